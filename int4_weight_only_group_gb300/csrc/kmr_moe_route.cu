// Expert router: the top k of each token's logits and their softmax weights.
//
//   p_i = exp(l_i - max l) / sum_j exp(l_j - max l);   ids = the k largest l, the lower index first among equals;
//   weight = p_i, or p_i / (sum of the chosen p).
// A logit of -inf or NaN takes no part; places that find no expert get id -1 and weight 0 (a row whose mask leaves
// nothing gets only those).  Logits of +inf share the weight equally.
//
// One warp per token: lane l holds the logits l, l + 32, ..., as keys whose unsigned order is the logits' order, so a
// round of the selection is one warp maximum over keys and one warp minimum over the indexes that hold it; the
// exponentials and their sum are fp32.  A token reads E logits and k rounds of two redux each follow: for one token
// the call is launch latency, for thousands the rounds (k * ~40 cycles a warp) hide behind each other.
#include "kmr_moe.cuh"

namespace kmr {

namespace {

constexpr int kRouteWarps = 4;

// Order of l as an unsigned key; 0 for what is never chosen.  -0 counts as 0.
__device__ __forceinline__ uint32_t order_key(float l) {
    if (!(l > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(l + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

template <int PER, bool BF16>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const MoeRouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    uint32_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        key[i] = 0u;
        if (e < p.E) {
            const size_t at = size_t(t) * p.E + e;
            key[i] = order_key(BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[at])
                                    : static_cast<const float*>(p.logits)[at]);
        }
    }
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = key[i] > best ? key[i] : best;
    const float most = key_value(__reduce_max_sync(0xffffffffu, best));       // (not used where no key is chosen)
    auto weight = [&](uint32_t k) {
        const float l = key_value(k);
        return k == 0u ? 0.f : (l == most ? 1.f : expf(l - most));
    };
    float total = 0.f;
    if (!p.renorm) {
#pragma unroll
        for (int i = 0; i < PER; ++i) total = __fadd_rn(total, weight(key[i]));
        total = warp_sum(total);
    }
    // lane j keeps the j-th choice
    int id = -1;
    float w = 0.f;
    for (int j = 0; j < p.k; ++j) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        if (top == 0u) break;
        uint32_t mine = 0xffffffffu;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (key[i] == top) mine = uint32_t(lane + 32 * i);
        const uint32_t e = __reduce_min_sync(0xffffffffu, mine);
        if (lane == j) {
            id = int(e);
            w = weight(top);
        }
        if (mine == e) {
            best = 0u;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (uint32_t(lane + 32 * i) == e) key[i] = 0u;
                best = key[i] > best ? key[i] : best;
            }
        }
    }
    if (p.renorm) total = warp_sum(w);
    if (lane < p.k) {
        const size_t at = size_t(t) * p.k + lane;
        p.ids[at] = id;
        p.weights[at] = id >= 0 ? __fdiv_rn(w, total) : 0.f;
    }
}

const void* route_fn(int E, bool bf16) {
#define KMR_ROUTE(n) \
    if (E <= 32 * n) return bf16 ? (const void*)moe_route_kernel<n, true> : (const void*)moe_route_kernel<n, false>
    KMR_ROUTE(1);
    KMR_ROUTE(2);
    KMR_ROUTE(4);
    KMR_ROUTE(8);
    KMR_ROUTE(16);
    KMR_ROUTE(32);
#undef KMR_ROUTE
    return nullptr;
}

}  // namespace

cudaError_t launch_moe_route(const MoeRouteParams& p, bool bf16, cudaStream_t st) {
    return launch_dependent(route_fn(p.E, bf16), dim3((p.T + kRouteWarps - 1) / kRouteWarps), kRouteWarps * 32, 0, 1, &p, st);
}

cudaError_t moe_route_set_attributes() {
    for (int E = 32; E <= kMoeMaxExperts; E *= 2)
        for (int b = 0; b < 2; ++b) {
            cudaFuncAttributes a;
            const cudaError_t e = cudaFuncGetAttributes(&a, route_fn(E, b != 0));
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

}  // namespace kmr
