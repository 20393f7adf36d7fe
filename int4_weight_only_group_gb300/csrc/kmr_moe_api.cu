// C ABI of the products whose weights each token chooses (declared in kmr.h): argument checks, then the launches of
// kmr_moe_route.cu, kmr_moe_small.cu and kmr_lora.cu.
#include "kmr_moe.cuh"

using namespace kmr;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int dtype) { return dtype == KMR_F32 || dtype == KMR_BF16; }

int view_of(const kmr_moe* m, MoeView* v) {
    if (!m || !m->gate_up || !m->down) return KMR_ERR_INVALID_ARG;
    if (!aligned(m->gate_up, 16) || !aligned(m->down, 16)) return KMR_ERR_INVALID_ARG;
    if (m->experts < 1 || m->experts > kMoeMaxExperts || m->group != 128) return KMR_ERR_SHAPE;
    for (const int n : {m->hidden, m->intermediate})
        if (n < 128 || n > kMoeMaxDim || n % 128) return KMR_ERR_SHAPE;
    v->gate_up = static_cast<const uint8_t*>(m->gate_up);
    v->down = static_cast<const uint8_t*>(m->down);
    v->E = m->experts;
    v->H = m->hidden;
    v->I = m->intermediate;
    return KMR_OK;
}

int counts_ok(int T, int top_k) {
    if (T < 1 || T > kMoeMaxTokens) return KMR_ERR_BATCH;
    return top_k < 1 || top_k > kMoeMaxTopK ? KMR_ERR_SHAPE : KMR_OK;
}

}  // namespace

extern "C" int kmr_moe_route(const void* logits, int dtype, int T, int experts, int top_k, int renormalise, int32_t* ids,
                             float* weights, void* stream) {
    if (!logits || !ids || !weights || !dtype_ok(dtype)) return KMR_ERR_INVALID_ARG;
    if (!aligned(logits, dtype == KMR_BF16 ? 2 : 4) || !aligned(ids, 4) || !aligned(weights, 4)) return KMR_ERR_INVALID_ARG;
    if (T < 1 || T > kMoeMaxTokens) return KMR_ERR_BATCH;
    if (experts < 1 || experts > kMoeMaxExperts || top_k < 1 || top_k > kMoeMaxTopK || top_k > experts) return KMR_ERR_SHAPE;
    if (ensure_kernel_attributes() != cudaSuccess) return KMR_ERR_CUDA;
    MoeRouteParams p = {};
    p.logits = logits;
    p.T = T;
    p.E = experts;
    p.k = top_k;
    p.renorm = renormalise != 0;
    p.ids = ids;
    p.weights = weights;
    return launch_moe_route(p, dtype == KMR_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}

extern "C" size_t kmr_moe_experts_workspace_size(const kmr_moe* moe, int dtype, int T, int top_k) {
    MoeView v;
    if (view_of(moe, &v) != KMR_OK || !dtype_ok(dtype) || counts_ok(T, top_k) != KMR_OK) return 0;
    return size_t(kMoeSmallPlaces) * v.I * 4;
}

extern "C" int kmr_moe_experts(const kmr_moe* moe, const void* x, int dtype, const int32_t* ids, const float* weights, int T,
                               int top_k, void* y, int epilogue, void* workspace, size_t workspace_bytes, void* stream) {
    MoeSmallParams p = {};
    int rc = view_of(moe, &p.w);
    if (rc != KMR_OK) return rc;
    if (!x || !ids || !weights || !y || !workspace || !dtype_ok(dtype)) return KMR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4))
        return KMR_ERR_INVALID_ARG;
    if (epilogue != KMR_EPI_NONE && epilogue != KMR_EPI_RESIDUAL) return KMR_ERR_INVALID_ARG;
    if ((rc = counts_ok(T, top_k)) != KMR_OK) return rc;
    if (workspace_bytes < kmr_moe_experts_workspace_size(moe, dtype, T, top_k)) return KMR_ERR_BUFFER_SIZE;
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    const bool bf16 = dtype == KMR_BF16;
    const size_t row = size_t(p.w.H) * (bf16 ? 2 : 4);
    p.k = top_k;
    p.act = static_cast<float*>(workspace);
    p.resid = epilogue == KMR_EPI_RESIDUAL;
    const int chunk = kMoeSmallPlaces / top_k;
    for (int t = 0; t < T; t += chunk) {
        p.x = static_cast<const uint8_t*>(x) + t * row;
        p.ids = ids + size_t(t) * top_k;
        p.weights = weights + size_t(t) * top_k;
        p.y = static_cast<uint8_t*>(y) + t * row;
        p.T = T - t < chunk ? T - t : chunk;
        if (launch_moe_small(p, bf16, num_sms(), static_cast<cudaStream_t>(stream)) != cudaSuccess) return KMR_ERR_CUDA;
    }
    return KMR_OK;
}

extern "C" int kmr_lora_apply(const kmr_lora* lora, const void* x, const void* base, void* y, int dtype,
                              const int32_t* adapter_ids, int T, long long ldx, long long ldy, void* stream) {
    if (!lora || !lora->a || !lora->b || !x || !y || !adapter_ids || !dtype_ok(dtype)) return KMR_ERR_INVALID_ARG;
    if (!aligned(lora->a, 16) || !aligned(lora->b, 16) || !aligned(lora->ranks, 4) || !aligned(lora->scales, 4) ||
        !aligned(x, 16) || !aligned(base, 16) || !aligned(y, 16) || !aligned(adapter_ids, 4))
        return KMR_ERR_INVALID_ARG;
    if (T < 1 || T > kMoeMaxTokens) return KMR_ERR_BATCH;
    if (lora->adapters < 1 || lora->inputs < 16 || lora->inputs % 16 || lora->outputs < 16 || lora->outputs % 16 ||
        lora->max_rank < 8 || lora->max_rank > kLoraMaxRank || lora->max_rank % 8)
        return KMR_ERR_SHAPE;
    if (ldx < lora->inputs || ldx % 8 || ldy < lora->outputs || ldy % 8) return KMR_ERR_SHAPE;
    LoraParams p = {};
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    p.a = lora->a;
    p.b = lora->b;
    p.ranks = lora->ranks;
    p.scales = lora->scales;
    p.L = lora->adapters;
    p.K = lora->inputs;
    p.N = lora->outputs;
    p.r = lora->max_rank;
    p.x = x;
    p.base = base;
    p.y = y;
    p.ldx = ldx;
    p.ldy = ldy;
    p.ids = adapter_ids;
    p.T = T;
    return launch_lora(p, dtype == KMR_BF16, num_sms(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}
