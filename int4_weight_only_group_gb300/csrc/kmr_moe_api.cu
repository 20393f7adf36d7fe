// C ABI of the products whose weights each token chooses (declared in kmr.h): argument checks, then the launches of
// kmr_moe_route.cu, kmr_moe_small.cu, kmr_moe_tc.cu and kmr_lora.cu.
#include "kmr_moe.cuh"

using namespace kmr;

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int dtype) { return dtype == KMR_F32 || dtype == KMR_BF16; }
bool dim_ok(int n) { return n >= 128 && n <= kMoeMaxDim && n % 128 == 0; }

int view_of(const kmr_moe* m, MoeView* v) {
    if (!m || !m->gate_up || !m->down || !m->factors) return KMR_ERR_INVALID_ARG;
    if (!aligned(m->gate_up, 16) || !aligned(m->down, 16) || !aligned(m->factors, 16)) return KMR_ERR_INVALID_ARG;
    if (m->experts < 1 || m->experts > kMoeMaxExperts || m->group != 128) return KMR_ERR_SHAPE;
    if (!dim_ok(m->hidden) || !dim_ok(m->intermediate)) return KMR_ERR_SHAPE;
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

// Tokens of one pass of the grouped form: bounds the workspace.
int chunk_of(int T, int top_k) {
    const int most = kMoeChunkPlaces / top_k;
    return T < most ? T : most;
}

struct Factors {
    float *gate_up, *down, *norms;
};
Factors factors_of(const kmr_moe* m) {
    float* f = m->factors;
    const size_t gate_up = size_t(m->experts) * 2 * m->intermediate;
    return {f, f + gate_up, f + gate_up + size_t(m->experts) * m->hidden};
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

extern "C" size_t kmr_moe_factors_size(int experts, int hidden, int intermediate) {
    if (experts < 1 || experts > kMoeMaxExperts || !dim_ok(hidden) || !dim_ok(intermediate)) return 0;
    return size_t(experts) * (2 * size_t(intermediate) + hidden + 3) * 4;      // (the last two words an expert are spare)
}

extern "C" int kmr_moe_prepare(const kmr_moe* moe, void* stream) {
    MoeView v;
    const int rc = view_of(moe, &v);
    if (rc != KMR_OK) return rc;
    if (ensure_kernel_attributes() != cudaSuccess) return KMR_ERR_CUDA;
    const Factors f = factors_of(moe);
    return launch_moe_factors(v, f.gate_up, f.down, f.norms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}

extern "C" size_t kmr_moe_experts_workspace_size(const kmr_moe* moe, int dtype, int T, int top_k) {
    MoeView v;
    if (view_of(moe, &v) != KMR_OK || !dtype_ok(dtype) || counts_ok(T, top_k) != KMR_OK) return 0;
    if (moe_small_fits(v, dtype == KMR_BF16, T, top_k)) return size_t(T) * top_k * v.I * 4;
    const size_t most = size_t(kMoeSmallPlaces) * v.I * 4, all = moe_tc_sizes(v, dtype == KMR_BF16, chunk_of(T, top_k), top_k).total;
    return all > most ? all : most;                      // (never less than for fewer tokens)
}

extern "C" int kmr_moe_experts(const kmr_moe* moe, const void* x, int dtype, const int32_t* ids, const float* weights, int T,
                               int top_k, void* y, int epilogue, void* workspace, size_t workspace_bytes, void* stream) {
    MoeView v;
    int rc = view_of(moe, &v);
    if (rc != KMR_OK) return rc;
    if (!x || !ids || !weights || !y || !workspace || !dtype_ok(dtype)) return KMR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4))
        return KMR_ERR_INVALID_ARG;
    if (epilogue != KMR_EPI_NONE && epilogue != KMR_EPI_RESIDUAL) return KMR_ERR_INVALID_ARG;
    if ((rc = counts_ok(T, top_k)) != KMR_OK) return rc;
    if (workspace_bytes < kmr_moe_experts_workspace_size(moe, dtype, T, top_k)) return KMR_ERR_BUFFER_SIZE;
    int* err = nullptr;
    if (ensure_kernel_attributes() != cudaSuccess || !(err = standalone_error_word())) return KMR_ERR_CUDA;
    const bool bf16 = dtype == KMR_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (moe_small_fits(v, bf16, T, top_k)) {
        MoeSmallParams p = {};
        p.w = v;
        p.x = x;
        p.ids = ids;
        p.weights = weights;
        p.T = T;
        p.k = top_k;
        p.act = static_cast<float*>(workspace);
        p.y = y;
        p.resid = epilogue == KMR_EPI_RESIDUAL;
        p.err = err;
        return launch_moe_small(p, bf16, num_sms(), st) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
    }
    const size_t row = size_t(v.H) * (bf16 ? 2 : 4);
    const int chunk = chunk_of(T, top_k);
    const MoeTcSizes z = moe_tc_sizes(v, bf16, chunk, top_k);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const Factors f = factors_of(moe);
    MoeTcParams p = {};
    p.w = v;
    p.rho_gate_up = f.gate_up;
    p.rho_down = f.down;
    p.norms = f.norms;
    p.k = top_k;
    p.ntiles = reinterpret_cast<int*>(ws);
    p.tiles = reinterpret_cast<int4*>(ws + z.tiles);
    p.pos = reinterpret_cast<int32_t*>(ws + z.pos);
    p.isx = reinterpret_cast<float*>(ws + z.isx);
    p.isa = reinterpret_cast<float*>(ws + z.isa);
    p.sout = reinterpret_cast<float*>(ws + z.sout);
    p.blocks = z.blocks;
    p.xs = ws + z.xs;
    p.as = ws + z.as;
    p.out = ws + z.out;
    p.resid = epilogue == KMR_EPI_RESIDUAL;
    p.err = err;
    for (int t = 0; t < T; t += chunk) {
        p.x = static_cast<const uint8_t*>(x) + t * row;
        p.ids = ids + size_t(t) * top_k;
        p.weights = weights + size_t(t) * top_k;
        p.y = static_cast<uint8_t*>(y) + t * row;
        p.T = T - t < chunk ? T - t : chunk;
        p.cap = moe_tc_cap((long long)p.T * top_k, v.E, bf16);
        if (launch_moe_tc(p, bf16, num_sms(), st) != cudaSuccess) return KMR_ERR_CUDA;
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
    if (lora->adapters < 1 || lora->inputs < 16 || lora->inputs % 16 || lora->inputs > kLoraMaxDim || lora->outputs < 16 ||
        lora->outputs % 16 || lora->outputs > kLoraMaxDim ||
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
