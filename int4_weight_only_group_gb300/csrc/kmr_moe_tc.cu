// Int4 experts for many tokens: the places (token, j) are grouped by expert and both products run as ragged grouped
// GEMMs on the 5th-generation tensor cores.
//
//   plan     counts the places of every expert and gives each a position; an expert's positions are padded to a multiple
//            of 16 and cut into tiles of at most `cap` (16..128) tokens
//   stage    token rows as fp16 into the tiles' operand layout (a copy per place)
//   gate_up  D = A B^T per (tile, 128 packed weight rows), silu(gate) * up, staged again for
//   down     the same product, fp32 rows of every place
//   combine  y[t] = sum_j weights[t, j] * row of place (t, j), in the order of the places: no atomics on values
//
// The product, D[row][token] = sum_k w[row][k] x[token][k], w = (q - 8) s + z:
//   * A = (q - 8) s rho: a 4-bit integer times a bf16 scale has 11 significant bits, so fp16 holds it exactly once a power of two
//     rho per row (laid out once, moe_factors_kernel) has brought the row's scales into fp16's range.
//   * the zero points' share sum_g z_g X_g, X_g = sum of the group's inputs, goes through the same accumulator as a few more
//     inputs: z rho 2^6 against X 2^-6 for every 64 inputs, X in two fp16 terms.
//   * B = x sigma (a power of two per row): exact for bf16 inputs, two terms (the fp16 rounding and what it left, two
//     MMAs on the same A) for fp32 ones.  So products are exact and sums are fp32 in both types.
//   * the activation's scale must be known before its row is complete: |silu(g) u| <= |g| |u| <= (|x| max |gate row|)
//     (|x| max |up row|) bounds it from the row's norm and per-expert constants.  The bound is loose by 2^7 to 2^13, which
//     fp16's range absorbs: the values stay far above its subnormals.
//
// Each CTA is persistent and warp-specialised: a weight producer and a token producer (cp.async.bulk rings), eight warps that turn
// KMR4 blocks into A in tensor memory (kmr_tcgemm.cu describes that layout), one thread that issues the MMAs, four epilogue
// warps on the other of two accumulators (for fp32 it also adds up chunks of a long sum, see kChunk).  Every wait is bounded; a timeout records KMR_ERR_DEVICE_TIMEOUT, skips the
// remaining work, drains the copies in flight and frees tensor memory.
#include <cuda_fp16.h>

#include "kmr_int4_mma.cuh"
#include "kmr_moe.cuh"
#include "kmr_tc.cuh"

namespace kmr {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = 128;                        // packed weight rows of a product (the MMA's M)
constexpr uint32_t kWBytes = 8 * kGroupBytes;     // a group of eight KMR4 tiles
constexpr uint32_t kBRing = 128 * 1024;
constexpr int kAQ = 4;                            // dequantised groups in tensor memory, 64 columns each
constexpr int kMaxStages = 16;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(max(1, min(253, e + 127))) << 23); }
// e such that |v| < 2^e, for v >= 0 (128 or more for what is not finite)
__device__ __forceinline__ int above(float v) { return int(__float_as_uint(v) >> 23) - 126; }
__device__ __forceinline__ float inverse_pow2(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// ------------------------------------------------------------------ weights, once
// Row factors rho (a power of two that brings max(8 |s|, 64 |z|) of the row to [2^13, 2^14)) and the largest row norm bound of
// each expert's gate and up rows: |w|^2 <= sum over groups of 128 max(|z - 8 s|, |z + 7 s|)^2.
__global__ void moe_factors_kernel(const uint8_t* w, int tiles, int G, float* rho, float* norms) {
    const int row = blockIdx.x * blockDim.x + threadIdx.x, e = blockIdx.y;
    if (row >= tiles * 16) return;
    const uint8_t* at = w + (size_t(e) * tiles + row / 16) * G * kGroupBytes + 1024 + (row & 15) * 4;
    float m = 0.f, n2 = 0.f;
    for (int g = 0; g < G; ++g) {
        const uint32_t sz = *reinterpret_cast<const uint32_t*>(at + size_t(g) * kGroupBytes);
        const float s = bf16_lo(sz), z = bf16_hi(sz);
        m = fmaxf(m, fmaxf(8.f * fabsf(s), 64.f * fabsf(z)));
        const float far = fmaxf(fabsf(__fmaf_rn(-8.f, s, z)), fabsf(__fmaf_rn(7.f, s, z)));
        n2 = __fmaf_rn(128.f * far, far, n2);
    }
    float r, ir;
    pow2_scale(__float_as_uint(m), r, ir);
    rho[size_t(e) * tiles * 16 + row] = r;
    // (a bound: rounded up; the bits of non-negative floats order like integers)
    if (norms) atomicMax(reinterpret_cast<int*>(norms + 2 * e + ((row & 15) >> 3)), __float_as_int(sqrtf(n2) * 1.001f));
}

// ------------------------------------------------------------------ plan
constexpr int kPlanThr = 1024;
__global__ void __launch_bounds__(kPlanThr) moe_plan_kernel(const MoeTcParams p) {
    __shared__ int count[kMoeMaxExperts], at[kMoeMaxExperts], wsum[2][32];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, S = p.T * p.k;
    count[tid] = 0;
    __syncthreads();
    for (int i = tid; i < S; i += kPlanThr) {
        const int e = p.ids[i];
        if (e >= 0 && e < p.w.E) atomicAdd(&count[e], 1);
        else if (e != -1) set_error(p.err, KMR_ERR_INVALID_ARG);
    }
    __syncthreads();
    // thread e: its expert's padded positions and tiles, and those before it
    const int n = count[tid], n16 = (n + 15) & ~15;
    const int nt = (n16 + p.cap - 1) / p.cap;
    int a = n16, b = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kFull, a, o), v = __shfl_up_sync(kFull, b, o);
        if (lane >= o) {
            a += u;
            b += v;
        }
    }
    if (lane == 31) {
        wsum[0][warp] = a;
        wsum[1][warp] = b;
    }
    __syncthreads();
    int pa = 0, pb = 0;
    for (int w = 0; w < warp; ++w) {
        pa += wsum[0][w];
        pb += wsum[1][w];
    }
    const int p0 = pa + a - n16, t0 = pb + b - nt;
    at[tid] = p0;
    if (nt > 0) {
        const int each = ((n16 + nt - 1) / nt + 15) & ~15;           // even tiles, whole sixteens
        for (int i = 0; i < nt; ++i) {
            const int len = min(each, n16 - i * each);
            p.tiles[t0 + i] = make_int4(tid, p0 + i * each, max(len, 0), 0);
        }
    }
    if (tid == kPlanThr - 1) *p.ntiles = pb + b;
    __syncthreads();
    // (which of its expert's positions a place gets does not change any result)
    for (int i = tid; i < S; i += kPlanThr) {
        const int e = p.ids[i];
        p.pos[i] = e >= 0 && e < p.w.E ? atomicAdd(&at[e], 1) : -1;
    }
}

// ------------------------------------------------------------------ operand layout
// Staged rows: blocks of 8 rows; within one, per group of 128 inputs NP (terms) x 2 atoms of [8 rows][64 inputs] fp16 with the
// 16-byte pieces of a row swizzled by the row (the MMA's 128-byte swizzle), then the sums' atoms, first terms and remainders.
// Input k of 16 sits at 2 (k % 8) - k % 2 + 2 (k / 8) (the order of A's columns in tensor memory).
__host__ __device__ constexpr int sum_atoms(int K) { return (K / 64 + 63) / 64; }
__host__ __device__ constexpr size_t block_bytes(int K, int np) {
    return size_t(K / 128) * np * 2048 + size_t(2) * sum_atoms(K) * 1024;
}
__device__ __forceinline__ uint32_t piece(int row, int c) { return uint32_t(row * 128 + ((c ^ row) << 4)); }
// Sum number h (of 64 inputs) of a row: its two terms.  `sums` is the block's first sum atom.
__device__ __forceinline__ void put_sum(uint8_t* sums, int K, int row, int h, float X) {
    const float x = X * 0.015625f;
    const __half hi = __float2half_rn(x);
    const __half lo = __float2half_rn(__fsub_rn(x, __half2float(hi)));
    uint8_t* at = sums + (h >> 6) * 1024 + piece(row, (h & 63) >> 3) + (h & 7) * 2;
    *reinterpret_cast<__half*>(at) = hi;
    *reinterpret_cast<__half*>(at + sum_atoms(K) * 1024) = lo;
}
// The places of sums past the last that an MMA step covers.
__device__ __forceinline__ void clear_sums(uint8_t* sums, int K, int row, int i) {
    const int h = K / 64 + i;
    if (h < ((K / 64 + 15) & ~15)) put_sum(sums, K, row, h, 0.f);
}

// ------------------------------------------------------------------ stage
constexpr int kStageThr = 256;
template <typename IN, int NP>
__global__ void __launch_bounds__(kStageThr) moe_stage_kernel(const MoeTcParams p) {
    __shared__ float red[2][kStageThr / 32];
    __shared__ int pos[kMoeMaxTopK];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.w.H, K4 = K >> 2;
    int n = 0;
    if (tid < 32) {
        const int at = tid < p.k ? p.pos[size_t(t) * p.k + tid] : -1;
        const uint32_t some = __ballot_sync(kFull, at >= 0);
        if (at >= 0) pos[__popc(some & ((1u << lane) - 1u))] = at;
        if (lane == 0) red[0][0] = __int_as_float(__popc(some));
    }
    __syncthreads();
    n = __float_as_int(red[0][0]);
    if (n == 0) return;
    __syncthreads();
    constexpr int kPer = kMoeMaxDim / 4 / kStageThr;
    float4 v[kPer];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k4 = tid + i * kStageThr;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k4 >= K4) continue;
        if constexpr (sizeof(IN) == 4) {
            v[i] = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + size_t(t) * K)[k4];
        } else {
            const uint2 r = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.x) + size_t(t) * K)[k4];
            v[i] = make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        }
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
    }
    m = warp_max(m);
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = red[0][0];
#pragma unroll
    for (int w = 1; w < kStageThr / 32; ++w) m = fmaxf(m, red[0][w]);
    float sig, isg;
    pow2_scale(__float_as_uint(m), sig, isg);
    float ss = 0.f;
    const size_t bb = block_bytes(K, NP);
    auto h2u = [](__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int k4 = tid + i * kStageThr;
        if (k4 >= K4) break;                                        // (whole warps: K4 is a multiple of 32)
        const int k = k4 * 4, m4 = k4 & 3;
        const float a[4] = {__fmul_rn(v[i].x, sig), __fmul_rn(v[i].y, sig), __fmul_rn(v[i].z, sig), __fmul_rn(v[i].w, sig)};
        float X = 0.f;
        uint2 out[NP];
        float r[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const __half2 h0 = __floats2half2_rn(r[0], r[1]), h1 = __floats2half2_rn(r[2], r[3]);
            const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
            X = __fadd_rn(X, __fadd_rn(__fadd_rn(f0.x, f0.y), __fadd_rn(f1.x, f1.y)));
            r[0] = __fsub_rn(r[0], f0.x);
            r[1] = __fsub_rn(r[1], f0.y);
            r[2] = __fsub_rn(r[2], f1.x);
            r[3] = __fsub_rn(r[3], f1.y);
            // a 16-byte piece holds inputs 0, 1, 8, 9, 2, 3, 10, 11 (or 4 more) of its 16: two lanes write its halves
            const uint32_t wa = h2u(h0), wb = h2u(h1);
            const uint32_t got = __shfl_xor_sync(kFull, m4 < 2 ? wb : wa, 2);
            out[q] = m4 < 2 ? make_uint2(wa, got) : make_uint2(got, wb);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) ss = __fmaf_rn(a[q], a[q], ss);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) X = __fadd_rn(X, __shfl_xor_sync(kFull, X, o));
        for (int j = 0; j < n; ++j) {
            const int at = pos[j], row = at & 7;
            uint8_t* blk = p.xs + size_t(at >> 3) * bb;
            uint8_t* to = blk + size_t(k >> 7) * NP * 2048 + ((k >> 6) & 1) * 1024 +
                          piece(row, ((k & 63) >> 4) * 2 + (m4 & 1)) + (m4 < 2 ? 0 : 8);
#pragma unroll
            for (int q = 0; q < NP; ++q) *reinterpret_cast<uint2*>(to + q * 2048) = out[q];
            if ((lane & 15) == 0) put_sum(blk + size_t(K >> 7) * NP * 2048, K, row, k >> 6, X);
        }
    }
    ss = warp_sum(ss);
    if (lane == 0) red[1][warp] = ss;
    __syncthreads();
    for (int i = tid; i < n * 16; i += kStageThr) {
        const int at = pos[i >> 4];
        clear_sums(p.xs + size_t(at >> 3) * bb + size_t(K >> 7) * NP * 2048, K, at & 7, i & 15);
    }
    if (tid < p.k) {
        const int at = p.pos[size_t(t) * p.k + tid];
        if (at < 0) return;
        ss = red[1][0];
        for (int w = 1; w < kStageThr / 32; ++w) ss = __fadd_rn(ss, red[1][w]);
        // |x|, and the bound of the place's activations: below 2^15 once scaled
        const int e = p.ids[size_t(t) * p.k + tid];
        const int ex = above(sqrtf(ss)) + above(isg) - 1;
        p.isx[at] = isg;
        p.sact[at] = pow2(15 - (2 * ex + above(p.norms[2 * e]) + above(p.norms[2 * e + 1])));
    }
}

// ------------------------------------------------------------------ the grouped product
constexpr int kUnpackWarps = 8, kTokenWarp = 10, kEpiWarp = 11, kEpiWarps = 4;
constexpr int kThr = (kEpiWarp + kEpiWarps) * 32;

struct Layout {
    uint32_t tile, w, z, bar, fac, psum, total;
};
__host__ __device__ constexpr int w_stages(int np, bool gate) { return gate && np == 2 ? 5 : 7; }
__host__ __device__ constexpr uint32_t z_pitch(int K) { return uint32_t((K / 128 + 7) & ~7) * 2; }   // bytes of a row's zeros
__host__ __device__ constexpr Layout layout(int np, bool gate, int K) {
    Layout l = {};
    l.tile = kBRing;
    l.w = l.tile + (gate ? 16384u * np : 0u);
    l.z = l.w + w_stages(np, gate) * kWBytes;
    l.bar = l.z + kRows * z_pitch(K);
    l.fac = l.bar + 512;
    l.psum = l.fac + 2 * 2 * 128 * 4;
    l.total = l.psum + (gate ? 4 * 128 * 4 : 0);
    return l;
}
static_assert(layout(1, true, kMoeMaxDim).total <= 227 * 1024 && layout(2, true, kMoeMaxDim).total <= 227 * 1024 &&
              layout(1, false, kMoeMaxDim).total <= 227 * 1024, "shared memory");

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, `stride` bytes between blocks of 8 rows.
__device__ __forceinline__ uint64_t swizzled_desc(uint32_t addr, uint32_t stride) {
    return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t((stride >> 4) & 0x3FFFu) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }
__device__ __forceinline__ float silu_mul(float x, float up) {
    return __fmul_rn(__fdiv_rn(x, __fadd_rn(1.f, expf(-x))), up);
}
__device__ __forceinline__ void tmem_store(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}

// The tensor cores cut a running sum off rather than round it, so a chain of n steps of 16 inputs comes out some n 2^-25 too
// small (measured: 1040 steps, 2.3e-5).  bf16 results do not show it.  For fp32 (two MMAs a step) the epilogue warps add
// up chunks of kChunk groups (64 steps: 1.4e-6) in registers, which limits a tile to 64 tokens.
constexpr int kChunk = 4;
template <int NP>
constexpr int kTileTokens = NP == 2 ? 64 : 128;
__device__ __forceinline__ bool chunk_end(int np, int g) { return np == 2 && g % kChunk == kChunk - 1; }

// A stage of a ring and the parity of its current round.
struct Turn {
    int s = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            ++round;
        }
    }
    __device__ __forceinline__ bool waits() const { return round > 0; }
    __device__ __forceinline__ uint32_t full() const { return round & 1u; }
    __device__ __forceinline__ uint32_t empty() const { return (round - 1u) & 1u; }
};

template <int NP, bool GATE>
__global__ void __launch_bounds__(kThr, 1) moe_product_kernel(const MoeTcParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const int K = GATE ? p.w.H : p.w.I, N = GATE ? 2 * p.w.I : p.w.H, G = K >> 7;
    const int R = N / kRows;                               // row tiles of an expert
    const Layout L = layout(NP, GATE, K);
    constexpr int WS = w_stages(NP, GATE);
    const uint32_t bstage = uint32_t(p.cap) * 256u * NP;
    const int BS = min(kMaxStages, int(kBRing / bstage));
    const int ZA = sum_atoms(K), ZK = (K / 64 + 15) / 16;  // atoms and MMA steps of the sums
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* w_full = reinterpret_cast<uint64_t*>(smem + L.bar);
    uint64_t* w_empty = w_full + WS;
    uint64_t* b_full = w_empty + WS;
    uint64_t* b_empty = b_full + kMaxStages;
    uint64_t* a_full = b_empty + kMaxStages;
    uint64_t* a_empty = a_full + kAQ;
    uint64_t* d_full = a_empty + kAQ;
    uint64_t* d_empty = d_full + 2;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(d_empty + 2);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    static_assert((2 * 7 + 2 * kMaxStages + 2 * kAQ + 4) * 8 + 8 <= 512, "barrier area");
    const uint32_t sbase = smem_u32(smem);

    if (tid == 0) {
        *abort_flag = 0;
        for (int s = 0; s < WS; ++s) {
            mbar_init(&w_full[s], 1);
            mbar_init(&w_empty[s], kUnpackWarps);
        }
        for (int s = 0; s < BS; ++s) {
            mbar_init(&b_full[s], 1);
            mbar_init(&b_empty[s], 1);
        }
        for (int s = 0; s < kAQ; ++s) {
            mbar_init(&a_full[s], kUnpackWarps);
            mbar_init(&a_empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&d_full[s], 1);
            mbar_init(&d_empty[s], kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 0) tc_alloc(tslot, 512);
    for (int i = tid; i < kRows * int(z_pitch(K)) / 4; i += kThr) reinterpret_cast<uint32_t*>(smem + L.z)[i] = 0u;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = *tslot;
    pdl_wait();
    pdl_launch_dependents();
    auto fail = [&]() { *abort_flag = 1; };
    // lane 0 waits, the warp follows its verdict
    auto warp_wait = [&](uint64_t* b, uint32_t parity) {
        int ok = 0;
        if (lane == 0) {
            ok = !*abort_flag && spin_wait(b, parity, p.err);
            if (!ok) fail();
        }
        return __shfl_sync(kFull, ok, 0) != 0;
    };
    const int items = *p.ntiles * R;
    const uint8_t* wsrc = GATE ? p.w.gate_up : p.w.down;
    const uint8_t* bsrc = GATE ? p.xs : p.as;
    const size_t bb = block_bytes(K, NP);
    Turn tw, tb;                                           // the producers' own rings (also for draining)
    bool ok = true;

    if (warp == 0) {
        // ---- weights: lanes 0..7 copy a group's eight blocks
        const uint64_t pol = policy_evict_first();
        for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
            const int4 tile = p.tiles[it / R];
            const uint8_t* src = wsrc + (size_t(tile.x) * (N / 16) + (it % R) * 8 + (lane & 7)) * G * kGroupBytes;
            for (int g = 0; g < G; ++g) {
                if (tw.waits() && !(ok = warp_wait(&w_empty[tw.s], tw.empty()))) break;
                if (lane == 0) mbar_arrive_expect_tx(&w_full[tw.s], kWBytes);
                __syncwarp();
                fence_proxy_async_smem();                  // the unpack warps' reads of the stage come first
                if (lane < 8)
                    bulk_g2s_stream(smem + L.w + tw.s * kWBytes + lane * kGroupBytes, src + size_t(g) * kGroupBytes, kGroupBytes,
                                    &w_full[tw.s], pol);
                tw.next(WS);
            }
        }
    } else if (warp == kTokenWarp) {
        // ---- staged tokens: one lane per block of 8 rows
        for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
            const int4 tile = p.tiles[it / R];
            const int nb = tile.z >> 3;
            const uint8_t* src = bsrc + size_t((tile.y >> 3) + lane) * bb;
            auto copy = [&](size_t from, uint32_t bytes) {
                if (tb.waits() && !warp_wait(&b_empty[tb.s], tb.empty())) return false;
                if (lane == 0) mbar_arrive_expect_tx(&b_full[tb.s], bytes * nb);
                __syncwarp();
                if (lane < nb) bulk_g2s(smem + size_t(tb.s) * bstage + lane * bytes, src + from, bytes, &b_full[tb.s]);
                tb.next(BS);
                return true;
            };
            for (int g = 0; g < G && ok; ++g) ok = copy(size_t(g) * NP * 2048, NP * 2048);
            for (int h = 0; h < 2 / NP && ok; ++h) ok = copy(size_t(G) * NP * 2048 + h * ZA * 1024, NP * ZA * 1024);
        }
    } else if (warp == 1) {
        // ---- MMA issue
        if (lane == 0) {
            Turn ta, tt, td;
            for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
                const uint32_t idesc = tc_idesc(kRows, p.tiles[it / R].z);
                bool begun = false;                        // the accumulator holds something of this chunk
                for (int g = 0; g <= G && ok; ++g) {
                    if (!begun && td.waits()) ok = spin_wait(&d_empty[td.s], td.empty(), p.err);
                    ok = ok && !*abort_flag && spin_wait(&a_full[ta.s], ta.full(), p.err);
                    const uint32_t acc = taddr + td.s * 128;
                    const int steps = g < G ? 8 : ZK;
                    const uint32_t a = taddr + 256 + ta.s * 64;
                    // the sums' first terms and remainders fill one stage (NP = 2) or two
                    for (int part = 0; part < (g < G ? 1 : 2 / NP) && ok; ++part) {
                        ok = spin_wait(&b_full[tt.s], tt.full(), p.err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t b = sbase + tt.s * bstage;
                        const uint32_t term = g < G ? 2048u : uint32_t(ZA) * 1024u;
#pragma unroll
                        for (int q = 0; q < NP; ++q)
                            for (int ks = 0; ks < steps; ++ks)
                                tc_mma_ta(acc, a + ks * 8, swizzled_desc(b + q * term + (ks >> 2) * 1024 + (ks & 3) * 32, NP * term),
                                          idesc, (begun || ks > 0 || q > 0) ? 1u : 0u);
                        begun = true;
                        tc_commit(&b_empty[tt.s]);
                        tt.next(BS);
                    }
                    tc_commit(&a_empty[ta.s]);
                    ta.next(kAQ);
                    if (g == G || (chunk_end(NP, g) && g + 1 < G)) {
                        tc_commit(&d_full[td.s]);
                        td.next(2);
                        begun = false;
                    }
                }
                if (!ok) fail();
            }
        }
    } else if (warp < kTokenWarp) {
        // ---- unpack: the two tiles of tensor-memory lane quarter warp % 4, half of a group's k-steps
        const int lq = warp & 3, kj = (warp - 2) >> 2, g8 = lane >> 2, t = lane & 3;
        const float* rho = GATE ? p.rho_gate_up : p.rho_down;
        uint8_t* zb = smem + L.z + (32 * lq + g8) * z_pitch(K);
        const __half2 m8 = __float2half2_rn(-1032.f), c16 = __float2half2_rn(0.0625f), m72 = __float2half2_rn(-72.f);
        auto h2 = [](uint32_t v) { return *reinterpret_cast<const __half2*>(&v); };
        auto u2 = [](__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); };
        Turn ta, tt;
        for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
            const int4 tile = p.tiles[it / R];
            float rr[4];                                   // of rows g8, g8 + 8, g8 + 16, g8 + 24 of the quarter
#pragma unroll
            for (int i = 0; i < 4; ++i) rr[i] = rho[size_t(tile.x) * N + (it % R) * kRows + 32 * lq + g8 + 8 * i];
            for (int g = 0; g < G; ++g) {
                if (!(ok = warp_wait(&w_full[tt.s], tt.full()))) break;
                if (ta.waits() && !(ok = warp_wait(&a_empty[ta.s], ta.empty()))) break;
                tc_fence_after();
                const uint8_t* wst = smem + L.w + tt.s * kWBytes + (2 * lq) * kGroupBytes;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* blk = wst + h * kGroupBytes;
                    const uint32_t sz0 = *reinterpret_cast<const uint32_t*>(blk + 1024 + g8 * 4);
                    const uint32_t sz1 = *reinterpret_cast<const uint32_t*>(blk + 1024 + (g8 + 8) * 4);
                    const __half2 s0 = __float2half2_rn(__fmul_rn(bf16_lo(sz0), rr[2 * h]));
                    const __half2 s1 = __float2half2_rn(__fmul_rn(bf16_lo(sz1), rr[2 * h + 1]));
                    if (kj == 0 && t == (g & 3)) {
                        *reinterpret_cast<uint16_t*>(zb + (16 * h) * z_pitch(K) + g * 2) = uint16_t(sz0 >> 16);
                        *reinterpret_cast<uint16_t*>(zb + (16 * h + 8) * z_pitch(K) + g * 2) = uint16_t(sz1 >> 16);
                    }
                    const uint32_t acol = taddr + 256 + ta.s * 64 + (uint32_t(32 * lq + 16 * h) << 16);
                    const uint4 wq = *reinterpret_cast<const uint4*>(blk + kj * 512 + lane * 16);
                    const uint32_t w4[4] = {wq.x, wq.y, wq.z, wq.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t w = w4[k], wh = w >> 8;
                        const __half2 qa = __hadd2(h2(and_or(w, 0x000F000Fu, 0x64006400u)), m8);
                        const __half2 qb = __hfma2(h2(and_or(w, 0x00F000F0u, 0x64006400u)), c16, m72);
                        const __half2 qc = __hadd2(h2(and_or(wh, 0x000F000Fu, 0x64006400u)), m8);
                        const __half2 qd = __hfma2(h2(and_or(wh, 0x00F000F0u, 0x64006400u)), c16, m72);
                        tmem_store(acol + (4 * kj + k) * 8, u2(__hmul2(qa, s0)), u2(__hmul2(qc, s0)), u2(__hmul2(qb, s1)),
                                   u2(__hmul2(qd, s1)));
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&a_full[ta.s]);
                    mbar_arrive(&w_empty[tt.s]);
                }
                tt.next(WS);
                ta.next(kAQ);
            }
            if (!ok) break;
            // the zero points: word column c of a step is group 8 step + c, twice
            if (ta.waits() && !(ok = warp_wait(&a_empty[ta.s], ta.empty()))) break;
            tc_fence_after();
            if (kj == 0) {
                __syncwarp();
                auto dup = [&](uint32_t bits, float r) { return u2(__float2half2_rn(__fmul_rn(__uint_as_float(bits << 16), 64.f * r))); };
                for (int ks = 0; ks < ZK; ++ks) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t z0 = *reinterpret_cast<const uint32_t*>(zb + (16 * h) * z_pitch(K) + (8 * ks + 2 * t) * 2);
                        const uint32_t z1 = *reinterpret_cast<const uint32_t*>(zb + (16 * h + 8) * z_pitch(K) + (8 * ks + 2 * t) * 2);
                        tmem_store(taddr + 256 + ta.s * 64 + (uint32_t(32 * lq + 16 * h) << 16) + ks * 8, dup(z0 & 0xFFFFu, rr[2 * h]),
                                   dup(z0 >> 16, rr[2 * h]), dup(z1 & 0xFFFFu, rr[2 * h + 1]), dup(z1 >> 16, rr[2 * h + 1]));
                    }
                }
                tc_wait_st();
                __syncwarp();                              // (the zeros are read before the next tile's come)
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&a_full[ta.s]);
            ta.next(kAQ);
        }
    } else if (warp >= kEpiWarp) {
        // ---- epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31 (its weight rows), all tokens
        const int q = warp & 3, et = tid - kEpiWarp * 32;
        float* fac = reinterpret_cast<float*>(smem + L.fac);       // [2][2][128]
        float* psum = reinterpret_cast<float*>(smem + L.psum);     // [4][128]
        uint8_t* tbuf = smem + L.tile;
        const float* rho = GATE ? p.rho_gate_up : p.rho_down;
        Turn td;
        int turn = 0;
        for (int it = blockIdx.x; it < items; it += gridDim.x, turn ^= 1) {
            const int4 tile = p.tiles[it / R];
            const int r = it % R, n = tile.z;
            float* f = fac + turn * 256;
            if (et < n) {
                f[et] = GATE ? p.isx[tile.y + et] : inverse_pow2(p.sact[tile.y + et]);
                if (GATE) f[128 + et] = p.sact[tile.y + et];
            }
            const float irho = inverse_pow2(rho[size_t(tile.x) * N + r * kRows + 32 * q + lane]);
            if (GATE && warp == kEpiWarp) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            epilogue_bar();                                // factors in place, the previous tile's copies have read the buffer
            // tokens c0 .. c0 + 15 of this lane's row
            auto finish = [&](int c0, const float (&v)[16]) {
                if (GATE) {
                    // in pairs: the gate lanes (tile rows 0..7) finish token c, the up lanes token c + 1
                    const bool lo = (lane & 15) < 8;
                    const int i16 = (lane >> 4) * 8 + (lane & 7);              // column of the warp's 16
                    const int at = 2 * (i16 & 7) - (i16 & 1) + ((i16 >> 3) << 1);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float xa = __fmul_rn(v[j], __fmul_rn(irho, f[c0 + j]));
                        const float xb = __fmul_rn(v[j + 1], __fmul_rn(irho, f[c0 + j + 1]));
                        const float other = __shfl_xor_sync(kFull, lo ? xb : xa, 8);
                        const int c = c0 + j + (lo ? 0 : 1);
                        float a = silu_mul(lo ? xa : other, lo ? other : xb);
                        a = __fmul_rn(a, f[128 + c]);
                        uint8_t* to = tbuf + size_t(c >> 3) * NP * 1024 + piece(c & 7, 2 * q + (at >> 3)) + (at & 7) * 2;
                        float X = 0.f;
#pragma unroll
                        for (int s = 0; s < NP; ++s) {
                            const __half hv = __float2half_rn(a);
                            const float hf = __half2float(hv);
                            *reinterpret_cast<__half*>(to + s * 1024) = hv;
                            X = __fadd_rn(X, hf);
                            a = __fsub_rn(a, hf);
                        }
                        X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 1));
                        X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 2));
                        X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 4));
                        X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 16));
                        if ((lane & 23) == 0) psum[q * 128 + c] = X;           // lanes 0 and 8
                    }
                } else {
                    float* out = p.out + size_t(tile.y + c0) * N + r * kRows + 32 * q + lane;
#pragma unroll
                    for (int j = 0; j < 16; ++j) out[size_t(j) * N] = __fmul_rn(v[j], __fmul_rn(irho, f[c0 + j]));
                }
            };
            // (after a timeout nothing is stored any more, but the barriers are kept)
            if constexpr (NP == 1) {
                ok = ok && warp_wait(&d_full[td.s], td.full());
                tc_fence_after();
                const uint32_t acc = taddr + td.s * 128 + (uint32_t(32 * q) << 16);
                for (int c0 = 0; c0 < n && ok; c0 += 16) {
                    float v[16];
                    tc_ld16(acc + uint32_t(c0), v);
                    finish(c0, v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[td.s]);
                td.next(2);
            } else {
                float sum[kTileTokens<NP> / 16][16];
#pragma unroll
                for (int i = 0; i < kTileTokens<NP> / 16; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[i][j] = 0.f;
                for (int g = 0; g < G; g += kChunk) {
                    ok = ok && warp_wait(&d_full[td.s], td.full());
                    tc_fence_after();
                    const uint32_t acc = taddr + td.s * 128 + (uint32_t(32 * q) << 16);
#pragma unroll
                    for (int i = 0; i < kTileTokens<NP> / 16; ++i) {
                        if (i * 16 >= n || !ok) continue;
                        float v[16];
                        tc_ld16(acc + uint32_t(i * 16), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] = __fadd_rn(sum[i][j], v[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[td.s]);
                    td.next(2);
                }
#pragma unroll
                for (int i = 0; i < kTileTokens<NP> / 16; ++i)
                    if (i * 16 < n && ok) finish(i * 16, sum[i]);
            }
            if (GATE) {
                fence_proxy_async_smem();
                epilogue_bar();
                const int GA = p.w.I >> 7;                 // groups of the activations; this tile is half of group r / 2
                const size_t ab = block_bytes(p.w.I, NP);
                uint8_t* blk = p.as + size_t(tile.y >> 3) * ab;
                if (ok && warp == kEpiWarp) {
                    if (lane < (n >> 3)) {
#pragma unroll
                        for (int s = 0; s < NP; ++s)
                            bulk_s2g(blk + lane * ab + (size_t(r >> 1) * NP + s) * 2048 + (r & 1) * 1024,
                                     tbuf + (size_t(lane) * NP + s) * 1024, 1024);
                    }
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                }
                if (ok && et < n) {
                    float X = psum[et];
#pragma unroll
                    for (int w = 1; w < 4; ++w) X = __fadd_rn(X, psum[w * 128 + et]);
                    uint8_t* sums = blk + size_t(et >> 3) * ab + size_t(GA) * NP * 2048;
                    put_sum(sums, p.w.I, et & 7, r, X);
                    if (r == 0)
                        for (int i = 0; i < 16; ++i) clear_sums(sums, p.w.I, et & 7, i);
                }
            }
        }
        if (GATE && warp == kEpiWarp) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (*abort_flag && lane == 0) {
        // the copies still in flight: the latest round of every stage
        if (warp == 0)
            for (int s = 0; s < WS; ++s)
                if (tw.round > 0 || s < tw.s) mbar_wait(&w_full[s], (s < tw.s ? tw.round : tw.round - 1) & 1u, p.err, 50000000ull);
        if (warp == kTokenWarp)
            for (int s = 0; s < BS; ++s)
                if (tb.round > 0 || s < tb.s) mbar_wait(&b_full[s], (s < tb.s ? tb.round : tb.round - 1) & 1u, p.err, 50000000ull);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, 512);
}

// ------------------------------------------------------------------ combine
constexpr int kCombineThr = 256;
template <typename OUT>
__global__ void __launch_bounds__(kCombineThr) moe_combine_kernel(const MoeTcParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, H = p.w.H;
    for (int h = threadIdx.x * 4; h < H; h += kCombineThr * 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < p.k; ++j) {
            const int at = p.pos[size_t(t) * p.k + j];
            if (at < 0) continue;
            const float w = p.weights[size_t(t) * p.k + j];
            const float4 o = *reinterpret_cast<const float4*>(p.out + size_t(at) * H + h);
            v.x = __fmaf_rn(w, o.x, v.x);
            v.y = __fmaf_rn(w, o.y, v.y);
            v.z = __fmaf_rn(w, o.z, v.z);
            v.w = __fmaf_rn(w, o.w, v.w);
        }
        const size_t at = size_t(t) * H + h;
        if constexpr (sizeof(OUT) == 4) {
            float4* y = reinterpret_cast<float4*>(static_cast<float*>(p.y) + at);
            if (p.resid) {
                const float4 o = *y;
                v = make_float4(__fadd_rn(o.x, v.x), __fadd_rn(o.y, v.y), __fadd_rn(o.z, v.z), __fadd_rn(o.w, v.w));
            }
            *y = v;
        } else {
            uint2* y = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at);
            if (p.resid) {
                const uint2 o = *y;
                v = make_float4(__fadd_rn(bf16_lo(o.x), v.x), __fadd_rn(bf16_hi(o.x), v.y), __fadd_rn(bf16_lo(o.y), v.z),
                                __fadd_rn(bf16_hi(o.y), v.w));
            }
            *y = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
    }
}

const void* product_fn(bool bf16, bool gate) {
    if (bf16) return gate ? (const void*)moe_product_kernel<1, true> : (const void*)moe_product_kernel<1, false>;
    return gate ? (const void*)moe_product_kernel<2, true> : (const void*)moe_product_kernel<2, false>;
}

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

// Tokens of a tile: enough for most experts at once when the places are spread evenly, and no more, since shorter stages mean
// more groups in flight.
int moe_tc_cap(long long places, int E, bool bf16) {
    const long long mean = places / E;
    return mean <= 6 ? 16 : (mean <= 14 ? 32 : (mean <= 40 || !bf16 ? kTileTokens<2> : kTileTokens<1>));
}

MoeTcSizes moe_tc_sizes(const MoeView& w, bool bf16, int T, int k) {
    const int np = bf16 ? 1 : 2;
    const size_t S = size_t(T) * k, experts = S < size_t(w.E) ? S : size_t(w.E);
    const size_t P = (S + 15 * experts + 15) & ~size_t(15);
    MoeTcSizes z = {};
    z.tiles = 16;
    z.pos = z.tiles + (experts + P / 16) * 16;
    z.isx = z.pos + up16(S * 4);
    z.sact = z.isx + up16(P * 4);
    z.xs = z.sact + up16(P * 4);
    z.as = z.xs + P / 8 * block_bytes(w.H, np);
    z.out = z.as + P / 8 * block_bytes(w.I, np);
    z.total = z.out + P * w.H * 4;
    return z;
}

cudaError_t launch_moe_tc(const MoeTcParams& p, bool bf16, int sms, cudaStream_t st) {
    const MoeTcParams* q = &p;
    cudaError_t e = launch_dependent((const void*)moe_plan_kernel, dim3(1), kPlanThr, 0, 1, q, st);
    if (e != cudaSuccess) return e;
    const void* stage = bf16 ? (const void*)moe_stage_kernel<uint16_t, 1> : (const void*)moe_stage_kernel<float, 2>;
    if ((e = launch_dependent(stage, dim3(p.T), kStageThr, 0, 1, q, st)) != cudaSuccess) return e;
    for (const bool gate : {true, false}) {
        const size_t smem = layout(bf16 ? 1 : 2, gate, gate ? p.w.H : p.w.I).total;
        if ((e = launch_dependent(product_fn(bf16, gate), dim3(sms), kThr, smem, 1, q, st)) != cudaSuccess) return e;
    }
    const void* combine = bf16 ? (const void*)moe_combine_kernel<uint16_t> : (const void*)moe_combine_kernel<float>;
    return launch_dependent(combine, dim3(p.T), kCombineThr, 0, 1, q, st);
}

cudaError_t launch_moe_factors(const MoeView& w, float* rho_gate_up, float* rho_down, float* norms, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(norms, 0, size_t(w.E) * 2 * 4, st);
    if (e != cudaSuccess) return e;
    moe_factors_kernel<<<dim3((2 * w.I + 127) / 128, w.E), 128, 0, st>>>(w.gate_up, w.I / 8, w.H / 128, rho_gate_up, norms);
    moe_factors_kernel<<<dim3((w.H + 127) / 128, w.E), 128, 0, st>>>(w.down, w.H / 16, w.I / 128, rho_down, nullptr);
    return cudaGetLastError();
}

cudaError_t moe_tc_set_attributes() {
    cudaError_t e;
    for (int b = 0; b < 2; ++b)
        for (int gate = 0; gate < 2; ++gate) {
            e = cudaFuncSetAttribute(product_fn(b != 0, gate != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(layout(b ? 1 : 2, gate != 0, kMoeMaxDim).total));
            if (e != cudaSuccess) return e;
        }
    const void* others[] = {(const void*)moe_plan_kernel, (const void*)moe_factors_kernel, (const void*)moe_stage_kernel<uint16_t, 1>,
                            (const void*)moe_stage_kernel<float, 2>, (const void*)moe_combine_kernel<uint16_t>,
                            (const void*)moe_combine_kernel<float>};
    for (const void* fn : others) {
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, fn)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kmr
