// Int4 experts for many tokens: the places (token, j) are grouped by expert and both products run as ragged grouped
// GEMMs on the 5th-generation tensor cores.
//
//   plan     counts the places of every expert and gives each a position; an expert's positions are padded to a multiple
//            of 16 and cut into tiles of at most `cap` (16..128) tokens
//   stage    token rows as fp16 into the tiles' operand layout (a copy per place)
//   gate_up  D = A B^T per (tile, 128 packed weight rows), silu(gate) * up, in fp32
//   act      the activations as fp16 in the operand layout, at the power of two of their row's largest
//   down     the same product, a row for every place
//   combine  y[t] = sum_j weights[t, j] * row of place (t, j), in the order of the places: no atomics on values
//
// The product, D[row][token] = sum_k w[row][k] x[token][k], w = (q - 8) s + z:
//   * A = (q - 8) s rho 2^-24: a 4-bit integer times a bf16 scale has 11 significant bits, so fp16 holds it exactly once a power of
//     two rho per row (laid out once, moe_factors_kernel) has brought the row's scales into its range (a group whose scale is below
//     2^-6 of the row's largest loses what lies below 2^-24, against a largest weight of 2^-8 or more).  A nibble under a zero mantissa is the
//     fp16 number q 2^-24 as it stands, so a weight is one AND and half an HFMA2: q 2^-24 * (s rho) - 8 s rho 2^-24.  (With 1024
//     + q, an addition and a multiplication the half-rate fp16 pipe is the bound.)
//   * the zero points' share sum_g z_g X_g, X_g = sum of the group's inputs, goes through the same accumulator as one more MMA for
//     every two groups: z rho 2^6 against X 2^-6 for every 64 inputs, X in two fp16 terms.
//   * B = x sigma (a power of two per row): exact for bf16 inputs down to 2^-30 of the row's largest, two terms (the fp16 rounding
//     and what it left, 22 bits down to 2^-16, two MMAs on the same A) for fp32 ones.  The products of these are exact, sums are fp32.
//   * the accumulators of a tile take a row's whole sum, so an activation row has one scale: that of its largest value, which is
//     known when all of its tiles are.  Hence act, a pass over the rows by itself.  (A scale from bounds, |silu(g) u| <= (|x|
//     max |gate row|) (|x| max |up row|), needs no pass but is loose by the spread of the rows' sizes twice over, and by
//     exp(-g) where the gates are shut: one gate and one up row of 256 times the others' size, fp32: 1.6e-2 of the result.)
//
// Each CTA is persistent and warp-specialised: a weight producer and a token producer (cp.async.bulk rings), eight or twelve warps
// that turn KMR4 blocks into A in tensor memory (kmr_tcgemm.cu describes that layout), one that lays out their zero points, one
// thread that issues the MMAs, eight epilogue warps on the accumulators that are done (for fp32 they also add up the groups'
// sums).  Every wait is bounded; a timeout records KMR_ERR_DEVICE_TIMEOUT, skips the remaining work, drains the copies in
// flight and frees tensor memory.
//
// Measured (us: plan, stage, gate_up, act, down, combine; hidden 2048).  128 experts of 768, 8 a token: 16 rows fp32 5, 5, 37, 4.5, 25,
// 4; 509 rows fp32 6, 9, 99, 8, 49, 9.5; 4096 rows bf16 10, 52, 165, 30, 103, 28.  8 experts of 6144, 2 a token, bf16: 1024 rows 5, 6,
// 89, 18, 60, 7.  What bounds the products: for small tiles the turning of KMR4 blocks into A (2,300 cycles for each of three sets of
// warps a pair of groups, 14 bytes of weights a cycle on an SM) and its hand-overs; for tiles of 128 the MMAs' 1,090 cycles a
// pair and theirs (1,550 in all); for fp32 tiles of 32 to 64 the epilogue, which reads every group's sums.
#include <cuda_fp16.h>

#include <type_traits>

#include "kmr_int4_mma.cuh"
#include "kmr_moe.cuh"
#include "kmr_tc.cuh"

namespace kmr {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kRows = 128;                        // packed weight rows of a product (the MMA's M)
constexpr uint32_t kWBytes = 16 * kGroupBytes;    // two groups of eight KMR4 tiles
constexpr int kMaxAcc = 8;                        // accumulators: as many as the columns beside A hold

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(max(1, min(253, e + 127))) << 23); }
// e such that |v| < 2^e, for v >= 0 (128 or more for what is not finite)
__device__ __forceinline__ int above(float v) { return int(__float_as_uint(v) >> 23) - 126; }
__device__ __forceinline__ float inverse_pow2(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }

// ------------------------------------------------------------------ weights, once
// Row factors rho (a power of two that brings max(|s|, 2^-18 |z|) of the row to [2^13, 2^14)) and, where norms is given, the largest
// row norm bound of each expert: |w|^2 <= sum over groups of 128 max(|z - 8 s|, |z + 7 s|)^2.
__global__ void moe_factors_kernel(const uint8_t* w, int tiles, int G, float* rho, float* norms) {
    const int row = blockIdx.x * blockDim.x + threadIdx.x, e = blockIdx.y;
    if (row >= tiles * 16) return;
    const uint8_t* at = w + (size_t(e) * tiles + row / 16) * G * kGroupBytes + 1024 + (row & 15) * 4;
    float m = 0.f, n2 = 0.f;
    for (int g = 0; g < G; ++g) {
        const uint32_t sz = *reinterpret_cast<const uint32_t*>(at + size_t(g) * kGroupBytes);
        const float s = bf16_lo(sz), z = bf16_hi(sz);
        m = fmaxf(m, fmaxf(fabsf(s), 0x1p-18f * fabsf(z)));
        const float far = fmaxf(fabsf(__fmaf_rn(-8.f, s, z)), fabsf(__fmaf_rn(7.f, s, z)));
        n2 = __fmaf_rn(128.f * far, far, n2);
    }
    float r, ir;
    pow2_scale(__float_as_uint(m), r, ir);
    rho[size_t(e) * tiles * 16 + row] = r;
    // (a bound: rounded up; the bits of non-negative floats order like integers)
    if (norms) atomicMax(reinterpret_cast<int*>(norms + e), __float_as_int(sqrtf(n2) * 1.001f));
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
    // each place's expert and its rank among the expert's places (which rank it gets does not change any result)
    constexpr int kPer = kMoeChunkPlaces / kPlanThr;
    uint32_t mine[kPer];
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
        const int i = b * kPlanThr + tid;
        mine[b] = i < S ? uint32_t(p.ids[i]) : 0xffffffffu;
    }
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
        if (b * kPlanThr >= S) break;
        const bool real = mine[b] < uint32_t(p.w.E);
        if (!real && mine[b] != 0xffffffffu) set_error(p.err, KMR_ERR_INVALID_ARG);
        mine[b] = real ? mine[b] << 16 | uint32_t(atomicAdd(&count[mine[b]], 1)) : 0xffffffffu;
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
            const int len = min(each, n16 - i * each);               // (above 0: each is at most cap)
            p.tiles[t0 + i] = make_int4(tid, p0 + i * each, len, min(len, n - i * each));
        }
    }
    if (tid == kPlanThr - 1) *p.ntiles = pb + b;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
        const int i = b * kPlanThr + tid;
        if (i < S) p.pos[i] = mine[b] == 0xffffffffu ? -1 : at[mine[b] >> 16] + int(mine[b] & 0xffffu);
    }
}

// ------------------------------------------------------------------ operand layout
// Staged rows, `blocks` blocks of 8: for every group of 128 inputs and each of the NP terms all the blocks side by side, each 2 atoms
// of [8 rows][64 inputs] fp16 with the 16-byte pieces of a row swizzled by the row (the MMA's 128-byte swizzle), so that a
// tile's share of a group is one run of memory.  Behind them, by pairs of groups, the sums of the four 64 inputs, [8
// rows][8]: per group the first terms of its two sums and their remainders (zeros for the group an odd last pair lacks).
// Input k of 16 sits at 2 (k % 8) - k % 2 + 2 (k / 8) (the order of A's columns in tensor memory).
__host__ __device__ constexpr int pairs_of(int K) { return (K / 128 + 1) / 2; }
__host__ __device__ constexpr size_t staged_bytes(int K, int np, size_t blocks) {
    return blocks * (size_t(K / 128) * np * 2048 + pairs_of(K) * 128);
}
__device__ __forceinline__ size_t atom_at(int h, int term, int np, size_t blocks, int block) {     // of 64 inputs number h
    return ((size_t(h >> 1) * np + term) * blocks + block) * 2048 + (h & 1) * 1024;
}
__device__ __forceinline__ size_t sums_at(int K, int np, size_t blocks) { return size_t(K / 128) * blocks * np * 2048; }
__device__ __forceinline__ uint32_t piece(int row, int c) { return uint32_t(row * 128 + ((c ^ row) << 4)); }
// Sum number h (of 64 inputs) of a row: its two terms, in the row's pieces of 8 numbers for each pair of groups.
__device__ __forceinline__ void put_sum(void* row, int h, float X) {
    const float x = X * 0.015625f;
    const __half hi = __float2half_rn(x);
    __half* to = reinterpret_cast<__half*>(static_cast<uint8_t*>(row) + (h >> 2) * 16) + ((h >> 1) & 1) * 4 + (h & 1);
    to[0] = hi;
    to[2] = __float2half_rn(__fsub_rn(x, __half2float(hi)));
}

// A lane's four inputs (k = 4 x its number), scaled, as NP terms: the 8 bytes of a piece that it writes (a 16-byte piece holds inputs
// 0, 1, 8, 9, 2, 3, 10, 11 (or 4 more) of its 16: two lanes write its halves), and the sum of its 16 lanes' 64.  By whole warps.
template <int NP>
__device__ __forceinline__ float stage4(const float (&a)[4], int m4, uint2 (&out)[NP]) {
    auto h2u = [](__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); };
    float X = 0.f;
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
        const uint32_t wa = h2u(h0), wb = h2u(h1);
        const uint32_t got = __shfl_xor_sync(kFull, m4 < 2 ? wb : wa, 2);
        out[q] = m4 < 2 ? make_uint2(wa, got) : make_uint2(got, wb);
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) X = __fadd_rn(X, __shfl_xor_sync(kFull, X, o));
    return X;
}
// Where they go: inputs k .. k + 3 of the row at position `at`.
__device__ __forceinline__ size_t four_at(int k, int at, int np, size_t blocks) {
    return atom_at(k >> 6, 0, np, blocks, at >> 3) + piece(at & 7, ((k & 63) >> 4) * 2 + ((k >> 2) & 1)) + ((k & 8) ? 8 : 0);
}
// A row's sums, from `sums` (put_sum's) to position `at`: pair number pr.
__device__ __forceinline__ void store_sums(uint8_t* to, const void* sums, int pr, int K, int np, size_t blocks, int at) {
    uint4 v = reinterpret_cast<const uint4*>(sums)[pr];
    if (2 * pr + 1 == K >> 7) v.z = v.w = 0u;              // (the half of the last pair that an odd number of groups leaves)
    *reinterpret_cast<uint4*>(to + sums_at(K, np, blocks) + (size_t(pr) * blocks + (at >> 3)) * 128 + (at & 7) * 16) = v;
}

// ------------------------------------------------------------------ stage
constexpr int kStageThr = 256;
template <typename IN, int NP, int PER>
__global__ void __launch_bounds__(kStageThr) moe_stage_kernel(const MoeTcParams p) {
    __shared__ float red[kStageThr / 32];
    __shared__ int pos[kMoeMaxTopK], places;
    __shared__ __align__(16) __half sums[kMoeMaxDim / 64 * 2];          // of the row, as a pair's 16 bytes
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = p.w.H, K4 = K >> 2;
    float4 v[PER];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k4 = tid + i * kStageThr;
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k4 >= K4) continue;
        if constexpr (sizeof(IN) == 4) {
            v[i] = reinterpret_cast<const float4*>(static_cast<const float*>(p.x) + size_t(t) * K)[k4];
        } else {
            const uint2 r = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.x) + size_t(t) * K)[k4];
            v[i] = make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        }
    }
    if (warp == 0) {
        const int at = lane < p.k ? p.pos[size_t(t) * p.k + lane] : -1;
        const uint32_t some = __ballot_sync(kFull, at >= 0);
        if (at >= 0) pos[__popc(some & ((1u << lane) - 1u))] = at;
        if (lane == 0) places = __popc(some);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
    m = warp_max(m);
    if (lane == 0) red[warp] = m;
    __syncthreads();
    const int n = places;
    if (n == 0) return;
    m = red[0];
#pragma unroll
    for (int w = 1; w < kStageThr / 32; ++w) m = fmaxf(m, red[w]);
    float sig, isg;
    pow2_scale(__float_as_uint(m), sig, isg);
    const size_t blocks = p.blocks;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int k4 = tid + i * kStageThr;
        if (k4 >= K4) break;                                        // (whole warps: K4 is a multiple of 32)
        const int k = k4 * 4, m4 = k4 & 3;
        const float a[4] = {__fmul_rn(v[i].x, sig), __fmul_rn(v[i].y, sig), __fmul_rn(v[i].z, sig), __fmul_rn(v[i].w, sig)};
        uint2 out[NP];
        const float X = stage4<NP>(a, m4, out);
        for (int j = 0; j < n; ++j) {
            uint8_t* to = p.xs + four_at(k, pos[j], NP, blocks);
#pragma unroll
            for (int q = 0; q < NP; ++q) *reinterpret_cast<uint2*>(to + q * blocks * 2048) = out[q];
        }
        if ((lane & 15) == 0) put_sum(sums, k >> 6, X);
    }
    __syncthreads();
    for (int i = tid; i < n * pairs_of(K); i += kStageThr) store_sums(p.xs, sums, i % pairs_of(K), K, NP, blocks, pos[i / pairs_of(K)]);
    if (tid < n) p.isx[pos[tid]] = isg;
}

// ------------------------------------------------------------------ the grouped product
// warps 0, 1, 2, 3: weights, MMA, tokens, zero points; then the unpack warps and the epilogue warps, from multiples of four on (a warp reaches the
// quarter warp % 4 of the tensor memory's lanes)
constexpr int kTokenWarp = 2, kZeroWarp = 3, kUnpackWarp = 4, kEpiWarps = 8, kMaxSets = 3;
constexpr int epilogue_warp(int sets) { return kUnpackWarp + 4 * sets; }
constexpr int product_threads(int sets) { return (epilogue_warp(sets) + kEpiWarps) * 32; }
constexpr uint32_t kSmem = 227 * 1024;

// The tensor cores cut a running sum off rather than round it, so a chain of n steps of 16 inputs comes out some n 2^-25 too
// small (measured: 1040 steps, 2.3e-5).  bf16 results do not show it.  For fp32 the epilogue warps add up the groups' sums (8
// steps) in registers, which limits a tile to 64 tokens.  (Four groups at a time: 3.7e-6 of the result.)
template <int NP>
constexpr int kTileTokens = NP == 2 ? 64 : 128;

// Shared memory: the zero points (of a pair of groups for each set), barriers, the tokens' factors, the token
// ring, 2 KB of zeros (behind whatever needs them as its second 16 bytes), the weight ring.  A stage of the token ring holds two
// groups of `cap` tokens and their sums; of 128 tokens one group, as two stages of 66 KB leave the MMAs waiting for the next (1024
// rows of 8 experts: 173 us against 163; for smaller tiles the second hand-over costs more than it gives, 80 rows: 87
// against 80).  Small tiles leave more of the memory to the weights, whose latency they have less work to hide.
constexpr uint32_t kZBytes = kRows * 16;
constexpr int kMaxStages = 8, kMaxWS = 8;
struct Layout {
    uint32_t z, bar, fac, ring;
};
__host__ __device__ constexpr Layout layout() {
    Layout l = {};
    l.bar = l.z + kMaxSets * kZBytes;
    l.fac = l.bar + 512;
    l.ring = (l.fac + 2 * 2 * 128 * 4 + 1023u) & ~1023u;
    return l;
}
__host__ __device__ constexpr int stage_groups(int cap) { return cap == 128 ? 1 : 2; }
__host__ __device__ constexpr uint32_t stage_bytes(int cap, int np) {
    return uint32_t(cap) * 256u * np * stage_groups(cap) + uint32_t(cap < 64 ? 1024 : cap * 16);
}
__host__ __device__ constexpr int token_stages(int cap, int np) {
    const int n = int(72u * 1024u / stage_bytes(cap, np)), least = stage_groups(cap) == 1 ? 4 : 2;
    return n < least ? least : (n > kMaxStages ? kMaxStages : n);
}
__host__ __device__ constexpr int weight_stages(int cap, int np) {
    const int n = int((kSmem - layout().ring - token_stages(cap, np) * stage_bytes(cap, np) - kZBytes) / kWBytes);
    return n > kMaxWS ? kMaxWS : n;
}
static_assert(weight_stages(128, 1) >= 3 && weight_stages(64, 2) >= 3, "shared memory");

// Shared-memory matrix descriptors, K-major.  Staged rows (128-byte swizzle, blocks of 8 rows 2 KB apart): the upper half is this
// constant, the lower the address and 1 << 16.
constexpr uint32_t kSwizzledHi = (2048u >> 4) | (1u << 14) | (2u << 29);
// No swizzle: 8 rows x 16 bytes side by side for consecutive blocks of 8 rows, the second 16 bytes `further` on.
// The upper half is a constant; the lower one of the next address `step` on, with the same second 16 bytes, is plain_step on.
constexpr uint32_t kPlainHi = (128u >> 4) | (1u << 14);
__device__ __forceinline__ uint32_t plain_lo(uint32_t addr, uint32_t second) {
    return ((addr >> 4) & 0x3FFFu) | (((second - addr) >> 4) & 0x3FFFu) << 16;
}
__device__ __forceinline__ constexpr uint32_t plain_step(uint32_t step) { return (step >> 4) - ((step >> 4) << 16); }
// D += A B^T for one K = 16 step, both in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t taddr, uint64_t ad, uint64_t bd, uint32_t idesc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(taddr),
                 "l"(ad), "l"(bd), "r"(idesc)
                 : "memory");
}
__device__ __forceinline__ void epilogue_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory"); }
// silu(x) * up.  bf16 results: __expf, documented to 2 + |1.17 x| units of 2^-23 (2^-18 at |x| = 30, 2^-16 where silu leaves the range of
// fp32), and __fdividef, to 2 units up to a divisor of 2^126 and 0 beyond (x below -87): far below the 11 bits that are kept.
template <bool FAST>
__device__ __forceinline__ float silu_mul(float x, float up) {
    if (FAST) return __fmul_rn(__fdividef(x, __fadd_rn(1.f, __expf(-x))), up);
    return __fmul_rn(__fdiv_rn(x, __fadd_rn(1.f, expf(-x))), up);
}
// Four steps of 8 columns at once.
__device__ __forceinline__ void tmem_store4(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void commit_at(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// Bounded wait; gives up at once when another warp has.
__device__ __forceinline__ bool wait_at(uint32_t b, uint32_t parity, volatile int* abort_flag, int* err) {
    if (try_at(b, parity)) return true;
    const long long c0 = clock64();
    for (uint32_t it = 1; it < (1u << 28); ++it) {
        if (try_at(b, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() - c0 > 4000000000ll) break;
    }
    set_error(err, KMR_ERR_DEVICE_TIMEOUT);
    *abort_flag = 1;
    return false;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t* b, uint32_t parity, volatile int* abort_flag, int* err) {
    return wait_at(smem_u32(b), parity, abort_flag, err);
}

// A stage of a ring and how often the ring has come round.
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

// Sets of unpack warps: three where tiles are small and that is what bounds the call, as far as the accumulators leave them tensor
// memory (80 rows of 60 experts: 74 us, with two 76), else two.
__host__ __device__ constexpr int unpack_sets(int cap, int np) { return cap * np <= 64 ? 3 : 2; }

// Roles.  Groups are handed over in pairs.  The unpack warps are SETS sets of four (one warp per quarter of the tensor memory's
// lanes) on every SETS-th pair, each with its own place in tensor memory: one set's waits and hand-over, some 900 cycles, fall
// under the others' arithmetic.  (Two sets on the two groups of one pair wait and work in step: 1650 cycles a pair instead of
// 1000; twice as many warps to a pair doubled the hand-overs' instructions.)
// GS: groups of a stage of the token ring.
template <int NP, bool GATE, int GS, int SETS>
__global__ void __launch_bounds__(product_threads(SETS), 1) moe_product_kernel(const MoeTcParams p) {
    constexpr int kEpiWarp = epilogue_warp(SETS), kThr = product_threads(SETS);
    extern __shared__ __align__(1024) uint8_t smem[];
    const int K = GATE ? p.w.H : p.w.I, N = GATE ? 2 * p.w.I : p.w.H, G = K >> 7;
    const int R = N / kRows;                               // row tiles of an expert
    constexpr Layout L = layout();
    const uint32_t bstage = stage_bytes(p.cap, NP);
    const int BS = token_stages(p.cap, NP), WS = weight_stages(p.cap, NP);
    const uint32_t zeros_at = L.ring + BS * bstage, wring = zeros_at + kZBytes;
    // accumulators: bf16 of a tile, fp32 of a pair's two groups side by side; where a token stage's sums begin
    const uint32_t dcols = uint32_t(p.cap) * NP, xoff = dcols * 256u * GS;
    const int DB = min(kMaxAcc, (512 - 128 * SETS) / int(dcols));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint64_t* w_full = reinterpret_cast<uint64_t*>(smem + L.bar);
    uint64_t* w_empty = w_full + kMaxWS;
    uint64_t* b_full = w_empty + kMaxWS;
    uint64_t* b_empty = b_full + kMaxStages;
    uint64_t* a_full = b_empty + kMaxStages;
    uint64_t* a_empty = a_full + kMaxSets;
    uint64_t* d_full = a_empty + kMaxSets;
    uint64_t* d_empty = d_full + kMaxAcc;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(d_empty + kMaxAcc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    static_assert(2 * (kMaxWS + kMaxStages + kMaxSets + kMaxAcc) * 8 + 8 <= 512, "barrier area");
    const uint32_t sbase = smem_u32(smem);

    if (tid == 0) {
        *abort_flag = 0;
        for (int s = 0; s < WS; ++s) {
            mbar_init(&w_full[s], 1);
            mbar_init(&w_empty[s], 4 + 1);           // a set and the zero points' warp
        }
        for (int s = 0; s < BS; ++s) {
            mbar_init(&b_full[s], 1);
            mbar_init(&b_empty[s], 1);
        }
        for (int s = 0; s < SETS; ++s) {
            mbar_init(&a_full[s], 4 + 1);
            mbar_init(&a_empty[s], 1);
        }
        for (int s = 0; s < DB; ++s) {
            mbar_init(&d_full[s], 1);
            mbar_init(&d_empty[s], kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == 0) tc_alloc(tslot, 512);
    for (int i = tid; i < int(kZBytes) / 4; i += kThr) reinterpret_cast<uint32_t*>(smem + zeros_at)[i] = 0u;
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = *tslot, abase = taddr + 512 - 128 * SETS;
    pdl_wait();
    pdl_launch_dependents();
    // a warp waits as one
    auto warp_wait = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(kFull, wait_or_abort(b, parity, abort_flag, p.err)) != 0;
    };
    const int items = *p.ntiles * R, step = int(gridDim.x);
    const uint8_t* wsrc = GATE ? p.w.gate_up : p.w.down;
    const uint8_t* bsrc = GATE ? p.xs : p.as;
    const float* rho = GATE ? p.rho_gate_up : p.rho_down;
    // what the tile of item `it` is (the next item's is always fetched ahead)
    auto tile_of = [&](int it) { return it < items ? p.tiles[it / R] : make_int4(0, 0, 0, 0); };
    Turn tw, tb;                                           // the producers' own rings
    bool ok = true;
    // after a timeout: the copies still in flight, the latest round of every stage
    auto drain = [&](uint64_t* full, int stages, const Turn& t) {
        if (!*abort_flag) return;
        for (int s = 0; s < stages; ++s)
            if (t.round > 0 || s < t.s) mbar_wait(&full[s], (s < t.s ? t.round : t.round - 1) & 1u, p.err, 50000000ull);
    };

    auto one_wait = [&](uint64_t* b, uint32_t parity) { return wait_or_abort(b, parity, abort_flag, p.err); };

    if (warp == 0) {
        // ---- weights: two groups of each of the eight tiles (they are neighbours in memory)
        if (elect_one()) {
            const uint64_t pol = policy_evict_first();
            int4 tile = tile_of(blockIdx.x);
            for (int it = blockIdx.x; it < items && ok; it += step) {
                const int4 ahead = tile_of(it + step);
                const uint8_t* src = wsrc + (size_t(tile.x) * (N / 16) + (it % R) * 8) * G * kGroupBytes;
#pragma unroll 1
                for (int g = 0; g < G; g += 2) {
                    if (tw.waits() && !(ok = one_wait(&w_empty[tw.s], tw.empty()))) break;
                    const uint32_t bytes = uint32_t(min(2, G - g)) * kGroupBytes;
                    mbar_arrive_expect_tx(&w_full[tw.s], 8 * bytes);
                    fence_proxy_async_smem();              // the unpack warps' reads of the stage come first
                    uint8_t* to = smem + wring + tw.s * kWBytes;
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        bulk_g2s_stream(to + t * bytes, src + (size_t(t) * G + g) * kGroupBytes, bytes, &w_full[tw.s], pol);
                    tw.next(WS);
                }
                tile = ahead;
            }
            drain(w_full, WS, tw);
        }
    } else if (warp == kTokenWarp) {
        // ---- staged tokens: the groups' shares of the tile, and with the last of a pair its sums
        if (elect_one()) {
            const size_t blocks = p.blocks, gstep = size_t(NP) * blocks * 2048;
            const uint8_t* sums = bsrc + sums_at(K, NP, blocks);
            int4 tile = tile_of(blockIdx.x);
            for (int it = blockIdx.x; it < items && ok; it += step) {
                const int4 ahead = tile_of(it + step);
                const uint32_t nb = uint32_t(tile.z) >> 3;
                const size_t first = size_t(tile.y >> 3);
                const uint8_t* src = bsrc + first * 2048;
#pragma unroll 1
                for (int g = 0; g < G; g += GS) {
                    const int both = min(GS, G - g);
                    const bool last = GS == 2 || (g & 1) || g + 1 == G;
                    if (tb.waits() && !(ok = one_wait(&b_empty[tb.s], tb.empty()))) break;
                    mbar_arrive_expect_tx(&b_full[tb.s], (2048u * NP * both + (last ? 128u : 0u)) * nb);
                    uint8_t* to = smem + L.ring + size_t(tb.s) * bstage;
#pragma unroll
                    for (int j = 0; j < GS; ++j) {
                        if (j < both) {
#pragma unroll
                            for (int q = 0; q < NP; ++q)
                                bulk_g2s(to + (j * NP + q) * nb * 2048, src + q * blocks * 2048, nb * 2048, &b_full[tb.s]);
                        }
                        src += gstep;
                    }
                    if (last) bulk_g2s(to + xoff, sums + (size_t(g >> 1) * blocks + first) * 128, nb * 128, &b_full[tb.s]);
                    tb.next(BS);
                }
                tile = ahead;
            }
            drain(b_full, BS, tb);
        }
    } else if (warp == 1) {
        // ---- MMA issue, by one elected thread (elect.sync: with `lane == 0` the compiler does not know that the operands are
        // uniform, and an MMA takes 55 cycles to issue instead of 6).  Alone on its path it takes some 6 cycles an instruction, so
        // everything that can be is kept in running registers: a loop of Turns and pointers took 1600 cycles a pair.
        if (elect_one()) {
            const uint32_t bars = smem_u32(b_full), bfull = bars, bempty = bars + 8 * kMaxStages, afull = smem_u32(a_full),
                           aempty = smem_u32(a_empty), dfull = smem_u32(d_full), dempty = smem_u32(d_empty);
            const uint32_t blo0 = (((sbase + L.ring) >> 4) & 0x3FFFu) | (1u << 16), bstep = bstage >> 4;
            const uint32_t zeros = sbase + zeros_at, zlo0 = plain_lo(sbase + L.z, zeros), xlo0 = plain_lo(sbase + L.ring + xoff, zeros);
            const uint32_t xstep = plain_step(bstage);
            uint32_t zlo = zlo0, xlo = xlo0;               // descriptors of the pair's zero points and sums
            uint32_t bs = 0, bph = 0, blo = blo0, as = 0, aph = 0, ds = 0, dph = 1, acc = taddr;
            auto wait = [&](uint32_t bar, uint32_t parity) { return wait_at(bar, parity, abort_flag, p.err); };
            auto eight = [&](uint32_t d, uint32_t a, uint32_t lo, uint32_t idesc, uint32_t begun) {
                const uint64_t desc = (uint64_t(kSwizzledHi) << 32) | lo;
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                    tc_mma_ta(d, a + ks * 8, desc + (ks >> 2) * 64 + (ks & 3) * 2, idesc, ks == 0 ? begun : 1u);
            };
            auto hand_over = [&]() {                       // the accumulator to the epilogue
                commit_at(dfull + 8 * ds);
                acc += dcols;
                if (++ds == uint32_t(DB)) {
                    ds = 0;
                    dph ^= 1;
                    acc = taddr;
                }
            };
            int4 tile = tile_of(blockIdx.x);
            for (int it = blockIdx.x; it < items && ok; it += step) {
                const int4 ahead = tile_of(it + step);
                const uint32_t idesc = tc_idesc(kRows, tile.z), rest = uint32_t(tile.z) * 16;   // (to the second terms, in 16 bytes)
                if (NP == 1 && !(ok = wait(dempty + 8 * ds, dph))) break;
#pragma unroll 1
                for (int g = 0; g < G; g += 2) {
                    if (!(ok = (NP == 1 || wait(dempty + 8 * ds, dph)) && wait(bfull + 8 * bs, bph) && wait(afull + 8 * as, aph))) break;
                    tc_fence_after();
                    const uint32_t a = abase + as * 128;
                    // (fp32: the small second terms first, so that only the first terms' 8 steps cut off from a sum of full size)
                    if (NP == 2) eight(acc, a, blo + rest, idesc, 0u);
                    eight(acc, a, blo, idesc, NP == 2 || g > 0 ? 1u : 0u);
                    auto next_stage = [&]() {
                        commit_at(bempty + 8 * bs);
                        blo += bstep;
                        xlo += xstep;
                        if (++bs == uint32_t(BS)) {
                            bs = 0;
                            bph ^= 1;
                            blo = blo0;
                            xlo = xlo0;
                        }
                    };
                    if (g + 1 < G) {
                        if (GS == 1) {
                            next_stage();
                            if (!(ok = wait(bfull + 8 * bs, bph))) break;
                            tc_fence_after();
                        }
                        const uint32_t d = NP == 2 ? acc + (dcols >> 1) : acc, lo = GS == 1 ? blo : blo + NP * rest;
                        if (NP == 2) eight(d, a + 64, lo + rest, idesc, 0u);
                        eight(d, a + 64, lo, idesc, 1u);
                    }
                    // the pair's zero points
                    mma_ss(acc, (uint64_t(kPlainHi) << 32) | zlo, (uint64_t(kPlainHi) << 32) | xlo, idesc);
                    commit_at(aempty + 8 * as);
                    next_stage();
                    if (NP == 2) hand_over();
                    zlo += plain_step(kZBytes);
                    if (++as == uint32_t(SETS)) {
                        as = 0;
                        aph ^= 1;
                        zlo = zlo0;
                    }
                }
                if (!ok) break;
                if (NP == 1) hand_over();
                tile = ahead;
            }
        }
    } else if (warp == kZeroWarp) {
        // ---- zero points of the pair's rows, four rows a lane, off the unpack warps' path
        auto dup = [&](uint32_t sz, float r) {
            const float z = __fmul_rn(bf16_hi(sz) * 0x1p-18f, r);
            const __half2 h = __floats2half2_rn(z, z);
            return *reinterpret_cast<const uint32_t*>(&h);
        };
        auto factors = [&](int it, const int4& tile, float (&to)[4]) {
            const float* at = rho + size_t(tile.x) * N + (it % R) * kRows + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = at[32 * i];
        };
        Turn tt, ta;
        float rr[4] = {1.f, 1.f, 1.f, 1.f}, rnext[4] = {1.f, 1.f, 1.f, 1.f};
        int4 ahead = tile_of(blockIdx.x);
        if (int(blockIdx.x) < items) factors(blockIdx.x, ahead, rnext);
        for (int it = blockIdx.x; it < items && ok; it += step) {
#pragma unroll
            for (int i = 0; i < 4; ++i) rr[i] = rnext[i];
            ahead = tile_of(it + step);
#pragma unroll 1
            for (int g = 0; g < G; g += 2) {
                const int both = min(2, G - g);
                if (g + 2 >= G && it + step < items) factors(it + step, ahead, rnext);
                if (!(ok = warp_wait(&w_full[tt.s], tt.full()))) break;
                // row 32 i + lane: tile 2 i + lane / 16, row lane % 16
                const uint8_t* at = smem + wring + tt.s * kWBytes + (lane >> 4) * both * kGroupBytes + 1024 + (lane & 15) * 4;
                uint32_t sz[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        sz[i][j] = j < both ? *reinterpret_cast<const uint32_t*>(at + (2 * i * both + j) * kGroupBytes) : 0u;
                if (ta.waits() && !(ok = warp_wait(&a_empty[ta.s], ta.empty()))) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t z0 = dup(sz[i][0], rr[i]), z1 = dup(sz[i][1], rr[i]);
                    *reinterpret_cast<uint4*>(smem + L.z + ta.s * kZBytes + (4 * i + (lane >> 3)) * 128 + (lane & 7) * 16) =
                        make_uint4(z0, z0, z1, z1);
                }
                fence_proxy_async_smem();                  // the MMA reads them through the async proxy
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&w_empty[tt.s]);
                    mbar_arrive(&a_full[ta.s]);
                }
                tt.next(WS);
                ta.next(SETS);
            }
        }
    } else if (warp >= kUnpackWarp && warp < kEpiWarp) {
        // ---- unpack: the two tiles of tensor-memory lane quarter warp % 4, every SETS-th pair of groups
        const int lq = warp & 3, set = (warp - kUnpackWarp) >> 2, g8 = lane >> 2;
        auto h2 = [](uint32_t v) { return *reinterpret_cast<const __half2*>(&v); };
        auto u2 = [](__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); };
        auto dup = [&](float v) { return __floats2half2_rn(v, v); };
        // factors of rows g8, g8 + 8, g8 + 16, g8 + 24 of the quarter
        auto factors = [&](int it, const int4& tile, float (&to)[4]) {
            const float* at = rho + size_t(tile.x) * N + (it % R) * kRows + 32 * lq;
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] = at[g8 + 8 * i];
        };
        const uint32_t aset = abase + set * 128 + (uint32_t(32 * lq) << 16);
        // this set's pairs are number set, set + SETS, ... of all: their stage of the weight ring, its parity, the place's parity
        uint32_t ws = set, wph = 0, aph = 1;
        int skip = set;                                    // pairs of the item that come before this set's next
        const int pairs = (G + 1) >> 1;
        const uint32_t wfull = smem_u32(w_full), aempty = smem_u32(a_empty + set);
        float rr[4] = {1.f, 1.f, 1.f, 1.f}, rnext[4] = {1.f, 1.f, 1.f, 1.f};
        int4 ahead = tile_of(blockIdx.x);
        if (int(blockIdx.x) < items) factors(blockIdx.x, ahead, rnext);
        for (int it = blockIdx.x; it < items && ok; it += step) {
#pragma unroll
            for (int i = 0; i < 4; ++i) rr[i] = rnext[i];
            ahead = tile_of(it + step);
            int pr = skip;
#pragma unroll 1
            for (; pr < pairs; pr += SETS) {
                const int both = min(2, G - 2 * pr);
                if (pr + SETS >= pairs && it + step < items) factors(it + step, ahead, rnext);
                if (!(ok = __all_sync(kFull, wait_at(wfull + 8 * ws, wph, abort_flag, p.err)))) break;
                const uint8_t* wst = smem + wring + ws * kWBytes + 2 * lq * both * kGroupBytes;
                // a group's words and scales
                uint4 wq[4];
                uint32_t sz[4];
                auto fetch = [&](int j) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint8_t* blk = wst + (h * both + j) * kGroupBytes;
                        sz[2 * h] = *reinterpret_cast<const uint32_t*>(blk + 1024 + g8 * 4);
                        sz[2 * h + 1] = *reinterpret_cast<const uint32_t*>(blk + 1024 + (g8 + 8) * 4);
                        wq[2 * h] = *reinterpret_cast<const uint4*>(blk + lane * 16);
                        wq[2 * h + 1] = *reinterpret_cast<const uint4*>(blk + 512 + lane * 16);
                    }
                };
                fetch(0);
                if (!(ok = __all_sync(kFull, wait_at(aempty, aph, abort_flag, p.err)))) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < both; ++j) {
                    if (j > 0) fetch(1);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // of rows g8 and g8 + 8: s rho, its 16th for the nibble one place up, and -8 of it 2^-24
                        const float r0 = __fmul_rn(bf16_lo(sz[2 * h]), rr[2 * h]), r1 = __fmul_rn(bf16_lo(sz[2 * h + 1]), rr[2 * h + 1]);
                        const __half2 s0 = dup(r0), n0 = dup(r0 * -0x1p-21f), s1 = dup(r1 * 0x1p-4f), n1 = dup(r1 * -0x1p-21f);
#pragma unroll
                        for (int kj = 0; kj < 2; ++kj) {
                            const uint4 q4 = wq[2 * h + kj];
                            const uint32_t w4[4] = {q4.x, q4.y, q4.z, q4.w};
                            uint32_t v[16];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t w = w4[k], wh = w >> 8;
                                v[4 * k] = u2(__hfma2(h2(w & 0x000F000Fu), s0, n0));
                                v[4 * k + 1] = u2(__hfma2(h2(wh & 0x000F000Fu), s0, n0));
                                v[4 * k + 2] = u2(__hfma2(h2(w & 0x00F000F0u), s1, n1));
                                v[4 * k + 3] = u2(__hfma2(h2(wh & 0x00F000F0u), s1, n1));
                            }
                            tmem_store4(aset + j * 64 + kj * 32 + (uint32_t(16 * h) << 16), v);
                        }
                    }
                }
                if (lane == 0) mbar_arrive(&w_empty[ws]);      // (all lanes' loads have been used by the stores above)
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&a_full[set]);
                aph ^= 1;
                ws += SETS;
                if (ws >= uint32_t(WS)) {
                    ws -= WS;
                    wph ^= 1;
                }
            }
            if (skip >= pairs && it + step < items) factors(it + step, ahead, rnext);
            skip = pr - pairs;
        }
    } else if (warp >= kEpiWarp) {
        // ---- epilogue: warp w reads tensor-memory lanes 32 (w % 4) .. + 31 (its weight rows), every second sixteen of the tokens
        const int q = warp & 3, et = tid - kEpiWarp * 32, half = (warp - kEpiWarp) >> 2;
        float* fac = reinterpret_cast<float*>(smem + L.fac);       // [2][2][128]
        const bool lo = (lane & 15) < 8;                           // gate_up: of the tile's 8 gate rows
        Turn td;
        int turn = 0;
        int4 tile = tile_of(blockIdx.x), ahead;
        float f0 = 0.f, f1 = 0.f, irho = 1.f;
        auto factors = [&](int it, const int4& tl) {
            if (et < tl.w) {
                f0 = GATE ? p.isx[tl.y + et] : p.isa[tl.y + et];
                if (!GATE && NP == 1) f1 = p.sout[tl.y + et];
            }
            irho = rho[size_t(tl.x) * N + (it % R) * kRows + 32 * q + lane];
        };
        if (int(blockIdx.x) < items) factors(blockIdx.x, tile);
        for (int it = blockIdx.x; it < items; it += step, turn ^= 1) {
            const int r = it % R, real = tile.w;
            float* f = fac + turn * 256;
            if (et < real) {
                f[et] = 0x1p12f * f0;
                if (!GATE && NP == 1) f[128 + et] = f1;
            }
            const float ir = 0x1p12f * inverse_pow2(irho);     // (the 2^24 of A, half of it with either factor)
            ahead = tile_of(it + step);
            // tokens c0 .. c0 + 15 of this lane's row
            auto finish = [&](int c0, const float (&v)[16]) {
                if (GATE) {
                    // in pairs: the gate lanes (tile rows 0..7) finish token c, the up lanes token c + 1
                    float* to = static_cast<float*>(p.out) + size_t(tile.y + c0 + (lo ? 0 : 1)) * p.w.I + r * 64 + 16 * q + (lane >> 4) * 8 + (lane & 7);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        if (c0 + j >= real) break;
                        const float2 u = *reinterpret_cast<const float2*>(f + c0 + j);
                        const float xa = __fmul_rn(v[j], __fmul_rn(ir, u.x)), xb = __fmul_rn(v[j + 1], __fmul_rn(ir, u.y));
                        const float other = __shfl_xor_sync(kFull, lo ? xb : xa, 8);
                        const float a = silu_mul<NP == 1>(lo ? xa : other, lo ? other : xb);
                        if (c0 + j + (lo ? 0 : 1) < real) to[size_t(j) * p.w.I] = a;
                    }
                } else {
                    // bf16: the rows wait for the weighted sum as fp16 (half a step: 2^-11, an eighth of the result's; fp32 rows would
                    // be 60% of the call's traffic), scaled by |act| max |down row|.  A value is typically 2^-5 (I 128) to 2^-10 (I
                    // 8192) of that bound, and fp16's normal range goes on for another 2^19: as far as that a row may be smaller than
                    // the expert's largest.  (Scales from the results' own maxima, one warp reduction for every 32 columns of a token:
                    // 4096 rows 406 -> 475 us.)
                    using Out = typename std::conditional<NP == 1, __half, float>::type;
                    Out* out = static_cast<Out*>(p.out) + size_t(tile.y + c0) * N + r * kRows + 32 * q + lane;
                    auto put = [&](int j) {
                        const float x = __fmul_rn(v[j], __fmul_rn(ir, f[c0 + j]));
                        if constexpr (NP == 1) out[size_t(j) * N] = __float2half_rn(__fmul_rn(x, f[128 + c0 + j]));
                        else out[size_t(j) * N] = x;
                    };
                    if (c0 + 16 <= real) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) put(j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c0 + j < real) put(j);
                    }
                }
            };
            // (after a timeout nothing is stored any more, but the barriers are kept)
            if constexpr (NP == 1) {
                epilogue_bar();                            // factors in place
                ok = ok && warp_wait(&d_full[td.s], td.full());
                if (it + step < items) factors(it + step, ahead);
                tc_fence_after();
                const uint32_t acc = taddr + td.s * dcols + (uint32_t(32 * q) << 16);
#pragma unroll 1
                for (int c0 = half * 16; c0 < real && ok; c0 += 32) {
                    float v[16];
                    tc_ld16(acc + uint32_t(c0), v);
                    finish(c0, v);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[td.s]);
                td.next(DB);
            } else {
                // the groups' sums
                constexpr int kSums = SETS == 3 ? 1 : kTileTokens<NP> / 32;
                float sum[kSums][16];
#pragma unroll
                for (int i = 0; i < kSums; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[i][j] = 0.f;
#pragma unroll 1
                for (int g = 0; g < G; g += 2) {
                    ok = ok && warp_wait(&d_full[td.s], td.full());
                    tc_fence_after();
                    const uint32_t acc = taddr + td.s * dcols + (uint32_t(32 * q) << 16);
#pragma unroll
                    for (int i = 0; i < kSums; ++i) {
                        const int c0 = i * 32 + half * 16;
                        if (c0 >= real || !ok) continue;
                        float v[16];
                        tc_ld16(acc + uint32_t(c0), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] = __fadd_rn(sum[i][j], v[j]);
                        if (g + 1 == G) continue;
                        tc_ld16(acc + (dcols >> 1) + uint32_t(c0), v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] = __fadd_rn(sum[i][j], v[j]);
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_empty[td.s]);
                    td.next(DB);
                }
                epilogue_bar();                            // factors in place
                if (it + step < items) factors(it + step, ahead);
                // (one copy of the code: the sums move down instead)
#pragma unroll 1
                for (int c0 = half * 16; c0 < real && ok; c0 += 32) {
                    finish(c0, sum[0]);
#pragma unroll
                    for (int i = 0; i + 1 < kSums; ++i)
#pragma unroll
                        for (int j = 0; j < 16; ++j) sum[i][j] = sum[i + 1][j];
                }
            }
            tile = ahead;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tc_dealloc(taddr, 512);
}

// ------------------------------------------------------------------ activations
// From gate_up's fp32 rows to down's operand: W warps (1, 2, 4 or 8) take a place's row, which they read once and hold.  4096 rows of
// 8 x 768: 30 us (150 MB, most of it L2: 5 TB/s); 1024 of 2 x 6144: 18.  (Four float4 a lane and twice the warps: 38 and 20; a bound
// of 48 or 40 registers spills.)
constexpr int kActThr = 256, kActPer = 8;                  // float4 of a lane: W x 1024 values of a row
template <int NP, int W>
__global__ void __launch_bounds__(kActThr) moe_act_kernel(const MoeTcParams p) {
    __shared__ float red[2][kActThr / 32];
    __shared__ __align__(16) __half sums[kActThr / 32 / W][W * kActPer * 4];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = warp / W, l = (warp % W) * 32 + lane;
    const int place = blockIdx.x * (kActThr / 32 / W) + row, K = p.w.I, K4 = K >> 2;
    const int at = place < p.T * p.k ? p.pos[place] : -1;
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(p.out) + size_t(max(at, 0)) * K);
    float4 v[kActPer];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kActPer; ++i) {
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (at >= 0 && l + i * W * 32 < K4) v[i] = __ldcs(src + l + i * W * 32);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(v[i].x), fabsf(v[i].y)), fmaxf(fabsf(v[i].z), fabsf(v[i].w))));
    }
    m = warp_max(m);
    if (W > 1) {
        if (lane == 0) red[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, red[0][row * W + w]);
    }
    float sig, isg;
    pow2_scale(__float_as_uint(m), sig, isg);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kActPer; ++i) {
        const int k4 = l + i * W * 32;
        if (at < 0 || k4 >= K4) break;                     // (whole warps: K4 is a multiple of 32)
        const float a[4] = {__fmul_rn(v[i].x, sig), __fmul_rn(v[i].y, sig), __fmul_rn(v[i].z, sig), __fmul_rn(v[i].w, sig)};
        uint2 out[NP];
        const float X = stage4<NP>(a, k4 & 3, out);
        if (NP == 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q) ss = __fmaf_rn(a[q], a[q], ss);
        }
        uint8_t* to = p.as + four_at(k4 * 4, at, NP, p.blocks);
#pragma unroll
        for (int q = 0; q < NP; ++q) *reinterpret_cast<uint2*>(to + q * p.blocks * 2048) = out[q];
        if ((lane & 15) == 0) put_sum(sums[row], k4 >> 4, X);
    }
    if (NP == 1) {
        ss = warp_sum(ss);
        if (W > 1 && lane == 0) red[1][warp] = ss;
    }
    if (W > 1) __syncthreads();
    else __syncwarp();
    if (at < 0) return;
    for (int pr = l; pr < pairs_of(K); pr += W * 32) store_sums(p.as, sums[row], pr, K, NP, p.blocks, at);
    if (l == 0) {
        p.isa[at] = isg;
        if (NP == 1) {
#pragma unroll
            for (int w = 1; w < W; ++w) ss = __fadd_rn(ss, red[1][row * W + w]);
            // the bound of the place's results: |act| |row| < 2^15 once scaled
            p.sout[at] = pow2(15 - (above(sqrtf(ss)) + above(isg) - 1 + above(p.norms[p.ids[place]])));
        }
    }
}

// ------------------------------------------------------------------ combine
// A CTA takes some columns of one token; rows of up to eight places are in flight.
constexpr int kCombineThr = 128;
template <bool BF16>
__global__ void __launch_bounds__(kCombineThr) moe_combine_kernel(const MoeTcParams p) {
    __shared__ int pos[kMoeMaxTopK];
    __shared__ float weight[kMoeMaxTopK], unscale[kMoeMaxTopK];
    constexpr int V = BF16 ? 8 : 4;                        // columns of a thread: 16 bytes of a row
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, H = p.w.H, h = (blockIdx.y * kCombineThr + threadIdx.x) * V;
    if (threadIdx.x < kMoeMaxTopK) {
        const int at = int(threadIdx.x) < p.k ? p.pos[size_t(t) * p.k + threadIdx.x] : -1;
        pos[threadIdx.x] = at;
        weight[threadIdx.x] = at >= 0 ? p.weights[size_t(t) * p.k + threadIdx.x] : 0.f;
        unscale[threadIdx.x] = BF16 && at >= 0 ? inverse_pow2(p.sout[at]) : 1.f;
    }
    __syncthreads();
    if (h >= H) return;
    float v[V];
#pragma unroll
    for (int c = 0; c < V; ++c) v[c] = 0.f;
    const size_t row = size_t(H) * (BF16 ? 2 : 4);
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        uint4 o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = j0 + j < kMoeMaxTopK ? pos[j0 + j] : -1;
            o[j] = at >= 0 ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.out) + at * row + size_t(h) * (16 / V)))
                           : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j >= kMoeMaxTopK || pos[j0 + j] < 0) continue;
            const float w = weight[j0 + j], u = unscale[j0 + j];
            const uint32_t a[4] = {o[j].x, o[j].y, o[j].z, o[j].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if constexpr (BF16) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a[c]));
                    v[2 * c] = __fmaf_rn(w, __fmul_rn(x.x, u), v[2 * c]);
                    v[2 * c + 1] = __fmaf_rn(w, __fmul_rn(x.y, u), v[2 * c + 1]);
                } else {
                    v[c] = __fmaf_rn(w, __uint_as_float(a[c]), v[c]);
                }
            }
        }
    }
    uint4* y = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + t * row + size_t(h) * (16 / V));
    uint32_t r[4] = {0u, 0u, 0u, 0u};
    if (p.resid) {
        const uint4 o = *y;
        r[0] = o.x;
        r[1] = o.y;
        r[2] = o.z;
        r[3] = o.w;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if constexpr (BF16) {
            if (p.resid) {
                v[2 * c] = __fadd_rn(bf16_lo(r[c]), v[2 * c]);
                v[2 * c + 1] = __fadd_rn(bf16_hi(r[c]), v[2 * c + 1]);
            }
            r[c] = pack_bf16x2(v[2 * c], v[2 * c + 1]);
        } else {
            r[c] = __float_as_uint(p.resid ? __fadd_rn(__uint_as_float(r[c]), v[c]) : v[c]);
        }
    }
    *y = make_uint4(r[0], r[1], r[2], r[3]);
}

const void* product_fn(bool bf16, bool gate, int cap) {
#define KMR_PRODUCT(np, gs, sets) (gate ? (const void*)moe_product_kernel<np, true, gs, sets> : (const void*)moe_product_kernel<np, false, gs, sets>)
    if (!bf16) return unpack_sets(cap, 2) == 3 ? KMR_PRODUCT(2, 2, 3) : KMR_PRODUCT(2, 2, 2);
    return stage_groups(cap) == 1 ? KMR_PRODUCT(1, 1, 2) : KMR_PRODUCT(1, 2, 3);
#undef KMR_PRODUCT
}

const void* stage_fn(bool bf16, int H) {
#define KMR_STAGE(n) \
    if (H <= n * kStageThr * 4) return bf16 ? (const void*)moe_stage_kernel<uint16_t, 1, n> : (const void*)moe_stage_kernel<float, 2, n>
    KMR_STAGE(1);
    KMR_STAGE(2);
    KMR_STAGE(4);
    KMR_STAGE(8);
#undef KMR_STAGE
    return nullptr;
}

// Warps to a row, and the kernel.
int act_warps(int I) { return I <= 1024 ? 1 : (I <= 2048 ? 2 : (I <= 4096 ? 4 : 8)); }
const void* act_fn(bool bf16, int I) {
#define KMR_ACT(w) \
    if (act_warps(I) == w) return bf16 ? (const void*)moe_act_kernel<1, w> : (const void*)moe_act_kernel<2, w>
    KMR_ACT(1);
    KMR_ACT(2);
    KMR_ACT(4);
    KMR_ACT(8);
#undef KMR_ACT
    return nullptr;
}

size_t up16(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

// Tokens of a tile: enough for most experts at once when the places are spread evenly; more of them mean longer waits for a stage's
// tokens.  By the mean of an expert's places (128 experts of 2048 x 768, us): fp32, 4: 16 tokens 99.6, 64 103.8; 8: 16 122, 32 115,
// 64 120; 14: 32 135, 64 142; 25: 32 164, 64 157.  bf16, 4: 16 86.7, 64 86.6; 16: 32 114, 64 108, 128 111; 32: 64 and 128 126; 48:
// 64 145, 128 136.
int moe_tc_cap(long long places, int E, bool bf16) {
    const long long mean = places / E;
    if (bf16) return mean <= 36 ? 64 : kTileTokens<1>;
    return mean <= 5 ? 16 : (mean <= 20 ? 32 : kTileTokens<2>);
}

MoeTcSizes moe_tc_sizes(const MoeView& w, bool bf16, int T, int k) {
    const int np = bf16 ? 1 : 2;
    const size_t S = size_t(T) * k, experts = S < size_t(w.E) ? S : size_t(w.E);
    const size_t P = (S + 15 * experts + 15) & ~size_t(15);
    MoeTcSizes z = {};
    z.tiles = 16;
    z.pos = z.tiles + (experts + P / 16) * 16;
    z.isx = z.pos + up16(S * 4);
    z.isa = z.isx + up16(P * 4);
    z.sout = z.isa + up16(P * 4);
    z.xs = z.sout + up16(P * 4);
    z.blocks = P / 8;
    z.as = z.xs + staged_bytes(w.H, np, P / 8);
    z.out = z.as + staged_bytes(w.I, np, P / 8);
    const size_t rows = size_t(w.H) * (bf16 ? 2 : 4), acts = size_t(w.I) * 4;      // (the activations are staged before the results come)
    z.total = z.out + P * (rows > acts ? rows : acts);
    return z;
}

cudaError_t launch_moe_tc(const MoeTcParams& p, bool bf16, int sms, cudaStream_t st) {
    const MoeTcParams* q = &p;
    cudaError_t e = launch_dependent((const void*)moe_plan_kernel, dim3(1), kPlanThr, 0, 1, q, st);
    if (e != cudaSuccess) return e;
    if ((e = launch_dependent(stage_fn(bf16, p.w.H), dim3(p.T), kStageThr, 0, 1, q, st)) != cudaSuccess) return e;
    const int threads = product_threads(unpack_sets(p.cap, bf16 ? 1 : 2)), rows = kActThr / 32 / act_warps(p.w.I);
    if ((e = launch_dependent(product_fn(bf16, true, p.cap), dim3(sms), threads, kSmem, 1, q, st)) != cudaSuccess) return e;
    if ((e = launch_dependent(act_fn(bf16, p.w.I), dim3((p.T * p.k + rows - 1) / rows), kActThr, 0, 1, q, st)) != cudaSuccess) return e;
    if ((e = launch_dependent(product_fn(bf16, false, p.cap), dim3(sms), threads, kSmem, 1, q, st)) != cudaSuccess) return e;
    const void* combine = bf16 ? (const void*)moe_combine_kernel<true> : (const void*)moe_combine_kernel<false>;
    const int cols = kCombineThr * (bf16 ? 8 : 4);
    return launch_dependent(combine, dim3(p.T, (p.w.H + cols - 1) / cols), kCombineThr, 0, 1, q, st);
}

cudaError_t launch_moe_factors(const MoeView& w, float* rho_gate_up, float* rho_down, float* norms, cudaStream_t st) {
    cudaError_t e = cudaMemsetAsync(norms, 0, size_t(w.E) * 4, st);
    if (e != cudaSuccess) return e;
    moe_factors_kernel<<<dim3((2 * w.I + 127) / 128, w.E), 128, 0, st>>>(w.gate_up, w.I / 8, w.H / 128, rho_gate_up, nullptr);
    moe_factors_kernel<<<dim3((w.H + 127) / 128, w.E), 128, 0, st>>>(w.down, w.H / 16, w.I / 128, rho_down, norms);
    return cudaGetLastError();
}

cudaError_t moe_tc_set_attributes() {
    cudaError_t e;
    for (int f = 0; f < 4; ++f)
        for (int gate = 0; gate < 2; ++gate) {
            const void* fn = product_fn(f > 1, gate != 0, f == 0 ? 32 : (f == 3 ? 128 : 64));
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
            if (e != cudaSuccess) return e;
        }
    const void* others[] = {(const void*)moe_plan_kernel, (const void*)moe_factors_kernel, stage_fn(true, 1024), stage_fn(true, 2048),
                            stage_fn(true, 4096), stage_fn(true, 8192), stage_fn(false, 1024), stage_fn(false, 2048),
                            stage_fn(false, 4096), stage_fn(false, 8192), act_fn(true, 1024), act_fn(true, 2048), act_fn(true, 4096),
                            act_fn(true, 8192), act_fn(false, 1024), act_fn(false, 2048), act_fn(false, 4096), act_fn(false, 8192),
                            (const void*)moe_combine_kernel<true>,
                            (const void*)moe_combine_kernel<false>};
    for (const void* fn : others) {
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, fn)) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kmr
