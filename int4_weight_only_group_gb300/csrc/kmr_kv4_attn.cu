// Decode attention of one token per row over the 4-bit KV cache (format: kmr_kv4.cuh).
//
// out = softmax(q K^T scale) V over positions 0..cache_position of the row's slot, and, where a mass
// is given, mass[slot][head][p] += the sum over the KV head's query heads of position p's weight.
// A (row, KV head) is cut into splits, whose softmax states (m, l, o) in base 2 merge in split order:
//   * caches of up to 2048 positions: one launch, the CTAs of a row's up to 8 splits are a thread-block cluster.  Each
//     pushes its states into the others' shared memory; after one cluster barrier each merges a slice of the output
//     and turns the scores of its own positions, kept in shared memory, into mass.  Of rows that share a slot the
//     first one's cluster takes all in turn, so that the mass gains them in row order.
//   * longer caches: up to 76 splits leave their states in the workspace (and, for the mass, every score); a
//     second launch, a programmatic dependent of the first, merges and adds, again in row order.
// One launch against two, 16/8 heads of 128, us: 5.6 / 5.6 (1 row of 1024), 6.0 / 8.1 (4 rows), 6.8 / 6.0 and 7.7 / 8.9 at
// 2048, 9.7 / 7.2 and 11.1 / 11.1 at 4096, where eight CTAs a head begin to be too few.
//
// The bound is HBM: 2 (d/2 + 4 d/g) bytes per position and KV head.  At d = 128, g = 32 an SM's share
// of the bandwidth is about 36 codes per cycle, too many for dequantising and multiplying on the CUDA
// cores, so both products run on the tensor cores, with the codes as the A operand.  mma m16n8k16 takes them from the
// registers in which a warp has unpacked them; a tcgen05 tile (128 positions as its rows, the heads' columns as N = 16)
// would be full as well, but wants the unpacked codes in shared or tensor memory first.  It has not been tried.
//   * a nibble c under the exponent of 1024 is the fp16 1024 + c (from bits 4..7: 1024 + 16 c); one packed fp16
//     operation takes the offset off again, exactly.  (As a bare subnormal c 2^-24 it would cost one operation
//     less, but a subnormal code was found to lose up to 10 of the accumulator's bits: outputs of a row of 8191
//     positions were off by 1e-4.)
//   * the other operand is fp32 split in two fp16 columns (high and low part, about 22 bits), so the result keeps
//     single precision: columns 2 h and 2 h + 1 belong to query head h and land in one lane's accumulators.
//   * scores: A = 16 positions x 16 dims, B = the query.  sum_j q_j (c_j s + z) = s sum q c + z sum q per group:
//     the group's accumulators are folded with its s and z and the query's group sum (fp32).
//   * output: A = 16 dims x 16 positions (two positions' units joined by a byte permute), B = weight times
//     the group's s, split in two.  The codes are taken as c - 8 at half of the positions and c - 7 at the
//     others (their mean is 7.5; fp16 has no 1031.5 to subtract), the base as z + 8 s or z + 7 s: a long
//     row's output is small against the codes' offset, and the sum of the offset codes would lose its bits (at
//     131072 positions an error of 5e-6 with c - 8 throughout).  The bases add per group in fp32.  The products
//     are scaled by a power of two per query head and group (fit_unit).
// Few query heads (rep <= 2) leave half of the columns empty.  With two groups or more the columns' halves then
// stand for the halves of the head's dims: column 4 f + 2 h + part is query head h in half f.  A step of the scores
// has 8 dims of either half (each half's columns are zero against the other's dims), a tile of the output 8
// dims of either half in its upper and lower rows.  The products are as many, but each lane folds, weighs and
// splits for its half's groups only: 413 instructions per tile of 16 positions at d = 128, g = 32 instead of 481 (one tile
// at a time; 392 now, two together).
//
// Measured, 16/8 heads of 128: 16 rows of 8192, group 32, 48.8 us (168 MB: 3.4 TB/s, 0.51 of the measured copy rate of 6.75); one
// row of 131072, 43.0 us (0.58), group 128, 39.2 us (143 MB, 0.54).  With the tiles' work left out the copies alone take 32 us
// for the long row (34 for 16 rows), with every row in L2 the 16 rows take 45.  No pipe is saturated (ALU 50% of the time, FMA
// 37%, tensor 21%): leaving the V codes' unpacking out gains 5.8 us of the long row's, the weights' splitting 1.3, the
// bases' sum and the shuffles 0.9 each, the K codes' unpacking 0.6, the products nothing.  Registers are at the 128 that
// four CTAs an SM allow; heads of 128 in groups of 32 with 3 or more query heads a KV head spill 12 to 80 bytes.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kmr_kv4.cuh"

namespace cg = cooperative_groups;

namespace kmr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThr = 128, kWarps = 4;
constexpr int kMergeThr = 256;

// KMR_OK, the row's error, or kEmptyRow: nothing to attend, which is no error.
constexpr int kEmptyRow = 1;
__device__ __forceinline__ int kv4_row_error(const Kv4AttnParams& p, int b) {
    const int slot = p.slot_ids[b], cp = p.cpos[b];
    if (cp == -1) return kEmptyRow;
    if (slot < 0 || slot >= p.c.slots) return KMR_ERR_SLOT_RANGE;
    return (cp < 0 || cp >= p.c.S) ? KMR_ERR_CACHE_FULL : KMR_OK;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// fp16 pair (low half a, high half b), rounded towards zero.
__device__ __forceinline__ uint32_t pack_f16_rz(float a, float b) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// The high part of x (mask 0: x itself, which the cut to fp16 shortens to its leading 11 significant bits) or its
// low part (mask 0xFFFFE000: what that cut leaves).
__device__ __forceinline__ float part_of(float x, uint32_t mask) {
    return __fsub_rn(x, __uint_as_float(__float_as_uint(x) & mask));
}
// The scale of a word times a power of two, which as a pair of bf16 is (0, itself): one operation instead of taking the
// base off and multiplying.  The sum with zero keeps a negative base from leaving -0 in the low half.
__device__ __forceinline__ float scaled_s(uint32_t word, float unit) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(word), "r"(__float_as_uint(unit)), "r"(0u));
    return __uint_as_float(r);
}
// The four codes of each half of a word as fp16 pairs c - OFF: nibbles (0, 4), (1, 5), (2, 6), (3, 7).
template <int OFF>
__device__ __forceinline__ void unpack_codes(uint32_t w, uint32_t (&c)[4]) {
    const __half2 low = __float2half2_rn(-1024.f - OFF), high = __float2half2_rn(-64.f - OFF);
    const __half2 sixteenth = __float2half2_rn(0.0625f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t a = and_or(w, 0x000F000Fu, 0x64006400u), b = and_or(w, 0x00F000F0u, 0x64006400u);
        const __half2 x = __hadd2(*reinterpret_cast<__half2*>(&a), low);
        const __half2 y = __hfma2(*reinterpret_cast<__half2*>(&b), sixteenth, high);
        c[2 * i] = *reinterpret_cast<const uint32_t*>(&x);
        c[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&y);
        w >>= 8;
    }
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ float exp2_approx(float x) {               // 2 ulp; 0 below 2^-126
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <int N>
__device__ __forceinline__ void lds_words(const void* p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 u = *static_cast<const uint4*>(p);
        w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else if constexpr (N == 2) {
        const uint2 u = *static_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
    } else {
        w[0] = *static_cast<const uint32_t*>(p);
    }
}

// How a CTA's four warps share the work.  Two tiles of 16 positions a warp at a time give two chains of products to
// interleave (when taken, one row of 8192: 9.1 -> 8.0 us; 16 rows 53.4 -> 47.4).  Up to 4 query heads a KV head fill one n-tile.  5 to 8
// need two: with heads of 64 every warp keeps both; with heads of 128 that takes 240 registers and two CTAs an SM, so
// warps 0, 1 have the first four heads and warps 2, 3 the others, over the same stage, and unpack it twice (16 rows of
// 8192, group 32, when taken: 8 heads on each of 4 KV heads 55.9 -> 48.6 us, 6 on each of 8 101 -> 87; one row of 4096 9.5 -> 10.3;
// now 49.6 and 89).
enum HeadClass { HEADS_2 = 0, HEADS_4 = 1, HEADS_8 = 2 };
template <int D, int HC>
struct Share {
    static constexpr int kHeadWarps = HC == HEADS_8 && D == 128 ? 2 : 1;       // groups of warps with heads of their own
    static constexpr int kTileWarps = kWarps / kHeadWarps;                     // warps that share out the tiles
    static constexpr int kNTiles = HC == HEADS_8 && D == 64 ? 2 : 1;           // n-tiles of a warp
    static constexpr int kTiles = 2;                                           // tiles of a warp at a time
    static constexpr int kCtas = kNTiles == 1 ? 4 : 3;                         // of an SM
};
template <int D, int G, int HC>
struct SplitSmem {
    using S = Share<D, HC>;
    static constexpr int kStagePos = 16 * S::kTileWarps * S::kTiles, kStages = 256 / kStagePos;
    static constexpr int kCodes = kStagePos * D / 2, kWords = kStagePos * (D / G) * 4;
    static constexpr int kStage = 2 * kCodes + 2 * kWords;
    static constexpr int kRing = kStages * kStage;
    __host__ __device__ static constexpr int merge(int rep) { return S::kTileWarps * rep * (D + 2) * 4; }
    static constexpr int kQuery = 4 * (D / 32) + 2 * (D / G);         // words of a lane's query per n-tile
    static constexpr int kQueryBytes = S::kHeadWarps * S::kNTiles * kQuery * 128;
    __host__ __device__ static constexpr int base(int rep) { return 128 + kQueryBytes + kRing + merge(rep); }
    // a cluster's additions: the states pushed here (a slice of o of every split; every m and l), the scores
    __host__ __device__ static constexpr int state(int rep, int ranks) {
        return kKv4ClusterSplits * (rep * D / ranks * 4 + rep * 8);
    }
    __host__ __device__ static constexpr int total(int rep, int ranks, int positions) {
        return base(rep) + state(rep, ranks) + rep * positions * 4;
    }
};

// Query head, half of the dims and part (0 high, 1 low) of an n-tile's column.
template <bool PAIR>
__device__ __forceinline__ int column_head(int g) { return PAIR ? (g >> 1) & 1 : g >> 1; }
template <bool PAIR>
__device__ __forceinline__ int column_half(int g) { return PAIR ? g >> 2 : 0; }

// The scaling of the output's weights times scales: a power of two from 2^-126 to 2^126 for each query head and group, so that
// neither a group beside others of far larger values nor a position of large values and no weight costs bits.  A product
// has to stay below 2^15 (fp16); its two parts hold 22 bits of it from 2^-2 on, and 2^-24 below.
//   * The scaling goes by the largest scale seen, brought to [2^kTop, 2^(kTop + 1)): weights are at most 2^kLag, so scales up
//     to twice as large (limit_of) need no look at the weights.
//   * Where that leaves the tiles' largest product below kEnough (what a long row's products lose below 2^-24 would begin to
//     show), because the large scale has no weight, the scaling goes by the product, brought to [2^7, 2^8).  Tiles with a
//     scale that may be too large are then looked at each (16 rows of 8192 whose V scales differ by up to 2^20 from
//     position to position: 48.8 -> 52.6 us).
//   * As the reference rises by `oct` whole octaves, what was added before falls by as much, and the scaling may rise by it.
// One scaling for all groups, as it was, kept 22 bits of the largest group only: beside one 10^4 (10^6) times larger
// a group was off by 3e-4 (2e-2).  This costs 0 to 2% (16 rows of 8192, group 32: 47.7 -> 48.7 us, 8 query heads a KV head 48.5 ->
// 48.7; one row of 131072, group 128: 38.5 -> 39.4); checking the products themselves in every tile cost 4 to 9%.
constexpr int kLag = 8, kTop = 13 - kLag;
constexpr float kEnough = 2.f;
__device__ __forceinline__ int unit_exponent(float u) { return int(__float_as_uint(u) >> 23); }
// The scaling that brings x to [2^top, 2^(top + 1)).
__device__ __forceinline__ float unit_for(float x, int top) {
    return __uint_as_float(uint32_t(min(max(254 + top - unit_exponent(x), 1), 253)) << 23);
}
__device__ __forceinline__ float fit_unit(float was, float smax, float pmax, float oct, bool first) {
    const float by_scale = unit_for(smax, kTop);
    // (at most 2^126 / smax: a weight of 0 times an infinity would be no number)
    const float cap = by_scale < 0x1p10f ? by_scale * 0x1p116f : 0x1p126f, by_product = fminf(unit_for(pmax, 7), cap);
    const bool enough = pmax * by_scale >= kEnough || pmax == 0.f;
    const float target = enough ? by_scale : by_product;
    if (first || (enough && smax * was >= float(1 << (kTop + 2)))) return target;
    if (pmax * was >= 0x1p15f) return by_product;
    was = fminf(was, cap);
    return pmax * was < kEnough ? fmaxf(was, fminf(target, was * exp2f(oct))) : was;
}
// Scales from here on (as bits) may be too large for a scaling: 2^(kTop + 2) / it.
__device__ __forceinline__ uint32_t limit_of(float u) { return uint32_t(min(256 + kTop - unit_exponent(u), 255)) << 23; }
// The largest over the lanes of one t, which hold the tile's rows.
__device__ __forceinline__ float max_over_rows(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}

// Query fragments of the scores' B operand (this lane's column), and the queries' group sums and factors of the head and
// half whose accumulators the lane holds (columns 2 t, 2 t + 1).  A head's query is scaled by a power of two per group, so that
// a group keeps its 22 bits beside others of far larger queries (with one for all, a K group 10^8 times larger where the
// query is as much smaller put outputs off by 1e-3); the group's s takes it back.  Heads from head0 on; past rep, zero.
template <int D, int G, int NT, bool PAIR>
__device__ __forceinline__ void query_fragments(const Kv4AttnParams& p, int b, int h, int rep, int head0, int lane,
                                                uint32_t* out) {
    constexpr int NB = D / 32 / (PAIR ? 2 : 1), NG = D / G / (PAIR ? 2 : 1), BPG = G / 32;     // of one half
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int hq = head0 + 4 * n + column_head<PAIR>(g);
        float x[NB][8], mx[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) mx[i] = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
            if (hq < rep) {
                const float4* src = reinterpret_cast<const float4*>(p.q + (size_t(b) * p.nq + h * rep + hq) * D +
                                                                    32 * (k + NB * column_half<PAIR>(g)) + 8 * t);
                u = src[0];
                v = src[1];
            }
            x[k][0] = u.x; x[k][1] = u.y; x[k][2] = u.z; x[k][3] = u.w;
            x[k][4] = v.x; x[k][5] = v.y; x[k][6] = v.z; x[k][7] = v.w;
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[k / BPG] = fmaxf(mx[k / BPG], fabsf(x[k][e]));
        }
        // each group's largest |q| sigma in [2^13, 2^14): sigma = 2^(13 - e), held within the normal range
        float gs[NG], sig[NG];
        uint32_t ex[NG];                                              // 2^e
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            const uint32_t e = max(__float_as_uint(mx[i]) >> 23, 14u);
            ex[i] = e << 23;
            sig[i] = __uint_as_float((267u - e) << 23);
            gs[i] = 0.f;
        }
        const uint32_t mask = (g & 1) ? 0xFFFFE000u : 0u;
        uint32_t* at = out + n * (4 * NB + 2 * NG) * 32 + lane;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                gs[k / BPG] += x[k][i];
                y[i] = part_of(x[k][i] * sig[k / BPG], mask);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) at[(4 * k + i) * 32] = pack_f16_rz(y[i], y[i + 4]);
        }
        const float base2 = p.scale * kLog2e;
        // columns 2 t, 2 t + 1 are lane 8 t's
#pragma unroll
        for (int i = 0; i < NG; ++i) {
            float v = gs[i];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            at[(4 * NB + i) * 32] = __float_as_uint(__shfl_sync(0xffffffffu, v * base2, 8 * t));
            at[(4 * NB + NG + i) * 32] = __shfl_sync(0xffffffffu, ex[i], 8 * t);
        }
    }
}

// One CTA of four warps, a ring of stages of 16 TT positions a warp filled by bulk copies (four lanes, one array each).
// A stage's four warps meet only at its barriers; a row's last tile masks by select, since what lies past the row's end
// may be NaN.  HC: the most query heads a KV head; with 2 and several groups the halves' groups are kept apart (PAIR,
// see above).
template <int D, int G, int HC, bool CL>
__global__ void __launch_bounds__(kThr, Share<D, HC>::kCtas) kv4_split_kernel(const Kv4AttnParams p) {
    using M = SplitSmem<D, G, HC>;
    using S = Share<D, HC>;
    constexpr int TT = S::kTiles, NT = S::kNTiles, kTileWarps = S::kTileWarps, kHeadWarps = S::kHeadWarps;
    constexpr bool PAIR = HC == HEADS_2 && G < D;
    constexpr int kStagePos = M::kStagePos, kStages = M::kStages;
    constexpr int NB = D / 32, NG = D / G, BPG = G / 32;
    constexpr int HB = PAIR ? NB / 2 : NB, HG = PAIR ? NG / 2 : NG;  // blocks and groups of a lane's half
    static_assert(!PAIR || (NT == 1 && NG >= 2), "two halves of whole groups");
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);              // [kStages]
    uint64_t* empty = full + kStages;                                // [kStages]
    uint8_t* ring = smem + 128 + M::kQueryBytes;
    const int s = blockIdx.x, h = blockIdx.y, b0 = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();                                   // nothing of the previous kernel's is read before
    if (!CL) pdl_launch_dependents();             // the merge, which waits for this kernel's end
    const int rep = p.nq / p.c.nkv;
    // warp 1 (and 2, for the second group of heads) prepares the query for all while warp 0 looks up the row and starts
    // its copies
    constexpr int kQueryWords = (4 * HB + 2 * HG) * 32;              // of an n-tile
    uint32_t* qsh = reinterpret_cast<uint32_t*>(smem + 128);         // [head group][n-tile][value][lane]
    // four groups' factors of the query are read from there each time where two warps have heads of their own (16 rows of
    // 8192, 6 heads a KV head: 89.2 us against 90.4 with them in registers; up to 4 heads, 4 KV heads: 32.8 against 32.3)
    constexpr bool kSharedExps = HG == 4 && kHeadWarps > 1;
    const int hw = warp / kTileWarps, wt = warp % kTileWarps, head0 = 4 * NT * hw;
    auto prepare_query = [&](int b) {
        if (warp >= 1 && warp <= kHeadWarps)
            query_fragments<D, G, NT, PAIR>(p, b, h, rep, 4 * NT * (warp - 1), lane, qsh + (warp - 1) * NT * kQueryWords);
    };
    prepare_query(b0);
    const int bad = kv4_row_error(p, b0);
    if (bad != KMR_OK) {                          // the same for the whole cluster
        if (CL && s == 0) {
            if (tid == 0 && h == 0 && bad != kEmptyRow) set_error(p.err, bad);
            for (int i = tid; i < rep * D; i += kThr) p.out[(size_t(b0) * p.nq + h * rep) * D + i] = 0.f;
        }
        return;
    }
    const int slot = p.slot_ids[b0];
    const size_t row = (size_t(slot) * p.c.nkv + h) * p.c.S;
    if (CL && p.mass) {
        // rows that share a slot belong to the first one's cluster
        int before = 0;
        for (int r = tid; r < b0; r += kThr) before |= p.slot_ids[r] == slot && kv4_row_error(p, r) == KMR_OK;
        if (__syncthreads_or(before)) return;
    }
    if (CL) cluster_arrive();                     // waited for before the first push: the others have started
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        fence_mbar_init();
    }
    __syncwarp();                                 // the other warps see the barriers after the first block barrier
    const int cgh = column_half<PAIR>(g), cth = PAIR ? t >> 1 : 0;   // halves of the lane's column and accumulators
    const uint32_t wmask = (g & 1) ? 0xFFFFE000u : 0u;
    uint32_t uses = 0;                            // stages filled so far: stage k of them was use k / kStages of its buffer
    bool first = true;
    // a lane looks through words of V of one position of a tile: of one group, or (d / g = 4) of two
    constexpr int kLook = (NG + 1) / 2;
    const int look_row = NG == 1 ? (lane & 15) : lane >> 1;
    auto look = [&](const uint8_t* buf, int i0, uint32_t (&mine)[kLook]) {
        lds_words(buf + 2 * M::kCodes + M::kWords + i0 * (4 * NG) + (NG == 1 ? 4 * look_row : lane * (2 * NG)), mine);
    };

    for (int b = b0; b < p.B; ++b) {
        if (CL && b != b0 && (!p.mass || p.slot_ids[b] != slot || kv4_row_error(p, b) != KMR_OK)) continue;
        const int L = p.cpos[b] + 1;
        int chunk, ns;
        if (CL)
            kv4_cluster_plan(L, chunk, ns);
        else
            kv4_split_plan(L, chunk, ns);
        // this CTA's splits, and the stages of all of them (a cluster's spare CTAs have none); one, beyond a cluster
        const int u0 = CL ? s * p.per : s, u1 = CL ? min(ns, u0 + p.per) : s + 1;
        if (!CL && u0 >= ns) return;
        const int end = min(L, u1 * chunk), per_split = (chunk + kStagePos - 1) / kStagePos;
        const int nst = u0 < u1 ? (u1 - u0 - 1) * per_split + (end - (u1 - 1) * chunk + kStagePos - 1) / kStagePos : 0;
        if (CL && !first) {
            cluster_arrive();
            cluster_wait();                           // what the last row pushed has been read, and the ring
            fence_proxy_async_smem();
        }

        // One stage: lanes 0..3 of the calling warp copy K codes, V codes, K words and V words of up to
        // kStagePos positions (rounded up to 16: within the row, whose length is a multiple of 16).
        auto issue = [&](int k) {
            const uint32_t slot_of = (uses + k) % kStages;
            uint8_t* buf = ring + slot_of * M::kStage;
            const int split0 = CL ? (u0 + k / per_split) * chunk : u0 * chunk;
            const int pa = split0 + (CL ? k % per_split : k) * kStagePos;
            const uint32_t np = uint32_t(min(kStagePos, (min(L, split0 + chunk) - pa + 15) & ~15));
            if (lane == 0) mbar_arrive_expect_tx(&full[slot_of], np * (D + 8 * NG));
            __syncwarp();
            if (lane < 4) {
                const bool words = lane >= 2, key = !(lane & 1);
                const void* src = words ? static_cast<const void*>((key ? p.c.ks : p.c.vs) + (row + pa) * NG)
                                        : static_cast<const void*>((key ? p.c.kc : p.c.vc) + (row + pa) * (D / 2));
                uint8_t* dst = buf + (words ? 2 * M::kCodes + (key ? 0 : M::kWords) : (key ? 0 : M::kCodes));
                bulk_g2s(dst, src, np * (words ? 4 * NG : D / 2), &full[slot_of]);
            }
            __syncwarp();
        };
        if (warp == 0)
            for (int i = 0; i < nst && i < kStages; ++i) issue(i);

        if (CL && !first) prepare_query(b);
        __syncthreads();
        uint32_t qf[NT][NB][4];                       // PAIR: [half][block of the half], zero for the other half
        float qsum[NT][HG], qex[NT][HG];
        const float unscore = p.scale * kLog2e * 0x1p-13f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint32_t* at = qsh + (hw * NT + n) * kQueryWords + lane;
#pragma unroll
            for (int k = 0; k < HB; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t v = at[(4 * k + i) * 32];
                    if constexpr (PAIR) {
                        qf[n][k][i] = cgh ? 0u : v;
                        qf[n][k + HB][i] = cgh ? v : 0u;
                    } else {
                        qf[n][k][i] = v;
                    }
                }
#pragma unroll
            for (int i = 0; i < HG; ++i) {
                qsum[n][i] = __uint_as_float(at[(4 * HB + i) * 32]);
                if constexpr (!kSharedExps) qex[n][i] = __uint_as_float(at[(4 * HB + HG + i) * 32]);
            }
        }

        // base-2 scores for the mass: [head][position], in shared memory from the CTA's first position on
        float* sc_out = nullptr;
        size_t sc_ld = p.c.S;
        if (CL && p.mass) {
            sc_ld = p.score_ld;
            sc_out = reinterpret_cast<float*>(smem + M::base(rep) + M::state(rep, int(gridDim.x))) - u0 * chunk;
        } else if (!CL && p.scores) {
            sc_out = p.scores + (size_t(b) * p.c.nkv + h) * rep * p.c.S;
        }

        float* wo = reinterpret_cast<float*>(ring + M::kRing);           // [warp of a head][rep][D]
        float* wml = wo + kTileWarps * rep * D;                          // [warp][rep][2]
        const int ranks = CL ? int(gridDim.x) : 1, slice = rep * D / ranks;         // of the output, for each rank
        float* recv = reinterpret_cast<float*>(smem + M::base(rep));                 // [split][slice]
        float* recv_ml = recv + kKv4ClusterSplits * slice;                           // [split][head][m, l]
        int k = 0;                                    // stage of the CTA
        for (int u = u0; u < u1; ++u) {
            const int t0 = u * chunk, t1 = min(L, t0 + chunk);
            float m[NT], l[NT], o[NT][2 * NB][4], zo[NT][HG];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                m[n] = -INFINITY;
                l[n] = 0.f;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
#pragma unroll
                for (int i = 0; i < HG; ++i) zo[n][i] = 0.f;
            }
            // the column's scaling in each of its groups, and the smallest V scale (as bits) of the groups whose words the
            // lane looks through that may be too large for it: both set by the first tiles
            float unit[NT][HG];
            uint32_t limit[kLook];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < HG; ++i) unit[n][i] = 1.f;
#pragma unroll
            for (int i = 0; i < kLook; ++i) limit[i] = 0u;
            for (int st = 0; t0 + st * kStagePos < t1; ++st, ++k) {
                const uint32_t slot_of = (uses + k) % kStages, phase = ((uses + k) / kStages) & 1u;
                const uint8_t* buf = ring + slot_of * M::kStage;
                mbar_wait(&full[slot_of], phase, p.err);
                const int base0 = t0 + st * kStagePos + wt * 16;         // the first tile's first position
                if (base0 < t1) {
                    // a tile is whole but for the row's last ones; one past the end counts for nothing
                    const bool whole = base0 + (TT - 1) * (16 * kTileWarps) + 16 <= t1;
                    // ---- scores of positions g and g + 8 of each tile for head 4 n + t, and the largest scales of the tiles' V
                    float sc[TT][NT][2];
                    uint32_t top[kLook] = {};
#pragma unroll
                    for (int u = 0; u < TT; ++u) {
                        const int i0 = (u * kTileWarps + wt) * 16, base = base0 + u * (16 * kTileWarps);
                        uint32_t k0[NB], k1[NB], w0[HG], w1[HG];
                        lds_words(buf + (i0 + g) * (D / 2) + t * (4 * NB), k0);
                        lds_words(buf + (i0 + g + 8) * (D / 2) + t * (4 * NB), k1);
                        lds_words(buf + 2 * M::kCodes + (i0 + g) * (4 * NG) + cth * (4 * HG), w0);
                        lds_words(buf + 2 * M::kCodes + (i0 + g + 8) * (4 * NG) + cth * (4 * HG), w1);
                        float zc[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n) sc[u][n][0] = sc[u][n][1] = zc[n][0] = zc[n][1] = 0.f;
#pragma unroll
                        for (int gr = 0; gr < HG; ++gr) {
                            float acc[NT][4];
#pragma unroll
                            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
                            for (int kb = 0; kb < BPG; ++kb) {
                                const int k = gr * BPG + kb;
                                uint32_t x[4], y[4];
                                unpack_codes<0>(k0[k], x);
                                unpack_codes<0>(k1[k], y);
                                if constexpr (PAIR) {
                                    uint32_t xh[4], yh[4];
                                    unpack_codes<0>(k0[k + HB], xh);
                                    unpack_codes<0>(k1[k + HB], yh);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        mma_f16(acc[0], x[i], y[i], xh[i], yh[i], qf[0][k][i], qf[0][k + HB][i]);
                                } else {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        mma_f16(acc[n], x[0], y[0], x[1], y[1], qf[n][k][0], qf[n][k][1]);
                                        mma_f16(acc[n], x[2], y[2], x[3], y[3], qf[n][k][2], qf[n][k][3]);
                                    }
                                }
                            }
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const float ex = kSharedExps ? __uint_as_float(qsh[(hw * NT + n) * kQueryWords + lane + (4 * HB + HG + gr) * 32])
                                                             : qex[n][gr];
                                sc[u][n][0] = __fmaf_rn(scaled_s(w0[gr], ex), acc[n][0] + acc[n][1], sc[u][n][0]);
                                sc[u][n][1] = __fmaf_rn(scaled_s(w1[gr], ex), acc[n][2] + acc[n][3], sc[u][n][1]);
                                zc[n][0] = __fmaf_rn(kv4_z(w0[gr]), qsum[n][gr], zc[n][0]);
                                zc[n][1] = __fmaf_rn(kv4_z(w1[gr]), qsum[n][gr], zc[n][1]);
                            }
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            sc[u][n][0] = __fmaf_rn(sc[u][n][0], unscore, zc[n][0]);
                            sc[u][n][1] = __fmaf_rn(sc[u][n][1], unscore, zc[n][1]);
                            if constexpr (PAIR) {
                                // the other half's part is two lanes away; both lanes add the same two numbers
                                sc[u][n][0] += __shfl_xor_sync(0xffffffffu, sc[u][n][0], 2);
                                sc[u][n][1] += __shfl_xor_sync(0xffffffffu, sc[u][n][1], 2);
                            }
                            if (!whole) {
                                if (base + g >= t1) sc[u][n][0] = -INFINITY;
                                if (base + g + 8 >= t1) sc[u][n][1] = -INFINITY;
                            }
                            const int hq = head0 + 4 * n + t;           // (PAIR: rep <= 2, the lanes of half 0)
                            if (sc_out && hq < rep) {
                                float* dst = sc_out + hq * sc_ld + base + g;
                                if (whole || base + g < t1) dst[0] = sc[u][n][0];
                                if (whole || base + g + 8 < t1) dst[8] = sc[u][n][1];
                            }
                        }
                        uint32_t mine[kLook];
                        look(buf, i0, mine);
                        if (whole || base + look_row < t1) {
#pragma unroll
                            for (int i = 0; i < kLook; ++i) top[i] = max(top[i], mine[i] & 0x7FFFFFFFu);
                        }
                    }
                    // ---- running reference of the weights, 2^(score - m): it follows the maximum once that is kLag octaves above,
                    // so that most tiles change neither it nor the scaling; weights stay below 2^kLag
                    float mn[NT];
                    bool over = false;
#pragma unroll
                    for (int i = 0; i < kLook; ++i) over |= top[i] >= limit[i];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c = fmaxf(sc[0][n][0], sc[0][n][1]);
                        c = fmaxf(c, fmaxf(sc[TT - 1][n][0], sc[TT - 1][n][1]));
                        c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 4));
                        c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 8));
                        c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, 16));
                        mn[n] = c > m[n] + float(kLag) ? c : m[n];
                        over |= mn[n] != m[n];
                    }
                    if (st == 0) {
                        // where every scale is 2^-4 of its group's largest or more, so is that of each head's best position, whose
                        // weight is 1: the scaling goes by the scales
                        float by_scale[NG];
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) {
                            const uint32_t v = NG == 1 || (lane & 1) == gr / kLook ? top[gr % kLook] : 0u;
                            by_scale[gr] = unit_for(__uint_as_float(__reduce_max_sync(0xffffffffu, v)), kTop);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int gr = 0; gr < HG; ++gr) unit[n][gr] = cgh ? by_scale[NG - HG + gr] : by_scale[gr];
                        over = false;
#pragma unroll
                        for (int i = 0; i < kLook; ++i) limit[i] = limit_of(NG > 1 && (lane & 1) ? by_scale[NG - kLook + i] : by_scale[i]);
#pragma unroll
                        for (int u = 0; u < TT; ++u) {
                            uint32_t mine[kLook];
                            look(buf, (u * kTileWarps + wt) * 16, mine);
#pragma unroll
                            for (int i = 0; i < kLook; ++i)
                                over |= (whole || base0 + u * (16 * kTileWarps) + look_row < t1) &&
                                        (mine[i] & 0x7FFFFFFFu) + (uint32_t(kTop + 1) << 23) < limit[i];
                        }
                    }
                    if (__builtin_expect(__any_sync(0xffffffffu, over), 0)) {
                        // the tiles' largest scale, and largest weight times scale of the lane's head, in each group
                        float smax[HG], pmax[NT][HG];
#pragma unroll
                        for (int gr = 0; gr < HG; ++gr) {
                            smax[gr] = 0.f;
#pragma unroll
                            for (int n = 0; n < NT; ++n) pmax[n][gr] = 0.f;
                        }
#pragma unroll
                        for (int u = 0; u < TT; ++u) {
                            const int i0 = (u * kTileWarps + wt) * 16, base = base0 + u * (16 * kTileWarps);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t v[HG];
                                lds_words(buf + 2 * M::kCodes + M::kWords + (i0 + g + 8 * e) * (4 * NG) + cth * (4 * HG), v);
#pragma unroll
                                for (int gr = 0; gr < HG; ++gr) {
                                    const float vs = base + g + 8 * e < t1 ? fabsf(kv4_s(v[gr])) : 0.f;
                                    smax[gr] = fmaxf(smax[gr], vs);
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        const float mm = mn[n] == -INFINITY ? 0.f : mn[n];
                                        pmax[n][gr] = fmaxf(pmax[n][gr], exp2_approx(__fsub_rn(sc[u][n][e], mm)) * vs);
                                    }
                                }
                            }
                        }
                        float most[HG];                              // largest scaling of any head
#pragma unroll
                        for (int gr = 0; gr < HG; ++gr) {
                            smax[gr] = max_over_rows(smax[gr]);
                            most[gr] = 0.f;
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const bool same = mn[n] == m[n];
                            const float fall = same ? 0.f : mn[n] - m[n], oct = same ? 0.f : floorf(mn[n]) - floorf(m[n]);
                            const float cf = exp2_approx(-fall);
                            l[n] *= cf;
#pragma unroll
                            for (int gr = 0; gr < HG; ++gr) {
                                const float was = __shfl_sync(0xffffffffu, unit[n][gr], 8 * t);      // column 2 t's
                                const float now = fit_unit(was, smax[gr], max_over_rows(pmax[n][gr]), oct, st == 0);
                                const float ce = exp2_approx(float(unit_exponent(now) - unit_exponent(was)) - fall);
                                zo[n][gr] *= cf;
                                constexpr int kEach = 2 * NB / HG;
#pragma unroll
                                for (int i = 0; i < kEach; ++i)
#pragma unroll
                                    for (int c = 0; c < 4; ++c) o[n][gr * kEach + i][c] *= ce;
                                most[gr] = fmaxf(most[gr], now);
                                unit[n][gr] = __shfl_sync(0xffffffffu, now, 2 * cgh + column_head<PAIR>(g));
                            }
                        }
                        uint32_t lim[HG];
#pragma unroll
                        for (int gr = 0; gr < HG; ++gr) {
                            most[gr] = fmaxf(most[gr], __shfl_xor_sync(0xffffffffu, most[gr], 1));
                            if (!PAIR) most[gr] = fmaxf(most[gr], __shfl_xor_sync(0xffffffffu, most[gr], 2));
                            lim[gr] = limit_of(most[gr]);
                        }
#pragma unroll
                        for (int i = 0; i < kLook; ++i) {
                            if constexpr (PAIR)
                                limit[i] = __shfl_sync(0xffffffffu, lim[i], 2 * (lane & 1));
                            else if constexpr (NG == 1)
                                limit[i] = lim[0];
                            else
                                limit[i] = (lane & 1) ? lim[NG / 2 + i] : lim[i];
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) m[n] = mn[n];
#pragma unroll
                    for (int u = 0; u < TT; ++u) {
                        const int i0 = (u * kTileWarps + wt) * 16, base = base0 + u * (16 * kTileWarps);
                        // ---- V words of positions g, g + 8 (the bases' sum) and t, t + 4, t + 8, t + 12 (the weights)
                        const uint8_t* words = buf + 2 * M::kCodes + M::kWords + i0 * (4 * NG);
                        uint32_t v0[HG], v1[HG], vw[4][HG];
                        lds_words(words + g * (4 * NG) + cth * (4 * HG), v0);
                        lds_words(words + (g + 8) * (4 * NG) + cth * (4 * HG), v1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) lds_words(words + (t + 4 * i) * (4 * NG) + cgh * (4 * HG), vw[i]);
                        if (!whole) {
                            // past the row's end the words are leftovers, and may be NaN: weight 0 would not hide that
#pragma unroll
                            for (int gr = 0; gr < HG; ++gr) {
                                if (base + g >= t1) v0[gr] = 0u;
                                if (base + g + 8 >= t1) v1[gr] = 0u;
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (base + t + 4 * i >= t1) vw[i][gr] = 0u;
                            }
                        }
                        // ---- weights of head 4 n + t at positions g, g + 8 and what the bases add; then of the lane's column's head at
                        // the lane's four positions
                        float w[NT][4];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const float mm = m[n] == -INFINITY ? 0.f : m[n];
                            const float p0 = exp2_approx(__fsub_rn(sc[u][n][0], mm)), p1 = exp2_approx(__fsub_rn(sc[u][n][1], mm));
                            l[n] += p0 + p1;
#pragma unroll
                            for (int gr = 0; gr < HG; ++gr) {
                                zo[n][gr] = __fmaf_rn(p0, __fmaf_rn(8.f, kv4_s(v0[gr]), kv4_z(v0[gr])), zo[n][gr]);
                                zo[n][gr] = __fmaf_rn(p1, __fmaf_rn(7.f, kv4_s(v1[gr]), kv4_z(v1[gr])), zo[n][gr]);
                            }
                            const int src = 4 * t + column_head<PAIR>(g);
                            w[n][0] = __shfl_sync(0xffffffffu, p0, src);
                            w[n][1] = __shfl_sync(0xffffffffu, p0, src + 16);
                            w[n][2] = __shfl_sync(0xffffffffu, p1, src);
                            w[n][3] = __shfl_sync(0xffffffffu, p1, src + 16);
                        }
                        // ---- output: dims 32 k + 4 g + j in rows g (j = 0, 2) and g + 8 (j = 1, 3); PAIR: dims 32 k + 4 g + j
                        // of half 0 in rows g, of half 1 in rows g + 8
                        uint32_t vc[4][NB / 2];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            lds_words(buf + M::kCodes + (i0 + t + 4 * i) * (D / 2) + g * (2 * NB), vc[i]);
                        auto unpack_block = [&](int k, uint32_t (&x)[4], uint32_t (&y)[4]) {
                            const uint32_t sel = (k & 1) ? 0x7632u : 0x5410u;
                            unpack_codes<8>(__byte_perm(vc[0][k >> 1], vc[1][k >> 1], sel), x);
                            unpack_codes<7>(__byte_perm(vc[2][k >> 1], vc[3][k >> 1], sel), y);
                        };
#pragma unroll
                        for (int gr = 0; gr < HG; ++gr) {
                            uint32_t wf[NT][2];
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                float a[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) a[i] = part_of(w[n][i] * scaled_s(vw[i][gr], unit[n][gr]), wmask);
                                wf[n][0] = pack_f16_rz(a[0], a[1]);
                                wf[n][1] = pack_f16_rz(a[2], a[3]);
                            }
#pragma unroll
                            for (int kb = 0; kb < BPG; ++kb) {
                                const int k = gr * BPG + kb;
                                uint32_t x[4], y[4];
                                unpack_block(k, x, y);
                                if constexpr (PAIR) {
                                    uint32_t xh[4], yh[4];
                                    unpack_block(k + HB, xh, yh);
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        mma_f16(o[0][4 * k + i], x[i], xh[i], y[i], yh[i], wf[0][0], wf[0][1]);
                                } else {
#pragma unroll
                                    for (int n = 0; n < NT; ++n) {
                                        mma_f16(o[n][2 * k], x[0], x[1], y[0], y[1], wf[n][0], wf[n][1]);
                                        mma_f16(o[n][2 * k + 1], x[2], x[3], y[2], y[3], wf[n][0], wf[n][1]);
                                    }
                                }
                            }
                        }
                    }
                }
                // the warps take turns to refill the stage once all are done with it
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot_of]);
                if (k + kStages < nst && warp == (k & (kWarps - 1))) {
                    mbar_wait(&empty[slot_of], phase, p.err);
                    fence_proxy_async_smem();
                    issue(k + kStages);
                }
            }

            // ---- the warp's state: o[head][dim], m, l
            if (u > u0) __syncthreads();                  // the split before this one has been merged
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int hq = PAIR ? t & 1 : head0 + 4 * n + t;
                float lt = l[n];
                lt += __shfl_xor_sync(0xffffffffu, lt, 4);
                lt += __shfl_xor_sync(0xffffffffu, lt, 8);
                lt += __shfl_xor_sync(0xffffffffu, lt, 16);
                float zt[HG], un[HG];                                         // un: the products' scaling, undone
#pragma unroll
                for (int gr = 0; gr < HG; ++gr) {
                    un[gr] = __uint_as_float(0x7F000000u - __float_as_uint(__shfl_sync(0xffffffffu, unit[n][gr], 8 * t)));
                    float v = zo[n][gr];
                    v += __shfl_xor_sync(0xffffffffu, v, 4);
                    v += __shfl_xor_sync(0xffffffffu, v, 8);
                    zt[gr] = v + __shfl_xor_sync(0xffffffffu, v, 16);
                }
                if (hq < rep) {
                    if (g == 0 && cth == 0) {
                        wml[(wt * rep + hq) * 2] = m[n];
                        wml[(wt * rep + hq) * 2 + 1] = lt;
                    }
#pragma unroll
                    for (int k = 0; k < HB; ++k) {
                        const float z = zt[k / BPG];
                        float v[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if constexpr (PAIR) {
                                const float(&a)[4] = o[n][4 * k + i];
                                v[i] = cth ? a[2] + a[3] : a[0] + a[1];
                            } else {
                                const float(&a)[4] = o[n][2 * k + i / 2];
                                v[i] = (i & 1) ? a[2] + a[3] : a[0] + a[1];
                            }
                            v[i] = __fmaf_rn(v[i], un[k / BPG], z);
                        }
                        *reinterpret_cast<float4*>(wo + (wt * rep + hq) * D + 32 * (k + cth * HB) + 4 * g) =
                            make_float4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            __syncthreads();
            float* part = CL ? nullptr : p.part + ((size_t(b) * p.c.nkv + h) * p.nsplit + u) * rep * (D + 2);
            if (CL && first && u == u0) cluster_wait();
            for (int i = tid; i < rep * (D / 4); i += kThr) {
                const int hq = i / (D / 4), dim = (i % (D / 4)) * 4;
                float mw[kTileWarps], mx = -INFINITY, den = 0.f;
#pragma unroll
                for (int w = 0; w < kTileWarps; ++w) mx = fmaxf(mx, mw[w] = wml[(w * rep + hq) * 2]);
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kTileWarps; ++w) {
                    const float f = mw[w] == -INFINITY ? 0.f : exp2_approx(__fsub_rn(mw[w], mx));
                    const float4 v = *reinterpret_cast<const float4*>(wo + (w * rep + hq) * D + dim);
                    den = __fmaf_rn(f, wml[(w * rep + hq) * 2 + 1], den);
                    num.x = __fmaf_rn(f, v.x, num.x);
                    num.y = __fmaf_rn(f, v.y, num.y);
                    num.z = __fmaf_rn(f, v.z, num.z);
                    num.w = __fmaf_rn(f, v.w, num.w);
                }
                if constexpr (CL) {
                    const int at = hq * D + dim;
                    float* to = cg::this_cluster().map_shared_rank(recv, at / slice);
                    *reinterpret_cast<float4*>(to + u * slice + at % slice) = num;
                    if (dim == 0)
                        for (int r = 0; r < ranks; ++r)
                            *reinterpret_cast<float2*>(cg::this_cluster().map_shared_rank(recv_ml, r) + (u * rep + hq) * 2) =
                                make_float2(mx, den);
                } else {
                    float* dst = part + hq * (D + 2);
                    *reinterpret_cast<float2*>(dst + 2 + dim) = make_float2(num.x, num.y);
                    *reinterpret_cast<float2*>(dst + 4 + dim) = make_float2(num.z, num.w);
                    if (dim == 0) *reinterpret_cast<float2*>(dst) = make_float2(mx, den);
                }
            }
        }
        uses += nst;
        if (CL && first && u0 >= u1) cluster_wait();
        if (!CL) return;
        // ---- every split's state is here: this rank's slice of the output, and its own positions' mass
        cluster_arrive();
        cluster_wait();
        for (int i = tid; i < slice; i += kThr) {
            const int hq = (s * slice + i) / D;
            float mx = -INFINITY, num = 0.f, den = 0.f;
            for (int r = 0; r < ns; ++r) mx = fmaxf(mx, recv_ml[(r * rep + hq) * 2]);
            for (int r = 0; r < ns; ++r) {
                const float mr = recv_ml[(r * rep + hq) * 2];
                const float f = mr == -INFINITY ? 0.f : exp2_approx(__fsub_rn(mr, mx));
                den = __fmaf_rn(f, recv_ml[(r * rep + hq) * 2 + 1], den);
                num = __fmaf_rn(f, recv[r * slice + i], num);
            }
            p.out[(size_t(b) * p.nq + h * rep) * D + s * slice + i] = num * __frcp_rn(den);
        }
        if (!p.mass) return;
        __shared__ float hm[kKv4MaxRep], hl[kKv4MaxRep];
        if (tid < rep) {
            float mx = -INFINITY, den = 0.f;
            for (int r = 0; r < ns; ++r) mx = fmaxf(mx, recv_ml[(r * rep + tid) * 2]);
            for (int r = 0; r < ns; ++r) {
                const float mr = recv_ml[(r * rep + tid) * 2];
                den = __fmaf_rn(mr == -INFINITY ? 0.f : exp2_approx(__fsub_rn(mr, mx)), recv_ml[(r * rep + tid) * 2 + 1], den);
            }
            hm[tid] = mx;
            hl[tid] = __frcp_rn(den);
        }
        __syncthreads();
        for (int i = u0 * chunk + tid; i < end; i += kThr) {
            float add = 0.f;
            for (int k = 0; k < rep; ++k) add = __fmaf_rn(exp2_approx(__fsub_rn(sc_out[k * sc_ld + i], hm[k])), hl[k], add);
            __stcg(p.mass + row + i, __ldcg(p.mass + row + i) + add);    // (another SM's, of the row before)
        }
        first = false;
    }
}

// Second launch, grid (rep + position blocks, KV head, row): block x < rep merges the splits of query head x, the
// others add the mass of kMassPos positions each.  Reads the states (1 KB per split and pair of heads) and, for the mass,
// the scores from L2: 3 to 4 us, most of it the launch.
constexpr int kMassPos = kMergeThr * 4;

// One query head's split states by one warp: weight[s] = 2^(m_s - max m) (if given), and max m and 1 / sum l.
__device__ __forceinline__ void merge_states(const float* part, size_t stride, int ns, int lane, float* weight, float& mx,
                                             float& inv) {
    float m[(kKv4MaxSplits + 31) / 32], l[(kKv4MaxSplits + 31) / 32];
    mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < (kKv4MaxSplits + 31) / 32; ++i) {
        const int s = lane + 32 * i;
        float2 v = make_float2(-INFINITY, 0.f);
        if (s < ns) v = *reinterpret_cast<const float2*>(part + s * stride);
        m[i] = v.x;
        l[i] = v.y;
        mx = fmaxf(mx, v.x);
    }
    mx = warp_max(mx);
    float den = 0.f;
#pragma unroll
    for (int i = 0; i < (kKv4MaxSplits + 31) / 32; ++i) {
        const float f = m[i] == -INFINITY ? 0.f : exp2_approx(__fsub_rn(m[i], mx));
        if (weight && lane + 32 * i < ns) weight[lane + 32 * i] = f;
        den = __fmaf_rn(f, l[i], den);
    }
    inv = __frcp_rn(warp_sum(den));
}

__global__ void __launch_bounds__(kMergeThr) kv4_merge_kernel(const Kv4AttnParams p) {
    __shared__ float weight[kKv4MaxSplits], hm[kKv4MaxRep], hl[kKv4MaxRep];
    __shared__ float2 acc[kMergeThr];
    const int h = blockIdx.y, b = blockIdx.z, d = p.c.d, rep = p.nq / p.c.nkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int err = kv4_row_error(p, b);
    const size_t stride = size_t(rep) * (d + 2);              // between the splits of a head
    int chunk, ns;
    if (int(blockIdx.x) < rep) {
        const int hq = blockIdx.x;
        float2* out = reinterpret_cast<float2*>(p.out + (size_t(b) * p.nq + h * rep + hq) * d);
        pdl_wait();
        const int pairs = d / 2, groups = kMergeThr / pairs, i = tid % pairs, grp = tid / pairs;
        if (err != KMR_OK) {
            if (tid == 0 && h == 0 && hq == 0 && err != kEmptyRow) set_error(p.err, err);
            if (grp == 0) out[i] = make_float2(0.f, 0.f);
            return;
        }
        kv4_split_plan(p.cpos[b] + 1, chunk, ns);
        const float* part = p.part + (size_t(b) * p.c.nkv + h) * p.nsplit * stride + size_t(hq) * (d + 2);
        if (warp == 0) {
            float mx, inv;
            merge_states(part, stride, ns, lane, weight, mx, inv);
            if (lane == 0) hl[0] = inv;
        }
        __syncthreads();
        // the splits in 4 (d = 128) or 8 interleaved groups, each in split order, then the groups in order
        float2 num = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int s = grp; s < ns; s += groups) {
            const float2 v = *reinterpret_cast<const float2*>(part + s * stride + 2 + 2 * i);
            num.x = __fmaf_rn(weight[s], v.x, num.x);
            num.y = __fmaf_rn(weight[s], v.y, num.y);
        }
        acc[tid] = num;
        __syncthreads();
        if (grp) return;
        for (int k = 1; k < groups; ++k) {
            num.x += acc[i + k * pairs].x;
            num.y += acc[i + k * pairs].y;
        }
        out[i] = make_float2(num.x * hl[0], num.y * hl[0]);
        return;
    }
    if (err != KMR_OK) return;
    const int block0 = (int(blockIdx.x) - rep) * kMassPos, pos = block0 + tid * 4;       // this thread's four positions
    const int slot = p.slot_ids[b];
    int before = 0, most = 0;
    for (int r = tid; r < p.B; r += kMergeThr) {
        if (p.slot_ids[r] != slot || kv4_row_error(p, r) != KMR_OK) continue;
        before |= r < b;
        most |= p.cpos[r] >= block0;
    }
    // the slot's first row adds for all of them; nothing to add past the longest
    before = __syncthreads_or(before);
    most = __syncthreads_or(most);
    if (before || !most) return;
    pdl_wait();
    float add[4] = {0.f, 0.f, 0.f, 0.f};
    int last = 0;
    for (int r = b; r < p.B; ++r) {
        if (p.slot_ids[r] != slot || kv4_row_error(p, r) != KMR_OK) continue;
        const int L = p.cpos[r] + 1;
        last = max(last, L);
        kv4_split_plan(L, chunk, ns);
        __syncthreads();
        if (warp < rep) {
            float mx, inv;
            merge_states(p.part + (size_t(r) * p.c.nkv + h) * p.nsplit * stride + size_t(warp) * (d + 2), stride, ns, lane,
                         nullptr, mx, inv);
            if (lane == 0) {
                hm[warp] = mx;
                hl[warp] = inv;
            }
        }
        __syncthreads();
        const float* sc = p.scores + (size_t(r) * p.c.nkv + h) * rep * p.c.S + pos;
        if (pos < L) {
#pragma unroll 2
            for (int k = 0; k < rep; ++k) {
                const float4 v = *reinterpret_cast<const float4*>(sc + size_t(k) * p.c.S);
                const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (pos + e < L) add[e] = __fmaf_rn(exp2_approx(__fsub_rn(x[e], hm[k])), hl[k], add[e]);
            }
        }
    }
    float* mass = p.mass + (size_t(slot) * p.c.nkv + h) * p.c.S + pos;
    if (pos + 4 <= last) {
        float4 v = *reinterpret_cast<float4*>(mass);
        v.x += add[0]; v.y += add[1]; v.z += add[2]; v.w += add[3];
        *reinterpret_cast<float4*>(mass) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (pos + e < last) mass[e] += add[e];
    }
}
static_assert(kMergeThr / 32 >= kKv4MaxRep, "a warp per query head");

template <int D, int G, int HC>
const void* split_fn(bool cl) {
    return cl ? (const void*)kv4_split_kernel<D, G, HC, true> : (const void*)kv4_split_kernel<D, G, HC, false>;
}
struct SplitVariant {
    const void* fn;
    int smem, ctas;                              // CTAs of an SM
};
// A cluster of `ranks` CTAs whose scores, `positions` of each, stay in shared memory (0: no mass); ranks 0: no cluster.
template <int D, int G, int HC>
SplitVariant split_variant(int rep, int ranks, int positions) {
    using M = SplitSmem<D, G, HC>;
    return {split_fn<D, G, HC>(ranks > 0), ranks ? M::total(rep, ranks, positions) : M::base(rep), Share<D, HC>::kCtas};
}
template <int D, int G>
SplitVariant split_variant(int rep, int ranks, int positions) {
    if constexpr (G < D) {
        if (rep <= 2) return split_variant<D, G, HEADS_2>(rep, ranks, positions);
    }
    if (rep <= 4) return split_variant<D, G, HEADS_4>(rep, ranks, positions);
    return split_variant<D, G, HEADS_8>(rep, ranks, positions);
}
SplitVariant split_variant(int d, int g, int rep, int ranks, int positions) {
    if (d == 64) return g == 32 ? split_variant<64, 32>(rep, ranks, positions) : split_variant<64, 64>(rep, ranks, positions);
    if (g == 32) return split_variant<128, 32>(rep, ranks, positions);
    return g == 64 ? split_variant<128, 64>(rep, ranks, positions) : split_variant<128, 128>(rep, ranks, positions);
}

}  // namespace

int kv4_attn_splits(int S) {
    if (S <= kKv4ClusterLen) return 0;            // merged inside a cluster
    // a shorter row can have more splits than the longest: 16 at most until the chunk is 256 (4096 positions),
    // then one per 256 up to 76
    const int large = (S + 255) / 256, most = large > 16 ? large : 16;
    return most < kKv4MaxSplits ? most : kKv4MaxSplits;
}
size_t kv4_attn_part_bytes(int B, int nq, int d, int nsplit) {
    return (size_t(B) * nq * nsplit * (d + 2) * 4 + 15) & ~size_t(15);
}
cudaError_t kv4_attn_set_attributes() {
    const int shapes[5][2] = {{64, 32}, {64, 64}, {128, 32}, {128, 64}, {128, 128}};
    for (const auto& sh : shapes)
        for (int rep : {2, 4, 8})
            for (int ranks : {0, 1}) {
                const SplitVariant v = split_variant(sh[0], sh[1], rep, ranks, kKv4ClusterLen);
                cudaError_t e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
                if (e != cudaSuccess) return e;
                e = cudaFuncSetAttribute(v.fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                         cudaSharedmemCarveoutMaxShared);
                if (e != cudaSuccess) return e;
            }
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kv4_merge_kernel);
}

cudaError_t launch_kv4_attn(const Kv4AttnParams& p, cudaStream_t st) {
    Kv4AttnParams q = p;
    void* args[] = {&q};
    const int rep = p.nq / p.c.nkv;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThr);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.c.S <= kKv4ClusterLen) {
        int chunk, splits, ranks = 1;
        kv4_cluster_plan(p.c.S, chunk, splits);
        while (ranks < splits) ranks *= 2;
        // CTAs that run at a time: more than that only queue, and pay their start and end each, so then a CTA takes
        // several splits of its row, one after the other, which changes no result (16 rows of 1024, when taken: 13.2 -> 10.3
        // us, 10.9 now; the longer caches' splits of 256 gained nothing by it, 47.4 against 48.2 us for 16 rows of 8192)
        const long long slots = (long long)split_variant(p.c.d, p.c.g, rep, 1, 0).ctas * num_sms();
        const long long rows = (long long)p.c.nkv * p.B;
        while (ranks > 1 && ranks * rows > slots) ranks /= 2;
        q.per = (splits + ranks - 1) / ranks;
        q.score_ld = q.per * chunk;
        const SplitVariant v = split_variant(p.c.d, p.c.g, rep, ranks, p.mass ? q.score_ld : 0);
        cfg.gridDim = dim3(ranks, p.c.nkv, p.B);
        cfg.dynamicSmemBytes = v.smem;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = ranks;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
        return cudaLaunchKernelExC(&cfg, v.fn, args);
    }
    const SplitVariant v = split_variant(p.c.d, p.c.g, rep, 0, 0);
    cfg.gridDim = dim3(p.nsplit, p.c.nkv, p.B);
    cfg.dynamicSmemBytes = v.smem;
    cudaError_t e = cudaLaunchKernelExC(&cfg, v.fn, args);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(rep + (p.mass ? (p.c.S + kMassPos - 1) / kMassPos : 0), p.c.nkv, p.B);
    cfg.blockDim = dim3(kMergeThr);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelExC(&cfg, (const void*)kv4_merge_kernel, args);
}

}  // namespace kmr
