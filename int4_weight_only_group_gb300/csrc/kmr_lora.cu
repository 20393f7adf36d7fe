// Adapters of many requests beside a shared projection: y = base + scale_a B_a (A_a x), a = the row's adapter.
//
// Both products are skinny (rank r at most 128), so the call is bound by reading x and base and writing y once; for a
// few rows by latency and the adapters' own bytes.
//   * A cluster of C = 1..8 CTAs takes R consecutive rows.  Each CTA multiplies its share of K (v = A x, all r ranks), the
//     partials meet through distributed shared memory in rank order, and each CTA adds its share of the N columns: x, base
//     and y pass through once, v never leaves the chip, one launch.
//   * Every warp has its own columns and streams them, rows of x (or base) and the same columns of A (or rows of B), through
//     a ring of its own by 16-byte cp.async, two to four units of 64 or 128 bytes a row deep: nothing but a wait for its own copies
//     stands between a warp and its products.  (Loads into registers, eight bytes a lane, held up by the L1's tags: 4077 rows
//     42 us against 27.5.  A ring per CTA, fed by one warp with bulk copies of 512 bytes or by four with cp.async: 52 and 45
//     us; a bulk copy costs the copy engine some 60 cycles, and 16 warps that all wait for each chunk proceed in step.)
//   * A tile's distinct adapters are taken in turn, other rows left out: runs of rows of one request (a prompt) cost one turn.
//     A row's result does not hang on its neighbours (on T only by the order of the sums over K).
//   * mma.m16n8k16 in bf16 with fp32 sums.  fp32 operands (x, v) are cut into three bf16 terms, which hold their 24 bits
//     whatever their exponent; the adapters are bf16 already, so the products are exact.
// Measured: one row, K 2048, N 4096, r 16: 4.5 us; 16 rows of 16 requests, K = N = 2048, r 64: 7.2 us; 4077 rows bf16, K 2048, N
// 4096, r 16: 27.3 us (3.0 TB/s); 8192 rows fp32, K 6144, N 2048, r 32: 79 us (4.3 TB/s of 6.8: the cutting into terms and the
// MMAs take half the issue slots).
#include <cooperative_groups.h>

#include "kmr_moe.cuh"

namespace kmr {

namespace cg = cooperative_groups;

namespace {

constexpr int kThr = 256, kWarps = kThr / 32, kMaxCluster = 8;

// {lo, hi} as bf16 (round to nearest), and what is left of them
__device__ __forceinline__ uint32_t cvt2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// term i of the pair: takes the term off lo and hi
__device__ __forceinline__ uint32_t take_term(float& lo, float& hi) {
    const uint32_t r = cvt2(lo, hi);
    lo = __fsub_rn(lo, bf16_lo(r));
    hi = __fsub_rn(hi, bf16_hi(r));
    return r;
}

__device__ __forceinline__ void clear4(float (&d)[4]) { d[0] = d[1] = d[2] = d[3] = 0.f; }

// The A operand of a step of 16 from fp32 values (rows g and g + 8, four consecutive k each): one of three terms, taken off.
__device__ __forceinline__ void term_of(float (&fa)[4], float (&fb)[4], uint32_t (&A)[4]) {
    A[0] = take_term(fa[0], fa[1]);
    A[1] = take_term(fb[0], fb[1]);
    A[2] = take_term(fa[2], fa[3]);
    A[3] = take_term(fb[2], fb[3]);
}

// Eight consecutive values of a row: fp32 or bf16.
template <bool BF16>
struct Eight {
    float4 v[2];
    __device__ __forceinline__ void values(float (&f)[8]) const {
        f[0] = v[0].x, f[1] = v[0].y, f[2] = v[0].z, f[3] = v[0].w;
        f[4] = v[1].x, f[5] = v[1].y, f[6] = v[1].z, f[7] = v[1].w;
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        v[0] = make_float4(f[0], f[1], f[2], f[3]);
        v[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ void store(void* p, size_t at) const {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        to[0] = v[0];
        to[1] = v[1];
    }
};
template <>
struct Eight<true> {
    uint4 v;
    __device__ __forceinline__ void values(float (&f)[8]) const {
        f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
    }
    __device__ __forceinline__ void set(const float (&f)[8]) {
        v = make_uint4(cvt2(f[0], f[1]), cvt2(f[2], f[3]), cvt2(f[4], f[5]), cvt2(f[6], f[7]));
    }
    __device__ __forceinline__ void store(void* p, size_t at) const { *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = v; }
};
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// A warp's ring: `stages` units, each 16 rows of x (or base) and the same columns of A (or rows of B).  Wide rows of A (many ranks)
// take shorter units, so that two CTAs fit to an SM as far as they can.  (Short units for all and four CTAs: 4077 rows 30.5 us
// instead of 27.5; a unit's fixed instructions count for more than the warps that hide their latency.)
template <bool BF16, int RT>
struct Cfg {
    static constexpr int RP = RT * 8;                                   // ranks, padded
    static constexpr int KS = (RT + 1) / 2;                             // steps of 16 ranks
    static constexpr int SZ = BF16 ? 2 : 4;
    static constexpr int ROW = BF16 && RT >= 4 ? 64 : 128;             // bytes of a row of x or base in a unit
    static constexpr int COLS = ROW / SZ, SUB = COLS / 32;              // its columns: 32 or 64, in runs of 32
    static constexpr int AROW = COLS * 2;                               // bytes of a row of A in a unit
    static constexpr int XBYTES = 16 * ROW, STAGE = XBYTES + RP * AROW;
    static constexpr int STAGES = RT == 1 ? 4 : (RT <= 4 ? 3 : (RT == 8 && !BF16 ? 4 : 2));
    static constexpr int CTAS = RT == 16 || (RT == 8 && !BF16) ? 1 : 2;     // to an SM
    static constexpr int TERMS = BF16 ? 2 : 3;                          // of v (bf16 results: two terms hold 16 bits)
    static constexpr size_t SMEM = size_t(kWarps) * STAGES * STAGE + size_t(kWarps / 2 + 2) * 16 * RP * 4;
};
// Where the 16-byte piece c of a row lies, so that eight lanes that read (two rows, four pieces) meet no bank twice: bf16 lanes
// read pieces t, t + 4 of rows of 128 bytes, fp32 lanes 2 t and 2 t + 1.
template <bool BF16, int ROW>
__device__ __forceinline__ int swizzled(int c, int row) {
    if (!BF16) return c ^ (row & 1);
    return ROW == 128 ? c ^ ((row & 1) << 2) : c;
}

// R rows to a tile: 16, or 1.  RT: 8-rank tiles.
template <bool BF16, int RT>
__global__ void __launch_bounds__(kThr, Cfg<BF16, RT>::CTAS) lora_kernel(const LoraParams p, int R) {
    using F = Cfg<BF16, RT>;
    constexpr int RP = F::RP, KS = F::KS, SZ = F::SZ, ROW = F::ROW, COLS = F::COLS, SUB = F::SUB, AROW = F::AROW, S = F::STAGES;
    constexpr int XP = ROW / 16, XR = 32 / XP, AP = AROW / 16, AR = 32 / AP;     // pieces of a row, rows of an instruction
    __shared__ __align__(16) int ids[32];
    __shared__ uint32_t leads;             // rows that are the first with their adapter
    extern __shared__ __align__(128) uint8_t sm[];
    float* vpart = reinterpret_cast<float*>(sm + size_t(kWarps) * S * F::STAGE);     // [kWarps / 2][16][RP]
    float* vloc = vpart + kWarps / 2 * 16 * RP;      // [16][RP]: this CTA's part of v, read by the cluster
    float* vsum = vloc + 16 * RP;          // [16][RP]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), C = int(cluster.num_blocks());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int row0 = int(blockIdx.x / C) * R;
    const int rows = min(R, p.T - row0);
    uint8_t* ring = sm + size_t(warp) * S * F::STAGE;
    const uint32_t ring32 = smem_u32(ring);
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 0) {
        int a = lane < rows ? p.ids[row0 + lane] : -1;
        if (a < -1 || a >= p.L) {
            if (rank == 0) set_error(p.err, KMR_ERR_INVALID_ARG);
            a = -1;
        }
        ids[lane] = a;
        const uint32_t same = __match_any_sync(0xffffffffu, a);       // (by the whole warp, whatever a is)
        const uint32_t m = __ballot_sync(0xffffffffu, a >= 0 && __ffs(same) - 1 == lane);
        if (lane == 0) leads = m;
    }
    __syncthreads();
    const int ida = ids[g], idb = ids[g + 8];             // of this lane's rows
    // this rank's units of the inputs and of the outputs, and this warp's of them
    auto share = [&](int n, int& from, int& to) {
        const int units = (n + COLS - 1) / COLS, u0 = units * rank / C, u1 = units * (rank + 1) / C;
        const int per = (u1 - u0 + kWarps - 1) / kWarps;
        from = u0 + warp * per;
        to = min(u1, from + per);
    };
    int kb, ke, nb, ne;
    share(p.K, kb, ke);
    share(p.N, nb, ne);

    // rows without an adapter
    if (p.base != p.y) {
        for (int r = 0; r < rows; ++r) {
            if (ids[r] >= 0) continue;
            const size_t at = size_t(row0 + r) * p.ldy * SZ;
            for (int c = nb * ROW + lane * 16; c < min(ne * ROW, p.N * SZ); c += 512) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (p.base) v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.base) + at + c);
                *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + at + c) = v;
            }
        }
    }

    bool pending = false;                  // the others may still read this CTA's part of v
    for (uint32_t left = leads; left; left &= left - 1) {
        const int a = ids[__ffs(left) - 1];
        const int rank_a = p.ranks ? max(0, min(p.r, p.ranks[a])) : p.r;
        const float scale = p.scales ? p.scales[a] : 1.f;
        const uint16_t* A = p.a + size_t(a) * p.r * p.K;
        const uint16_t* B = p.b + size_t(a) * p.N * p.r;
        uint32_t mine = 0;                 // bit i: row lane / XP + XR i is one of the adapter's
#pragma unroll
        for (int i = 0; i < 16 / XR; ++i) mine |= (ids[lane / XP + XR * i] == a ? 1u : 0u) << i;
        const int xrow = lane / XP, xpiece = lane % XP, arow = lane / AP, apiece = lane % AP;
        // unit u of x or base, `n` columns wide
        auto copy_rows = [&](const void* from, long long ld, int n, int u, uint32_t to) {
            const int col = u * COLS + xpiece * (16 / SZ);
            const bool real = col < n;
            const uint8_t* at = static_cast<const uint8_t*>(from) + (size_t(row0 + xrow) * ld + (real ? col : 0)) * SZ;
#pragma unroll
            for (int i = 0; i < 16 / XR; ++i)
                if (mine >> i & 1u) {
                    const int row = xrow + XR * i;
                    copy16(to + row * ROW + swizzled<BF16, ROW>(xpiece, row) * 16, at + size_t(XR * i) * ld * SZ, real);
                }
        };
        auto copy_in = [&](int u, int stage) {
            if (u < ke) {
                const uint32_t to = ring32 + stage * F::STAGE;
                copy_rows(p.x, p.ldx, p.K, u, to);
                const int col = u * COLS + apiece * 8;
                const bool real = col < p.K;               // (past the inputs both sides are zero)
                const uint16_t* at = A + size_t(arow) * p.K + (real ? col : 0);
#pragma unroll
                for (int i = 0; i < RP / AR; ++i) {
                    const int n = arow + AR * i;
                    const int c = BF16 ? swizzled<BF16, AROW>(apiece, n) : apiece;
                    if (n < rank_a) copy16(to + F::XBYTES + n * AROW + c * 16, at + size_t(AR * i) * p.K, real);
                }
            }
            commit_copies();
        };
        auto copy_out = [&](int u, int stage) {
            if (u < ne) {
                const uint32_t to = ring32 + stage * F::STAGE;
                if (p.base) copy_rows(p.base, p.ldy, p.N, u, to);
                const int pieces = min(COLS, p.N - u * COLS) * p.r >> 3;
                const uint16_t* at = B + size_t(u) * COLS * p.r;
#pragma unroll 4
                for (int i = lane; i < pieces; i += 32) copy16(to + F::XBYTES + i * 16, at + i * 8, true);
            }
            commit_copies();
        };
        __syncwarp();
#pragma unroll
        for (int i = 0; i < S - 1; ++i) copy_in(kb + i, i);
        {                                  // B's bytes are on their way while v is formed
            const size_t from = size_t(nb) * COLS * p.r, to = size_t(min(ne * COLS, p.N)) * p.r;
            for (size_t i = from + lane * 64; i < to; i += 32 * 64) prefetch_l2(B + i);
        }

        // ---- v = A x over this warp's units
        float d[RT][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) clear4(d[j]);
        for (int u = kb, stage = 0; u < ke; ++u) {
            wait_copies<S - 2>();
            __syncwarp();
            copy_in(u + S - 1, stage == 0 ? S - 1 : stage - 1);
            const uint8_t* at = ring + stage * F::STAGE;
            stage = stage == S - 1 ? 0 : stage + 1;
            // (the tensor cores cut a running sum off rather than round it: fp32 sums are taken over in short runs, the small terms first,
            // so that only two steps do so at a run's full size)
            float c[RT][4];
            if (!BF16) {
#pragma unroll
                for (int j = 0; j < RT; ++j) clear4(c[j]);
            }
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                // a lane's eight inputs 8 t .. of 32 make two steps of 16 (any order of the inputs will do)
                const uint8_t* wat = at + F::XBYTES + g * AROW + (BF16 ? swizzled<BF16, AROW>(sub * 4 + t, g) : t) * 16;
                if constexpr (BF16) {
                    const uint4 xa = *reinterpret_cast<const uint4*>(at + g * ROW + swizzled<BF16, ROW>(sub * 4 + t, g) * 16);
                    const uint4 xb = *reinterpret_cast<const uint4*>(at + (g + 8) * ROW + swizzled<BF16, ROW>(sub * 4 + t, g) * 16);
                    const uint32_t A0[4] = {xa.x, xb.x, xa.y, xb.y}, A1[4] = {xa.z, xb.z, xa.w, xb.w};
#pragma unroll
                    for (int j = 0; j < RT; ++j) {
                        const uint4 w = *reinterpret_cast<const uint4*>(wat + j * 8 * AROW);
                        mma_bf16(d[j], A0, w.x, w.y);
                        mma_bf16(d[j], A1, w.z, w.w);
                    }
                } else {
                    float fa[2][4], fb[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float4 xa = *reinterpret_cast<const float4*>(at + g * ROW + swizzled<BF16, ROW>(2 * t + h, g) * 16);
                        const float4 xb = *reinterpret_cast<const float4*>(at + (g + 8) * ROW + swizzled<BF16, ROW>(2 * t + h, g) * 16);
                        fa[h][0] = xa.x, fa[h][1] = xa.y, fa[h][2] = xa.z, fa[h][3] = xa.w;
                        fb[h][0] = xb.x, fb[h][1] = xb.y, fb[h][2] = xb.z, fb[h][3] = xb.w;
                    }
                    uint4 w[RT <= 8 ? RT : 1];
                    if (RT <= 8) {
#pragma unroll
                        for (int j = 0; j < RT; ++j) w[RT <= 8 ? j : 0] = *reinterpret_cast<const uint4*>(wat + j * 8 * AROW);
                    }
                    uint32_t A0[3][4], A1[3][4];           // (multiplied the smallest first, as below)
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        term_of(fa[0], fb[0], A0[term]);
                        term_of(fa[1], fb[1], A1[term]);
                    }
#pragma unroll
                    for (int term = 2; term >= 0; --term) {
#pragma unroll
                        for (int j = 0; j < RT; ++j) {
                            const uint4 wj = RT <= 8 ? w[RT <= 8 ? j : 0] : *reinterpret_cast<const uint4*>(wat + j * 8 * AROW);
                            mma_bf16(c[j], A0[term], wj.x, wj.y);
                            mma_bf16(c[j], A1[term], wj.z, wj.w);
                        }
                    }
                }
            }
            if (!BF16) {
#pragma unroll
                for (int j = 0; j < RT; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[j][q] = __fadd_rn(d[j][q], c[j][q]);
            }
        }
        wait_copies<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < S - 1; ++i) copy_out(nb + i, i);

        // the warps' parts meet: the upper four warps' with the lower four's, then those
        float* slot = vpart + ((warp & (kWarps / 2 - 1)) * 16 + g) * RP + 2 * t;
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            if (step == 1) __syncthreads();
            if ((warp < kWarps / 2) != (step == 1)) continue;
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float2* to = reinterpret_cast<float2*>(slot + h * 8 * RP + 8 * j);
                    float2 v = make_float2(d[j][2 * h], d[j][2 * h + 1]);
                    if (step == 1) v = make_float2(__fadd_rn(v.x, to->x), __fadd_rn(v.y, to->y));
                    *to = v;
                }
        }
        if (pending) cluster.barrier_wait();
        __syncthreads();
        const int live = rows * RP;
        for (int i = threadIdx.x; i < live; i += kThr) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps / 2; ++w) v = __fadd_rn(v, vpart[w * 16 * RP + i]);
            vloc[i] = v;
        }
        cluster.sync();
        for (int i = threadIdx.x; i < live; i += kThr) {
            float q[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) q[c] = c < C ? cluster.map_shared_rank(vloc, c)[i] : 0.f;
            float v = q[0];
#pragma unroll
            for (int c = 1; c < kMaxCluster; ++c) v = __fadd_rn(v, q[c]);
            // (ranks past this adapter's: whatever the ring held there)
            vsum[i] = int(unsigned(i) % RP) < rank_a ? v : 0.f;
        }
        cluster.barrier_arrive();
        pending = true;
        __syncthreads();
        uint32_t V[KS][F::TERMS][4];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int k = ks * 16 + 4 * t;
            float fa[4], fb[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                fa[q] = k < RP && g < rows ? vsum[g * RP + k + q] : 0.f;
                fb[q] = k < RP && g + 8 < rows ? vsum[(g + 8) * RP + k + q] : 0.f;
            }
#pragma unroll
            for (int term = 0; term < F::TERMS; ++term) term_of(fa, fb, V[ks][term]);
        }

        // ---- y = base + scale B v over this warp's units of the outputs
        for (int u = nb, stage = 0; u < ne; ++u) {
            wait_copies<S - 2>();
            __syncwarp();
            copy_out(u + S - 1, stage == 0 ? S - 1 : stage - 1);
            const uint8_t* at = ring + stage * F::STAGE;
            stage = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                float e[4][4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint2 ws[KS];
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        // column g of n-tile h: output column 8 (g / 2) + 2 h + g % 2 of the run; ranks k .. k + 3
                        const int n = sub * 32 + 8 * (g >> 1) + 2 * h + (g & 1), k = ks * 16 + 4 * t;
                        uint2 w = k < p.r ? *reinterpret_cast<const uint2*>(at + F::XBYTES + (n * p.r + k) * 2) : make_uint2(0u, 0u);
                        if (p.ranks) {
                            if (k + 0 >= rank_a) w.x &= 0xFFFF0000u;
                            if (k + 1 >= rank_a) w.x &= 0x0000FFFFu;
                            if (k + 2 >= rank_a) w.y &= 0xFFFF0000u;
                            if (k + 3 >= rank_a) w.y &= 0x0000FFFFu;
                        }
                        ws[ks] = w;
                    }
                    // the small terms first here, too (largest first in both products, fp32: rank 16 2.7e-7 and rank 128 6.1e-7 of the result
                    // instead of 1.1e-7 and 1.8e-7)
                    clear4(e[h]);
#pragma unroll
                    for (int term = F::TERMS - 1; term >= 0; --term)
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks) mma_bf16(e[h], V[ks][term], ws[ks].x, ws[ks].y);
                }
                const int col = u * COLS + sub * 32 + 8 * t;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((h ? idb : ida) != a || col >= p.N) continue;
                    Eight<BF16> v;
                    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                    if (p.base) {
                        const uint8_t* bat = at + (g + 8 * h) * ROW;
                        if constexpr (BF16) {
                            v.v = *reinterpret_cast<const uint4*>(bat + swizzled<BF16, ROW>(sub * 4 + t, g) * 16);
                        } else {
                            v.v[0] = *reinterpret_cast<const float4*>(bat + swizzled<BF16, ROW>(2 * t, g) * 16);
                            v.v[1] = *reinterpret_cast<const float4*>(bat + swizzled<BF16, ROW>(2 * t + 1, g) * 16);
                        }
                        v.values(o);
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) o[q] = __fmaf_rn(scale, e[q >> 1][2 * h + (q & 1)], o[q]);
                    v.set(o);
                    v.store(p.y, size_t(row0 + g + 8 * h) * p.ldy + col);
                }
            }
        }
        wait_copies<0>();
    }
    if (pending) cluster.barrier_wait();
}

template <bool BF16, int RT>
cudaError_t run(const LoraParams& p, int R, int C, cudaStream_t st, bool set_only) {
    const size_t smem = Cfg<BF16, RT>::SMEM;
    if (set_only) return cudaFuncSetAttribute((const void*)lora_kernel<BF16, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(C);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((p.T + R - 1) / R) * C);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_kernel<BF16, RT>, p, R);
}
template <bool BF16>
cudaError_t by_rank(const LoraParams& p, int R, int C, cudaStream_t st, bool set_only) {
    if (p.r <= 8) return run<BF16, 1>(p, R, C, st, set_only);
    if (p.r <= 16) return run<BF16, 2>(p, R, C, st, set_only);
    if (p.r <= 32) return run<BF16, 4>(p, R, C, st, set_only);
    if (p.r <= 64) return run<BF16, 8>(p, R, C, st, set_only);
    return run<BF16, 16>(p, R, C, st, set_only);
}

}  // namespace

cudaError_t launch_lora(const LoraParams& p, bool bf16, int sms, cudaStream_t st) {
    // One row a tile up to two rows an SM, else 16.  The ids are on the device, so the rule does not know how rows share adapters: single
    // rows read an adapter again for each, tiles of 16 take a tile's adapters in turn.  us, single rows against tiles (best cluster
    // each; K 2048, N 4096), where every row has its own adapter / 16 requests / one:
    //   bf16, rank 16    64 rows  6.3 : 43 / 6.2 : 18 / 4.9 : 5.6      256  15 : 59 / 14 : 14 / 10 : 6.2      400  26 : 63 / 23 : 14 / 17 : 6.4
    //   fp32, rank 64    64 rows  17 : 113 / 16 : 44 / 16 : 9.7        256  56 : 154 / 53 : 27 / 53 : 13      400  82 : 156 / 70 : 33 / 79 : 13
    //   fp32, rank 128   64 rows  29 : 169 / 27 : 77 / 19 : 10         256  98 : 268 / 94 : 48 / 63 : 14      400  150 : 274 / 140 : 47 / 94 : 14
    // So the worst case decides for small batches (decoding: requests of their own), and short prompts of one request pay for it up
    // to four times.  Then the largest cluster whose CTAs number up to 2.5 an SM: two places each, or for the ranks that take an SM to a
    // CTA some waves (1000 rows of 16 requests, rank 16: 14 in clusters of 4, 27 by themselves, 16 in clusters of 8; fp32 rank 128: 66, 156,
    // 79; 64 single rows of fp32 rank 64 are quicker in clusters of 2, 16 against 20; 4077 rows 28, and 36 in clusters of 4).
    const int R = p.T <= 2 * sms ? 1 : 16, tiles = (p.T + R - 1) / R;
    int C = kMaxCluster;
    while (C > 1 && tiles * C > 2 * sms + sms / 2) C /= 2;
    return bf16 ? by_rank<true>(p, R, C, st, false) : by_rank<false>(p, R, C, st, false);
}

cudaError_t lora_set_attributes() {
    LoraParams p = {};
    for (p.r = 8; p.r <= kLoraMaxRank; p.r *= 2) {
        cudaError_t e = by_rank<true>(p, 0, 1, nullptr, true);
        if (e == cudaSuccess) e = by_rank<false>(p, 0, 1, nullptr, true);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kmr
