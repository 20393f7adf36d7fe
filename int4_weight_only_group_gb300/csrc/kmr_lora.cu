// Adapters of many requests beside a shared projection: y = base + scale_a B_a (A_a x), a = the row's adapter.
//
// Both products are skinny (rank r at most 128), so the call is bound by reading x and base and writing y once; for a
// few rows by latency and the adapters' own bytes.
//   * A cluster of 8 CTAs takes R consecutive rows.  Each CTA multiplies an eighth of K (v = A x, all r ranks), the eight
//     partials meet through distributed shared memory in rank order, and each CTA adds its eighth of the N columns: x,
//     base and y pass through once, v never leaves the chip, one launch.
//   * A tile's distinct adapters are taken in turn, other rows masked: runs of rows of one request (a prompt) cost
//     one turn.  A row's result does not hang on its neighbours (on R only by the order of the sums over K).
//   * mma.m16n8k16 in bf16 with fp32 sums.  fp32 operands (x, v) are cut into three bf16 terms, which hold their 24 bits
//     whatever their exponent; the adapters are bf16 already, so the products are exact.
//   * The k and n indexes are dealt to the lanes so that each loads 16 bytes of a row at a time (any order of the
//     contraction will do, as long as both operands follow it).
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

// Four values of a row: fp32 or bf16.
template <bool BF16>
struct Four {
    float4 v;
    __device__ __forceinline__ void load(const void* p, size_t at, bool real) {
        v = real ? *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void store(void* p, size_t at) const { *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = v; }
    __device__ __forceinline__ void values(float (&f)[4]) const {
        f[0] = v.x;
        f[1] = v.y;
        f[2] = v.z;
        f[3] = v.w;
    }
};
template <>
struct Four<true> {
    uint2 v;
    __device__ __forceinline__ void load(const void* p, size_t at, bool real) {
        v = real ? *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at) : make_uint2(0u, 0u);
    }
    __device__ __forceinline__ void store(void* p, size_t at) const { *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = v; }
    __device__ __forceinline__ void values(float (&f)[4]) const {
        f[0] = bf16_lo(v.x);
        f[1] = bf16_hi(v.x);
        f[2] = bf16_lo(v.y);
        f[3] = bf16_hi(v.y);
    }
};
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Rows of a tile: MT m-tiles of 16 (R = 16 MT, or R = 1 with MT = 1: `rows` says how many are real).  RT: 8-rank tiles.
template <bool BF16, int RT, int MT>
__global__ void __launch_bounds__(kThr, RT >= 16 ? 1 : 2) lora_kernel(const LoraParams p, int R) {
    constexpr int RP = RT * 8;             // ranks, padded
    constexpr int KS = (RT + 1) / 2;       // steps of 16 ranks
    constexpr int KW = kWarps / MT;        // warps that share an m-tile
    constexpr int U = RT <= 2 ? (BF16 ? 8 : 4) : (RT == 4 ? 4 : (RT == 8 ? 2 : 1));       // steps of 16 inputs in flight
    constexpr int UN = RT <= 4 ? 4 : (RT == 8 ? 2 : 1);                      // blocks of 16 outputs in flight
    __shared__ __align__(16) int ids[16 * MT < 32 ? 32 : 16 * MT];
    __shared__ uint32_t leads[2];          // rows that are the first with their adapter
    extern __shared__ __align__(16) float sm[];
    float* vpart = sm;                     // [KW][16 MT][RP]
    float* vloc = vpart + KW * 16 * MT * RP;   // [16 MT][RP]: this CTA's part of v, read by the cluster
    float* vsum = vloc + 16 * MT * RP;     // [16 MT][RP]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), C = int(cluster.num_blocks());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int mt = warp / KW, kw = warp % KW;
    const int row0 = int(blockIdx.x / C) * R;
    const int rows = min(R, p.T - row0);
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x < 16 * MT) {
        int a = threadIdx.x < rows ? p.ids[row0 + threadIdx.x] : -1;
        if (a < -1 || a >= p.L) {
            if (rank == 0) set_error(p.err, KMR_ERR_INVALID_ARG);
            a = -1;
        }
        ids[threadIdx.x] = a;
    }
    __syncthreads();
    if (warp < 2) {
        const int i = threadIdx.x;
        const int a = i < 16 * MT ? ids[i] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, a);       // (by the whole warp, whatever a is)
        bool lead = a >= 0 && __ffs(same) - 1 == lane;
        if (MT > 2 && warp == 1) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int4 o = reinterpret_cast<const int4*>(ids)[j];
                lead = lead && o.x != a && o.y != a && o.z != a && o.w != a;
            }
        }
        const uint32_t m = __ballot_sync(0xffffffffu, lead);
        if (lane == 0) leads[warp] = m;
    }
    __syncthreads();
    const int ra = 16 * mt + g, rb = ra + 8;              // this lane's rows
    const int ida = ids[ra], idb = ids[rb];
    // this rank's columns of the output: whole blocks of 16, and this warp's part of its k-steps
    const int blocks = p.N >> 4;
    const int n0 = blocks * rank / C, n1 = blocks * (rank + 1) / C;
    const int k0 = (p.K / 16) * rank / C, k1 = (p.K / 16) * (rank + 1) / C;
    const int kper = (k1 - k0 + KW - 1) / KW, kb = k0 + kw * kper, ke = min(k1, kb + kper);

    // rows without an adapter
    for (int r = warp; r < rows; r += kWarps) {
        if (ids[r] >= 0 || p.base == p.y) continue;
        const size_t at = size_t(row0 + r) * p.ldy;
        for (int c = n0 * 16 + lane * 4; c < n1 * 16; c += 128) {
            Four<BF16> f;
            f.load(p.base, at + c, p.base != nullptr);
            f.store(p.y, at + c);
        }
    }

    bool pending = false;                  // the others may still read this CTA's part of v
    for (uint64_t left = leads[0] | (uint64_t(leads[1]) << 32); left; left &= left - 1) {
        const int a = ids[__ffsll(left) - 1];
        const int rank_a = p.ranks ? max(0, min(p.r, p.ranks[a])) : p.r;
        const float scale = p.scales ? p.scales[a] : 1.f;
        const uint16_t* A = p.a + size_t(a) * p.r * p.K;
        const uint16_t* B = p.b + size_t(a) * p.N * p.r;
        const bool ua = ida == a, ub = idb == a;
        const size_t xa = size_t(row0 + ra) * p.ldx, xb = size_t(row0 + rb) * p.ldx;
        const size_t ya = size_t(row0 + ra) * p.ldy, yb = size_t(row0 + rb) * p.ldy;

        uint2 w2[UN][KS][2];
        Four<BF16> oa[UN], ob[UN];
        auto load_out = [&](int nb0) {
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int nb = nb0 + i;
                const bool real = nb < n1;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // column g of n-tile h: output columns 4 (g / 2) + 2 h + g % 2 of the block; ranks k .. k + 3
                        const int k = ks * 16 + 4 * t, n = nb * 16 + 4 * (g >> 1) + 2 * h + (g & 1);
                        w2[i][ks][h] = real && k < p.r ? *reinterpret_cast<const uint2*>(B + size_t(n) * p.r + k) : make_uint2(0u, 0u);
                    }
                oa[i].load(p.base, ya + nb * 16 + 4 * t, real && ua && p.base);
                ob[i].load(p.base, yb + nb * 16 + 4 * t, real && ub && p.base);
            }
        };
        if (MT == 1) {                     // few rows: B's bytes are on their way while v is formed
            const size_t from = size_t(n0) * 16 * p.r, to = size_t(n1) * 16 * p.r;
            for (size_t i = from + threadIdx.x * 64; i < to; i += kThr * 64) prefetch_l2(B + i);
        }

        // ---- v = A x over this warp's k-steps
        float d[RT][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) clear4(d[j]);
        for (int ks = kb; ks < ke; ks += U) {
            Four<BF16> va[U], vb[U];
            uint2 w[U][RT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = (ks + u) * 16 + 4 * t;
                const bool real = ks + u < ke;
                va[u].load(p.x, xa + k, real && ua);
                vb[u].load(p.x, xb + k, real && ub);
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    const int n = 8 * j + g;
                    w[u][j] = real && n < rank_a ? *reinterpret_cast<const uint2*>(A + size_t(n) * p.K + k) : make_uint2(0u, 0u);
                }
            }
            // (the tensor cores cut a running sum off rather than round it: fp32 sums are taken over in short runs)
            float c[RT][4];
            if (!BF16) {
#pragma unroll
                for (int j = 0; j < RT; ++j) clear4(c[j]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if constexpr (BF16) {
                    const uint32_t A0[4] = {(va[u].v.x), (vb[u].v.x), (va[u].v.y), (vb[u].v.y)};
#pragma unroll
                    for (int j = 0; j < RT; ++j) mma_bf16(d[j], A0, w[u][j].x, w[u][j].y);
                } else {
                    float fa[4], fb[4];
                    va[u].values(fa);
                    vb[u].values(fb);
#pragma unroll
                    for (int term = 0; term < 3; ++term) {
                        uint32_t A0[4];
                        term_of(fa, fb, A0);
#pragma unroll
                        for (int j = 0; j < RT; ++j) mma_bf16(c[j], A0, w[u][j].x, w[u][j].y);
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
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            float* to = vpart + (size_t(kw) * 16 * MT + ra) * RP + 8 * j + 2 * t;
            *reinterpret_cast<float2*>(to) = make_float2(d[j][0], d[j][1]);
            *reinterpret_cast<float2*>(to + 8 * RP) = make_float2(d[j][2], d[j][3]);
        }
        if (pending) cluster.barrier_wait();
        __syncthreads();
        const int live = min(16 * MT, rows) * RP;
        for (int i = threadIdx.x; i < live; i += kThr) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) s = __fadd_rn(s, vpart[size_t(w) * 16 * MT * RP + i]);
            vloc[i] = s;
        }
        cluster.sync();
        for (int i = threadIdx.x; i < live; i += kThr) {
            float q[kMaxCluster];
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c) q[c] = c < C ? cluster.map_shared_rank(vloc, c)[i] : 0.f;
            float s = q[0];
#pragma unroll
            for (int c = 1; c < kMaxCluster; ++c) s = __fadd_rn(s, q[c]);
            // (ranks past this adapter's: whatever its arrays hold there)
            vsum[i] = int(unsigned(i) % RP) < rank_a ? s : 0.f;
        }
        cluster.barrier_arrive();
        pending = true;
        __syncthreads();

        // ---- y = base + scale B v over this rank's columns: a warp takes UN blocks of 16 at a time
        for (int nb0 = n0 + kw * UN; nb0 < n1; nb0 += KW * UN) {
            load_out(nb0);
            float e[UN][2][4];
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                clear4(e[i][0]);
                clear4(e[i][1]);
            }
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const int k = ks * 16 + 4 * t;
                float fa[4] = {0.f, 0.f, 0.f, 0.f}, fb[4] = {0.f, 0.f, 0.f, 0.f};
                if (k < RP) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        fa[q] = ra < rows ? vsum[ra * RP + k + q] : 0.f;
                        fb[q] = rb < rows ? vsum[rb * RP + k + q] : 0.f;
                    }
                }
                if (p.ranks) {
#pragma unroll
                    for (int i = 0; i < UN; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (k + 0 >= rank_a) w2[i][ks][h].x &= 0xFFFF0000u;
                            if (k + 1 >= rank_a) w2[i][ks][h].x &= 0x0000FFFFu;
                            if (k + 2 >= rank_a) w2[i][ks][h].y &= 0xFFFF0000u;
                            if (k + 3 >= rank_a) w2[i][ks][h].y &= 0x0000FFFFu;
                        }
                }
                // (bf16 results: two terms hold 16 bits)
#pragma unroll
                for (int term = 0; term < (BF16 ? 2 : 3); ++term) {
                    uint32_t A0[4];
                    term_of(fa, fb, A0);
#pragma unroll
                    for (int i = 0; i < UN; ++i) {
                        mma_bf16(e[i][0], A0, w2[i][ks][0].x, w2[i][ks][0].y);
                        mma_bf16(e[i][1], A0, w2[i][ks][1].x, w2[i][ks][1].y);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                if (nb0 + i >= n1) continue;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(h ? ub : ua)) continue;
                    float o[4];
                    (h ? ob[i] : oa[i]).values(o);
                    o[0] = __fmaf_rn(scale, e[i][0][2 * h], o[0]);
                    o[1] = __fmaf_rn(scale, e[i][0][2 * h + 1], o[1]);
                    o[2] = __fmaf_rn(scale, e[i][1][2 * h], o[2]);
                    o[3] = __fmaf_rn(scale, e[i][1][2 * h + 1], o[3]);
                    const size_t at = (h ? yb : ya) + (nb0 + i) * 16 + 4 * t;
                    Four<BF16> r;
                    if constexpr (BF16) r.v = make_uint2(cvt2(o[0], o[1]), cvt2(o[2], o[3]));
                    else r.v = make_float4(o[0], o[1], o[2], o[3]);
                    r.store(p.y, at);
                }
            }
        }
    }
    if (pending) cluster.barrier_wait();
}

template <bool BF16, int RT, int MT>
cudaError_t run(const LoraParams& p, int R, int C, cudaStream_t st, bool set_only) {
    const size_t smem = size_t(kWarps / MT + 2) * 16 * MT * RT * 8 * 4;
    const void* fn = (const void*)lora_kernel<BF16, RT, MT>;
    if (set_only) return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
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
    return cudaLaunchKernelEx(&cfg, lora_kernel<BF16, RT, MT>, p, R);
}
template <bool BF16, int RT>
cudaError_t by_rows(const LoraParams& p, int R, int C, cudaStream_t st, bool set_only) {
    if (set_only) {
        return run<BF16, RT, 1>(p, R, C, st, true);
    }
    return run<BF16, RT, 1>(p, R, C, st, false);
}
template <bool BF16>
cudaError_t by_rank(const LoraParams& p, int R, int C, cudaStream_t st, bool set_only) {
    if (p.r <= 8) return by_rows<BF16, 1>(p, R, C, st, set_only);
    if (p.r <= 16) return by_rows<BF16, 2>(p, R, C, st, set_only);
    if (p.r <= 32) return by_rows<BF16, 4>(p, R, C, st, set_only);
    if (p.r <= 64) return by_rows<BF16, 8>(p, R, C, st, set_only);
    return by_rows<BF16, 16>(p, R, C, st, set_only);
}

}  // namespace

cudaError_t launch_lora(const LoraParams& p, bool bf16, int sms, cudaStream_t st) {
    // One row a tile up to two rows a SM: rows of a small batch have adapters of their own (64 rows of 64 adapters: 7 us against
    // 55 with tiles of 16; of 4 adapters 8 against 9).  More rows are taken 16 at a time (32 and 64 are no faster even for one
    // adapter: their phases overlap less).  Then the smallest cluster that gives every SM a CTA or two.
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
