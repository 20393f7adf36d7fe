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

constexpr int kThr = 256, kWarps = kThr / 32, kCluster = 8;

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

// Rows of a tile: MT m-tiles of 16 (R = 16 MT, or R = 1 with MT = 1: `rows` says how many are real).
template <bool BF16, int RT, int MT>       // RT: 8-rank tiles
__global__ void __launch_bounds__(kThr) lora_kernel(const LoraParams p, int R) {
    constexpr int RP = RT * 8;             // ranks, padded
    constexpr int KW = kWarps / MT;        // warps that share an m-tile
    __shared__ int ids[16 * MT];
    extern __shared__ __align__(16) float sm[];
    float* vpart = sm;                     // [KW][16 MT][RP]
    float* vloc = vpart + KW * 16 * MT * RP;   // [16 MT][RP]: this CTA's part of v, read by the cluster
    float* vsum = vloc + 16 * MT * RP;     // [16 MT][RP]
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank());
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int mt = warp / KW, kw = warp % KW;
    const int row0 = int(blockIdx.x / kCluster) * R;
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
    const int ra = 16 * mt + g, rb = ra + 8;              // this lane's rows
    const int ida = ids[ra], idb = ids[rb];
    // this rank's columns of the output: whole blocks of 16
    const int blocks = p.N >> 4;
    const int n0 = blocks * rank / kCluster, n1 = blocks * (rank + 1) / kCluster;
    const int k0 = (p.K / 16) * rank / kCluster, k1 = (p.K / 16) * (rank + 1) / kCluster;      // k-steps of 16

    // rows without an adapter
    for (int r = warp; r < rows; r += kWarps) {
        if (ids[r] >= 0 || p.base == p.y) continue;
        const size_t at = size_t(row0 + r) * p.ldy;
        for (int c = n0 * 16 + lane; c < n1 * 16; c += 32) {
            if (BF16)
                static_cast<uint16_t*>(p.y)[at + c] = p.base ? static_cast<const uint16_t*>(p.base)[at + c] : uint16_t(0);
            else
                static_cast<float*>(p.y)[at + c] = p.base ? static_cast<const float*>(p.base)[at + c] : 0.f;
        }
    }

    for (int lead = 0; lead < rows; ++lead) {
        const int a = ids[lead];
        if (a < 0) continue;
        bool first = true;
        for (int r = 0; r < lead; ++r) first = first && ids[r] != a;
        if (!first) continue;
        const int rank_a = p.ranks ? max(0, min(p.r, p.ranks[a])) : p.r;
        const uint16_t* A = p.a + size_t(a) * p.r * p.K;
        const uint16_t* B = p.b + size_t(a) * p.N * p.r;
        // ---- v = A x over this rank's k-steps
        float d[RT][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) clear4(d[j]);
        const bool ua = ida == a, ub = idb == a;
        const size_t xa = size_t(row0 + ra) * p.ldx, xb = size_t(row0 + rb) * p.ldx;
        for (int ks = k0 + kw; ks < k1; ks += KW) {
            const int k = ks * 16 + 4 * t;
            float fa[4] = {0.f, 0.f, 0.f, 0.f}, fb[4] = {0.f, 0.f, 0.f, 0.f};
            uint32_t A0[4] = {0, 0, 0, 0};
            if (BF16) {
                const uint16_t* x = static_cast<const uint16_t*>(p.x);
                const uint2 va = ua ? *reinterpret_cast<const uint2*>(x + xa + k) : make_uint2(0, 0);
                const uint2 vb = ub ? *reinterpret_cast<const uint2*>(x + xb + k) : make_uint2(0, 0);
                A0[0] = va.x; A0[1] = vb.x; A0[2] = va.y; A0[3] = vb.y;
            } else {
                const float* x = static_cast<const float*>(p.x);
                const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 va = ua ? *reinterpret_cast<const float4*>(x + xa + k) : z;
                const float4 vb = ub ? *reinterpret_cast<const float4*>(x + xb + k) : z;
                fa[0] = va.x; fa[1] = va.y; fa[2] = va.z; fa[3] = va.w;
                fb[0] = vb.x; fb[1] = vb.y; fb[2] = vb.z; fb[3] = vb.w;
            }
            uint2 w[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int n = 8 * j + g;
                w[j] = n < rank_a ? *reinterpret_cast<const uint2*>(A + size_t(n) * p.K + k) : make_uint2(0, 0);
            }
#pragma unroll
            for (int term = 0; term < (BF16 ? 1 : 3); ++term) {
                if (!BF16) {
                    A0[0] = take_term(fa[0], fa[1]);
                    A0[1] = take_term(fb[0], fb[1]);
                    A0[2] = take_term(fa[2], fa[3]);
                    A0[3] = take_term(fb[2], fb[3]);
                }
#pragma unroll
                for (int j = 0; j < RT; ++j) mma_bf16(d[j], A0, w[j].x, w[j].y);
            }
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            float* to = vpart + (size_t(kw) * 16 * MT + ra) * RP + 8 * j + 2 * t;
            *reinterpret_cast<float2*>(to) = make_float2(d[j][0], d[j][1]);
            *reinterpret_cast<float2*>(to + 8 * RP) = make_float2(d[j][2], d[j][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * MT * RP; i += kThr) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) s = __fadd_rn(s, vpart[size_t(w) * 16 * MT * RP + i]);
            vloc[i] = s;
        }
        cluster.sync();
        for (int i = threadIdx.x; i < 16 * MT * RP; i += kThr) {
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kCluster; ++q) s = __fadd_rn(s, cluster.map_shared_rank(vloc, q)[i]);
            vsum[i] = s;
        }
        __syncthreads();
        // ---- y = base + scale B v over this rank's columns: a warp takes blocks of 16
        const float scale = p.scales ? p.scales[a] : 1.f;
        for (int nb = n0 + kw; nb < n1; nb += KW) {
            float e[2][4];
            clear4(e[0]);
            clear4(e[1]);
#pragma unroll
            for (int ks = 0; ks < (RT + 1) / 2; ++ks) {
                const int k = ks * 16 + 4 * t;                   // ranks k..k + 3
                float fa[4], fb[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool in = k + q < rank_a;
                    fa[q] = in ? vsum[ra * RP + k + q] : 0.f;
                    fb[q] = in ? vsum[rb * RP + k + q] : 0.f;
                }
                uint2 w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // column g of n-tile h: output columns 4 (g / 2) + 2 h + g % 2 of the block
                    const int n = nb * 16 + 4 * (g >> 1) + 2 * h + (g & 1);
                    w[h] = k < p.r ? *reinterpret_cast<const uint2*>(B + size_t(n) * p.r + k) : make_uint2(0, 0);
                    // ranks past this adapter's: whatever the array holds there
                    if (k + 0 >= rank_a) w[h].x &= 0xFFFF0000u;
                    if (k + 1 >= rank_a) w[h].x &= 0x0000FFFFu;
                    if (k + 2 >= rank_a) w[h].y &= 0xFFFF0000u;
                    if (k + 3 >= rank_a) w[h].y &= 0x0000FFFFu;
                }
#pragma unroll
                for (int term = 0; term < 3; ++term) {
                    uint32_t A0[4];
                    A0[0] = take_term(fa[0], fa[1]);
                    A0[1] = take_term(fb[0], fb[1]);
                    A0[2] = take_term(fa[2], fa[3]);
                    A0[3] = take_term(fb[2], fb[3]);
                    mma_bf16(e[0], A0, w[0].x, w[0].y);
                    mma_bf16(e[1], A0, w[1].x, w[1].y);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!(h ? ub : ua)) continue;
                const size_t at = size_t(row0 + (h ? rb : ra)) * p.ldy + nb * 16 + 4 * t;
                float o[4] = {e[0][2 * h], e[0][2 * h + 1], e[1][2 * h], e[1][2 * h + 1]};
                if (BF16) {
                    uint2 b = make_uint2(0, 0);
                    if (p.base) b = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.base) + at);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
                        make_uint2(cvt2(__fmaf_rn(scale, o[0], bf16_lo(b.x)), __fmaf_rn(scale, o[1], bf16_hi(b.x))),
                                   cvt2(__fmaf_rn(scale, o[2], bf16_lo(b.y)), __fmaf_rn(scale, o[3], bf16_hi(b.y))));
                } else {
                    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p.base) b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.base) + at);
                    *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) =
                        make_float4(__fmaf_rn(scale, o[0], b.x), __fmaf_rn(scale, o[1], b.y), __fmaf_rn(scale, o[2], b.z),
                                    __fmaf_rn(scale, o[3], b.w));
                }
            }
        }
        cluster.sync();                    // the others have read this CTA's part of v
    }
}

template <bool BF16, int RT, int MT>
cudaError_t run(const LoraParams& p, int R, cudaStream_t st, bool set_only) {
    const size_t smem = size_t(kWarps / MT + 2) * 16 * MT * RT * 8 * 4;
    const void* fn = (const void*)lora_kernel<BF16, RT, MT>;
    if (set_only) return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((p.T + R - 1) / R) * kCluster);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, lora_kernel<BF16, RT, MT>, p, R);
}
template <bool BF16, int RT>
cudaError_t by_rows(const LoraParams& p, int R, cudaStream_t st, bool set_only) {
    if (set_only) {
        const cudaError_t e = run<BF16, RT, 1>(p, R, st, true);
        return e != cudaSuccess ? e : run<BF16, RT, 4>(p, R, st, true);
    }
    return R > 16 ? run<BF16, RT, 4>(p, R, st, false) : run<BF16, RT, 1>(p, R, st, false);
}
template <bool BF16>
cudaError_t by_rank(const LoraParams& p, int R, cudaStream_t st, bool set_only) {
    if (p.r <= 8) return by_rows<BF16, 1>(p, R, st, set_only);
    if (p.r <= 16) return by_rows<BF16, 2>(p, R, st, set_only);
    if (p.r <= 32) return by_rows<BF16, 4>(p, R, st, set_only);
    if (p.r <= 64) return by_rows<BF16, 8>(p, R, st, set_only);
    return by_rows<BF16, 16>(p, R, st, set_only);
}

}  // namespace

cudaError_t launch_lora(const LoraParams& p, bool bf16, int sms, cudaStream_t st) {
    const int R = p.T <= 64 ? 1 : (p.T < 2048 ? 16 : 64);
    return bf16 ? by_rank<true>(p, R, st, false) : by_rank<false>(p, R, st, false);
}

cudaError_t lora_set_attributes() {
    LoraParams p = {};
    for (p.r = 8; p.r <= kLoraMaxRank; p.r *= 2) {
        cudaError_t e = by_rank<true>(p, 0, nullptr, true);
        if (e == cudaSuccess) e = by_rank<false>(p, 0, nullptr, true);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kmr
