// Int4 experts for a few tokens: gate_up + SiLU * up, then down + the weighted sum, two launches.
//
//   act[t, j] = silu(gate_e x[t]) * (up_e x[t]),  y[t] = sum_j weights[t, j] * down_e act[t, j],  e = ids[t, j],
//   rows of gate_e, up_e, down_e: w = (q - 8) s + z in the KMR4 layout (include/kmr.h).
//
// What bounds it: every expert that a token is sent to is read once (1.0625 bytes per 2 weights), so HBM; for one
// token the latency of two dependent kernels.  A warp plans the call by itself: its lanes hold the (at most 32)
// expert ids, one match gives the distinct experts.
//   * gate_up: (expert, 16-row tile) pairs are dealt out evenly over one CTA per SM, which fetches its tiles with
//     cp.async.bulk into a ring of two halves.
//   * down: a CTA owns 16 output columns and fetches that tile of every expert used, so a token's sum is formed in
//     one place, in the order of its places, without atomics.  Its weights' copies start while gate_up still runs.
//   * warp w multiplies the 128-input groups w, w + 16, ... of a tile (fewer groups: several tiles at once).  The codes
//     are the A operand of mma.m16n8k16, as exact fp16 integers q - 8; the inputs are B, scaled by a power of two per
//     (row, group): one column per token in bf16, two (the fp16 rounding and what it left) in fp32, so that products
//     and sums keep single precision.  Per group, y += (s D + z X) / sigma with D = sum (q - 8) x and X = sum x.
//   * partial sums meet in shared memory and are added in a fixed order that hangs on K alone: a token's result does not
//     change with the other tokens of the call.
#include <cuda_fp16.h>

#include "kmr_int4_mma.cuh"
#include "kmr_moe.cuh"
#include "kmr_tc.cuh"

namespace kmr {

namespace {

constexpr int kThr = 512, kWarps = kThr / 32;
constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ the call's plan, in a warp's registers
struct Plan {
    int id;                  // expert of place `lane`, or -1
    uint32_t leaders;        // first place of each distinct expert
};
__device__ __forceinline__ Plan make_plan(const int32_t* ids, int S, int E, int* err, bool report) {
    const int lane = threadIdx.x & 31;
    Plan pl;
    pl.id = lane < S ? ids[lane] : -1;
    if (pl.id < -1 || pl.id >= E) {
        if (report) set_error(err, KMR_ERR_INVALID_ARG);
        pl.id = -1;
    }
    const uint32_t same = __match_any_sync(kFull, pl.id);
    pl.leaders = __ballot_sync(kFull, pl.id >= 0 && __ffs(same) - 1 == lane);
    return pl;
}
// The n-th set bit of m, n < popc(m).
__device__ __forceinline__ int nth_bit(uint32_t m, int n) {
    int at = 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
        const int below = __popc((m >> at) & ((1u << w) - 1u));
        if (n >= below) {
            n -= below;
            at += w;
        }
    }
    return at;
}

// ------------------------------------------------------------------ operands
// B fragments of one 128-input group of up to 8 (SPLIT: 4) rows for this lane, and the group's fold constants.
struct Frag {
    uint32_t b[16];
    float X0, is0, X1, is1;  // of columns 2t and 2t + 1: sum of the staged values, 1 / sigma
};
// This lane's inputs of one group: row (column lane / 4, SPLIT: (lane / 4) % 4 with the remainders in columns 4..7) at the
// group's first input.  A lane without a row reads another's and takes zeros, so that all loads go out together.
template <typename IN>
__device__ __forceinline__ void load_raw(float (&v)[32], const IN* row, bool real, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 u;
        if constexpr (sizeof(IN) == 4) {
            u = __ldcg(reinterpret_cast<const float2*>(row + 8 * i + 2 * t));
        } else {
            const uint32_t r = __ldcg(reinterpret_cast<const uint32_t*>(row + 8 * i + 2 * t));
            u = make_float2(bf16_lo(r), bf16_hi(r));
        }
        v[2 * i] = real ? u.x : 0.f;
        v[2 * i + 1] = real ? u.y : 0.f;
    }
}
template <bool SPLIT>
__device__ __forceinline__ void make_frag(Frag& f, const float (&v)[32], int lane) {
    const int t = lane & 3;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 1));
    m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
    float sig, isg;
    pow2_scale(__float_as_uint(m), sig, isg);
    float X = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float a = __fmul_rn(v[2 * i], sig), b = __fmul_rn(v[2 * i + 1], sig);
        __half2 h = __floats2half2_rn(a, b);
        if (SPLIT) {
            const float2 r = __half22float2(h);
            const __half2 l = __floats2half2_rn(__fsub_rn(a, r.x), __fsub_rn(b, r.y));
            h = lane >= 16 ? l : h;
        }
        const float2 s = __half22float2(h);
        X = __fadd_rn(X, __fadd_rn(s.x, s.y));
        f.b[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 1));
    X = __fadd_rn(X, __shfl_xor_sync(kFull, X, 2));
    f.X0 = __shfl_sync(kFull, X, 8 * t);
    f.X1 = __shfl_sync(kFull, X, 8 * t + 4);
    f.is0 = __shfl_sync(kFull, isg, 8 * t);
    f.is1 = __shfl_sync(kFull, isg, 8 * t + 4);
}

// acc (rows g and g + 8, columns 2t and 2t + 1) += one (16-row tile, 128-input group) block times the fragments.
__device__ __forceinline__ void block_product(const uint8_t* gb, const Frag& f, int lane, float (&acc)[4]) {
    const int g = lane >> 2;
    const __half2 m8 = __float2half2_rn(-1032.f), c16 = __float2half2_rn(0.0625f), m72 = __float2half2_rn(-72.f);
    auto h2 = [](uint32_t v) { return *reinterpret_cast<const __half2*>(&v); };
    auto u2 = [](__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); };
    float d[2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) d[c][0] = d[c][1] = d[c][2] = d[c][3] = 0.f;
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
        const uint4 wq = *reinterpret_cast<const uint4*>(gb + blk * 512 + lane * 16);
        const uint32_t w4[4] = {wq.x, wq.y, wq.z, wq.w};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const uint32_t w = w4[ks], w2 = w >> 8;
            // 1024 + q less 1032, and (1024 + 16 q) / 16 less 72: exact
            mma16816(d[ks & 1], u2(__hadd2(h2(and_or(w, 0x000F000Fu, 0x64006400u)), m8)),
                     u2(__hfma2(h2(and_or(w, 0x00F000F0u, 0x64006400u)), c16, m72)),
                     u2(__hadd2(h2(and_or(w2, 0x000F000Fu, 0x64006400u)), m8)),
                     u2(__hfma2(h2(and_or(w2, 0x00F000F0u, 0x64006400u)), c16, m72)), f.b[blk * 8 + 2 * ks],
                     f.b[blk * 8 + 2 * ks + 1]);
        }
    }
    const uint32_t sz0 = *reinterpret_cast<const uint32_t*>(gb + 1024 + g * 4);
    const uint32_t sz1 = *reinterpret_cast<const uint32_t*>(gb + 1024 + (g + 8) * 4);
    auto fold = [](uint32_t sz, float D, float X) { return __fmaf_rn(bf16_lo(sz), D, __fmul_rn(bf16_hi(sz), X)); };
    acc[0] = __fmaf_rn(fold(sz0, __fadd_rn(d[0][0], d[1][0]), f.X0), f.is0, acc[0]);
    acc[1] = __fmaf_rn(fold(sz0, __fadd_rn(d[0][1], d[1][1]), f.X1), f.is1, acc[1]);
    acc[2] = __fmaf_rn(fold(sz1, __fadd_rn(d[0][2], d[1][2]), f.X0), f.is0, acc[2]);
    acc[3] = __fmaf_rn(fold(sz1, __fadd_rn(d[0][3], d[1][3]), f.X1), f.is1, acc[3]);
}

// This warp's partial of a tile, [16 rows][8 columns].
__device__ __forceinline__ void store_part8(float* to, int lane, const float (&acc)[4]) {
    const int g = lane >> 2, c = 2 * (lane & 3);
    *reinterpret_cast<float2*>(to + g * 8 + c) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(to + (g + 8) * 8 + c) = make_float2(acc[2], acc[3]);
}

// Warps that share a tile: the smallest power of two that covers its groups, 16 at most.
__host__ __device__ constexpr int group_warps(int G) { return G >= kWarps ? kWarps : pow2_at_least(G); }

// ------------------------------------------------------------------ the ring of tiles
// Tile i of the CTA's sequence lives in stage i % stages; the tiles of a batch (half the ring) are fetched together
// once the batch before the previous one has been used up.
struct Ring {
    uint8_t* data;
    uint64_t* full;
    int tile_bytes, stages;
};
__device__ __forceinline__ void fetch(const Ring& r, int i, const uint8_t* from, uint64_t pol) {      // by warp 0
    if (!elect_one()) return;
    const int s = i % r.stages;
    mbar_arrive_expect_tx(&r.full[s], uint32_t(r.tile_bytes));
    bulk_g2s_stream(r.data + size_t(s) * r.tile_bytes, from, uint32_t(r.tile_bytes), &r.full[s], pol);
}

__device__ __forceinline__ float silu_mul(float x, float up) {
    return __fmul_rn(__fdiv_rn(x, __fadd_rn(1.f, expf(-x))), up);
}

// ------------------------------------------------------------------ gate_up
template <typename IN, bool SPLIT, int GPW>
__global__ void __launch_bounds__(kThr, 1) moe_gate_up_kernel(const MoeSmallParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int CAP = SPLIT ? 4 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.w.H >> 7, GW = group_warps(G), NT = kWarps / GW, wg = warp & (GW - 1), wt = warp / GW;
    const int tiles = p.w.I >> 3;                       // 16-row tiles (8 gate, 8 up) of an expert
    const Ring ring = {smem, reinterpret_cast<uint64_t*>(smem + size_t(p.stages) * G * kGroupBytes), G * kGroupBytes, p.stages};
    float* part = reinterpret_cast<float*>(ring.full + p.stages + (p.stages & 1));   // [batch][GW][16][8]
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&ring.full[s], 1);
        fence_mbar_init();
    }
    pdl_wait();
    pdl_launch_dependents();                            // (after the wait: see the down kernel's prologue)
    const Plan pl = make_plan(p.ids, p.T * p.k, p.w.E, p.err, blockIdx.x == 0 && warp == 0);
    const long long W = (long long)__popc(pl.leaders) * tiles;
    const long long first = W * blockIdx.x / gridDim.x;
    const int n = int(W * (blockIdx.x + 1) / gridDim.x - first);
    const int u0 = int(first / tiles), r0 = int(first % tiles);
    // tile i of the sequence: row tile (r0 + i) % tiles of the (u0 + (r0 + i) / tiles)-th distinct expert
    auto expert = [&](int i) { return __shfl_sync(kFull, pl.id, nth_bit(pl.leaders, u0 + (r0 + i) / tiles)); };
    __syncthreads();
    const uint64_t pol = policy_evict_first();
    auto fill = [&](int from, int to) {                 // warp 0
        for (int i = from; i < to; ++i)
            fetch(ring, i, p.w.gate_up + (size_t(expert(i)) * tiles + (r0 + i) % tiles) * ring.tile_bytes, pol);
    };
    if (warp == 0) fill(0, min(n, p.stages));
    Frag f[GPW];
    int staged = -1;                                    // expert and pass whose rows the fragments hold
    for (int b0 = 0; b0 < n; b0 += p.batch) {
        const int nb = min(p.batch, n - b0);
        int passes = 0;
        for (int i = b0; i < b0 + nb; ++i) {
            const int used = __popc(__ballot_sync(kFull, pl.id == expert(i)));
            passes = max(passes, (used + CAP - 1) / CAP);
        }
        for (int ps = 0; ps < passes; ++ps) {
            for (int i = b0 + wt; i < b0 + nb; i += NT) {
                const int e = expert(i);
                const uint32_t places = __ballot_sync(kFull, pl.id == e);
                const int cols = __popc(places) - ps * CAP;
                if (cols <= 0 || wg >= G) continue;
                if (staged != e * kMoeSmallPlaces + ps) {
                    staged = e * kMoeSmallPlaces + ps;
                    const int col = SPLIT ? (lane >> 2) & 3 : lane >> 2;
                    const int place = col < cols ? nth_bit(places, ps * CAP + col) : -1;
#pragma unroll
                    for (int j = 0; j < GPW; ++j) {
                        const int grp = min(wg + j * kWarps, G - 1);
                        float v[32];
                        load_raw(v, static_cast<const IN*>(p.x) + size_t(max(place, 0) / p.k) * p.w.H + size_t(grp) * 128, place >= 0, lane);
                        make_frag<SPLIT>(f[j], v, lane);
                    }
                }
                const int s = i % p.stages;
                if (!__all_sync(kFull, mbar_wait(&ring.full[s], uint32_t((i / p.stages) & 1), p.err))) continue;
                const uint8_t* tile = ring.data + size_t(s) * ring.tile_bytes;
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < GPW; ++j)
                    if (wg + j * kWarps < G) block_product(tile + (wg + j * kWarps) * kGroupBytes, f[j], lane, acc);
                store_part8(part + (size_t(i - b0) * GW + wg) * 128, lane, acc);
            }
            __syncthreads();
            // two (row, column) of a tile a warp at a time, eight lanes for each row of its gate and its up: a lane sums two of the
            // (at most 16) partials, then the eight lanes' sums meet
            int done = 0;                               // (row, column) pairs of the tiles before
            for (int i = 0; i < nb; ++i) {
                const uint32_t places = __ballot_sync(kFull, pl.id == expert(b0 + i));
                const int cols = max(0, min(CAP, __popc(places) - ps * CAP));
                const int jt = (r0 + b0 + i) % tiles;
                for (int o = 2 * ((warp - (done >> 1)) & (kWarps - 1)); o < 8 * cols; o += 2 * kWarps) {
                    const int r = (o & 7) + (lane >> 4), c = o >> 3, w = lane & 7;
                    const float* at = part + size_t(i) * GW * 128 + (r + ((lane >> 3) & 1) * 8) * 8 + c;
                    float v = 0.f;
                    if (w < GW && w < G) v = SPLIT ? __fadd_rn(at[w * 128], at[w * 128 + 4]) : at[w * 128];
                    if (w + 8 < GW && w + 8 < G) {
                        const float* b = at + (w + 8) * 128;
                        v = __fadd_rn(v, SPLIT ? __fadd_rn(b[0], b[4]) : b[0]);
                    }
                    v = __fadd_rn(v, __shfl_xor_sync(kFull, v, 4));
                    v = __fadd_rn(v, __shfl_xor_sync(kFull, v, 2));
                    v = __fadd_rn(v, __shfl_xor_sync(kFull, v, 1));
                    const float up = __shfl_sync(kFull, v, lane + 8);
                    if ((lane & 15) == 0) p.act[size_t(nth_bit(places, ps * CAP + c)) * p.w.I + jt * 8 + r] = silu_mul(v, up);
                }
                done += 8 * cols;
            }
            __syncthreads();
        }
        if (warp == 0 && b0 + p.stages < n) {
            fence_proxy_async_smem();
            fill(b0 + p.stages, min(n, b0 + nb + p.stages));
        }
    }
}

// ------------------------------------------------------------------ down
template <typename OUT, bool SPLIT, int GPW>
__global__ void __launch_bounds__(kThr, 1) moe_down_kernel(const MoeSmallParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int CAP = SPLIT ? 4 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.w.I >> 7, GW = group_warps(G), NT = kWarps / GW, wg = warp & (GW - 1), wt = warp / GW;
    const int tiles = p.w.H >> 4, S = p.T * p.k;
    const Ring ring = {smem, reinterpret_cast<uint64_t*>(smem + size_t(p.stages) * G * kGroupBytes), G * kGroupBytes, p.stages};
    float* part = reinterpret_cast<float*>(ring.full + p.stages + (p.stages & 1));   // [place][GW][16]
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&ring.full[s], 1);
        fence_mbar_init();
    }
    // The ids were written before gate_up began (it waited for them before it let this kernel start), and the weights
    // are constant: both are read before the wait for gate_up's results.
    const Plan pl = make_plan(p.ids, S, p.w.E, p.err, false);
    const int n = __popc(pl.leaders);
    __syncthreads();
    const uint64_t pol = policy_evict_first();
    auto fill = [&](int from, int to) {                 // warp 0
        for (int i = from; i < to; ++i)
            fetch(ring, i, p.w.down + (size_t(__shfl_sync(kFull, pl.id, nth_bit(pl.leaders, i))) * tiles + blockIdx.x) * ring.tile_bytes,
                  pol);
    };
    if (warp == 0) fill(0, min(n, p.stages));
    pdl_wait();
    pdl_launch_dependents();
    for (int b0 = 0; b0 < n; b0 += p.batch) {
        const int nb = min(p.batch, n - b0);
        for (int i = b0 + wt; i < b0 + nb; i += NT) {
            if (wg >= G) break;
            const int e = __shfl_sync(kFull, pl.id, nth_bit(pl.leaders, i));
            const uint32_t places = __ballot_sync(kFull, pl.id == e);
            const int used = __popc(places);
            const int s = i % p.stages;
            if (!__all_sync(kFull, mbar_wait(&ring.full[s], uint32_t((i / p.stages) & 1), p.err))) continue;
            for (int c0 = 0; c0 < used; c0 += CAP) {
                const int col = SPLIT ? (lane >> 2) & 3 : lane >> 2;
                const int place = c0 + col < used ? nth_bit(places, c0 + col) : -1;
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < GPW; ++j) {
                    const int grp = wg + j * kWarps;
                    if (grp >= G) break;
                    Frag f;
                    float v[32];
                    load_raw(v, p.act + size_t(max(place, 0)) * p.w.I + size_t(grp) * 128, place >= 0, lane);
                    make_frag<SPLIT>(f, v, lane);
                    block_product(ring.data + size_t(s) * ring.tile_bytes + grp * kGroupBytes, f, lane, acc);
                }
                // columns 2t and 2t + 1 of rows g and g + 8; the remainders' columns add to their token's
                if (SPLIT) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[q] = __fadd_rn(acc[q], __shfl_xor_sync(kFull, acc[q], 2));
                }
                const int t = lane & 3, g = lane >> 2;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int c = 2 * t + q;
                    if (c < CAP && c0 + c < used) {
                        float* to = part + (size_t(nth_bit(places, c0 + c)) * GW + wg) * 16;
                        to[g] = acc[q];
                        to[g + 8] = acc[2 + q];
                    }
                }
            }
        }
        if (b0 + p.stages < n) {                        // the batch's stages are refilled once every warp is through
            __syncthreads();
            if (warp == 0) {
                fence_proxy_async_smem();
                fill(b0 + p.stages, min(n, b0 + nb + p.stages));
            }
        }
    }
    __syncthreads();
    // y[t, r] = sum over places in order, each the sum of its groups' partials
    OUT* y = static_cast<OUT*>(p.y);
    for (int o = threadIdx.x; o < p.T * 16; o += kThr) {
        const int t = o >> 4, r = o & 15;
        float v = 0.f;
        for (int j = 0; j < p.k; ++j) {
            const int place = t * p.k + j;
            const int e = p.ids[place];
            if (e < 0 || e >= p.w.E) continue;
            float a = 0.f;
            const int parts = GW < G ? GW : G;
            for (int w = 0; w < parts; ++w) a = __fadd_rn(a, part[(size_t(place) * GW + w) * 16 + r]);
            v = __fmaf_rn(p.weights[place], a, v);
        }
        const size_t at = size_t(t) * p.w.H + blockIdx.x * 16 + r;
        if constexpr (sizeof(OUT) == 4) {
            y[at] = p.resid ? __fadd_rn(y[at], v) : v;
        } else {
            y[at] = f32_to_bf16_rn(p.resid ? __fadd_rn(bf16_to_f32(y[at]), v) : v);
        }
    }
}

constexpr size_t kSmem = 227 * 1024;

const void* small_fn(bool down, bool bf16, int K) {
    const int gpw = K <= 2048 ? 1 : (K <= 4096 ? 2 : 4);
#define KMR_SMALL(kernel) \
    (gpw == 1 ? (bf16 ? (const void*)kernel<uint16_t, false, 1> : (const void*)kernel<float, true, 1>) \
     : gpw == 2 ? (bf16 ? (const void*)kernel<uint16_t, false, 2> : (const void*)kernel<float, true, 2>) \
                : (bf16 ? (const void*)kernel<uint16_t, false, 4> : (const void*)kernel<float, true, 4>))
    return down ? KMR_SMALL(moe_down_kernel) : KMR_SMALL(moe_gate_up_kernel);
#undef KMR_SMALL
}

// Ring of `most` tiles at the most, one batch where all of them fit and else two; `per_batch_tile` bytes for each tile of a batch
// and `fixed` bytes beside the tiles.
size_t plan_ring(int most, int K, size_t per_batch_tile, size_t fixed, int* stages, int* batch) {
    const size_t tile = size_t(K / 128) * kGroupBytes;
    auto bytes = [&](int st, int batch) { return st * tile + (st + (st & 1)) * 8 + batch * per_batch_tile + fixed; };
    *stages = *batch = most;
    if (bytes(most, most) <= kSmem) return bytes(most, most);
    int st = most + (most & 1);
    while (st > 2 && bytes(st, st / 2) > kSmem) st -= 2;
    *stages = st;
    *batch = st / 2;
    return bytes(st, st / 2);
}

}  // namespace

cudaError_t launch_moe_small(const MoeSmallParams& p, bool bf16, int sms, cudaStream_t st) {
    const int S = p.T * p.k, distinct = S < p.w.E ? S : p.w.E;
    MoeSmallParams q = p;
    // gate_up: at most `distinct` experts' tiles over the CTAs
    const long long tiles = (long long)distinct * (p.w.I / 8);
    const int grid = int(tiles < sms ? tiles : sms);
    const int G = p.w.H / 128;
    size_t smem = plan_ring(int((tiles + grid - 1) / grid), p.w.H, size_t(group_warps(G)) * 128 * 4, 0, &q.stages, &q.batch);
    cudaError_t e = launch_dependent(small_fn(false, bf16, p.w.H), dim3(grid), kThr, smem, 1, &q, st);
    if (e != cudaSuccess) return e;
    smem = plan_ring(distinct, p.w.I, 0, size_t(S) * group_warps(p.w.I / 128) * 16 * 4, &q.stages, &q.batch);
    return launch_dependent(small_fn(true, bf16, p.w.I), dim3(p.w.H / 16), kThr, smem, 1, &q, st);
}

cudaError_t moe_small_set_attributes() {
    for (int down = 0; down < 2; ++down)
        for (int b = 0; b < 2; ++b)
            for (int K = 2048; K <= kMoeMaxDim; K *= 2) {
                const cudaError_t e = cudaFuncSetAttribute(small_fn(down != 0, b != 0, K),
                                                           cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
                if (e != cudaSuccess) return e;
            }
    return cudaSuccess;
}

}  // namespace kmr
