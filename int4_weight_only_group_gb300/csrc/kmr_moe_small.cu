// Int4 experts for a few tokens: gate_up + SiLU * up, then down + the weighted sum, two launches.
//
//   act[t, j] = silu(gate_e x[t]) * (up_e x[t]),  y[t] = sum_j weights[t, j] * down_e act[t, j],  e = ids[t, j],
//   rows of gate_e, up_e, down_e: w = (q - 8) s + z in the KMR4 layout (include/kmr.h).
//
// What bounds it: every expert that a token is sent to is read once (1.0625 bytes per 2 weights), so HBM; for one
// token the latency of two dependent kernels.
//   * gate_up: (expert, 16-row tile) pairs are dealt out evenly over one CTA per SM, which fetches its tiles with
//     cp.async.bulk into a ring (of two halves, if they do not all fit).
//   * down: a CTA owns 16 output columns and fetches that tile of every expert used, so a token's sum is formed in
//     one place, in the order of its places, without atomics.  Its weights' copies start before its inputs are there.
//   * One warp plans the call: its lanes hold the (at most 32) expert ids, one match gives the distinct experts, and each lane
//     lists and fetches a tile.  The others meanwhile turn the rows into the MMAs' B fragments, once for the whole CTA.
//   * (tile, 128-input group) products are dealt to 32 warps, at most 16 to a tile, which then take the groups w, w + 16, ...
//     The codes are the A operand of mma.m16n8k16, as exact fp16 numbers; the inputs are B, scaled by a power of two per
//     (row, group): one column per token in bf16, two (the fp16 rounding and what it left) in fp32, so that products and
//     sums keep single precision.  Per group, y += (s D + z X) / sigma with D = sum (q - 8) x and X = sum x.
//   * partial sums meet in shared memory and are added in a fixed order that hangs on K alone: a token's result does not
//     change with the other tokens of the call.
// Measured: one token, 8 of 128 experts of 2048 x 768 (20 MB), fp32: 14.8 us, gate_up 8 (its first weights arrive after 3.4: the
// wait for the ids, the plan, HBM), down 5, launches; four tokens (32 places) 43 us.  With 16 warps, each of which planned
// the call, made its own fragments and divided for every tile: 25.7.  A product of one warp takes
// 1,400 cycles with 16 warps at work, for some 150 instructions and 8 MMAs (64 cycles): latency, which 32 warps hide better.
#include <cuda_fp16.h>

#include "kmr_int4_mma.cuh"
#include "kmr_moe.cuh"

namespace kmr {

namespace {

constexpr int kThr = 1024, kWarps = kThr / 32, kParts = 16;
constexpr uint32_t kFull = 0xffffffffu;

// ------------------------------------------------------------------ the call's plan, in a warp's registers
struct Plan {
    int id;                  // expert of place `lane`, or -1
    uint32_t same;           // the places of that expert
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
    pl.same = __match_any_sync(kFull, pl.id);
    pl.leaders = __ballot_sync(kFull, pl.id >= 0 && __ffs(pl.same) - 1 == lane);
    return pl;
}
// Most places of one expert.
__device__ __forceinline__ int most_places(const Plan& pl) {
    return int(__reduce_max_sync(kFull, pl.id >= 0 ? uint32_t(__popc(pl.same)) : 0u));
}
// The n-th set bit of m (the last one, if it has no more).
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

// A tile of the CTA's sequence: its number among the experts' tiles and within its expert, and its expert's places.
struct __align__(16) Tile {
    int from, row;
    uint32_t places;
    int unused;
};

// ------------------------------------------------------------------ operands
// The rows wait in shared memory as B fragments: per (row, group of 128) the four quarters t of the lanes, each the 16 registers of
// its 8 steps (inputs 8 i + 2 t and + 1 in register i), in 16-byte pieces that two quarters exchange so that a load meets no
// bank twice; SPLIT: the remainders behind them.  An item of zeros stands last.  Beside them, for each term, its sum and 1 / sigma,
// as the codes' 2^-9 needs them.
template <bool SPLIT>
constexpr int kItemBytes = SPLIT ? 512 : 256;
template <typename IN, bool SPLIT>
__device__ __forceinline__ void stage_rows(uint8_t* to, float4* fold, const IN* x, int items) {
    const int lane = threadIdx.x & 31, i = lane & 15;      // half a warp to an item, a lane its inputs 8 i .. 8 i + 7: register i of each quarter
    if (threadIdx.x >= kThr - 32) {
        reinterpret_cast<uint4*>(to + size_t(items) * kItemBytes<SPLIT>)[lane & (kItemBytes<SPLIT> / 16 - 1)] = make_uint4(0u, 0u, 0u, 0u);
        fold[items] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i0 = (threadIdx.x >> 5) * 2; i0 < items; i0 += kWarps * 2) {
        const int item = min(i0 + (lane >> 4), items - 1);
        float r[8];
        if constexpr (sizeof(IN) == 4) {
            const float4* src = reinterpret_cast<const float4*>(x + size_t(item) * 128 + i * 8);
            const float4 v0 = __ldcg(src), v1 = __ldcg(src + 1);
            r[0] = v0.x, r[1] = v0.y, r[2] = v0.z, r[3] = v0.w, r[4] = v1.x, r[5] = v1.y, r[6] = v1.z, r[7] = v1.w;
        } else {
            const uint4 v = __ldcg(reinterpret_cast<const uint4*>(x + size_t(item) * 128 + i * 8));
            r[0] = bf16_lo(v.x), r[1] = bf16_hi(v.x), r[2] = bf16_lo(v.y), r[3] = bf16_hi(v.y);
            r[4] = bf16_lo(v.z), r[5] = bf16_hi(v.z), r[6] = bf16_lo(v.w), r[7] = bf16_hi(v.w);
        }
        uint32_t m = 0u;                                   // (bits of non-negative numbers order like integers, NaN above all)
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(fabsf(r[q])));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        float sig, isg;
        pow2_scale(m, sig, isg);
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = __fmul_rn(r[q], sig);
        float X[2] = {0.f, 0.f};
        uint8_t* dst = to + size_t(item) * kItemBytes<SPLIT> + (i & 3) * 4;
#pragma unroll
        for (int term = 0; term < (SPLIT ? 2 : 1); ++term) {
            float part[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const __half2 h = __floats2half2_rn(r[2 * t], r[2 * t + 1]);
                const float2 f = __half22float2(h);
                part[t] = __fadd_rn(f.x, f.y);
                r[2 * t] = __fsub_rn(r[2 * t], f.x);
                r[2 * t + 1] = __fsub_rn(r[2 * t + 1], f.y);
                *reinterpret_cast<__half2*>(dst + term * 256 + t * 64 + (((i >> 2) ^ (t >> 1)) << 4)) = h;
            }
            X[term] = __fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3]));
        }
        // the lower lanes of the half sum the first terms, the upper ones the remainders
        float sum = __fadd_rn(i < 8 ? X[0] : X[1], __shfl_xor_sync(kFull, i < 8 ? X[1] : X[0], 8));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
        if ((i & 7) == 0)
            reinterpret_cast<float2*>(fold + item)[i >> 3] = make_float2(sum * 0x1p-9f, isg * 0x1p9f);      // (isg is 2^114 at the most)
    }
}

// B fragments of one 128-input group of up to 8 (SPLIT: 4) rows for this lane, and the group's fold constants.
struct Frag {
    uint32_t b[16];
    float X0, is0, X1, is1;  // of columns 2t and 2t + 1: sum of the staged values 2^-9, 2^9 / sigma
};
// Column lane / 4 takes staged item `item` (SPLIT: columns 4..7 its remainders).
template <bool SPLIT>
__device__ __forceinline__ void load_frag(Frag& f, const uint8_t* staged, const float4* fold, int item, int lane) {
    const int t = lane & 3, rest = SPLIT ? lane >> 4 : 0;
    const uint8_t* at = staged + size_t(item) * kItemBytes<SPLIT> + rest * 256 + t * 64;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(at + ((c ^ (t >> 1)) << 4));
        f.b[4 * c] = v.x;
        f.b[4 * c + 1] = v.y;
        f.b[4 * c + 2] = v.z;
        f.b[4 * c + 3] = v.w;
    }
    const float2 k = reinterpret_cast<const float2*>(fold + item)[rest];
    f.X0 = __shfl_sync(kFull, k.x, 8 * t);
    f.X1 = __shfl_sync(kFull, k.x, 8 * t + 4);
    f.is0 = __shfl_sync(kFull, k.y, 8 * t);
    f.is1 = __shfl_sync(kFull, k.y, 8 * t + 4);
}

// acc (rows g and g + 8, columns 2t and 2t + 1) += one (16-row tile, 128-input group) block times the fragments.
// A code's four bits are themselves an fp16, q 2^-24 (rows g + 8: 16 q 2^-24), so that half an AND and half an HFMA2 give (q - 8)
// 2^-9.  (The MMA takes the subnormal numbers as they are, too, but aligns their products as if they were 2^10 larger: 2.2e-6
// of the result instead of 4e-7.)
__device__ __forceinline__ void block_product(const uint8_t* gb, const Frag& f, int lane, float (&acc)[4]) {
    const int g = lane >> 2;
    const __half2 m8 = __float2half2_rn(-0x1p-6f), up0 = __float2half2_rn(0x1p15f), up1 = __float2half2_rn(0x1p11f);
    auto codes = [&](uint32_t v, __half2 up) {
        const __half2 a = __hfma2(*reinterpret_cast<const __half2*>(&v), up, m8);
        return *reinterpret_cast<const uint32_t*>(&a);
    };
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
            mma16816(d[ks & 1], codes(w & 0x000F000Fu, up0), codes(w & 0x00F000F0u, up1), codes(w2 & 0x000F000Fu, up0),
                     codes(w2 & 0x00F000F0u, up1), f.b[blk * 8 + 2 * ks], f.b[blk * 8 + 2 * ks + 1]);
        }
    }
    auto fold = [](uint32_t sz, float D, float X, float is, float a) {
        return __fmaf_rn(__fmaf_rn(bf16_lo(sz), D, __fmul_rn(bf16_hi(sz), X)), is, a);
    };
    const uint32_t sz0 = *reinterpret_cast<const uint32_t*>(gb + 1024 + g * 4);
    const uint32_t sz1 = *reinterpret_cast<const uint32_t*>(gb + 1024 + (g + 8) * 4);
    acc[0] = fold(sz0, __fadd_rn(d[0][0], d[1][0]), f.X0, f.is0, acc[0]);
    acc[1] = fold(sz0, __fadd_rn(d[0][1], d[1][1]), f.X1, f.is1, acc[1]);
    acc[2] = fold(sz1, __fadd_rn(d[0][2], d[1][2]), f.X0, f.is0, acc[2]);
    acc[3] = fold(sz1, __fadd_rn(d[0][3], d[1][3]), f.X1, f.is1, acc[3]);
}

// The columns' sums of one warp's groups w, w + 16, ... of a tile: acc (rows g and g + 8, columns 2t and 2t + 1).  `row` is the
// staged row of column lane / 4 (of 8, SPLIT: of 4 and again), `rows` (zeros) for none; SPLIT: the remainders' columns are
// added to their rows'.
template <bool SPLIT>
__device__ __forceinline__ void tile_product(const uint8_t* tile, const uint8_t* staged, const float4* fold, int row, int rows, int G,
                                             int w, int lane, float (&acc)[4]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = 0.f;
    for (int grp = w; grp < G; grp += kParts) {
        Frag f;
        load_frag<SPLIT>(f, staged, fold, row * G + (row < rows ? grp : 0), lane);
        block_product(tile + grp * kGroupBytes, f, lane, acc);
    }
    if (SPLIT) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = __fadd_rn(acc[q], __shfl_xor_sync(kFull, acc[q], 2));
    }
}
// (tile i, part w) of a batch in the order of the warps, one for each at a time, without a division for each.
struct Turn {
    int i, w;
};
__device__ __forceinline__ Turn first_turn(int warp, int P) { return {warp / P, warp % P}; }
__device__ __forceinline__ void next_turn(Turn& t, int P, int di, int dw) {
    t.i += di;
    t.w += dw;
    if (t.w >= P) {
        t.w -= P;
        ++t.i;
    }
}

// ------------------------------------------------------------------ the ring of tiles
// Tile i of the CTA's sequence lives in stage i % stages; the tiles of a batch (half the ring) are fetched together
// once the batch before the previous one has been used up.
struct Ring {
    uint8_t* data;
    uint64_t* full;
    int tile_bytes, stages;
};
__device__ __forceinline__ void fetch(const Ring& r, int i, const uint8_t* from, uint64_t pol) {      // by one lane
    const int s = i % r.stages;
    mbar_arrive_expect_tx(&r.full[s], uint32_t(r.tile_bytes));
    bulk_g2s_stream(r.data + size_t(s) * r.tile_bytes, from, uint32_t(r.tile_bytes), &r.full[s], pol);
}
// Where everything lies in shared memory: ring, barriers, tile list, fold constants, staged rows, partial sums.
__host__ __device__ constexpr int parts_of(int G) { return G < kParts ? G : kParts; }
struct Layout {
    size_t full, list, fold, staged, part, total;
};
__host__ __device__ inline Layout layout_of(bool down, bool split, int K, int rows, int stages, int batch, int tiles) {
    const int G = K >> 7;
    Layout l;
    l.full = size_t(stages) * G * kGroupBytes;
    l.list = l.full + size_t(stages + (stages & 1)) * 8;
    l.fold = l.list + size_t(tiles) * sizeof(Tile);
    l.staged = l.fold + (size_t(rows) * G + 1) * 16;    // (one item more, of zeros)
    l.part = l.staged + (size_t(rows) * G + 1) * (split ? 512 : 256);
    // gate_up: [batch][part][16 rows][columns]; down: [place][part][16 rows]
    l.total = l.part + size_t(down ? rows : batch * (split ? 4 : 8)) * parts_of(G) * 64;
    return l;
}

__device__ __forceinline__ float silu_mul(float x, float up) {
    return __fmul_rn(__fdiv_rn(x, __fadd_rn(1.f, expf(-x))), up);
}

// ------------------------------------------------------------------ gate_up
template <typename IN, bool SPLIT>
__global__ void __launch_bounds__(kThr, 1) moe_gate_up_kernel(const MoeSmallParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int most, n_tiles;
    constexpr int CAP = SPLIT ? 4 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.w.H >> 7, P = parts_of(G);
    const int tiles = p.w.I >> 3;                       // 16-row tiles (8 gate, 8 up) of an expert
    const Layout l = layout_of(false, SPLIT, p.w.H, p.T, p.stages, p.batch, p.list);
    const Ring ring = {smem, reinterpret_cast<uint64_t*>(smem + l.full), G * kGroupBytes, p.stages};
    Tile* list = reinterpret_cast<Tile*>(smem + l.list);
    float4* fold = reinterpret_cast<float4*>(smem + l.fold);
    uint8_t* staged = smem + l.staged;
    float* part = reinterpret_cast<float*>(smem + l.part);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&ring.full[s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_launch_dependents();                            // (after the wait: see the down kernel's prologue)
    const uint64_t pol = policy_evict_first();
    if (warp == 0) {
        const Plan pl = make_plan(p.ids, p.T * p.k, p.w.E, p.err, blockIdx.x == 0);
        // (products with the rounded-up 2^32 / d for divisions by d: exact, n * d stays below 2^32)
        const int W = __popc(pl.leaders) * tiles, per = __umulhi(W, p.by_grid), more = W - per * int(gridDim.x);
        const int first = int(blockIdx.x) * per + min(int(blockIdx.x), more), mine = per + (int(blockIdx.x) < more ? 1 : 0);
        const int u0 = __umulhi(first, p.by_tiles), r0 = first - u0 * tiles;
        for (int i0 = 0; i0 < mine; i0 += 32) {         // tile i: row tile (r0 + i) % tiles of a distinct expert
            const int i = min(i0 + lane, mine - 1), u = __umulhi(r0 + i, p.by_tiles), at = nth_bit(pl.leaders, u0 + u);
            Tile t;
            t.row = r0 + i - u * tiles;
            t.from = __shfl_sync(kFull, pl.id, at) * tiles + t.row;
            t.places = __shfl_sync(kFull, pl.same, at);
            t.unused = 0;
            if (i0 + lane < mine) {
                list[i] = t;
                if (i < p.stages) fetch(ring, i, p.w.gate_up + size_t(t.from) * ring.tile_bytes, pol);
            }
        }
        const int m = most_places(pl);
        if (lane == 0) {
            most = m;
            n_tiles = mine;
        }
    }
    stage_rows<IN, SPLIT>(staged, fold, static_cast<const IN*>(p.x), p.T * G);
    const int token = lane / p.k;                       // of place `lane`
    __syncthreads();
    const int n = n_tiles, columns = min(most, CAP), di = kWarps / P, dw = kWarps % P;
    const Turn t0 = first_turn(warp, P);
    bool ok = true;                                     // (a wait that ran out: no other is made)
    for (int b0 = 0, s0 = 0, phase = 0; b0 < n; b0 += p.batch) {
        const int nb = min(p.batch, n - b0);
        for (int c0 = 0; c0 < most; c0 += CAP) {
            for (Turn t = t0; t.i < nb; next_turn(t, P, di, dw)) {
                const uint32_t places = list[b0 + t.i].places;
                const int cols = __popc(places) - c0, col = SPLIT ? (lane >> 2) & 3 : lane >> 2;
                if (cols <= 0) continue;
                int at = 0;                             // column's token
                if (p.T > 1) at = __shfl_sync(kFull, token, nth_bit(places, c0 + min(col, cols - 1)));
                if (!(ok = ok && __all_sync(kFull, mbar_wait(&ring.full[s0 + t.i], uint32_t(phase), p.err)))) continue;
                float acc[4];
                tile_product<SPLIT>(ring.data + size_t(s0 + t.i) * ring.tile_bytes, staged, fold, col < cols ? at : p.T, p.T, G, t.w, lane, acc);
                const int g = lane >> 2, c = 2 * (lane & 3);
                if (c < CAP) {
                    float* to = part + ((t.i * P + t.w) * 16 + g) * CAP + c;
                    *reinterpret_cast<float2*>(to) = make_float2(acc[0], acc[1]);
                    *reinterpret_cast<float2*>(to + 8 * CAP) = make_float2(acc[2], acc[3]);
                }
            }
            __syncthreads();
            // four outputs of a (tile, column) a warp at a time, four lanes for each row of its gate and its up: a lane sums four of
            // the (at most 16) partials, then the four lanes' sums meet
            for (int c = 0; c < columns; ++c) {
                for (int o = warp; o < nb * 2; o += kWarps) {
                    const Tile t = list[b0 + (o >> 1)];
                    if (c0 + c >= __popc(t.places)) continue;
                    const int r = (o & 1) * 4 + ((lane >> 2) & 3), w = lane & 3;
                    const float* at = part + ((o >> 1) * P * 16 + r + (lane >> 4) * 8) * CAP + c;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = w + 4 * q < P ? at[(w + 4 * q) * 16 * CAP] : 0.f;
                    float a = __fadd_rn(__fadd_rn(v[0], v[1]), __fadd_rn(v[2], v[3]));
                    a = __fadd_rn(a, __shfl_xor_sync(kFull, a, 1));
                    a = __fadd_rn(a, __shfl_xor_sync(kFull, a, 2));
                    const float up = __shfl_sync(kFull, a, (lane + 16) & 31);
                    const int place = c0 + c == 0 ? __ffs(t.places) - 1 : nth_bit(t.places, c0 + c);
                    if (lane < 16 && w == 0) p.act[size_t(place) * p.w.I + t.row * 8 + r] = silu_mul(a, up);
                }
            }
            if (c0 + CAP >= most && b0 + nb >= n) return;
            __syncthreads();
        }
        if (warp == 0) {
            fence_proxy_async_smem();
            for (int i = b0 + p.stages + lane; i < min(n, b0 + nb + p.stages); i += 32)
                fetch(ring, i, p.w.gate_up + size_t(list[i].from) * ring.tile_bytes, pol);
        }
        s0 += p.batch;
        if (s0 == p.stages) {
            s0 = 0;
            phase ^= 1;
        }
    }
}

// ------------------------------------------------------------------ down
template <typename OUT, bool SPLIT>
__global__ void __launch_bounds__(kThr, 1) moe_down_kernel(const MoeSmallParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int ids[32], experts;
    __shared__ float weights[32];
    constexpr int CAP = SPLIT ? 4 : 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = p.w.I >> 7, P = parts_of(G);
    const int tiles = p.w.H >> 4, S = p.T * p.k;
    const Layout l = layout_of(true, SPLIT, p.w.I, S, p.stages, p.batch, p.list);
    const Ring ring = {smem, reinterpret_cast<uint64_t*>(smem + l.full), G * kGroupBytes, p.stages};
    Tile* list = reinterpret_cast<Tile*>(smem + l.list);
    float4* fold = reinterpret_cast<float4*>(smem + l.fold);
    uint8_t* staged = smem + l.staged;
    float* part = reinterpret_cast<float*>(smem + l.part);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) mbar_init(&ring.full[s], 1);
        fence_mbar_init();
    }
    __syncwarp();
    // The ids and weights were written before gate_up began (it waited for them before it let this kernel start), and the
    // experts are constant: they are read before the wait for gate_up's results.
    const uint64_t pol = policy_evict_first();
    if (warp == 0) {
        const Plan pl = make_plan(p.ids, S, p.w.E, p.err, false);
        const int distinct = __popc(pl.leaders), at = nth_bit(pl.leaders, lane) & 31;
        Tile t;
        t.row = blockIdx.x;
        t.from = __shfl_sync(kFull, pl.id, at) * tiles + t.row;
        t.places = __shfl_sync(kFull, pl.same, at);
        t.unused = 0;
        if (lane < distinct) {
            list[lane] = t;
            if (lane < p.stages) fetch(ring, lane, p.w.down + size_t(t.from) * ring.tile_bytes, pol);
        }
        ids[lane] = pl.id;
        weights[lane] = lane < S ? p.weights[lane] : 0.f;
        if (lane == 0) experts = distinct;
    }
    pdl_wait();
    pdl_launch_dependents();
    OUT* y = static_cast<OUT*>(p.y);
    const size_t out = size_t(threadIdx.x >> 4) * p.w.H + blockIdx.x * 16 + (threadIdx.x & 15);     // (T * 16 <= kThr)
    const bool mine = int(threadIdx.x) < p.T * 16;
    float before = 0.f;
    if (mine && p.resid) {
        if constexpr (sizeof(OUT) == 4) before = y[out];
        else before = bf16_to_f32(y[out]);
    }
    stage_rows<float, SPLIT>(staged, fold, p.act, S * G);
    __syncthreads();
    const int n = experts, di = kWarps / P, dw = kWarps % P;
    const Turn t0 = first_turn(warp, P);
    bool ok = true;                                     // (a wait that ran out: no other is made)
    for (int b0 = 0, s0 = 0, phase = 0; b0 < n; b0 += p.batch) {
        const int nb = min(p.batch, n - b0);
        for (Turn t = t0; t.i < nb; next_turn(t, P, di, dw)) {
            const uint32_t places = list[b0 + t.i].places;
            const int used = __popc(places);
            if (!(ok = ok && __all_sync(kFull, mbar_wait(&ring.full[s0 + t.i], uint32_t(phase), p.err)))) continue;
            for (int c0 = 0; c0 < used; c0 += CAP) {
                const int col = SPLIT ? (lane >> 2) & 3 : lane >> 2;
                int place = col == 0 ? __ffs(places) - 1 : -1;
                if (used > 1) place = c0 + col < used ? nth_bit(places, c0 + col) : -1;
                float acc[4];
                tile_product<SPLIT>(ring.data + size_t(s0 + t.i) * ring.tile_bytes, staged, fold, place < 0 ? S : place, S, G, t.w, lane, acc);
                const int g = lane >> 2;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int to = __shfl_sync(kFull, place, 8 * (lane & 3) + 4 * q);      // of column 2t + q
                    if (to >= 0 && 2 * (lane & 3) < CAP) {
                        part[(to * P + t.w) * 16 + g] = acc[q];
                        part[(to * P + t.w) * 16 + g + 8] = acc[2 + q];
                    }
                }
            }
        }
        if (b0 + p.stages < n) {                        // the batch's stages are refilled once every warp is through
            __syncthreads();
            if (warp == 0) {
                fence_proxy_async_smem();
                for (int i = b0 + p.stages + lane; i < min(n, b0 + nb + p.stages); i += 32)
                    fetch(ring, i, p.w.down + size_t(list[i].from) * ring.tile_bytes, pol);
            }
        }
        s0 += p.batch;
        if (s0 == p.stages) {
            s0 = 0;
            phase ^= 1;
        }
    }
    __syncthreads();
    // y[t, r] = sum over places in order, each the sum of its parts in order
    for (int o = threadIdx.x; o < S * 16; o += kThr) {
        if (ids[o >> 4] < 0) continue;
        float* at = part + (o >> 4) * P * 16 + (o & 15);
        float a = at[0];
#pragma unroll 4
        for (int w = 1; w < P; ++w) a = __fadd_rn(a, at[w * 16]);
        at[0] = a;
    }
    __syncthreads();
    if (!mine) return;
    float v = 0.f;
#pragma unroll 4
    for (int j = 0; j < p.k; ++j) {
        const int place = int(threadIdx.x >> 4) * p.k + j;
        if (ids[place] >= 0) v = __fmaf_rn(weights[place], part[place * P * 16 + (threadIdx.x & 15)], v);
    }
    if (p.resid) v = __fadd_rn(before, v);
    if constexpr (sizeof(OUT) == 4) y[out] = v;
    else y[out] = f32_to_bf16_rn(v);
}

constexpr size_t kSmem = 227 * 1024 - 512;               // (less the kernels' static variables)

const void* small_fn(bool down, bool bf16) {
    if (down) return bf16 ? (const void*)moe_down_kernel<uint16_t, false> : (const void*)moe_down_kernel<float, true>;
    return bf16 ? (const void*)moe_gate_up_kernel<uint16_t, false> : (const void*)moe_gate_up_kernel<float, true>;
}

// Ring of `most` tiles at the most, one batch where all of them fit and else two.
size_t plan_ring(bool down, bool bf16, int K, int rows, int most, int* stages, int* batch) {
    auto bytes = [&](int st, int b) { return layout_of(down, !bf16, K, rows, st, b, most).total; };
    *stages = *batch = most;
    if (bytes(most, most) <= kSmem) return bytes(most, most);
    int st = most + (most & 1);
    while (st > 2 && bytes(st, st / 2) > kSmem) st -= 2;
    *stages = st;
    *batch = st / 2;
    return bytes(st, st / 2);
}
int distinct_of(const MoeView& w, int S) { return S < w.E ? S : w.E; }
int gate_tiles(const MoeView& w, int S, int ctas) {      // the longest sequence of a CTA
    const int all = distinct_of(w, S) * (w.I / 8);
    return all <= ctas ? 1 : (all + ctas - 1) / ctas;
}

}  // namespace

// (a larger call, of weights or of tokens, is quicker in the grouped form, whose kernels cost 22 us in any case but read the
// weights faster: 16 experts of 4096 x 2048, two a token, fp32: four tokens 48 us against 52, five 65 against 53; 64 experts of
// 2048 x 768, one a token, bf16: 16 tokens 27 against 31, 32 tokens 49 against 34)
bool moe_small_fits(const MoeView& w, bool bf16, int T, int k) {
    const int S = T * k;
    int st, b;
    if (S > kMoeSmallPlaces || T > kMoeSmallTokens || (long long)S * w.H * w.I * 3 > kMoeSmallWeights) return false;
    return plan_ring(false, bf16, w.H, T, gate_tiles(w, S, kMoeSmallCtas), &st, &b) <= kSmem &&
           plan_ring(true, bf16, w.I, S, distinct_of(w, S), &st, &b) <= kSmem;
}

cudaError_t launch_moe_small(const MoeSmallParams& p, bool bf16, int sms, cudaStream_t st) {
    const int S = p.T * p.k, all = distinct_of(p.w, S) * (p.w.I / 8);
    MoeSmallParams q = p;
    const int ctas = sms > kMoeSmallCtas ? sms : kMoeSmallCtas;      // (a CTA waits for no other: fewer SMs run them in turn)
    const int grid = all < ctas ? all : ctas;
    q.list = gate_tiles(p.w, S, ctas);
    q.by_tiles = uint32_t((0x100000000ull + p.w.I / 8 - 1) / (p.w.I / 8));
    q.by_grid = uint32_t((0x100000000ull + grid - 1) / grid);
    size_t smem = plan_ring(false, bf16, p.w.H, p.T, q.list, &q.stages, &q.batch);
    cudaError_t e = launch_dependent(small_fn(false, bf16), dim3(grid), kThr, smem, 1, &q, st);
    if (e != cudaSuccess) return e;
    q.list = distinct_of(p.w, S);
    smem = plan_ring(true, bf16, p.w.I, S, q.list, &q.stages, &q.batch);
    return launch_dependent(small_fn(true, bf16), dim3(p.w.H / 16), kThr, smem, 1, &q, st);
}

cudaError_t moe_small_set_attributes() {
    for (int f = 0; f < 4; ++f) {
        const cudaError_t e = cudaFuncSetAttribute(small_fn((f & 1) != 0, (f & 2) != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kmr
