// Writes of the 4-bit KV cache: new tokens (q/k RMSNorm, M-RoPE and quantisation in one pass),
// conversions from and to a bf16 cache, and eviction into another row.  The format is in kmr_kv4.cuh.
//
// All are bound by HBM where there is enough to move; measured at d = 128, group 32, 8 KV heads, against the measured
// copy rate of 6.75 TB/s:
//   append, a prompt of 8192 (16 query heads): 37.7 us for 212 MB, 5.6 TB/s (0.83); one token: 3.2 us, most of it launch
//   bf16 -> 4 bits, 16 rows of up to 8192 (96 thousand positions): 86.6 us for 516 MB, 6.0 TB/s (0.88)
//   4 bits -> bf16, the same: 82.1 us, 6.3 TB/s (0.93)
//   evict, 16 rows of up to 8192 to 2048: 29.2 us for 90 MB (3.1 TB/s, 0.46); the selection alone (2 kept) takes 10.7 us
#include <type_traits>

#include "kmr_kv4.cuh"

namespace kmr {
namespace {

constexpr int kThr = 128;

// ------------------------------------------------------------------ a vector on four lanes
// Every kernel here holds a vector of D dims on four neighbouring lanes: lane l has dims 32 b + 8 l .. + 7 of each
// of the NB = D / 32 blocks.  That is one 16-byte piece of a bf16 row per block, both halves of every rotation
// pair (dim i + D / 2 is block b + NB / 2), and 4 NB contiguous bytes of a row of codes: lane l's words of
// a K row, lanes 2 l and 2 l + 1's units of a V row.

__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// (w << 8) | codes hi, lo held within 0..15
__device__ __forceinline__ uint32_t pack_code(int hi, int lo, uint32_t w) {
    uint32_t r;
    asm("cvt.pack.sat.u4.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(hi), "r"(lo), "r"(w));
    return r;
}

// Extremes of a vector's NG groups over its four lanes, as v = min over lanes of each; lane l ends with group l
// (NG 4), l / 2 (NG 2) or the only one: each lane then works out one group's scale instead of all of them.
template <int NG, typename T, typename Min>
__device__ __forceinline__ T lane_group_min(const T (&v)[NG], int l, Min&& mn) {
    T u[NG > 1 ? NG / 2 : 1];
    if constexpr (NG == 1) {
        u[0] = mn(v[0], T(__shfl_xor_sync(0xffffffffu, v[0], 2)));
    } else {
        const bool up = (l & 2) != 0;
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) {
            const T keep = up ? v[i + NG / 2] : v[i], send = up ? v[i] : v[i + NG / 2];
            u[i] = mn(keep, T(__shfl_xor_sync(0xffffffffu, send, 2)));
        }
    }
    if constexpr (NG < 4) return mn(u[0], T(__shfl_xor_sync(0xffffffffu, u[0], 1)));
    const bool odd = (l & 1) != 0;
    const T keep = odd ? u[NG / 2 - 1] : u[0], send = odd ? u[0] : u[NG / 2 - 1];
    return mn(keep, T(__shfl_xor_sync(0xffffffffu, send, 1)));
}

// A group's word (z, s) and reciprocal from its extremes.  s = bf16((hi - lo) / 15), 0 below 2^-126 (its reciprocal would
// leave the normal range); z = bf16(lo).  A group that holds a NaN or an infinity, or whose range overflows, stores
// s = 0 and z = NaN (kBadWord): it reads back as NaN.  The quotient by 15 is the correctly rounded one (as below).
constexpr uint32_t kBadWord = 0x7FC0u;
__device__ __forceinline__ uint32_t group_word(float lo, float hi, float& r) {
    const float range = __fsub_rn(hi, lo), fifteenth = 1.f / 15.f;
    const float s0 = __fmul_rn(range, fifteenth);
    const float s1 = __fmaf_rn(__fmaf_rn(-15.f, s0, range), fifteenth, s0);
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(s1), "f"(lo));
    if (u < 0x00800000u) u &= 0xFFFFu;
    if ((u & 0x7F800000u) == 0x7F800000u || (u & 0x7F80u) == 0x7F80u) u = kBadWord;
    const float s = kv4_s(u);
    r = 0.f;
    if (s > 0.f) {
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
        r = __fmaf_rn(__fmaf_rn(-s, r, 1.f), r, r);
    }
    return u;
}

// The lane's codes (word k: dims 32 k + 8 l + i in nibble i) under the vector's group words: c = rint((x - z) / s)
// within 0..15, 0 where s is 0.  The quotient is the correctly rounded one (Markstein 1990: with r near 1 / s,
// q0 = rn(a r), e = a - q0 s exactly, rn(q0 + e r)), so a value half-way between two codes is seen as half-way and goes
// to the even one.  own, r: the word and reciprocal of the lane's group (lane_group_min).
template <int D, int G>
__device__ __forceinline__ void code_words(const float (&x)[D / 32][8], uint32_t own, float own_r, uint32_t (&w)[D / 32]) {
    constexpr int NG = D / G, BPG = G / 32;
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        const uint32_t u = NG == 1 ? own : __shfl_sync(0xffffffffu, own, gr * (4 / NG), 4);
        const float r = NG == 1 ? own_r : __shfl_sync(0xffffffffu, own_r, gr * (4 / NG), 4);
        const float s = kv4_s(u), z = kv4_z(u);
#pragma unroll
        for (int kb = 0; kb < BPG; ++kb) {
            const int k = gr * BPG + kb;
            int c[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float a = __fsub_rn(x[k][i], z);
                const float q0 = __fmul_rn(a, r);
                const float q = __fmaf_rn(__fmaf_rn(-q0, s, a), r, q0);
                // 1.5 * 2^23 + q rounds q to a whole number (half to even) in the low bits
                c[i] = __float_as_int(__fadd_rn(q, 12582912.f)) - 0x4B400000;
            }
            uint32_t v = pack_code(c[7], c[6], 0u);
            v = pack_code(c[5], c[4], v);
            v = pack_code(c[3], c[2], v);
            v = pack_code(c[1], c[0], v);
            w[k] = u == kBadWord ? 0u : v;
        }
    }
}
// Codes of a vector and the word of the lane's group.
template <int D, int G>
__device__ __forceinline__ uint32_t quantize(const float (&x)[D / 32][8], int l, uint32_t (&w)[D / 32]) {
    constexpr int NG = D / G, BPG = G / 32;
    float lo[NG], hi[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        lo[gr] = hi[gr] = x[gr * BPG][0];
#pragma unroll
        for (int k = 0; k < BPG; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo[gr] = min_nan(lo[gr], x[gr * BPG + k][i]);
                hi[gr] = max_nan(hi[gr], x[gr * BPG + k][i]);
            }
    }
    const float mylo = lane_group_min<NG>(lo, l, [](float a, float b) { return min_nan(a, b); });
    const float myhi = lane_group_min<NG>(hi, l, [](float a, float b) { return max_nan(a, b); });
    float r;
    const uint32_t own = group_word(mylo, myhi, r);
    code_words<D, G>(x, own, r, w);
    return own;
}
// The same of bf16 pairs, whose extremes are found two at a time and cross the lanes as one pair (lo, -hi).
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int D, int G>
__device__ __forceinline__ uint32_t quantize_bf16(const uint4 (&raw)[D / 32], int l, uint32_t (&w)[D / 32]) {
    constexpr int NB = D / 32, NG = D / G, BPG = G / 32;
    float x[NB][8];
    uint32_t ends[NG];
#pragma unroll
    for (int gr = 0; gr < NG; ++gr) {
        uint32_t lo2 = raw[gr * BPG].x, hi2 = lo2;
#pragma unroll
        for (int kb = 0; kb < BPG; ++kb) {
            const int k = gr * BPG + kb;
            const uint32_t v[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo2 = min2_nan(lo2, v[i]);
                asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi2) : "r"(v[i]));
                x[k][2 * i] = bf16_lo(v[i]);
                x[k][2 * i + 1] = bf16_hi(v[i]);
            }
        }
        hi2 ^= 0x80008000u;
        ends[gr] = min2_nan(__byte_perm(lo2, hi2, 0x5410), __byte_perm(lo2, hi2, 0x7632));
    }
    const uint32_t mine = lane_group_min<NG>(ends, l, [](uint32_t a, uint32_t b) { return min2_nan(a, b); });
    float r;
    const uint32_t own = group_word(bf16_lo(mine), -bf16_hi(mine), r);
    code_words<D, G>(x, own, r, w);
    return own;
}

// Words of a lane <-> its 4 NB bytes of a row of codes.
template <int NB>
__device__ __forceinline__ void store_codes(uint8_t* row, const uint32_t (&w)[NB], bool key, int l) {
    uint32_t v[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) v[i] = w[i];
    if (!key) {
        // units of dims 8 l .. 8 l + 3 of all blocks, then those of 8 l + 4 .. 8 l + 7
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            v[i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
            v[NB / 2 + i] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
        }
    }
    if constexpr (NB == 4)
        *reinterpret_cast<uint4*>(row + l * 16) = make_uint4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2*>(row + l * 8) = make_uint2(v[0], v[1]);
}
template <int NB>
__device__ __forceinline__ void load_codes(const uint8_t* row, uint32_t (&w)[NB], bool key, int l) {
    uint32_t v[NB];
    if constexpr (NB == 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(row + l * 16);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(row + l * 8);
        v[0] = u.x; v[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) w[i] = v[i];
    if (!key) {
#pragma unroll
        for (int i = 0; i < NB / 2; ++i) {
            w[2 * i] = __byte_perm(v[i], v[NB / 2 + i], 0x5410);
            w[2 * i + 1] = __byte_perm(v[i], v[NB / 2 + i], 0x7632);
        }
    }
}
// Group words of a vector: each by (one of) the lanes that worked it out.
template <int NG>
__device__ __forceinline__ void store_word(uint32_t* row, uint32_t own, int l) {
    if (NG == 4 || (l & (4 / NG - 1)) == 0) row[l / (4 / NG)] = own;
}

// Whether a later row of the call writes one of positions [p0, p1) of the slot too: its values stay.  `refused(r)`
// says whether row r is refused, for whatever reason: such a row writes nothing and claims nothing.
// Uniform over the CTA (every thread takes part).
template <typename Refused>
__device__ __forceinline__ bool later_row_writes(int b, int B, int slot, int p0, int p1, const int32_t* slots,
                                                 const int32_t* start, const int32_t* len, int T, Refused&& refused) {
    if (b + 1 >= B) return false;
    int hit = 0;
    for (int r = b + 1 + threadIdx.x; r < B; r += blockDim.x) {
        if (slots[r] != slot || refused(r)) continue;
        const int s0 = start[r], n = len ? len[r] : T;
        hit |= p1 > s0 && p0 < s0 + n;
    }
    return __syncthreads_or(hit) != 0;
}

// KMR_OK or why row b of an append is refused; a row of no tokens never is.
__device__ __forceinline__ int append_row_error(const Kv4AppendParams& p, int b) {
    const int n = p.n_tokens ? p.n_tokens[b] : p.T;
    if (n < 0 || n > p.T) return KMR_ERR_INVALID_ARG;
    if (n == 0) return KMR_OK;
    const int slot = p.slot_ids[b], c0 = p.cpos[b];
    if (slot < 0 || slot >= p.c.slots) return KMR_ERR_SLOT_RANGE;
    return c0 < 0 || c0 > p.c.S - n ? KMR_ERR_CACHE_FULL : KMR_OK;
}
// The same of a conversion's span b, which both caches have to hold.
__device__ __forceinline__ int convert_row_error(const Kv4ConvertParams& p, int b) {
    const int n = p.lengths[b];
    if (n < 0 || n > p.T) return KMR_ERR_INVALID_ARG;
    if (n == 0) return KMR_OK;
    const int slot = p.slot_ids[b], s0 = p.start[b], slot16 = p.slot16[b], s16 = p.start16[b];
    if (slot < 0 || slot >= p.c.slots || slot16 < 0 || slot16 >= p.slots16) return KMR_ERR_SLOT_RANGE;
    return s0 < 0 || s0 > p.c.S - n || s16 < 0 || s16 > p.S16 - n ? KMR_ERR_CACHE_FULL : KMR_OK;
}

// ------------------------------------------------------------------ new tokens
// Cosine and sine of an angle of turn / 2^64 turns, to 0.53 ulp (a sine below 2^-28 turns to 2^-22 of itself): the nearest quarter
// turn is taken off exactly, the rest (at most pi / 4) is a pair of floats th + tl, the Taylor series' first terms are
// formed as pairs too, and one addition at the end rounds.
__device__ __forceinline__ void cos_sin_turn(unsigned long long turn, float& c, float& s) {
    // the nearest 2^-32 turns and what is left, of either sign: a small negative angle is no difference of large parts
    const int low = int(uint32_t(turn));
    const uint32_t high = uint32_t(turn >> 32) + (uint32_t(low) >> 31);
    const int quarter = int((high + (1u << 29)) >> 30);
    const int rem = int(high - (uint32_t(quarter) << 30));                // [-2^29, 2^29), and low / 2^32
    constexpr double kUnit = 6.283185307179586477 / 4294967296.0;
    const float uh = float(kUnit), ul = float(kUnit - double(uh));
    const float rh = __int2float_rn(rem);
    const float rl = __fmaf_rn(__int2float_rn(low), 0x1p-32f, __int2float_rn(rem - __float2int_rn(rh)));
    const float th = __fmul_rn(rh, uh);
    const float tl = __fmaf_rn(rl, uh, __fmaf_rn(rh, ul, __fmaf_rn(rh, uh, -th)));
    const float u = __fmul_rn(th, th);
    const float ul2 = __fmaf_rn(th, th, -u), u2 = __fmaf_rn(2.f * th, tl, ul2);        // th squared is u + ul2, th + tl squared u + u2
    // a constant as two floats, and x times it as product and what its rounding lost
    constexpr float k6 = float(-1.0 / 6), k6l = float(-1.0 / 6 - double(k6)), k24 = float(1.0 / 24), k24l = float(1.0 / 24 - double(k24));
    // sine: th - th^3 / 6 and the rest
    const float c3 = __fmul_rn(th, u), p3 = __fmul_rn(c3, k6);
    const float c3l = __fmaf_rn(th, ul2, __fmaf_rn(th, u, -c3));
    const float p3l = __fmaf_rn(c3l, k6, __fmaf_rn(c3, k6l, __fmaf_rn(c3, k6, -p3)));
    const float ps = __fmul_rn(u, __fmaf_rn(u, __fmaf_rn(u, __fmaf_rn(u, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f), 1.f / 120.f));
    const float s0 = __fadd_rn(th, p3), s0l = __fadd_rn(p3, -__fsub_rn(s0, th));
    const float sn = __fadd_rn(s0, __fadd_rn(s0l, __fmaf_rn(c3, ps, __fadd_rn(p3l, __fmaf_rn(-0.5f * u, tl, tl)))));
    // cosine: 1 - th^2 / 2 + th^4 / 24 and the rest
    const float lead = __fmaf_rn(-0.5f, u, 1.f);
    const float left = __fmaf_rn(-0.5f, u2, __fmaf_rn(-0.5f, u, __fsub_rn(1.f, lead)));
    const float c4 = __fmul_rn(u, u), p4 = __fmul_rn(c4, k24);
    const float p4l = __fmaf_rn(__fmaf_rn(2.f * u, u2, __fmaf_rn(u, u, -c4)), k24, __fmaf_rn(c4, k24l, __fmaf_rn(c4, k24, -p4)));
    const float pc = __fmul_rn(u, __fmaf_rn(u, __fmaf_rn(u, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f));
    const float c0 = __fadd_rn(lead, p4), c0l = __fadd_rn(p4, -__fsub_rn(c0, lead));
    const float cn = __fadd_rn(c0, __fadd_rn(c0l, __fmaf_rn(c4, pc, __fadd_rn(p4l, left))));
    const float a = (quarter & 1) ? sn : cn, b = (quarter & 1) ? cn : sn;
    c = ((quarter + 1) & 2) ? -a : a;
    s = (quarter & 2) ? -b : b;
}

// One CTA per token.  The token's angles are formed once: frequency i advances by theta^(-2i/d) / 2 pi
// turns per position, held as a 64-bit fraction, so that position x fraction mod 1 needs no rounding: the angle of
// position p is off by |p| 2^-65 turns, 2^-34 (4e-10 radians) at most.  Then each warp takes eight heads at a time.
template <int D, int G>
__global__ void __launch_bounds__(kThr) kv4_append_kernel(const __grid_constant__ Kv4AppendParams p) {
    constexpr int NB = D / 32, NG = D / G;
    __shared__ __align__(16) float cs[D / 2], sn[D / 2];
    const int t = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    pdl_wait();
    const int nkv = p.c.nkv;
    const int n = p.n_tokens ? p.n_tokens[b] : p.T, slot = p.slot_ids[b], c0 = p.cpos[b];
    if (const int bad = append_row_error(p, b)) {
        if (t == 0 && tid == 0) set_error(p.err, bad);
        return;
    }
    if (t >= n) return;
    const int pos = c0 + t;
    const int heads = p.nq + 2 * nkv, l = tid & 3;
    const float* row = p.qkv + (size_t(b) * p.T + t) * heads * D;
    if (tid < D / 2) {
        const int axis = tid < p.sec0 ? 0 : (tid < p.sec0 + p.sec1 ? 1 : 2);
        const long long x = p.positions[(size_t(axis) * p.B + b) * p.T + t];
        cos_sin_turn((unsigned long long)x * p.turn[tid], cs[tid], sn[tid]);
    }
    const bool lose = later_row_writes(b, p.B, slot, pos, pos + 1, p.slot_ids, p.cpos, p.n_tokens, p.T,
                                       [&](int r) { return append_row_error(p, r) != KMR_OK; });
    __syncthreads();
    // every lane of a warp runs the same number of rounds, so that the shuffles are complete
    for (int h0 = 0; h0 < heads; h0 += kThr / 4) {
        const int hh = h0 + tid / 4;
        const bool on = hh < heads;
        const int h = on ? hh : heads - 1;
        const bool isq = h < p.nq, isk = !isq && h < p.nq + nkv;
        float x[NB][8];
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const float4* src = reinterpret_cast<const float4*>(row + size_t(h) * D + 32 * k + 8 * l);
            const float4 u = __ldcs(src), v = __ldcs(src + 1);
            x[k][0] = u.x; x[k][1] = u.y; x[k][2] = u.z; x[k][3] = u.w;
            x[k][4] = v.x; x[k][5] = v.y; x[k][6] = v.z; x[k][7] = v.w;
        }
        const uint16_t* w = isq ? p.qn_w : p.kn_w;
        // the sum of squares: over the blocks first, then a tree of neighbours, as a plain reduction by a warp of one dim a lane
        // has it.  The codes hang on the last bits of what is quantised: in this order 0.1% of the values differ from those of
        // a plain norm and rotation in their last bit (by the cosines' rounding), in another order of as many additions 12%.
        float part[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            part[i] = __fmul_rn(x[0][i], x[0][i]);
#pragma unroll
            for (int k = 1; k < NB; ++k) part[i] = __fadd_rn(part[i], __fmul_rn(x[k][i], x[k][i]));
        }
        float ss = __fadd_rn(__fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3])),
                             __fadd_rn(__fadd_rn(part[4], part[5]), __fadd_rn(part[6], part[7])));
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        if (isq || isk) {
            if (w) {
                const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.f / float(D)), p.eps));     // D is a power of two
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const uint4 u = *reinterpret_cast<const uint4*>(w + 32 * k + 8 * l);
                    const uint32_t wv[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[k][2 * i] = __fmul_rn(__fmul_rn(x[k][2 * i], r), bf16_lo(wv[i]));
                        x[k][2 * i + 1] = __fmul_rn(__fmul_rn(x[k][2 * i + 1], r), bf16_hi(wv[i]));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < NB / 2; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float c = cs[32 * k + 8 * l + i], s = sn[32 * k + 8 * l + i];
                    const float lo = x[k][i], hi = x[k + NB / 2][i];
                    x[k][i] = __fsub_rn(__fmul_rn(lo, c), __fmul_rn(hi, s));
                    x[k + NB / 2][i] = __fadd_rn(__fmul_rn(hi, c), __fmul_rn(lo, s));
                }
        }
        if (isq && on) {
            float4* dst = reinterpret_cast<float4*>(p.q_out + ((size_t(b) * p.T + t) * p.nq + h) * D + 8 * l);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                dst[8 * k] = make_float4(x[k][0], x[k][1], x[k][2], x[k][3]);
                dst[8 * k + 1] = make_float4(x[k][4], x[k][5], x[k][6], x[k][7]);
            }
        }
        if (__all_sync(0xffffffffu, isq)) continue;
        uint32_t codes[NB];
        const uint32_t word = quantize<D, G>(x, l, codes);
        if (!on || isq || lose) continue;
        const int kvh = isk ? h - p.nq : h - p.nq - nkv;
        const size_t at = (size_t(slot) * nkv + kvh) * p.c.S + pos;
        store_codes<NB>((isk ? p.c.kc : p.c.vc) + at * (D / 2), codes, isk, l);
        store_word<NG>((isk ? p.c.ks : p.c.vs) + at * NG, word, l);
        if (isk && p.mass && l == 0) p.mass[at] = 0.f;
    }
}

// ------------------------------------------------------------------ bf16 <-> 4 bits
// Grid (positions / span, 2 n_kv, row): a warp takes eight neighbouring positions of K or V of one head at a time.  A CTA's
// span is long where that still gives every SM four of them (the loads of the row's state, some 2 us, are paid per
// CTA), short otherwise.
constexpr int kSpanLong = 256, kSpanShort = 64;

__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

template <int D, int G, bool TO16>
__global__ void __launch_bounds__(kThr) kv4_convert_kernel(const Kv4ConvertParams p) {
    constexpr int NB = D / 32, NG = D / G, BPG = G / 32;
    const int b = blockIdx.z, tid = threadIdx.x, l = tid & 3;
    pdl_wait();
    const int nkv = p.c.nkv, n = p.lengths[b];
    const int slot = p.slot_ids[b], s0 = p.start[b], slot16 = p.slot16[b], s16 = p.start16[b];
    if (const int bad = convert_row_error(p, b)) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) set_error(p.err, bad);
        return;
    }
    const int t0 = blockIdx.x * p.span, t1 = min(n, t0 + p.span);
    if (t0 >= t1) return;
    const int wslot = TO16 ? slot16 : slot, w0 = TO16 ? s16 : s0;
    const int32_t* wslots = TO16 ? p.slot16 : p.slot_ids;
    const int32_t* wstart = TO16 ? p.start16 : p.start;
    const bool clash = later_row_writes(b, p.B, wslot, w0 + t0, w0 + t1, wslots, wstart, p.lengths, p.T,
                                        [&](int r) { return convert_row_error(p, r) != KMR_OK; });
    const bool key = int(blockIdx.y) < nkv;
    const int kvh = key ? blockIdx.y : blockIdx.y - nkv;
    const size_t row = (size_t(slot) * nkv + kvh) * p.c.S + s0, row16 = (size_t(slot16) * nkv + kvh) * p.S16 + s16;
    auto mine = [&](int t) {
        if (t >= t1) return false;
        if (clash)
            for (int r = b + 1; r < p.B; ++r) {
                const int m = p.lengths[r], q = wstart[r];
                if (wslots[r] == wslot && convert_row_error(p, r) == KMR_OK && w0 + t >= q && w0 + t < q + m) return false;
            }
        return true;
    };
    uint16_t* vals0 = (key ? p.k16 : p.v16) + row16 * D + 8 * l;
    uint8_t* codes0 = (key ? p.c.kc : p.c.vc) + row * (D / 2);
    uint32_t* words0 = (key ? p.c.ks : p.c.vs) + row * NG;
    if constexpr (TO16) {
#pragma unroll 2
        for (int t = t0 + tid / 4; t < t1; t += kThr / 4) {
            uint32_t w[NB], word[NG];
            load_codes<NB>(codes0 + size_t(t) * (D / 2), w, key, l);
#pragma unroll
            for (int i = 0; i < NG; ++i) word[i] = words0[size_t(t) * NG + i];
            if (!mine(t)) continue;
            uint4* vals = reinterpret_cast<uint4*>(vals0 + size_t(t) * D);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t u = word[k / BPG];
                const uint32_t s2 = __byte_perm(u, 0u, 0x3232), z2 = __byte_perm(u, 0u, 0x1010);
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // a nibble under the exponent of 128 is the bf16 128 + c; nibbles (i, i + 4)
                    const uint32_t c = fma_bf16x2(and_or(w[k] >> (4 * i), 0x000F000Fu, 0x43004300u), 0x3F803F80u,
                                                  0xC300C300u);
                    y[i] = fma_bf16x2(c, s2, z2);
                }
                __stcs(vals + 4 * k, make_uint4(__byte_perm(y[0], y[1], 0x5410), __byte_perm(y[2], y[3], 0x5410),
                                                __byte_perm(y[0], y[1], 0x7632), __byte_perm(y[2], y[3], 0x7632)));
            }
        }
    } else {
        // every lane of a warp runs the same number of rounds (the shuffles); the next round's loads are in flight
        uint4 next[NB];
        auto load = [&](int t) {
            const uint4* vals = reinterpret_cast<const uint4*>(vals0 + size_t(t < t1 ? t : t0) * D);
#pragma unroll
            for (int k = 0; k < NB; ++k) next[k] = __ldcs(vals + 4 * k);
        };
        load(t0 + tid / 4);
        for (int i0 = t0; i0 < t1; i0 += kThr / 4) {
            const int t = i0 + tid / 4;
            uint4 raw[NB];
#pragma unroll
            for (int k = 0; k < NB; ++k) raw[k] = next[k];
            if (i0 + kThr / 4 < t1) load(t + kThr / 4);
            uint32_t w[NB];
            const uint32_t word = quantize_bf16<D, G>(raw, l, w);
            if (!mine(t)) continue;
            store_codes<NB>(codes0 + size_t(t) * (D / 2), w, key, l);
            store_word<NG>(words0 + size_t(t) * NG, word, l);
        }
    }
}

// ------------------------------------------------------------------ eviction
constexpr int kSelThr = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelCache = 48 * 1024;      // keys held in shared memory (192 KB); longer rows read them again each pass

// Order-preserving integer of a mass: larger mass, larger key; -0 counts as 0, NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = __float_as_uint(m + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// KMR_OK or why a row of some length is refused for itself.
__device__ __forceinline__ int evict_own_error(const Kv4EvictParams& p, int b) {
    const int src = p.src_ids[b], dst = p.dst_ids[b], n = p.lengths[b];
    if (src < 0 || src >= p.src.slots || dst < 0 || dst >= p.dst.slots) return KMR_ERR_SLOT_RANGE;
    return n < 0 || n > p.src.S ? KMR_ERR_CACHE_FULL : KMR_OK;
}
// Whether the row may be evicted: KMR_OK or the error.  A row that is refused for itself moves nothing, so it stands in no
// other's way.  Uniform over the CTA.
__device__ __forceinline__ int evict_row_error(const Kv4EvictParams& p, int b) {
    if (p.lengths[b] == 0) return KMR_OK;            // an idle row: nothing moves
    const int own = evict_own_error(p, b), dst = p.dst_ids[b];
    int clash = 0;
    for (int r = threadIdx.x; r < p.B; r += blockDim.x) {
        if (p.lengths[r] == 0 || evict_own_error(p, r) != KMR_OK) continue;
        clash |= r != b && p.dst_ids[r] == dst;
        clash |= p.same && p.src_ids[r] == dst;
    }
    clash = __syncthreads_or(clash);
    return own != KMR_OK ? own : (clash ? KMR_ERR_SLOT_RANGE : KMR_OK);
}

// Positions kept of one (row, head): the newest `recent`, and of the older ones the heaviest, the
// lower index first among equals.  The smallest kept key is found digit by digit (11, 11 and 10 bits: a
// histogram each, searched from the top by a scan over the CTA), then one ordered pass writes the kept
// indices in ascending order.  The keys are formed once and kept in shared memory.  What bounds it is the chain
// of some fifteen barriers: a row of 8192 masses is 32 KB.
__device__ __forceinline__ void select_positions(const Kv4EvictParams& p, int h, int b, int bad) {
    extern __shared__ uint32_t keys[];
    __shared__ int hist[kSelBins];
    __shared__ int wsum[2][32];
    __shared__ int found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* kept = p.kept + (size_t(b) * p.src.nkv + h) * p.keep;
    const int n = bad ? 0 : p.lengths[b];
    const int total = n < p.keep ? n : p.keep, newest = p.recent < total ? p.recent : total;
    if (tid == 0 && h == 0) {
        if (bad) set_error(p.err, bad);
        p.new_lengths[b] = total;
    }
    for (int i = total + tid; i < p.keep; i += kSelThr) kept[i] = -1;
    if (total == n) {                                // everything stays
        for (int i = tid; i < n; i += kSelThr) kept[i] = i;
        return;
    }
    const int old = n - newest, need = total - newest;
    for (int i = tid; i < newest; i += kSelThr) kept[need + i] = old + i;
    if (need == 0) return;
    const float* m = p.mass + (size_t(p.src_ids[b]) * p.src.nkv + h) * p.src.S;
    const bool cached = old <= kSelCache;
    if (cached)
        for (int i = tid; i < old; i += kSelThr) keys[i] = mass_key(m[i]);
    auto key_at = [&](int i) { return cached ? keys[i] : mass_key(m[i]); };
    uint32_t prefix = 0;
    int left = need;                                 // how many of the keys that share the prefix are kept
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass < 2 ? 11 : 10;
        const uint32_t above = pass == 0 ? 0u : 0xFFFFFFFFu << (shift + bits), digits = (1u << bits) - 1u;
        hist[tid] = 0;
        hist[tid + kSelThr] = 0;
        __syncthreads();                             // (also: the keys are there)
        for (int i = tid; i < old; i += kSelThr) {
            const uint32_t k = key_at(i);
            if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & digits], 1);
        }
        __syncthreads();
        // thread i holds bins 2047 - 2 i and 2046 - 2 i: an inclusive scan counts from the top
        const int top = kSelBins - 1 - 2 * tid, c0 = hist[top], c1 = hist[top - 1];
        int sum = c0 + c1;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) wsum[0][warp] = sum;
        __syncthreads();
        int before = sum - c0 - c1;
        for (int w = 0; w < warp; ++w) before += wsum[0][w];
        if (before < left && left <= before + c0 + c1) {
            const bool second = before + c0 < left;
            found[0] = second ? top - 1 : top;
            found[1] = left - before - (second ? c0 : 0);
        }
        __syncthreads();
        prefix |= uint32_t(found[0]) << shift;
        left = found[1];
    }
    // keys above `prefix` are kept, and the first `left` of those equal to it
    const int per = ((old + kSelThr - 1) / kSelThr) * 32;      // positions of a warp, a multiple of 32
    const int i0 = warp * per, i1 = min(old, i0 + per);
    int gt = 0, eq = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = key_at(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = warp_sum(gt);
    eq = warp_sum(eq);
    if (lane == 0) {
        wsum[0][warp] = gt;
        wsum[1][warp] = eq;
    }
    __syncthreads();
    gt = warp_sum(lane < warp ? wsum[0][lane] : 0);
    eq = warp_sum(lane < warp ? wsum[1][lane] : 0);
    for (int i = i0; i < i1; i += 32) {
        const bool in = i + lane < i1;
        const uint32_t k = in ? key_at(i + lane) : 0u;
        const bool isg = in && k > prefix, ise = in && k == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
        const uint32_t below = (1u << lane) - 1u;
        const int g0 = gt + __popc(mg & below), e0 = eq + __popc(me & below);
        if (isg || (ise && e0 < left)) kept[g0 + min(e0, left)] = i + lane;
        gt += __popc(mg);
        eq += __popc(me);
    }
}

// One (row, head) per thread-block cluster: its first CTA selects, then all move the kept positions' codes, scales
// and mass to positions 0, 1, ... of the destination row: four lanes a position (as above), kMove positions of a
// lane in flight.  The cluster is as large as the SMs allow (up to 8): a call of few rows needs more than one SM's
// bandwidth for a row, one of many rows has an SM for each.
constexpr int kMove = 2;

template <int D, int G>
__global__ void __launch_bounds__(kSelThr, 1) kv4_evict_kernel(const Kv4EvictParams p) {
    constexpr int NG = D / G;
    using Piece = typename std::conditional<D == 128, uint4, uint2>::type;
    const int h = blockIdx.y, b = blockIdx.z, l = threadIdx.x & 3;
    pdl_wait();
    const int bad = evict_row_error(p, b);
    if (blockIdx.x == 0) select_positions(p, h, b, bad);
    if (gridDim.x > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
    if (bad) return;
    const int32_t* kept = p.kept + (size_t(b) * p.src.nkv + h) * p.keep;
    const int n = p.lengths[b], total = n < p.keep ? n : p.keep;
    const size_t srow = (size_t(p.src_ids[b]) * p.src.nkv + h) * p.src.S;
    const size_t drow = (size_t(p.dst_ids[b]) * p.src.nkv + h) * p.dst.S;
    constexpr int kLanes = kSelThr / 4;
    for (int j0 = int(blockIdx.x) * kLanes * kMove + threadIdx.x / 4; j0 < total; j0 += gridDim.x * kLanes * kMove) {
        size_t from[kMove];
        Piece k[kMove], v[kMove];
        uint32_t kw[kMove], vw[kMove];
        float m[kMove];
#pragma unroll
        for (int i = 0; i < kMove; ++i) {
            const int j = j0 + i * kLanes;
            from[i] = srow + __ldcg(kept + (j < total ? j : j0));
        }
#pragma unroll
        for (int i = 0; i < kMove; ++i) {
            k[i] = __ldcs(reinterpret_cast<const Piece*>(p.src.kc + from[i] * (D / 2)) + l);
            v[i] = __ldcs(reinterpret_cast<const Piece*>(p.src.vc + from[i] * (D / 2)) + l);
            kw[i] = l < NG ? __ldcs(p.src.ks + from[i] * NG + l) : 0u;
            vw[i] = l < NG ? __ldcs(p.src.vs + from[i] * NG + l) : 0u;
            m[i] = l == 0 ? p.mass[from[i]] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kMove; ++i) {
            const int j = j0 + i * kLanes;
            if (j >= total) break;
            const size_t to = drow + j;
            reinterpret_cast<Piece*>(p.dst.kc + to * (D / 2))[l] = k[i];
            reinterpret_cast<Piece*>(p.dst.vc + to * (D / 2))[l] = v[i];
            if (l < NG) {
                p.dst.ks[to * NG + l] = kw[i];
                p.dst.vs[to * NG + l] = vw[i];
            }
            if (l == 0 && p.dst_mass) p.dst_mass[to] = m[i];
        }
    }
}

template <int D, int G>
const void* write_fn(int which) {
    if (which == 0) return (const void*)kv4_append_kernel<D, G>;
    if (which == 3) return (const void*)kv4_evict_kernel<D, G>;
    return which == 1 ? (const void*)kv4_convert_kernel<D, G, false> : (const void*)kv4_convert_kernel<D, G, true>;
}
const void* write_fn(int d, int g, int which) {
    if (d == 64) return g == 32 ? write_fn<64, 32>(which) : write_fn<64, 64>(which);
    return g == 32 ? write_fn<128, 32>(which) : (g == 64 ? write_fn<128, 64>(which) : write_fn<128, 128>(which));
}

}  // namespace

// Every kernel of the cache is launched as a programmatic dependent of whatever ran before it on the stream, and
// waits for that at its start: the launch itself overlaps the end of the previous kernel.
static cudaError_t launch(const void* fn, dim3 grid, int threads, size_t smem, int cluster, const void* params,
                          cudaStream_t st) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    void* args[] = {const_cast<void*>(params)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t st) {
    return launch(write_fn(p.c.d, p.c.g, 0), dim3(p.T, p.B), kThr, 0, 1, &p, st);
}

cudaError_t launch_kv4_convert(const Kv4ConvertParams& p, bool to_bf16, cudaStream_t st) {
    Kv4ConvertParams q = p;
    const long long ctas = (long long)((p.T + kSpanLong - 1) / kSpanLong) * 2 * p.c.nkv * p.B;
    q.span = ctas >= 4LL * num_sms() ? kSpanLong : kSpanShort;
    return launch(write_fn(p.c.d, p.c.g, to_bf16 ? 2 : 1), dim3((p.T + q.span - 1) / q.span, 2 * p.c.nkv, p.B), kThr, 0, 1,
                  &q, st);
}

// Also loads every kernel, so that a later call can be captured into a graph whatever its shape.
cudaError_t kv4_set_attributes() {
    const int shapes[5][2] = {{64, 32}, {64, 64}, {128, 32}, {128, 64}, {128, 128}};
    for (const auto& sh : shapes) {
        cudaFuncAttributes a;
        cudaError_t e;
        for (int which = 0; which < 3; ++which)
            if ((e = cudaFuncGetAttributes(&a, write_fn(sh[0], sh[1], which))) != cudaSuccess) return e;
        e = cudaFuncSetAttribute(write_fn(sh[0], sh[1], 3), cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCache * 4);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t st) {
    int cluster = 8;
    while (cluster > 1 && (long long)cluster * p.src.nkv * p.B > num_sms()) cluster /= 2;
    return launch(write_fn(p.src.d, p.src.g, 3), dim3(cluster, p.src.nkv, p.B), kSelThr,
                  size_t(p.src.S < kSelCache ? p.src.S : kSelCache) * 4, cluster, &p, st);
}

}  // namespace kmr
