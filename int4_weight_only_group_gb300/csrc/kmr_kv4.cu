// Writes of the 4-bit KV cache: new tokens (q/k RMSNorm, M-RoPE and quantisation in one pass),
// conversions from and to a bf16 cache, and eviction into another row.  The format and the
// quantiser are in kmr_kv4.cuh.
#include "kmr_kv4.cuh"

namespace kmr {
namespace {

constexpr int kThr = 256;

// Whether a later row of the call writes this (slot, position) too: then that row's values stay.
// Uniform over the CTA (every thread takes part).
__device__ __forceinline__ bool later_row_writes(int b, int B, int slot, int pos, const int32_t* slots,
                                                 const int32_t* start, const int32_t* len, int T, int S) {
    if (b + 1 >= B) return false;
    int hit = 0;
    for (int r = b + 1 + threadIdx.x; r < B; r += blockDim.x) {
        if (slots[r] != slot) continue;
        const int s0 = start[r], n = len ? len[r] : T;
        if (n < 0 || n > T || s0 < 0 || s0 > S - n) continue;      // a refused row writes nothing
        hit |= pos >= s0 && pos < s0 + n;
    }
    return __syncthreads_or(hit) != 0;
}

// ------------------------------------------------------------------ new tokens
// One CTA per token.  The token's angles are formed once: frequency i advances by theta^(-2i/d) / 2 pi
// turns per position, held as a 64-bit fraction, so that position x fraction mod 1 is exact for any
// position and the angle keeps its bits far into a long context.  Then d / 4 lanes take a head at a
// time, four dims each: the rotation's partner dim is d / 8 lanes away.
__global__ void __launch_bounds__(kThr) kv4_append_kernel(const __grid_constant__ Kv4AppendParams p) {
    __shared__ float cs[64], sn[64];
    const int t = blockIdx.x, b = blockIdx.y;
    const int d = p.c.d, nkv = p.c.nkv;
    const int n = p.n_tokens ? p.n_tokens[b] : p.T;
    const int slot = p.slot_ids[b], c0 = p.cpos[b];
    const bool bad_n = n < 0 || n > p.T, bad_slot = slot < 0 || slot >= p.c.slots;
    const bool bad_pos = !bad_n && (c0 < 0 || c0 > p.c.S - n);
    if (bad_n || (n > 0 && (bad_slot || bad_pos))) {
        if (t == 0 && threadIdx.x == 0)
            set_error(p.err, bad_n ? KMR_ERR_INVALID_ARG : (bad_slot ? KMR_ERR_SLOT_RANGE : KMR_ERR_CACHE_FULL));
        return;
    }
    if (t >= n) return;
    const int pos = c0 + t;
    if (threadIdx.x < d / 2) {
        const int f = threadIdx.x, axis = f < p.sec0 ? 0 : (f < p.sec0 + p.sec1 ? 1 : 2);
        const long long x = p.positions[(size_t(axis) * p.B + b) * p.T + t];
        const unsigned long long turn = (unsigned long long)x * p.turn[f];
        const float frac = float(int(turn >> 32)) * 0x1p-31f;          // half turns in [-1, 1)
        sincospif(frac, &sn[f], &cs[f]);
    }
    __syncthreads();
    const bool lose = later_row_writes(b, p.B, slot, pos, p.slot_ids, p.cpos, p.n_tokens, p.T, p.c.S);
    const int lpr = d / 4, lane = threadIdx.x % lpr, sub = threadIdx.x / lpr, nsub = kThr / lpr;
    const int heads = p.nq + 2 * nkv, nb = d / 32, ng = d / p.c.g;
    const float* row = p.qkv + (size_t(b) * p.T + t) * heads * d;
    // every lane of a warp runs the same number of rounds, so that the shuffles are complete
    for (int h0 = 0; h0 < heads; h0 += nsub) {
        const int hh = h0 + sub;
        const bool on = hh < heads;
        const int h = on ? hh : heads - 1;
        const bool isq = h < p.nq, isk = !isq && h < p.nq + nkv;
        const float4 v = *reinterpret_cast<const float4*>(row + size_t(h) * d + lane * 4);
        float x[4] = {v.x, v.y, v.z, v.w};
        const uint16_t* w = isq ? p.qn_w : p.kn_w;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = __fmaf_rn(x[e], x[e], ss);
        for (int o = 1; o < lpr; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((isq || isk) && w) {
            const float r = rsqrtf(ss / float(d) + p.eps);
            const uint2 wv = *reinterpret_cast<const uint2*>(w + lane * 4);
            x[0] = x[0] * r * bf16_lo(wv.x);
            x[1] = x[1] * r * bf16_hi(wv.x);
            x[2] = x[2] * r * bf16_lo(wv.y);
            x[3] = x[3] * r * bf16_hi(wv.y);
        }
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], lpr / 2);
        if (isq || isk) {
            const bool lo = lane < lpr / 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int f = (lane * 4 + e) % (d / 2);
                x[e] = lo ? x[e] * cs[f] - y[e] * sn[f] : x[e] * cs[f] + y[e] * sn[f];
            }
        }
        uint32_t word;
        const uint32_t c = kv4_quantize(x, p.c.g / 4, word);
        if (!on) continue;
        if (isq) {
            *reinterpret_cast<float4*>(p.q_out + ((size_t(b) * p.T + t) * p.nq + h) * d + lane * 4) =
                make_float4(x[0], x[1], x[2], x[3]);
            continue;
        }
        if (lose) continue;
        const int kvh = isk ? h - p.nq : h - p.nq - nkv;
        const size_t at = (size_t(slot) * nkv + kvh) * p.c.S + pos;
        uint16_t* codes = reinterpret_cast<uint16_t*>((isk ? p.c.kc : p.c.vc) + at * (d / 2));
        codes[kv4_unit(lane, nb, isk)] = uint16_t(c);
        if (lane % (p.c.g / 4) == 0) (isk ? p.c.ks : p.c.vs)[at * ng + lane * 4 / p.c.g] = word;
        if (isk && p.mass && lane == 0) p.mass[at] = 0.f;
    }
}

// ------------------------------------------------------------------ bf16 <-> 4 bits
template <bool TO16>
__global__ void __launch_bounds__(kThr) kv4_convert_kernel(const Kv4ConvertParams p) {
    const int b = blockIdx.y, t = blockIdx.x;
    const int d = p.c.d, nkv = p.c.nkv, n = p.lengths[b];
    const int slot = p.slot_ids[b], s0 = p.start[b], slot16 = p.slot16[b], s16 = p.start16[b];
    const bool bad_n = n < 0 || n > p.T;
    const bool bad_slot = slot < 0 || slot >= p.c.slots || slot16 < 0 || slot16 >= p.slots16;
    const bool bad_pos = !bad_n && (s0 < 0 || s0 > p.c.S - n || s16 < 0 || s16 > p.S16 - n);
    if (bad_n || (n > 0 && (bad_slot || bad_pos))) {
        if (t == 0 && threadIdx.x == 0)
            set_error(p.err, bad_n ? KMR_ERR_INVALID_ARG : (bad_slot ? KMR_ERR_SLOT_RANGE : KMR_ERR_CACHE_FULL));
        return;
    }
    if (t >= n) return;
    if (TO16 ? later_row_writes(b, p.B, slot16, s16 + t, p.slot16, p.start16, p.lengths, p.T, p.S16)
             : later_row_writes(b, p.B, slot, s0 + t, p.slot_ids, p.start, p.lengths, p.T, p.c.S))
        return;
    const int lpr = d / 4, lane = threadIdx.x % lpr, sub = threadIdx.x / lpr, nsub = kThr / lpr;
    const int nb = d / 32, ng = d / p.c.g;
    for (int h0 = 0; h0 < 2 * nkv; h0 += nsub) {
        const int hh = h0 + sub;
        const bool on = hh < 2 * nkv;
        const int h = on ? hh : 0, kvh = h % nkv;
        const bool isk = h < nkv;
        const size_t at = (size_t(slot) * nkv + kvh) * p.c.S + s0 + t;
        const size_t at16 = ((size_t(slot16) * nkv + kvh) * p.S16 + s16 + t) * d + lane * 4;
        uint16_t* codes = reinterpret_cast<uint16_t*>((isk ? p.c.kc : p.c.vc) + at * (d / 2)) + kv4_unit(lane, nb, isk);
        uint32_t* words = (isk ? p.c.ks : p.c.vs) + at * ng + lane * 4 / p.c.g;
        uint2* vals = reinterpret_cast<uint2*>((isk ? p.k16 : p.v16) + at16);
        if constexpr (TO16) {
            if (!on) continue;
            const uint32_t c = *codes, w = *words;
            const float s = kv4_s(w), z = kv4_z(w);
            *vals = make_uint2(pack_bf16x2(__fmaf_rn(float(c & 15), s, z), __fmaf_rn(float((c >> 4) & 15), s, z)),
                               pack_bf16x2(__fmaf_rn(float((c >> 8) & 15), s, z), __fmaf_rn(float(c >> 12), s, z)));
        } else {
            const uint2 u = *vals;
            const float x[4] = {bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
            uint32_t word;
            const uint32_t c = kv4_quantize(x, p.c.g / 4, word);
            if (!on) continue;
            *codes = uint16_t(c);
            if (lane % (p.c.g / 4) == 0) *words = word;
        }
    }
}

// ------------------------------------------------------------------ eviction
constexpr int kSelThr = 1024;

// Order-preserving integer of a mass: larger mass, larger key; -0 counts as 0, NaN below everything.
__device__ __forceinline__ uint32_t mass_key(float m) {
    if (m != m) return 0u;
    const uint32_t u = __float_as_uint(m + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Whether the row may be evicted: -1, or the error code.  Uniform over the CTA.
__device__ __forceinline__ int evict_row_error(const Kv4EvictParams& p, int b) {
    const int src = p.src_ids[b], dst = p.dst_ids[b], n = p.lengths[b];
    int clash = 0;
    for (int r = threadIdx.x; r < p.B; r += blockDim.x) {
        clash |= r != b && p.dst_ids[r] == dst;
        clash |= p.same && p.src_ids[r] == dst;
    }
    clash = __syncthreads_or(clash);
    if (src < 0 || src >= p.src.slots || dst < 0 || dst >= p.dst.slots || clash) return KMR_ERR_SLOT_RANGE;
    return (n < 0 || n > p.src.S) ? KMR_ERR_CACHE_FULL : KMR_OK;
}

// Positions kept of one (row, head): the newest `recent`, and of the older ones the heaviest, the
// lower index first among equals.  The smallest kept key is found digit by digit (8 bits at a time,
// a histogram each), then one ordered pass writes the kept indices in ascending order.
__global__ void __launch_bounds__(kSelThr) kv4_select_kernel(const Kv4EvictParams p) {
    __shared__ int hist[256];
    __shared__ int wsum[2][32];
    __shared__ uint32_t sh_prefix;
    __shared__ int sh_need;
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bad = evict_row_error(p, b);
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
    uint32_t prefix = 0;
    int left = need;                                 // how many of the keys that share the prefix are kept
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t above = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
        for (int i = tid; i < old; i += kSelThr) {
            const uint32_t k = mass_key(m[i]);
            if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int got = 0, dig = 255;
            while (dig > 0 && got + hist[dig] < left) got += hist[dig--];
            sh_prefix = prefix | (uint32_t(dig) << shift);
            sh_need = left - got;
        }
        __syncthreads();
        prefix = sh_prefix;
        left = sh_need;
    }
    // keys above `prefix` are kept, and the first `left` of those equal to it
    const int per = ((old + 1023) / 1024) * 32;      // positions of a warp, a multiple of 32
    const int i0 = warp * per, i1 = min(old, i0 + per);
    int gt = 0, eq = 0;
    for (int i = i0 + lane; i < i1; i += 32) {
        const uint32_t k = mass_key(m[i]);
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
    gt = eq = 0;
    for (int w = 0; w < warp; ++w) {
        gt += wsum[0][w];
        eq += wsum[1][w];
    }
    for (int i = i0; i < i1; i += 32) {
        const uint32_t k = i + lane < i1 ? mass_key(m[i + lane]) : 0u;
        const bool in = i + lane < i1, isg = in && k > prefix, ise = in && k == prefix;
        const uint32_t mg = __ballot_sync(0xffffffffu, isg), me = __ballot_sync(0xffffffffu, ise);
        const uint32_t below = (1u << lane) - 1u;
        const int g0 = gt + __popc(mg & below), e0 = eq + __popc(me & below);
        if (isg || (ise && e0 < left)) kept[g0 + min(e0, left)] = i + lane;
        gt += __popc(mg);
        eq += __popc(me);
    }
}

// The kept positions' codes, scales and mass, moved to positions 0, 1, ... of the destination row.
__global__ void __launch_bounds__(kThr) kv4_gather_kernel(const Kv4EvictParams p) {
    const int h = blockIdx.y, b = blockIdx.z;
    const int d = p.src.d, ng = d / p.src.g, units = d / 32;       // 16-byte units of a row of codes
    const int32_t* kept = p.kept + (size_t(b) * p.src.nkv + h) * p.keep;
    const int total = p.new_lengths[b];
    if (total == 0) return;
    const size_t srow = (size_t(p.src_ids[b]) * p.src.nkv + h) * p.src.S;
    const size_t drow = (size_t(p.dst_ids[b]) * p.src.nkv + h) * p.dst.S;
    for (int j = blockIdx.x * kThr + threadIdx.x; j < total; j += gridDim.x * kThr) {
        const size_t s = srow + kept[j], t = drow + j;
        const uint4* ksrc = reinterpret_cast<const uint4*>(p.src.kc + s * (d / 2));
        const uint4* vsrc = reinterpret_cast<const uint4*>(p.src.vc + s * (d / 2));
        uint4* kdst = reinterpret_cast<uint4*>(p.dst.kc + t * (d / 2));
        uint4* vdst = reinterpret_cast<uint4*>(p.dst.vc + t * (d / 2));
        for (int u = 0; u < units; ++u) {
            kdst[u] = ksrc[u];
            vdst[u] = vsrc[u];
        }
        for (int u = 0; u < ng; ++u) {
            p.dst.ks[t * ng + u] = p.src.ks[s * ng + u];
            p.dst.vs[t * ng + u] = p.src.vs[s * ng + u];
        }
        if (p.dst_mass) p.dst_mass[t] = p.mass[s];
    }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t st) {
    kv4_append_kernel<<<dim3(p.T, p.B), kThr, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_convert(const Kv4ConvertParams& p, bool to_bf16, cudaStream_t st) {
    if (to_bf16)
        kv4_convert_kernel<true><<<dim3(p.T, p.B), kThr, 0, st>>>(p);
    else
        kv4_convert_kernel<false><<<dim3(p.T, p.B), kThr, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t st) {
    kv4_select_kernel<<<dim3(p.src.nkv, p.B), kSelThr, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    kv4_gather_kernel<<<dim3((p.keep + kThr - 1) / kThr, p.src.nkv, p.B), kThr, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kmr
