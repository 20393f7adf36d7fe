// Decode attention of one token per row over the 4-bit KV cache (format: kmr_kv4.cuh).
//
// out = softmax(q K^T scale) V over positions 0..cache_position of the row's slot, and, where a mass
// is given, mass[slot][head][p] += the sum over the KV head's query heads of position p's weight.
// Two launches: the splits of every (row, KV head) leave their softmax states (m, l, o) in base 2 in
// the workspace (and, for the mass, every score); the second merges the states in split order and
// turns the scores into weights.  Rows that share a slot add to its mass in row order.
#include <math.h>

#include "kmr_kv4.cuh"

namespace kmr {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kThr = 256, kWarps = 8;

__device__ __forceinline__ int kv4_row_error(const Kv4AttnParams& p, int b) {
    const int slot = p.slot_ids[b], cp = p.cpos[b];
    if (slot < 0 || slot >= p.c.slots) return KMR_ERR_SLOT_RANGE;
    return (cp < 0 || cp >= p.c.S) ? KMR_ERR_CACHE_FULL : KMR_OK;
}

template <int D>
__global__ void __launch_bounds__(kThr) kv4_split_kernel(const Kv4AttnParams p) {
    constexpr int NB = D / 32, LPR = D / 4, SUBS = 32 / LPR;
    __shared__ float wm[kWarps * 2][kKv4MaxRep], wl[kWarps * 2][kKv4MaxRep];
    __shared__ float wo[kWarps * SUBS][D];
    const int s = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    if (kv4_row_error(p, b) != KMR_OK) return;
    const int L = p.cpos[b] + 1, rep = p.nq / p.c.nkv;
    int chunk, ns;
    kv4_split_plan(L, chunk, ns);
    if (s >= ns) return;
    const int t0 = s * chunk, t1 = min(L, t0 + chunk);
    const int tid = threadIdx.x, warp = tid >> 5, wl32 = tid & 31, lane = wl32 % LPR, sub = warp * SUBS + wl32 / LPR;
    const size_t row = (size_t(p.slot_ids[b]) * p.c.nkv + h) * p.c.S;
    const int ng = D / p.c.g, gi = lane * 4 / p.c.g;
    const float qs = p.scale * kLog2e;
    for (int r = 0; r < rep; ++r) {
        const float4 qv = *reinterpret_cast<const float4*>(p.q + (size_t(b) * p.nq + h * rep + r) * D + lane * 4);
        float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
        float* sc = p.scores ? p.scores + ((size_t(b) * p.c.nkv + h) * rep + r) * p.c.S : nullptr;
        for (int i0 = t0; i0 < t1; i0 += kWarps * SUBS) {
            const int i = i0 + sub;
            const size_t at = row + (i < t1 ? i : t0);
            const uint32_t kc = reinterpret_cast<const uint16_t*>(p.c.kc + at * (D / 2))[kv4_unit(lane, NB, true)];
            const uint32_t vc = reinterpret_cast<const uint16_t*>(p.c.vc + at * (D / 2))[kv4_unit(lane, NB, false)];
            const uint32_t kw = p.c.ks[at * ng + gi], vw = p.c.vs[at * ng + gi];
            const float s4 = kv4_s(kw), z4 = kv4_z(kw);
            float a = qv.x * fmaf(float(kc & 15), s4, z4) + qv.y * fmaf(float((kc >> 4) & 15), s4, z4) +
                      qv.z * fmaf(float((kc >> 8) & 15), s4, z4) + qv.w * fmaf(float(kc >> 12), s4, z4);
            for (int off = 1; off < LPR; off <<= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
            if (i >= t1) continue;
            a *= qs;
            if (sc && lane == 0) sc[i] = a;
            const float mn = fmaxf(m, a), cf = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(a - mn);
            const float vs = kv4_s(vw), vz = kv4_z(vw);
            m = mn;
            l = l * cf + w;
            for (int e = 0; e < 4; ++e) o[e] = o[e] * cf + w * fmaf(float((vc >> (4 * e)) & 15), vs, vz);
        }
        __syncthreads();
        if (lane == 0) {
            wm[sub][r] = m;
            wl[sub][r] = l;
        }
        for (int e = 0; e < 4; ++e) wo[sub][lane * 4 + e] = o[e];
        __syncthreads();
        float* part = p.part + (((size_t(b) * p.c.nkv + h) * p.nsplit + s) * rep + r) * (D + 2);
        for (int i = tid; i < D; i += kThr) {
            float mx = -INFINITY, num = 0.f, den = 0.f;
            for (int w = 0; w < kWarps * SUBS; ++w) mx = fmaxf(mx, wm[w][r]);
            for (int w = 0; w < kWarps * SUBS; ++w) {
                const float f = wm[w][r] == -INFINITY ? 0.f : exp2f(wm[w][r] - mx);
                den += f * wl[w][r];
                num += f * wo[w][i];
            }
            part[2 + i] = num;
            if (i == 0) {
                part[0] = mx;
                part[1] = den;
            }
        }
    }
}

__global__ void __launch_bounds__(kThr) kv4_merge_kernel(const Kv4AttnParams p) {
    const int h = blockIdx.y, b = blockIdx.z, d = p.c.d, rep = p.nq / p.c.nkv, tid = threadIdx.x;
    const int err = kv4_row_error(p, b);
    float* out = p.out + (size_t(b) * p.nq + h * rep) * d;
    if (err != KMR_OK) {
        if (blockIdx.x == 0) {
            if (tid == 0 && h == 0) set_error(p.err, err);
            for (int i = tid; i < rep * d; i += kThr) out[i] = 0.f;
        }
        return;
    }
    int chunk, ns;
    if (blockIdx.x == 0) {
        kv4_split_plan(p.cpos[b] + 1, chunk, ns);
        const float* part = p.part + (size_t(b) * p.c.nkv + h) * p.nsplit * rep * (d + 2);
        for (int i = tid; i < rep * d; i += kThr) {
            const float* mine = part + size_t(i / d) * (d + 2);
            float mx = -INFINITY, num = 0.f, den = 0.f;
            for (int s = 0; s < ns; ++s) mx = fmaxf(mx, mine[size_t(s) * rep * (d + 2)]);
            for (int s = 0; s < ns; ++s) {
                const float* q = mine + size_t(s) * rep * (d + 2);
                const float f = q[0] == -INFINITY ? 0.f : exp2f(q[0] - mx);
                den += f * q[1];
                num += f * q[2 + i % d];
            }
            out[i] = num / den;
        }
    }
    if (!p.mass) return;
    const int slot = p.slot_ids[b];
    int before = 0;
    for (int r = tid; r < b; r += kThr) before |= p.slot_ids[r] == slot && kv4_row_error(p, r) == KMR_OK;
    if (__syncthreads_or(before)) return;            // the slot's first row adds for all of them
    __shared__ float sm[kKv4MaxRep], sl[kKv4MaxRep];
    const int i = blockIdx.x * kThr + tid;
    float add = 0.f;
    int most = 0;
    for (int r = b; r < p.B; ++r) {
        if (p.slot_ids[r] != slot || kv4_row_error(p, r) != KMR_OK) continue;
        const int L = p.cpos[r] + 1;
        most = max(most, L);
        kv4_split_plan(L, chunk, ns);
        __syncthreads();
        if (tid < rep) {
            const float* q = p.part + ((size_t(r) * p.c.nkv + h) * p.nsplit * rep + tid) * (d + 2);
            float mx = -INFINITY, den = 0.f;
            for (int s = 0; s < ns; ++s) mx = fmaxf(mx, q[size_t(s) * rep * (d + 2)]);
            for (int s = 0; s < ns; ++s) {
                const float m = q[size_t(s) * rep * (d + 2)];
                den += m == -INFINITY ? 0.f : exp2f(m - mx) * q[size_t(s) * rep * (d + 2) + 1];
            }
            sm[tid] = mx;
            sl[tid] = 1.f / den;
        }
        __syncthreads();
        if (i < L) {
            const float* sc = p.scores + (size_t(r) * p.c.nkv + h) * rep * p.c.S + i;
            for (int k = 0; k < rep; ++k) add += exp2f(sc[size_t(k) * p.c.S] - sm[k]) * sl[k];
        }
    }
    if (i < most) p.mass[(size_t(slot) * p.c.nkv + h) * p.c.S + i] += add;
}

}  // namespace

int kv4_attn_splits(int S) {
    int chunk, ns;
    kv4_split_plan(S, chunk, ns);
    // a shorter row can have more splits than the longest (the chunk is rounded up), never more than 32
    const int most = (S + kKv4MinChunk - 1) / kKv4MinChunk;
    return most < kKv4MaxSplits ? most : kKv4MaxSplits;
}
size_t kv4_attn_part_bytes(int B, int nq, int d, int nsplit) {
    return (size_t(B) * nq * nsplit * (d + 2) * 4 + 15) & ~size_t(15);
}
cudaError_t kv4_attn_set_attributes() { return cudaSuccess; }

cudaError_t launch_kv4_attn(const Kv4AttnParams& p, cudaStream_t st) {
    const dim3 grid(p.nsplit, p.c.nkv, p.B);
    if (p.c.d == 64)
        kv4_split_kernel<64><<<grid, kThr, 0, st>>>(p);
    else
        kv4_split_kernel<128><<<grid, kThr, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    kv4_merge_kernel<<<dim3(p.mass ? (p.c.S + kThr - 1) / kThr : 1, p.c.nkv, p.B), kThr, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace kmr
