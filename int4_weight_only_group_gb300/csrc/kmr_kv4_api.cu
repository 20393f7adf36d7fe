// C ABI of the 4-bit KV cache (declared in kmr.h): argument checks, then the launches of kmr_kv4.cu
// and kmr_kv4_attn.cu.
#include <cmath>
#include <initializer_list>

#include "kmr_kv4.cuh"

using namespace kmr;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int view_of(const kmr_kv4_cache* c, Kv4View* v) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_sz || !c->v_sz) return KMR_ERR_INVALID_ARG;
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_sz) || !aligned16(c->v_sz))
        return KMR_ERR_INVALID_ARG;
    if (c->slots < 1 || c->n_kv_heads < 1 || c->n_kv_heads > kKv4MaxHeads) return KMR_ERR_SHAPE;
    if (c->max_len < 16 || c->max_len % 16 || c->max_len > kKv4MaxLen) return KMR_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return KMR_ERR_SHAPE;
    if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->head_dim) return KMR_ERR_SHAPE;
    v->kc = static_cast<uint8_t*>(c->k_codes);
    v->vc = static_cast<uint8_t*>(c->v_codes);
    v->ks = static_cast<uint32_t*>(c->k_sz);
    v->vs = static_cast<uint32_t*>(c->v_sz);
    v->slots = c->slots;
    v->nkv = c->n_kv_heads;
    v->S = c->max_len;
    v->d = c->head_dim;
    v->g = c->group;
    return KMR_OK;
}

bool overlap(const void* a, size_t abytes, const void* b, size_t bbytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bbytes && y < x + abytes;
}

bool heads_ok(int nq, int nkv) { return nq >= 1 && nq % nkv == 0 && nq / nkv <= kKv4MaxRep; }

int convert(const kmr_kv4_cache* cache, uint16_t* k16, uint16_t* v16, int slots16, int max_len16, const int32_t* slot16,
            const int32_t* start16, const int32_t* slot_ids, const int32_t* start, const int32_t* lengths, int B, int T,
            bool to_bf16, void* stream) {
    Kv4ConvertParams p = {};
    const int rc = view_of(cache, &p.c);
    if (rc != KMR_OK) return rc;
    if (!k16 || !v16 || !slot16 || !start16 || !slot_ids || !start || !lengths) return KMR_ERR_INVALID_ARG;
    if (!aligned16(k16) || !aligned16(v16) || T < 1 || T > kKv4MaxLen) return KMR_ERR_INVALID_ARG;
    if (slots16 < 1 || max_len16 < 1) return KMR_ERR_SHAPE;
    if (B < 1 || B > kKv4MaxRows) return KMR_ERR_BATCH;
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    p.k16 = k16;
    p.v16 = v16;
    p.slots16 = slots16;
    p.S16 = max_len16;
    p.slot16 = slot16;
    p.start16 = start16;
    p.slot_ids = slot_ids;
    p.start = start;
    p.lengths = lengths;
    p.B = B;
    p.T = T;
    return launch_kv4_convert(p, to_bf16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}

// A number as the sum of two doubles, some 2^-104 of it (Dekker 1971; products by an exact fused multiply-add).
struct Two {
    double hi, lo;
};
Two sum_of(double a, double b) {                        // |a| >= |b|
    const double s = a + b;
    return {s, b - (s - a)};
}
Two operator*(Two a, Two b) {
    const double p = a.hi * b.hi, e = std::fma(a.hi, b.hi, -p);
    return sum_of(p, e + (a.hi * b.lo + a.lo * b.hi));
}
Two root(Two a) {
    const double x = std::sqrt(a.hi), e = std::fma(-x, x, a.hi);
    return sum_of(x, (e + a.lo) / (2.0 * x));
}
// The fraction of x, rounded to 2^-64.
unsigned long long fraction_of(Two x) {
    const double top = (x.hi - std::floor(x.hi)) * 0x1p64, whole = std::floor(top);      // exact
    const double rest = (x.lo - std::floor(x.lo + 0.5)) * 0x1p64 + (top - whole);
    return (unsigned long long)whole + (unsigned long long)std::llrint(std::fmin(rest, 0x1.fffffffffffffp62));
}

// theta^(-i / half) / 2 pi turns per position, modulo one turn, as 64-bit fractions: half is 32 or 64, so the step
// theta^(-1 / half) is five or six square roots.
void rope_turns(float theta, int half, unsigned long long* turn) {
    const double t = theta, q = 1.0 / t;
    Two step = {q, std::fma(-q, t, 1.0) / t};
    for (int n = half; n > 1; n /= 2) step = root(step);
    constexpr int kChains = 8;
    Two v[kChains] = {{0.15915494309189535, -9.839338337591243e-18}}, far = step;
    for (int i = 1; i < kChains; ++i) v[i] = v[i - 1] * step;
    for (int n = 1; n < kChains; n *= 2) far = far * far;
    for (int i = 0; i < half; ++i) {
        turn[i] = fraction_of(v[i % kChains]);
        v[i % kChains] = v[i % kChains] * far;
    }
}

}  // namespace

extern "C" int kmr_kv4_append(const kmr_kv4_cache* cache, const float* qkv, const int32_t* positions,
                              const int32_t* slot_ids, const int32_t* cache_position, const int32_t* n_tokens, int B,
                              int T, int nq, const uint16_t* q_norm, const uint16_t* k_norm, float eps,
                              float rope_theta, const int* sections, float* q_out, float* mass, void* stream) {
    Kv4AppendParams p = {};
    const int rc = view_of(cache, &p.c);
    if (rc != KMR_OK) return rc;
    if (!qkv || !positions || !slot_ids || !cache_position || !sections || !q_out) return KMR_ERR_INVALID_ARG;
    if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(q_norm) || !aligned16(k_norm)) return KMR_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps) || !(rope_theta > 0.f) || std::isinf(rope_theta) || T < 1 || T > kKv4MaxLen)
        return KMR_ERR_INVALID_ARG;
    if (B < 1 || B > kKv4MaxRows) return KMR_ERR_BATCH;
    if (!heads_ok(nq, p.c.nkv)) return KMR_ERR_SHAPE;
    const int half = p.c.d / 2;
    if (sections[0] < 0 || sections[1] < 0 || sections[2] < 0 || sections[0] > half || sections[1] > half ||
        sections[2] > half || sections[0] + sections[1] + sections[2] != half)
        return KMR_ERR_SHAPE;
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    p.qkv = qkv;
    p.positions = positions;
    p.slot_ids = slot_ids;
    p.cpos = cache_position;
    p.n_tokens = n_tokens;
    p.B = B;
    p.T = T;
    p.nq = nq;
    p.qn_w = q_norm;
    p.kn_w = k_norm;
    p.eps = eps;
    p.sec0 = sections[0];
    p.sec1 = sections[1];
    p.q_out = q_out;
    p.mass = mass;
    rope_turns(rope_theta, half, p.turn);
    return launch_kv4_append(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}

extern "C" int kmr_kv4_from_bf16(const kmr_kv4_cache* cache, const uint16_t* k_bf16, const uint16_t* v_bf16,
                                 int bf16_slots, int bf16_max_len, const int32_t* bf16_slot_ids,
                                 const int32_t* bf16_start, const int32_t* slot_ids, const int32_t* start,
                                 const int32_t* lengths, int B, int max_tokens, void* stream) {
    return convert(cache, const_cast<uint16_t*>(k_bf16), const_cast<uint16_t*>(v_bf16), bf16_slots, bf16_max_len,
                   bf16_slot_ids, bf16_start, slot_ids, start, lengths, B, max_tokens, false, stream);
}

extern "C" int kmr_kv4_to_bf16(const kmr_kv4_cache* cache, uint16_t* k_bf16, uint16_t* v_bf16, int bf16_slots,
                               int bf16_max_len, const int32_t* bf16_slot_ids, const int32_t* bf16_start,
                               const int32_t* slot_ids, const int32_t* start, const int32_t* lengths, int B,
                               int max_tokens, void* stream) {
    return convert(cache, k_bf16, v_bf16, bf16_slots, bf16_max_len, bf16_slot_ids, bf16_start, slot_ids, start, lengths,
                   B, max_tokens, true, stream);
}

extern "C" size_t kmr_decode_attn_kv4_workspace_size(const kmr_kv4_cache* cache, int B, int nq, int with_mass) {
    Kv4View v;
    if (view_of(cache, &v) != KMR_OK || B < 1 || B > kKv4MaxRows || !heads_ok(nq, v.nkv)) return 0;
    const int ns = kv4_attn_splits(v.S);
    if (ns == 0) return 16;                       // merged on chip: any buffer will do
    return kv4_attn_part_bytes(B, nq, v.d, ns) + (with_mass ? size_t(B) * nq * v.S * 4 : 0);
}

extern "C" int kmr_decode_attn_kv4(const kmr_kv4_cache* cache, const float* q, const int32_t* slot_ids,
                                   const int32_t* cache_position, int B, int nq, float scale, float* mass, float* out,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    Kv4AttnParams p = {};
    const int rc = view_of(cache, &p.c);
    if (rc != KMR_OK) return rc;
    if (!q || !slot_ids || !cache_position || !out || !workspace) return KMR_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned16(mass) || !std::isfinite(scale))
        return KMR_ERR_INVALID_ARG;
    if (B < 1 || B > kKv4MaxRows) return KMR_ERR_BATCH;
    if (!heads_ok(nq, p.c.nkv)) return KMR_ERR_SHAPE;
    if (workspace_bytes < kmr_decode_attn_kv4_workspace_size(cache, B, nq, mass != nullptr)) return KMR_ERR_BUFFER_SIZE;
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    p.q = q;
    p.slot_ids = slot_ids;
    p.cpos = cache_position;
    p.B = B;
    p.nq = nq;
    p.scale = scale;
    p.mass = mass;
    p.out = out;
    p.nsplit = kv4_attn_splits(p.c.S);
    p.part = static_cast<float*>(workspace);
    p.scores = mass ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                               kv4_attn_part_bytes(B, nq, p.c.d, p.nsplit))
                    : nullptr;
    return launch_kv4_attn(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}

extern "C" int kmr_kv4_evict(const kmr_kv4_cache* src, const kmr_kv4_cache* dst, const int32_t* src_slot_ids,
                             const int32_t* dst_slot_ids, const int32_t* lengths, int B, int keep, int recent,
                             const float* mass, float* dst_mass, int32_t* kept, int32_t* new_lengths, void* stream) {
    Kv4EvictParams p = {};
    int rc = view_of(src, &p.src);
    if (rc == KMR_OK) rc = view_of(dst, &p.dst);
    if (rc != KMR_OK) return rc;
    if (!src_slot_ids || !dst_slot_ids || !lengths || !mass || !kept || !new_lengths) return KMR_ERR_INVALID_ARG;
    if (keep < 1 || recent < 0 || recent > keep) return KMR_ERR_INVALID_ARG;
    if (B < 1 || B > kKv4MaxRows) return KMR_ERR_BATCH;
    if (p.src.nkv != p.dst.nkv || p.src.d != p.dst.d || p.src.g != p.dst.g) return KMR_ERR_SHAPE;
    if (keep > p.dst.S) return KMR_ERR_CACHE_FULL;
    p.same = p.src.kc == p.dst.kc;
    // one cache has one shape, and one mass only together with it
    if (p.same && (p.src.slots != p.dst.slots || p.src.S != p.dst.S)) return KMR_ERR_SHAPE;
    if (!p.same && mass == dst_mass) return KMR_ERR_INVALID_ARG;
    // every head's CTAs read the row's ids and length, each row those of the others: what is written lies elsewhere
    const size_t ids = size_t(B) * 4, list = ids * p.src.nkv * keep;
    for (const int32_t* in : {src_slot_ids, dst_slot_ids, lengths})
        if (overlap(new_lengths, ids, in, ids) || overlap(kept, list, in, ids)) return KMR_ERR_INVALID_ARG;
    if (overlap(kept, list, new_lengths, ids)) return KMR_ERR_INVALID_ARG;
    if (ensure_kernel_attributes() != cudaSuccess || !(p.err = standalone_error_word())) return KMR_ERR_CUDA;
    p.src_ids = src_slot_ids;
    p.dst_ids = dst_slot_ids;
    p.lengths = lengths;
    p.B = B;
    p.keep = keep;
    p.recent = recent;
    p.mass = mass;
    p.dst_mass = dst_mass;
    p.kept = kept;
    p.new_lengths = new_lengths;
    return launch_kv4_evict(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KMR_OK : KMR_ERR_CUDA;
}
