// The 4-bit KV cache: its format, the attention's split plans and the parameter blocks of its kernels.
//
// A cached vector (one slot, KV head and position; d = 64 or 128 dims) holds 4-bit codes c and,
// for every group of 32, 64 or 128 dims, a bf16 scale s and a bf16 base z: value = c s + z.
// Codes are ordered for the attention kernel's tensor-core fragments (kmr_kv4_attn.cu): with
// nb = d / 32 blocks of 32 dims,
//   K row: [4][nb][8] nibbles, dim 32 b + 8 t + i at [t][b][i]: lane t of a fragment's four lanes
//          reads its 8 dims of every block in one load;
//   V row: [8][nb][4] nibbles, dim 32 b + 4 u + j at [u][b][j]: likewise lane u of eight.
#pragma once

#include "kmr_internal.cuh"

namespace kmr {

constexpr int kKv4MaxRows = 1024;        // rows of one call (each row looks at the others for clashes)
constexpr int kKv4MaxHeads = 1024;       // KV heads
constexpr int kKv4MaxLen = 1 << 28;      // positions of a row
constexpr int kKv4MaxRep = 8;            // query heads per KV head
constexpr int kKv4MaxSplits = 76;        // of a row: with 8 KV heads, four CTAs for each of 152 SMs (fewer heads fill fewer)
constexpr int kKv4ClusterSplits = 8;     // of a row of a short cache: one cluster
constexpr int kKv4ClusterLen = 2048;     // longest max_len of a short cache (measured: kmr_kv4_attn.cu)
constexpr int kKv4MinChunk = 128;        // positions per split, at least

struct Kv4View {
    uint8_t* kc;                         // [slots][nkv][S][d / 2]
    uint8_t* vc;
    uint32_t* ks;                        // [slots][nkv][S][d / g]: z in the low half, s in the high half
    uint32_t* vs;
    int slots, nkv, S, d, g;
};

__device__ __forceinline__ float kv4_s(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float kv4_z(uint32_t w) { return __uint_as_float(w << 16); }

struct Kv4AppendParams {
    Kv4View c;
    const float* qkv;                    // [B][T][(nq + 2 nkv) d]
    const int32_t* positions;            // [3][B][T]
    const int32_t* slot_ids;             // [B]
    const int32_t* cpos;                 // [B]: cache position of the row's token 0
    const int32_t* n_tokens;             // [B] or null: T
    int B, T, nq;
    const uint16_t* qn_w;                // bf16 [d] or null
    const uint16_t* kn_w;
    float eps;
    int sec0, sec1;
    float* q_out;                        // [B][T][nq][d]
    float* mass;                         // [slots][nkv][S] or null
    int* err;
    unsigned long long turn[64];         // frequency i in turns per position, as a 64-bit fraction
};
cudaError_t kv4_set_attributes();
cudaError_t launch_kv4_append(const Kv4AppendParams& p, cudaStream_t st);

struct Kv4ConvertParams {
    Kv4View c;
    uint16_t* k16;                       // bf16 [slots16][nkv][S16][d]
    uint16_t* v16;
    int slots16, S16;
    const int32_t* slot16;               // [B]
    const int32_t* start16;
    const int32_t* slot_ids;
    const int32_t* start;
    const int32_t* lengths;
    int B, T;
    int span;                            // positions of a CTA (set by the launch)
    int* err;
};
cudaError_t launch_kv4_convert(const Kv4ConvertParams& p, bool to_bf16, cudaStream_t st);

struct Kv4AttnParams {
    Kv4View c;
    const float* q;                      // [B][nq][d]
    const int32_t* slot_ids;
    const int32_t* cpos;
    int B, nq;
    float scale;
    float* mass;                         // [slots][nkv][S] or null
    float* out;                          // [B][nq][d]
    float* part;                         // [B][nkv][nsplit][rep][d + 2]
    float* scores;                       // [B][nkv][rep][S] base-2 scores (mass only)
    int nsplit;                          // the most splits a row of a long cache can have (0: a short cache)
    int per;                             // short cache: splits of a CTA (this and the next: set by the launch)
    int score_ld;                        // short cache: positions whose scores a CTA keeps
    int* err;
};
size_t kv4_attn_part_bytes(int B, int nq, int d, int nsplit);
int kv4_attn_splits(int S);
cudaError_t kv4_attn_set_attributes();
cudaError_t launch_kv4_attn(const Kv4AttnParams& p, cudaStream_t st);

struct Kv4EvictParams {
    Kv4View src, dst;
    const int32_t* src_ids;              // [B]
    const int32_t* dst_ids;
    const int32_t* lengths;
    int B, keep, recent;
    int same;                            // source and destination are one cache (or one mass)
    const float* mass;                   // [src.slots][nkv][src.S]
    float* dst_mass;                     // [dst.slots][nkv][dst.S] or null
    int32_t* kept;                       // [B][nkv][keep]
    int32_t* new_lengths;                // [B]
    int* err;
};
cudaError_t launch_kv4_evict(const Kv4EvictParams& p, cudaStream_t st);

// Positions of a row are cut into splits of `chunk` positions (a multiple of 16), by the row's own length
// (and, through the form chosen, by max_len) alone, so that a row's result does not depend on the others of the call.
// Long caches: 128 for short rows, growing to 256 by 4096 positions, and beyond 76 splits with the length.
__host__ __device__ __forceinline__ void kv4_split_plan(int L, int& chunk, int& ns) {
    const int grow = (L + 15) >> 4;
    chunk = (L + kKv4MaxSplits - 1) / kKv4MaxSplits;
    if (chunk < kKv4MinChunk) chunk = kKv4MinChunk;
    if (grow > chunk) chunk = grow < 256 ? grow : (chunk < 256 ? 256 : chunk);
    chunk = (chunk + 15) & ~15;
    ns = (L + chunk - 1) / chunk;
}
// Short caches: 128 to 256 positions, at most 8 splits.
__host__ __device__ __forceinline__ void kv4_cluster_plan(int L, int& chunk, int& ns) {
    chunk = ((L + kKv4ClusterSplits - 1) / kKv4ClusterSplits + 15) & ~15;
    if (chunk < kKv4MinChunk) chunk = kKv4MinChunk;
    ns = (L + chunk - 1) / chunk;
}

}  // namespace kmr
