// Products whose weights each token chooses: the expert router, the int4 experts and the adapters
// (parameter blocks and launches; the C ABI in kmr_moe_api.cu checks the arguments).
#pragma once

#include "kmr_internal.cuh"

namespace kmr {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;
constexpr int kMoeMaxDim = 8192;             // hidden and intermediate sizes, multiples of 128
constexpr int kMoeMaxTokens = 1 << 20;
constexpr int kMoeSmallPlaces = 32;          // most places (token, j) of the small form: a warp's lanes
constexpr int kMoeSmallTokens = 16;          // its most tokens
constexpr long long kMoeSmallWeights = 3ll << 26;    // and weights of the places' experts, each counted by itself
constexpr int kMoeSmallCtas = 128;           // fewest CTAs of gate_up, which its sizes are made for (a GB300 has 152 SMs)

// ------------------------------------------------------------------ router
struct MoeRouteParams {
    const void* logits;                      // [T][E] fp32 or bf16
    int T, E, k, renorm;
    int32_t* ids;                            // [T][k]
    float* weights;                          // [T][k]
};
cudaError_t launch_moe_route(const MoeRouteParams& p, bool bf16, cudaStream_t st);
cudaError_t moe_route_set_attributes();

// ------------------------------------------------------------------ experts
struct MoeView {
    const uint8_t* gate_up;                  // [E] KMR4 matrices [2I, H], gate / up tiles interleaved
    const uint8_t* down;                     // [E] KMR4 matrices [H, I]
    int E, H, I;
};
// Small form: up to kMoeSmallPlaces places whose rows fit into shared memory beside two tiles of weights.
struct MoeSmallParams {
    MoeView w;
    const void* x;                           // [T][H]
    const int32_t* ids;                      // [T][k]
    const float* weights;                    // [T][k]
    int T, k;                                // T * k <= kMoeSmallPlaces
    float* act;                              // [T * k][I]
    void* y;                                 // [T][H]
    int resid;                               // add to y
    int stages, batch, list;                 // ring of `stages` tiles, `batch` of them at a time, `list` in all (set by the launch)
    uint32_t by_tiles, by_grid;              // 2^32 / gate_up tiles of an expert, 2^32 / CTAs, rounded up (set by the launch)
    int* err;
};
bool moe_small_fits(const MoeView& w, bool bf16, int T, int k);
cudaError_t launch_moe_small(const MoeSmallParams& p, bool bf16, int sms, cudaStream_t st);
cudaError_t moe_small_set_attributes();

// Grouped form (kmr_moe_tc.cu).
constexpr int kMoeChunkPlaces = 32768;       // places of one pass (a rank within an expert fits 16 bits)
struct MoeTcParams {
    MoeView w;
    const float* rho_gate_up;                // [E][2I] row factors, packed row order
    const float* rho_down;                   // [E][H]
    const float* norms;                      // [E] bounds of the down rows' norms
    const void* x;                           // [T][H]
    const int32_t* ids;                      // [T][k]
    const float* weights;                    // [T][k]
    int T, k, cap;                           // most tokens of a tile: 16, 32, 64 or 128
    int* ntiles;
    int4* tiles;                             // (expert, first position, tokens with padding, tokens)
    int32_t* pos;                            // [T][k]: the place's position, or -1
    float* isx;                              // [P] 1 / scale of the position's inputs
    float* isa;                              // [P] 1 / scale of its activations
    float* sout;                             // [P] bf16: scale of its result while it waits for the sum (fp32: not used)
    size_t blocks;                           // P / 8
    uint8_t* xs;                             // staged inputs
    uint8_t* as;                             // staged activations
    void* out;                               // [P][I] fp32: activations; then [P][H]: results, fp16 (bf16) or fp32
    void* y;                                 // [T][H]
    int resid;
    int* err;
};
// Byte offsets into the workspace (the tile count comes first), and the blocks of 8 positions.
struct MoeTcSizes {
    size_t tiles, pos, isx, isa, sout, xs, as, out, total, blocks;
};
int moe_tc_cap(long long places, int E, bool bf16);
MoeTcSizes moe_tc_sizes(const MoeView& w, bool bf16, int T, int k);
cudaError_t launch_moe_tc(const MoeTcParams& p, bool bf16, int sms, cudaStream_t st);
cudaError_t launch_moe_factors(const MoeView& w, float* rho_gate_up, float* rho_down, float* norms, cudaStream_t st);
cudaError_t moe_tc_set_attributes();

// ------------------------------------------------------------------ adapters
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxDim = 1 << 28;         // inputs and outputs: a row's byte offsets are 32-bit numbers
struct LoraParams {
    const uint16_t* a;                       // bf16 [L][r][K]
    const uint16_t* b;                       // bf16 [L][N][r]
    const int32_t* ranks;                    // [L] or null: r
    const float* scales;                     // [L] or null: 1
    int L, K, N, r;
    const void* x;                           // [T] rows of K, ldx apart
    const void* base;                        // [T] rows of N, ldy apart, or null (zeros)
    void* y;                                 // [T] rows of N, ldy apart
    long long ldx, ldy;
    const int32_t* ids;                      // [T]
    int T;
    int* err;
};
cudaError_t launch_lora(const LoraParams& p, bool bf16, int sms, cudaStream_t st);
cudaError_t lora_set_attributes();

// Every kernel of this part is launched as a programmatic dependent of whatever ran before it on the stream and
// waits for that before it reads or writes memory: the launch itself overlaps the end of the previous kernel.
inline cudaError_t launch_dependent(const void* fn, dim3 grid, int threads, size_t smem, int cluster, const void* params,
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

}  // namespace kmr
