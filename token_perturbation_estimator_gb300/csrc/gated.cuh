// Launch interfaces of the gated block's tensor-core products (k_gated_tc.cu)
// and of its few rows on the CUDA cores (k_gated_few.cu).
#pragma once
#include "head.cuh"
#include "step.cuh"

namespace dust {

// g and u tile by tile: h of them, or with gh their gradients D.
struct GatedTiles {
    Planes X, Wg, Wu;      // [T][d], [f][d]
    int64_t T, d, f;
    int act;
    void* h;               // forward
    int64_t ld_h;
    const void* gh;        // backward: rows that start on 16 bytes
    int64_t ld_gh;
    Planes D;              // [T rounded up to a tile][2 gated_half(f)]: dG, dU
};
// Columns of D that dG and dU take each: whole tiles.
inline int64_t gated_half(int64_t f) { return (f + kHeadTile - 1) / kHeadTile * kHeadTile; }
cudaError_t launch_gated_tiles(const GatedTiles& a, cudaStream_t s);

// gX = D [Wg; Wu], [gWg; gWu] = D^T X in one launch, and one more where sums
// are cut into slices.
struct GatedCuts { int x, w; };
GatedCuts gated_cuts(int64_t T, int64_t d, int64_t f, int planes);
int64_t gated_acc_floats(int64_t rows, int64_t d, int planes, int cut);
struct GatedProducts {
    Planes X, Wg, Wu, D;
    int64_t T, d, f;
    void* gX;              // or null
    int64_t ld_gx;
    void *gWg, *gWu;       // or null
    bool bf16, gW_bf16, accumulate;
    GatedCuts cuts;
    float *gx_acc, *gw_acc;  // slices' sums (or null)
};
cudaError_t launch_gated_products(const GatedProducts& a, cudaStream_t s);

constexpr int64_t kGatedFew = 4;  // rows that take the CUDA cores (forward)
cudaError_t launch_gated_few(const GatedProblem& p, void* h, int64_t ld_h, cudaStream_t s);

}  // namespace dust
