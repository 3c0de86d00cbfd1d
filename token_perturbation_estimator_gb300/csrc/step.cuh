// Launch interfaces of the operators of a training step around the estimator:
// k_gated.cu (gated feed-forward block), k_rope.cu (queries' and keys' norms
// and rotation), k_policy.cu (policy loss), k_clip.cu (gradient norm).
#pragma once
#include "internal.cuh"

namespace dust {

struct GatedProblem {
    const void *X, *Wg, *Wu;
    int64_t ld_x, ld_wg, ld_wu;
    bool bf16;
    int64_t T, d, f;
    int act;                   // dust_act
};
size_t gated_workspace_bytes(const GatedProblem& p);
size_t gated_grad_workspace_bytes(const GatedProblem& p);
cudaError_t launch_gated(const GatedProblem& p, void* h, int64_t ld_h, void* ws, cudaStream_t s);
cudaError_t launch_gated_grad(const GatedProblem& p, const void* gh, int64_t ld_gh, bool accumulate,
                              void* gX, int64_t ld_gx, void* gWg, void* gWu, bool gW_bf16, void* ws,
                              cudaStream_t s);

// The heads of one operand, and those of its output and gradient.
struct RopeSide {
    dust_heads x, y, gy;       // input; output or input's gradient; output's gradient
    int64_t heads;
    const float* w;            // or null
    float* gw;                 // or null
};
struct RopeProblem {
    RopeSide side[2];          // queries, keys
    bool bf16;
    int64_t T, D;
    float eps;
    const int32_t* positions;
    const float *cosine, *sine;
    int64_t n_pos, rot;
    int layout;                // dust_rope_layout
};
size_t rope_grad_workspace_bytes(int64_t T, int64_t heads, int64_t D);
cudaError_t launch_rope(const RopeProblem& p, cudaStream_t s);
cudaError_t launch_rope_grad(const RopeProblem& p, bool accumulate, void* ws, cudaStream_t s);

struct PolicyProblem {
    const float *nll, *old, *ref, *advantages;
    bool per_token;
    const int32_t *offsets, *targets;
    int64_t n_seq, S, T;
    double low, high;          // bounds of old - nll
    float low32, high32;       // the same, rounded
    float least, most;         // the ratio's bounds
    float beta;
    bool by_sequence;
};
size_t policy_workspace_bytes(int64_t S, int64_t T, int64_t n_seq);
cudaError_t launch_policy(const PolicyProblem& p, float* loss, float* total, float* kl,
                          float* clipped, float* delta, void* ws, cudaStream_t s);
cudaError_t launch_policy_grad(const PolicyProblem& p, const float* gtotal, float* gnll, void* ws,
                               cudaStream_t s);

constexpr int64_t kMaxGrads = 4096;
size_t clip_workspace_bytes();
cudaError_t launch_clip(const dust_grad* grads, int64_t n, float max_norm, float* norm, void* ws,
                        cudaStream_t s);

}  // namespace dust
