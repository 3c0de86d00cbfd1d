// Launch interface of the head's losses and gradients (k_head.cu).
#pragma once
#include "internal.cuh"

namespace dust {

// What each token is to be scored against: one target id (K = 1, no teacher),
// or K teacher entries.
struct HeadTargets {
    const int32_t* ids;     // [T][K]; outside [0, V): absent
    const float* teacher;   // [T][K] teacher logits, or null
    int64_t K;
};

struct HeadProblem {
    const void* H;          // [S * T][d], row stride ld_h
    const void* E;          // [V][d], row stride ld_e
    int64_t ld_h, ld_e;
    bool bf16;
    int64_t S, T, d, V;
    HeadTargets tg;
    float scale;
};

size_t head_loss_workspace_bytes(int64_t R, int64_t d, int64_t V, bool distill, bool bf16);
size_t head_grad_workspace_bytes(int64_t R, int64_t d, int64_t V, bool bf16);
// student: the picked logits [S * T][K] (distillation only).
cudaError_t launch_head_loss(const HeadProblem& p, float* loss, float* lse, float* student,
                             float* delta, void* ws, cudaStream_t s);
cudaError_t launch_head_grad(const HeadProblem& p, const float* lse, const float* student,
                             const float* gloss, bool accumulate, void* gH, int64_t ld_gh,
                             void* gE, bool gE_bf16, void* ws, cudaStream_t s);

}  // namespace dust
