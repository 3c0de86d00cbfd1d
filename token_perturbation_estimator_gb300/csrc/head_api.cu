// C ABI of the layer norm, the head's losses and the distillation
// (include/dust.h): argument checks and dispatch.
#include <cmath>

#include "dust.h"
#include "head.cuh"

using namespace dust;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Of the head's rows, columns and ids: their numbers, padded to whole tiles
// and to the row pass's thousands, fit 32 bits (the kernels' and TMA's).
constexpr int64_t kMaxHeadDim = (int64_t(1) << 31) - (int64_t(1) << 16);
constexpr int64_t kMaxHeadTiles = int64_t(1) << 30;  // of 256 rows x 128 ids, in a launch

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

dust_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DUST_OK : DUST_ERR_CUDA; }

bool value_dtype(dust_dtype t) { return t == DUST_F32 || t == DUST_BF16; }

// Whether p is a multiple of its element's size (any pointer a program gets
// from an allocation or by stepping whole elements is).
bool aligned_to(const void* p, dust_dtype t) {
    return reinterpret_cast<uintptr_t>(p) % (t == DUST_BF16 ? 2 : 4) == 0;
}

bool ws_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}

dust_status check_norm(dust_dtype dtype, int64_t T, int64_t d) {
    if (T < 0 || d < 0 || !value_dtype(dtype)) return DUST_ERR_INVALID_ARG;
    if (T > kMaxDim || d > kMaxDim || (d > 0 && T > kMaxElems / d)) return DUST_ERR_RANGE;
    return DUST_OK;
}

dust_status check_head_sizes(int64_t S, int64_t T, int64_t d, int64_t V, dust_dtype dtype) {
    if (S < 1 || T < 0 || d < 1 || V < 1 || !value_dtype(dtype)) return DUST_ERR_INVALID_ARG;
    if (T > kMaxHeadDim / S || d > kMaxHeadDim || V > kMaxHeadDim) return DUST_ERR_RANGE;
    if ((T > 0 && S * T > kMaxElems / d) || V > kMaxElems / d) return DUST_ERR_RANGE;
    if ((S * T + 255) / 256 * ((V + 127) / 128) > kMaxHeadTiles) return DUST_ERR_RANGE;
    return DUST_OK;
}

dust_status check_teacher_sizes(int64_t S, int64_t T, int64_t K) {
    if (K < 1) return DUST_ERR_INVALID_ARG;
    if (K > DUST_MAX_TEACHER || (T > 0 && S * T > kMaxElems / K)) return DUST_ERR_RANGE;
    return DUST_OK;
}

// A problem's sizes alone, for the workspace queries.
HeadProblem sizes(int64_t S, int64_t T, int64_t d, int64_t V, int64_t K, bool distill,
                  dust_dtype dtype) {
    return {nullptr, nullptr, d, d, dtype == DUST_BF16, S, T, d, V, {nullptr, nullptr, K, distill},
            1.0f};
}

// The checks shared by the four head calls, in one place: sizes, scale,
// strides, and (for T > 0) the inputs' pointers.
dust_status check_head(const void* H, int64_t ld_h, const void* E, int64_t ld_e, dust_dtype dtype,
                       int64_t S, int64_t T, int64_t d, int64_t V, const int32_t* ids,
                       float scale) {
    const dust_status st = check_head_sizes(S, T, d, V, dtype);
    if (st != DUST_OK) return st;
    if (!std::isfinite(scale) || ld_h < d || ld_e < d) return DUST_ERR_INVALID_ARG;
    // Strides too: no row may start beyond 2^40 elements.
    if ((T > 0 && ld_h > kMaxElems / (S * T)) || ld_e > kMaxElems / V) return DUST_ERR_RANGE;
    if (T > 0 && (!H || !E || !ids || !aligned_to(H, dtype) || !aligned_to(E, dtype)))
        return DUST_ERR_INVALID_ARG;
    return DUST_OK;
}

dust_status run_loss(const HeadProblem& p, float* loss, float* lse, float* student, float* delta,
                     size_t need, void* ws, size_t ws_bytes, void* stream) {
    if (!lse || (p.tg.many && !student)) return DUST_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, need)) return DUST_ERR_WORKSPACE;
    return cuda_status(launch_head_loss(p, loss, lse, student, delta, ws,
                                        static_cast<cudaStream_t>(stream)));
}

dust_status check_grad(uint32_t flags, dust_dtype dtype, int64_t S, int64_t T, int64_t d,
                       const void* gH, int64_t ld_gh, const void* gE, dust_dtype gE_dtype) {
    if (flags & ~static_cast<uint32_t>(DUST_ACCUMULATE)) return DUST_ERR_INVALID_ARG;
    if (gE) {
        if (!value_dtype(gE_dtype) || (gE_dtype == DUST_BF16 && dtype != DUST_BF16))
            return DUST_ERR_INVALID_ARG;
        if ((flags & DUST_ACCUMULATE) && gE_dtype != DUST_F32) return DUST_ERR_INVALID_ARG;
        if (!aligned_to(gE, gE_dtype)) return DUST_ERR_INVALID_ARG;
    }
    if (gH) {
        if (ld_gh < d || !aligned_to(gH, dtype)) return DUST_ERR_INVALID_ARG;
        if (T > 0 && ld_gh > kMaxElems / (S * T)) return DUST_ERR_RANGE;
    }
    return DUST_OK;
}

// T = 0: no row adds to gE.
dust_status empty_grad(int64_t V, int64_t d, uint32_t flags, void* gE, dust_dtype gE_dtype,
                       void* stream) {
    if (!gE || (flags & DUST_ACCUMULATE)) return DUST_OK;
    return cuda_status(cudaMemsetAsync(
        gE, 0, static_cast<size_t>(V) * static_cast<size_t>(d) * (gE_dtype == DUST_BF16 ? 2 : 4),
        static_cast<cudaStream_t>(stream)));
}

dust_status run_grad(const HeadProblem& p, const float* lse, const float* student,
                     const float* gloss, uint32_t flags, void* gH, int64_t ld_gh, void* gE,
                     dust_dtype gE_dtype, size_t need, void* ws, size_t ws_bytes, void* stream) {
    if (!lse || !gloss || (p.tg.many && !student)) return DUST_ERR_INVALID_ARG;
    if (!gH && !gE) return DUST_OK;
    if (!ws_ok(ws, ws_bytes, need)) return DUST_ERR_WORKSPACE;
    return cuda_status(launch_head_grad(p, lse, student, gloss, (flags & DUST_ACCUMULATE) != 0, gH,
                                        ld_gh, gE, gE_dtype == DUST_BF16, ws,
                                        static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

dust_status dust_layer_norm(const void* x, dust_dtype dtype, int64_t ld_x, int64_t T, int64_t d,
                            const float* weight, const float* bias, float eps, void* y,
                            int64_t ld_y, float* mean, float* rstd, void* stream) {
    const dust_status st = check_norm(dtype, T, d);
    if (st != DUST_OK) return st;
    if (ld_x < d || ld_y < d || !std::isfinite(eps) || eps < 0.0f) return DUST_ERR_INVALID_ARG;
    if (T * d == 0) return DUST_OK;
    if (ld_x > kMaxElems / T || ld_y > kMaxElems / T) return DUST_ERR_RANGE;
    if (!x || !y || !aligned_to(x, dtype) || !aligned_to(y, dtype)) return DUST_ERR_INVALID_ARG;
    return cuda_status(launch_layer_norm(x, dtype == DUST_BF16, ld_x, T, d, weight, bias, eps, y,
                                         ld_y, mean, rstd, static_cast<cudaStream_t>(stream)));
}

dust_status dust_layer_norm_grad_workspace(size_t* bytes, int64_t T, int64_t d) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_norm(DUST_F32, T, d);
    if (st != DUST_OK) return st;
    *bytes = a256(layer_norm_grad_workspace_bytes(T, d));
    return DUST_OK;
}

dust_status dust_layer_norm_grad(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x,
                                 dust_dtype dtype, int64_t T, int64_t d, const float* weight,
                                 const float* mean, const float* rstd, uint32_t flags, void* gx,
                                 int64_t ld_gx, float* gweight, float* gbias, void* workspace,
                                 size_t ws_bytes, void* stream) {
    const dust_status st = check_norm(dtype, T, d);
    if (st != DUST_OK) return st;
    if (ld_gy < d || ld_x < d || (gx && ld_gx < d)) return DUST_ERR_INVALID_ARG;
    if (flags & ~static_cast<uint32_t>(DUST_ACCUMULATE)) return DUST_ERR_INVALID_ARG;
    const bool acc = (flags & DUST_ACCUMULATE) != 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d == 0 || (!gx && !gweight && !gbias)) return DUST_OK;
    if (T == 0) {
        for (float* p : {gweight, gbias})
            if (p && !acc) {
                const cudaError_t e = cudaMemsetAsync(p, 0, sizeof(float) * static_cast<size_t>(d), s);
                if (e != cudaSuccess) return DUST_ERR_CUDA;
            }
        return DUST_OK;
    }
    if (ld_gy > kMaxElems / T || ld_x > kMaxElems / T || (gx && ld_gx > kMaxElems / T))
        return DUST_ERR_RANGE;
    if (!gy || !x || !mean || !rstd) return DUST_ERR_INVALID_ARG;
    if (!aligned_to(gy, dtype) || !aligned_to(x, dtype) || !aligned_to(gx, dtype))
        return DUST_ERR_INVALID_ARG;
    if ((gweight || gbias) &&
        !ws_ok(workspace, ws_bytes, a256(layer_norm_grad_workspace_bytes(T, d))))
        return DUST_ERR_WORKSPACE;
    return cuda_status(launch_layer_norm_grad(gy, ld_gy, x, ld_x, dtype == DUST_BF16, T, d, weight,
                                              mean, rstd, acc, gx, ld_gx, gweight, gbias,
                                              static_cast<float*>(workspace), s));
}

dust_status dust_head_loss_workspace(size_t* bytes, int64_t S, int64_t T, int64_t d, int64_t V,
                                     dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_head_sizes(S, T, d, V, dtype);
    if (st != DUST_OK) return st;
    *bytes = head_loss_workspace_bytes(sizes(S, T, d, V, 1, false, dtype));
    return DUST_OK;
}

dust_status dust_head_loss(const void* H, int64_t ld_h, const void* E, int64_t ld_e,
                           dust_dtype dtype, int64_t S, int64_t T, int64_t d, int64_t V,
                           const int32_t* targets, float scale, float* loss, float* lse,
                           float* delta, void* workspace, size_t ws_bytes, void* stream) {
    const dust_status st = check_head(H, ld_h, E, ld_e, dtype, S, T, d, V, targets, scale);
    if (st != DUST_OK || T == 0) return st;
    const HeadProblem p = {H, E, ld_h, ld_e, dtype == DUST_BF16, S, T, d, V,
                           {targets, nullptr, 1, false}, scale};
    return run_loss(p, loss, lse, nullptr, delta,
                    head_loss_workspace_bytes(p), workspace, ws_bytes,
                    stream);
}

dust_status dust_head_loss_grad_workspace(size_t* bytes, int64_t S, int64_t T, int64_t d,
                                          int64_t V, dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_head_sizes(S, T, d, V, dtype);
    if (st != DUST_OK) return st;
    *bytes = head_grad_workspace_bytes(sizes(S, T, d, V, 1, false, dtype));
    return DUST_OK;
}

dust_status dust_head_loss_grad(const void* H, int64_t ld_h, const void* E, int64_t ld_e,
                                dust_dtype dtype, int64_t S, int64_t T, int64_t d, int64_t V,
                                const int32_t* targets, float scale, const float* lse,
                                const float* gloss, uint32_t flags, void* gH, int64_t ld_gh,
                                void* gE, dust_dtype gE_dtype, void* workspace, size_t ws_bytes,
                                void* stream) {
    dust_status st = check_head(H, ld_h, E, ld_e, dtype, S, T, d, V, targets, scale);
    if (st == DUST_OK) st = check_grad(flags, dtype, S, T, d, gH, ld_gh, gE, gE_dtype);
    if (st != DUST_OK) return st;
    if (T == 0) return empty_grad(V, d, flags, gE, gE_dtype, stream);
    const HeadProblem p = {H, E, ld_h, ld_e, dtype == DUST_BF16, S, T, d, V,
                           {targets, nullptr, 1, false}, scale};
    return run_grad(p, lse, nullptr, gloss, flags, gH, ld_gh, gE, gE_dtype,
                    head_grad_workspace_bytes(p), workspace, ws_bytes, stream);
}

dust_status dust_distill_loss_workspace(size_t* bytes, int64_t S, int64_t T, int64_t d,
                                        int64_t V, int64_t K, dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    dust_status st = check_head_sizes(S, T, d, V, dtype);
    if (st == DUST_OK) st = check_teacher_sizes(S, T, K);
    if (st != DUST_OK) return st;
    *bytes = head_loss_workspace_bytes(sizes(S, T, d, V, K, true, dtype));
    return DUST_OK;
}

dust_status dust_distill_loss(const void* H, int64_t ld_h, const void* E, int64_t ld_e,
                              dust_dtype dtype, int64_t S, int64_t T, int64_t d, int64_t V,
                              const int32_t* ids, const float* teacher, int64_t K, float scale,
                              float* loss, float* lse, float* student, float* delta,
                              void* workspace, size_t ws_bytes, void* stream) {
    dust_status st = check_head(H, ld_h, E, ld_e, dtype, S, T, d, V, ids, scale);
    if (st == DUST_OK) st = check_teacher_sizes(S, T, K);
    if (st != DUST_OK || T == 0) return st;
    if (!teacher) return DUST_ERR_INVALID_ARG;
    const HeadProblem p = {H, E, ld_h, ld_e, dtype == DUST_BF16, S, T, d, V,
                           {ids, teacher, K, true}, scale};
    return run_loss(p, loss, lse, student, delta,
                    head_loss_workspace_bytes(p), workspace, ws_bytes,
                    stream);
}

dust_status dust_distill_loss_grad_workspace(size_t* bytes, int64_t S, int64_t T, int64_t d,
                                             int64_t V, int64_t K, dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    dust_status st = check_head_sizes(S, T, d, V, dtype);
    if (st == DUST_OK) st = check_teacher_sizes(S, T, K);
    if (st != DUST_OK) return st;
    *bytes = head_grad_workspace_bytes(sizes(S, T, d, V, K, true, dtype));
    return DUST_OK;
}

dust_status dust_distill_loss_grad(const void* H, int64_t ld_h, const void* E, int64_t ld_e,
                                   dust_dtype dtype, int64_t S, int64_t T, int64_t d, int64_t V,
                                   const int32_t* ids, const float* teacher, int64_t K,
                                   float scale, const float* lse, const float* student,
                                   const float* gloss, uint32_t flags, void* gH, int64_t ld_gh,
                                   void* gE, dust_dtype gE_dtype, void* workspace,
                                   size_t ws_bytes, void* stream) {
    dust_status st = check_head(H, ld_h, E, ld_e, dtype, S, T, d, V, ids, scale);
    if (st == DUST_OK) st = check_teacher_sizes(S, T, K);
    if (st == DUST_OK) st = check_grad(flags, dtype, S, T, d, gH, ld_gh, gE, gE_dtype);
    if (st != DUST_OK) return st;
    if (T == 0) return empty_grad(V, d, flags, gE, gE_dtype, stream);
    if (!teacher) return DUST_ERR_INVALID_ARG;
    const HeadProblem p = {H, E, ld_h, ld_e, dtype == DUST_BF16, S, T, d, V,
                           {ids, teacher, K, true}, scale};
    return run_grad(p, lse, student, gloss, flags, gH, ld_gh, gE, gE_dtype,
                    head_grad_workspace_bytes(p), workspace, ws_bytes, stream);
}

}  // extern "C"
