// Layer norm, forward and backward. Per row of d values, n = (x - mean) rstd:
//     y  = n weight + bias
//     gx = rstd (gn - mean(gn) - n mean(gn n)),  gn = gy weight
//     gweight = sum_t gy n,  gbias = sum_t gy
// Bound by memory: the forward reads x and writes y once, the backward reads
// gy and x and writes gx once.
//
// A warp takes a row and goes over it once per sum (the later passes come
// from L1/L2). The gradients of weight and bias are summed per row chunk by
// a thread per column, then over the chunks in order: deterministic.
#include "internal.cuh"

namespace dust {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

constexpr int kRows = 8;           // rows (warps) per CTA
constexpr int kColRows = 8;        // row lanes of the column sums
constexpr int64_t kMaxChunks = 256;  // row chunks of the column sums

template <typename TX>
__global__ void __launch_bounds__(32 * kRows)
    k_norm(const TX* x, int64_t ld_x, int64_t T, int64_t d, const float* __restrict__ weight,
           const float* __restrict__ bias, float eps, TX* y, int64_t ld_y, float* mean,
           float* rstd) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x >> 5);
    if (t >= T) return;
    const TX* xr = x + t * ld_x;
    float s = 0.0f;
    for (int64_t c = lane; c < d; c += 32) s += to_f(xr[c]);
    const float mu = warp_sum(s) / static_cast<float>(d);
    float q = 0.0f;
    for (int64_t c = lane; c < d; c += 32) {
        const float e = to_f(xr[c]) - mu;
        q = fmaf(e, e, q);
    }
    const float r = 1.0f / sqrtf(warp_sum(q) / static_cast<float>(d) + eps);
    TX* yr = y + t * ld_y;
    for (int64_t c = lane; c < d; c += 32) {
        const float n = (to_f(xr[c]) - mu) * r;
        yr[c] = from_f<TX>(fmaf(n, weight ? weight[c] : 1.0f, bias ? bias[c] : 0.0f));
    }
    if (lane == 0) {
        if (mean) mean[t] = mu;
        if (rstd) rstd[t] = r;
    }
}

template <typename TX>
__global__ void __launch_bounds__(256)
    k_norm_cols(const TX* __restrict__ gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x,
                int64_t T, int64_t d, const float* __restrict__ mean,
                const float* __restrict__ rstd, int64_t chunk, float* __restrict__ part) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sw[kColRows][32], sb[kColRows][32];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * chunk;
    const int64_t t1 = t0 + chunk < T ? t0 + chunk : T;
    float w = 0.0f, b = 0.0f;
    if (c < d) {
        for (int64_t t = t0 + rl; t < t1; t += kColRows) {
            const float g = to_f(gy[t * ld_gy + c]);
            w = fmaf(g, (to_f(x[t * ld_x + c]) - mean[t]) * rstd[t], w);
            b += g;
        }
    }
    sw[rl][lane] = w;
    sb[rl][lane] = b;
    __syncthreads();
    if (rl == 0 && c < d) {
        for (int i = 1; i < kColRows; ++i) {
            w += sw[i][lane];
            b += sb[i][lane];
        }
        float* p = part + static_cast<int64_t>(blockIdx.y) * 2 * d;
        p[c] = w;
        p[d + c] = b;
    }
}

__global__ void __launch_bounds__(256)
    k_norm_finish(const float* __restrict__ part, int64_t n_chunks, int64_t d, int accumulate,
                  float* gweight, float* gbias) {
    pdl_wait();
    pdl_trigger();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= 2 * d) return;
    float* out = c < d ? gweight : gbias;
    if (!out) return;
    out += c < d ? c : c - d;
    float v = 0.0f;
    for (int64_t k = 0; k < n_chunks; ++k) v += part[k * 2 * d + c];
    *out = accumulate ? *out + v : v;
}

template <typename TX>
__global__ void __launch_bounds__(32 * kRows)
    k_norm_gx(const TX* gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x, int64_t T,
              int64_t d, const float* __restrict__ weight, const float* __restrict__ mean,
              const float* __restrict__ rstd, TX* gx, int64_t ld_gx) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + (threadIdx.x >> 5);
    if (t >= T) return;
    const TX* gr = gy + t * ld_gy;
    const TX* xr = x + t * ld_x;
    const float mu = mean[t], r = rstd[t];
    float a = 0.0f, b = 0.0f;
    for (int64_t c = lane; c < d; c += 32) {
        const float gn = to_f(gr[c]) * (weight ? weight[c] : 1.0f);
        a += gn;
        b = fmaf(gn, (to_f(xr[c]) - mu) * r, b);
    }
    a = warp_sum(a) / static_cast<float>(d);
    b = warp_sum(b) / static_cast<float>(d);
    TX* o = gx + t * ld_gx;
    for (int64_t c = lane; c < d; c += 32) {
        const float gn = to_f(gr[c]) * (weight ? weight[c] : 1.0f);
        const float n = (to_f(xr[c]) - mu) * r;
        o[c] = from_f<TX>(r * (gn - a - n * b));
    }
}

int64_t row_chunk(int64_t T) {
    int64_t chunk = (T + kMaxChunks - 1) / kMaxChunks;
    return chunk < 64 ? 64 : chunk;
}

template <typename TX>
cudaError_t grad_typed(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x, int64_t T,
                       int64_t d, const float* weight, const float* mean, const float* rstd,
                       bool accumulate, void* gx, int64_t ld_gx, float* gweight, float* gbias,
                       float* part, cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    const TX* g = static_cast<const TX*>(gy);
    const TX* xx = static_cast<const TX*>(x);
    cudaError_t e = cudaSuccess;
    if (gweight || gbias) {  // before gx, which may overwrite gy
        const int64_t chunk = row_chunk(T), n = (T + chunk - 1) / chunk;
        e = launch_pdl(k_norm_cols<TX>,
                       dim3(static_cast<unsigned>((d + 31) / 32), static_cast<unsigned>(n)),
                       dim3(256), 0, s, g, ld_gy, xx, ld_x, T, d, mean, rstd, chunk, part);
        if (e != cudaSuccess) return e;
        e = launch_pdl(k_norm_finish, dim3(static_cast<unsigned>((2 * d + 255) / 256)), dim3(256),
                       0, s, part, n, d, accumulate ? 1 : 0, gweight, gbias);
        if (e != cudaSuccess) return e;
    }
    if (gx)
        e = launch_pdl(k_norm_gx<TX>, dim3(static_cast<unsigned>((T + kRows - 1) / kRows)),
                       dim3(32 * kRows), 0, s, g, ld_gy, xx, ld_x, T, d, weight, mean, rstd,
                       static_cast<TX*>(gx), ld_gx);
    return e;
}

}  // namespace

cudaError_t launch_layer_norm(const void* x, int bf16, int64_t ld_x, int64_t T, int64_t d,
                              const float* weight, const float* bias, float eps, void* y,
                              int64_t ld_y, float* mean, float* rstd, cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    const dim3 grid(static_cast<unsigned>((T + kRows - 1) / kRows)), block(32 * kRows);
    if (bf16)
        return launch_pdl(k_norm<__nv_bfloat16>, grid, block, 0, s,
                          static_cast<const __nv_bfloat16*>(x), ld_x, T, d, weight, bias, eps,
                          static_cast<__nv_bfloat16*>(y), ld_y, mean, rstd);
    return launch_pdl(k_norm<float>, grid, block, 0, s, static_cast<const float*>(x), ld_x, T, d,
                      weight, bias, eps, static_cast<float*>(y), ld_y, mean, rstd);
}

size_t layer_norm_grad_workspace_bytes(int64_t T, int64_t d) {
    const int64_t chunk = row_chunk(T), n = (T + chunk - 1) / chunk;
    return sizeof(float) * static_cast<size_t>(2 * n * d);
}

cudaError_t launch_layer_norm_grad(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x,
                                   int bf16, int64_t T, int64_t d, const float* weight,
                                   const float* mean, const float* rstd, bool accumulate, void* gx,
                                   int64_t ld_gx, float* gweight, float* gbias, float* part,
                                   cudaStream_t s) {
    return bf16 ? grad_typed<__nv_bfloat16>(gy, ld_gy, x, ld_x, T, d, weight, mean, rstd,
                                            accumulate, gx, ld_gx, gweight, gbias, part, s)
                : grad_typed<float>(gy, ld_gy, x, ld_x, T, d, weight, mean, rstd, accumulate, gx,
                                    ld_gx, gweight, gbias, part, s);
}

}  // namespace dust
