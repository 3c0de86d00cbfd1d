// The head's per-token losses and their gradients, over the vocabulary in
// pieces and without keeping the logits (include/dust.h gives the formulas):
// softmax cross entropy against a target id, and distillation from a
// teacher's largest logits.
//
// One piece of the vocabulary at a time, the logits x = scale H E^T of all
// rows are formed in the workspace. The forward keeps a running maximum and
// sum per row (rescaled when the maximum grows) and picks the logits of the
// target or of the teacher's entries; the backward turns the piece into
// G = gloss (exp(x - lse) - wanted) in place and adds its part of gH = G E,
// and its rows of gE = G^T H. The products run on the CUDA cores in fp32.
#include <cmath>

#include "head.cuh"

namespace dust {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

constexpr int64_t kPiece = 4096;  // vocabulary rows a piece

constexpr int kTile = 64, kDepth = 16;

// C[m][n] = scale sum_k A(m, k) B(n, k) (+ C when `add`), operands by strides.
// A zero in A hides whatever B holds (rows that take no part).
template <typename TA, typename TB, typename TC>
__global__ void __launch_bounds__(256)
    k_head_mm(const TA* __restrict__ A, int64_t am, int64_t ak, const TB* __restrict__ B,
              int64_t bn, int64_t bk, int64_t M, int64_t N, int64_t K, float scale, TC* C,
              int64_t ldc, int add) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile; n0 < N;
         n0 += static_cast<int64_t>(gridDim.y) * kTile) {
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < K; k0 += kDepth) {
            for (int i = threadIdx.x; i < kTile * kDepth; i += 256) {
                // The faster index runs along whichever stride is 1.
                const int ma = ak == 1 ? i / kDepth : i % kTile;
                const int ka = ak == 1 ? i % kDepth : i / kTile;
                sa[ka][ma] = m0 + ma < M && k0 + ka < K
                                 ? to_f(A[(m0 + ma) * am + (k0 + ka) * ak]) : 0.0f;
                const int nb = bk == 1 ? i / kDepth : i % kTile;
                const int kb = bk == 1 ? i % kDepth : i / kTile;
                sb[kb][nb] = n0 + nb < N && k0 + kb < K
                                 ? to_f(B[(n0 + nb) * bn + (k0 + kb) * bk]) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kDepth; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float a = sa[k][ty * 4 + i];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (a != 0.0f) acc[i][j] = fmaf(a, sb[k][tx * 4 + j], acc[i][j]);
                }
            }
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
                if (m >= M || n >= N) continue;
                TC* c = C + m * ldc + n;
                put(c, scale * acc[i][j] + (add ? to_f(*c) : 0.0f));
            }
    }
}

template <typename TA, typename TB, typename TC>
cudaError_t mm(const TA* A, int64_t am, int64_t ak, const TB* B, int64_t bn, int64_t bk, int64_t M,
               int64_t N, int64_t K, float scale, TC* C, int64_t ldc, bool add, cudaStream_t s) {
    const int64_t gx = (M + kTile - 1) / kTile, gy = (N + kTile - 1) / kTile;
    return launch_pdl(k_head_mm<TA, TB, TC>,
                      dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy < 65535 ? gy : 65535)),
                      dim3(256), 0, s, A, am, ak, B, bn, bk, M, N, K, scale, C, ldc, add ? 1 : 0);
}

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* sh) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, off);
        v = is_max ? fmaxf(v, o) : v + o;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh[0];
    for (int i = 1; i < static_cast<int>(blockDim.x >> 5); ++i)
        v = is_max ? fmaxf(v, sh[i]) : v + sh[i];
    return v;
}

// One row of a piece: the running maximum and sum, and the picked logits.
__global__ void __launch_bounds__(256)
    k_head_rows(const float* __restrict__ x, int64_t v0, int64_t n, int64_t T, HeadTargets tg,
                int64_t V, int first, float* __restrict__ run_max, float* __restrict__ run_sum,
                float* __restrict__ picked, unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[8];
    const int64_t r = blockIdx.x, t = r % T;
    const float* xr = x + r * n;
    float m = -INFINITY;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) m = fmaxf(m, xr[i]);
    m = block_reduce(m, true, sh);
    const float old_m = first ? -INFINITY : run_max[r];
    const float nm = fmaxf(m, old_m);
    const float base = nm == -INFINITY ? 0.0f : nm;
    float q = 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) q += expf(xr[i] - base);
    q = block_reduce(q, false, sh);
    if (threadIdx.x == 0) {
        run_max[r] = nm;
        run_sum[r] = (first ? 0.0f : run_sum[r] * expf(old_m - base)) + q;
    }
    for (int64_t j = threadIdx.x; j < tg.K; j += blockDim.x) {
        const int64_t id = tg.ids[t * tg.K + j];
        if (id >= V) {
            if (first) atomicExch(status, 1u /* DUST_ERR_INVALID_ARG */);
        }
        if (first && (id < 0 || id >= V)) picked[r * tg.K + j] = 0.0f;
        if (id >= v0 && id < v0 + n) picked[r * tg.K + j] = xr[id - v0];
    }
}

// The teacher's largest scaled logit and the sum of exponentials over the
// entries present; `any` tells whether there is one. Whole block.
__device__ __forceinline__ void teacher_stats(const HeadTargets& tg, int64_t t, int64_t V,
                                              float scale, float* sh, float& m, float& sum,
                                              bool& any) {
    float a = -INFINITY, have = 0.0f;
    for (int64_t j = threadIdx.x; j < tg.K; j += blockDim.x) {
        const int64_t id = tg.ids[t * tg.K + j];
        if (id < 0 || id >= V) continue;
        have = 1.0f;
        a = fmaxf(a, scale * tg.teacher[t * tg.K + j]);
    }
    any = block_reduce(have, true, sh) > 0.0f;
    m = block_reduce(a, true, sh);
    if (m == -INFINITY) {  // no entry has any probability
        any = false;
        m = 0.0f;
    }
    float q = 0.0f;
    for (int64_t j = threadIdx.x; j < tg.K; j += blockDim.x) {
        const int64_t id = tg.ids[t * tg.K + j];
        if (id >= 0 && id < V) q += expf(scale * tg.teacher[t * tg.K + j] - m);
    }
    sum = block_reduce(q, false, sh);
}

__global__ void __launch_bounds__(128)
    k_head_finish(int64_t T, HeadTargets tg, int64_t V, float scale,
                  const float* __restrict__ run_max, const float* __restrict__ run_sum,
                  const float* __restrict__ picked, float* loss, float* lse) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[8];
    const int64_t r = blockIdx.x, t = r % T;
    const float l = run_max[r] + logf(run_sum[r]);
    float out = 0.0f;
    if (!tg.teacher) {
        const int64_t id = tg.ids[t];
        if (id >= 0 && id < V) out = l - picked[r];
    } else {
        float m, sum;
        bool any;
        teacher_stats(tg, t, V, scale, sh, m, sum, any);
        float a = 0.0f;
        for (int64_t j = threadIdx.x; any && j < tg.K; j += blockDim.x) {
            const int64_t id = tg.ids[t * tg.K + j];
            if (id < 0 || id >= V) continue;
            const float lq = scale * tg.teacher[t * tg.K + j] - m - logf(sum);
            const float q = expf(lq);
            if (q > 0.0f) a += q * (lq - (picked[r * tg.K + j] - l));
        }
        out = block_reduce(a, false, sh);
    }
    if (threadIdx.x == 0) {
        lse[r] = l;
        if (loss) loss[r] = out;
    }
}

__global__ void __launch_bounds__(256)
    k_head_changes(const float* __restrict__ loss, int64_t T, int64_t n, float* delta) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) delta[i] = loss[T + i] - loss[i % T];
}

// A piece of logits into G, in place (block per row).
__global__ void __launch_bounds__(256)
    k_head_factor(float* x, int64_t v0, int64_t n, int64_t T, HeadTargets tg, int64_t V,
                  float scale, const float* __restrict__ lse, const float* __restrict__ gloss,
                  unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[8];
    const int64_t r = blockIdx.x, t = r % T;
    float* xr = x + r * n;
    const float g = gloss[r];
    bool any;
    float m = 0.0f, sum = 1.0f;
    if (tg.teacher) {
        teacher_stats(tg, t, V, scale, sh, m, sum, any);
    } else {
        const int64_t id = tg.ids[t];
        any = id >= 0 && id < V;
    }
    if (v0 == 0)
        for (int64_t j = threadIdx.x; j < tg.K; j += blockDim.x)
            if (tg.ids[t * tg.K + j] >= V) atomicExch(status, 1u /* DUST_ERR_INVALID_ARG */);
    const bool live = any && g != 0.0f;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
        xr[i] = live ? g * expf(xr[i] - lse[r]) : 0.0f;
    __syncthreads();
    if (!live || threadIdx.x != 0) return;
    for (int64_t j = 0; j < tg.K; ++j) {
        const int64_t id = tg.ids[t * tg.K + j];
        if (id < v0 || id >= v0 + n) continue;
        const float q = tg.teacher ? expf(scale * tg.teacher[t * tg.K + j] - m - logf(sum)) : 1.0f;
        xr[id - v0] -= g * q;
    }
}

template <typename TX>
__global__ void __launch_bounds__(256)
    k_head_cast(const float* __restrict__ src, int64_t R, int64_t d, TX* dst, int64_t ld) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < R * d) put(dst + (i / d) * ld + i % d, src[i]);
}

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct Space {
    float *x, *run_max, *run_sum, *picked, *loss, *gh;
    size_t total;
};

Space carve(void* ws, int64_t R, int64_t d, int64_t V, int64_t K, bool grad) {
    Space w = {};
    unsigned char* p = static_cast<unsigned char*>(ws);
    size_t at = 0;
    auto take = [&](int64_t n) {
        float* q = ws ? reinterpret_cast<float*>(p + at) : nullptr;
        at += a256(sizeof(float) * static_cast<size_t>(n));
        return q;
    };
    w.x = take(R * (V < kPiece ? V : kPiece));
    if (grad) {
        w.gh = take(R * d);
    } else {
        w.run_max = take(R);
        w.run_sum = take(R);
        w.picked = take(K);  // cross entropy: R logits
        w.loss = take(R);
    }
    w.total = at;
    return w;
}

template <typename TX>
cudaError_t loss_typed(const HeadProblem& p, float* loss, float* lse, float* student, float* delta,
                       void* ws, cudaStream_t s) {
    const int64_t R = p.S * p.T;
    const bool distill = p.tg.teacher != nullptr;
    Space w = carve(ws, R, p.d, p.V, distill ? 0 : R, false);
    float* picked = distill ? student : w.picked;
    if (!loss && delta) loss = w.loss;
    unsigned int* st = status_word();
    if (!st) return cudaErrorUnknown;
    cudaError_t e;
    for (int64_t v0 = 0; v0 < p.V; v0 += kPiece) {
        const int64_t n = p.V - v0 < kPiece ? p.V - v0 : kPiece;
        e = mm(static_cast<const TX*>(p.H), p.ld_h, int64_t(1),
               static_cast<const TX*>(p.E) + v0 * p.ld_e, p.ld_e, int64_t(1), R, n, p.d, p.scale,
               w.x, n, false, s);
        if (e != cudaSuccess) return e;
        e = launch_pdl(k_head_rows, dim3(static_cast<unsigned>(R)), dim3(256), 0, s, w.x, v0, n,
                       p.T, p.tg, p.V, v0 == 0 ? 1 : 0, w.run_max, w.run_sum, picked, st);
        if (e != cudaSuccess) return e;
    }
    e = launch_pdl(k_head_finish, dim3(static_cast<unsigned>(R)), dim3(128), 0, s, p.T, p.tg, p.V,
                   p.scale, w.run_max, w.run_sum, picked, loss, lse);
    if (e != cudaSuccess || !delta || p.S < 2) return e;
    const int64_t n = R - p.T;
    return launch_pdl(k_head_changes, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0,
                      s, loss, p.T, n, delta);
}

template <typename TX>
cudaError_t grad_typed(const HeadProblem& p, const float* lse, const float* gloss, bool accumulate,
                       void* gH, int64_t ld_gh, void* gE, bool gE_bf16, void* ws,
                       cudaStream_t s) {
    const int64_t R = p.S * p.T;
    Space w = carve(ws, R, p.d, p.V, 0, true);
    const TX* H = static_cast<const TX*>(p.H);
    unsigned int* st = status_word();
    if (!st) return cudaErrorUnknown;
    cudaError_t e = cudaSuccess;
    for (int64_t v0 = 0; v0 < p.V; v0 += kPiece) {
        const int64_t n = p.V - v0 < kPiece ? p.V - v0 : kPiece;
        const TX* E = static_cast<const TX*>(p.E) + v0 * p.ld_e;
        e = mm(H, p.ld_h, int64_t(1), E, p.ld_e, int64_t(1), R, n, p.d, p.scale, w.x, n, false, s);
        if (e != cudaSuccess) return e;
        e = launch_pdl(k_head_factor, dim3(static_cast<unsigned>(R)), dim3(256), 0, s, w.x, v0, n,
                       p.T, p.tg, p.V, p.scale, lse, gloss, st);
        if (e != cudaSuccess) return e;
        if (gH) {
            e = mm(w.x, n, int64_t(1), E, int64_t(1), p.ld_e, R, p.d, n, p.scale, w.gh, p.d,
                   v0 > 0, s);
            if (e != cudaSuccess) return e;
        }
        if (!gE) continue;
        if (gE_bf16)
            e = mm(w.x, int64_t(1), n, H, int64_t(1), p.ld_h, n, p.d, R, p.scale,
                   static_cast<__nv_bfloat16*>(gE) + v0 * p.d, p.d, false, s);
        else
            e = mm(w.x, int64_t(1), n, H, int64_t(1), p.ld_h, n, p.d, R, p.scale,
                   static_cast<float*>(gE) + v0 * p.d, p.d, accumulate, s);
        if (e != cudaSuccess) return e;
    }
    if (!gH) return e;
    return launch_pdl(k_head_cast<TX>, dim3(static_cast<unsigned>((R * p.d + 255) / 256)),
                      dim3(256), 0, s, w.gh, R, p.d, static_cast<TX*>(gH), ld_gh);
}

}  // namespace

size_t head_loss_workspace_bytes(int64_t R, int64_t d, int64_t V, bool distill, bool bf16) {
    (void)bf16;
    return carve(nullptr, R, d, V, distill ? 0 : R, false).total;
}

size_t head_grad_workspace_bytes(int64_t R, int64_t d, int64_t V, bool bf16) {
    (void)bf16;
    return carve(nullptr, R, d, V, 0, true).total;
}

cudaError_t launch_head_loss(const HeadProblem& p, float* loss, float* lse, float* student,
                             float* delta, void* ws, cudaStream_t s) {
    ProfScope ps(kStageHead, s);
    return p.bf16 ? loss_typed<__nv_bfloat16>(p, loss, lse, student, delta, ws, s)
                  : loss_typed<float>(p, loss, lse, student, delta, ws, s);
}

cudaError_t launch_head_grad(const HeadProblem& p, const float* lse, const float* student,
                             const float* gloss, bool accumulate, void* gH, int64_t ld_gh,
                             void* gE, bool gE_bf16, void* ws, cudaStream_t s) {
    (void)student;
    ProfScope ps(kStageHead, s);
    return p.bf16 ? grad_typed<__nv_bfloat16>(p, lse, gloss, accumulate, gH, ld_gh, gE, gE_bf16,
                                              ws, s)
                  : grad_typed<float>(p, lse, gloss, accumulate, gH, ld_gh, gE, gE_bf16, ws, s);
}

}  // namespace dust
