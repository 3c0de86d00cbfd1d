// The gated feed-forward block's first half, h = act(X Wg^T) (X Wu^T), and its
// gradients (include/dust.h gives the formulas): tiles of 64 x 64 on the CUDA
// cores, fp32 sums.
#include <algorithm>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256, kTile = 64, kDeep = 16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// act(g) and its slope.
__device__ __forceinline__ float2 act_of(int act, float g) {
    if (act == DUST_ACT_RELU2) {
        const float r = g > 0.0f ? g : g == g ? 0.0f : g;
        return make_float2(r * r, 2.0f * r);
    }
    constexpr float kB = 0.044715f, kC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float z = act == DUST_ACT_SILU ? g : kC * fmaf(kB * g * g, g, g);
    const float p = 1.0f / (1.0f + expf(-z));
    const float q = 1.0f / (1.0f + expf(z));  // 1 - p
    // Where p q is 0 the slope of z may be infinite.
    const float slope = act == DUST_ACT_SILU ? 1.0f : kC * fmaf(3.0f * kB * g, g, 1.0f);
    const float pq = p * q;
    return make_float2(g * p, pq == 0.0f ? p : fmaf(g * pq, slope, p));
}

// acc[a][b] += sum over k < depth of A(row0 + 4 ty + a, k) B(col0 + 4 tx + b, k).
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(FA A, FB B, int64_t depth, float (&acc)[4][4]) {
    __shared__ float sa[kDeep][kTile + 4], sb[kDeep][kTile + 4];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    for (int64_t k0 = 0; k0 < depth; k0 += kDeep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kDeep; i += kThreads) {
            const int k = i % kDeep, r = i / kDeep;
            sa[k][r] = k0 + k < depth ? A(r, k0 + k) : 0.0f;
            sb[k][r] = k0 + k < depth ? B(r, k0 + k) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < 4; ++b) acc[a][b] = fmaf(sa[k][4 * ty + a], sb[k][4 * tx + b], acc[a][b]);
    }
}

struct Args {
    GatedProblem p;
    const void* gh;
    int64_t ld_gh;
    void* h;
    int64_t ld_h;
    void* D;              // [T][2 f]
    void *gX, *gWg, *gWu;
    int64_t ld_gx;
    bool accumulate;
    int64_t cols;         // tiles of columns
};

template <typename TX, bool BACK>
__global__ void __launch_bounds__(kThreads) k_gated_up(const Args a) {
    pdl_wait();
    pdl_trigger();
    const GatedProblem& p = a.p;
    const int64_t r0 = blockIdx.x / a.cols * kTile, c0 = blockIdx.x % a.cols * kTile;
    const auto at = [&](const void* m, int64_t ld, int64_t rows, int64_t first) {
        return [=](int r, int64_t k) {
            return first + r < rows ? to_f(static_cast<const TX*>(m)[(first + r) * ld + k]) : 0.0f;
        };
    };
    float g[4][4] = {}, u[4][4] = {};
    tile_product(at(p.X, p.ld_x, p.T, r0), at(p.Wg, p.ld_wg, p.f, c0), p.d, g);
    tile_product(at(p.X, p.ld_x, p.T, r0), at(p.Wu, p.ld_wu, p.f, c0), p.d, u);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + threadIdx.x / 16 * 4 + i, c = c0 + threadIdx.x % 16 * 4 + j;
            if (r >= p.T || c >= p.f) continue;
            const float2 act = act_of(p.act, g[i][j]);
            if constexpr (BACK) {
                const float gh = to_f(static_cast<const TX*>(a.gh)[r * a.ld_gh + c]);
                TX* D = static_cast<TX*>(a.D) + r * 2 * p.f + c;
                from_f(gh * u[i][j] * act.y, D[0]);
                from_f(gh * act.x, D[p.f]);
            } else {
                from_f(act.x * u[i][j], static_cast<TX*>(a.h)[r * a.ld_h + c]);
            }
        }
}

template <typename TX>
__global__ void __launch_bounds__(kThreads) k_gated_gx(const Args a) {
    pdl_wait();
    pdl_trigger();
    const GatedProblem& p = a.p;
    const int64_t r0 = blockIdx.x / a.cols * kTile, c0 = blockIdx.x % a.cols * kTile;
    float acc[4][4] = {};
    tile_product([&](int r, int64_t k) {
        return r0 + r < p.T ? to_f(static_cast<const TX*>(a.D)[(r0 + r) * 2 * p.f + k]) : 0.0f;
    }, [&](int c, int64_t k) {
        if (c0 + c >= p.d) return 0.0f;
        return k < p.f ? to_f(static_cast<const TX*>(p.Wg)[k * p.ld_wg + c0 + c])
                       : to_f(static_cast<const TX*>(p.Wu)[(k - p.f) * p.ld_wu + c0 + c]);
    }, 2 * p.f, acc);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + threadIdx.x / 16 * 4 + i, c = c0 + threadIdx.x % 16 * 4 + j;
            if (r < p.T && c < p.d) from_f(acc[i][j], static_cast<TX*>(a.gX)[r * a.ld_gx + c]);
        }
}

template <typename TX, typename TW>
__global__ void __launch_bounds__(kThreads) k_gated_gw(const Args a) {
    pdl_wait();
    pdl_trigger();
    const GatedProblem& p = a.p;
    const int64_t r0 = blockIdx.x / a.cols * kTile, c0 = blockIdx.x % a.cols * kTile;
    float acc[4][4] = {};
    tile_product([&](int r, int64_t k) {
        return r0 + r < 2 * p.f ? to_f(static_cast<const TX*>(a.D)[k * 2 * p.f + r0 + r]) : 0.0f;
    }, [&](int c, int64_t k) {
        return c0 + c < p.d ? to_f(static_cast<const TX*>(p.X)[k * p.ld_x + c0 + c]) : 0.0f;
    }, p.T, acc);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t r = r0 + threadIdx.x / 16 * 4 + i, c = c0 + threadIdx.x % 16 * 4 + j;
            if (r >= 2 * p.f || c >= p.d) continue;
            TW* out = static_cast<TW*>(r < p.f ? a.gWg : a.gWu);
            if (!out) continue;
            out += (r < p.f ? r : r - p.f) * p.d + c;
            from_f(a.accumulate ? to_f(*out) + acc[i][j] : acc[i][j], *out);
        }
}

int64_t tiles(int64_t n) { return (n + kTile - 1) / kTile; }

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

template <typename TX>
cudaError_t grad_typed(Args a, bool gW_bf16, cudaStream_t s) {
    const GatedProblem& p = a.p;
    a.cols = tiles(p.f);
    DUST_TRY(launch_pdl(k_gated_up<TX, true>, dim3(static_cast<unsigned>(tiles(p.T) * a.cols)),
                        dim3(kThreads), 0, s, a));
    a.cols = tiles(p.d);
    if (a.gX)
        DUST_TRY(launch_pdl(k_gated_gx<TX>, dim3(static_cast<unsigned>(tiles(p.T) * a.cols)),
                            dim3(kThreads), 0, s, a));
    if (!a.gWg && !a.gWu) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(tiles(2 * p.f) * a.cols));
    return gW_bf16 ? launch_pdl(k_gated_gw<TX, __nv_bfloat16>, grid, dim3(kThreads), 0, s, a)
                   : launch_pdl(k_gated_gw<TX, float>, grid, dim3(kThreads), 0, s, a);
}

}  // namespace

size_t gated_workspace_bytes(const GatedProblem&) { return 0; }
size_t gated_grad_workspace_bytes(const GatedProblem& p) {
    return static_cast<size_t>(p.T * p.f) * 2 * (p.bf16 ? 2 : 4);
}

cudaError_t launch_gated(const GatedProblem& p, void* h, int64_t ld_h, void*, cudaStream_t s) {
    ProfScope ps(kStageGated, s);
    Args a = {};
    a.p = p;
    a.h = h;
    a.ld_h = ld_h;
    a.cols = tiles(p.f);
    const dim3 grid(static_cast<unsigned>(tiles(p.T) * a.cols));
    return p.bf16 ? launch_pdl(k_gated_up<__nv_bfloat16, false>, grid, dim3(kThreads), 0, s, a)
                  : launch_pdl(k_gated_up<float, false>, grid, dim3(kThreads), 0, s, a);
}

cudaError_t launch_gated_grad(const GatedProblem& p, const void* gh, int64_t ld_gh, bool accumulate,
                              void* gX, int64_t ld_gx, void* gWg, void* gWu, bool gW_bf16, void* ws,
                              cudaStream_t s) {
    ProfScope ps(kStageGated, s);
    Args a = {};
    a.p = p;
    a.gh = gh;
    a.ld_gh = ld_gh;
    a.D = ws;
    a.gX = gX;
    a.gWg = gWg;
    a.gWu = gWu;
    a.ld_gx = ld_gx;
    a.accumulate = accumulate;
    return p.bf16 ? grad_typed<__nv_bfloat16>(a, gW_bf16, s) : grad_typed<float>(a, false, s);
}

}  // namespace dust
