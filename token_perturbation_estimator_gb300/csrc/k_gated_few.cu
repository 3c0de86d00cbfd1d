// The gated block of a few rows (up to kGatedFew) on the CUDA cores: the
// weights are read once as they lie and everything is summed in fp32. On the
// tensor cores a 256-row tile would be mostly empty, the weights of a few units
// would be all that a pair of CTAs has on its way, and fp32 weights would be
// copied into planes first.
//
// A warp takes two units, four rows of weights, over the whole width or a part
// of it: `split` warps of a CTA share a pair of units, so that there are
// CTAs for the whole GPU. X comes from the L1 after its first use.
//
// 1 row, d 512, f 2048 bf16 is a round trip to memory: 5.0 us alone (10 as tiles),
// 2.2 in a row of captured calls, 2.7 with weights that are not in the L2. 1 row, d
// 2048, f 8192, 67 MB of weights: 13.2 us from memory, 5.1 TB/s, 7.1 from the L2; 4
// rows 18.0 and 14.0, where their products and X's loads, four times as many, show
// beside the weights (16 rows as tiles 20.2 and 18.8). HBM's rate makes 9.9 of
// either: a warp has few loads on their way while it waits for those it has begun.
#include <algorithm>

#include "gated.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

struct Args {
    const void *X, *Wg, *Wu;
    int64_t ld_x, ld_g, ld_u;
    int T;
    int64_t d, f;
    int act, split;
    void* h;
    int64_t ld_h;
};

__device__ __forceinline__ float activation(int act, float g) {
    if (act == DUST_ACT_RELU2) {
        const float r = g > 0.0f ? g : g == g ? 0.0f : g;
        return r * r;
    }
    const float z = act == DUST_ACT_SILU ? g : 1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f);
    return g / (1.0f + expf(-z));
}

// PER values from p: 16 bytes at once, or one.
template <typename TX, int PER>
__device__ __forceinline__ void load(const TX* p, float (&v)[PER]) {
    if constexpr (PER == 1) {
        v[0] = to_f(*p);
    } else {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (PER == 8) {
                v[2 * i] = __uint_as_float(r[i] << 16);
                v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(r[i]);
            }
        }
    }
}

// ROWS: the rows rounded up to 1, 2 or 4; the last one stands in for those
// that there are not.
template <typename TX, int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads) k_gated_few(const Args a) {
    pdl_wait();
    pdl_trigger();
    constexpr int kPer = VEC ? 16 / static_cast<int>(sizeof(TX)) : 1;
    __shared__ float part[kWarps][ROWS * 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int pairs = kWarps / a.split, mine = warp / a.split, slice = warp % a.split;
    const int64_t unit = 2 * (static_cast<int64_t>(blockIdx.x) * pairs + mine);
    float acc[ROWS][4] = {};  // of each row: the units' gates, their ups
    if (unit < a.f) {
        const int64_t other = min(unit + 1, a.f - 1);
        const TX* w[4] = {static_cast<const TX*>(a.Wg) + unit * a.ld_g, static_cast<const TX*>(a.Wg) + other * a.ld_g,
                          static_cast<const TX*>(a.Wu) + unit * a.ld_u, static_cast<const TX*>(a.Wu) + other * a.ld_u};
        const TX* x[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) x[r] = static_cast<const TX*>(a.X) + min(r, a.T - 1) * a.ld_x;
        // Steps of 32 lanes' values, dealt to the slices in turn.
        const int64_t step = 32 * kPer * a.split;
#pragma unroll 2
        for (int64_t c = (static_cast<int64_t>(slice) * 32 + lane) * kPer; c < a.d; c += step) {
            float wv[4][kPer];
#pragma unroll
            for (int i = 0; i < 4; ++i) load<TX, kPer>(w[i] + c, wv[i]);
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float xv[kPer];
                load<TX, kPer>(x[r] + c, xv);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < kPer; ++k) acc[r][i] = fmaf(wv[i][k], xv[k], acc[r][i]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v = acc[r][i];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            if (lane == 0) part[warp][4 * r + i] = v;
        }
    __syncthreads();
    // A thread per row and unit.
    const int n = threadIdx.x;
    if (n >= pairs * ROWS * 2) return;
    const int p = n / (ROWS * 2), r = n / 2 % ROWS, u = n & 1;
    const int64_t to = 2 * (static_cast<int64_t>(blockIdx.x) * pairs + p) + u;
    if (r >= a.T || to >= a.f) return;
    float g = 0.0f, up = 0.0f;
    for (int s = 0; s < a.split; ++s) {
        g += part[p * a.split + s][4 * r + u];
        up += part[p * a.split + s][4 * r + 2 + u];
    }
    from_f(activation(a.act, g) * up, static_cast<TX*>(a.h)[r * a.ld_h + to]);
}

template <typename TX, int ROWS>
cudaError_t launch_rows(const Args& a, bool vec, unsigned grid, cudaStream_t s) {
    return vec ? launch_pdl(k_gated_few<TX, ROWS, true>, dim3(grid), dim3(kThreads), 0, s, a)
               : launch_pdl(k_gated_few<TX, ROWS, false>, dim3(grid), dim3(kThreads), 0, s, a);
}

template <typename TX>
cudaError_t launch_typed(const Args& a, bool vec, unsigned grid, cudaStream_t s) {
    return a.T == 1   ? launch_rows<TX, 1>(a, vec, grid, s)
           : a.T == 2 ? launch_rows<TX, 2>(a, vec, grid, s)
                      : launch_rows<TX, 4>(a, vec, grid, s);
}

}  // namespace

cudaError_t launch_gated_few(const GatedProblem& p, void* h, int64_t ld_h, cudaStream_t s) {
    const int64_t size = p.bf16 ? 2 : 4, per = 16 / size;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.X) | reinterpret_cast<uintptr_t>(p.Wg) |
                         reinterpret_cast<uintptr_t>(p.Wu) |
                         static_cast<uintptr_t>((p.ld_wg | p.ld_wu | (p.T > 1 ? p.ld_x : 0)) * size);
    const bool vec = at % 16 == 0 && p.d % per == 0;
    Args a = {p.X, p.Wg, p.Wu, p.ld_x, p.ld_wg, p.ld_wu, static_cast<int>(p.T), p.d, p.f, p.act, 1, h, ld_h};
    // Two CTAs per SM, if the width gives every warp something to read.
    const int64_t pairs = (p.f + 1) / 2, step = 32 * (vec ? per : 1);
    while (a.split < kWarps && pairs * a.split < 304 * kWarps && a.split * step < p.d) a.split *= 2;
    const int64_t units = kWarps / a.split;
    const unsigned grid = static_cast<unsigned>((pairs + units - 1) / units);
    return p.bf16 ? launch_typed<__nv_bfloat16>(a, vec, grid, s) : launch_typed<float>(a, vec, grid, s);
}

}  // namespace dust
