// The head's loss and gradients for a few rows (single tokens being scored).
// Loss: every row of E is read once, as it lies, and multiplied with all rows
// of H on the CUDA cores, fp32 throughout. Bound by E's bytes; the tensor-core kernel spends a
// 256-row tile on these rows, and first copies an fp32 E into three planes.
//
// A warp takes 16 / NR rows of E at a time (NR: the rows of H, rounded up to
// a power of two), so that it keeps 16 sums, as many 16-byte loads per lane in
// flight as it has rows of E, and uses what it reads of H that often; H lies
// in shared memory. The 16 sums are added up over the lanes by halving: each
// step a lane hands over half of its sums, and ends with one. That lane keeps
// the running maximum and sum of its row of H; they are joined per CTA, and
// over the CTAs by the same kernel that joins the tiles' partial sums.
//
// Distillation: the teacher's entries are further dots, a warp each.
//
// One row, d 2048, V 50257: the loss takes 43 us in bf16 and 75 us in fp32
// (4.8 and 5.5 TB/s of E), the gradients 105 and 187 us (E and gE: 3.9 and
// 4.4 TB/s).
#include <algorithm>
#include <cmath>

#include "head.cuh"

namespace dust {

namespace {

constexpr int kWarps = 8;
constexpr int kSums = 16;
constexpr int kMaxRows = 8;
// Floats of H in shared memory: two CTAs per SM for the loss, one for a
// gradient, which keeps as many sums.
constexpr int64_t kMaxH = 24 * 1024;
constexpr int kMaxGradSmem = 208 * 1024;
constexpr int kMaxCtas = 152 * 2;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Values that a lane loads at once: 16 bytes of a row, or one.
template <typename TX, bool VEC> constexpr int per_load() {
    return VEC ? 16 / static_cast<int>(sizeof(TX)) : 1;
}

template <typename TX, bool VEC>
struct Loaded {
    static constexpr int P = per_load<TX, VEC>();
    union {
        uint4 q;
        TX x[P];
    };
    __device__ Loaded() {}
    __device__ __forceinline__ void load(const TX* p, bool in) {
        if constexpr (VEC)
            q = in ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
        else
            x[0] = in ? *p : TX(0.0f);
    }
    __device__ __forceinline__ float at(int k) const { return to_f(x[k]); }
};

struct FewArgs {
    int64_t ld_h, ld_e, T, V, K;
    int R, d;
    float scale;
    const int32_t* targets;  // or null
    const int32_t* ids;      // distillation, else null
    float* student;
    HeadPart* part;
    int64_t ld_part;
    float* picked;
    unsigned int* status;
};

// Where value k of lane l in column block b (32 P columns) lies in shared
// memory: lanes read neighbouring 16 bytes.
template <int P>
__device__ __forceinline__ int place(int b, int l, int k) {
    return P >= 4 ? ((b * (P / 4) + k / 4) * 32 + l) * 4 + k % 4 : b * 32 + l;
}

// H's rows [0, R) into shared memory, zero past them and past column d, and
// where a row is not wanted.
template <typename TX, int P, int NR, typename F>
__device__ __forceinline__ void stage_rows(float* h, const TX* H, int64_t ld, int R, int d, int pitch,
                                           F wanted) {
    for (int i = threadIdx.x; i < NR * pitch; i += blockDim.x) {
        const int r = i / pitch, c = i - r * pitch;
        const int b = c / (32 * P), l = c / P % 32, k = c % P;
        h[r * pitch + place<P>(b, l, k)] =
            r < R && c < d && wanted(r) ? to_f(H[r * ld + c]) : 0.0f;
    }
}

// P values of a row of H, for column block b.
template <int P>
__device__ __forceinline__ void staged(const float* h, int b, int lane, float (&v)[P]) {
    if constexpr (P >= 4) {
#pragma unroll
        for (int k = 0; k < P; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(h + place<P>(b, lane, k));
            v[k] = f.x;
            v[k + 1] = f.y;
            v[k + 2] = f.z;
            v[k + 3] = f.w;
        }
    } else {
        v[0] = h[place<P>(b, lane, 0)];
    }
}

// Products of U rows of E (those below `left`) with NR staged rows. Of every
// 32 / (U NR) lanes, all end with the i-th: row i / NR of E, row i % NR of H.
template <typename TX, bool VEC, int NR, int U>
__device__ __forceinline__ float few_dots(const TX* E, int64_t ld, int64_t left, const float* h,
                                          int d, int pitch, int lane) {
    constexpr int P = per_load<TX, VEC>(), N = U * NR;
    const int blocks = pitch / (32 * P);
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    const TX* e = E + lane * P;
    for (int b = 0; b < blocks; ++b) {
        const bool in = (b * 32 + lane) * P < d;
        Loaded<TX, VEC> x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) x[i].load(e + i * ld + b * 32 * P, in && i < left);
#pragma unroll
        for (int q = 0; q < NR; ++q) {
            float hv[P];
            staged<P>(h + q * pitch, b, lane, hv);
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int k = 0; k < P; ++k)
                    acc[i * NR + q] = fmaf(x[i].at(k), hv[k], acc[i * NR + q]);
        }
    }
#pragma unroll
    for (int n = N / 2, off = 16; n > 0; n >>= 1, off >>= 1) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool up = (lane & off) != 0;
            const float keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
#pragma unroll
    for (int off = 16 / N; off > 0; off >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], off);
    return acc[0];
}

template <typename TX, bool VEC, int NR>
__global__ void __launch_bounds__(32 * kWarps, 2)
    k_head_few(const TX* __restrict__ H, const TX* __restrict__ E, const FewArgs a) {
    constexpr int P = per_load<TX, VEC>(), U = kSums / NR;
    extern __shared__ __align__(16) float h[];  // [NR][blocks 32 P]
    __shared__ HeadPart meet[kWarps][NR];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int blocks = (a.d + 32 * P - 1) / (32 * P), pitch = blocks * 32 * P;
    pdl_wait();
    pdl_trigger();
    stage_rows<TX, P, NR>(h, H, a.ld_h, a.R, a.d, pitch, [](int) { return true; });
    __syncthreads();

    // The sum a lane ends with: that of E row v0 + u with H row r.
    const int u = lane / 2 / NR, r = lane / 2 % NR;
    const bool mine = (lane & 1) == 0 && r < a.R;
    const int32_t target = mine && a.targets ? a.targets[r % a.T] : -1;
    const float c = a.scale * kLog2e;
    float m = -INFINITY, s = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * U;
    for (int64_t v0 = (static_cast<int64_t>(blockIdx.x) * kWarps + w) * U; v0 < a.V; v0 += step) {
        const float x = few_dots<TX, VEC, NR, U>(E + v0 * a.ld_e, a.ld_e, a.V - v0, h, a.d, pitch, lane);
        const int64_t v = v0 + u;
        if (!mine || v >= a.V) continue;
        if (v == target) a.picked[r] = a.scale * x;
        const float nm = fmaxf(m, ceilf(c * x));
        const float base = nm == -INFINITY ? 0.0f : nm;
        s = s * exp2f(m - base) + exp2f(fmaf(c, x, -base));
        m = nm;
    }
    if (!mine) {
        m = -INFINITY;
        s = 0.0f;
    }
    const auto join = [&](float pm, float ps) {
        const float nm = fmaxf(m, pm);
        const float base = nm == -INFINITY ? 0.0f : nm;
        s = s * exp2f(m - base) + ps * exp2f(pm - base);
        m = nm;
    };
#pragma unroll
    for (int off = 2 * NR; off < 32; off <<= 1) {  // over u
        const float pm = __shfl_xor_sync(0xffffffffu, m, off);
        const float ps = __shfl_xor_sync(0xffffffffu, s, off);
        join(pm, ps);
    }
    if (u == 0 && (lane & 1) == 0) meet[w][r] = {m, s};
    __syncthreads();
    if (threadIdx.x < a.R) {
        m = meet[0][threadIdx.x].m;
        s = meet[0][threadIdx.x].s;
        for (int i = 1; i < kWarps; ++i) join(meet[i][threadIdx.x].m, meet[i][threadIdx.x].s);
        a.part[static_cast<int64_t>(blockIdx.x) * a.ld_part + threadIdx.x] = {m, s};
    }
    if (!a.ids) return;
    const int64_t items = a.R * a.K;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + w; i < items;
         i += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int q = static_cast<int>(i / a.K);
        const int64_t t = q % a.T;
        const int64_t id = a.ids[t * a.K + (i - q * a.K)];
        if (id >= a.V && lane == 0) atomicExch(a.status, 1u /* DUST_ERR_INVALID_ARG */);
        float dot = 0.0f;
        if (id >= 0 && id < a.V) {
            const TX* e = E + id * a.ld_e + lane * P;
            for (int b = 0; b < blocks; ++b) {
                Loaded<TX, VEC> x;
                x.load(e + b * 32 * P, (b * 32 + lane) * P < a.d);
#pragma unroll
                for (int k = 0; k < P; ++k)
                    dot = fmaf(x.at(k), h[q * pitch + place<P>(b, lane, k)], dot);
            }
            dot = warp_sum(dot);
        }
        if (lane == 0) a.student[i] = a.scale * dot;
    }
}

// ------------------------------------------------------------- gradients

struct FewGrad {
    int64_t ld_h, ld_e, T, V;
    int R, d, groups;
    float scale;
    const int32_t* targets;  // or null
    HeadPicks picks;         // distillation: exp(x - lse) - q at the entries, in order
    const int32_t* alive;    // distillation
    const float *lse, *gloss;
    float* part;             // [CTAs][R][d], or null
    void* gE;                // or null
    int ge_bf16, accumulate;
    unsigned int* status;
};

// Writes P neighbouring values.
template <int P>
__device__ __forceinline__ void write_values(void* out, int64_t at, const float (&v)[P], bool bf16,
                                             bool add) {
    if (bf16) {
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(out) + at;
        alignas(16) __nv_bfloat16 b[P];
#pragma unroll
        for (int k = 0; k < P; ++k) b[k] = __float2bfloat16_rn(v[k]);
        if constexpr (P == 8) *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(b);
        else if constexpr (P == 4) *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(b);
        else o[0] = b[0];
    } else {
        float* o = static_cast<float*>(out) + at;
        if constexpr (P >= 4) {
#pragma unroll
            for (int k = 0; k < P; k += 4) {
                float4 x = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                if (add) {
                    const float4 y = *reinterpret_cast<const float4*>(o + k);
                    x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
                }
                *reinterpret_cast<float4*>(o + k) = x;
            }
        } else {
            o[0] = add ? o[0] + v[0] : v[0];
        }
    }
}

// Rows of E per warp and block, of NR rows of H: few, so that a block's rows
// are still near when they are read again (one fp32 row, d 2048, V 50257:
// 8 rows 206 us, 4 rows 187).
__host__ __device__ constexpr int grad_rows(int NR) { return NR <= 4 ? 4 : kSums / NR; }

// Both gradients of a few rows, fp32 throughout. A CTA takes kWarps grad_rows(NR)
// rows of E at a time: its warps form their logits as above and leave
// g = gloss (exp(x - lse) - wanted) in shared memory; then each thread takes
// 16 bytes of the columns, reads those rows again (out of the caches), adds
// g E to its part of gH, which lies in shared memory between the blocks, and
// writes gE = sum g H. Where the columns are fewer than the threads, groups of
// threads take every so manieth row. The CTAs' parts of gH are added up by
// k_head_few_sum, in order.
template <typename TX, bool VEC, int NR>
__global__ void __launch_bounds__(32 * kWarps, 2)
    k_head_few_grad(const TX* __restrict__ H, const TX* __restrict__ E, const FewGrad a) {
    constexpr int P = per_load<TX, VEC>(), U = grad_rows(NR), kRows = kWarps * U;
    constexpr int kLanes = 32 / (U * NR), kAhead = NR * P > 16 ? 4 : 8;
    extern __shared__ __align__(16) float h[];  // [NR][pitch], then groups of as many sums
    __shared__ float g[kRows][NR];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int blocks = (a.d + 32 * P - 1) / (32 * P), pitch = blocks * 32 * P;
    float* sums = h + NR * pitch;
    pdl_wait();
    pdl_trigger();
    const auto wanted = [&](int r) {
        if (a.gloss[r] == 0.0f) return false;
        if (!a.targets) return a.alive[r] != 0;
        const int32_t id = a.targets[r % a.T];
        return id >= 0 && id < a.V;
    };
    // Rows that take no part are not read.
    stage_rows<TX, P, NR>(h, H, a.ld_h, a.R, a.d, pitch, wanted);
    for (int i = threadIdx.x; i < a.groups * NR * pitch; i += blockDim.x) sums[i] = 0.0f;
    if (blockIdx.x == 0 && threadIdx.x < a.R && a.targets && a.targets[threadIdx.x % a.T] >= a.V)
        atomicExch(a.status, 1u /* DUST_ERR_INVALID_ARG */);

    const int u = lane / kLanes / NR, r = lane / kLanes % NR;
    const bool live = r < a.R && wanted(r), mine = lane % kLanes == 0;
    const float weight = live ? a.gloss[r] : 0.0f, l = live ? a.lse[r] : 0.0f;
    const int32_t target = live && a.targets ? a.targets[r % a.T] : -1;
    // This thread's columns and rows in the second part.
    const int wide = 8 / a.groups, group = w / wide, col = w % wide;  // in warps
    __syncthreads();
    int64_t block = blockIdx.x;
    for (int64_t v0 = block * kRows; v0 < a.V; v0 += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t from = v0 + w * U;
        const float x = few_dots<TX, VEC, NR, U>(E + from * a.ld_e, a.ld_e, a.V - from, h, a.d, pitch, lane);
        if (mine) {
            float f = 0.0f;  // rows of H that take no part, and rows past E's
            if (live && from + u < a.V) {
                f = expf(fmaf(a.scale, x, -l));
                if (from + u == target) f -= 1.0f;
                f *= weight;
            }
            g[w * U + u][r] = f;
        }
        __syncthreads();
        if (a.picks.entries) {
            const int64_t bin = v0 / kRows;
            for (int q = w; q < a.R; q += kWarps) {
                if (!wanted(q)) continue;
                const uint16_t* at = a.picks.starts + q * (a.picks.bins + 1) + bin;
                for (int j = at[0] + lane; j < at[1]; j += 32) {
                    const int2 e = a.picks.entries[q * a.picks.K + j];
                    g[e.x - v0][q] = a.gloss[q] * __int_as_float(e.y);
                }
            }
            __syncthreads();
        }
        const int rows = a.V - v0 < kRows ? static_cast<int>(a.V - v0) : kRows;
        for (int b = col; b < blocks; b += wide) {
            const int c = (b * 32 + lane) * P;
            if (c >= a.d) continue;
            float hv[NR][P], acc[NR][P];
#pragma unroll
            for (int q = 0; q < NR; ++q) {
                staged<P>(h + q * pitch, b, lane, hv[q]);
                staged<P>(sums + (group * NR + q) * pitch, b, lane, acc[q]);
            }
            for (int first = group; first < rows; first += kAhead * a.groups) {
                Loaded<TX, VEC> e[kAhead];  // together on their way
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int v = first + i * a.groups;
                    e[i].load(E + (v0 + v) * a.ld_e + c, v < rows);
                }
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int v = first + i * a.groups;
                    if (v >= rows) break;
                    float out[P];
#pragma unroll
                    for (int k = 0; k < P; ++k) out[k] = 0.0f;
#pragma unroll
                    for (int q = 0; q < NR; ++q) {
                        const float f = g[v][q];
#pragma unroll
                        for (int k = 0; k < P; ++k) {
                            acc[q][k] = fmaf(f, e[i].at(k), acc[q][k]);
                            out[k] = fmaf(f, hv[q][k], out[k]);
                        }
                    }
                    if (!a.gE) continue;
#pragma unroll
                    for (int k = 0; k < P; ++k) out[k] *= a.scale;
                    write_values<P>(a.gE, (v0 + v) * a.d + c, out, a.ge_bf16, a.accumulate);
                }
            }
#pragma unroll
            for (int q = 0; q < NR; ++q)
#pragma unroll
                for (int k = 0; k < P; ++k)
                    sums[(group * NR + q) * pitch + place<P>(b, lane, k)] = acc[q][k];
        }
        __syncthreads();
    }
    if (!a.part) return;
    for (int i = threadIdx.x; i < a.R * a.d; i += blockDim.x) {
        const int q = i / a.d, c = i - q * a.d;
        const int at = q * pitch + place<P>(c / (32 * P), c / P % 32, c % P);
        float v = 0.0f;
        for (int k = 0; k < a.groups; ++k) v += sums[k * NR * pitch + at];
        // What a row of E holds does not reach a row that takes no part.
        a.part[static_cast<int64_t>(blockIdx.x) * a.R * a.d + i] = wanted(q) ? v : 0.0f;
    }
}

// gH = scale times the sum of n parts of R d values: 32 columns by kWarps
// slices of the parts per CTA.
__global__ void __launch_bounds__(32 * kWarps)
    k_head_few_sum(const float* __restrict__ part, int n, int R, int d, float scale, void* gH,
                   int64_t ld, int bf16) {
    __shared__ float sh[kWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t all = static_cast<int64_t>(R) * d, i = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (i < all)
#pragma unroll 8
        for (int k = w; k < n; k += kWarps) v += part[k * all + i];
    sh[w][lane] = v;
    __syncthreads();
    if (w != 0 || i >= all) return;
    for (int k = 1; k < kWarps; ++k) v += sh[k][lane];
    const int64_t at = i / d * ld + i % d;
    if (bf16) static_cast<__nv_bfloat16*>(gH)[at] = __float2bfloat16_rn(scale * v);
    else static_cast<float*>(gH)[at] = scale * v;
}

int rows_up(int64_t R) { return R <= 1 ? 1 : R <= 2 ? 2 : R <= 4 ? 4 : 8; }

template <typename TX, bool VEC, int NR>
cudaError_t launch_few(const HeadProblem& p, const FewArgs& a, int ctas, cudaStream_t s) {
    constexpr int P = per_load<TX, VEC>();
    const int64_t pitch = (p.d + 32 * P - 1) / (32 * P) * (32 * P);
    const size_t smem = sizeof(float) * static_cast<size_t>(NR * pitch);
    static const auto kernel = k_head_few<TX, VEC, NR>;
    const cudaError_t e =
        ensure_smem_limit(reinterpret_cast<const void*>(kernel), 4 * kMaxH + 4 * kMaxRows * 256);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * kWarps), smem, s,
                      static_cast<const TX*>(p.H), static_cast<const TX*>(p.E), a);
}

template <typename TX, bool VEC>
cudaError_t by_rows(const HeadProblem& p, const FewArgs& a, int ctas, cudaStream_t s) {
    switch (rows_up(a.R)) {
        case 1: return launch_few<TX, VEC, 1>(p, a, ctas, s);
        case 2: return launch_few<TX, VEC, 2>(p, a, ctas, s);
        case 4: return launch_few<TX, VEC, 4>(p, a, ctas, s);
        default:
            if constexpr (sizeof(TX) == 4) return launch_few<TX, VEC, 8>(p, a, ctas, s);
            return cudaErrorInvalidValue;
    }
}

template <typename TX, bool VEC, int NR>
cudaError_t launch_few_grad(const HeadProblem& p, FewGrad a, int ctas, cudaStream_t s) {
    constexpr int P = per_load<TX, VEC>();
    const int blocks = static_cast<int>((p.d + 32 * P - 1) / (32 * P)), pitch = blocks * 32 * P;
    a.groups = blocks > 4 ? 1 : blocks > 2 ? 2 : blocks > 1 ? 4 : 8;
    const size_t smem = sizeof(float) * static_cast<size_t>((1 + a.groups) * NR * pitch);
    static const auto kernel = k_head_few_grad<TX, VEC, NR>;
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), kMaxGradSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(32 * kWarps), smem, s,
                      static_cast<const TX*>(p.H), static_cast<const TX*>(p.E), a);
}

template <typename TX, bool VEC>
cudaError_t grad_by_rows(const HeadProblem& p, const FewGrad& a, int ctas, cudaStream_t s) {
    switch (rows_up(a.R)) {
        case 1: return launch_few_grad<TX, VEC, 1>(p, a, ctas, s);
        case 2: return launch_few_grad<TX, VEC, 2>(p, a, ctas, s);
        case 4: return launch_few_grad<TX, VEC, 4>(p, a, ctas, s);
        default:
            if constexpr (sizeof(TX) == 4) return launch_few_grad<TX, VEC, 8>(p, a, ctas, s);
            return cudaErrorInvalidValue;
    }
}

}  // namespace

// Few enough that this is faster than the tensor cores' tiles, loss and
// gradients together. us here / there (with the launches that join), V 4096,
// d 512 and V 50257, d 2048:
//   loss       bf16  R 1  6 / 9,  43 / 62     R 2  6 / 9,  46 / 55
//                    R 4  7 / 9,  65 / 54     R 8  10 / 9, 96 / 54
//              fp32  R 1  7 / 29, 75 / 477    R 8  9 / 27, 142 / 458
//   gradients  bf16  R 1  9 / 24, 105 / 236   R 2  11 / 24, 120 / 236
//                    R 4  16 / 24, 158 / 236
//              fp32  R 1  9 / 45, 187 / 1160  R 8  25 / 45, 527 / 1156
// (bf16 rows of 1001 values, V 20000: loss of R 4 33 / 38, R 8 40 / 38; with d
// 4096, V 32000, where one CTA fits an SM, gradients of bf16 R 4 346 / 287).
// With E out of the L2, the loss of four bf16 rows takes 81 / 105 (d 2048, V
// 50257) and 32 / 38 (d 1024, V 20000), as the binding calls it.
// One rule for loss and gradients: the gradient takes exp(x - lse) with the x
// that lse was formed from, and the two ways' sums of x differ by what the
// tensor cores cut off (loss of a token 1e-4, target's logit 30: gH was 0.1 to
// 0.2 off by row; summed alike 0.02 and less).
bool head_few(const HeadProblem& p) {
    const int64_t R = p.S * p.T;
    if (R > kMaxRows || rows_up(R) * p.d > kMaxH) return false;
    return !p.bf16 || R <= 2 || (R <= 4 && p.d <= kMaxH / 8);
}

int head_few_parts(const HeadProblem& p) {
    const int64_t per = kWarps * kSums / rows_up(p.S * p.T);  // rows of E a CTA takes at a time
    return static_cast<int>(std::min<int64_t>((p.V + per - 1) / per, kMaxCtas));
}

cudaError_t launch_head_few(const HeadProblem& p, HeadPart* part, int64_t ld_part, float* picked,
                            float* student, cudaStream_t s) {
    FewArgs a = {};
    a.ld_h = p.ld_h;
    a.ld_e = p.ld_e;
    a.T = p.T;
    a.V = p.V;
    a.K = p.tg.K;
    a.R = static_cast<int>(p.S * p.T);
    a.d = static_cast<int>(p.d);
    a.scale = p.scale;
    a.targets = p.tg.many ? nullptr : p.tg.ids;
    a.ids = p.tg.many ? p.tg.ids : nullptr;
    a.student = student;
    a.part = part;
    a.ld_part = ld_part;
    a.picked = picked;
    a.status = status_word();
    if (!a.status) return cudaErrorUnknown;
    const int size = p.bf16 ? 2 : 4, ctas = head_few_parts(p);
    const bool vec = p.d * size % 16 == 0 && p.ld_e * size % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(p.E) % 16 == 0;
    if (p.bf16)
        return vec ? by_rows<__nv_bfloat16, true>(p, a, ctas, s)
                   : by_rows<__nv_bfloat16, false>(p, a, ctas, s);
    return vec ? by_rows<float, true>(p, a, ctas, s) : by_rows<float, false>(p, a, ctas, s);
}

int head_few_grad_rows(const HeadProblem& p) { return kWarps * grad_rows(rows_up(p.S * p.T)); }

int head_few_grad_parts(const HeadProblem& p) {
    const int64_t per = head_few_grad_rows(p);
    return static_cast<int>(std::min<int64_t>((p.V + per - 1) / per, kMaxCtas));
}

cudaError_t launch_head_few_grad(const HeadProblem& p, const HeadPicks& picks, const int32_t* alive,
                                 const float* lse, const float* gloss, bool accumulate, float* part,
                                 void* gH, int64_t ld_gh, void* gE, bool gE_bf16, cudaStream_t s) {
    FewGrad a = {};
    a.ld_h = p.ld_h;
    a.ld_e = p.ld_e;
    a.T = p.T;
    a.V = p.V;
    a.R = static_cast<int>(p.S * p.T);
    a.d = static_cast<int>(p.d);
    a.scale = p.scale;
    a.targets = p.tg.many ? nullptr : p.tg.ids;
    a.picks = picks;
    a.alive = alive;
    a.lse = lse;
    a.gloss = gloss;
    a.part = gH ? part : nullptr;
    a.gE = gE;
    a.ge_bf16 = gE_bf16;
    a.accumulate = accumulate;
    a.status = status_word();
    if (!a.status) return cudaErrorUnknown;
    const int size = p.bf16 ? 2 : 4, ctas = head_few_grad_parts(p);
    // gE's rows are as long as E's, and start on 16 bytes with them (on 8 if
    // they are of the shorter type).
    const bool vec = p.d * size % 16 == 0 && p.ld_e * size % 16 == 0 &&
                     (reinterpret_cast<uintptr_t>(p.E) | reinterpret_cast<uintptr_t>(gE)) % 16 == 0;
    cudaError_t e;
    if (p.bf16)
        e = vec ? grad_by_rows<__nv_bfloat16, true>(p, a, ctas, s)
                : grad_by_rows<__nv_bfloat16, false>(p, a, ctas, s);
    else
        e = vec ? grad_by_rows<float, true>(p, a, ctas, s) : grad_by_rows<float, false>(p, a, ctas, s);
    if (e != cudaSuccess || !gH) return e;
    return launch_pdl(k_head_few_sum, dim3(static_cast<unsigned>((a.R * p.d + 31) / 32)),
                      dim3(32 * kWarps), 0, s, static_cast<const float*>(part), ctas, a.R, a.d,
                      p.scale, gH, ld_gh, static_cast<int>(p.bf16));
}

}  // namespace dust
