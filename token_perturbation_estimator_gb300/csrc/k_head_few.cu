// The head's loss for a few rows (single tokens being scored): every row of E
// is read once, as it lies, and multiplied with all rows of H on the CUDA
// cores, fp32 throughout. Bound by E's bytes; the tensor-core kernel spends a
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
#include <algorithm>
#include <cmath>

#include "head.cuh"

namespace dust {

namespace {

constexpr int kWarps = 8;
constexpr int kSums = 16;
constexpr int kMaxRows = 8;
constexpr int64_t kMaxH = 24 * 1024;  // floats of H in shared memory: two CTAs per SM
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
    for (int i = threadIdx.x; i < NR * pitch; i += blockDim.x) {
        const int r = i / pitch, c = i - r * pitch;
        const int b = c / (32 * P), l = c / P % 32, k = c % P;
        h[r * pitch + place<P>(b, l, k)] =
            r < a.R && c < a.d ? to_f(H[r * a.ld_h + c]) : 0.0f;
    }
    __syncthreads();

    // The sum a lane ends with: that of E row v0 + u with H row r.
    const int u = lane / 2 / NR, r = lane / 2 % NR;
    const bool mine = (lane & 1) == 0 && r < a.R;
    const int32_t target = mine && a.targets ? a.targets[r % a.T] : -1;
    const float c = a.scale * kLog2e;
    float m = -INFINITY, s = 0.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps * U;
    for (int64_t v0 = (static_cast<int64_t>(blockIdx.x) * kWarps + w) * U; v0 < a.V; v0 += step) {
        float acc[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) acc[i] = 0.0f;
        const TX* e = E + v0 * a.ld_e + lane * P;
        for (int b = 0; b < blocks; ++b) {
            const bool in = (b * 32 + lane) * P < a.d;
            Loaded<TX, VEC> x[U];
#pragma unroll
            for (int i = 0; i < U; ++i)
                x[i].load(e + i * a.ld_e + b * 32 * P, in && v0 + i < a.V);
#pragma unroll
            for (int q = 0; q < NR; ++q) {
                float hv[P];
                if constexpr (P >= 4) {
#pragma unroll
                    for (int k = 0; k < P; k += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(
                            h + q * pitch + place<P>(b, lane, k));
                        hv[k] = f.x;
                        hv[k + 1] = f.y;
                        hv[k + 2] = f.z;
                        hv[k + 3] = f.w;
                    }
                } else {
                    hv[0] = h[q * pitch + place<P>(b, lane, 0)];
                }
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int k = 0; k < P; ++k)
                        acc[i * NR + q] = fmaf(x[i].at(k), hv[k], acc[i * NR + q]);
            }
        }
#pragma unroll
        for (int n = kSums / 2, off = 16; n > 0; n >>= 1, off >>= 1) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const bool up = (lane & off) != 0;
                const float keep = up ? acc[i + n] : acc[i], give = up ? acc[i] : acc[i + n];
                acc[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
            }
        }
        const float x = acc[0] + __shfl_xor_sync(0xffffffffu, acc[0], 1);
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
        default: return launch_few<TX, VEC, 8>(p, a, ctas, s);
    }
}

}  // namespace

// Few enough that this is faster than the tensor cores' tiles. us here / there
// (both with the joining launch), V 4096, d 512 and V 50257, d 2048:
//   bf16  R 1  6 / 9,  43 / 62     R 2  6 / 9,  46 / 55
//         R 4  7 / 9,  65 / 54     R 8  10 / 9, 96 / 54
//   fp32  R 1  7 / 29, 75 / 477    R 8  9 / 27, 142 / 458
// (bf16 rows of 1001 values, V 20000: R 4 33 / 38, R 8 40 / 38).
bool head_few(const HeadProblem& p) {
    const int64_t R = p.S * p.T;
    if (R > kMaxRows || rows_up(R) * p.d > kMaxH) return false;
    return !p.bf16 || R <= 2 || (R <= 4 && p.V * p.d <= (int64_t(1) << 24));
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

}  // namespace dust
