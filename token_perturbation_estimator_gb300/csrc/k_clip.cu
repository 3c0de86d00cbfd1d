// The norm over all gradients of a step, and the gradients scaled to it:
//     norm = sqrt(sum g^2),  out = g min(1, max_norm / norm)
//
// Two passes over chunks of kChunk values, each CTA's one after another: the first
// leaves one sum per CTA, the second adds those up in every CTA (in one order,
// so that all have the same factor) and scales, each CTA its chunks in reverse:
// what was read last is still in the L2. Squares are summed 16 at a
// time in fp32, those sums in 64 bits.
//
// Bound by memory: g is read twice and out written once.
#include <algorithm>
#include <cmath>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;                  // squares summed in fp32
constexpr int kChunk = kThreads * kGroup * 2;
constexpr int kCtas = 4;                    // per SM
constexpr int kMaxParts = 152 * kCtas;      // CTAs of a launch
constexpr int64_t kBatch = 512;             // tensors of a launch

// The tensors of a launch (in the kernel's parameters) and their chunks,
// numbered one tensor after another.
template <int N>
struct Batch {
    const void* g[N];
    void* out[N];
    int64_t n[N];
    int64_t first[N + 1];
    uint8_t bf16[N];
    int count;
    int64_t chunks;

    __device__ int tensor_of(int64_t chunk) const {
        int lo = 0, hi = count - 1;  // the last tensor whose first chunk is not past it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first[mid] <= chunk) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// The squares of a group.
__device__ __forceinline__ double squares(const float (&v)[kGroup]) {
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kGroup; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    // Above, what squares below fp32's range lose is less than the sum's last bit.
    if (sum >= 0x1p-90f && sum <= 0x1p127f) return static_cast<double>(sum);
    double d = 0.0;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) any |= __float_as_uint(v[i]) << 1;
    if (any == 0) return 0.0;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
    return d;
}

// A thread's group k of the chunk: 16 bytes at a time where g allows, else
// value by value, neighbouring lanes on neighbouring ones; zeros past the end.
template <typename TX>
__device__ __forceinline__ void load_group(const TX* p, int n, bool vec, int k, float (&v)[kGroup]) {
    constexpr int per = 16 / static_cast<int>(sizeof(TX));
    const int base = k * kThreads * kGroup;
    if (vec) {
#pragma unroll
        for (int j = 0; j < kGroup / per; ++j) {
            const int at = base + (j * kThreads + static_cast<int>(threadIdx.x)) * per;
            if (at + per <= n) {
                const uint4 q = *reinterpret_cast<const uint4*>(p + at);
                const TX* x = reinterpret_cast<const TX*>(&q);
#pragma unroll
                for (int i = 0; i < per; ++i) v[j * per + i] = to_f(x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < per; ++i) v[j * per + i] = at + i < n ? to_f(p[at + i]) : 0.0f;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            const int at = base + j * kThreads + static_cast<int>(threadIdx.x);
            v[j] = at < n ? to_f(p[at]) : 0.0f;
        }
    }
}

__device__ __forceinline__ float from_f(float v, float) { return v; }
__device__ __forceinline__ __nv_bfloat16 from_f(float v, __nv_bfloat16) { return __float2bfloat16_rn(v); }

template <typename TX>
__device__ __forceinline__ void store_group(TX* p, int n, bool vec, int k, const float (&v)[kGroup]) {
    constexpr int per = 16 / static_cast<int>(sizeof(TX));
    const int base = k * kThreads * kGroup;
    if (vec) {
#pragma unroll
        for (int j = 0; j < kGroup / per; ++j) {
            const int at = base + (j * kThreads + static_cast<int>(threadIdx.x)) * per;
            alignas(16) TX x[per];
#pragma unroll
            for (int i = 0; i < per; ++i) x[i] = from_f(v[j * per + i], TX());
            if (at + per <= n) {
                *reinterpret_cast<uint4*>(p + at) = *reinterpret_cast<const uint4*>(x);
            } else {
#pragma unroll
                for (int i = 0; i < per; ++i)
                    if (at + i < n) p[at + i] = x[i];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            const int at = base + j * kThreads + static_cast<int>(threadIdx.x);
            if (at < n) p[at] = from_f(v[j], TX());
        }
    }
}

__device__ __forceinline__ bool on_16(const void* a, const void* b) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

template <typename TX>
__device__ __forceinline__ double chunk_squares(const void* g, int64_t from, int n) {
    const TX* p = static_cast<const TX*>(g) + from;
    const bool vec = on_16(g, nullptr);
    float a[kGroup], b[kGroup];
    load_group(p, n, vec, 0, a);
    load_group(p, n, vec, 1, b);
    return squares(a) + squares(b);
}

template <typename TX>
__device__ __forceinline__ void chunk_scale(const void* g, void* out, int64_t from, int n, float c) {
    const TX* p = static_cast<const TX*>(g) + from;
    const bool vec = on_16(g, out);
    float a[kGroup], b[kGroup];
    load_group(p, n, vec, 0, a);
    load_group(p, n, vec, 1, b);
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
        a[i] *= c;
        b[i] *= c;
    }
    store_group(static_cast<TX*>(out) + from, n, vec, 0, a);
    store_group(static_cast<TX*>(out) + from, n, vec, 1, b);
}

// The CTA's sum, to all its threads.
__device__ __forceinline__ double cta_sum(double v) {
    __shared__ double sh[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += sh[i];
    return v;
}

// A CTA's chunks, and the tensor that one of them lies in.
template <int N>
struct Walk {
    const Batch<N>& b;
    int64_t from, to;
    int t;

    __device__ explicit Walk(const Batch<N>& batch) : b(batch) {
        from = b.chunks * blockIdx.x / gridDim.x;
        to = b.chunks * (blockIdx.x + 1) / gridDim.x;
    }
    __device__ __forceinline__ int count(int64_t chunk) const {
        return static_cast<int>(min(b.n[t] - (chunk - b.first[t]) * kChunk, static_cast<int64_t>(kChunk)));
    }
    __device__ __forceinline__ int64_t start(int64_t chunk) const { return (chunk - b.first[t]) * kChunk; }
};

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_clip_sum(const __grid_constant__ Batch<N> b, double* __restrict__ parts) {
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
    Walk<N> w(b);
    if (w.from < w.to) w.t = b.tensor_of(w.from);
    for (int64_t c = w.from; c < w.to; ++c) {
        while (c >= b.first[w.t + 1]) ++w.t;
        s += b.bf16[w.t] ? chunk_squares<__nv_bfloat16>(b.g[w.t], w.start(c), w.count(c))
                         : chunk_squares<float>(b.g[w.t], w.start(c), w.count(c));
    }
    s = cta_sum(s);
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_clip_scale(const __grid_constant__ Batch<N> b, const double* __restrict__ parts, int n_parts,
                 double max_norm, float* norm) {
    pdl_wait();
    pdl_trigger();
    double s = 0.0;
    for (int i = threadIdx.x; i < n_parts; i += kThreads) s += parts[i];
    const double length = sqrt(cta_sum(s));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(length);
    const float f = length <= max_norm ? 1.0f : static_cast<float>(max_norm / length);
    Walk<N> w(b);
    if (w.from < w.to) w.t = b.tensor_of(w.to - 1);
    for (int64_t c = w.to - 1; c >= w.from; --c) {
        while (c < b.first[w.t]) --w.t;
        if (!b.out[w.t] || (f == 1.0f && b.out[w.t] == b.g[w.t])) continue;
        if (b.bf16[w.t]) chunk_scale<__nv_bfloat16>(b.g[w.t], b.out[w.t], w.start(c), w.count(c), f);
        else chunk_scale<float>(b.g[w.t], b.out[w.t], w.start(c), w.count(c), f);
    }
}

template <int N>
Batch<N> batch_of(const dust_grad* g, int64_t n) {
    Batch<N> b;
    b.count = 0;
    b.chunks = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (g[i].n == 0) continue;
        const int k = b.count++;
        b.g[k] = g[i].g;
        b.out[k] = g[i].out;
        b.n[k] = g[i].n;
        b.bf16[k] = g[i].dtype == DUST_BF16;
        b.first[k] = b.chunks;
        b.chunks += (g[i].n + kChunk - 1) / kChunk;
    }
    b.first[b.count] = b.chunks;
    return b;
}

unsigned grid_of(int64_t chunks) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(chunks, kMaxParts)));
}

}  // namespace

size_t clip_workspace_bytes() { return sizeof(double) * kMaxParts * ((kMaxGrads + kBatch - 1) / kBatch); }

template <int N>
static cudaError_t launch_clip_by(const dust_grad* grads, int64_t n, float max_norm, float* norm,
                                  double* parts, cudaStream_t s) {
    int n_parts = 0;
    for (int64_t i = 0; i < n || i == 0; i += N) {
        const Batch<N> b = batch_of<N>(grads + i, std::min<int64_t>(N, n - i));
        const unsigned grid = grid_of(b.chunks);
        const cudaError_t e = launch_pdl(k_clip_sum<N>, dim3(grid), dim3(kThreads), 0, s, b, parts + n_parts);
        if (e != cudaSuccess) return e;
        n_parts += static_cast<int>(grid);
    }
    for (int64_t i = 0; i < n || i == 0; i += N) {
        const Batch<N> b = batch_of<N>(grads + i, std::min<int64_t>(N, n - i));
        const cudaError_t e = launch_pdl(k_clip_scale<N>, dim3(grid_of(b.chunks)), dim3(kThreads), 0, s, b,
                                         parts, n_parts, static_cast<double>(max_norm),
                                         i == 0 ? norm : nullptr);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_clip(const dust_grad* grads, int64_t n, float max_norm, float* norm, void* ws,
                        cudaStream_t s) {
    ProfScope ps(kStageClip, s);
    double* parts = static_cast<double*>(ws);
    return n <= 64 ? launch_clip_by<64>(grads, n, max_norm, norm, parts, s)
                   : launch_clip_by<kBatch>(grads, n, max_norm, norm, parts, s);
}

}  // namespace dust
