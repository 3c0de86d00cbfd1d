// The norm over all gradients of a step, and the gradients scaled to it:
//     norm = sqrt(sum g^2),  out = g min(1, max_norm / norm)
//
// Two passes over chunks of kChunk values, each CTA's one after another: the
// first leaves one sum per CTA, the second adds those up in every CTA (in one
// order, so that all have the same factor) and scales, each CTA its chunks in
// reverse: what was read last may still be in the L2 (151 MB of gradients: 80 us
// instead of 86). Squares are summed 16 at a time in fp32, those sums in 64 bits.
// Few values take one launch of a cluster, whose CTAs hand their sums to one
// another.
//
// Bound by memory: g is read twice and out written once. 48 tensors, 151 MB fp32:
// 75 us = 6.1 TB/s, of which 27 for the norm; 5 tensors, 0.3 MB bf16: 11 us.
#include <algorithm>
#include <cmath>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 16;                  // squares summed in fp32
constexpr int kChunk = kThreads * kGroup;
constexpr int kCtas = 4;                    // per SM
constexpr int kMaxParts = 152 * kCtas;      // CTAs of a launch
constexpr int64_t kBatch = 512;             // tensors of a launch
constexpr int kFewTensors = 64;             // of a launch of few, whose parameters are shorter
constexpr int kCluster = 8;                 // CTAs that share few values,
constexpr int kTeams = 4;                   // each as several teams of kThreads
constexpr int64_t kFewChunks = kCluster * kTeams * 4;

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
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// A sum of squares: hi + lo, hi the running sum in fp32 and lo what its
// roundings lost; and `far`, what lies outside of the range where that is exact
// enough.
struct Squares {
    float hi = 0.0f, lo = 0.0f;
    double far = 0.0;

    // The sum and its error, exactly (Knuth).
    __device__ __forceinline__ void add(float v) {
        const float s = hi + v, t = s - hi;
        lo += (hi - (s - t)) + (v - t);
        hi = s;
    }
    __device__ __forceinline__ void add(const float (&v)[kGroup]) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kGroup; ++i) s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
        const float sum = (s[0] + s[1]) + (s[2] + s[3]);
        // From 2^-90 on, what squares below fp32's range lose is less than the
        // sum's last bit; up to 2^80, the sums of 2^40 groups stay in the range.
        if (sum >= 0x1p-90f && sum <= 0x1p80f) {
            add(sum);
            return;
        }
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) any |= __float_as_uint(v[i]) << 1;
        if (any == 0) return;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) far = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), far);
    }
    __device__ __forceinline__ double value() const {
        return static_cast<double>(hi) + static_cast<double>(lo) + far;
    }
};

// What values are multiplied by, one after the other: a factor below fp32's
// normal numbers, which would have few bits as one of them or none, is a number
// below 1 times a power of two; else that is 1. (Values whose squares overflow are
// scaled so: 1e38 to a norm of 1. A product of them and `normal` does not overflow
// and loses bits only where the result has none left; `normal` has all of its own
// where that is above 2^-147.)
struct Factor {
    float normal, power;
};

// A thread's group of a chunk: 16 bytes at a time (VEC), or value by value,
// neighbouring lanes on neighbouring ones.
template <typename TX, bool VEC>
struct Group {
    static constexpr int kPer = VEC ? 16 / static_cast<int>(sizeof(TX)) : 1;
    static __device__ __forceinline__ int at(int j) {
        return (j * kThreads + static_cast<int>(threadIdx.x) % kThreads) * kPer;
    }
    struct alignas(sizeof(TX) * kPer) Raw { TX x[kPer]; };

    // Of a chunk of n values (FULL: kChunk), zeros past them.
    template <bool FULL>
    static __device__ __forceinline__ void load(const TX* p, int n, float (&v)[kGroup]) {
#pragma unroll
        for (int j = 0; j < kGroup / kPer; ++j) {
            if (FULL || at(j) + kPer <= n) {
                const Raw q = *reinterpret_cast<const Raw*>(p + at(j));
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[j * kPer + i] = to_f(q.x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i) v[j * kPer + i] = at(j) + i < n ? to_f(p[at(j) + i]) : 0.0f;
            }
        }
    }
    template <bool FULL>
    static __device__ __forceinline__ void store(TX* p, int n, const float (&v)[kGroup], Factor c) {
#pragma unroll
        for (int j = 0; j < kGroup / kPer; ++j) {
            Raw q;
#pragma unroll
            for (int i = 0; i < kPer; ++i) from_f(v[j * kPer + i] * c.normal * c.power, q.x[i]);
            if (FULL || at(j) + kPer <= n) {
                *reinterpret_cast<Raw*>(p + at(j)) = q;
            } else {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (at(j) + i < n) p[at(j) + i] = q.x[i];
            }
        }
    }
};

// The squares of n values from p, by kThreads threads.
template <typename TX, bool VEC>
__device__ void add_squares(Squares& s, const TX* p, int64_t n) {
    using G = Group<TX, VEC>;
    for (; n >= 2 * kChunk; n -= 2 * kChunk, p += 2 * kChunk) {  // two at once
        float v[kGroup], u[kGroup];
        G::template load<true>(p, kChunk, v);
        G::template load<true>(p + kChunk, kChunk, u);
        s.add(v);
        s.add(u);
    }
    for (; n > 0; n -= kChunk, p += kChunk) {
        float v[kGroup];
        G::template load<false>(p, static_cast<int>(min(n, static_cast<int64_t>(kChunk))), v);
        s.add(v);
    }
}

// n values from p to out, times c, the last ones first.
template <typename TX, bool VEC>
__device__ void scale_to(const TX* p, TX* out, int64_t n, Factor c) {
    using G = Group<TX, VEC>;
    const int64_t full = n / kChunk * kChunk;
    if (n > full) {
        float v[kGroup];
        G::template load<false>(p + full, static_cast<int>(n - full), v);
        G::template store<false>(out + full, static_cast<int>(n - full), v, c);
    }
    for (int64_t i = full - kChunk; i >= kChunk; i -= 2 * kChunk) {  // two at once
        float v[kGroup], u[kGroup];
        G::template load<true>(p + i, kChunk, v);
        G::template load<true>(p + i - kChunk, kChunk, u);
        G::template store<true>(out + i, kChunk, v, c);
        G::template store<true>(out + i - kChunk, kChunk, u, c);
    }
    if (full / kChunk % 2 != 0) {
        float v[kGroup];
        G::template load<true>(p, kChunk, v);
        G::template store<true>(out, kChunk, v, c);
    }
}

__device__ __forceinline__ bool on_16(const void* a, const void* b) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 15) == 0;
}

template <typename TX>
__device__ __forceinline__ void squares_by(Squares& s, const void* g, int64_t from, int64_t n) {
    const TX* p = static_cast<const TX*>(g) + from;
    if (on_16(g, nullptr)) add_squares<TX, true>(s, p, n);
    else add_squares<TX, false>(s, p, n);
}

template <typename TX>
__device__ __forceinline__ void scale_by(const void* g, void* out, int64_t from, int64_t n, Factor c) {
    const TX* p = static_cast<const TX*>(g) + from;
    TX* o = static_cast<TX*>(out) + from;
    if (on_16(g, out)) scale_to<TX, true>(p, o, n, c);
    else scale_to<TX, false>(p, o, n, c);
}

// The chunks [from, to) of a CTA, or of a team of one, tensor by tensor.
template <int N>
struct Walk {
    const Batch<N>& b;
    int64_t from, to;

    __device__ Walk(const Batch<N>& batch, int cta, int ctas) : b(batch) {
        from = b.chunks * cta / ctas;
        to = b.chunks * (cta + 1) / ctas;
    }

    __device__ Squares squares() const {
        Squares s;
        if (from >= to) return s;
        for (int t = b.tensor_of(from); t < b.count && b.first[t] < to; ++t) {
            const int64_t at = (max(from, b.first[t]) - b.first[t]) * kChunk;
            const int64_t n = min(b.n[t], (to - b.first[t]) * kChunk) - at;
            if (b.bf16[t]) squares_by<__nv_bfloat16>(s, b.g[t], at, n);
            else squares_by<float>(s, b.g[t], at, n);
        }
        return s;
    }

    __device__ void scale(Factor c) const {
        if (from >= to) return;
        for (int t = b.tensor_of(to - 1); t >= 0 && b.first[t + 1] > from; --t) {
            if (!b.out[t] || (c.normal == 1.0f && b.out[t] == b.g[t])) continue;
            const int64_t at = (max(from, b.first[t]) - b.first[t]) * kChunk;
            const int64_t n = min(b.n[t], (to - b.first[t]) * kChunk) - at;
            if (b.bf16[t]) scale_by<__nv_bfloat16>(b.g[t], b.out[t], at, n, c);
            else scale_by<float>(b.g[t], b.out[t], at, n, c);
        }
    }
};

// The CTA's sum, to thread 0.
template <int THREADS>
__device__ __forceinline__ double cta_sum(Squares s) {
    __shared__ double sh[THREADS / 32];
    if (__any_sync(0xffffffffu, s.far != 0.0))
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s.far += __shfl_xor_sync(0xffffffffu, s.far, off);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        s.lo += __shfl_xor_sync(0xffffffffu, s.lo, off);
        s.add(__shfl_xor_sync(0xffffffffu, s.hi, off));
    }
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = s.value();
    __syncthreads();
    double v = 0.0;
    if (threadIdx.x < 32) {
        if (threadIdx.x < THREADS / 32) v = sh[threadIdx.x];
#pragma unroll
        for (int off = THREADS / 64; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    return v;
}

// min(1, max_norm / length).
__device__ __forceinline__ Factor factor(double length, double max_norm) {
    if (length <= max_norm) return {1.0f, 1.0f};
    const double c = max_norm / length;
    if (!(c > 0.0 && c < 0x1p-126)) return {static_cast<float>(c), 1.0f};
    const int up = min(-1 - ilogb(c), 149);  // 2^-149 is the least power that there is
    return {static_cast<float>(scalbn(c, up)), scalbnf(1.0f, -up)};
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_clip_sum(const __grid_constant__ Batch<N> b, double* __restrict__ parts) {
    pdl_wait();
    pdl_trigger();
    const double s = cta_sum<kThreads>(Walk<N>(b, blockIdx.x, gridDim.x).squares());
    if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_clip_scale(const __grid_constant__ Batch<N> b, const double* __restrict__ parts, int n_parts,
                 double max_norm, float* norm) {
    __shared__ Factor shared_factor;
    pdl_wait();
    pdl_trigger();
    if (threadIdx.x < 32) {
        double s = 0.0;
#pragma unroll 8
        for (int i = threadIdx.x; i < n_parts; i += 32) s += parts[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (threadIdx.x == 0) {
            const double length = sqrt(s);
            shared_factor = factor(length, max_norm);
            if (norm && blockIdx.x == 0) *norm = static_cast<float>(length);
        }
    }
    __syncthreads();
    Walk<N>(b, blockIdx.x, gridDim.x).scale(shared_factor);
}

// The same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ double read_at_rank(const double* p, int rank) {
    uint32_t at;
    double v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
    return v;
}

// The lanes of a warp meet first: .aligned wants them to arrive together.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Both passes by one cluster.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kTeams * kThreads)
    k_clip_few(const __grid_constant__ Batch<kFewTensors> b, double max_norm, float* norm) {
    __shared__ double mine;
    __shared__ Factor shared_factor;
    pdl_wait();
    pdl_trigger();
    const Walk<kFewTensors> w(b, blockIdx.x * kTeams + threadIdx.x / kThreads, kCluster * kTeams);
    const double s = cta_sum<kTeams * kThreads>(w.squares());
    if (threadIdx.x == 0) mine = s;
    cluster_barrier();
    if (threadIdx.x == 0) {
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < kCluster; ++i) all += read_at_rank(&mine, i);
        const double length = sqrt(all);
        shared_factor = factor(length, max_norm);
        if (blockIdx.x == 0) *norm = static_cast<float>(length);
    }
    cluster_barrier();  // nobody leaves before its sum is read
    w.scale(shared_factor);
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

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

template <int N>
cudaError_t launch_sum(const Batch<N>& b, double* parts, int* n_parts, cudaStream_t s) {
    const unsigned grid = grid_of(b.chunks);
    double* to = parts + *n_parts;
    *n_parts += static_cast<int>(grid);
    return launch_pdl(k_clip_sum<N>, dim3(grid), dim3(kThreads), 0, s, b, to);
}

template <int N>
cudaError_t launch_scale(const Batch<N>& b, const double* parts, int n_parts, float max_norm, float* norm,
                         cudaStream_t s) {
    return launch_pdl(k_clip_scale<N>, dim3(grid_of(b.chunks)), dim3(kThreads), 0, s, b, parts, n_parts,
                      static_cast<double>(max_norm), norm);
}

}  // namespace

size_t clip_workspace_bytes() { return sizeof(double) * kMaxParts * ((kMaxGrads + kBatch - 1) / kBatch); }

cudaError_t launch_clip(const dust_grad* grads, int64_t n, float max_norm, float* norm, void* ws,
                        cudaStream_t s) {
    ProfScope ps(kStageClip, s);
    double* parts = static_cast<double*>(ws);
    int n_parts = 0;
    if (n <= kFewTensors) {
        const Batch<kFewTensors> b = batch_of<kFewTensors>(grads, n);
        if (b.chunks <= kFewChunks)
            return launch_pdl(k_clip_few, dim3(kCluster), dim3(kTeams * kThreads), 0, s, b,
                              static_cast<double>(max_norm), norm);
        DUST_TRY(launch_sum(b, parts, &n_parts, s));
        return launch_scale(b, parts, n_parts, max_norm, norm, s);
    }
    for (int64_t i = 0; i < n; i += kBatch)
        DUST_TRY(launch_sum(batch_of<kBatch>(grads + i, std::min(kBatch, n - i)), parts, &n_parts, s));
    for (int64_t i = 0; i < n; i += kBatch)
        DUST_TRY(launch_scale(batch_of<kBatch>(grads + i, std::min(kBatch, n - i)), parts, n_parts, max_norm,
                              i == 0 ? norm : nullptr, s));
    return cudaSuccess;
}

}  // namespace dust
