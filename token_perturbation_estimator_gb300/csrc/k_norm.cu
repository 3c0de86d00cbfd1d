// Layer norm, forward and backward. Per row of d values, n = (x - mean) rstd:
//     y  = n weight + bias
//     gx = rstd (gn - mean(gn) - n mean(gn n)),  gn = gy weight
//     gweight = sum_t gy n,  gbias = sum_t gy
// Bound by memory: the forward reads x and writes y once, the backward reads
// gy and x and writes gx once, up to a width of kMaxWidth.
//
// A row is held in registers by one warp (half or a quarter of one for narrow
// rows, several for wide ones), E values a lane as they were loaded: the
// mean, then the deviations, then the result come from them without a second
// read, and a sum over a row needs ten shuffles, no barrier. While a row is
// worked on, the warp's next two are on their way into shared memory
// (cp.async, each thread's own values, so again no barrier). Both matter:
// with 8 values a thread and rows spread over a CTA, two thirds of the
// instructions were reductions and the forward at 65536 x 2048 bf16 was bound
// by issue at 118 us; with a warp per row but loads straight into registers,
// it was bound by latency at the same 118 us.
// Rows that start on 16 bytes are read and written 16 bytes a lane; others
// value by value, neighbouring lanes on neighbouring values (bf16 ones, 2
// bytes, straight into registers: cp.async takes 4 at least).
//
// The backward adds its rows' gy n and gy per column in registers, the CTA's
// warps add theirs up in shared memory, and each CTA leaves one partial row;
// k_norm_finish sums the partial rows in order. No atomics: the result
// depends on T, d, the type and the alignment only.
//
// Wider rows are read once per pass by one CTA.
#include <algorithm>
#include <mutex>

#include "f32x2.cuh"
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

constexpr int kThreads = 256;     // of a CTA whose rows take a warp or less
constexpr int kMaxThreads = 512;  // of one whose rows take several warps, 16 values a lane
constexpr int64_t kMaxWidth = kMaxThreads * 16;
constexpr int kRing = 2;          // rows on their way per warp
constexpr int kOwnParams = 16;    // values per lane up to which weight and bias stay in registers

// Where a thread's E values of a row lie, thread l of the g that share it.
// VEC: 16 bytes at a time, load j being columns [(j g + l) per, + per); else
// single values, per = 1.
template <typename TX, bool VEC, int E>
struct Layout {
    static constexpr int kPer = VEC ? 16 / static_cast<int>(sizeof(TX)) : 1;
    static constexpr int kLoads = E / kPer;
    // A thread's bytes of one row in the ring; 0 where rows come straight.
    static constexpr bool kAsync = VEC || sizeof(TX) == 4;
    static constexpr int kPiece = VEC ? 16 : 4;
    static constexpr int kBytes = kAsync ? kLoads * kPiece : 0;

    static __device__ __forceinline__ int column(int l, int g, int j) { return (j * g + l) * kPer; }
};

// Starts the copy of a row (none if !any: zeros) to this thread's places in a
// slot of the ring, zeros past column d.
template <typename TX, bool VEC, int E>
__device__ __forceinline__ void fetch_row(uint32_t slot, const TX* row, bool any, int l, int g,
                                          int d) {
    using L = Layout<TX, VEC, E>;
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        const int c = L::column(l, g, j);
        const bool in = any && c < d;
        const uint32_t to = slot + (j * blockDim.x + threadIdx.x) * L::kPiece;
        const TX* from = in ? row + c : row;
        if constexpr (VEC)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                         "r"(in ? 16 : 0)
                         : "memory");
        else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from),
                         "r"(in ? 4 : 0)
                         : "memory");
    }
}

__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of this thread's copies have landed.
template <int N> __device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The two values of a 32-bit word of bf16.
__device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// A row's values from a slot of the ring, or straight from the row.
template <typename TX, bool VEC, int E>
__device__ __forceinline__ void get_row(float2 (&v)[E / 2], const unsigned char* slot,
                                        const TX* row, int l, int g, int d) {
    using L = Layout<TX, VEC, E>;
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) {
            const uint4 q =
                *reinterpret_cast<const uint4*>(slot + (j * blockDim.x + threadIdx.x) * 16);
            if constexpr (sizeof(TX) == 2) {
                v[4 * j] = unpack(q.x);
                v[4 * j + 1] = unpack(q.y);
                v[4 * j + 2] = unpack(q.z);
                v[4 * j + 3] = unpack(q.w);
            } else {
                v[2 * j] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
                v[2 * j + 1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float x;
            if constexpr (L::kAsync) {
                x = *reinterpret_cast<const float*>(slot + (j * blockDim.x + threadIdx.x) * 4);
            } else {
                const int c = L::column(l, g, j);
                x = c < d ? to_f(row[c]) : 0.0f;
            }
            (j & 1 ? v[j / 2].y : v[j / 2].x) = x;
        }
    }
}

// Sets the values past column d to 0.
template <typename TX, bool VEC, int E>
__device__ __forceinline__ void clear_past(float2 (&v)[E / 2], int l, int g, int d) {
    using L = Layout<TX, VEC, E>;
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        if (L::column(l, g, j) < d) continue;
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < L::kPer / 2; ++k) v[j * L::kPer / 2 + k] = make_float2(0.0f, 0.0f);
        } else {
            (j & 1 ? v[j / 2].y : v[j / 2].x) = 0.0f;
        }
    }
}

template <typename TX, bool VEC, int E>
__device__ __forceinline__ void put_row(TX* row, const float2 (&v)[E / 2], int l, int g, int d) {
    using L = Layout<TX, VEC, E>;
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        const int c = L::column(l, g, j);
        if (c >= d) continue;
        if constexpr (VEC && sizeof(TX) == 2) {
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[4 * j + k].x, v[4 * j + k].y);
                q[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(row + c) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if constexpr (VEC) {
            *reinterpret_cast<float4*>(row + c) =
                make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
        } else {
            row[c] = from_f<TX>(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    }
}

// A parameter's values at this thread's columns (`none` where there is no
// parameter): kept in registers, or (many values a lane) one copy per CTA in
// shared memory, laid out so that lanes read neighbouring 16 bytes.
template <typename TX, bool VEC, int E>
__device__ __forceinline__ void own_param(float2 (&w)[E / 2], const float* p, float none, int l,
                                          int g, int d) {
    using L = Layout<TX, VEC, E>;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = L::column(l, g, i / L::kPer) + i % L::kPer;
        (i & 1 ? w[i / 2].y : w[i / 2].x) = p && c < d ? p[c] : none;
    }
}
template <typename TX, bool VEC, int E, int G>
__device__ __forceinline__ void share_param(float* to, const float* p, float none, int d) {
    using L = Layout<TX, VEC, E>;
    constexpr int N = L::kPer < 4 ? L::kPer : 4;  // floats that a lane reads at once
    for (int i = threadIdx.x; i < G * E; i += blockDim.x) {
        // i = (chunk G + l) N + k: the k-th of the chunk-th N values of lane l
        const int k = i % N, l = i / N % G, chunk = i / N / G;
        const int at = chunk * N + k;  // its place among the lane's values
        const int c = L::column(l, G, at / L::kPer) + at % L::kPer;
        to[i] = p && c < d ? p[c] : none;
    }
}
template <typename TX, bool VEC, int E, int G>
__device__ __forceinline__ float2 shared_param(const float* at, int l, int pair) {
    using L = Layout<TX, VEC, E>;
    if constexpr (L::kPer == 1) {
        return make_float2(at[2 * pair * G + l], at[(2 * pair + 1) * G + l]);
    } else {  // pairs 2 i and 2 i + 1 share 16 bytes: one load for both
        const float4 q = reinterpret_cast<const float4*>(at)[(pair / 2) * G + l];
        return pair & 1 ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
    }
}

// Sums of N values over the threads that share a row, to all of them. G lanes
// of a warp, or (MULTI) `warps` warps, which meet in shared memory: two slots
// used in turn, so that one barrier per sum is enough.
template <int G, int MULTI, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float (*sh)[N * 16], int& slot, int warps) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    if constexpr (MULTI > 0) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) sh[slot][k * 16 + warp] = v[k];
        __syncthreads();
        const int first = warp / warps * warps;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0.0f;
            for (int i = 0; i < warps; ++i) s += sh[slot][k * 16 + first + i];
            v[k] = s;
        }
        slot ^= 1;
    }
}

// A thread's part of a sum over pairs, in two chains.
template <int E>
__device__ __forceinline__ float total(const float2 (&v)[E / 2]) {
    float2 a = v[0], b = v[1];
#pragma unroll
    for (int i = 2; i < E / 2; i += 2) {
        a = add2(a, v[i]);
        b = add2(b, v[i + 1]);
    }
    a = add2(a, b);
    return a.x + a.y;
}

template <typename TX, bool VEC, int G, int E, int MULTI>
__global__ void __launch_bounds__(MULTI == 2 ? kMaxThreads : kThreads, MULTI ? 1 : E <= 32 ? 3 : 2)
    k_norm(const TX* x, int64_t ld_x, int64_t T, int d, int warps,
           const float* __restrict__ weight, const float* __restrict__ bias, float eps, TX* y,
           int64_t ld_y, float* mean, float* rstd) {
    using L = Layout<TX, VEC, E>;
    constexpr bool kOwn = E <= kOwnParams;
    static_assert(kOwn || MULTI == 0, "shared parameters are laid out for one warp per row");
    __shared__ float sh[2][16];
    extern __shared__ __align__(16) unsigned char ring[];
    int slot = 0;
    const int g = MULTI ? 32 * warps : G;
    const int l = threadIdx.x % g, sub = threadIdx.x / g, rows = blockDim.x / g;
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows;
    const uint32_t slot_bytes = blockDim.x * L::kBytes;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const TX* from = x + (first + sub) * ld_x;  // the next row to fetch
    int64_t ahead = first + sub;
    const auto fetch = [&](int at) {
        const bool any = ahead < T;
        fetch_row<TX, VEC, E>(ring_at + at * slot_bytes, any ? from : x, any, l, g, d);
        copies_begun();
        from += step * ld_x;
        ahead += step;
    };
    pdl_wait();
    pdl_trigger();
    if constexpr (L::kAsync) {
        fetch(0);
        fetch(1);
    }
    float2 w[kOwn ? E / 2 : 1], b[kOwn ? E / 2 : 1];
    float* params = reinterpret_cast<float*>(ring + kRing * slot_bytes);
    if constexpr (kOwn) {
        own_param<TX, VEC, E>(w, weight, 1.0f, l, g, d);
        own_param<TX, VEC, E>(b, bias, 0.0f, l, g, d);
    } else {
        share_param<TX, VEC, E, G>(params, weight, 1.0f, d);
        share_param<TX, VEC, E, G>(params + G * E, bias, 0.0f, d);
        __syncthreads();
    }
    TX* to = y + (first + sub) * ld_y;
    int at = 0;
    for (int64_t t0 = first; t0 < T; t0 += step, at ^= 1, to += step * ld_y) {
        const int64_t t = t0 + sub;  // every thread of the CTA goes as often
        const bool in = t < T;
        float2 v[E / 2];
        if constexpr (L::kAsync) copies_landed<kRing - 1>();
        get_row<TX, VEC, E>(v, ring + at * slot_bytes, in ? x + t * ld_x : x, l, g, d);
        float s[1] = {total<E>(v)};
        // The row has been read (its sum needs it): its slot is free.
        if constexpr (L::kAsync) fetch(at);
        row_sum<G, MULTI, 1>(s, sh, slot, warps);
        const float mu = s[0] * inv;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[i] = add2(v[i], both(-mu));
        clear_past<TX, VEC, E>(v, l, g, d);
        float2 q[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int i = 0; i < E / 2; ++i) q[i & 1] = fma2(v[i], v[i], q[i & 1]);
        q[0] = add2(q[0], q[1]);
        s[0] = q[0].x + q[0].y;
        row_sum<G, MULTI, 1>(s, sh, slot, warps);
        const float r = 1.0f / sqrtf(fmaf(s[0], inv, eps));
        if (!in) continue;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float2 wi, bi;
            if constexpr (kOwn) {
                wi = w[i];
                bi = b[i];
            } else {
                wi = shared_param<TX, VEC, E, G>(params, l, i);
                bi = shared_param<TX, VEC, E, G>(params + G * E, l, i);
            }
            v[i] = fma2(mul2(v[i], both(r)), wi, bi);
        }
        put_row<TX, VEC, E>(to, v, l, g, d);
        if (l == 0) {
            if (mean) mean[t] = mu;
            if (rstd) rstd[t] = r;
        }
    }
}

template <typename TX, bool VEC, int G, int E, int MULTI>
__global__ void __launch_bounds__(MULTI == 2 ? kMaxThreads : kThreads, MULTI ? 1 : 2)
    k_norm_grad(const TX* gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x, int64_t T,
                int d, int warps, const float* __restrict__ weight,
                const float* __restrict__ mean, const float* __restrict__ rstd, TX* gx,
                int64_t ld_gx, float* __restrict__ part) {
    using L = Layout<TX, VEC, E>;
    __shared__ float sh[2][32];
    // The ring; then, for one sum at a time, floats [rows of the CTA][g E].
    extern __shared__ __align__(16) unsigned char ring[];
    int slot = 0;
    const int g = MULTI ? 32 * warps : G;
    const int l = threadIdx.x % g, sub = threadIdx.x / g, rows = blockDim.x / g;
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * rows;
    const uint32_t slot_bytes = blockDim.x * L::kBytes;
    const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const TX* from_g = gy + (first + sub) * ld_gy;  // the next rows to fetch
    const TX* from_x = x + (first + sub) * ld_x;
    int64_t ahead = first + sub;
    const auto fetch = [&](int at) {
        const bool any = ahead < T;
        fetch_row<TX, VEC, E>(ring_at + 2 * at * slot_bytes, any ? from_g : gy, any, l, g, d);
        fetch_row<TX, VEC, E>(ring_at + (2 * at + 1) * slot_bytes, any ? from_x : x, any, l, g, d);
        copies_begun();
        from_g += step * ld_gy;
        from_x += step * ld_x;
        ahead += step;
    };
    pdl_wait();
    pdl_trigger();
    if constexpr (L::kAsync) {
        fetch(0);
        fetch(1);
    }
    float2 w[E / 2], aw[E / 2], ab[E / 2];
    own_param<TX, VEC, E>(w, weight, 1.0f, l, g, d);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) aw[i] = ab[i] = make_float2(0.0f, 0.0f);
    float next_mu = 0.0f, next_r = 0.0f;
    if (first + sub < T) {
        next_mu = mean[first + sub];
        next_r = rstd[first + sub];
    }
    TX* to = gx + (first + sub) * ld_gx;
    int at = 0;
    for (int64_t t0 = first; t0 < T; t0 += step, at ^= 1, to += step * ld_gx) {
        const int64_t t = t0 + sub;
        const bool in = t < T;
        const float mu = next_mu, r = next_r;
        if (t + step < T) {
            next_mu = mean[t + step];
            next_r = rstd[t + step];
        }
        float s[2] = {0.0f, 0.0f};
        float2 gn[E / 2], n[E / 2];
        if constexpr (L::kAsync) copies_landed<kRing - 1>();
        get_row<TX, VEC, E>(gn, ring + 2 * at * slot_bytes, in ? gy + t * ld_gy : gy, l, g, d);
        get_row<TX, VEC, E>(n, ring + (2 * at + 1) * slot_bytes, in ? x + t * ld_x : x, l, g, d);
        if (in) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) n[i] = mul2(add2(n[i], both(-mu)), both(r));
            clear_past<TX, VEC, E>(n, l, g, d);  // gy is 0 there
            float2 q0 = {0.0f, 0.0f}, q1 = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                aw[i] = fma2(gn[i], n[i], aw[i]);
                ab[i] = add2(ab[i], gn[i]);
                gn[i] = mul2(gn[i], w[i]);
                q0 = add2(q0, gn[i]);
                q1 = fma2(gn[i], n[i], q1);
            }
            s[0] = q0.x + q0.y;
            s[1] = q1.x + q1.y;
        }
        // Both rows have been read (the sums need them): their slots are free.
        if constexpr (L::kAsync) fetch(at);
        row_sum<G, MULTI, 2>(s, sh, slot, warps);
        if (!in || !gx) continue;
        const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            gn[i] = mul2(fma2(n[i], both(-b), add2(gn[i], both(-a))), both(r));
        put_row<TX, VEC, E>(to, gn, l, g, d);
    }
    if (!part) return;
    if constexpr (L::kAsync) copies_landed<0>();  // the ring is about to hold the sums
    float* cols = reinterpret_cast<float*>(ring);
    float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += d) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float2 p = which ? ab[i / 2] : aw[i / 2];
            cols[sub * g * E + L::column(l, g, i / L::kPer) + i % L::kPer] = i & 1 ? p.y : p.x;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            float v = 0.0f;
            for (int i = 0; i < rows; ++i) v += cols[i * g * E + c];
            out[c] = v;
        }
    }
}

// gweight and gbias from n partial rows of 2 d values: 32 columns a CTA, the
// partial rows dealt to 32 warps, whose sums are added in order.
__global__ void __launch_bounds__(1024)
    k_norm_finish(const float* __restrict__ part, int64_t n, int64_t d, int accumulate,
                  float* gweight, float* gbias) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float v = 0.0f;
    if (c < 2 * d) {
#pragma unroll 8
        for (int64_t i = k; i < n; i += 32) v += part[i * 2 * d + c];
    }
    sh[k][lane] = v;
    __syncthreads();
    if (k != 0 || c >= 2 * d) return;
    float* out = c < d ? gweight : gbias;
    if (!out) return;
    out += c < d ? c : c - d;
    v = 0.0f;
    for (int i = 0; i < 32; ++i) v += sh[i][lane];
    *out = accumulate ? *out + v : v;
}

// ---------------------------------------------------------- wide rows

constexpr int kWideThreads = 512;
constexpr int64_t kWideChunks = 256;  // row chunks of the column sums

template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* sh) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        for (int k = 0; k < N; ++k) sh[k * 32 + (threadIdx.x >> 5)] = v[k];
    __syncthreads();
    for (int k = 0; k < N; ++k) {
        v[k] = 0.0f;
        for (int i = 0; i < kWideThreads / 32; ++i) v[k] += sh[k * 32 + i];
    }
}

template <typename TX>
__global__ void __launch_bounds__(kWideThreads)
    k_norm_wide(const TX* x, int64_t ld_x, int64_t T, int64_t d, const float* __restrict__ weight,
                const float* __restrict__ bias, float eps, TX* y, int64_t ld_y, float* mean,
                float* rstd) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[64];
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const TX* xr = x + t * ld_x;
        float s[1] = {0.0f};
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) s[0] += to_f(xr[c]);
        block_sum<1>(s, sh);
        const float mu = s[0] / static_cast<float>(d);
        s[0] = 0.0f;
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float e = to_f(xr[c]) - mu;
            s[0] = fmaf(e, e, s[0]);
        }
        block_sum<1>(s, sh);
        const float r = 1.0f / sqrtf(s[0] / static_cast<float>(d) + eps);
        TX* yr = y + t * ld_y;
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads)
            yr[c] = from_f<TX>(fmaf((to_f(xr[c]) - mu) * r, weight ? weight[c] : 1.0f,
                                    bias ? bias[c] : 0.0f));
        if (threadIdx.x == 0) {
            if (mean) mean[t] = mu;
            if (rstd) rstd[t] = r;
        }
    }
}

// Column sums of one row chunk: 32 columns a CTA, eight row lanes.
template <typename TX>
__global__ void __launch_bounds__(256)
    k_norm_cols(const TX* __restrict__ gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x,
                int64_t T, int64_t d, const float* __restrict__ mean,
                const float* __restrict__ rstd, int64_t chunk, float* __restrict__ part) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sw[8][32], sb[8][32];
    const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * chunk;
    const int64_t t1 = t0 + chunk < T ? t0 + chunk : T;
    float w = 0.0f, b = 0.0f;
    if (c < d) {
        for (int64_t t = t0 + rl; t < t1; t += 8) {
            const float g = to_f(gy[t * ld_gy + c]);
            w = fmaf(g, (to_f(x[t * ld_x + c]) - mean[t]) * rstd[t], w);
            b += g;
        }
    }
    sw[rl][lane] = w;
    sb[rl][lane] = b;
    __syncthreads();
    if (rl != 0 || c >= d) return;
    for (int i = 1; i < 8; ++i) {
        w += sw[i][lane];
        b += sb[i][lane];
    }
    float* p = part + static_cast<int64_t>(blockIdx.y) * 2 * d;
    p[c] = w;
    p[d + c] = b;
}

template <typename TX>
__global__ void __launch_bounds__(kWideThreads)
    k_norm_gx_wide(const TX* gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x, int64_t T,
                   int64_t d, const float* __restrict__ weight, const float* __restrict__ mean,
                   const float* __restrict__ rstd, TX* gx, int64_t ld_gx) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[64];
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const TX* gr = gy + t * ld_gy;
        const TX* xr = x + t * ld_x;
        const float mu = mean[t], r = rstd[t];
        float s[2] = {0.0f, 0.0f};
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float gn = to_f(gr[c]) * (weight ? weight[c] : 1.0f);
            s[0] += gn;
            s[1] = fmaf(gn, (to_f(xr[c]) - mu) * r, s[1]);
        }
        block_sum<2>(s, sh);
        const float a = s[0] / static_cast<float>(d), b = s[1] / static_cast<float>(d);
        TX* o = gx + t * ld_gx;
        for (int64_t c = threadIdx.x; c < d; c += kWideThreads) {
            const float gn = to_f(gr[c]) * (weight ? weight[c] : 1.0f);
            o[c] = from_f<TX>(r * (gn - a - (to_f(xr[c]) - mu) * r * b));
        }
    }
}

// ------------------------------------------------------------------ host

constexpr int kMaxResident = 1024;  // partial rows: no more CTAs than this run the backward

// CTAs that fill the current device; Kernel names the kernel that `kernel` is.
template <typename Kernel, typename K>
int resident(K kernel, int threads, int smem) {
    constexpr int kMaxDev = 64, kShapes = kMaxThreads / 32 + 1;
    static int cache[kMaxDev][kShapes] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lk(mu);
    int& n = cache[dev][threads / 32];
    if (n == 0) {
        int per = 0, sms = 0;
        if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        n = per * sms;
    }
    return n;
}

// How a width is laid out: warps per row, and threads per CTA for G lanes.
template <int G, int MULTI> int cta_threads(int warps) {
    return MULTI ? 32 * warps * std::max(1, 8 / warps) : kThreads;
}

struct NormArgs {
    const void *gy, *x;
    int64_t ld_gy, ld_x, T, d;
    const float *weight, *bias;
    float eps;
    void* out;  // y or gx
    int64_t ld_out;
    float *mean, *rstd, *part;
    int64_t* parts;
    cudaStream_t s;
};

template <typename TX, bool VEC, int G, int E, int MULTI>
struct Forward {
    static cudaError_t run(const NormArgs& a, int warps) {
        const int threads = cta_threads<G, MULTI>(warps);
        const int rows = threads / (MULTI ? 32 * warps : G);
        const int smem = kRing * threads * Layout<TX, VEC, E>::kBytes +
                         (E <= kOwnParams ? 0 : 2 * G * E * static_cast<int>(sizeof(float)));
        static const auto kernel = k_norm<TX, VEC, G, E, MULTI>;
        const int fill = resident<Forward>(kernel, threads, smem);
        if (fill <= 0) return cudaErrorUnknown;
        const int64_t blocks = std::min<int64_t>((a.T + rows - 1) / rows, fill);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads),
                          static_cast<size_t>(smem), a.s, static_cast<const TX*>(a.x), a.ld_x, a.T,
                          static_cast<int>(a.d), warps, a.weight, a.bias, a.eps, static_cast<TX*>(a.out), a.ld_out,
                          a.mean, a.rstd);
    }
};

template <typename TX, bool VEC, int G, int E, int MULTI>
struct Backward {
    static cudaError_t run(const NormArgs& a, int warps) {
        const int threads = cta_threads<G, MULTI>(warps);
        const int rows = threads / (MULTI ? 32 * warps : G);
        const int smem = threads * std::max(2 * kRing * Layout<TX, VEC, E>::kBytes,
                                            E * static_cast<int>(sizeof(float)));
        static const auto kernel = k_norm_grad<TX, VEC, G, E, MULTI>;
        const int fill = resident<Backward>(kernel, threads, smem);
        if (fill <= 0) return cudaErrorUnknown;
        const int64_t blocks =
            std::min<int64_t>({(a.T + rows - 1) / rows, fill, int64_t(kMaxResident)});
        *a.parts = blocks;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads),
                          static_cast<size_t>(smem), a.s, static_cast<const TX*>(a.gy), a.ld_gy,
                          static_cast<const TX*>(a.x), a.ld_x, a.T, static_cast<int>(a.d), warps,
                          a.weight, a.mean, a.rstd, static_cast<TX*>(a.out), a.ld_out,
                          a.part);
    }
};

// Lanes and values per lane for a width: the fewest that hold it, so that
// few lanes carry columns past d. Wide rows take as many warps as it needs.
template <typename TX, bool VEC>
cudaError_t forward_by_width(const NormArgs& a) {
    const int64_t d = a.d;
    if (d <= 64) return Forward<TX, VEC, 8, 8, 0>::run(a, 1);
    if (d <= 128) return Forward<TX, VEC, 16, 8, 0>::run(a, 1);
    if (d <= 256) return Forward<TX, VEC, 32, 8, 0>::run(a, 1);
    if (d <= 512) return Forward<TX, VEC, 32, 16, 0>::run(a, 1);
    if (d <= 768) return Forward<TX, VEC, 32, 24, 0>::run(a, 1);
    if (d <= 1024) return Forward<TX, VEC, 32, 32, 0>::run(a, 1);
    if constexpr (VEC && sizeof(TX) == 2) {
        if (d <= 1536) return Forward<TX, VEC, 32, 48, 0>::run(a, 1);
        if (d <= 2048) return Forward<TX, VEC, 32, 64, 0>::run(a, 1);
    }
    const int warps = static_cast<int>((d + 511) / 512);
    return warps <= 8 ? Forward<TX, VEC, 32, 16, 1>::run(a, warps)
                      : Forward<TX, VEC, 32, 16, 2>::run(a, warps);
}

template <typename TX, bool VEC>
cudaError_t backward_by_width(const NormArgs& a) {
    const int64_t d = a.d;
    if (d <= 64) return Backward<TX, VEC, 8, 8, 0>::run(a, 1);
    if (d <= 128) return Backward<TX, VEC, 16, 8, 0>::run(a, 1);
    if (d <= 256) return Backward<TX, VEC, 32, 8, 0>::run(a, 1);
    if (d <= 512) return Backward<TX, VEC, 32, 16, 0>::run(a, 1);
    const int warps = static_cast<int>((d + 511) / 512);
    return warps <= 8 ? Backward<TX, VEC, 32, 16, 1>::run(a, warps)
                      : Backward<TX, VEC, 32, 16, 2>::run(a, warps);
}

// Whether every row starts on 16 bytes and ends on them.
template <typename TX>
bool rows16(const void* p, int64_t ld, int64_t d) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(TX) % 16 == 0 &&
           d * sizeof(TX) % 16 == 0;
}

int64_t wide_chunk(int64_t T) { return std::max<int64_t>((T + kWideChunks - 1) / kWideChunks, 64); }

template <typename TX>
cudaError_t norm_typed(const NormArgs& a) {
    const TX* x = static_cast<const TX*>(a.x);
    const bool vec = rows16<TX>(a.x, a.ld_x, a.d) && rows16<TX>(a.out, a.ld_out, a.d);
    if (a.d > kMaxWidth)
        return launch_pdl(k_norm_wide<TX>,
                          dim3(static_cast<unsigned>(std::min<int64_t>(a.T, 152 * 4))),
                          dim3(kWideThreads), 0, a.s, x, a.ld_x, a.T, a.d, a.weight, a.bias, a.eps,
                          static_cast<TX*>(a.out), a.ld_out, a.mean, a.rstd);
    return vec ? forward_by_width<TX, true>(a) : forward_by_width<TX, false>(a);
}

template <typename TX>
cudaError_t grad_typed(const NormArgs& a, bool accumulate, float* gweight, float* gbias) {
    cudaError_t e = cudaSuccess;
    const bool vec = rows16<TX>(a.gy, a.ld_gy, a.d) && rows16<TX>(a.x, a.ld_x, a.d) &&
                     (!a.out || rows16<TX>(a.out, a.ld_out, a.d));
    if (a.d > kMaxWidth) {
        const TX* gy = static_cast<const TX*>(a.gy);
        const TX* x = static_cast<const TX*>(a.x);
        if (a.part) {  // before gx, which may overwrite gy
            const int64_t chunk = wide_chunk(a.T);
            *a.parts = (a.T + chunk - 1) / chunk;
            e = launch_pdl(k_norm_cols<TX>,
                           dim3(static_cast<unsigned>((a.d + 31) / 32),
                                static_cast<unsigned>(*a.parts)),
                           dim3(256), 0, a.s, gy, a.ld_gy, x, a.ld_x, a.T, a.d, a.mean, a.rstd,
                           chunk, a.part);
            if (e != cudaSuccess) return e;
        }
        if (a.out)
            e = launch_pdl(k_norm_gx_wide<TX>,
                           dim3(static_cast<unsigned>(std::min<int64_t>(a.T, 152 * 4))),
                           dim3(kWideThreads), 0, a.s, gy, a.ld_gy, x, a.ld_x, a.T, a.d, a.weight,
                           a.mean, a.rstd, static_cast<TX*>(a.out), a.ld_out);
    } else {
        e = vec ? backward_by_width<TX, true>(a) : backward_by_width<TX, false>(a);
    }
    if (e != cudaSuccess || !a.part) return e;
    return launch_pdl(k_norm_finish, dim3(static_cast<unsigned>((2 * a.d + 31) / 32)), dim3(1024),
                      0, a.s, a.part, *a.parts, a.d, accumulate ? 1 : 0, gweight, gbias);
}

}  // namespace

cudaError_t launch_layer_norm(const void* x, int bf16, int64_t ld_x, int64_t T, int64_t d,
                              const float* weight, const float* bias, float eps, void* y,
                              int64_t ld_y, float* mean, float* rstd, cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    NormArgs a = {};
    a.x = x;
    a.ld_x = ld_x;
    a.T = T;
    a.d = d;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.out = y;
    a.ld_out = ld_y;
    a.mean = mean;
    a.rstd = rstd;
    a.s = s;
    return bf16 ? norm_typed<__nv_bfloat16>(a) : norm_typed<float>(a);
}

size_t layer_norm_grad_workspace_bytes(int64_t T, int64_t d) {
    // Wide rows leave a partial row per chunk, no more than kWideChunks of them.
    const int64_t n = std::min<int64_t>(T, kMaxResident);
    return sizeof(float) * static_cast<size_t>(2 * n * d);
}

cudaError_t launch_layer_norm_grad(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x,
                                   int bf16, int64_t T, int64_t d, const float* weight,
                                   const float* mean, const float* rstd, bool accumulate, void* gx,
                                   int64_t ld_gx, float* gweight, float* gbias, float* part,
                                   cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    int64_t parts = 0;
    NormArgs a = {};
    a.gy = gy;
    a.ld_gy = ld_gy;
    a.x = x;
    a.ld_x = ld_x;
    a.T = T;
    a.d = d;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.out = gx;
    a.ld_out = ld_gx;
    a.part = gweight || gbias ? part : nullptr;
    a.parts = &parts;
    a.s = s;
    return bf16 ? grad_typed<__nv_bfloat16>(a, accumulate, gweight, gbias)
                : grad_typed<float>(a, accumulate, gweight, gbias);
}

}  // namespace dust
