// Layer norm, forward and backward. Per row of d values, n = (x - mean) rstd:
//     y  = n weight + bias
//     gx = rstd (gn - mean(gn) - n mean(gn n)),  gn = gy weight
//     gweight = sum_t gy n,  gbias = sum_t gy
// Bound by memory: the forward reads x and writes y once, the backward reads
// gy and x and writes gx once, whatever the width up to kMaxWidth.
//
// A row is held in registers by a group of G threads, E values each (G a power
// of two, the smallest with G E >= d): mean, then deviations, then the
// result, without a second read. A group goes over many rows, so weight and
// bias stay in registers too, and the next row's loads are in flight while
// this one is reduced and written. Rows that start on 16 bytes are read and
// written 16 bytes a thread; others value by value, neighbouring threads on
// neighbouring values.
//
// The backward adds its rows' gy n and gy per column in registers, the CTA's
// groups add theirs up in shared memory, and each CTA leaves one partial row;
// k_norm_finish sums the partial rows in order. No atomics: the result
// depends on T, d, the type and the alignment only.
//
// Wider rows (more than kMaxWidth values) are read once per pass by one CTA.
#include <algorithm>
#include <mutex>

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

constexpr int kMinThreads = 256;   // threads per CTA of narrow groups
constexpr int kValues = 8;         // E
constexpr int kRingRows = 4;         // rows in the ring of a group: one in use, the others in flight
constexpr int kMinF = 5, kMinB = 3;  // CTAs of 256 threads that an SM has registers for
constexpr int64_t kMaxWidth = 1024 * kValues;

// E values of one row, as loaded. VEC: 16 bytes at a time; value i of thread
// l is column ((i / per) G + l) per + i % per with per values in 16 bytes
// (per = 1 without VEC).
template <typename TX, bool VEC, int G, int E>
struct Held {
    static constexpr int kPer = VEC ? 16 / static_cast<int>(sizeof(TX)) : 1;
    static constexpr int kLoads = E / kPer;
    union {
        uint4 q[VEC ? kLoads : 1];
        TX x[E];
    };
    __device__ Held() {}

    static __device__ __forceinline__ int column(int l, int i) {
        return ((i / kPer) * G + l) * kPer + i % kPer;
    }
    // A thread's bytes of one row in its ring, 0 where rows go through registers.
    static constexpr bool kRing = VEC || sizeof(TX) == 4;
    static constexpr int kBytes = kRing ? E * static_cast<int>(sizeof(TX)) : 0;
    static constexpr int kPiece = VEC ? 16 : 4;

    __device__ __forceinline__ void load(const TX* row, int l, int d) {
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int c = (j * G + l) * kPer;
            x[j] = c < d ? row[c] : from_f<TX>(0.0f);
        }
    }
    // Starts the row's copy into this thread's slots (zeros past d, or of no
    // row at all); get() reads them once the copies have landed. A thread
    // reads what it copied itself, so no barrier is needed.
    static __device__ __forceinline__ void fetch(unsigned char* slot, const TX* row, bool any,
                                                 int l, int d) {
        const int threads = blockDim.x;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int c = (j * G + l) * kPer;
            const bool in = any && c < d;
            const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(slot)) +
                                (j * threads + threadIdx.x) * kPiece;
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
    __device__ __forceinline__ void get(const unsigned char* slot) {
        const int threads = blockDim.x;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const unsigned char* at = slot + (j * threads + threadIdx.x) * kPiece;
            if constexpr (VEC)
                q[j] = *reinterpret_cast<const uint4*>(at);
            else
                x[j] = *reinterpret_cast<const TX*>(at);
        }
    }
    __device__ __forceinline__ float at(int i) const { return to_f(x[i]); }
};

template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ void store_row(TX* row, int l, int d, const float (&v)[E]) {
    using H = Held<TX, VEC, G, E>;
#pragma unroll
    for (int j = 0; j < H::kLoads; ++j) {
        const int c = (j * G + l) * H::kPer;
        if (c >= d) continue;
        if constexpr (VEC) {
            union {
                uint4 q;
                TX x[H::kPer];
            } o;
#pragma unroll
            for (int k = 0; k < H::kPer; ++k) o.x[k] = from_f<TX>(v[j * H::kPer + k]);
            *reinterpret_cast<uint4*>(row + c) = o.q;
        } else {
            row[c] = from_f<TX>(v[j]);
        }
    }
}

// Sums of N values over a group, to all its threads. Groups of several warps
// meet in shared memory: `sh` has two slots, used in turn, so that one barrier
// per sum is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*sh)[N * 32], int& slot) {
#pragma unroll
    for (int off = (G < 32 ? G : 32) / 2; off > 0; off >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    if constexpr (G > 32) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) sh[slot][k * 32 + warp] = v[k];
        __syncthreads();
        const int first = warp / (G / 32) * (G / 32);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < G / 32; ++i) s += sh[slot][k * 32 + first + i];
            v[k] = s;
        }
        slot ^= 1;
    }
}

__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of copies of this thread have landed.
template <int N> __device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The backward's ring, two operands: as long as shared memory takes.
template <typename TX, int G> constexpr int ring_rows_grad() {
    return sizeof(TX) == 4 && G == 1024 ? 3 : kRingRows;
}

template <int G> constexpr int threads_of() { return G > kMinThreads ? G : kMinThreads; }

template <typename TX, bool VEC, int G>
__global__ void __launch_bounds__(threads_of<G>(), G > 256 ? 256 * kMinF / G : kMinF)
    k_norm(const TX* x, int64_t ld_x, int64_t T, int d, const float* __restrict__ weight,
           const float* __restrict__ bias, float eps, TX* y, int64_t ld_y, float* mean,
           float* rstd) {
    constexpr int E = kValues, kRows = threads_of<G>() / G;
    using H = Held<TX, VEC, G, E>;
    __shared__ float sh[2][32];
    extern __shared__ __align__(16) unsigned char ring[];
    constexpr int kSlot = threads_of<G>() * H::kBytes;
    int slot = 0;
    const int l = threadIdx.x % G, sub = threadIdx.x / G;
    float w[E], b[E];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = H::column(l, i);
        w[i] = c < d && weight ? weight[c] : 1.0f;
        b[i] = c < d && bias ? bias[c] : 0.0f;
    }
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows;
    H next;
    int at = 0;  // ring slot of the row in use
    if constexpr (H::kRing) {
#pragma unroll
        for (int k = 0; k < kRingRows - 1; ++k) {
            const int64_t t = t0 + sub + k * step;
            H::fetch(ring + k * kSlot, x + (t < T ? t : 0) * ld_x, t < T, l, d);
            copies_begun();
        }
    } else if (t0 + sub < T) {
        next.load(x + (t0 + sub) * ld_x, l, d);
    }
    for (; t0 < T; t0 += step) {  // every thread of the CTA as often
        const int64_t t = t0 + sub;
        H row;
        if constexpr (H::kRing) {
            const int64_t u = t + (kRingRows - 1) * step;
            const int to = at == 0 ? kRingRows - 1 : at - 1;
            H::fetch(ring + to * kSlot, x + (u < T ? u : 0) * ld_x, u < T, l, d);
            copies_begun();
            copies_landed<kRingRows - 1>();
            row.get(ring + at * kSlot);
            at = at + 1 == kRingRows ? 0 : at + 1;
        } else {
            row = next;
            if (t + step < T) next.load(x + (t + step) * ld_x, l, d);
        }
        float v[E];
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = row.at(i);
            if (t < T) s[0] += v[i];
        }
        group_sum<G, 1>(s, sh, slot);
        const float mu = s[0] * inv;
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] -= mu;
            if (H::column(l, i) < d) s[0] = fmaf(v[i], v[i], s[0]);
        }
        group_sum<G, 1>(s, sh, slot);
        const float r = 1.0f / sqrtf(fmaf(s[0], inv, eps));
        if (t >= T) continue;
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = fmaf(v[i] * r, w[i], b[i]);
        store_row<TX, VEC, G, E>(y + t * ld_y, l, d, v);
        if (l == 0) {
            if (mean) mean[t] = mu;
            if (rstd) rstd[t] = r;
        }
    }
}

template <typename TX, bool VEC, int G>
__global__ void __launch_bounds__(threads_of<G>(), 256 * kMinB > G ? (G > 256 ? 256 * kMinB / G : kMinB) : 1)
    k_norm_grad(const TX* gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x, int64_t T,
                int d, const float* __restrict__ weight, const float* __restrict__ mean,
                const float* __restrict__ rstd, TX* gx, int64_t ld_gx, float* __restrict__ part) {
    constexpr int E = kValues, kRows = threads_of<G>() / G, kAhead = ring_rows_grad<TX, G>();
    using H = Held<TX, VEC, G, E>;
    __shared__ float sh[2][64];
    __shared__ float cols[kRows > 1 ? 2 : 1][kRows > 1 ? threads_of<G>() * E : 1];
    extern __shared__ __align__(16) unsigned char ring[];
    constexpr int kSlot = threads_of<G>() * H::kBytes;
    int slot = 0;
    const int l = threadIdx.x % G, sub = threadIdx.x / G;
    float w[E], aw[E], ab[E];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = H::column(l, i);
        w[i] = c < d && weight ? weight[c] : 1.0f;
        aw[i] = ab[i] = 0.0f;
    }
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows;
    H next_g, next_x;
    float next_mu = 0.0f, next_r = 0.0f;
    int at = 0;
    const auto fetch = [&](int k, int64_t t) {
        const int64_t u = t < T ? t : 0;
        H::fetch(ring + 2 * k * kSlot, gy + u * ld_gy, t < T, l, d);
        H::fetch(ring + (2 * k + 1) * kSlot, x + u * ld_x, t < T, l, d);
        copies_begun();
    };
    const auto load = [&](int64_t t) {
        if (t >= T) return;
        if constexpr (!H::kRing) {
            next_g.load(gy + t * ld_gy, l, d);
            next_x.load(x + t * ld_x, l, d);
        }
        next_mu = mean[t];
        next_r = rstd[t];
    };
    if constexpr (H::kRing) {
#pragma unroll
        for (int k = 0; k < kAhead - 1; ++k) fetch(k, t0 + sub + k * step);
    }
    load(t0 + sub);
    for (; t0 < T; t0 += step) {
        const int64_t t = t0 + sub;
        H rg, rx;
        if constexpr (H::kRing) {
            fetch(at == 0 ? kAhead - 1 : at - 1, t + (kAhead - 1) * step);
            copies_landed<kAhead - 1>();
            rg.get(ring + 2 * at * kSlot);
            rx.get(ring + (2 * at + 1) * kSlot);
            at = at + 1 == kAhead ? 0 : at + 1;
        } else {
            rg = next_g;
            rx = next_x;
        }
        const float mu = next_mu, r = next_r;
        load(t + step);
        float g[E], n[E];
        float s[2] = {0.0f, 0.0f};
        if (t < T) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                // Columns past d hold zeros in both rows: n there is not, so
                // their gy, 0, has to come first in every product; a rstd or
                // mean that is not finite would not vanish.
                const bool in = H::column(l, i) < d;
                const float gv = rg.at(i);
                n[i] = in ? (rx.at(i) - mu) * r : 0.0f;
                aw[i] = fmaf(gv, n[i], aw[i]);
                ab[i] += gv;
                g[i] = gv * w[i];
                s[0] += g[i];
                s[1] = fmaf(g[i], n[i], s[1]);
            }
        }
        group_sum<G, 2>(s, sh, slot);
        if (t >= T || !gx) continue;
        const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
        for (int i = 0; i < E; ++i) g[i] = r * (g[i] - a - n[i] * b);
        store_row<TX, VEC, G, E>(gx + t * ld_gx, l, d, g);
    }
    if (!part) return;
    float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = H::column(l, i);
            if (c >= d) continue;
            out[c] = aw[i];
            out[d + c] = ab[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const int c = sub * G * E + H::column(l, i);
            cols[0][c] = aw[i];
            cols[1][c] = ab[i];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            float sw = 0.0f, sb = 0.0f;
            for (int k = 0; k < kRows; ++k) {
                sw += cols[0][k * G * E + c];
                sb += cols[1][k * G * E + c];
            }
            out[c] = sw;
            out[d + c] = sb;
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
#pragma unroll 4
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
    constexpr int kMaxDev = 64;
    static int cache[kMaxDev] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0) {
        int per = 0, sms = 0;
        if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), smem) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        cache[dev] = per * sms;
    }
    return cache[dev];
}

template <typename TX, bool VEC, int G>
struct Forward {
    static cudaError_t run(const void* x, int64_t ld_x, int64_t T, int64_t d, const float* weight,
                           const float* bias, float eps, void* y, int64_t ld_y, float* mean,
                           float* rstd, cudaStream_t s) {
        constexpr int threads = threads_of<G>(), rows = threads / G;
        constexpr int smem = kRingRows * threads * Held<TX, VEC, G, kValues>::kBytes;
        static const auto kernel = k_norm<TX, VEC, G>;
        const int fill = resident<Forward>(kernel, threads, smem);
        if (fill <= 0) return cudaErrorUnknown;
        const int64_t blocks = std::min<int64_t>((T + rows - 1) / rows, fill);
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, s,
                          static_cast<const TX*>(x), ld_x, T, static_cast<int>(d), weight, bias,
                          eps, static_cast<TX*>(y), ld_y, mean, rstd);
    }
};

template <typename TX, bool VEC, int G>
struct Backward {
    static cudaError_t run(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x, int64_t T,
                           int64_t d, const float* weight, const float* mean, const float* rstd,
                           void* gx, int64_t ld_gx, float* part, int64_t* parts, cudaStream_t s) {
        constexpr int threads = threads_of<G>(), rows = threads / G;
        constexpr int smem = 2 * ring_rows_grad<TX, G>() * threads * Held<TX, VEC, G, kValues>::kBytes;
        static const auto kernel = k_norm_grad<TX, VEC, G>;
        const int fill = resident<Backward>(kernel, threads, smem);
        if (fill <= 0) return cudaErrorUnknown;
        const int64_t blocks =
            std::min<int64_t>({(T + rows - 1) / rows, fill, int64_t(kMaxResident)});
        *parts = blocks;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), smem, s,
                          static_cast<const TX*>(gy), ld_gy, static_cast<const TX*>(x), ld_x, T,
                          static_cast<int>(d), weight, mean, rstd, static_cast<TX*>(gx), ld_gx,
                          part);
    }
};

// The group size for d at E values a thread.
template <template <typename, bool, int> class Op, typename TX, bool VEC, typename... Args>
cudaError_t by_width(int64_t d, int E, Args... args) {
    if (d <= 8 * E) return Op<TX, VEC, 8>::run(args...);
    if (d <= 16 * E) return Op<TX, VEC, 16>::run(args...);
    if (d <= 32 * E) return Op<TX, VEC, 32>::run(args...);
    if (d <= 64 * E) return Op<TX, VEC, 64>::run(args...);
    if (d <= 128 * E) return Op<TX, VEC, 128>::run(args...);
    if (d <= 256 * E) return Op<TX, VEC, 256>::run(args...);
    if (d <= 512 * E) return Op<TX, VEC, 512>::run(args...);
    return Op<TX, VEC, 1024>::run(args...);
}

// Whether every row starts on 16 bytes and ends on them.
template <typename TX>
bool rows16(const void* p, int64_t ld, int64_t d) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(TX) % 16 == 0 &&
           d * sizeof(TX) % 16 == 0;
}

int64_t wide_chunk(int64_t T) { return std::max<int64_t>((T + kWideChunks - 1) / kWideChunks, 64); }

template <typename TX>
cudaError_t norm_typed(const void* x, int64_t ld_x, int64_t T, int64_t d, const float* weight,
                       const float* bias, float eps, void* y, int64_t ld_y, float* mean,
                       float* rstd, cudaStream_t s) {
    if (d > kMaxWidth)
        return launch_pdl(k_norm_wide<TX>, dim3(static_cast<unsigned>(std::min<int64_t>(T, 152 * 4))),
                          dim3(kWideThreads), 0, s, static_cast<const TX*>(x), ld_x, T, d, weight,
                          bias, eps, static_cast<TX*>(y), ld_y, mean, rstd);
    if (rows16<TX>(x, ld_x, d) && rows16<TX>(y, ld_y, d))
        return by_width<Forward, TX, true>(d, kValues, x, ld_x, T, d, weight, bias, eps, y, ld_y,
                                           mean, rstd, s);
    return by_width<Forward, TX, false>(d, kValues, x, ld_x, T, d, weight, bias, eps, y, ld_y,
                                        mean, rstd, s);
}

template <typename TX>
cudaError_t grad_typed(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x, int64_t T,
                       int64_t d, const float* weight, const float* mean, const float* rstd,
                       bool accumulate, void* gx, int64_t ld_gx, float* gweight, float* gbias,
                       float* part, cudaStream_t s) {
    cudaError_t e;
    int64_t parts = 0;
    if (!gweight && !gbias) part = nullptr;
    if (d > kMaxWidth) {
        const TX* g = static_cast<const TX*>(gy);
        const TX* xx = static_cast<const TX*>(x);
        if (part) {  // before gx, which may overwrite gy
            const int64_t chunk = wide_chunk(T);
            parts = (T + chunk - 1) / chunk;
            e = launch_pdl(k_norm_cols<TX>,
                           dim3(static_cast<unsigned>((d + 31) / 32), static_cast<unsigned>(parts)),
                           dim3(256), 0, s, g, ld_gy, xx, ld_x, T, d, mean, rstd, chunk, part);
            if (e != cudaSuccess) return e;
        }
        if (gx) {
            e = launch_pdl(k_norm_gx_wide<TX>,
                           dim3(static_cast<unsigned>(std::min<int64_t>(T, 152 * 4))),
                           dim3(kWideThreads), 0, s, g, ld_gy, xx, ld_x, T, d, weight, mean, rstd,
                           static_cast<TX*>(gx), ld_gx);
            if (e != cudaSuccess) return e;
        }
    } else {
        const bool vec = rows16<TX>(gy, ld_gy, d) && rows16<TX>(x, ld_x, d) &&
                         (!gx || rows16<TX>(gx, ld_gx, d));
        e = vec ? by_width<Backward, TX, true>(d, kValues, gy, ld_gy, x, ld_x, T, d, weight,
                                               mean, rstd, gx, ld_gx, part, &parts, s)
                : by_width<Backward, TX, false>(d, kValues, gy, ld_gy, x, ld_x, T, d, weight,
                                                mean, rstd, gx, ld_gx, part, &parts, s);
        if (e != cudaSuccess) return e;
    }
    if (!part) return cudaSuccess;
    return launch_pdl(k_norm_finish, dim3(static_cast<unsigned>((2 * d + 31) / 32)), dim3(1024), 0,
                      s, part, parts, d, accumulate ? 1 : 0, gweight, gbias);
}

}  // namespace

cudaError_t launch_layer_norm(const void* x, int bf16, int64_t ld_x, int64_t T, int64_t d,
                              const float* weight, const float* bias, float eps, void* y,
                              int64_t ld_y, float* mean, float* rstd, cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    return bf16 ? norm_typed<__nv_bfloat16>(x, ld_x, T, d, weight, bias, eps, y, ld_y, mean, rstd, s)
                : norm_typed<float>(x, ld_x, T, d, weight, bias, eps, y, ld_y, mean, rstd, s);
}

size_t layer_norm_grad_workspace_bytes(int64_t T, int64_t d) {
    int64_t n = std::min<int64_t>(T, kMaxResident);
    if (d > kMaxWidth) {
        const int64_t chunk = wide_chunk(T);
        n = (T + chunk - 1) / chunk;
    }
    return sizeof(float) * static_cast<size_t>(2 * n * d);
}

cudaError_t launch_layer_norm_grad(const void* gy, int64_t ld_gy, const void* x, int64_t ld_x,
                                   int bf16, int64_t T, int64_t d, const float* weight,
                                   const float* mean, const float* rstd, bool accumulate, void* gx,
                                   int64_t ld_gx, float* gweight, float* gbias, float* part,
                                   cudaStream_t s) {
    ProfScope ps(kStageNorm, s);
    return bf16 ? grad_typed<__nv_bfloat16>(gy, ld_gy, x, ld_x, T, d, weight, mean, rstd,
                                            accumulate, gx, ld_gx, gweight, gbias, part, s)
                : grad_typed<float>(gy, ld_gy, x, ld_x, T, d, weight, mean, rstd, accumulate, gx,
                                    ld_gx, gweight, gbias, part, s);
}

}  // namespace dust
