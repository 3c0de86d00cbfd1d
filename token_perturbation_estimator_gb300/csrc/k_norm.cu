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
// Rows that start on 16 bytes are read and written 16 bytes a lane. Others are
// copied as they lie, from the 16 bytes that hold their first value on, and
// taken from shared memory value by value, neighbouring lanes on neighbouring
// values.
//
// The backward adds its rows' gy n and gy per column in registers, the CTA's
// warps add theirs up in shared memory, and each CTA leaves one partial row;
// k_norm_finish sums the partial rows in order. No atomics: the result
// depends on T, d, the type and the alignment only.
//
// Wider rows are read once per pass by one CTA.
//
// Measured: forward, 65536 x 2048 bf16, 94 us = 5.7 TB/s (0.85 of a copy's
// rate); backward, 65536 x 512 bf16, 37 us = 5.5 TB/s; backward, 9973 x 1531
// fp32, whose rows start on 4 bytes, 38 us = 4.8 TB/s.
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

// A thread's E values of a row: of the segment of G E columns that its warp (or
// part of a warp) holds, the whole row unless the row takes several warps.
// VEC: 16 bytes at a time, load j being the segment's columns [(j G + lane)
// per, + per); else single values, per = 1.
template <typename TX, bool VEC, int G, int E>
struct Layout {
    static constexpr int kSize = static_cast<int>(sizeof(TX));
    static constexpr int kPer = VEC ? 16 / kSize : 1;
    static constexpr int kLoads = E / kPer;
    // A segment's bytes in the ring: each thread's own places, or the
    // segment's image, with room for what shares its first 16 bytes.
    static constexpr int kBytes = G * E * kSize + (VEC ? 0 : 16);

    static __device__ __forceinline__ int column(int lane, int j) { return (j * G + lane) * kPer; }
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes)
                 : "memory");
}

// Starts the copy of a segment of n columns (or more: FULL) into its place in
// the ring. VEC: this thread's own values, zeros past the segment. Else 16
// bytes at a time from the 16 that hold its first value, as long as these do
// not start before the tensor (`base`); the few values before the next 16 are
// then copied one by one.
template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ void fetch_row(uint32_t slot, const TX* seg, const TX* base, int lane,
                                          int n) {
    using L = Layout<TX, VEC, G, E>;
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) {
            const int c = L::column(lane, j);
            const bool in = c < n;
            copy16(slot + (j * G + lane) * 16, in ? seg + c : base, in ? 16 : 0);
        }
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(seg);
        const int head = static_cast<int>(at & 15);
        const uintptr_t from = at - head;
        const int bytes = head + min(n, G * E) * L::kSize;
        const bool whole = from >= reinterpret_cast<uintptr_t>(base);
        constexpr int kTurns = E * L::kSize / 16 + 1;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int c = (i * G + lane) * 16;
            if (c < bytes && (c > 0 || whole))
                copy16(slot + c, reinterpret_cast<const void*>(from + c), min(16, bytes - c));
        }
        if (!whole && lane == 0) {
            const int k = min(n, (16 - head) / L::kSize);
            for (int i = 0; i < k; ++i) {
                const uint32_t to = slot + head + i * L::kSize;
                if constexpr (sizeof(TX) == 2)
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to),
                                 "h"(*reinterpret_cast<const uint16_t*>(seg + i))
                                 : "memory");
                else
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to),
                                 "r"(*reinterpret_cast<const uint32_t*>(seg + i))
                                 : "memory");
            }
        }
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

// A segment's values from its place in the ring (`head`: the low 4 bits of
// where it lay), zeros past its n columns.
template <typename TX, bool VEC, int G, int E, bool FULL>
__device__ __forceinline__ void get_row(float2 (&v)[E / 2], const unsigned char* slot, int head,
                                        int lane, int n) {
    using L = Layout<TX, VEC, G, E>;
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < L::kLoads; ++j) {
            const uint4 q = *reinterpret_cast<const uint4*>(slot + (j * G + lane) * 16);
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
        const TX* at = reinterpret_cast<const TX*>(slot + head) + lane;
#pragma unroll
        for (int j = 0; j < E; ++j) {
            float x = 0.0f;
            if (FULL || j * G + lane < n) x = to_f(at[j * G]);
            (j & 1 ? v[j / 2].y : v[j / 2].x) = x;
        }
    }
}

// Sets the values past the segment's n columns to 0.
template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ void clear_past(float2 (&v)[E / 2], int lane, int n) {
    using L = Layout<TX, VEC, G, E>;
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        if (L::column(lane, j) < n) continue;
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < L::kPer / 2; ++k) v[j * L::kPer / 2 + k] = make_float2(0.0f, 0.0f);
        } else {
            (j & 1 ? v[j / 2].y : v[j / 2].x) = 0.0f;
        }
    }
}

template <typename TX, bool VEC, int G, int E, bool FULL>
__device__ __forceinline__ void put_row(TX* seg, const float2 (&v)[E / 2], int lane, int n) {
    using L = Layout<TX, VEC, G, E>;
    TX* to = seg + lane * L::kPer;
#pragma unroll
    for (int j = 0; j < L::kLoads; ++j) {
        if (!FULL && L::column(lane, j) >= n) continue;
        if constexpr (VEC && sizeof(TX) == 2) {
            uint32_t q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[4 * j + k].x, v[4 * j + k].y);
                q[k] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(to + j * G * L::kPer) = make_uint4(q[0], q[1], q[2], q[3]);
        } else if constexpr (VEC) {
            *reinterpret_cast<float4*>(to + j * G * L::kPer) =
                make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
        } else {
            to[j * G] = from_f<TX>(j & 1 ? v[j / 2].y : v[j / 2].x);
        }
    }
}

// A parameter's values at this thread's columns (`none` where there is no
// parameter; p: at the segment's first): kept in registers, or (many values a
// lane) one copy per CTA in shared memory, laid out so that lanes read
// neighbouring 16 bytes.
template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ void own_param(float2 (&w)[E / 2], const float* p, float none, int lane,
                                          int n) {
    using L = Layout<TX, VEC, G, E>;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int c = L::column(lane, i / L::kPer) + i % L::kPer;
        (i & 1 ? w[i / 2].y : w[i / 2].x) = p && c < n ? p[c] : none;
    }
}
template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ void share_param(float* to, const float* p, float none, int d) {
    using L = Layout<TX, VEC, G, E>;
    constexpr int N = L::kPer < 4 ? L::kPer : 4;  // floats that a lane reads at once
    for (int i = threadIdx.x; i < G * E; i += blockDim.x) {
        // i = (chunk G + lane) N + k: the k-th of a lane's chunk-th N values
        const int k = i % N, lane = i / N % G, chunk = i / N / G;
        const int at = chunk * N + k;  // its place among the lane's values
        const int c = L::column(lane, at / L::kPer) + at % L::kPer;
        to[i] = p && c < d ? p[c] : none;
    }
}
template <typename TX, bool VEC, int G, int E>
__device__ __forceinline__ float2 shared_param(const float* at, int lane, int pair) {
    using L = Layout<TX, VEC, G, E>;
    if constexpr (L::kPer == 1) {
        return make_float2(at[2 * pair * G + lane], at[(2 * pair + 1) * G + lane]);
    } else {  // pairs 2 i and 2 i + 1 share 16 bytes: one load for both
        const float4 q = reinterpret_cast<const float4*>(at)[(pair / 2) * G + lane];
        return pair & 1 ? make_float2(q.z, q.w) : make_float2(q.x, q.y);
    }
}

// The threads that share a row meet: the lanes of a warp, or (MULTI) the
// row's own warps, so that a CTA's rows do not wait for one another. (bar.sync
// wants the lanes of a warp to arrive together.)
template <int MULTI>
__device__ __forceinline__ void row_sync(int warps) {
    __syncwarp();
    if constexpr (MULTI > 0)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x >> 5) / warps),
                     "r"(32 * warps)
                     : "memory");
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
        row_sync<MULTI>(warps);
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

// The launch bounds of the kernels below are what sets their registers: 80 a
// thread for the forward (two CTAs of 9-warp rows where 128 would leave one:
// 16384 x 4099 bf16, 148 -> 103 us), 128 for the backward, which spills below.

// Where a thread stands: its row among the CTA's, and its segment of it.
template <int G, int E, int MULTI>
struct Stand {
    int rows, sub, lane, seg, n;  // n: the segment's columns, G E or fewer
    bool full;
    __device__ Stand(int warps, int d) {
        const int warp = threadIdx.x >> 5;
        rows = MULTI ? (blockDim.x >> 5) / warps : blockDim.x / G;
        sub = MULTI ? warp / warps : threadIdx.x / G;
        lane = threadIdx.x % G;
        seg = MULTI ? (warp - sub * warps) * (G * E) : 0;
        n = d - seg;
        full = n >= G * E;
    }
};

template <typename TX, bool VEC, int G, int E, int MULTI>
__global__ void __launch_bounds__(MULTI == 2 ? 768 : kThreads, MULTI == 2 ? 1 : E > 32 ? 2 : 3)
    k_norm(const TX* x, int64_t ld_x, int64_t T, int d, int warps,
           const float* __restrict__ weight, const float* __restrict__ bias, float eps, TX* y,
           int64_t ld_y, float* mean, float* rstd) {
    using L = Layout<TX, VEC, G, E>;
    constexpr bool kOwn = E <= kOwnParams;
    static_assert(kOwn || MULTI == 0, "shared parameters are laid out for one warp per row");
    __shared__ float sh[2][16];
    extern __shared__ __align__(16) unsigned char ring[];
    int slot = 0;
    const Stand<G, E, MULTI> me(warps, d);
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * me.rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * me.rows;
    // The ring's slots are one after another, a segment's place in each.
    const int slot_bytes = static_cast<int>(blockDim.x) / G * L::kBytes;
    const unsigned char* mine = ring + threadIdx.x / G * L::kBytes;
    const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    const TX* cur = x + (first + me.sub) * ld_x + me.seg;  // this row, and the next to fetch
    const TX* from = cur;
    int64_t ahead = first + me.sub;
    const auto fetch = [&](int at) {
        if (ahead < T) fetch_row<TX, VEC, G, E>(mine_at + at * slot_bytes, from, x, me.lane, me.n);
        copies_begun();
        from += step * ld_x;
        ahead += step;
    };
    pdl_wait();
    pdl_trigger();
    fetch(0);
    fetch(1);
    float2 w[kOwn ? E / 2 : 1], b[kOwn ? E / 2 : 1];
    float* params = reinterpret_cast<float*>(ring + kRing * slot_bytes);  // past the ring
    if constexpr (kOwn) {
        own_param<TX, VEC, G, E>(w, weight ? weight + me.seg : nullptr, 1.0f, me.lane, me.n);
        own_param<TX, VEC, G, E>(b, bias ? bias + me.seg : nullptr, 0.0f, me.lane, me.n);
    } else {
        share_param<TX, VEC, G, E>(params, weight, 1.0f, d);
        share_param<TX, VEC, G, E>(params + G * E, bias, 0.0f, d);
        __syncthreads();
    }
    TX* to = y + (first + me.sub) * ld_y + me.seg;
    int at = 0;
    for (int64_t t0 = first; t0 < T; t0 += step, at ^= 1, to += step * ld_y, cur += step * ld_x) {
        const int64_t t = t0 + me.sub;  // every thread of the CTA goes as often
        float2 v[E / 2];
        copies_landed<kRing - 1>();
        if constexpr (!VEC) __syncwarp();  // the other lanes' copies too
        const int head = static_cast<int>(reinterpret_cast<uintptr_t>(cur) & 15);
        if (me.full)
            get_row<TX, VEC, G, E, true>(v, mine + at * slot_bytes, head, me.lane, me.n);
        else
            get_row<TX, VEC, G, E, false>(v, mine + at * slot_bytes, head, me.lane, me.n);
        float s[1] = {total<E>(v)};
        // The row has been read (its sum needs it): its place is free, an
        // image's after every lane's part of the sum.
        if constexpr (VEC) fetch(at);
        row_sum<G, MULTI, 1>(s, sh, slot, warps);
        if constexpr (!VEC) fetch(at);
        const float mu = s[0] * inv;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) v[i] = add2(v[i], both(-mu));
        if (!me.full) clear_past<TX, VEC, G, E>(v, me.lane, me.n);
        float2 q[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
        for (int i = 0; i < E / 2; ++i) q[i & 1] = fma2(v[i], v[i], q[i & 1]);
        q[0] = add2(q[0], q[1]);
        s[0] = q[0].x + q[0].y;
        row_sum<G, MULTI, 1>(s, sh, slot, warps);
        const float r = 1.0f / sqrtf(fmaf(s[0], inv, eps));
        if (t >= T) continue;
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            float2 wi, bi;
            if constexpr (kOwn) {
                wi = w[i];
                bi = b[i];
            } else {
                wi = shared_param<TX, VEC, G, E>(params, me.lane, i);
                bi = shared_param<TX, VEC, G, E>(params + G * E, me.lane, i);
            }
            v[i] = fma2(mul2(v[i], both(r)), wi, bi);
        }
        if (me.full)
            put_row<TX, VEC, G, E, true>(to, v, me.lane, me.n);
        else
            put_row<TX, VEC, G, E, false>(to, v, me.lane, me.n);
        if (me.lane == 0 && me.seg == 0) {
            if (mean) mean[t] = mu;
            if (rstd) rstd[t] = r;
        }
    }
}

template <typename TX, bool VEC, int G, int E, int MULTI>
__global__ void __launch_bounds__(MULTI == 2 ? kMaxThreads : kThreads, MULTI == 2 ? 1 : 2)
    k_norm_grad(const TX* gy, int64_t ld_gy, const TX* __restrict__ x, int64_t ld_x, int64_t T,
                int d, int warps, const float* __restrict__ weight,
                const float* __restrict__ mean, const float* __restrict__ rstd, TX* gx,
                int64_t ld_gx, float* __restrict__ part) {
    using L = Layout<TX, VEC, G, E>;
    __shared__ float sh[2][32];
    // The ring; then, for one sum at a time, floats [rows of the CTA][columns].
    extern __shared__ __align__(16) unsigned char ring[];
    int slot = 0;
    const Stand<G, E, MULTI> me(warps, d);
    const float inv = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * me.rows;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * me.rows;
    const int slot_bytes = static_cast<int>(blockDim.x) / G * L::kBytes;
    const unsigned char* mine = ring + threadIdx.x / G * L::kBytes;
    const uint32_t mine_at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
    const TX* cur_g = gy + (first + me.sub) * ld_gy + me.seg;  // these rows, and the next to fetch
    const TX* cur_x = x + (first + me.sub) * ld_x + me.seg;
    const TX *from_g = cur_g, *from_x = cur_x;
    int64_t ahead = first + me.sub;
    const auto fetch = [&](int at) {
        if (ahead < T) {
            fetch_row<TX, VEC, G, E>(mine_at + 2 * at * slot_bytes, from_g, gy, me.lane, me.n);
            fetch_row<TX, VEC, G, E>(mine_at + (2 * at + 1) * slot_bytes, from_x, x, me.lane, me.n);
        }
        copies_begun();
        from_g += step * ld_gy;
        from_x += step * ld_x;
        ahead += step;
    };
    pdl_wait();
    pdl_trigger();
    fetch(0);
    fetch(1);
    float2 w[E / 2], aw[E / 2], ab[E / 2];
    own_param<TX, VEC, G, E>(w, weight ? weight + me.seg : nullptr, 1.0f, me.lane, me.n);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) aw[i] = ab[i] = make_float2(0.0f, 0.0f);
    float next_mu = 0.0f, next_r = 0.0f;
    if (first + me.sub < T) {
        next_mu = mean[first + me.sub];
        next_r = rstd[first + me.sub];
    }
    TX* to = gx + (first + me.sub) * ld_gx + me.seg;
    int at = 0;
    for (int64_t t0 = first; t0 < T; t0 += step, at ^= 1, to += step * ld_gx,
                 cur_g += step * ld_gy, cur_x += step * ld_x) {
        const int64_t t = t0 + me.sub;
        const bool in = t < T;
        const float mu = next_mu, r = next_r;
        if (t + step < T) {
            next_mu = mean[t + step];
            next_r = rstd[t + step];
        }
        float s[2] = {0.0f, 0.0f};
        float2 gn[E / 2], n[E / 2];
        copies_landed<kRing - 1>();
        if constexpr (!VEC) __syncwarp();
        const int head_g = static_cast<int>(reinterpret_cast<uintptr_t>(cur_g) & 15);
        const int head_x = static_cast<int>(reinterpret_cast<uintptr_t>(cur_x) & 15);
        const unsigned char* at_g = mine + 2 * at * slot_bytes;
        if (me.full) {
            get_row<TX, VEC, G, E, true>(gn, at_g, head_g, me.lane, me.n);
            get_row<TX, VEC, G, E, true>(n, at_g + slot_bytes, head_x, me.lane, me.n);
        } else {
            get_row<TX, VEC, G, E, false>(gn, at_g, head_g, me.lane, me.n);
            get_row<TX, VEC, G, E, false>(n, at_g + slot_bytes, head_x, me.lane, me.n);
        }
        if (in) {
#pragma unroll
            for (int i = 0; i < E / 2; ++i) n[i] = mul2(add2(n[i], both(-mu)), both(r));
            if (!me.full) clear_past<TX, VEC, G, E>(n, me.lane, me.n);  // gy is 0 there
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
        if constexpr (VEC) fetch(at);
        row_sum<G, MULTI, 2>(s, sh, slot, warps);
        if constexpr (!VEC) fetch(at);
        if (!in || !gx) continue;
        const float a = s[0] * inv, b = s[1] * inv;
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            gn[i] = mul2(fma2(n[i], both(-b), add2(gn[i], both(-a))), both(r));
        if (me.full)
            put_row<TX, VEC, G, E, true>(to, gn, me.lane, me.n);
        else
            put_row<TX, VEC, G, E, false>(to, gn, me.lane, me.n);
    }
    if (!part) return;
    copies_landed<0>();  // the ring is about to hold the sums
    float* cols = reinterpret_cast<float*>(ring);
    const int width = (MULTI ? warps : 1) * G * E;
    float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += d) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float2 p = which ? ab[i / 2] : aw[i / 2];
            cols[me.sub * width + me.seg + L::column(me.lane, i / L::kPer) + i % L::kPer] =
                i & 1 ? p.y : p.x;
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d; c += blockDim.x) {
            float v = 0.0f;
            for (int i = 0; i < me.rows; ++i) v += cols[i * width + c];
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

// CTAs that fill the current device; Kernel names the kernel that `kernel` is,
// `threads` tells its `smem`.
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
        const int smem = kRing * (threads / G) * Layout<TX, VEC, G, E>::kBytes +
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
        const int smem = std::max(2 * kRing * (threads / G) * Layout<TX, VEC, G, E>::kBytes,
                                  threads * E * static_cast<int>(sizeof(float)));
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
    if constexpr (sizeof(TX) == 2) {
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
