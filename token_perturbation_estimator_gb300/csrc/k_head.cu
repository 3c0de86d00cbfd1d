// The head's per-token losses and their gradients, over the vocabulary in
// pieces and without keeping the logits (include/dust.h gives the formulas):
// softmax cross entropy against a target id, and distillation from a
// teacher's largest logits. The products are k_head_tc.cu's.
//
// Loss (of more than a few rows, which k_head_few.cu takes): one launch forms the logits tile by tile and leaves per row a partial
// maximum and sum for every half tile, and the target's logit; a second one
// joins them. For distillation the pass over the tiles also picks the logits
// of the teacher's entries, which a first launch has put in order. (Formed
// apart, as products of a row of H with K rows of E, they took 74 us beside
// the 183 us of the logits, 4096 rows, d 1024, V 32768, K 64.)
//
// Gradient, per piece of the vocabulary (a piece's G stays below 2^27
// values): the logits again as G = weight (exp(x - lse) - wanted) in bf16,
// then gH += G E and gE = G^T H in one launch. Rows that take no part (no
// target, no weight) are left out of all products: the others' H rows are
// moved together first if there are such rows.
//
// fp32 inputs, and bf16 ones whose rows do not start on 16 bytes, are first
// copied into the workspace, as three bf16 planes or padded rows.
#include <algorithm>
#include <cmath>

#include "head.cuh"

namespace dust {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The same shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ int2 read_at_rank(const int2* p, int rank) {
    uint32_t at;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void report_id(unsigned int* status) {
    atomicExch(status, 1u /* DUST_ERR_INVALID_ARG */);
}

// ------------------------------------------------------------------ loss

constexpr int kJoinLanes = 32;  // threads that share a row's partial sums, at most

// A row's partial sums joined, and its cross entropy. The threads of a row (8
// to 32, one per warp) each take every so manieth partial; theirs are joined
// in order.
__global__ void __launch_bounds__(32 * kJoinLanes)
    k_head_join(const HeadPart* __restrict__ part, int64_t ld, int n_part, int64_t R, int64_t T,
                const int32_t* __restrict__ targets, int64_t V,
                const float* __restrict__ picked, float* loss, float* lse, unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    __shared__ HeadPart sh[kJoinLanes][32];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, lanes = blockDim.x >> 5;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + lane;
    float m = -INFINITY, s = 0.0f;
    const auto join = [&](const HeadPart& p) {
        const float nm = fmaxf(m, p.m);
        // An empty partial has m = -inf and s = 0. NaN sums pass through.
        const float base = nm == -INFINITY ? 0.0f : nm;
        s = s * exp2f(m - base) + p.s * exp2f(p.m - base);
        m = nm;
    };
    if (r < R)
#pragma unroll 4
        for (int i = k; i < n_part; i += lanes) join(part[i * ld + r]);
    sh[k][lane] = {m, s};
    __syncthreads();
    if (k != 0 || r >= R) return;
    for (int i = 1; i < lanes; ++i) join(sh[i][lane]);
    // m is a whole number of powers of two; one rounding for each result.
    const double l = static_cast<double>(m) * 0.69314718055994530942 +
                     static_cast<double>(logf(s));
    lse[r] = static_cast<float>(l);
    if (!targets) return;
    const int64_t id = targets[r % T];
    const bool has = id >= 0 && id < V;
    if (id >= V) report_id(status);
    if (loss) loss[r] = has ? static_cast<float>(l - static_cast<double>(picked[r])) : 0.0f;
}

// A token's entries in order of their ids, for the loss's pass over the
// columns to pick their logits on its way: a warp per token sorts them (a
// bitonic network in shared memory), writes them out, and looks up where each
// half tile's first one is. Entries that are absent come last and are not
// counted; their logits are written here, 0.
__global__ void __launch_bounds__(256)
    k_head_bins(int64_t S, int64_t T, const int32_t* __restrict__ ids, int K, int size, int64_t V,
                int columns, int bins, int2* __restrict__ entries, uint16_t* __restrict__ starts,
                float* __restrict__ student, unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t bins_smem[];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5);
    if (t >= T) return;
    uint32_t* id = bins_smem + (threadIdx.x >> 5) * 2 * size;  // size: K or more, a power of two
    uint32_t* place = id + size;
    int n = 0;
    bool bad = false;
    for (int j = lane; j < size; j += 32) {
        const int32_t v = j < K ? ids[t * K + j] : -1;
        const bool in = v >= 0 && v < V;
        bad |= v >= V;
        id[j] = in ? static_cast<uint32_t>(v) : 0xffffffffu;
        place[j] = static_cast<uint32_t>(j);
        n += __popc(__ballot_sync(0xffffffffu, in));
        if (j < K && !in)
            for (int64_t s = 0; s < S; ++s) student[(s * T + t) * K + j] = 0.0f;
    }
    if (bad) report_id(status);
    __syncwarp();
    for (int k = 2; k <= size; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = lane; i < size / 2; i += 32) {
                const int p = 2 * i - (i & (j - 1)), q = p + j;  // bit j of p is 0
                const bool rising = (p & k) == 0;
                // The place breaks ties: the order is the same every time.
                const bool over = id[p] > id[q] || (id[p] == id[q] && place[p] > place[q]);
                if (over == rising) {
                    const uint32_t u = id[p], v = place[p];
                    id[p] = id[q];
                    place[p] = place[q];
                    id[q] = u;
                    place[q] = v;
                }
            }
            __syncwarp();
        }
    }
    for (int j = lane; j < n; j += 32)
        entries[t * K + j] = make_int2(static_cast<int>(id[j]), static_cast<int>(place[j]));
    for (int b = lane; b <= bins; b += 32) {
        const uint32_t from = static_cast<uint32_t>(b) * static_cast<uint32_t>(columns);
        int lo = 0, hi = n;  // the first entry at or past `from`
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (id[mid] < from) lo = mid + 1;
            else hi = mid;
        }
        starts[t * (bins + 1) + b] = static_cast<uint16_t>(lo);
    }
}

// The teacher of a token over its entries present: the largest scaled logit
// and the logarithm of the sum of exponentials over it; largest -inf where no
// entry has any probability. Whole warp.
__device__ __forceinline__ float2 teacher_stats(const int32_t* ids, const float* z, int64_t K,
                                                int64_t V, float scale, unsigned int* status) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    bool bad = false;
    for (int64_t j = lane; j < K; j += 32) {
        const int32_t id = ids[j];
        bad |= id >= V;
        if (id >= 0 && id < V) m = fmaxf(m, scale * z[j]);
    }
    if (bad && status) report_id(status);
    m = warp_max(m);
    float q = 0.0f;
    for (int64_t j = lane; j < K; j += 32) {
        const int32_t id = ids[j];
        if (m != -INFINITY && id >= 0 && id < V) q += expf(scale * z[j] - m);
    }
    q = warp_sum(q);
    return make_float2(m, logf(q));
}

__global__ void __launch_bounds__(256)
    k_head_distill(int64_t R, int64_t T, HeadTargets tg, int64_t V, float scale,
                   const float* __restrict__ lse, const float* __restrict__ student,
                   float* __restrict__ loss) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (r >= R) return;
    const int64_t t = r % T;
    const int32_t* ids = tg.ids + t * tg.K;
    const float* z = tg.teacher + t * tg.K;
    const float2 st = teacher_stats(ids, z, tg.K, V, scale, nullptr);
    const float l = lse[r];
    float a = 0.0f;
    for (int64_t j = lane; j < tg.K; j += 32) {
        const int32_t id = ids[j];
        if (st.x == -INFINITY || id < 0 || id >= V) continue;
        const float lq = scale * z[j] - st.x - st.y;
        const float q = expf(lq);
        // q = 0 adds nothing, whatever its logarithm.
        if (q != 0.0f) a = fmaf(q, lq - (student[r * tg.K + j] - l), a);
    }
    a = warp_sum(a);
    if (lane == 0) loss[r] = a;
}

__global__ void __launch_bounds__(256)
    k_head_changes(const float* __restrict__ loss, int64_t T, int64_t n, float* delta) {
    pdl_wait();
    pdl_trigger();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < n) delta[i] = loss[T + i] - loss[i % T];
}

// -------------------------------------------------------------- gradients

__global__ void __launch_bounds__(256)
    k_head_teacher(int64_t T, HeadTargets tg, int64_t V, float scale, float2* __restrict__ stats,
                   unsigned int* status) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= T) return;
    const float2 st = teacher_stats(tg.ids + t * tg.K, tg.teacher + t * tg.K, tg.K, V, scale,
                                    status);
    if ((threadIdx.x & 31) == 0) stats[t] = st;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634074 - 1.4426950408889634f);

// The rows that take part, in order: k_head_live writes which they are, their
// places (or -1), and what the factor needs of each; and the largest |gloss|.
// One cluster of eight CTAs: CTA c takes the c-th part of the rows, 1024 at a
// time, twice: counting, then, with the counts of the CTAs before it (read
// through the cluster's shared memory), writing.
constexpr int kLiveCtas = 8, kLiveThreads = 1024;

struct LiveRows {
    int32_t R, T;              // rows, tokens
    int64_t V;
    const int32_t* targets;    // or null
    const float2* teacher;
    const float* gloss;

    // Whether row r takes part; its target and weight.
    __device__ __forceinline__ bool wanted(int64_t r, int32_t& id, float& g) const {
        id = -1;
        g = 0.0f;
        if (r >= R) return false;
        const uint32_t t = R == T ? static_cast<uint32_t>(r)
                                  : static_cast<uint32_t>(r) % static_cast<uint32_t>(T);
        g = gloss[r];
        if (!targets) return teacher[t].x != -INFINITY && g != 0.0f;
        id = targets[t];
        return id >= 0 && id < V && g != 0.0f;
    }
};

__global__ void __cluster_dims__(kLiveCtas, 1, 1) __launch_bounds__(kLiveThreads, 1)
    k_head_live(LiveRows a, const float* __restrict__ lse, HeadCounts* counts,
                HeadRow* __restrict__ rows, int32_t* __restrict__ row_of,
                int32_t* __restrict__ place, unsigned int* status) {
    __shared__ int s_n[32];
    __shared__ float s_g[32];
    __shared__ int2 s_cta;  // this CTA's rows that take part; bits of its largest |gloss|
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, cta = blockIdx.x;
    // Parts of whole thousands of rows, each warp's rows in one run of it.
    const int32_t per = (a.R + kLiveCtas * kLiveThreads - 1) / (kLiveCtas * kLiveThreads);
    const int64_t r0 = (static_cast<int64_t>(cta) * kLiveThreads + w * 32) * per;
    int n = 0;
    float g = 0.0f;
    bool bad = false;
#pragma unroll 4
    for (int32_t i = 0; i < per; ++i) {
        int32_t id;
        float gl;
        const bool live = a.wanted(r0 + i * 32 + lane, id, gl);
        bad |= id >= a.V;
        if (live) g = fmaxf(g, fabsf(gl));  // NaN is passed over
        n += __popc(__ballot_sync(0xffffffffu, live));
    }
    if (bad) report_id(status);
    g = warp_max(g);
    if (lane == 0) {
        s_n[w] = n;
        s_g[w] = g;
    }
    __syncthreads();
    int at = __reduce_add_sync(0xffffffffu, lane < w ? s_n[lane] : 0);
    if (w == 0) {
        const int all = __reduce_add_sync(0xffffffffu, s_n[lane]);
        g = warp_max(s_g[lane]);
        if (lane == 0) s_cta = make_int2(all, __float_as_int(g));
    }
    cluster_barrier();
    int all = 0;
    g = 0.0f;
#pragma unroll
    for (int c = 0; c < kLiveCtas; ++c) {
        const int2 o = read_at_rank(&s_cta, c);
        if (c < cta) at += o.x;
        all += o.x;
        g = fmaxf(g, __int_as_float(o.y));
    }
    cluster_barrier();  // nobody leaves before its counts are read
    if (!(g > 0.0f) || g == INFINITY) g = 1.0f;
    if (cta == 0 && threadIdx.x == 0) *counts = {all, g};
#pragma unroll 4
    for (int32_t i = 0; i < per; ++i) {
        const int64_t r = r0 + i * 32 + lane;
        int32_t id;
        float gl;
        const bool live = a.wanted(r, id, gl);
        const unsigned int mask = __ballot_sync(0xffffffffu, live);
        const int to = at + __popc(mask & ((1u << lane) - 1u));
        at += __popc(mask);
        if (r >= a.R) continue;
        place[r] = live ? to : -1;
        if (!live) continue;
        const float l = lse[r];
        HeadRow h;
        h.lse_hi = l * kLog2e;
        h.lse_lo = fmaf(l, kLog2e, -h.lse_hi) + l * kLog2eRest;
        h.weight = gl / g;
        h.target = id;
        rows[to] = h;
        row_of[to] = static_cast<int32_t>(r);
    }
}

// Rows into the workspace as bf16 (one plane) or as three bf16 planes, zero
// from column d to dp. With counts, row i is the i-th that takes part, rows
// up to the next multiple of 64 are zeroed, and rows of `zero` (gH) that take
// no part are cleared; if all take part and `only_if_some` is set there is
// nothing to do.
template <typename TX, int PLANES>
__global__ void __launch_bounds__(256)
    k_head_pack(const TX* __restrict__ src, int64_t ld, int64_t n, int64_t d, int64_t dp, int vec,
                __nv_bfloat16* __restrict__ dst, const HeadCounts* counts,
                const int32_t* __restrict__ row_of, int only_if_some,
                const int32_t* __restrict__ place, TX* zero, int64_t ld_zero) {
    pdl_wait();
    pdl_trigger();
    const int64_t live = counts ? counts->rows : n;
    if (only_if_some && live == n) return;
    int64_t end = n;
    if (counts) {
        end = (live + 63) / 64 * 64;
        if (end > n) end = n;
    }
    const int lane = threadIdx.x & 31;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < n;
         i += static_cast<int64_t>(gridDim.x) * 8) {
        if (zero && place[i] < 0)
            for (int64_t c = lane; c < d; c += 32) zero[i * ld_zero + c] = TX(0.0f);
        if (i >= end || !dst) continue;
        const TX* s = i < live ? src + (row_of ? row_of[i] : i) * ld : nullptr;
        __nv_bfloat16* o = dst + i * dp;
        for (int64_t c = lane * 8; c < dp; c += 256) {
            float v[8];
            if (s && vec && c + 8 <= d) {
#pragma unroll
                for (int u = 0; u < static_cast<int>(sizeof(TX)) / 2; ++u) {
                    const uint4 x = reinterpret_cast<const uint4*>(s + c)[u];
                    const TX* xs = reinterpret_cast<const TX*>(&x);
                    constexpr int per = 16 / sizeof(TX);
#pragma unroll
                    for (int k = 0; k < per; ++k) v[u * per + k] = to_f(xs[k]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = s && c + k < d ? to_f(s[c + k]) : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                __nv_bfloat16 b[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    b[k] = __float2bfloat16_rn(v[k]);
                    // What this plane leaves (nothing of an infinity).
                    v[k] = __builtin_isinf(v[k]) ? 0.0f : v[k] - __bfloat162float(b[k]);
                }
                *reinterpret_cast<uint4*>(o + p * n * dp + c) = *reinterpret_cast<const uint4*>(b);
            }
        }
    }
}

// Distillation: G at the teacher's entries of a piece, weight (exp(x - lse) -
// q), with q summed over the entries of the same id. A warp per row; the
// row's ids and probabilities in shared memory.
template <int PLANES>
__global__ void __launch_bounds__(256)
    k_head_patch(const HeadCounts* __restrict__ counts, const HeadRow* __restrict__ rows,
                 const int32_t* __restrict__ row_of, int64_t T, HeadTargets tg, float scale,
                 const float2* __restrict__ teacher, const float* __restrict__ student, int64_t v0,
                 int64_t n, __nv_bfloat16* __restrict__ G, int64_t ld_g, int64_t plane) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ unsigned char patch_smem[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int K = static_cast<int>(tg.K);
    int32_t* s_id = reinterpret_cast<int32_t*>(patch_smem) + w * 2 * K;
    float* s_q = reinterpret_cast<float*>(s_id + K);
    const int live = counts->rows;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * warps + w; i < live;
         i += static_cast<int64_t>(gridDim.x) * warps) {
        const int64_t r = row_of[i], t = r % T;
        const float2 st = teacher[t];
        const HeadRow h = rows[i];
        __syncwarp();
        for (int j = lane; j < K; j += 32) {
            const int64_t id = tg.ids[t * K + j];
            const bool in = id >= v0 && id < v0 + n;
            s_id[j] = in ? static_cast<int32_t>(id - v0) : -1;
            s_q[j] = in ? expf(scale * tg.teacher[t * K + j] - st.x - st.y) : 0.0f;
        }
        __syncwarp();
        for (int j = lane; j < K; j += 32) {
            const int32_t id = s_id[j];
            if (id < 0) continue;
            float q = 0.0f;
            bool first = true;
            for (int u = 0; u < K; ++u) {
                if (s_id[u] != id) continue;
                first = first && u >= j;
                q += s_q[u];
            }
            if (!first) continue;
            const float x = student[r * K + j];
            const float p = exp2f(fmaf(x, kLog2e, -h.lse_hi) - h.lse_lo + x * kLog2eRest);
            float g = h.weight * (p - q);
            __nv_bfloat16* o = G + i * ld_g + id;
#pragma unroll
            for (int u = 0; u < PLANES; ++u) {
                const __nv_bfloat16 b = __float2bfloat16_rn(g);
                o[u * plane] = b;
                g -= __bfloat162float(b);
            }
        }
    }
}

// ------------------------------------------------------------------ host

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t up(int64_t x, int64_t by) { return (x + by - 1) / by * by; }

// Whether TMA can read the rows where they lie.
bool direct(const void* p, int64_t ld, bool bf16) {
    return bf16 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// Vocabulary rows of a piece: whole tiles, G at most 2^27 values over its
// planes (256 MB), so that a large vocabulary's G is never whole.
int64_t piece_of(int64_t R, int64_t V, int planes) {
    const int64_t cap = (int64_t(1) << 27) / (up(R, kHeadTile) * planes);
    const int64_t whole = up(V, kHeadTile);
    int64_t n = std::min(whole, std::max<int64_t>(cap / kHeadTile * kHeadTile, 4 * kHeadTile));
    // Pieces of about one size.
    const int64_t pieces = (whole + n - 1) / n;
    return up((whole + pieces - 1) / pieces, kHeadTile);
}

struct Carver {
    unsigned char* base;
    size_t at = 0;
    template <typename T> T* take(int64_t n) {
        T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
        at += a256(sizeof(T) * static_cast<size_t>(n));
        return p;
    }
};

struct LossSpace {
    int2* entries;
    uint16_t* starts;
    __nv_bfloat16 *h, *e;
    HeadPart* part;
    float *picked, *loss;
    size_t total;
};

// Partial sums per row.
int loss_parts(const HeadProblem& p) {
    if (head_few(p)) return head_few_parts(p);
    const int64_t bn = head_loss_columns(p.S * p.T, p.V);
    return static_cast<int>(2 * ((p.V + bn - 1) / bn));
}

// H and E are sized as if copied, wherever they lie: the size must not
// depend on addresses. Only what a call needs is touched.
LossSpace carve_loss(void* ws, const HeadProblem& p) {
    const int64_t R = p.S * p.T, dp = up(p.d, 8), planes = p.bf16 ? 1 : 3;
    const int64_t parts = loss_parts(p);
    const bool tiles = !head_few(p);
    Carver c{static_cast<unsigned char*>(ws)};
    LossSpace w;
    w.part = c.take<HeadPart>(parts * up(R, 32));
    w.picked = c.take<float>(R);
    const bool picks = p.tg.many && tiles;
    w.entries = c.take<int2>(picks ? p.T * p.tg.K : 0);
    w.starts = c.take<uint16_t>(picks ? p.T * (parts + 1) : 0);
    w.loss = c.take<float>(R);
    w.h = c.take<__nv_bfloat16>(tiles ? planes * R * dp : 0);
    w.e = c.take<__nv_bfloat16>(tiles ? planes * p.V * dp : 0);
    w.total = c.at;
    return w;
}

struct GradSpace {
    HeadCounts* counts;
    HeadRow* rows;
    int32_t *row_of, *place;
    float2* teacher;
    __nv_bfloat16 *h, *e, *g;
    float *gh_acc, *ge_acc;
    HeadCuts cuts;
    int64_t piece;
    size_t total;
};

GradSpace carve_grad(void* ws, const HeadProblem& p) {
    const int64_t R = p.S * p.T, dp = up(p.d, 8), planes = p.bf16 ? 1 : 3;
    Carver c{static_cast<unsigned char*>(ws)};
    GradSpace w;
    w.piece = piece_of(R, p.V, static_cast<int>(planes));
    w.counts = c.take<HeadCounts>(1);
    w.rows = c.take<HeadRow>(R);
    w.row_of = c.take<int32_t>(R);
    w.place = c.take<int32_t>(R);
    w.teacher = c.take<float2>(p.T);
    // As for both gradients, whichever are asked for.
    w.cuts = head_cuts(R, std::min(w.piece, p.V), p.d, static_cast<int>(planes));
    w.gh_acc = c.take<float>(w.piece < p.V || w.cuts.gh > 1 ? head_acc_floats(R, p.d, w.cuts.gh) : 0);
    w.ge_acc = c.take<float>(w.cuts.ge > 1 ? head_acc_floats(w.piece, p.d, w.cuts.ge) : 0);
    w.g = c.take<__nv_bfloat16>(planes * up(R, kHeadTile) * w.piece);
    w.h = c.take<__nv_bfloat16>(planes * R * dp);
    w.e = c.take<__nv_bfloat16>(planes * p.V * dp);
    w.total = c.at;
    return w;
}

template <typename TX>
cudaError_t pack(const void* src, int64_t ld, int64_t n, int64_t d, __nv_bfloat16* dst,
                 const HeadCounts* counts, const int32_t* row_of, bool only_if_some,
                 const int32_t* place, void* zero, int64_t ld_zero, cudaStream_t s) {
    constexpr int P = sizeof(TX) == 2 ? 1 : 3;
    const int vec = ld * sizeof(TX) % 16 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0;
    const int64_t blocks = std::min<int64_t>((n + 7) / 8, 152 * 8);
    return launch_pdl(k_head_pack<TX, P>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                      static_cast<const TX*>(src), ld, n, d, up(d, 8), vec, dst, counts, row_of,
                      only_if_some ? 1 : 0, place, static_cast<TX*>(zero), ld_zero);
}

// The matrix as an operand: where it lies, or copied.
template <typename TX>
cudaError_t operand(const void* src, int64_t ld, int64_t n, int64_t d, __nv_bfloat16* copy,
                    Planes* out, cudaStream_t s) {
    constexpr bool bf16 = sizeof(TX) == 2;
    if (direct(src, ld, bf16)) {
        *out = {src, n, d, ld, 1};
        return cudaSuccess;
    }
    *out = {copy, n, up(d, 8), up(d, 8), bf16 ? 1 : 3};
    return pack<TX>(src, ld, n, d, copy, nullptr, nullptr, false, nullptr, nullptr, 0, s);
}

unsigned grid_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

template <typename TX>
cudaError_t loss_typed(const HeadProblem& p, float* loss, float* lse, float* student, float* delta,
                       void* ws, cudaStream_t s) {
    const int64_t R = p.S * p.T;
    const bool distill = p.tg.many;
    const LossSpace w = carve_loss(ws, p);
    if (!loss && delta) loss = w.loss;
    unsigned int* st = status_word();
    if (!st) return cudaErrorUnknown;
    const int32_t* targets = distill ? nullptr : p.tg.ids;
    const int64_t ld_part = up(R, 32);
    int parts = loss_parts(p);
    if (head_few(p)) {
        DUST_TRY(launch_head_few(p, w.part, ld_part, w.picked, student, s));
    } else {
        HeadLogits a = {};
        DUST_TRY(operand<TX>(p.H, p.ld_h, R, p.d, w.h, &a.H, s));
        DUST_TRY(operand<TX>(p.E, p.ld_e, p.V, p.d, w.e, &a.E, s));
        a.n = p.V;
        a.scale = p.scale;
        a.targets = targets;
        a.T = p.T;
        a.part = w.part;
        a.ld_part = ld_part;
        a.picked = w.picked;
        if (distill) {
            const int K = static_cast<int>(p.tg.K), warps = K <= 512 ? 8 : 4;
            int size = 32;
            while (size < K) size *= 2;
            DUST_TRY(launch_pdl(k_head_bins, dim3(grid_of(p.T, warps)), dim3(32 * warps),
                                static_cast<size_t>(warps) * 8 * size, s, p.S, p.T, p.tg.ids, K,
                                size, p.V, head_loss_columns(R, p.V) / 2, parts, w.entries,
                                w.starts, student, st));
            a.picks = {w.entries, w.starts, parts, p.tg.K, student};
        }
        DUST_TRY(launch_head_lse(a, s));
    }
    const int join_lanes = std::min(kJoinLanes, std::max(8, parts / 8));
    DUST_TRY(launch_pdl(k_head_join, dim3(grid_of(R, 32)), dim3(32 * join_lanes), 0, s, w.part,
                        ld_part, parts, R, p.T, targets, p.V, w.picked, loss, lse, st));
    if (distill && loss)
        DUST_TRY(launch_pdl(k_head_distill, dim3(grid_of(R, 8)), dim3(256), 0, s, R, p.T, p.tg,
                            p.V, p.scale, lse, student, loss));
    if (!delta || p.S < 2) return cudaSuccess;
    return launch_pdl(k_head_changes, dim3(grid_of(R - p.T, 256)), dim3(256), 0, s, loss, p.T,
                      R - p.T, delta);
}

template <typename TX>
cudaError_t grad_typed(const HeadProblem& p, const float* lse, const float* student,
                       const float* gloss, bool accumulate, void* gH, int64_t ld_gh, void* gE,
                       bool gE_bf16, void* ws, cudaStream_t s) {
    constexpr bool bf16 = sizeof(TX) == 2;
    const int64_t R = p.S * p.T, planes = bf16 ? 1 : 3;
    const bool distill = p.tg.many;
    const GradSpace w = carve_grad(ws, p);
    unsigned int* st = status_word();
    if (!st) return cudaErrorUnknown;
    if (distill)
        DUST_TRY(launch_pdl(k_head_teacher, dim3(grid_of(p.T, 8)), dim3(256), 0, s, p.T, p.tg, p.V,
                            p.scale, w.teacher, st));
    const LiveRows live = {static_cast<int32_t>(R), static_cast<int32_t>(p.T), p.V,
                           distill ? nullptr : p.tg.ids, w.teacher, gloss};
    DUST_TRY(launch_pdl(k_head_live, dim3(kLiveCtas), dim3(kLiveThreads), 0, s, live, lse,
                        w.counts, w.rows, w.row_of, w.place, st));
    HeadLogits a = {};
    const bool in_place = direct(p.H, p.ld_h, bf16);
    const Planes copy = {w.h, R, up(p.d, 8), up(p.d, 8), static_cast<int>(planes)};
    a.H = in_place ? Planes{p.H, R, p.d, p.ld_h, 1} : copy;
    if (in_place) a.Hc = copy;
    DUST_TRY(pack<TX>(p.H, p.ld_h, R, p.d, w.h, w.counts, w.row_of, in_place, w.place, gH, ld_gh,
                      s));
    DUST_TRY(operand<TX>(p.E, p.ld_e, p.V, p.d, w.e, &a.E, s));
    a.scale = p.scale;
    a.counts = w.counts;
    a.rows = w.rows;
    const int64_t g_rows = up(R, kHeadTile);
    a.G = {w.g, g_rows, w.piece, w.piece, static_cast<int>(planes)};
    for (int64_t v0 = 0; v0 < p.V; v0 += w.piece) {
        const int64_t n = std::min(w.piece, p.V - v0);
        a.v0 = v0;
        a.n = n;
        DUST_TRY(launch_head_factor(a, s));
        if (distill) {
            const int warps = p.tg.K <= 512 ? 8 : 4;
            const size_t smem = static_cast<size_t>(warps) * 8 * static_cast<size_t>(p.tg.K);
            const unsigned blocks = std::min(grid_of(R, warps), 152u * 8u);
            DUST_TRY(launch_pdl(k_head_patch<bf16 ? 1 : 3>, dim3(blocks), dim3(32 * warps), smem, s,
                                w.counts, w.rows, w.row_of, p.T, p.tg, p.scale, w.teacher, student,
                                v0, n, w.g, w.piece, g_rows * w.piece));
        }
        HeadProducts m = {};
        m.G = a.G;
        m.E = a.E;
        m.H = a.H;
        m.Hc = a.Hc;
        m.v0 = v0;
        m.n = n;
        m.d = p.d;
        m.scale = p.scale;
        m.counts = w.counts;
        m.row_of = w.row_of;
        m.gH = gH;
        m.ld_gh = ld_gh;
        m.gh_bf16 = bf16;
        // One choice for all pieces: gH's slices run on across them.
        m.cuts = w.cuts;
        m.gh_acc = w.piece < p.V || w.cuts.gh > 1 ? w.gh_acc : nullptr;
        m.ge_acc = w.cuts.ge > 1 ? w.ge_acc : nullptr;
        m.first = v0 == 0;
        m.last = v0 + n == p.V;
        m.gE = gE ? static_cast<unsigned char*>(gE) + v0 * p.d * (gE_bf16 ? 2 : 4) : nullptr;
        m.ge_bf16 = gE_bf16;
        m.accumulate = accumulate;
        DUST_TRY(launch_head_products(m, s));
    }
    return cudaSuccess;
}

}  // namespace

size_t head_loss_workspace_bytes(const HeadProblem& p) { return carve_loss(nullptr, p).total; }
size_t head_grad_workspace_bytes(const HeadProblem& p) { return carve_grad(nullptr, p).total; }

cudaError_t launch_head_loss(const HeadProblem& p, float* loss, float* lse, float* student,
                             float* delta, void* ws, cudaStream_t s) {
    ProfScope ps(kStageHead, s);
    return p.bf16 ? loss_typed<__nv_bfloat16>(p, loss, lse, student, delta, ws, s)
                  : loss_typed<float>(p, loss, lse, student, delta, ws, s);
}

cudaError_t launch_head_grad(const HeadProblem& p, const float* lse, const float* student,
                             const float* gloss, bool accumulate, void* gH, int64_t ld_gh,
                             void* gE, bool gE_bf16, void* ws, cudaStream_t s) {
    ProfScope ps(kStageHead, s);
    return p.bf16 ? grad_typed<__nv_bfloat16>(p, lse, student, gloss, accumulate, gH, ld_gh, gE,
                                              gE_bf16, ws, s)
                  : grad_typed<float>(p, lse, student, gloss, accumulate, gH, ld_gh, gE, gE_bf16,
                                      ws, s);
}

}  // namespace dust
