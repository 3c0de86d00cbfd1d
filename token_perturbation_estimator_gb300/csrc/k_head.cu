// The head's per-token losses and their gradients, over the vocabulary in
// pieces and without keeping the logits (include/dust.h gives the formulas):
// softmax cross entropy against a target id, and distillation from a
// teacher's largest logits. The products are k_head_tc.cu's.
//
// A few rows go to k_head_few.cu.
//
// Loss: one launch forms the logits tile by tile and leaves per row a partial
// maximum and sum for every half tile, and the target's logit; a second one
// joins them. For distillation the pass over the tiles also picks the logits
// of the teacher's entries, which a first launch has put in order. (Formed
// apart, as products of a row of H with K rows of E, they took 74 us beside
// the logits' then 183 us, 4096 rows, d 1024, V 32768, K 64.)
//
// Gradient, per piece of the vocabulary (a piece's G has at most 2^28 values
// over its planes, or 1024 ids of every row where that is more: head_piece()):
// the logits again as G = weight (exp(x - lse) - wanted) in bf16,
// then gH += G E and gE = G^T H in one launch. For distillation a first launch
// puts each row's entries in order and forms exp(x - lse) - q at them, which
// the pass over the columns puts in their places. Rows that take no part (no
// target, no weight) are left out of all products: the others' H rows are
// moved together first if there are such rows.
//
// fp32 inputs, and bf16 ones whose rows do not start on 16 bytes, are first
// copied into the workspace, as three bf16 planes or padded rows.
//
// What is here is bound by latency but for the copies: 4 to 8 us a launch
// (16384 rows: which take part 5 us, joining 128 partials of 4096 rows 7 us,
// ordering 64 entries of 4096 tokens 14 us).
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

// The lanes of a warp meet first: .aligned wants them to arrive together.
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();
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

// The teacher of a token over its entries present: the largest scaled logit
// and the logarithm of the sum of exponentials over it; largest -inf where no
// entry has any probability. Whole warp.
__device__ __forceinline__ float2 teacher_stats(const int32_t* ids, const float* z, int64_t K,
                                                int64_t V, float scale) {
    const int lane = threadIdx.x & 31;
    float m = -INFINITY;
    bool nan = false;
    for (int64_t j = lane; j < K; j += 32) {
        const int32_t id = ids[j];
        if (id < 0 || id >= V) continue;
        m = fmaxf(m, scale * z[j]);  // passes NaN over
        nan |= isnan(z[j]);
    }
    m = __any_sync(0xffffffffu, nan) ? NAN : warp_max(m);
    float q = 0.0f;
    for (int64_t j = lane; j < K; j += 32) {
        const int32_t id = ids[j];
        if (m != -INFINITY && id >= 0 && id < V) q += expf(scale * z[j] - m);
    }
    q = warp_sum(q);
    return make_float2(m, logf(q));
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634074 - 1.4426950408889634f);

constexpr int kRankSize = 256;  // entries that are sorted by counting, at most

struct BinArgs {
    int64_t items;           // tokens (loss) or rows (gradient)
    int64_t S, T, V;
    HeadTargets tg;
    int size;                // K or more, a power of two, 32 at least
    int columns, bins;       // half tiles
    float scale;
    int2* entries;
    uint16_t* starts;
    float* student;          // loss: 0 written where an entry is absent; gradient: read
    const float* lse;        // gradient
    int32_t* alive;          // gradient: whether any entry has a probability
    unsigned int* status;
};

// Entries in order of their ids, so that the passes over the columns meet
// them on their way: a warp per token (loss) or row (gradient) sorts them (by
// counting, or many of them by a bitonic network, in shared memory), writes
// them out, and looks up where each half tile's first one is. Absent entries
// come last and are not counted.
// The loss is to write an entry's logit to its place; the gradient is to put
// exp(x - lse) - q there, which is formed here, with q the teacher's
// probability summed over the entries of the same id.
template <bool GRAD>
__global__ void __launch_bounds__(256) k_head_bins(const BinArgs a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t bins_smem[];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, size = a.size;
    const int K = static_cast<int>(a.tg.K);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5);
    if (item >= a.items) return;
    const int64_t t = GRAD ? item % a.T : item;
    const int32_t* ids = a.tg.ids + t * K;
    const float* z = a.tg.teacher + t * K;
    uint32_t* id = bins_smem + (threadIdx.x >> 5) * 3 * size;
    uint32_t* place = id + size;
    float* q = reinterpret_cast<float*>(place + size);
    int n = 0;
    bool bad = false;
    uint32_t* raw = reinterpret_cast<uint32_t*>(q);  // the ids in their own order, at first
    for (int j = lane; j < size; j += 32) {
        const int32_t v = j < K ? ids[j] : -1;
        const bool in = v >= 0 && v < a.V;
        bad |= v >= a.V;
        raw[j] = in ? static_cast<uint32_t>(v) : 0xffffffffu;
        n += __popc(__ballot_sync(0xffffffffu, in));
        if (!GRAD && j < K && !in)
            for (int64_t s = 0; s < a.S; ++s) a.student[(s * a.T + t) * K + j] = 0.0f;
    }
    if (bad) report_id(a.status);
    __syncwarp();
    // In both ways the place breaks ties: the order is the same every time.
    if (size <= kRankSize) {
        // An entry's position is the number of entries before it: comparisons
        // that do not wait for one another, where the network's every stage
        // waits for the one before (128 entries: 1600 clocks against 8000).
        for (int j = lane; j < K; j += 32) {
            const uint32_t mine = raw[j];
            int at = 0;
            for (int i = 0; i < K; ++i) {
                const uint32_t other = raw[i];
                at += other < mine || (other == mine && i < j);
            }
            id[at] = mine;
            place[at] = static_cast<uint32_t>(j);
        }
        __syncwarp();
    } else {
        for (int j = lane; j < size; j += 32) {
            id[j] = raw[j];
            place[j] = static_cast<uint32_t>(j);
        }
        __syncwarp();
        for (int k = 2; k <= size; k <<= 1) {
            for (int j = k >> 1; j > 0; j >>= 1) {
                for (int i = lane; i < size / 2; i += 32) {
                    const int p = 2 * i - (i & (j - 1)), u = p + j;  // bit j of p is 0
                    const bool rising = (p & k) == 0;
                    const bool over = id[p] > id[u] || (id[p] == id[u] && place[p] > place[u]);
                    if (over == rising) {
                        const uint32_t x = id[p], y = place[p];
                        id[p] = id[u];
                        place[p] = place[u];
                        id[u] = x;
                        place[u] = y;
                    }
                }
                __syncwarp();
            }
        }
    }
    if constexpr (GRAD) {
        const float2 st = teacher_stats(ids, z, K, a.V, a.scale);
        if (lane == 0) a.alive[item] = st.x != -INFINITY;
        if (st.x == -INFINITY) return;  // the row takes no part
        for (int j = lane; j < n; j += 32) q[j] = expf(a.scale * z[place[j]] - st.x - st.y);
        __syncwarp();
        const float l = a.lse[item];
        for (int j = lane; j < n; j += 32) {
            int from = j, to = j + 1;  // the entries of this id
            while (from > 0 && id[from - 1] == id[j]) --from;
            while (to < n && id[to] == id[j]) ++to;
            float sum = 0.0f;
            for (int i = from; i < to; ++i) sum += q[i];
            const float p = expf(a.student[item * K + place[j]] - l);
            a.entries[item * K + j] = make_int2(static_cast<int>(id[j]), __float_as_int(p - sum));
        }
    } else {
        for (int j = lane; j < n; j += 32)
            a.entries[item * K + j] = make_int2(static_cast<int>(id[j]), static_cast<int>(place[j]));
    }
    for (int b = lane; b <= a.bins; b += 32) {
        const uint32_t from = static_cast<uint32_t>(b) * static_cast<uint32_t>(a.columns);
        int lo = 0, hi = n;  // the first entry at or past `from`
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (id[mid] < from) lo = mid + 1;
            else hi = mid;
        }
        a.starts[item * (a.bins + 1) + b] = static_cast<uint16_t>(lo);
    }
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
    const float2 st = teacher_stats(ids, z, tg.K, V, scale);
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
    const int32_t* alive;      // distillation
    const float* gloss;

    // Whether row r takes part; its target and weight.
    __device__ __forceinline__ bool wanted(int64_t r, int32_t& id, float& g) const {
        id = -1;
        g = 0.0f;
        if (r >= R) return false;
        g = gloss[r];
        if (!targets) return alive[r] != 0 && g != 0.0f;
        id = targets[R == T ? static_cast<uint32_t>(r)
                            : static_cast<uint32_t>(r) % static_cast<uint32_t>(T)];
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
        h.target = a.targets ? id : static_cast<int32_t>(r);
        rows[to] = h;
        row_of[to] = static_cast<int32_t>(r);
    }
}

// Rows into the workspace as bf16 (one plane) or as three bf16 planes, zero
// from column d to dp.
template <typename TX>
struct PackJob {
    const TX* src;
    int64_t ld, n, d, dp;
    int vec;                   // rows can be read 16 bytes at a time
    __nv_bfloat16* dst;
    // With counts, row i is the i-th that takes part, rows up to the next
    // multiple of 64 are zeroed, and the rows of `zero` (gH) that take no part
    // are cleared; if all take part and only_if_some is set there is nothing
    // to do.
    const HeadCounts* counts;
    const int32_t* row_of;
    int only_if_some;
    const int32_t* place;
    TX* zero;
    int64_t ld_zero;
    unsigned blocks;           // CTAs that work on it
};

template <typename TX>
__device__ void pack_rows(const PackJob<TX>& a, int64_t block) {
    constexpr int PLANES = sizeof(TX) == 2 ? 1 : 3;
    const int64_t live = a.counts ? a.counts->rows : a.n;
    if (a.only_if_some && live == a.n) return;
    const int64_t end = a.counts ? min((live + 63) / 64 * 64, a.n) : a.n;
    const int lane = threadIdx.x & 31;
    for (int64_t i = block * 8 + (threadIdx.x >> 5); i < a.n;
         i += static_cast<int64_t>(a.blocks) * 8) {
        if (a.zero && a.place[i] < 0)
            for (int64_t c = lane; c < a.d; c += 32) a.zero[i * a.ld_zero + c] = TX(0.0f);
        if (i >= end) continue;
        const TX* s = i < live ? a.src + (a.row_of ? a.row_of[i] : i) * a.ld : nullptr;
        __nv_bfloat16* o = a.dst + i * a.dp;
        for (int64_t c = lane * 8; c < a.dp; c += 256) {
            float v[8];
            if (s && a.vec && c + 8 <= a.d) {
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
                for (int k = 0; k < 8; ++k) v[k] = s && c + k < a.d ? to_f(s[c + k]) : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
                alignas(16) __nv_bfloat16 b[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    b[k] = __float2bfloat16_rn(v[k]);
                    // Not up to infinity; and of an infinity nothing is left.
                    if (__hisinf(b[k])) b[k] = __float2bfloat16_rz(v[k]);
                    v[k] = __hisinf(b[k]) ? 0.0f : v[k] - __bfloat162float(b[k]);
                }
                *reinterpret_cast<uint4*>(o + p * a.n * a.dp + c) = *reinterpret_cast<const uint4*>(b);
            }
        }
    }
}

template <typename TX>
__global__ void __launch_bounds__(256) k_head_pack(const PackJob<TX> a, const PackJob<TX> b) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x < a.blocks)
        pack_rows(a, blockIdx.x);
    else
        pack_rows(b, blockIdx.x - a.blocks);
}

// ------------------------------------------------------------------ host

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t up(int64_t x, int64_t by) { return (x + by - 1) / by * by; }

// Whether TMA can read the rows where they lie.
bool direct(const void* p, int64_t ld, bool bf16) {
    return bf16 && ld % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
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
    const int64_t bn = head_columns(p.S * p.T, p.V, p.d);
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
    int32_t* alive;
    int2* entries;
    uint16_t* starts;
    int bins;
    __nv_bfloat16 *h, *e, *g;
    float *gh_acc, *ge_acc;
    HeadCuts cuts;
    int64_t piece;
    size_t total;
};

// Columns of the tiles of G, whose logits are summed as the loss's are.
int grad_columns(const HeadProblem& p, int64_t piece) {
    return head_columns(p.S * p.T, std::min(piece, p.V), p.d);
}

GradSpace carve_grad(void* ws, const HeadProblem& p) {
    const int64_t R = p.S * p.T, dp = up(p.d, 8), planes = p.bf16 ? 1 : 3;
    Carver c{static_cast<unsigned char*>(ws)};
    GradSpace w = {};
    w.alive = c.take<int32_t>(p.tg.many ? R : 0);
    w.entries = c.take<int2>(p.tg.many ? R * p.tg.K : 0);
    if (head_few(p)) {
        w.bins = static_cast<int>((p.V + head_few_grad_rows(p) - 1) / head_few_grad_rows(p));
        w.starts = c.take<uint16_t>(p.tg.many ? R * (w.bins + 1) : 0);
        w.gh_acc = c.take<float>(head_few_grad_parts(p) * R * p.d);
        w.total = c.at;
        return w;
    }
    w.piece = head_piece(R, p.V, p.d, static_cast<int>(planes));
    w.counts = c.take<HeadCounts>(1);
    w.rows = c.take<HeadRow>(R);
    w.row_of = c.take<int32_t>(R);
    w.place = c.take<int32_t>(R);
    const int64_t bn = grad_columns(p, w.piece);
    w.bins = static_cast<int>(2 * ((p.V + bn - 1) / bn));
    w.starts = c.take<uint16_t>(p.tg.many ? R * (w.bins + 1) : 0);
    // As for both gradients, whichever are asked for.
    w.cuts = head_cuts(R, std::min(w.piece, p.V), p.d, static_cast<int>(planes));
    const int n_planes = static_cast<int>(planes);
    w.gh_acc = c.take<float>(
        w.piece < p.V || w.cuts.gh > 1 ? head_acc_floats(R, p.d, n_planes, w.cuts.gh) : 0);
    w.ge_acc = c.take<float>(
        w.cuts.ge > 1 ? head_acc_floats(w.piece, p.d, n_planes, w.cuts.ge) : 0);
    w.g = c.take<__nv_bfloat16>(planes * up(R, kHeadTile) * w.piece);
    w.h = c.take<__nv_bfloat16>(planes * R * dp);
    w.e = c.take<__nv_bfloat16>(planes * p.V * dp);
    w.total = c.at;
    return w;
}

// The copy of a matrix of n rows.
template <typename TX>
PackJob<TX> pack_job(const void* src, int64_t ld, int64_t n, int64_t d, __nv_bfloat16* dst) {
    PackJob<TX> j = {};
    j.src = static_cast<const TX*>(src);
    j.ld = ld;
    j.n = n;
    j.d = d;
    j.dp = up(d, 8);
    j.vec = ld * sizeof(TX) % 16 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0;
    j.dst = dst;
    j.blocks = static_cast<unsigned>(std::min<int64_t>((n + 7) / 8, 152 * 8));
    return j;
}

template <typename TX>
cudaError_t pack(const PackJob<TX>& a, const PackJob<TX>& b, cudaStream_t s) {
    if (a.blocks + b.blocks == 0) return cudaSuccess;
    return launch_pdl(k_head_pack<TX>, dim3(a.blocks + b.blocks), dim3(256), 0, s, a, b);
}

// The matrix as an operand: where it lies, or the copy that *job is to make.
template <typename TX>
Planes operand(const void* src, int64_t ld, int64_t n, int64_t d, __nv_bfloat16* copy,
               PackJob<TX>* job) {
    constexpr bool bf16 = sizeof(TX) == 2;
    *job = {};
    if (direct(src, ld, bf16)) return {src, n, d, ld, 1};
    *job = pack_job<TX>(src, ld, n, d, copy);
    return {copy, n, up(d, 8), up(d, 8), bf16 ? 1 : 3};
}

int sort_size(int64_t K) {
    int size = 32;
    while (size < K) size *= 2;
    return size;
}

unsigned grid_of(int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); }

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

template <bool GRAD>
cudaError_t launch_bins(BinArgs b, const HeadProblem& p, cudaStream_t s) {
    b.S = p.S;
    b.T = p.T;
    b.V = p.V;
    b.tg = p.tg;
    b.scale = p.scale;
    b.size = sort_size(p.tg.K);
    b.status = status_word();
    const int warps = b.size <= 256 ? 8 : 4;  // at most 48 KB of shared memory
    return launch_pdl(k_head_bins<GRAD>, dim3(grid_of(b.items, warps)), dim3(32 * warps),
                      static_cast<size_t>(warps) * 12 * b.size, s, b);
}

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
        PackJob<TX> jh, je;
        a.H = operand<TX>(p.H, p.ld_h, R, p.d, w.h, &jh);
        a.E = operand<TX>(p.E, p.ld_e, p.V, p.d, w.e, &je);
        DUST_TRY(pack(jh, je, s));
        a.n = p.V;
        a.bn = head_columns(R, p.V, p.d);
        a.scale = p.scale;
        a.targets = targets;
        a.T = p.T;
        a.part = w.part;
        a.ld_part = ld_part;
        a.picked = w.picked;
        if (distill) {
            BinArgs b = {};
            b.items = p.T;
            b.columns = a.bn / 2;
            b.bins = parts;
            b.entries = w.entries;
            b.starts = w.starts;
            b.student = student;
            DUST_TRY(launch_bins<false>(b, p, s));
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
    const bool few = head_few(p);
    HeadLogits a = {};
    if (!few) a.bn = grad_columns(p, w.piece);
    if (distill) {
        BinArgs b = {};
        b.items = R;
        b.columns = few ? head_few_grad_rows(p) : a.bn / 2;
        b.bins = w.bins;
        b.entries = w.entries;
        b.starts = w.starts;
        b.student = const_cast<float*>(student);
        b.lse = lse;
        b.alive = w.alive;
        DUST_TRY(launch_bins<true>(b, p, s));
        a.picks = {w.entries, w.starts, b.bins, p.tg.K, nullptr};
    }
    if (few)
        return launch_head_few_grad(p, a.picks, w.alive, lse, gloss, accumulate, w.gh_acc, gH, ld_gh,
                                    gE, gE_bf16, s);
    const LiveRows live = {static_cast<int32_t>(R), static_cast<int32_t>(p.T), p.V,
                           distill ? nullptr : p.tg.ids, w.alive, gloss};
    DUST_TRY(launch_pdl(k_head_live, dim3(kLiveCtas), dim3(kLiveThreads), 0, s, live, lse,
                        w.counts, w.rows, w.row_of, w.place, st));
    const bool in_place = direct(p.H, p.ld_h, bf16);
    const Planes copy = {w.h, R, up(p.d, 8), up(p.d, 8), static_cast<int>(planes)};
    a.H = in_place ? Planes{p.H, R, p.d, p.ld_h, 1} : copy;
    if (in_place) a.Hc = copy;
    PackJob<TX> jh = pack_job<TX>(p.H, p.ld_h, R, p.d, w.h), je;
    jh.counts = w.counts;
    jh.row_of = w.row_of;
    jh.only_if_some = in_place;
    jh.place = w.place;
    jh.zero = static_cast<TX*>(gH);
    jh.ld_zero = ld_gh;
    a.E = operand<TX>(p.E, p.ld_e, p.V, p.d, w.e, &je);
    DUST_TRY(pack(jh, je, s));
    a.scale = p.scale;
    a.counts = w.counts;
    a.rows = w.rows;
    a.G = {w.g, up(R, kHeadTile), w.piece, w.piece, static_cast<int>(planes)};
    HeadMaps maps;
    if (!make_head_maps(&maps, a.H, a.Hc, a.E, a.G)) return cudaErrorInvalidValue;
    for (int64_t v0 = 0; v0 < p.V; v0 += w.piece) {
        const int64_t n = std::min(w.piece, p.V - v0);
        a.v0 = v0;
        a.n = n;
        DUST_TRY(launch_head_factor(a, maps, s));
        HeadProducts m = {};
        m.rows = R;
        m.planes = static_cast<int>(planes);
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
        DUST_TRY(launch_head_products(m, maps, s));
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
