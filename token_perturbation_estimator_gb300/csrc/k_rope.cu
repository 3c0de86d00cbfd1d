// The root-mean-square norm of each head's query and key and the rotation by
// the token's position, and the gradients (include/dust.h gives the formulas).
// Bound by memory: each head's values are read once and written once.
//
// A head's D values are held by G lanes of a warp, in pairs of vectors of V
// values: the two vectors of a pair are those that are turned into one another
// (halves of the rotated part), or neighbours (pairs turned within a vector,
// values that are not turned), so that the rotation needs no exchange between
// lanes. The warp's 32 / G groups take the heads of one token in turn, queries
// before keys, and keep its cosines and sines in registers.
//
// The backward keeps each lane's sums of gm n for its own columns in
// registers, queries' and keys' apart, over all the tokens of the warp; a
// CTA's warps leave one partial row, and k_rope_finish adds those up in order.
#include <algorithm>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCtas = 152 * 4;     // of the backward: partial rows

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

struct Side {
    const void *x, *gy;
    void* y;
    int64_t x_token, x_head, y_token, y_head, gy_token, gy_head;
    const float* w;
};

struct Args {
    Side side[2];
    int hq, heads;             // queries' heads, all heads
    int64_t T;
    int D, rot;
    float eps;
    const int32_t* positions;
    const float *cosine, *sine;
    int64_t n_pos;
    int turned, pairs;         // vector pairs that are turned (halves), all of them
    unsigned int* status;
};

template <typename TX, int V>
__device__ __forceinline__ void load(const TX* p, float (&v)[V]) {
    struct alignas(sizeof(TX) * V) Vec { TX x[V]; };
    const Vec q = *reinterpret_cast<const Vec*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = to_f(q.x[i]);
}

template <typename TX, int V>
__device__ __forceinline__ void store(TX* p, const float (&v)[V]) {
    struct alignas(sizeof(TX) * V) Vec { TX x[V]; };
    Vec q;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f(v[i], q.x[i]);
    *reinterpret_cast<Vec*>(p) = q;
}

// A lane's vector pairs: the first value of each, and how many vectors there
// are (0 to 2).
template <int V, int G, int PER, bool HALVES>
struct Columns {
    int a[PER], b[PER], have[PER];

    __device__ Columns(const Args& g, int lane) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int p = lane + i * G;
            if (HALVES && p < g.turned) {
                a[i] = p * V;
                b[i] = a[i] + g.rot / 2;
            } else {
                const int from = HALVES ? g.rot : 0, q = HALVES ? p - g.turned : p;
                a[i] = from + 2 * q * V;
                b[i] = a[i] + V;
            }
            have[i] = p >= g.pairs ? 0 : b[i] + V <= g.D ? 2 : 1;
        }
    }
};

// The angles' cosines and sines of a lane's vector pairs. Halves: those of a
// pair's V turns. Pairs: V / 2 turns of either vector.
template <int V, int PER>
struct Turns {
    float c[PER][V], s[PER][V];
};

template <int V, int G, int PER, bool HALVES>
__device__ __forceinline__ void load_turns(const Args& g, const Columns<V, G, PER, HALVES>& col, int lane,
                                           int64_t pos, float sign, Turns<V, PER>& t) {
    const float* cs = g.cosine + pos * (g.rot / 2);
    const float* sn = g.sine + pos * (g.rot / 2);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            t.c[i][k] = 1.0f;
            t.s[i][k] = 0.0f;
        }
        if constexpr (HALVES) {
            if (lane + i * G < g.turned) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    t.c[i][k] = cs[col.a[i] + k];
                    t.s[i][k] = sign * sn[col.a[i] + k];
                }
            }
        } else if constexpr (V >= 2) {
#pragma unroll
            for (int k = 0; k < V; ++k) {  // turn k of the two vectors together
                const int e = col.a[i] + 2 * k;
                if (col.have[i] && e < g.rot) {
                    t.c[i][k] = cs[e / 2];
                    t.s[i][k] = sign * sn[e / 2];
                }
            }
        } else if (col.have[i] == 2 && col.a[i] < g.rot) {
            t.c[i][0] = cs[col.a[i] / 2];
            t.s[i][0] = sign * sn[col.a[i] / 2];
        }
    }
}

// Turns a lane's values: x its first vectors, y its second ones.
template <int V, int PER, bool HALVES>
__device__ __forceinline__ void turn(float (&x)[PER][V], float (&y)[PER][V], const Turns<V, PER>& t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (HALVES || V == 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float u = x[i][k], v = y[i][k];
                x[i][k] = u * t.c[i][k] - v * t.s[i][k];
                y[i][k] = v * t.c[i][k] + u * t.s[i][k];
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float* z = k < V / 2 ? &x[i][2 * k] : &y[i][2 * k - V];
                const float u = z[0], v = z[1];
                z[0] = u * t.c[i][k] - v * t.s[i][k];
                z[1] = v * t.c[i][k] + u * t.s[i][k];
            }
        }
    }
}

template <int V, int G, int PER, bool HALVES, typename TX>
__device__ __forceinline__ void load_head(const Columns<V, G, PER, HALVES>& col, const TX* p,
                                          float (&x)[PER][V], float (&y)[PER][V]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) x[i][k] = y[i][k] = 0.0f;
        if (col.have[i] > 0) load<TX, V>(p + col.a[i], x[i]);
        if (col.have[i] > 1) load<TX, V>(p + col.b[i], y[i]);
    }
}

template <int V, int G, int PER, bool HALVES, typename TX>
__device__ __forceinline__ void store_head(const Columns<V, G, PER, HALVES>& col, TX* p,
                                           const float (&x)[PER][V], const float (&y)[PER][V]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (col.have[i] > 0) store<TX, V>(p + col.a[i], x[i]);
        if (col.have[i] > 1) store<TX, V>(p + col.b[i], y[i]);
    }
}

// A parameter at a lane's columns, 1 where there is none.
template <int V, int G, int PER, bool HALVES>
__device__ __forceinline__ void load_weight(const Columns<V, G, PER, HALVES>& col, const float* w,
                                            float (&x)[PER][V], float (&y)[PER][V]) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            x[i][k] = w && col.have[i] > 0 ? w[col.a[i] + k] : 1.0f;
            y[i][k] = w && col.have[i] > 1 ? w[col.b[i] + k] : 1.0f;
        }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The position of token t, or -1 where it is padding; one out of range is reported.
__device__ __forceinline__ int64_t position_of(const Args& g, int64_t t) {
    const int64_t p = g.positions[t];
    if (p < g.n_pos) return p < 0 ? -1 : p;
    atomicExch(g.status, 1u /* DUST_ERR_INVALID_ARG */);
    return -1;
}

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_rope(const Args g) {
    pdl_wait();
    pdl_trigger();
    constexpr int kGroups = 32 / G;
    const int lane = threadIdx.x % G, group = threadIdx.x % 32 / G;
    const Columns<V, G, PER, HALVES> col(g, lane);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; t < g.T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t pos = position_of(g, t);
        Turns<V, PER> turns;
        load_turns<V, G, PER, HALVES>(g, col, lane, max(pos, static_cast<int64_t>(0)), 1.0f, turns);
        for (int h0 = 0; h0 < g.heads; h0 += kGroups) {
            const int h = h0 + group;
            const bool in = h < g.heads;
            const Side& side = g.side[in && h >= g.hq ? 1 : 0];
            const int64_t n = h - (h >= g.hq ? g.hq : 0);
            float x[PER][V] = {}, y[PER][V] = {};
            if (in && pos >= 0)
                load_head<V, G, PER, HALVES>(
                    col, static_cast<const TX*>(side.x) + t * side.x_token + n * side.x_head, x, y);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) s = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], s));
            s = group_sum<G>(s);
            const float rstd = 1.0f / sqrtf(s / static_cast<float>(g.D) + g.eps);
            if (!in) continue;
            float wx[PER][V], wy[PER][V];
            load_weight<V, G, PER, HALVES>(col, side.w, wx, wy);
            if (pos >= 0) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        x[i][k] *= rstd * wx[i][k];
                        y[i][k] *= rstd * wy[i][k];
                    }
                turn<V, PER, HALVES>(x, y, turns);
            }
            store_head<V, G, PER, HALVES>(
                col, static_cast<TX*>(side.y) + t * side.y_token + n * side.y_head, x, y);
        }
    }
}

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads) k_rope_grad(const Args g, float* __restrict__ parts) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ float rows[];  // [2][D]
    constexpr int kGroups = 32 / G;
    const int lane = threadIdx.x % G, group = threadIdx.x % 32 / G;
    const Columns<V, G, PER, HALVES> col(g, lane);
    float sum[2][2][PER][V] = {};  // queries' and keys', first and second vectors
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32; t < g.T;
         t += static_cast<int64_t>(gridDim.x) * kWarps) {
        const int64_t pos = position_of(g, t);
        Turns<V, PER> turns;
        load_turns<V, G, PER, HALVES>(g, col, lane, max(pos, static_cast<int64_t>(0)), -1.0f, turns);
        // Queries, then keys: each lane knows which of its sums it adds to.
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const Side& side = g.side[kind];
            const int heads = kind ? g.heads - g.hq : g.hq;
            for (int h0 = 0; h0 < heads; h0 += kGroups) {
                const int64_t n = h0 + group;
                const bool in = n < heads;
                float x[PER][V] = {}, y[PER][V] = {}, u[PER][V] = {}, v[PER][V] = {};
                if (in && pos >= 0) {
                    load_head<V, G, PER, HALVES>(
                        col, static_cast<const TX*>(side.x) + t * side.x_token + n * side.x_head, x, y);
                    load_head<V, G, PER, HALVES>(
                        col, static_cast<const TX*>(side.gy) + t * side.gy_token + n * side.gy_head, u, v);
                }
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k) s = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], s));
                s = group_sum<G>(s);
                const float rstd = 1.0f / sqrtf(s / static_cast<float>(g.D) + g.eps);
                turn<V, PER, HALVES>(u, v, turns);  // gm
                float wx[PER][V], wy[PER][V];
                load_weight<V, G, PER, HALVES>(col, side.w, wx, wy);
                float dot = 0.0f;
                if (pos >= 0 && in) {
#pragma unroll
                    for (int i = 0; i < PER; ++i)
#pragma unroll
                        for (int k = 0; k < V; ++k) {
                            x[i][k] *= rstd;  // n
                            y[i][k] *= rstd;
                            sum[kind][0][i][k] = fmaf(u[i][k], x[i][k], sum[kind][0][i][k]);
                            sum[kind][1][i][k] = fmaf(v[i][k], y[i][k], sum[kind][1][i][k]);
                            u[i][k] *= wx[i][k];
                            v[i][k] *= wy[i][k];
                            dot = fmaf(u[i][k], x[i][k], fmaf(v[i][k], y[i][k], dot));
                        }
                }
                dot = group_sum<G>(dot) / static_cast<float>(g.D);
                if (!in) continue;
                if (pos >= 0) {
#pragma unroll
                    for (int i = 0; i < PER; ++i)
#pragma unroll
                        for (int k = 0; k < V; ++k) {
                            u[i][k] = rstd * (u[i][k] - x[i][k] * dot);
                            v[i][k] = rstd * (v[i][k] - y[i][k] * dot);
                        }
                }
                store_head<V, G, PER, HALVES>(
                    col, static_cast<TX*>(side.y) + t * side.y_token + n * side.y_head, u, v);
            }
        }
    }
    if (!parts) return;
    // The groups of a warp, then the warps one after another.
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float& s = sum[kind][half][i][k];
#pragma unroll
                    for (int off = 16; off >= G; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
                }
    for (int w = 0; w < kWarps; ++w) {
        if (static_cast<int>(threadIdx.x) / 32 == w && group == 0) {
#pragma unroll
            for (int kind = 0; kind < 2; ++kind)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < PER; ++i)
                        if (col.have[i] > half)
#pragma unroll
                            for (int k = 0; k < V; ++k) {
                                float* to = rows + kind * g.D + (half ? col.b[i] : col.a[i]) + k;
                                *to = w == 0 ? sum[kind][half][i][k] : *to + sum[kind][half][i][k];
                            }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * g.D; i += kThreads) parts[static_cast<int64_t>(blockIdx.x) * 2 * g.D + i] = rows[i];
}

// The partial rows added up: a warp per 32 columns... one CTA per 32 columns,
// its warps each every eighth row.
__global__ void __launch_bounds__(kThreads)
    k_rope_finish(const float* __restrict__ parts, int n, int D, bool accumulate, float* gwq, float* gwk) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * D)
#pragma unroll 4
        for (int i = warp; i < n; i += kWarps) s += parts[static_cast<int64_t>(i) * 2 * D + c];
    sh[warp][lane] = s;
    __syncthreads();
    if (warp != 0 || c >= 2 * D) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += sh[w][lane];
    float* out = c < D ? gwq : gwk;
    if (!out) return;
    out += c < D ? c : c - D;
    *out = accumulate ? *out + s : s;
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

unsigned grad_grid(int64_t T) {
    return static_cast<unsigned>(std::min<int64_t>((T + kWarps - 1) / kWarps, kMaxCtas));
}

template <typename TX, int V, int G, int PER, bool HALVES>
cudaError_t launch_with(const Args& g, bool grad, float* parts, cudaStream_t s) {
    const int64_t ctas = (g.T + kWarps - 1) / kWarps;
    if (!grad)
        return launch_pdl(k_rope<TX, V, G, PER, HALVES>,
                          dim3(static_cast<unsigned>(std::min<int64_t>(ctas, 152 * 64))), dim3(kThreads), 0,
                          s, g);
    return launch_pdl(k_rope_grad<TX, V, G, PER, HALVES>, dim3(grad_grid(g.T)), dim3(kThreads),
                      sizeof(float) * 2 * static_cast<size_t>(g.D), s, g, parts);
}

template <typename TX, int V, int PER, bool HALVES>
cudaError_t launch_groups(const Args& g, bool grad, float* parts, cudaStream_t s) {
    if constexpr (PER == 1) {
        if (g.pairs <= 4) return launch_with<TX, V, 4, 1, HALVES>(g, grad, parts, s);
        if (g.pairs <= 8) return launch_with<TX, V, 8, 1, HALVES>(g, grad, parts, s);
        if (g.pairs <= 16) return launch_with<TX, V, 16, 1, HALVES>(g, grad, parts, s);
    }
    return launch_with<TX, V, 32, PER, HALVES>(g, grad, parts, s);
}

template <typename TX, bool HALVES>
cudaError_t launch_vectors(const Args& g, int V, bool grad, float* parts, cudaStream_t s) {
    const int per = (g.pairs + 31) / 32;
    if constexpr (sizeof(TX) == 2)
        if (V == 8) return launch_groups<TX, 8, 1, HALVES>(g, grad, parts, s);
    if (V == 4)
        return per == 1 ? launch_groups<TX, 4, 1, HALVES>(g, grad, parts, s)
                        : launch_groups<TX, 4, 2, HALVES>(g, grad, parts, s);
    return per <= 2 ? launch_groups<TX, 1, 2, HALVES>(g, grad, parts, s)
                    : launch_groups<TX, 1, 8, HALVES>(g, grad, parts, s);
}

cudaError_t run(const RopeProblem& p, bool grad, float* parts, cudaStream_t s) {
    Args g = {};
    const int size = p.bf16 ? 2 : 4;
    int V = 16 / size;
    const auto fits = [&](int v) {
        if (p.layout == DUST_ROPE_HALVES ? (p.rot / 2) % v || (p.D - p.rot) % v : p.D % v) return false;
        for (const RopeSide& d : p.side) {
            if (d.heads == 0) continue;
            const auto on = [&](const dust_heads& h) {
                return !h.data || ((reinterpret_cast<uintptr_t>(h.data) |
                                    static_cast<uintptr_t>(h.token_stride * size) |
                                    static_cast<uintptr_t>(h.head_stride * size)) % (v * size)) == 0;
            };
            if (!on(d.x) || !on(d.y) || !on(d.gy)) return false;
        }
        return true;
    };
    while (V > 1 && !fits(V)) V = V > 4 ? 4 : 1;
    for (int i = 0; i < 2; ++i) {
        const RopeSide& d = p.side[i];
        g.side[i] = {d.x.data, d.gy.data, d.y.data, d.x.token_stride, d.x.head_stride, d.y.token_stride,
                     d.y.head_stride, d.gy.token_stride, d.gy.head_stride, d.w};
    }
    g.hq = static_cast<int>(p.side[0].heads);
    g.heads = static_cast<int>(p.side[0].heads + p.side[1].heads);
    g.T = p.T;
    g.D = static_cast<int>(p.D);
    g.rot = static_cast<int>(p.rot);
    g.eps = p.eps;
    g.positions = p.positions;
    g.cosine = p.cosine;
    g.sine = p.sine;
    g.n_pos = p.n_pos;
    const bool halves = p.layout == DUST_ROPE_HALVES;
    g.turned = halves ? g.rot / 2 / V : 0;
    g.pairs = g.turned + ((halves ? g.D - g.rot : g.D) + 2 * V - 1) / (2 * V);
    g.status = status_word();
    if (!g.status) return cudaErrorUnknown;
    if (p.bf16)
        return halves ? launch_vectors<__nv_bfloat16, true>(g, V, grad, parts, s)
                      : launch_vectors<__nv_bfloat16, false>(g, V, grad, parts, s);
    return halves ? launch_vectors<float, true>(g, V, grad, parts, s)
                  : launch_vectors<float, false>(g, V, grad, parts, s);
}

}  // namespace

size_t rope_grad_workspace_bytes(int64_t T, int64_t heads, int64_t D) {
    return heads == 0 ? 0 : sizeof(float) * 2 * static_cast<size_t>(D) * grad_grid(T);
}

cudaError_t launch_rope(const RopeProblem& p, cudaStream_t s) {
    ProfScope ps(kStageRope, s);
    return run(p, false, nullptr, s);
}

cudaError_t launch_rope_grad(const RopeProblem& p, bool accumulate, void* ws, cudaStream_t s) {
    ProfScope ps(kStageRope, s);
    const bool sums = p.side[0].gw || p.side[1].gw;
    DUST_TRY(run(p, true, sums ? static_cast<float*>(ws) : nullptr, s));
    if (!sums) return cudaSuccess;
    return launch_pdl(k_rope_finish, dim3(static_cast<unsigned>((2 * p.D + 31) / 32)), dim3(kThreads), 0, s,
                      static_cast<const float*>(ws), static_cast<int>(grad_grid(p.T)),
                      static_cast<int>(p.D), accumulate, p.side[0].gw, p.side[1].gw);
}

}  // namespace dust
