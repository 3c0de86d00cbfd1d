// The root-mean-square norm of each head's query and key and the rotation by
// the token's position, and the gradients (include/dust.h gives the formulas).
// Bound by memory: each head's values are read once and written once.
//
// A head's D values are held by G lanes of a warp, in pairs of vectors of V
// values: the two vectors of a pair are those that are turned into one another
// (halves of the rotated part), or neighbours (pairs turned within a vector,
// values that are not turned), so that the rotation needs no exchange between
// lanes. A warp keeps the same 32 / G heads, queries before keys, and goes from
// token to token: weights and addresses then stay in registers, and the next
// token's values are on their way meanwhile. (A warp that went from head to
// head of a token took 280 instructions a head for the addresses, weights and
// the queries' and keys' cases, and at 65536 tokens of 8 and 8 heads of 64
// 80 us, a third of HBM's rate.)
//
// The backward keeps each lane's sums of gm n for its own columns in registers
// over all the tokens of the warp; a CTA's warps leave one partial row, and
// k_rope_finish adds those up in order.
#include <algorithm>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kForwardCtas = 3, kBackwardCtas = 2;  // per SM
constexpr int kMaxCtas = 152 * kBackwardCtas;       // of the backward: partial rows

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
    float inv_d;
    int turned, pairs;         // vector pairs that are turned (halves), all of them
    unsigned int* status;
};

// V values as they lie.
template <typename TX, int V>
struct alignas(sizeof(TX) * V) Raw {
    TX x[V];
};

template <typename TX, int V>
__device__ __forceinline__ void store(TX* p, const float (&v)[V]) {
    Raw<TX, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) from_f(v[i], q.x[i]);
    *reinterpret_cast<Raw<TX, V>*>(p) = q;
}

// V floats of a table, on 16 bytes where V allows it.
template <int V>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 q = reinterpret_cast<const float4*>(p)[i];
            v[4 * i] = q.x;
            v[4 * i + 1] = q.y;
            v[4 * i + 2] = q.z;
            v[4 * i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = p[i];
    }
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
// pair's V turns. Pairs: V / 2 turns of either vector, one after another in the
// tables too.
template <int V, int PER>
struct Turns {
    float c[PER][V], s[PER][V];
};

template <int V, int G, int PER, bool HALVES>
__device__ __forceinline__ void load_turns(const Args& g, const Columns<V, G, PER, HALVES>& col, int lane,
                                           int64_t pos, Turns<V, PER>& t) {
    const float* cs = g.cosine + pos * (g.rot / 2);
    const float* sn = g.sine + pos * (g.rot / 2);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int from = HALVES ? col.a[i] : col.a[i] / 2;
        // The turns that there are: all or none (halves, or a single one).
        const int n = HALVES ? (lane + i * G < g.turned ? V : 0) : col.have[i] ? g.rot / 2 - from : 0;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            t.c[i][k] = 1.0f;
            t.s[i][k] = 0.0f;
        }
        if (n >= V) {
            load_floats<V>(cs + from, t.c[i]);
            load_floats<V>(sn + from, t.s[i]);
        } else if (!HALVES && n > 0) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (k < n) {
                    t.c[i][k] = cs[from + k];
                    t.s[i][k] = sn[from + k];
                }
        }
    }
}

// Turns a lane's values: x its first vectors, y its second ones; BACK: the other
// way round.
template <bool BACK, int V, int PER, bool HALVES>
__device__ __forceinline__ void turn(float (&x)[PER][V], float (&y)[PER][V], const Turns<V, PER>& t) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (HALVES || V == 1) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float u = x[i][k], v = y[i][k], n = BACK ? -t.s[i][k] : t.s[i][k];
                x[i][k] = u * t.c[i][k] - v * n;
                y[i][k] = v * t.c[i][k] + u * n;
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float* z = k < V / 2 ? &x[i][2 * k] : &y[i][2 * k - V];
                const float u = z[0], v = z[1], n = BACK ? -t.s[i][k] : t.s[i][k];
                z[0] = u * t.c[i][k] - v * n;
                z[1] = v * t.c[i][k] + u * n;
            }
        }
    }
}

// A head's values of a lane as they lie, and as numbers, zeros where there are
// none.
template <typename TX, int V, int PER>
struct Head {
    Raw<TX, V> a[PER], b[PER];

    template <int G, bool HALVES>
    __device__ __forceinline__ void fetch(const Columns<V, G, PER, HALVES>& col, const TX* p) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (col.have[i] > 0) a[i] = *reinterpret_cast<const Raw<TX, V>*>(p + col.a[i]);
            if (col.have[i] > 1) b[i] = *reinterpret_cast<const Raw<TX, V>*>(p + col.b[i]);
        }
    }
    template <int G, bool HALVES>
    __device__ __forceinline__ void values(const Columns<V, G, PER, HALVES>& col, bool there,
                                           float (&x)[PER][V], float (&y)[PER][V]) const {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                x[i][k] = there && col.have[i] > 0 ? to_f(a[i].x[k]) : 0.0f;
                y[i][k] = there && col.have[i] > 1 ? to_f(b[i].x[k]) : 0.0f;
            }
    }
};

template <int V, int G, int PER, bool HALVES, typename TX>
__device__ __forceinline__ void store_head(const Columns<V, G, PER, HALVES>& col, TX* p,
                                           const float (&x)[PER][V], const float (&y)[PER][V]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (col.have[i] > 0) store<TX, V>(p + col.a[i], x[i]);
        if (col.have[i] > 1) store<TX, V>(p + col.b[i], y[i]);
    }
}

// A head's weights at a lane's columns, 1 where there are none.
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

// A position, or -1 where the token is padding; one out of range is reported.
__device__ __forceinline__ int64_t position_of(const Args& g, int32_t p) {
    if (p < g.n_pos) return p < 0 ? -1 : p;
    atomicExch(g.status, 1u /* DUST_ERR_INVALID_ARG */);
    return -1;
}

// The heads and tokens of a warp: its group's head (or none), its first token
// and the step to the next one. Neighbouring warps take a token's heads in
// turn, so that its angles are read from HBM once.
template <int G>
struct Walk {
    int64_t t, step, head;  // head: among the queries' or the keys'
    bool in, key;

    __device__ explicit Walk(const Args& g) {
        constexpr int kGroups = 32 / G;
        const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
        const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
        const int64_t chunks = (g.heads + kGroups - 1) / kGroups;
        step = warps / chunks;  // 1 at least: see grid_of()
        t = warp / chunks;
        if (t >= step) t = g.T;  // the last warps, fewer than there are chunks
        head = warp % chunks * kGroups + threadIdx.x % 32 / G;
        in = head < g.heads;
        key = in && head >= g.hq;
        if (key) head -= g.hq;
        if (!in) head = 0;
    }
};

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads, kForwardCtas) k_rope(const Args g) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % G;
    const Columns<V, G, PER, HALVES> col(g, lane);
    const Walk<G> w(g);
    const Side& side = g.side[w.key];
    const TX* x_at = static_cast<const TX*>(side.x) + w.head * side.x_head;
    TX* y_at = static_cast<TX*>(side.y) + w.head * side.y_head;
    float wx[PER][V], wy[PER][V];
    load_weight(col, side.w, wx, wy);
    Head<TX, V, PER> next;
    int32_t next_pos = -1;
    const auto fetch = [&](int64_t t) {
        if (t >= g.T) return;
        next_pos = g.positions[t];
        if (w.in) next.fetch(col, x_at + t * side.x_token);
    };
    fetch(w.t);
    for (int64_t t = w.t; t < g.T; t += w.step) {
        const int64_t pos = position_of(g, next_pos);
        float x[PER][V], y[PER][V];
        next.values(col, w.in && pos >= 0, x, y);
        fetch(t + w.step);
        Turns<V, PER> turns;
        load_turns<V, G, PER, HALVES>(g, col, lane, max(pos, static_cast<int64_t>(0)), turns);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) s = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], s));
        s = group_sum<G>(s);
        if (!w.in) continue;
        if (pos >= 0) {
            const float rstd = rsqrtf(fmaf(s, g.inv_d, g.eps));
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    x[i][k] *= rstd * wx[i][k];
                    y[i][k] *= rstd * wy[i][k];
                }
            turn<false, V, PER, HALVES>(x, y, turns);
        }
        store_head<V, G, PER, HALVES>(col, y_at + t * side.y_token, x, y);
    }
}

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    k_rope_grad(const Args g, float* __restrict__ parts) {
    extern __shared__ float rows[];  // [kWarps][2][D]
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x % G, group = threadIdx.x % 32 / G;
    const Columns<V, G, PER, HALVES> col(g, lane);
    const Walk<G> w(g);
    const Side& side = g.side[w.key];
    const TX* x_at = static_cast<const TX*>(side.x) + w.head * side.x_head;
    const TX* g_at = static_cast<const TX*>(side.gy) + w.head * side.gy_head;
    TX* y_at = static_cast<TX*>(side.y) + w.head * side.y_head;
    float wx[PER][V], wy[PER][V];
    load_weight(col, side.w, wx, wy);
    float sx[PER][V] = {}, sy[PER][V] = {};  // of gm n
    Head<TX, V, PER> next_x, next_g;
    int32_t next_pos = -1;
    const auto fetch = [&](int64_t t) {
        if (t >= g.T) return;
        next_pos = g.positions[t];
        if (!w.in) return;
        next_x.fetch(col, x_at + t * side.x_token);
        next_g.fetch(col, g_at + t * side.gy_token);
    };
    fetch(w.t);
    for (int64_t t = w.t; t < g.T; t += w.step) {
        const int64_t pos = position_of(g, next_pos);
        float x[PER][V], y[PER][V], u[PER][V], v[PER][V];
        next_x.values(col, w.in && pos >= 0, x, y);
        next_g.values(col, w.in && pos >= 0, u, v);
        fetch(t + w.step);
        Turns<V, PER> turns;
        load_turns<V, G, PER, HALVES>(g, col, lane, max(pos, static_cast<int64_t>(0)), turns);
        turn<true, V, PER, HALVES>(u, v, turns);  // gm
        // sum x^2 and sum gm w x together; the root comes to the second later.
        float s = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s = fmaf(x[i][k], x[i][k], fmaf(y[i][k], y[i][k], s));
                dot = fmaf(u[i][k] * wx[i][k], x[i][k], fmaf(v[i][k] * wy[i][k], y[i][k], dot));
            }
        s = group_sum<G>(s);
        dot = group_sum<G>(dot);
        if (!w.in) continue;
        if (pos >= 0) {
            const float rstd = rsqrtf(fmaf(s, g.inv_d, g.eps));
            dot *= rstd * g.inv_d;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    x[i][k] *= rstd;  // n
                    y[i][k] *= rstd;
                    sx[i][k] = fmaf(u[i][k], x[i][k], sx[i][k]);
                    sy[i][k] = fmaf(v[i][k], y[i][k], sy[i][k]);
                    u[i][k] = rstd * fmaf(-x[i][k], dot, u[i][k] * wx[i][k]);
                    v[i][k] = rstd * fmaf(-y[i][k], dot, v[i][k] * wy[i][k]);
                }
        }
        store_head<V, G, PER, HALVES>(col, y_at + t * side.y_token, u, v);
    }
    if (!parts) return;
    // The groups of a warp one after another, then the warps.
    float* mine = rows + static_cast<int>(threadIdx.x) / 32 * 2 * g.D;
    for (int i = threadIdx.x % 32; i < 2 * g.D; i += 32) mine[i] = 0.0f;
    __syncwarp();
    for (int k = 0; k < 32 / G; ++k) {
        if (group == k && w.in) {
            float* to = mine + (w.key ? g.D : 0);
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (col.have[i] > 0) to[col.a[i] + e] += sx[i][e];
                    if (col.have[i] > 1) to[col.b[i] + e] += sy[i][e];
                }
        }
        __syncwarp();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.D; i += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += rows[k * 2 * g.D + i];
        parts[static_cast<int64_t>(blockIdx.x) * 2 * g.D + i] = s;
    }
}

// The partial rows added up: a CTA per 32 columns, its warps every 32nd row each.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads)
    k_rope_finish(const float* __restrict__ parts, int n, int D, bool accumulate, float* gwq, float* gwk) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sh[kFinishThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < 2 * D)
#pragma unroll 10
        for (int i = warp; i < n; i += kFinishThreads / 32) s += parts[static_cast<int64_t>(i) * 2 * D + c];
    sh[warp][lane] = s;
    __syncthreads();
    // Each warp one column.
    s = sh[lane][warp];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int col = blockIdx.x * 32 + warp;
    if (lane != 0 || col >= 2 * D) return;
    float* out = col < D ? gwq : gwk;
    if (!out) return;
    out += col < D ? col : col - D;
    *out = accumulate ? *out + s : s;
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

// CTAs: a warp per token and chunk of `groups` heads, as far as the GPU holds
// them, and at least one for every chunk.
unsigned grid_of(int64_t T, int64_t heads, int groups, int most) {
    const int64_t chunks = (heads + groups - 1) / groups;
    const int64_t ctas = (std::min<int64_t>(T, int64_t(1) << 20) * chunks + kWarps - 1) / kWarps;
    return static_cast<unsigned>(std::max((chunks + kWarps - 1) / kWarps, std::min<int64_t>(ctas, most)));
}
// Partial rows: for any split of the warps into groups.
int64_t most_parts(int64_t T, int64_t heads) { return grid_of(T, heads, 1, kMaxCtas); }

struct Launch {
    bool grad;
    float* parts;
    unsigned* n_parts;
    cudaStream_t s;
};

template <typename TX, int V, int G, int PER, bool HALVES>
cudaError_t launch_with(const Args& g, const Launch& l) {
    if (!l.grad)
        return launch_pdl(k_rope<TX, V, G, PER, HALVES>,
                          dim3(grid_of(g.T, g.heads, 32 / G, 152 * kForwardCtas)), dim3(kThreads), 0, l.s, g);
    *l.n_parts = grid_of(g.T, g.heads, 32 / G, kMaxCtas);
    return launch_pdl(k_rope_grad<TX, V, G, PER, HALVES>, dim3(*l.n_parts), dim3(kThreads),
                      sizeof(float) * 2 * kWarps * static_cast<size_t>(g.D), l.s, g, l.parts);
}

template <typename TX, int V, int LEAST, bool HALVES>
cudaError_t launch_groups(const Args& g, const Launch& l) {
    if (g.pairs <= 4 && LEAST <= 4) return launch_with<TX, V, LEAST, 1, HALVES>(g, l);
    if (g.pairs <= 8 && LEAST <= 8) return launch_with<TX, V, std::max(LEAST, 8), 1, HALVES>(g, l);
    if (g.pairs <= 16) return launch_with<TX, V, 16, 1, HALVES>(g, l);
    return launch_with<TX, V, 32, 1, HALVES>(g, l);
}

template <typename TX, bool HALVES>
cudaError_t launch_vectors(const Args& g, int V, const Launch& l) {
    const int per = (g.pairs + 31) / 32;
    if constexpr (sizeof(TX) == 2)
        if (V == 8) return launch_groups<TX, 8, 4, HALVES>(g, l);
    if (V == 4) return per == 1 ? launch_groups<TX, 4, 4, HALVES>(g, l) : launch_with<TX, 4, 32, 2, HALVES>(g, l);
    if (V == 2)
        return per == 1   ? launch_groups<TX, 2, 16, HALVES>(g, l)
               : per == 2 ? launch_with<TX, 2, 32, 2, HALVES>(g, l)
                          : launch_with<TX, 2, 32, 4, HALVES>(g, l);
    return per <= 2 ? launch_with<TX, 1, 32, 2, HALVES>(g, l) : launch_with<TX, 1, 32, 8, HALVES>(g, l);
}

cudaError_t run(const RopeProblem& p, const Launch& l) {
    Args g = {};
    const int size = p.bf16 ? 2 : 4;
    int V = 16 / size;
    const auto fits = [&](int v) {
        if (p.layout == DUST_ROPE_HALVES ? (p.rot / 2) % v || (p.D - p.rot) % v
                                         : p.D % v || (v >= 4 && (p.rot / 2) % 4))
            return false;
        if (v >= 4 && p.rot &&
            (reinterpret_cast<uintptr_t>(p.cosine) | reinterpret_cast<uintptr_t>(p.sine)) % 16)
            return false;
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
    while (V > 1 && !fits(V)) V /= 2;
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
    g.inv_d = 1.0f / static_cast<float>(p.D);
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
        return halves ? launch_vectors<__nv_bfloat16, true>(g, V, l)
                      : launch_vectors<__nv_bfloat16, false>(g, V, l);
    return halves ? launch_vectors<float, true>(g, V, l)
                  : launch_vectors<float, false>(g, V, l);
}

}  // namespace

size_t rope_grad_workspace_bytes(int64_t T, int64_t heads, int64_t D) {
    return T == 0 || heads == 0
               ? 0
               : sizeof(float) * 2 * static_cast<size_t>(D) * static_cast<size_t>(most_parts(T, heads));
}

cudaError_t launch_rope(const RopeProblem& p, cudaStream_t s) {
    ProfScope ps(kStageRope, s);
    return run(p, {false, nullptr, nullptr, s});
}

cudaError_t launch_rope_grad(const RopeProblem& p, bool accumulate, void* ws, cudaStream_t s) {
    ProfScope ps(kStageRope, s);
    const bool sums = p.side[0].gw || p.side[1].gw;
    unsigned n = 0;
    DUST_TRY(run(p, {true, sums ? static_cast<float*>(ws) : nullptr, &n, s}));
    if (!sums) return cudaSuccess;
    return launch_pdl(k_rope_finish, dim3(static_cast<unsigned>((2 * p.D + 31) / 32)), dim3(kFinishThreads),
                      0, s, static_cast<const float*>(ws), static_cast<int>(n), static_cast<int>(p.D),
                      accumulate, p.side[0].gw, p.side[1].gw);
}

}  // namespace dust
