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
// tokens' values are on their way meanwhile.
//
// Heads whose vectors are 16 bytes go through k_rope_fast, with the next kRing
// tokens' values in shared memory (cp.async, each thread's own) and two values
// an instruction; other sizes and alignments through k_rope, value by value or
// in smaller vectors, the next tokens' values in registers. Those lanes move
// fewer bytes each, so that latency bounds them: 1.2 to 3.4 TB/s, by single
// bf16 values the least (head sizes of 13 to 201).
//
// Measured, bf16: 65536 tokens of 8 and 8 heads of 64 in rows of 24, 45 to 48 us
// = 5.9 to 6.4 TB/s; backward of 16384 tokens of 32 and 8 heads of 128, 91 to 94
// us = 5.5 TB/s. (A warp that went from head to head of a token took 280
// instructions a head, for addresses, weights and the two kinds, and 73 to 83
// us; loads of one token ahead into registers 73 and 171 us. 2, 3 and 4 tokens
// in the ring take the same time, 6 two to five per cent more; two CTAs an SM
// instead of three 54 us, four 60.)
//
// The backward keeps each lane's sums of gm n for its own columns in registers
// over all the tokens of the warp; a CTA's warps leave one partial row, and
// k_rope_finish adds those up in order.
#include <algorithm>

#include "f32x2.cuh"
#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRing = 2;              // tokens on their way per warp
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
    if constexpr (sizeof(TX) == 2 && V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            *reinterpret_cast<__nv_bfloat162*>(q.x + i) = __floats2bfloat162_rn(v[i], v[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) from_f(v[i], q.x[i]);
    }
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
    int turns[PER];  // angles: all V or none (halves), or what is left of the tables (pairs)

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
            turns[i] = HALVES ? (p < g.turned ? V : 0) : have[i] ? g.rot / 2 - a[i] / 2 : 0;
        }
    }
};

// The angles' cosines and sines of a lane's vector pairs, 1 and 0 where nothing
// turns. Halves: those of a pair's V turns. Pairs: V / 2 turns of either vector,
// one after another in the tables too.
template <int V, int PER>
struct Turns {
    float c[PER][V], s[PER][V];

    __device__ Turns() {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                c[i][k] = 1.0f;
                s[i][k] = 0.0f;
            }
    }

    // Of a position. How many there are is the same for all of them.
    template <int G, bool HALVES>
    __device__ __forceinline__ void load(const Args& g, const Columns<V, G, PER, HALVES>& col, int64_t pos) {
        const float* cs = g.cosine + pos * (g.rot / 2);
        const float* sn = g.sine + pos * (g.rot / 2);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int from = HALVES ? col.a[i] : col.a[i] / 2;
            if (col.turns[i] >= V) {
                load_floats<V>(cs + from, c[i]);
                load_floats<V>(sn + from, s[i]);
            } else if (!HALVES && col.turns[i] > 0) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (k < col.turns[i]) {
                        c[i][k] = cs[from + k];
                        s[i][k] = sn[from + k];
                    }
            }
        }
    }
};

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

// A head's values of a lane as they lie, and as numbers; zeros where there are
// none, which no load touches.
template <typename TX, int V, int PER>
struct Head {
    Raw<TX, V> a[PER], b[PER];

    __device__ Head() {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) a[i].x[k] = b[i].x[k] = TX(0.0f);
    }

    template <int G, bool HALVES>
    __device__ __forceinline__ void fetch(const Columns<V, G, PER, HALVES>& col, const TX* p) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (col.have[i] > 0) a[i] = *reinterpret_cast<const Raw<TX, V>*>(p + col.a[i]);
            if (col.have[i] > 1) b[i] = *reinterpret_cast<const Raw<TX, V>*>(p + col.b[i]);
        }
    }
    __device__ __forceinline__ void values(float (&x)[PER][V], float (&y)[PER][V]) const {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                x[i][k] = to_f(a[i].x[k]);
                y[i][k] = to_f(b[i].x[k]);
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
        if (!in) head = 0;  // stands at a head that there is
        key = head >= g.hq;
        if (key) head -= g.hq;
    }
};

// The warps' sums of gm n, [kWarps][2][D], as the CTA's partial row.
__device__ __forceinline__ void join_rows(const Args& g, const float* rows, float* parts) {
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * g.D; i += kThreads) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) s += rows[k * 2 * g.D + i];
        parts[static_cast<int64_t>(blockIdx.x) * 2 * g.D + i] = s;
    }
}

template <int V, int PER>
__device__ __forceinline__ void clear(float (&x)[PER][V], float (&y)[PER][V]) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) x[i][k] = y[i][k] = 0.0f;
}

// Tokens that a warp of k_rope and k_rope_grad takes at once, and has on their
// way, and CTAs per SM, for lanes of PER vector pairs, `values` in all: as far
// as registers go. Measured at 20000 tokens of 20 heads of 80 (turned by 40,
// bf16: vectors of 4) and of 16 heads of 201 (4 pairs of single values): forward
// one token at once 58 and 102 us, two 78 and 113; backward 106 and 183, two 158
// and 334. Of 25751 x 20 heads of 45: forward 62 us with two or 64 with four,
// backward 114.
constexpr int at_once(int values, bool grad) {
    return grad ? (values <= 1 ? 4 : values <= 2 ? 2 : 1) : values <= 1 ? 2 : 1;
}
constexpr int forward_ctas(int values, int per) { return values <= 2 || per == 1 ? 4 : 3; }

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads, forward_ctas(V * PER, PER)) k_rope(const Args g) {
    pdl_wait();
    pdl_trigger();
    constexpr int N = at_once(V * PER, false);
    const int lane = threadIdx.x % G;
    const Columns<V, G, PER, HALVES> col(g, lane);
    const Walk<G> w(g);
    const Side& side = g.side[w.key];
    const TX* x_at = static_cast<const TX*>(side.x) + w.head * side.x_head;
    TX* y_at = static_cast<TX*>(side.y) + w.head * side.y_head;
    float wx[PER][V], wy[PER][V];
    load_weight(col, side.w, wx, wy);
    Head<TX, V, PER> next[N];
    Turns<V, PER> turns[N];
    int32_t next_pos[N];
    const int64_t x_step = w.step * side.x_token, y_step = w.step * side.y_token;
    const TX* x_next = x_at + w.t * side.x_token;
    const int32_t* pos_next = g.positions + w.t;
    int64_t t_next = w.t;
    const auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            next_pos[j] = -1;
            if (t_next < g.T) {
                next_pos[j] = *pos_next;
                if (w.in) next[j].fetch(col, x_next);
            }
            t_next += w.step;
            pos_next += w.step;
            x_next += x_step;
        }
    };
    fetch();
    y_at += w.t * side.y_token;
    for (int64_t t0 = w.t; t0 < g.T; t0 += N * w.step) {
        bool there[N];
        float x[N][PER][V], y[N][PER][V];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t pos = position_of(g, next_pos[j]);
            there[j] = pos >= 0;
            next[j].values(x[j], y[j]);
            if (there[j]) turns[j].load(g, col, pos);
        }
        fetch();
#pragma unroll
        for (int j = 0; j < N; ++j, y_at += y_step) {
            const int64_t t = t0 + j * w.step;
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) s = fmaf(x[j][i][k], x[j][i][k], fmaf(y[j][i][k], y[j][i][k], s));
            s = group_sum<G>(s);
            if (!w.in || t >= g.T) continue;
            if (there[j]) {
                const float rstd = rsqrtf(fmaf(s, g.inv_d, g.eps));
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        x[j][i][k] *= rstd * wx[i][k];
                        y[j][i][k] *= rstd * wy[i][k];
                    }
                turn<false, V, PER, HALVES>(x[j], y[j], turns[j]);
            } else {
                clear(x[j], y[j]);
            }
            store_head<V, G, PER, HALVES>(col, y_at, x[j], y[j]);
        }
    }
}

template <typename TX, int V, int G, int PER, bool HALVES>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    k_rope_grad(const Args g, float* __restrict__ parts) {
    extern __shared__ float rows[];  // [kWarps][2][D]
    pdl_wait();
    pdl_trigger();
    constexpr int N = at_once(V * PER, true);
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
    Head<TX, V, PER> next_x[N], next_g[N];
    Turns<V, PER> turns[N];
    int32_t next_pos[N];
    const int64_t x_step = w.step * side.x_token, y_step = w.step * side.y_token;
    const int64_t g_step = w.step * side.gy_token;
    const TX *x_next = x_at + w.t * side.x_token, *g_next = g_at + w.t * side.gy_token;
    const int32_t* pos_next = g.positions + w.t;
    int64_t t_next = w.t;
    const auto fetch = [&] {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            next_pos[j] = -1;
            if (t_next < g.T) {
                next_pos[j] = *pos_next;
                if (w.in) {
                    next_x[j].fetch(col, x_next);
                    next_g[j].fetch(col, g_next);
                }
            }
            t_next += w.step;
            pos_next += w.step;
            x_next += x_step;
            g_next += g_step;
        }
    };
    fetch();
    y_at += w.t * side.y_token;
    for (int64_t t0 = w.t; t0 < g.T; t0 += N * w.step) {
        bool there[N];
        float x[N][PER][V], y[N][PER][V], u[N][PER][V], v[N][PER][V];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int64_t pos = position_of(g, next_pos[j]);
            there[j] = pos >= 0;
            next_x[j].values(x[j], y[j]);
            next_g[j].values(u[j], v[j]);
            if (there[j]) turns[j].load(g, col, pos);
        }
        fetch();
#pragma unroll
        for (int j = 0; j < N; ++j, y_at += y_step) {
            const int64_t t = t0 + j * w.step;
            turn<true, V, PER, HALVES>(u[j], v[j], turns[j]);  // gm
            // sum x^2 and sum gm w x together; the root comes to the second later.
            float s = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < PER; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    s = fmaf(x[j][i][k], x[j][i][k], fmaf(y[j][i][k], y[j][i][k], s));
                    dot = fmaf(u[j][i][k] * wx[i][k], x[j][i][k], fmaf(v[j][i][k] * wy[i][k], y[j][i][k], dot));
                }
            s = group_sum<G>(s);
            dot = group_sum<G>(dot);
            if (!w.in || t >= g.T) continue;
            if (there[j]) {
                const float rstd = rsqrtf(fmaf(s, g.inv_d, g.eps));
                dot *= rstd * g.inv_d;
#pragma unroll
                for (int i = 0; i < PER; ++i)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        x[j][i][k] *= rstd;  // n
                        y[j][i][k] *= rstd;
                        sx[i][k] = fmaf(u[j][i][k], x[j][i][k], sx[i][k]);
                        sy[i][k] = fmaf(v[j][i][k], y[j][i][k], sy[i][k]);
                        u[j][i][k] = rstd * fmaf(-x[j][i][k], dot, u[j][i][k] * wx[i][k]);
                        v[j][i][k] = rstd * fmaf(-y[j][i][k], dot, v[j][i][k] * wy[i][k]);
                    }
            } else {
                clear(u[j], v[j]);
            }
            store_head<V, G, PER, HALVES>(col, y_at, u[j], v[j]);
        }
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
    join_rows(g, rows, parts);
}

// ---- vectors of 16 bytes

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copies_landed() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 16 bytes as numbers, in twos, and back.
template <typename TX, int N>
__device__ __forceinline__ void unpack(const uint4& q, float2 (&v)[N]) {
    const uint32_t r[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = sizeof(TX) == 2
                   ? make_float2(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u))
                   : make_float2(__uint_as_float(r[(2 * i) % 4]), __uint_as_float(r[(2 * i + 1) % 4]));
}
template <typename TX, int N>
__device__ __forceinline__ uint4 pack(const float2 (&v)[N]) {
    if constexpr (sizeof(TX) == 2) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                          __float_as_uint(v[1].y));
    }
}

template <int N>
__device__ __forceinline__ void load_twos(const float* p, float2 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float4 q = reinterpret_cast<const float4*>(p)[i];
        v[2 * i] = make_float2(q.x, q.y);
        v[2 * i + 1] = make_float2(q.z, q.w);
    }
}

// A lane's place in its head: a pair of vectors, wholly turned or not at all.
// Lanes past the last pair stand at the first one and neither add nor write.
template <typename TX, int G, bool HALVES>
struct Place {
    static constexpr int V = 16 / static_cast<int>(sizeof(TX));
    int a, b, turn;   // first values of its vectors, its first angle
    bool own, turned;

    __device__ explicit Place(const Args& g) {
        const int lane = threadIdx.x % G;
        own = lane < g.pairs;
        const int p = own ? lane : 0;
        if (HALVES) {
            turned = p < g.turned;
            a = turned ? p * V : g.rot + 2 * (p - g.turned) * V;
            b = turned ? a + g.rot / 2 : a + V;
            turn = a;
        } else {
            a = 2 * p * V;
            b = a + V;
            turned = a < g.rot;
            turn = a / 2;
        }
    }
};

// Turns x and y by c and s (BACK: the other way round). Pairs: x has the first
// V / 2 turns, y the others.
template <bool BACK, bool HALVES, int N>
__device__ __forceinline__ void turn_twos(float2 (&x)[N], float2 (&y)[N], const float2 (&c)[N],
                                          const float2 (&s)[N]) {
    if constexpr (HALVES) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 n = make_float2(-s[i].x, -s[i].y), u = x[i], v = y[i];
            x[i] = fma2(v, BACK ? s[i] : n, mul2(u, c[i]));
            y[i] = fma2(u, BACK ? n : s[i], mul2(v, c[i]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 2 * N; ++k) {
            float2& z = k < N ? x[k] : y[k - N];
            const float ck = k & 1 ? c[k / 2].y : c[k / 2].x, sk = k & 1 ? s[k / 2].y : s[k / 2].x;
            z = fma2(make_float2(z.y, z.x), BACK ? make_float2(sk, -sk) : make_float2(-sk, sk),
                     mul2(z, both(ck)));
        }
    }
}

template <int N>
__device__ __forceinline__ float dot_twos(const float2 (&x)[N], const float2 (&y)[N], const float2 (&u)[N],
                                          const float2 (&v)[N]) {
    float2 s = mul2(x[0], u[0]), t = mul2(y[0], v[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) {
        s = fma2(x[i], u[i], s);
        t = fma2(y[i], v[i], t);
    }
    s = add2(s, t);
    return s.x + s.y;
}

// One warp's way through its tokens: positions, angles and values ahead.
template <typename TX, int G, bool HALVES, bool GRAD>
struct Stream {
    using P = Place<TX, G, HALVES>;
    static constexpr int N = P::V / 2, kVecs = GRAD ? 4 : 2;
    static constexpr int kBytes = kThreads * kVecs * 16;  // of a token in the ring
    const Args& g;
    const Walk<G> w;
    const P at;
    const TX *x, *gy;        // the next token to fetch
    TX* y;                   // the token at hand
    int64_t x_step, gy_step, y_step, ahead;
    const int32_t* position;
    int32_t next;            // position of the token after the one at hand
    uint32_t ring;
    const unsigned char* mine;
    int slot = 0, free = 0;
    float2 c[N], s[N];

    __device__ Stream(const Args& args, unsigned char* smem) : g(args), w(args), at(args) {
        const Side& side = g.side[w.key];
        x = static_cast<const TX*>(side.x) + w.head * side.x_head + w.t * side.x_token;
        y = static_cast<TX*>(side.y) + w.head * side.y_head + w.t * side.y_token;
        x_step = w.step * side.x_token;
        y_step = w.step * side.y_token;
        if (GRAD) {
            gy = static_cast<const TX*>(side.gy) + w.head * side.gy_head + w.t * side.gy_token;
            gy_step = w.step * side.gy_token;
        }
        position = g.positions + w.t;
        mine = smem + threadIdx.x * 16;
        ring = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
        ahead = w.t;
        next = w.t < g.T ? *position : -1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            c[i] = both(1.0f);
            s[i] = both(0.0f);
        }
#pragma unroll
        for (int i = 0; i < kRing; ++i) fetch();
    }

    __device__ __forceinline__ void fetch() {
        if (ahead < g.T) {
            const uint32_t to = ring + free * kBytes;
            copy16(to, x + at.a);
            copy16(to + kThreads * 16, x + at.b);
            x += x_step;
            if (GRAD) {
                copy16(to + 2 * kThreads * 16, gy + at.a);
                copy16(to + 3 * kThreads * 16, gy + at.b);
                gy += gy_step;
            }
        }
        copies_begun();
        ahead += w.step;
        free = free + 1 == kRing ? 0 : free + 1;
    }

    // The k-th vector of the token at hand.
    __device__ __forceinline__ uint4 vec(int k) const {
        return *reinterpret_cast<const uint4*>(mine + slot * kBytes + k * kThreads * 16);
    }

    // The position of token t, -1 where it is padding, and its angles.
    __device__ __forceinline__ bool begin(int64_t t) {
        const int64_t pos = position_of(g, next);
        position += w.step;
        if (t + w.step < g.T) next = *position;
        if (at.turned && pos >= 0) {
            const int64_t from = pos * (g.rot / 2) + at.turn;
            load_twos(g.cosine + from, c);
            load_twos(g.sine + from, s);
        }
        copies_landed<kRing - 1>();
        return pos >= 0;
    }

    __device__ __forceinline__ void end() {
        slot = slot + 1 == kRing ? 0 : slot + 1;
        y += y_step;
        fetch();
    }

    __device__ __forceinline__ void write(const float2 (&a)[N], const float2 (&b)[N]) const {
        if (!at.own || !w.in) return;
        *reinterpret_cast<uint4*>(y + at.a) = pack<TX>(a);
        *reinterpret_cast<uint4*>(y + at.b) = pack<TX>(b);
    }

    // The head's weights at the lane's columns, 1 where there are none.
    __device__ void weights(float2 (&a)[N], float2 (&b)[N]) const {
        const float* p = g.side[w.key].w;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = p ? make_float2(p[at.a + 2 * i], p[at.a + 2 * i + 1]) : both(1.0f);
            b[i] = p ? make_float2(p[at.b + 2 * i], p[at.b + 2 * i + 1]) : both(1.0f);
        }
    }
};

template <typename TX, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads, kForwardCtas) k_rope_fast(const Args g) {
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_wait();
    pdl_trigger();
    Stream<TX, G, HALVES, false> f(g, ring);
    constexpr int N = decltype(f)::N;
    float2 wx[N], wy[N];
    f.weights(wx, wy);
    for (int64_t t = f.w.t; t < g.T; t += f.w.step) {
        const bool there = f.begin(t);
        float2 x[N], y[N];
        unpack<TX>(f.vec(0), x);
        unpack<TX>(f.vec(1), y);
        if (there) {
            const float s = group_sum<G>(f.at.own ? dot_twos(x, y, x, y) : 0.0f);
            const float2 r = both(rsqrtf(fmaf(s, g.inv_d, g.eps)));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = mul2(mul2(x[i], r), wx[i]);
                y[i] = mul2(mul2(y[i], r), wy[i]);
            }
            turn_twos<false, HALVES>(x, y, f.c, f.s);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = y[i] = both(0.0f);
        }
        f.write(x, y);
        f.end();
    }
}

template <typename TX, int G, bool HALVES>
__global__ void __launch_bounds__(kThreads, kBackwardCtas)
    k_rope_grad_fast(const Args g, float* __restrict__ parts) {
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_wait();
    pdl_trigger();
    Stream<TX, G, HALVES, true> f(g, ring);
    constexpr int N = decltype(f)::N;
    float2 wx[N], wy[N], sx[N], sy[N];  // weights, sums of gm n
    f.weights(wx, wy);
#pragma unroll
    for (int i = 0; i < N; ++i) sx[i] = sy[i] = both(0.0f);
    for (int64_t t = f.w.t; t < g.T; t += f.w.step) {
        const bool there = f.begin(t);
        float2 x[N], y[N], u[N], v[N];
        unpack<TX>(f.vec(0), x);
        unpack<TX>(f.vec(1), y);
        unpack<TX>(f.vec(2), u);
        unpack<TX>(f.vec(3), v);
        if (there) {
            turn_twos<true, HALVES>(u, v, f.c, f.s);  // gm
            float s = f.at.own ? dot_twos(x, y, x, y) : 0.0f;
            s = group_sum<G>(s);
            const float rstd = rsqrtf(fmaf(s, g.inv_d, g.eps));
            const float2 r = both(rstd);
            float2 dots = both(0.0f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                x[i] = mul2(x[i], r);  // n
                y[i] = mul2(y[i], r);
                sx[i] = fma2(u[i], x[i], sx[i]);
                sy[i] = fma2(v[i], y[i], sy[i]);
                u[i] = mul2(u[i], wx[i]);
                v[i] = mul2(v[i], wy[i]);
                dots = fma2(u[i], x[i], fma2(v[i], y[i], dots));
            }
            const float dot = group_sum<G>(f.at.own ? dots.x + dots.y : 0.0f) * g.inv_d;
            const float2 m = both(-dot);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                u[i] = mul2(r, fma2(x[i], m, u[i]));
                v[i] = mul2(r, fma2(y[i], m, v[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) u[i] = v[i] = both(0.0f);
        }
        f.write(u, v);
        f.end();
    }
    if (!parts) return;
    copies_landed<0>();
    __syncthreads();  // the ring is done with: the sums take its place
    float* rows = reinterpret_cast<float*>(ring);
    float* mine = rows + static_cast<int>(threadIdx.x) / 32 * 2 * g.D;
    for (int i = threadIdx.x % 32; i < 2 * g.D; i += 32) mine[i] = 0.0f;
    __syncwarp();
    for (int k = 0; k < 32 / G; ++k) {
        if (static_cast<int>(threadIdx.x) % 32 / G == k && f.w.in && f.at.own) {
            float* to = mine + (f.w.key ? g.D : 0);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                to[f.at.a + 2 * i] += sx[i].x;
                to[f.at.a + 2 * i + 1] += sx[i].y;
                to[f.at.b + 2 * i] += sy[i].x;
                to[f.at.b + 2 * i + 1] += sy[i].y;
            }
        }
        __syncwarp();
    }
    join_rows(g, rows, parts);
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
                          dim3(grid_of(g.T, g.heads, 32 / G, 152 * forward_ctas(V * PER, PER))), dim3(kThreads), 0, l.s, g);
    *l.n_parts = grid_of(g.T, g.heads, 32 / G, kMaxCtas);
    return launch_pdl(k_rope_grad<TX, V, G, PER, HALVES>, dim3(*l.n_parts), dim3(kThreads),
                      sizeof(float) * 2 * kWarps * static_cast<size_t>(g.D), l.s, g, l.parts);
}

template <typename TX, int G, bool HALVES>
cudaError_t launch_fast(const Args& g, const Launch& l) {
    using F = Stream<TX, G, HALVES, false>;
    using B = Stream<TX, G, HALVES, true>;
    if (!l.grad) {
        const void* k = reinterpret_cast<const void*>(k_rope_fast<TX, G, HALVES>);
        DUST_TRY(ensure_smem_limit(k, kRing * F::kBytes));
        return launch_pdl(k_rope_fast<TX, G, HALVES>,
                          dim3(grid_of(g.T, g.heads, 32 / G, 152 * kForwardCtas)), dim3(kThreads),
                          kRing * F::kBytes, l.s, g);
    }
    *l.n_parts = grid_of(g.T, g.heads, 32 / G, kMaxCtas);
    const size_t smem = std::max<size_t>(kRing * B::kBytes, sizeof(float) * 2 * kWarps * static_cast<size_t>(g.D));
    const void* k = reinterpret_cast<const void*>(k_rope_grad_fast<TX, G, HALVES>);
    DUST_TRY(ensure_smem_limit(k, kRing * B::kBytes));
    return launch_pdl(k_rope_grad_fast<TX, G, HALVES>, dim3(*l.n_parts), dim3(kThreads), smem, l.s, g, l.parts);
}

template <typename TX, bool HALVES>
cudaError_t launch_vectors(const Args& g, int V, const Launch& l) {
    if (V * static_cast<int>(sizeof(TX)) == 16 && g.pairs <= 32)
        return g.pairs <= 2    ? launch_fast<TX, 2, HALVES>(g, l)
               : g.pairs <= 4  ? launch_fast<TX, 4, HALVES>(g, l)
               : g.pairs <= 8  ? launch_fast<TX, 8, HALVES>(g, l)
               : g.pairs <= 16 ? launch_fast<TX, 16, HALVES>(g, l)
                               : launch_fast<TX, 32, HALVES>(g, l);
    if constexpr (sizeof(TX) == 2)
        if (V == 4)
            return g.pairs <= 8    ? launch_with<TX, 4, 8, 1, HALVES>(g, l)
                   : g.pairs <= 16 ? launch_with<TX, 4, 16, 1, HALVES>(g, l)
                   : g.pairs <= 32 ? launch_with<TX, 4, 32, 1, HALVES>(g, l)
                                   : launch_with<TX, 4, 32, 2, HALVES>(g, l);
    if (V >= 2)
        return g.pairs <= 8    ? launch_with<TX, 2, 8, 1, HALVES>(g, l)
               : g.pairs <= 16 ? launch_with<TX, 2, 16, 1, HALVES>(g, l)
               : g.pairs <= 32 ? launch_with<TX, 2, 32, 1, HALVES>(g, l)
               : g.pairs <= 64 ? launch_with<TX, 2, 32, 2, HALVES>(g, l)
                               : launch_with<TX, 2, 32, 4, HALVES>(g, l);
    return g.pairs <= 8     ? launch_with<TX, 1, 8, 1, HALVES>(g, l)
           : g.pairs <= 16  ? launch_with<TX, 1, 16, 1, HALVES>(g, l)
           : g.pairs <= 32  ? launch_with<TX, 1, 32, 1, HALVES>(g, l)
           : g.pairs <= 64  ? launch_with<TX, 1, 32, 2, HALVES>(g, l)
           : g.pairs <= 128 ? launch_with<TX, 1, 32, 4, HALVES>(g, l)
                            : launch_with<TX, 1, 32, 8, HALVES>(g, l);
}

cudaError_t run(const RopeProblem& p, const Launch& l) {
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
        // From 4 values on the tables' vectors are 16 bytes too; and of 16 bytes,
        // whole pairs of vectors, each turned or not.
        return v == 2 || (p.rot % (2 * v) == 0 && (v * size < 16 || p.D % (2 * v) == 0) &&
                          (p.rot == 0 || (reinterpret_cast<uintptr_t>(p.cosine) |
                                          reinterpret_cast<uintptr_t>(p.sine)) % 16 == 0));
    };
    if (!fits(V) || p.D > 64 * V) V = p.bf16 && fits(4) ? 4 : fits(2) ? 2 : 1;
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
