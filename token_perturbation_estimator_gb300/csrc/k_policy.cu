// A policy's clipped loss with a KL term on per-token losses, and its gradient
// (include/dust.h gives the formulas).
//
// A first pass finds each token's sequence and counts the scored tokens (whole
// numbers, so that the order of the additions does not show); a second one
// forms the tokens' losses, or gradients, whose weights come from those counts,
// and leaves each CTA's sums, which the CTA that is done last adds up in order.
// Few tokens go through all of it in one CTA and one launch.
//
// Bound by latency: clearing, counting, one wave of CTAs that start, wait for
// their first values and join, one after another. One slice of 65536 tokens takes
// 14.5 us, 33 of them 24.7. A loss takes about 115 instructions (two exponentials,
// a series, the sums), which are a third of the second pass (36 % of its cycles
// issue one, 58 % of those in which an SM has work), and its 12 bytes a value less;
// each group of slices forms the clean one's losses again. A gradient of one slice
// takes 9.2 us, 1531 tokens 4.7 (7 alone).
//
// The losses' signs cancel in their mean, so that it is added up in 64 bits beyond
// a thread's 4 tokens, or with what roundings lose, and what the weights'
// roundings leave (of the counts, their product and its inverse) is added as
// well. Whether a ratio is beyond its bound is decided in fp32 where that is
// certain, else in 64 bits, of which the GPU does a 64th as many a second: in 64
// bits throughout, 33 slices took 48 us.
#include <algorithm>
#include <cmath>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kSlices = 5;   // slices that a CTA takes, at most
constexpr int kPer = 4;      // tokens that a thread takes
constexpr int kTokens = kThreads * kPer;
constexpr int kCountTokens = 512;            // of a CTA of the first pass, one a thread
constexpr int kWindow = kCountTokens + 1;    // sequences' starts that it holds

struct Counts {
    int32_t tokens, sequences;  // scored, with scored tokens
    unsigned int done;          // CTAs of the second pass that have left their sums
};

struct Space {
    Counts* counts;
    int32_t* of_seq;   // [n_seq] scored tokens
    int32_t* seq_of;   // [T] sequence of a scored token, or -1
    double* parts;     // [blocks][S][3]
    size_t clear;      // bytes that start at 0, from counts on
    size_t total;
};

int64_t blocks_of(int64_t T) { return (T + kTokens - 1) / kTokens; }
int64_t groups_of(int64_t S) { return (S + kSlices - 1) / kSlices; }

Space carve(void* ws, int64_t S, int64_t T, int64_t n_seq) {
    unsigned char* base = static_cast<unsigned char*>(ws);
    size_t at = 0;
    const auto take = [&](int64_t bytes) {
        unsigned char* p = base ? base + at : nullptr;
        at += (static_cast<size_t>(bytes) + 255) & ~static_cast<size_t>(255);
        return p;
    };
    Space w;
    w.counts = reinterpret_cast<Counts*>(take(256));
    w.of_seq = reinterpret_cast<int32_t*>(take(4 * n_seq));
    w.clear = at;
    w.seq_of = reinterpret_cast<int32_t*>(take(4 * T));
    w.parts = reinterpret_cast<double*>(take(24 * blocks_of(T) * S));
    w.total = at;
    return w;
}

// How many of the sequences' n starts (and the last one's end) are at or before
// token t; whole warp. The starts do not decrease, so it narrows a range down
// to one, 32 parts at a time; whatever they are, it ends and stays inside.
__device__ __forceinline__ int64_t starts_until(const int32_t* offsets, int64_t n, int64_t t) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const bool before = at < hi && offsets[at] <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, before));
        hi = min(hi, lo + k * step);
        lo = k == 0 ? hi : lo + (k - 1) * step + 1;
    }
    return lo;
}

// The same by one thread.
__device__ __forceinline__ int64_t starts_until_alone(const int32_t* offsets, int64_t n, int64_t t) {
    int64_t lo = 0, hi = n;
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The starts around a CTA's tokens, from the first one's sequence on, or all
// starts where they are few.
struct Window {
    int64_t first;  // number of the first start held, -1 where the first token precedes all
    int32_t at[kWindow];

    __device__ void load(const int32_t* offsets, int64_t n_seq, int64_t t0) {
        if (n_seq < kWindow) {  // all of them
            if (threadIdx.x == 0) first = 0;
        } else if (threadIdx.x < 32) {
            const int64_t k = starts_until(offsets, n_seq + 1, t0);
            if (threadIdx.x == 0) first = k - 1;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kWindow; i += blockDim.x) {
            const int64_t k = first + i;
            at[i] = k < 0 ? INT32_MIN : k <= n_seq ? offsets[k] : INT32_MAX;
        }
        __syncthreads();
    }

    // The sequence of token t, or -1; held: whether its start is.
    __device__ int32_t sequence(const int32_t* offsets, int64_t n_seq, int64_t t, bool& held) const {
        int lo = 0, hi = kWindow;  // starts held that are at or before t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (at[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        int64_t seq = first + lo - 1;
        held = lo < kWindow;
        if (!held)  // more sequences than tokens: empty ones
            seq = starts_until_alone(offsets, n_seq + 1, t) - 1;
        return seq >= 0 && seq < n_seq ? static_cast<int32_t>(seq) : -1;
    }
};

__device__ __forceinline__ bool has_target(const PolicyProblem& p, int64_t t) {
    return t < p.T && (!p.targets || p.targets[t] >= 0);
}

// Adds 1 at each lane's place (-1: none), one addition per warp and place.
__device__ __forceinline__ void count_places(int32_t place, int32_t* counts) {
    const unsigned same = __match_any_sync(0xffffffffu, place);
    if (place >= 0 && __ffs(same) - 1 == static_cast<int>(threadIdx.x & 31))
        atomicAdd(counts + place, __popc(same));
}

// The tokens of each sequence are counted in shared memory, then added to the
// others' once per sequence: additions that return a value take a microsecond
// each.
__global__ void __launch_bounds__(kCountTokens)
    k_policy_count(const PolicyProblem p, Counts* counts, int32_t* of_seq, int32_t* __restrict__ seq_of) {
    __shared__ Window window;
    __shared__ int32_t here[kWindow];
    pdl_wait();
    pdl_trigger();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kCountTokens + threadIdx.x;
    const bool has = has_target(p, t);
    for (int i = threadIdx.x; i < kWindow; i += kCountTokens) here[i] = 0;
    window.load(p.offsets, p.n_seq, static_cast<int64_t>(blockIdx.x) * kCountTokens);
    bool held = true;
    const int32_t seq = has ? window.sequence(p.offsets, p.n_seq, t, held) : -1;
    if (t < p.T) seq_of[t] = seq;
    count_places(seq >= 0 && held ? static_cast<int32_t>(seq - window.first) : -1, here);
    int opened = 0;
    if (seq >= 0 && !held) opened = atomicAdd(of_seq + seq, 1) == 0;
    const int scored = __syncthreads_count(seq >= 0);
    for (int i = threadIdx.x; i < kWindow; i += kCountTokens)
        if (here[i] > 0) opened += atomicAdd(of_seq + window.first + i, here[i]) == 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) opened += __shfl_xor_sync(0xffffffffu, opened, off);
    if (opened > 0 && (threadIdx.x & 31) == 0) atomicAdd(&counts->sequences, opened);
    if (threadIdx.x == 0 && scored > 0) atomicAdd(&counts->tokens, scored);
}

// exp(r) - r - 1 without cancellation: its series where |r| < 1 (what it leaves
// out is below 2^-27 of it).
__device__ __forceinline__ float kl_of(float r) {
    float s = 1.0f / 479001600.0f;  // 1 / 12!
    s = fmaf(s, r, 1.0f / 39916800.0f);
    s = fmaf(s, r, 1.0f / 3628800.0f);
    s = fmaf(s, r, 1.0f / 362880.0f);
    s = fmaf(s, r, 1.0f / 40320.0f);
    s = fmaf(s, r, 1.0f / 5040.0f);
    s = fmaf(s, r, 1.0f / 720.0f);
    s = fmaf(s, r, 1.0f / 120.0f);
    s = fmaf(s, r, 1.0f / 24.0f);
    s = fmaf(s, r, 1.0f / 6.0f);
    s = fmaf(s, r, 0.5f);
    const float far = expf(r) - (1.0f + r);
    return fabsf(r) < 1.0f ? s * r * r : far;
}

// What the rounding of a count v >= 0 to f leaves (2^31, which it may round to,
// fits 32 bits without a sign).
__device__ __forceinline__ float beyond_fp32(int32_t v, float f) {
    return static_cast<float>(static_cast<int32_t>(static_cast<uint32_t>(v) - static_cast<uint32_t>(f)));
}

// What a token needs of everything but nll.
struct Token {
    bool scored;
    float old, ref, adv;
    float weight, rest;  // and what its rounding leaves, the same for a whole sequence

    __device__ __forceinline__ void load(const PolicyProblem& p, const Counts& c, const int32_t* of_seq,
                                         int32_t seq, int64_t t) {
        scored = seq >= 0;
        old = ref = adv = weight = rest = 0.0f;
        if (!scored) return;
        old = p.old[t];
        ref = p.ref ? p.ref[t] : 0.0f;
        adv = p.advantages[p.per_token ? t : seq];
        // The tokens that share the mean: a product that has up to 62 bits, as n and
        // what is beyond it.
        const int32_t a = p.by_sequence ? c.sequences : 1, b = p.by_sequence ? of_seq[seq] : c.tokens;
        const float fa = static_cast<float>(a), fb = static_cast<float>(b), n = fa * fb;
        const float beyond = fmaf(beyond_fp32(a, fa), fb, fmaf(fa, beyond_fp32(b, fb), fmaf(fa, fb, -n)));
        weight = 1.0f / n;
        rest = fmaf(-weight, beyond, fmaf(-weight, n, 1.0f)) * weight;
    }
};

// Whether the ratio is beyond the bound on its advantage's side. The fp32
// difference is off by half a step, as the bound is: further apart than 4
// steps, they stand as the exact ones do, and what is nearer is rare. An infinite
// bound is the exception: everything seems near it and is decided all the same,
// which is asked last, as it would cost the common way 2 per cent. (With all
// tokens in 64 bits there, 33 slices of 65536 tokens took 46 us without a bound.)
struct Side {
    bool beyond, near;
    float bound;

    __device__ __forceinline__ Side(const PolicyProblem& p, const Token& k, float nll) {
        const bool up = k.adv > 0.0f;
        bound = up ? p.high32 : p.low32;
        const float step = k.old - nll;
        near = !(fabsf(step - bound) > 0x1p-22f * fabsf(bound));
        beyond = up ? step > bound : k.adv < 0.0f && step < bound;
    }
    __device__ __forceinline__ bool open() const { return near && !isinf(bound); }
    // Decided in 64 bits. A call of its own: in line, the compiler would
    // form the exact differences of every value.
    static __device__ __noinline__ bool exactly(const PolicyProblem& p, float adv, float old, float nll) {
        const double step = static_cast<double>(old) - static_cast<double>(nll);
        return adv > 0.0f ? step > p.high : adv < 0.0f && step < p.low;
    }
};

// The ratio that the advantage is multiplied by: exp(step), but finite where the
// product is 0 whatever it is.
__device__ __forceinline__ float ratio_of(float step, float adv) {
    return expf(adv == 0.0f && step > 0.0f ? 0.0f : step);
}

// N tokens' losses side by side, without branches but for the rare ones.
template <int N>
__device__ __forceinline__ void losses_of(const PolicyProblem& p, const Token (&k)[N], const float (&nll)[N],
                                          float (&loss)[N], float (&kl)[N], bool (&clipped)[N]) {
    bool near = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const Side d(p, k[i], nll[i]);
        clipped[i] = d.beyond;
        near |= d.near;
    }
    if (near)
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (Side(p, k[i], nll[i]).open()) clipped[i] = Side::exactly(p, k[i].adv, k[i].old, nll[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float bound = k[i].adv > 0.0f ? p.most : p.least;
        const float ratio = ratio_of(k[i].old - nll[i], k[i].adv);
        loss[i] = -(clipped[i] ? bound : ratio) * k[i].adv;
        kl[i] = 0.0f;
        if (p.ref) {
            kl[i] = kl_of(nll[i] - k[i].ref);
            if (p.beta != 0.0f) loss[i] = fmaf(p.beta, kl[i], loss[i]);
        }
        if (!k[i].scored) {
            loss[i] = kl[i] = 0.0f;
            clipped[i] = false;
        }
    }
}

__device__ __forceinline__ float slope_of(const PolicyProblem& p, const Token& k, float nll) {
    Side d(p, k, nll);
    if (d.open()) d.beyond = Side::exactly(p, k.adv, k.old, nll);
    float g = d.beyond ? 0.0f : ratio_of(k.old - nll, k.adv) * k.adv;
    if (p.ref && p.beta != 0.0f) g = fmaf(p.beta, expm1f(nll - k.ref), g);
    return g;
}

// A sum over the lanes: of terms of one sign (the KL term, clipped tokens) ...
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// ... and of the losses, whose signs cancel: what the roundings lose (and have
// lost) is added up as well (Knuth), and counts unless the sum has overflowed,
// where it is no number. In fp32, the sum of 12 sequences' 325 tokens was 1.2e-6
// off where its losses' own roundings make 0.8e-6.
__device__ __forceinline__ double with_rest(double v, double lost) { return isfinite(v) ? v + lost : v; }
__device__ __forceinline__ void add_exactly(float& v, float& lost, float u) {
    const float s = v + u, t = s - v;
    lost += (v - (s - t)) + (u - t);
    v = s;
}
__device__ __forceinline__ double warp_sum_exact(float v, float lost) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        lost += __shfl_xor_sync(0xffffffffu, lost, off);
        add_exactly(v, lost, __shfl_xor_sync(0xffffffffu, v, off));
    }
    return with_rest(v, lost);
}

struct Outputs {
    float *loss, *total, *kl, *clipped, *delta;
};

// The CTAs' sums [blocks][n] added up: each column by a power of two of threads,
// then theirs by halves.
__device__ __forceinline__ void join_parts(const double* parts, int64_t blocks, int64_t n, const Outputs& o) {
    __shared__ double sh[kThreads];
    for (int64_t c0 = 0; c0 < n; c0 += kThreads) {
        const int cols = static_cast<int>(min(n - c0, static_cast<int64_t>(kThreads)));
        const int turns = 1 << (31 - __clz(kThreads / cols)), c = threadIdx.x % cols, turn = threadIdx.x / cols;
        double v = 0.0;
        if (turn < turns)
#pragma unroll 8
            for (int64_t b = turn; b < blocks; b += turns) v += __ldcg(parts + b * n + c0 + c);
        sh[threadIdx.x] = v;
        __syncthreads();
        for (int h = turns / 2; h > 0; h /= 2) {
            if (turn < h) sh[threadIdx.x] += sh[threadIdx.x + h * cols];
            __syncthreads();
        }
        if (turn == 0) {
            const int64_t s = (c0 + c) / 3;
            float* out = (c0 + c) % 3 == 0 ? o.total : (c0 + c) % 3 == 1 ? o.kl : o.clipped;
            if (out) out[s] = static_cast<float>(sh[threadIdx.x]);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads, 3)
    k_policy(const PolicyProblem p, const Outputs o, int64_t blocks, int64_t groups, Counts* counts,
             const int32_t* __restrict__ of_seq, const int32_t* __restrict__ seq_of, double* parts) {
    pdl_wait();
    pdl_trigger();
    __shared__ float losses[kSlices][kThreads];  // each thread's
    __shared__ float sums[kThreads / 32][kSlices][3];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t block = blockIdx.x % blocks, group = blockIdx.x / blocks;
    const int64_t t0 = block * kTokens + threadIdx.x;
    const int s0 = static_cast<int>(p.S * group / groups), s1 = static_cast<int>(p.S * (group + 1) / groups);
    const int here = static_cast<int>(min(p.T - block * kTokens, static_cast<int64_t>(kTokens)));
    // This thread's tokens that there are, the first one's place in its slice.
    const int mine = max(0, (here - static_cast<int>(threadIdx.x) + kThreads - 1) / kThreads);
    const float* nll = p.nll + s0 * p.T + t0;
    Token k[kPer];
    float clean[kPer], next[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        next[i] = i < mine ? nll[i * kThreads] : 0.0f;
        clean[i] = o.delta && i < mine ? p.nll[t0 + i * kThreads] : 0.0f;
    }
    const Counts c = *counts;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        k[i].load(p, c, of_seq, i < mine ? seq_of[t0 + i * kThreads] : -1, t0 + i * kThreads);
    float l[kPer], kl[kPer];
    bool clipped[kPer];
    if (o.delta) {
        losses_of(p, k, clean, l, kl, clipped);
#pragma unroll
        for (int i = 0; i < kPer; ++i) clean[i] = l[i];
    }
    float* loss = o.loss ? o.loss + s0 * p.T + t0 : nullptr;
    float* delta = o.delta ? o.delta + (s0 - 1) * p.T + t0 : nullptr;
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        float now[kPer];
        nll += p.T;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            now[i] = next[i];
            if (s + 1 < s1 && i < mine) next[i] = nll[i * kThreads];
        }
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        losses_of(p, k, now, l, kl, clipped);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            sum[0] = fmaf(k[i].weight, l[i], sum[0]);
            sum[3] = fmaf(k[i].rest, l[i], sum[3]);
            sum[1] = fmaf(k[i].weight, kl[i], sum[1]);
            if (clipped[i]) sum[2] += k[i].weight;
            if (loss && i < mine) loss[i * kThreads] = l[i];
            if (delta && s > 0 && i < mine) delta[i * kThreads] = l[i] - clean[i];
        }
        if (loss) loss += p.T;
        if (delta) delta += p.T;
        losses[s - s0][threadIdx.x] = sum[0];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            sum[j + 1] = warp_sum(sum[j + 1]);
            if (lane == 0) sums[warp][s - s0][j] = sum[j + 1];
        }
    }
    if (!o.total && !o.kl && !o.clipped) return;
    __syncthreads();
    // The losses' signs cancel: their sums in 64 bits, a warp per slice.
    for (int s = warp; s < s1 - s0; s += kThreads / 32) {
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) v += static_cast<double>(losses[s][32 * i + lane]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        float own = 0.0f;
        if (lane < 3)
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) own += sums[w][s][lane];
        const double rest = static_cast<double>(__shfl_sync(0xffffffffu, own, 2));
        double* to = parts + (block * p.S + s0 + s) * 3;
        if (lane < 2) __stcg(to + 1 + lane, static_cast<double>(own));
        if (lane == 0) __stcg(to, with_rest(v, rest));
    }
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) last = atomicAdd(&counts->done, 1u) + 1 == gridDim.x;
    __syncthreads();
    if (!last) return;
    __threadfence();
    join_parts(parts, blocks, 3 * p.S, o);
}

__global__ void __launch_bounds__(kThreads)
    k_policy_grad(const PolicyProblem p, int64_t blocks, int64_t groups, const Counts* counts,
                  const int32_t* __restrict__ of_seq, const int32_t* __restrict__ seq_of,
                  const float* __restrict__ gtotal, float* gnll) {
    pdl_wait();
    pdl_trigger();
    const Counts c = *counts;
    const int64_t t = blockIdx.x % blocks * kThreads + threadIdx.x, group = blockIdx.x / blocks;
    if (t >= p.T) return;
    Token k;
    k.load(p, c, of_seq, seq_of[t], t);
    const int64_t s0 = p.S * group / groups, s1 = p.S * (group + 1) / groups;
#pragma unroll 2
    for (int64_t s = s0; s < s1; ++s)
        gnll[s * p.T + t] = k.scored ? gtotal[s] * k.weight * slope_of(p, k, p.nll[s * p.T + t]) : 0.0f;
}

// Few tokens: everything by one CTA, the counts in shared memory. The sums are
// a warp's 32 tokens' at a time, then its turns', then the warps', in order.
constexpr int kFewThreads = 1024;
constexpr int kFewTokens = 2 * kFewThreads, kFewSequences = 4096, kFewSlices = 4;

template <bool GRAD>
__global__ void __launch_bounds__(kFewThreads)
    k_policy_few(const PolicyProblem p, const Outputs o, const float* __restrict__ gtotal, float* gnll) {
    __shared__ Counts counts;
    __shared__ int32_t of_seq[kFewSequences];
    __shared__ double sums[kFewThreads / 32][kFewSlices][3];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = static_cast<int>(p.T), S = static_cast<int>(p.S);
    for (int i = threadIdx.x; i < p.n_seq; i += kFewThreads) of_seq[i] = 0;
    if (threadIdx.x == 0) counts = {0, 0, 0};
    __syncthreads();
    int32_t seq[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = i * kFewThreads + threadIdx.x;
        seq[i] = -1;
        if (has_target(p, t)) {
            const int64_t k = starts_until_alone(p.offsets, p.n_seq + 1, t) - 1;
            if (k >= 0 && k < p.n_seq) seq[i] = static_cast<int32_t>(k);
        }
        count_places(seq[i], of_seq);
    }
    const int scored = __syncthreads_count(seq[0] >= 0) + __syncthreads_count(seq[1] >= 0);
    int open = 0;
    for (int i0 = 0; i0 < p.n_seq; i0 += kFewThreads) {
        const int i = i0 + threadIdx.x;
        open += __syncthreads_count(i < p.n_seq && of_seq[i] > 0);
    }
    if (threadIdx.x == 0) counts = {scored, open, 0};
    __syncthreads();
    float sum[kFewSlices][4] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = i * kFewThreads + threadIdx.x;
        if (t >= T) continue;
        Token k;
        k.load(p, counts, of_seq, seq[i], t);
        float clean = 0.0f;
#pragma unroll
        for (int s = 0; s < kFewSlices; ++s) {
            if (s >= S) continue;
            const float nll = p.nll[s * T + t];
            if constexpr (GRAD) {
                gnll[s * T + t] = k.scored ? gtotal[s] * k.weight * slope_of(p, k, nll) : 0.0f;
            } else {
                float l[1], kl[1];
                bool clipped[1];
                const Token one[1] = {k};
                const float value[1] = {nll};
                losses_of(p, one, value, l, kl, clipped);
                const float term = k.weight * l[0];
                sum[s][3] += fmaf(k.rest, l[0], fmaf(k.weight, l[0], -term));
                add_exactly(sum[s][0], sum[s][3], term);
                sum[s][1] = fmaf(k.weight, kl[0], sum[s][1]);
                if (clipped[0]) sum[s][2] += k.weight;
                if (s == 0) clean = l[0];
                if (o.loss) o.loss[s * T + t] = l[0];
                if (o.delta && s > 0) o.delta[(s - 1) * T + t] = l[0] - clean;
            }
        }
    }
    if constexpr (!GRAD) {
#pragma unroll
        for (int s = 0; s < kFewSlices; ++s) {
            if (s >= S) continue;
            const double total = warp_sum_exact(sum[s][0], sum[s][3]);
            sum[s][1] = warp_sum(sum[s][1]);
            sum[s][2] = warp_sum(sum[s][2]);
            if (lane == 0) {
                sums[warp][s][0] = total;
                sums[warp][s][1] = sum[s][1];
                sums[warp][s][2] = sum[s][2];
            }
        }
        __syncthreads();
        if (warp < 3 * S) {
            const int s = warp / 3, j = warp % 3;
            double v = sums[lane][s][j];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            float* out = j == 0 ? o.total : j == 1 ? o.kl : o.clipped;
            if (lane == 0 && out) out[s] = static_cast<float>(v);
        }
    }
}

bool few(int64_t S, int64_t T, int64_t n_seq) {
    return T <= kFewTokens && n_seq <= kFewSequences && S <= kFewSlices;
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

cudaError_t count(const PolicyProblem& p, const Space& w, cudaStream_t s) {
    DUST_TRY(cudaMemsetAsync(w.counts, 0, w.clear, s));
    const unsigned grid = static_cast<unsigned>((p.T + kCountTokens - 1) / kCountTokens);
    return launch_pdl(k_policy_count, dim3(grid), dim3(kCountTokens), 0, s, p, w.counts, w.of_seq, w.seq_of);
}

}  // namespace

size_t policy_workspace_bytes(int64_t S, int64_t T, int64_t n_seq) {
    return few(S, T, n_seq) ? 0 : carve(nullptr, S, T, n_seq).total;
}

cudaError_t launch_policy(const PolicyProblem& p, float* loss, float* total, float* kl,
                          float* clipped, float* delta, void* ws, cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    const Outputs o = {loss, total, kl, clipped, delta};
    if (few(p.S, p.T, p.n_seq))
        return launch_pdl(k_policy_few<false>, dim3(1), dim3(kFewThreads), 0, s, p, o, nullptr, nullptr);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = blocks_of(p.T), groups = groups_of(p.S);
    return launch_pdl(k_policy, dim3(static_cast<unsigned>(blocks * groups)), dim3(kThreads), 0, s, p, o,
                      blocks, groups, w.counts, w.of_seq, w.seq_of, w.parts);
}

cudaError_t launch_policy_grad(const PolicyProblem& p, const float* gtotal, float* gnll, void* ws,
                               cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    if (few(p.S, p.T, p.n_seq))
        return launch_pdl(k_policy_few<true>, dim3(1), dim3(kFewThreads), 0, s, p, Outputs{}, gtotal, gnll);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = (p.T + kThreads - 1) / kThreads, groups = groups_of(p.S);
    return launch_pdl(k_policy_grad, dim3(static_cast<unsigned>(blocks * groups)), dim3(kThreads), 0, s, p,
                      blocks, groups, w.counts, w.of_seq, w.seq_of, gtotal, gnll);
}

}  // namespace dust
