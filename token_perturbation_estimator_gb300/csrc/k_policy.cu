// A policy's clipped loss with a KL term on per-token losses, and its gradient
// (include/dust.h gives the formulas).
//
// A first pass finds each token's sequence and counts the scored tokens (whole
// numbers, so that the order of the additions does not show); a second one
// forms the tokens' losses, or gradients, whose weights come from those counts,
// and leaves each CTA's sums; a third adds the sums up in order. Few tokens
// go through all of it in one CTA and one launch.
//
// A loss takes about a hundred instructions (two exponentials, a series, the
// sums), so that many slices are bound by issue rather than by their 12 bytes
// a value, and single ones by the launches' latency. Whether a ratio is beyond
// its bound is decided in fp32 where that is certain, else in 64 bits, of which
// the GPU does a 64th as many a second: in 64 bits throughout, 33 slices of
// 65536 tokens took 48 us.
#include <algorithm>
#include <cmath>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kSlices = 8;   // slices that a CTA takes
constexpr int kPer = 4;      // tokens that a thread takes
constexpr int kTokens = kThreads * kPer;
constexpr int kWindow = kTokens + 1;  // sequences' starts that a CTA holds

struct Counts {
    int32_t tokens, sequences;  // scored, with scored tokens
};

struct Space {
    Counts* counts;
    int32_t* of_seq;   // [n_seq] scored tokens
    int32_t* seq_of;   // [T] sequence of a scored token, or -1
    float* parts;      // [blocks][S][3]
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
    w.parts = reinterpret_cast<float*>(take(12 * blocks_of(T) * S));
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

// The starts around a CTA's tokens, from the first one's sequence on.
struct Window {
    int64_t first;  // number of the first start held, -1 where the first token precedes all
    int32_t at[kWindow];

    __device__ void load(const int32_t* offsets, int64_t n_seq, int64_t t0) {
        if (threadIdx.x < 32) {
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

    // The sequence of token t, or -1.
    __device__ int32_t sequence(const int32_t* offsets, int64_t n_seq, int64_t t) const {
        int lo = 0, hi = kWindow;  // starts held that are at or before t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (at[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
        int64_t seq = first + lo - 1;
        if (lo == kWindow)  // more sequences than tokens: empty ones
            seq = starts_until_alone(offsets, n_seq + 1, t) - 1;
        return seq >= 0 && seq < n_seq ? static_cast<int32_t>(seq) : -1;
    }
};

// Adds a warp's scored tokens to the counts, one addition per sequence.
__device__ __forceinline__ void count_tokens(int32_t seq, Counts* counts, int32_t* of_seq) {
    const unsigned same = __match_any_sync(0xffffffffu, seq);
    const int lane = threadIdx.x & 31;
    bool opened = false;
    if (seq >= 0 && __ffs(same) - 1 == lane) opened = atomicAdd(of_seq + seq, __popc(same)) == 0;
    const unsigned scored = __ballot_sync(0xffffffffu, seq >= 0);
    const unsigned open = __ballot_sync(0xffffffffu, opened);
    if (lane == 0 && scored) {
        atomicAdd(&counts->tokens, __popc(scored));
        if (open) atomicAdd(&counts->sequences, __popc(open));
    }
}

__device__ __forceinline__ bool has_target(const PolicyProblem& p, int64_t t) {
    return t < p.T && (!p.targets || p.targets[t] >= 0);
}

__global__ void __launch_bounds__(kThreads)
    k_policy_count(const PolicyProblem p, Counts* counts, int32_t* of_seq, int32_t* __restrict__ seq_of) {
    __shared__ Window window;
    pdl_wait();
    pdl_trigger();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
    bool has[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) has[i] = has_target(p, t0 + i * kThreads + threadIdx.x);
    window.load(p.offsets, p.n_seq, t0);
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + i * kThreads + threadIdx.x;
        const int32_t seq = has[i] ? window.sequence(p.offsets, p.n_seq, t) : -1;
        if (t < p.T) seq_of[t] = seq;
        count_tokens(seq, counts, of_seq);
    }
}

// exp(r) - r - 1 without cancellation: its series where |r| < 1 (what it leaves
// out is below 2^-27 of it).
__device__ __forceinline__ float kl_of(float r) {
    if (fabsf(r) < 1.0f) {
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
        return s * r * r;
    }
    return expm1f(r) - r;
}

// What a token needs of everything but nll.
struct Token {
    bool scored;
    float old, ref, adv, weight;

    __device__ __forceinline__ void load(const PolicyProblem& p, const Counts& c, const int32_t* of_seq,
                                         int32_t seq, int64_t t) {
        scored = seq >= 0;
        if (!scored) return;
        old = p.old[t];
        ref = p.ref ? p.ref[t] : 0.0f;
        adv = p.advantages[p.per_token ? t : seq];
        weight = 1.0f / (p.by_sequence ? static_cast<float>(c.sequences) * static_cast<float>(of_seq[seq])
                                       : static_cast<float>(c.tokens));
    }
};

// Whether the ratio is beyond the bound on its advantage's side. The fp32
// difference is off by half a step, as the bound is: further apart than 4
// steps, they stand as the exact ones do. (The exact ones in a call of their
// own: in line, the compiler forms them for every value.)
__device__ __noinline__ int compare_exactly(double old, double nll, double bound) {
    const double step = old - nll;
    return step > bound ? 1 : step < bound ? -1 : 0;
}

__device__ __forceinline__ bool beyond(const PolicyProblem& p, float adv, float old, float nll) {
    const bool up = adv > 0.0f;
    const float bound = up ? p.high32 : p.low32, step = old - nll;
    if (!(fabsf(step - bound) > 0x1p-22f * fabsf(bound))) {
        const int c = compare_exactly(old, nll, up ? p.high : p.low);
        return up ? c > 0 : adv < 0.0f && c < 0;
    }
    return up ? step > bound : adv < 0.0f && step < bound;
}

__device__ __forceinline__ float loss_of(const PolicyProblem& p, const Token& k, float nll, float& kl,
                                         bool& clipped) {
    clipped = beyond(p, k.adv, k.old, nll);
    const float bound = k.adv > 0.0f ? 1.0f + p.clip_high : 1.0f - p.clip_low;
    const float loss = -(clipped ? bound : expf(k.old - nll)) * k.adv;
    kl = p.ref ? kl_of(nll - k.ref) : 0.0f;
    return p.ref ? fmaf(p.beta, kl, loss) : loss;
}

__device__ __forceinline__ float slope_of(const PolicyProblem& p, const Token& k, float nll) {
    float g = beyond(p, k.adv, k.old, nll) ? 0.0f : expf(k.old - nll) * k.adv;
    if (p.ref) g = fmaf(p.beta, expm1f(nll - k.ref), g);
    return g;
}

// A slice's sums over the lanes, to lane 0.
__device__ __forceinline__ void warp_sums(float (&sum)[3]) {
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
}

struct Outputs {
    float *loss, *total, *kl, *clipped, *delta;
};

__global__ void __launch_bounds__(kThreads)
    k_policy(const PolicyProblem p, const Outputs o, int64_t blocks, int64_t groups, const Counts* counts,
             const int32_t* __restrict__ of_seq, const int32_t* __restrict__ seq_of,
             float* __restrict__ parts) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sums[kThreads / 32][kSlices][3];
    const Counts c = *counts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t block = blockIdx.x % blocks, group = blockIdx.x / blocks;
    const int64_t t0 = block * kTokens + threadIdx.x;
    const int64_t s0 = p.S * group / groups, s1 = p.S * (group + 1) / groups;
    Token k[kPer];
    float clean[kPer], next[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + i * kThreads;
        next[i] = t < p.T ? p.nll[s0 * p.T + t] : 0.0f;
        clean[i] = o.delta && t < p.T ? p.nll[t] : 0.0f;
        k[i].load(p, c, of_seq, t < p.T ? seq_of[t] : -1, t);
    }
    if (o.delta) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float kl;
            bool clipped;
            clean[i] = k[i].scored ? loss_of(p, k[i], clean[i], kl, clipped) : 0.0f;
        }
    }
#pragma unroll 1
    for (int64_t s = s0; s < s1; ++s) {
        float now[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = t0 + i * kThreads;
            now[i] = next[i];
            if (s + 1 < s1 && t < p.T) next[i] = p.nll[(s + 1) * p.T + t];
        }
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = t0 + i * kThreads;
            if (t >= p.T) continue;
            float l = 0.0f, kl = 0.0f;
            bool clipped = false;
            if (k[i].scored) {
                l = loss_of(p, k[i], now[i], kl, clipped);
                sum[0] = fmaf(k[i].weight, l, sum[0]);
                sum[1] = fmaf(k[i].weight, kl, sum[1]);
                if (clipped) sum[2] += k[i].weight;
            }
            if (o.loss) o.loss[s * p.T + t] = l;
            if (o.delta && s > 0) o.delta[(s - 1) * p.T + t] = l - clean[i];
        }
        warp_sums(sum);
        if (lane == 0)
#pragma unroll
            for (int j = 0; j < 3; ++j) sums[warp][s - s0][j] = sum[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (s1 - s0) * 3; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v += sums[w][i / 3][i % 3];
        parts[(block * p.S + s0) * 3 + i] = v;
    }
}

// Sums over the blocks, a warp per slice and kind.
__global__ void __launch_bounds__(96) k_policy_join(const float* __restrict__ parts, int64_t blocks,
                                                    int64_t S, const Outputs o) {
    pdl_wait();
    pdl_trigger();
    const int64_t s = blockIdx.x;
    const int j = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double v = 0.0;
    for (int64_t b = lane; b < blocks; b += 32) v += static_cast<double>(parts[(b * S + s) * 3 + j]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    float* out = j == 0 ? o.total : j == 1 ? o.kl : o.clipped;
    if (lane == 0 && out) out[s] = static_cast<float>(v);
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
    __shared__ float sums[kFewThreads / 32][kFewSlices][3];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = static_cast<int>(p.T), S = static_cast<int>(p.S);
    for (int i = threadIdx.x; i < p.n_seq; i += kFewThreads) of_seq[i] = 0;
    if (threadIdx.x == 0) counts = {0, 0};
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
        if (i * kFewThreads < T) count_tokens(seq[i], &counts, of_seq);
    }
    __syncthreads();
    float sum[kFewSlices][3] = {};
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
                float l = 0.0f, kl = 0.0f;
                bool clipped = false;
                if (k.scored) {
                    l = loss_of(p, k, nll, kl, clipped);
                    sum[s][0] = fmaf(k.weight, l, sum[s][0]);
                    sum[s][1] = fmaf(k.weight, kl, sum[s][1]);
                    if (clipped) sum[s][2] += k.weight;
                }
                if (s == 0) clean = l;
                if (o.loss) o.loss[s * T + t] = l;
                if (o.delta && s > 0) o.delta[(s - 1) * T + t] = l - clean;
            }
        }
    }
    if constexpr (!GRAD) {
#pragma unroll
        for (int s = 0; s < kFewSlices; ++s) {
            if (s >= S) continue;
            warp_sums(sum[s]);
            if (lane == 0)
#pragma unroll
                for (int j = 0; j < 3; ++j) sums[warp][s][j] = sum[s][j];
        }
        __syncthreads();
        if (warp < 3 * S) {
            const int s = warp / 3, j = warp % 3;
            double v = static_cast<double>(sums[lane][s][j]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            float* out = j == 0 ? o.total : j == 1 ? o.kl : o.clipped;
            if (lane == 0 && out) out[s] = static_cast<float>(v);
        }
    }
}

bool few(const PolicyProblem& p) {
    return p.T <= kFewTokens && p.n_seq <= kFewSequences && p.S <= kFewSlices;
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

cudaError_t count(const PolicyProblem& p, const Space& w, cudaStream_t s) {
    DUST_TRY(cudaMemsetAsync(w.counts, 0, w.clear, s));
    return launch_pdl(k_policy_count, dim3(static_cast<unsigned>(blocks_of(p.T))), dim3(kThreads), 0, s, p,
                      w.counts, w.of_seq, w.seq_of);
}

}  // namespace

size_t policy_workspace_bytes(int64_t S, int64_t T, int64_t n_seq) {
    return carve(nullptr, S, T, n_seq).total;
}

cudaError_t launch_policy(const PolicyProblem& p, float* loss, float* total, float* kl,
                          float* clipped, float* delta, void* ws, cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    const Outputs o = {loss, total, kl, clipped, delta};
    if (few(p))
        return launch_pdl(k_policy_few<false>, dim3(1), dim3(kFewThreads), 0, s, p, o, nullptr, nullptr);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = blocks_of(p.T), groups = groups_of(p.S);
    DUST_TRY(launch_pdl(k_policy, dim3(static_cast<unsigned>(blocks * groups)), dim3(kThreads), 0, s, p, o,
                        blocks, groups, w.counts, w.of_seq, w.seq_of, w.parts));
    if (!total && !kl && !clipped) return cudaSuccess;
    return launch_pdl(k_policy_join, dim3(static_cast<unsigned>(p.S)), dim3(96), 0, s, w.parts, blocks, p.S, o);
}

cudaError_t launch_policy_grad(const PolicyProblem& p, const float* gtotal, float* gnll, void* ws,
                               cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    if (few(p))
        return launch_pdl(k_policy_few<true>, dim3(1), dim3(kFewThreads), 0, s, p, Outputs{}, gtotal, gnll);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = (p.T + kThreads - 1) / kThreads, groups = groups_of(p.S);
    return launch_pdl(k_policy_grad, dim3(static_cast<unsigned>(blocks * groups)), dim3(kThreads), 0, s, p,
                      blocks, groups, w.counts, w.of_seq, w.seq_of, gtotal, gnll);
}

}  // namespace dust
