// A policy's clipped loss with a KL term on per-token losses, and its gradient
// (include/dust.h gives the formulas).
//
// A first pass counts each sequence's scored tokens (whole numbers, so that
// the order of the additions does not show); a second one forms the tokens'
// losses, or gradients, whose weights come from those counts, and leaves each
// CTA's sums; a third adds the sums up in order.
#include <algorithm>

#include "step.cuh"

namespace dust {

namespace {

constexpr int kThreads = 256;
constexpr int kSlices = 8;   // slices that a CTA takes
constexpr int kPer = 4;      // tokens that a thread takes
constexpr int kTokens = kThreads * kPer;

struct Counts {
    int32_t tokens, sequences;  // scored, with scored tokens
};

struct Space {
    Counts* counts;
    int32_t* of_seq;   // [n_seq] scored tokens
    float* parts;      // [blocks][S][3]
    size_t clear;      // bytes that start at 0, from counts on
    size_t total;
};

int64_t blocks_of(int64_t T) { return (T + kTokens - 1) / kTokens; }

Space carve(void* ws, int64_t S, int64_t T, int64_t n_seq) {
    unsigned char* base = static_cast<unsigned char*>(ws);
    const auto a256 = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    Space w;
    w.counts = reinterpret_cast<Counts*>(base);
    w.of_seq = reinterpret_cast<int32_t*>(base + 256);
    w.clear = 256 + sizeof(int32_t) * static_cast<size_t>(n_seq);
    size_t at = a256(w.clear);
    w.parts = reinterpret_cast<float*>(base + at);
    at += a256(sizeof(float) * 3 * static_cast<size_t>(blocks_of(T) * S));
    w.total = at;
    return w;
}

// The sequence of token t, or -1: the last one that does not start past it,
// if it has not ended.
__device__ __forceinline__ int64_t sequence_of(const int32_t* offsets, int64_t n_seq, int64_t t) {
    int64_t lo = 0, hi = n_seq;  // offsets[lo] <= t < offsets[hi], once both hold
    if (n_seq == 0 || offsets[0] > t || offsets[n_seq] <= t) return -1;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) k_policy_count(const PolicyProblem p, Counts* counts,
                                                           int32_t* of_seq) {
    pdl_wait();
    pdl_trigger();
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    int64_t seq = -1;
    if (t < p.T && (!p.targets || p.targets[t] >= 0)) seq = sequence_of(p.offsets, p.n_seq, t);
    // One addition per warp and sequence.
    const unsigned same = __match_any_sync(0xffffffffu, static_cast<int>(seq));
    const int lane = threadIdx.x & 31;
    const bool first = __ffs(same) - 1 == lane;
    bool opened = false;
    if (seq >= 0 && first) opened = atomicAdd(of_seq + seq, __popc(same)) == 0;
    const unsigned scored = __ballot_sync(0xffffffffu, seq >= 0);
    const unsigned open = __ballot_sync(0xffffffffu, opened);
    if (lane == 0 && scored) {
        atomicAdd(&counts->tokens, __popc(scored));
        if (open) atomicAdd(&counts->sequences, __popc(open));
    }
}

// exp(r) - r - 1 without cancellation: its series where r is small.
__device__ __forceinline__ float kl_of(float r) {
    if (fabsf(r) < 0.5f) {
        float s = 1.0f / 3628800.0f;  // 1 / 10!
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

    __device__ void load(const PolicyProblem& p, const Counts& c, const int32_t* of_seq, int64_t t) {
        scored = t < p.T && (!p.targets || p.targets[t] >= 0);
        const int64_t seq = scored ? sequence_of(p.offsets, p.n_seq, t) : -1;
        scored = seq >= 0;
        if (!scored) return;
        old = p.old[t];
        ref = p.ref ? p.ref[t] : 0.0f;
        adv = p.advantages[p.per_token ? t : seq];
        weight = p.by_sequence
                     ? static_cast<float>(1.0 / (static_cast<double>(c.sequences) * of_seq[seq]))
                     : 1.0f / static_cast<float>(c.tokens);
    }
};

__device__ __forceinline__ bool beyond(const PolicyProblem& p, float adv, float old, float nll) {
    const double step = static_cast<double>(old) - static_cast<double>(nll);
    return adv > 0.0f ? step > p.high : adv < 0.0f && step < p.low;
}

__device__ __forceinline__ float loss_of(const PolicyProblem& p, const Token& k, float nll, float& kl,
                                         bool& clipped) {
    clipped = beyond(p, k.adv, k.old, nll);
    const float bound = k.adv > 0.0f ? 1.0f + p.clip_high : 1.0f - p.clip_low;
    const float loss = -(clipped ? bound : expf(k.old - nll)) * k.adv;
    kl = p.ref ? kl_of(nll - k.ref) : 0.0f;
    return p.ref ? fmaf(p.beta, kl, loss) : loss;
}

__global__ void __launch_bounds__(kThreads)
    k_policy(const PolicyProblem p, int64_t blocks, const Counts* counts,
             const int32_t* __restrict__ of_seq, float* __restrict__ loss, float* __restrict__ delta, float* __restrict__ parts) {
    pdl_wait();
    pdl_trigger();
    __shared__ float sums[kThreads / 32][kSlices][3];
    const Counts c = *counts;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t block = blockIdx.x % blocks;
    const int64_t t0 = block * kTokens + threadIdx.x;
    const int64_t s0 = blockIdx.x / blocks * kSlices;
    const int slices = static_cast<int>(min(p.S - s0, static_cast<int64_t>(kSlices)));
    Token k[kPer];
    float clean[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int64_t t = t0 + i * kThreads;
        k[i].load(p, c, of_seq, t);
        clean[i] = 0.0f;
        if (delta && k[i].scored) {
            float kl;
            bool clipped;
            clean[i] = loss_of(p, k[i], p.nll[t], kl, clipped);
        }
    }
    for (int s = 0; s < slices; ++s) {
        float sum[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = t0 + i * kThreads;
            if (t >= p.T) continue;
            float l = 0.0f, kl = 0.0f;
            bool clipped = false;
            if (k[i].scored) {
                l = loss_of(p, k[i], p.nll[(s0 + s) * p.T + t], kl, clipped);
                sum[0] = fmaf(k[i].weight, l, sum[0]);
                sum[1] = fmaf(k[i].weight, kl, sum[1]);
                if (clipped) sum[2] += k[i].weight;
            }
            if (loss) loss[(s0 + s) * p.T + t] = l;
            if (delta && s0 + s > 0) delta[(s0 + s - 1) * p.T + t] = l - clean[i];
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
            if (lane == 0) sums[warp][s][j] = sum[j];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slices * 3; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v += sums[w][i / 3][i % 3];
        parts[(block * p.S + s0) * 3 + i] = v;
    }
}

// Sums over the blocks, a warp per slice and kind.
__global__ void __launch_bounds__(96) k_policy_join(const float* __restrict__ parts, int64_t blocks,
                                                    int64_t S, float* total, float* kl, float* clipped) {
    pdl_wait();
    pdl_trigger();
    const int64_t s = blockIdx.x;
    const int j = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double v = 0.0;
    for (int64_t b = lane; b < blocks; b += 32) v += static_cast<double>(parts[(b * S + s) * 3 + j]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    float* out = j == 0 ? total : j == 1 ? kl : clipped;
    if (lane == 0 && out) out[s] = static_cast<float>(v);
}

__global__ void __launch_bounds__(kThreads)
    k_policy_grad(const PolicyProblem p, int64_t blocks, const Counts* counts,
                  const int32_t* __restrict__ of_seq, const float* __restrict__ gtotal, float* gnll) {
    pdl_wait();
    pdl_trigger();
    const Counts c = *counts;
    const int64_t t = blockIdx.x % blocks * kThreads + threadIdx.x;
    if (t >= p.T) return;
    Token k;
    k.load(p, c, of_seq, t);
    const int64_t s0 = blockIdx.x / blocks * kSlices;
    const int64_t s1 = min(p.S, s0 + kSlices);
    for (int64_t s = s0; s < s1; ++s) {
        float g = 0.0f;
        if (k.scored) {
            const float nll = p.nll[s * p.T + t];
            if (!beyond(p, k.adv, k.old, nll)) g = expf(k.old - nll) * k.adv;
            if (p.ref) g = fmaf(p.beta, expm1f(nll - k.ref), g);
            g *= gtotal[s] * k.weight;
        }
        gnll[s * p.T + t] = g;
    }
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

cudaError_t count(const PolicyProblem& p, const Space& w, cudaStream_t s) {
    DUST_TRY(cudaMemsetAsync(w.counts, 0, w.clear, s));
    return launch_pdl(k_policy_count, dim3(static_cast<unsigned>((p.T + kThreads - 1) / kThreads)),
                      dim3(kThreads), 0, s, p, w.counts, w.of_seq);
}

int64_t slice_groups(int64_t S) { return (S + kSlices - 1) / kSlices; }

}  // namespace

size_t policy_workspace_bytes(int64_t S, int64_t T, int64_t n_seq) {
    return carve(nullptr, S, T, n_seq).total;
}

cudaError_t launch_policy(const PolicyProblem& p, float* loss, float* total, float* kl,
                          float* clipped, float* delta, void* ws, cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = blocks_of(p.T);
    DUST_TRY(launch_pdl(k_policy, dim3(static_cast<unsigned>(blocks * slice_groups(p.S))), dim3(kThreads),
                        0, s, p, blocks, w.counts, w.of_seq, loss, delta, w.parts));
    if (!total && !kl && !clipped) return cudaSuccess;
    return launch_pdl(k_policy_join, dim3(static_cast<unsigned>(p.S)), dim3(96), 0, s, w.parts, blocks, p.S,
                      total, kl, clipped);
}

cudaError_t launch_policy_grad(const PolicyProblem& p, const float* gtotal, float* gnll, void* ws,
                               cudaStream_t s) {
    ProfScope ps(kStagePolicy, s);
    const Space w = carve(ws, p.S, p.T, p.n_seq);
    DUST_TRY(count(p, w, s));
    const int64_t blocks = (p.T + kThreads - 1) / kThreads;
    return launch_pdl(k_policy_grad, dim3(static_cast<unsigned>(blocks * slice_groups(p.S))),
                      dim3(kThreads), 0, s, p, blocks, w.counts, w.of_seq, gtotal, gnll);
}

}  // namespace dust
