// C ABI of the gated feed-forward block, the queries' and keys' norms and
// rotation, the policy loss and the gradient clipping (include/dust.h):
// argument checks and dispatch.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "step.cuh"

using namespace dust;

namespace {

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Of the block's rows, columns and units: padded to whole tiles they fit 32
// bits, the units twice over; a plane of a matrix, padded, stays within 2^40
// bytes (TMA's limit).
constexpr int64_t kMaxGatedDim = (int64_t(1) << 31) - (int64_t(1) << 16);
constexpr int64_t kMaxGatedUnits = (int64_t(1) << 30) - (int64_t(1) << 16);
constexpr int64_t kMaxGatedElems = int64_t(1) << 37;
constexpr int64_t kMaxGatedTiles = int64_t(1) << 30;  // of 256 rows x 64 columns, in a launch

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

dust_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DUST_OK : DUST_ERR_CUDA; }

bool value_dtype(int32_t t) { return t == DUST_F32 || t == DUST_BF16; }

int size_of(int32_t t) { return t == DUST_BF16 ? 2 : 4; }

bool aligned_to(const void* p, int32_t t) {
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(size_of(t)) == 0;
}

bool ws_ok(const void* ws, size_t have, size_t need) {
    return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}

// ------------------------------------------------------------------ gated

dust_status check_gated_sizes(int64_t T, int64_t d, int64_t f, dust_dtype dtype) {
    if (T < 0 || d < 1 || f < 1 || !value_dtype(dtype)) return DUST_ERR_INVALID_ARG;
    if (T > kMaxGatedDim || d > kMaxGatedDim || f > kMaxGatedUnits) return DUST_ERR_RANGE;
    const auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    if (up(T) > kMaxGatedElems / up(f) || up(T) > kMaxGatedElems / up(d) || up(f) > kMaxGatedElems / up(d))
        return DUST_ERR_RANGE;
    const auto tiles = [](int64_t rows, int64_t cols) { return (rows + 255) / 256 * ((cols + 63) / 64); };
    if (std::max({tiles(T, f), tiles(T, d), tiles(2 * f, d)}) > kMaxGatedTiles) return DUST_ERR_RANGE;
    return DUST_OK;
}

GatedProblem gated_sizes(int64_t T, int64_t d, int64_t f, dust_dtype dtype) {
    return {nullptr, nullptr, nullptr, d, d, d, dtype == DUST_BF16, T, d, f, 0};
}

dust_status check_gated(const void* X, int64_t ld_x, const void* Wg, int64_t ld_wg, const void* Wu,
                        int64_t ld_wu, dust_dtype dtype, int64_t T, int64_t d, int64_t f, dust_act act) {
    const dust_status st = check_gated_sizes(T, d, f, dtype);
    if (st != DUST_OK) return st;
    if (act != DUST_ACT_SILU && act != DUST_ACT_GELU && act != DUST_ACT_RELU2) return DUST_ERR_INVALID_ARG;
    if (ld_x < d || ld_wg < d || ld_wu < d) return DUST_ERR_INVALID_ARG;
    if ((T > 0 && ld_x > kMaxElems / T) || ld_wg > kMaxElems / f || ld_wu > kMaxElems / f)
        return DUST_ERR_RANGE;
    if (T > 0 && (!X || !Wg || !Wu || !aligned_to(X, dtype) || !aligned_to(Wg, dtype) ||
                  !aligned_to(Wu, dtype)))
        return DUST_ERR_INVALID_ARG;
    return DUST_OK;
}

// A matrix of T rows that is read or written.
dust_status check_rows(const void* p, int64_t ld, int64_t T, int64_t cols, dust_dtype dtype) {
    if (ld < cols || !p || !aligned_to(p, dtype)) return DUST_ERR_INVALID_ARG;
    return ld > kMaxElems / T ? DUST_ERR_RANGE : DUST_OK;
}

// ------------------------------------------------------------------- rope

dust_status check_rope_sizes(int64_t T, int64_t hq, int64_t hk, int64_t D) {
    if (T < 0 || hq < 0 || hk < 0 || D < 1) return DUST_ERR_INVALID_ARG;
    if (D > DUST_MAX_HEAD || T > kMaxDim || hq > kMaxDim - hk || hk > kMaxDim) return DUST_ERR_RANGE;
    if (T > 0 && hq + hk > 0 && (hq + hk) * D > kMaxElems / T) return DUST_ERR_RANGE;
    return DUST_OK;
}

// Operand of T tokens of `heads` heads.
dust_status check_heads(const dust_heads* h, int64_t heads, int64_t T, int64_t D, dust_dtype dtype) {
    if (heads == 0) return DUST_OK;
    if (!h || !h->data || !aligned_to(h->data, dtype)) return DUST_ERR_INVALID_ARG;
    const int64_t t = h->token_stride, n = h->head_stride;
    if (t < 0 || n < 0) return DUST_ERR_INVALID_ARG;
    if ((T > 1 && t > kMaxElems / T) || (heads > 1 && n > kMaxElems / heads)) return DUST_ERR_RANGE;
    // Tokens around heads, or heads around tokens; the stride of a single one says nothing.
    const bool ok = heads == 1 ? T == 1 || t >= D
                    : T == 1   ? n >= D
                               : (n >= D && t >= (heads - 1) * n + D) || (t >= D && n >= (T - 1) * t + D);
    return ok ? DUST_OK : DUST_ERR_INVALID_ARG;
}

dust_heads heads_of(const dust_heads* h, int64_t heads) {
    return h && heads > 0 ? *h : dust_heads{nullptr, 0, 0};
}

struct RopeCall {
    const dust_heads *q, *k;
    int64_t hq, hk;
    dust_dtype dtype;
    int64_t T, D;
    const float *wq, *wk;
    float eps;
    const int32_t* positions;
    const float *cosine, *sine;
    int64_t n_pos, rot;
    dust_rope_layout layout;
    const dust_heads *yq, *yk, *gyq, *gyk;
    bool grad;
};

// The checks of both calls; on DUST_OK with *go false there is nothing to launch.
dust_status check_rope(const RopeCall& c, RopeProblem* p, bool* go) {
    *go = false;
    dust_status st = check_rope_sizes(c.T, c.hq, c.hk, c.D);
    if (st != DUST_OK) return st;
    if (!value_dtype(c.dtype) || !std::isfinite(c.eps) || c.eps < 0.0f) return DUST_ERR_INVALID_ARG;
    if (c.rot < 0 || c.rot > c.D || c.rot % 2 || c.n_pos < 0) return DUST_ERR_INVALID_ARG;
    if (c.layout != DUST_ROPE_HALVES && c.layout != DUST_ROPE_PAIRS) return DUST_ERR_INVALID_ARG;
    if (c.rot > 0 && c.n_pos > kMaxElems / c.rot) return DUST_ERR_RANGE;
    if (c.T == 0 || c.hq + c.hk == 0) return DUST_OK;
    if (!c.positions || (c.rot > 0 && c.n_pos > 0 && (!c.cosine || !c.sine))) return DUST_ERR_INVALID_ARG;
    const struct { const dust_heads* h; int64_t n; } all[6] = {
        {c.q, c.hq}, {c.k, c.hk}, {c.yq, c.hq}, {c.yk, c.hk}, {c.gyq, c.hq}, {c.gyk, c.hk}};
    for (int i = 0; i < (c.grad ? 6 : 4); ++i) {
        st = check_heads(all[i].h, all[i].n, c.T, c.D, c.dtype);
        if (st != DUST_OK) return st;
    }
    *p = {{{heads_of(c.q, c.hq), heads_of(c.yq, c.hq), heads_of(c.gyq, c.hq), c.hq, c.wq, nullptr},
           {heads_of(c.k, c.hk), heads_of(c.yk, c.hk), heads_of(c.gyk, c.hk), c.hk, c.wk, nullptr}},
          c.dtype == DUST_BF16, c.T, c.D, c.eps, c.positions, c.cosine, c.sine, c.n_pos, c.rot, c.layout};
    *go = true;
    return DUST_OK;
}

dust_status zero_weights(float* gwq, float* gwk, int64_t D, cudaStream_t s) {
    for (float* w : {gwq, gwk})
        if (w && cudaMemsetAsync(w, 0, sizeof(float) * static_cast<size_t>(D), s) != cudaSuccess)
            return DUST_ERR_CUDA;
    return DUST_OK;
}

// ----------------------------------------------------------------- policy

dust_status check_policy_sizes(int64_t S, int64_t T, int64_t n_seq) {
    if (S < 1 || T < 0 || n_seq < 0) return DUST_ERR_INVALID_ARG;
    if (S > kMaxDim || T > kMaxDim / S || n_seq > kMaxDim) return DUST_ERR_RANGE;
    return DUST_OK;
}

dust_status check_policy(const PolicyProblem& p, double clip_low, double clip_high, dust_mean mean,
                         const void* ws, size_t ws_bytes) {
    const dust_status st = check_policy_sizes(p.S, p.T, p.n_seq);
    if (st != DUST_OK) return st;
    if (!(clip_low >= 0.0 && clip_low <= 1.0) || !(clip_high >= 0.0) || !std::isfinite(p.beta))
        return DUST_ERR_INVALID_ARG;
    if (mean != DUST_MEAN_TOKEN && mean != DUST_MEAN_SEQUENCE) return DUST_ERR_INVALID_ARG;
    if (p.T > 0 && (!p.nll || !p.old || !p.offsets)) return DUST_ERR_INVALID_ARG;
    if (p.T > 0 && !p.advantages && (p.per_token || p.n_seq > 0)) return DUST_ERR_INVALID_ARG;
    if (!ws_ok(ws, ws_bytes, policy_workspace_bytes(p.S, p.T, p.n_seq))) return DUST_ERR_WORKSPACE;
    return DUST_OK;
}

PolicyProblem policy_problem(const float* nll, const float* old, const float* ref,
                             const float* advantages, int32_t per_token, const int32_t* seq_offsets,
                             int64_t n_seq, const int32_t* targets, int64_t S, int64_t T,
                             double clip_low, double clip_high, float beta, dust_mean mean) {
    const double low = std::log1p(-clip_low), high = std::log1p(clip_high);
    return {nll, old, ref, advantages, per_token != 0, seq_offsets, targets, n_seq, S, T, low, high,
            static_cast<float>(low), static_cast<float>(high), static_cast<float>(1.0 - clip_low),
            static_cast<float>(1.0 + clip_high), beta,
            mean == DUST_MEAN_SEQUENCE};
}

// ------------------------------------------------------------------- clip

struct Span {
    uintptr_t from, to;
    bool out;
};

// Whether an output overlaps another tensor's input or output (or its own
// input without being it). spans: room for 2 n.
bool clip_overlaps(const dust_grad* g, int64_t n, Span* spans) {
    int64_t m = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (g[i].n == 0) continue;
        const uintptr_t bytes = static_cast<uintptr_t>(g[i].n) * static_cast<uintptr_t>(size_of(g[i].dtype));
        const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].g), b = reinterpret_cast<uintptr_t>(g[i].out);
        spans[m++] = {b, b + bytes, true};
        if (a != b) spans[m++] = {a, a + bytes, false};
    }
    std::sort(spans, spans + m, [](const Span& x, const Span& y) { return x.from < y.from; });
    uintptr_t out_end = 0, any_end = 0;  // of the spans so far
    for (int64_t i = 0; i < m; ++i) {
        if (spans[i].from < (spans[i].out ? any_end : out_end)) return true;
        any_end = std::max(any_end, spans[i].to);
        if (spans[i].out) out_end = std::max(out_end, spans[i].to);
    }
    return false;
}

}  // namespace

extern "C" {

dust_status dust_gated_up_workspace(size_t* bytes, int64_t T, int64_t d, int64_t f, dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_gated_sizes(T, d, f, dtype);
    if (st != DUST_OK) return st;
    *bytes = a256(gated_workspace_bytes(gated_sizes(T, d, f, dtype)));
    return DUST_OK;
}

dust_status dust_gated_up(const void* X, int64_t ld_x, const void* Wg, int64_t ld_wg, const void* Wu,
                          int64_t ld_wu, dust_dtype dtype, int64_t T, int64_t d, int64_t f,
                          dust_act act, void* h, int64_t ld_h, void* workspace, size_t ws_bytes,
                          void* stream) {
    dust_status st = check_gated(X, ld_x, Wg, ld_wg, Wu, ld_wu, dtype, T, d, f, act);
    if (st != DUST_OK || T == 0) return st;
    st = check_rows(h, ld_h, T, f, dtype);
    if (st != DUST_OK) return st;
    const GatedProblem p = {X, Wg, Wu, ld_x, ld_wg, ld_wu, dtype == DUST_BF16, T, d, f, act};
    if (!ws_ok(workspace, ws_bytes, a256(gated_workspace_bytes(p)))) return DUST_ERR_WORKSPACE;
    return cuda_status(launch_gated(p, h, ld_h, workspace, static_cast<cudaStream_t>(stream)));
}

dust_status dust_gated_up_grad_workspace(size_t* bytes, int64_t T, int64_t d, int64_t f,
                                         dust_dtype dtype) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_gated_sizes(T, d, f, dtype);
    if (st != DUST_OK) return st;
    *bytes = a256(gated_grad_workspace_bytes(gated_sizes(T, d, f, dtype)));
    return DUST_OK;
}

dust_status dust_gated_up_grad(const void* gh, int64_t ld_gh, const void* X, int64_t ld_x,
                               const void* Wg, int64_t ld_wg, const void* Wu, int64_t ld_wu,
                               dust_dtype dtype, int64_t T, int64_t d, int64_t f, dust_act act,
                               uint32_t flags, void* gX, int64_t ld_gx, void* gWg, void* gWu,
                               dust_dtype gW_dtype, void* workspace, size_t ws_bytes, void* stream) {
    dust_status st = check_gated(X, ld_x, Wg, ld_wg, Wu, ld_wu, dtype, T, d, f, act);
    if (st != DUST_OK) return st;
    if (flags & ~static_cast<uint32_t>(DUST_ACCUMULATE)) return DUST_ERR_INVALID_ARG;
    const bool acc = (flags & DUST_ACCUMULATE) != 0;
    if (gWg || gWu) {
        if (!value_dtype(gW_dtype) || (gW_dtype == DUST_BF16 && (dtype != DUST_BF16 || acc)))
            return DUST_ERR_INVALID_ARG;
        if (!aligned_to(gWg, gW_dtype) || !aligned_to(gWu, gW_dtype)) return DUST_ERR_INVALID_ARG;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        for (void* w : {gWg, gWu})
            if (w && !acc && cudaMemsetAsync(w, 0, static_cast<size_t>(f) * static_cast<size_t>(d) *
                                                       static_cast<size_t>(size_of(gW_dtype)), s) != cudaSuccess)
                return DUST_ERR_CUDA;
        return DUST_OK;
    }
    if (!gX && !gWg && !gWu) return DUST_OK;
    st = check_rows(gh, ld_gh, T, f, dtype);
    if (st == DUST_OK && gX) st = check_rows(gX, ld_gx, T, d, dtype);
    if (st != DUST_OK) return st;
    const GatedProblem p = {X, Wg, Wu, ld_x, ld_wg, ld_wu, dtype == DUST_BF16, T, d, f, act};
    if (!ws_ok(workspace, ws_bytes, a256(gated_grad_workspace_bytes(p)))) return DUST_ERR_WORKSPACE;
    return cuda_status(launch_gated_grad(p, gh, ld_gh, acc, gX, ld_gx, gWg, gWu, gW_dtype == DUST_BF16,
                                         workspace, s));
}

dust_status dust_qk_norm_rope(const dust_heads* q, int64_t hq, const dust_heads* k, int64_t hk,
                              dust_dtype dtype, int64_t T, int64_t D, const float* wq,
                              const float* wk, float eps, const int32_t* positions,
                              const float* cosine, const float* sine, int64_t n_pos, int64_t rot,
                              dust_rope_layout layout, const dust_heads* yq, const dust_heads* yk,
                              void* stream) {
    RopeProblem p;
    bool go;
    const dust_status st = check_rope({q, k, hq, hk, dtype, T, D, wq, wk, eps, positions, cosine, sine,
                                       n_pos, rot, layout, yq, yk, nullptr, nullptr, false}, &p, &go);
    if (st != DUST_OK || !go) return st;
    return cuda_status(launch_rope(p, static_cast<cudaStream_t>(stream)));
}

dust_status dust_qk_norm_rope_grad_workspace(size_t* bytes, int64_t T, int64_t hq, int64_t hk,
                                             int64_t D) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_rope_sizes(T, hq, hk, D);
    if (st != DUST_OK) return st;
    *bytes = a256(rope_grad_workspace_bytes(T, hq + hk, D));
    return DUST_OK;
}

dust_status dust_qk_norm_rope_grad(const dust_heads* gyq, const dust_heads* gyk,
                                   const dust_heads* q, int64_t hq, const dust_heads* k,
                                   int64_t hk, dust_dtype dtype, int64_t T, int64_t D,
                                   const float* wq, const float* wk, float eps,
                                   const int32_t* positions, const float* cosine,
                                   const float* sine, int64_t n_pos, int64_t rot,
                                   dust_rope_layout layout, uint32_t flags, const dust_heads* gq,
                                   const dust_heads* gk, float* gwq, float* gwk, void* workspace,
                                   size_t ws_bytes, void* stream) {
    RopeProblem p;
    bool go;
    const dust_status st = check_rope({q, k, hq, hk, dtype, T, D, wq, wk, eps, positions, cosine, sine,
                                       n_pos, rot, layout, gq, gk, gyq, gyk, true}, &p, &go);
    if (st != DUST_OK) return st;
    if (flags & ~static_cast<uint32_t>(DUST_ACCUMULATE)) return DUST_ERR_INVALID_ARG;
    const bool acc = (flags & DUST_ACCUMULATE) != 0;
    if (!go) return acc ? DUST_OK : zero_weights(gwq, gwk, D, static_cast<cudaStream_t>(stream));
    if ((gwq || gwk) && !ws_ok(workspace, ws_bytes, a256(rope_grad_workspace_bytes(T, hq + hk, D))))
        return DUST_ERR_WORKSPACE;
    p.side[0].gw = gwq;
    p.side[1].gw = gwk;
    return cuda_status(launch_rope_grad(p, acc, workspace, static_cast<cudaStream_t>(stream)));
}

dust_status dust_policy_loss_workspace(size_t* bytes, int64_t S, int64_t T, int64_t n_seq) {
    if (!bytes) return DUST_ERR_INVALID_ARG;
    const dust_status st = check_policy_sizes(S, T, n_seq);
    if (st != DUST_OK) return st;
    *bytes = policy_workspace_bytes(S, T, n_seq);
    return DUST_OK;
}

dust_status dust_policy_loss(const float* nll, const float* old, const float* ref,
                             const float* advantages, int32_t per_token, const int32_t* seq_offsets,
                             int64_t n_seq, const int32_t* targets, int64_t S, int64_t T,
                             double clip_low, double clip_high, float beta, dust_mean mean, float* loss,
                             float* total, float* kl_mean, float* clipped, float* delta,
                             void* workspace, size_t ws_bytes, void* stream) {
    const PolicyProblem p = policy_problem(nll, old, ref, advantages, per_token, seq_offsets, n_seq, targets,
                                           S, T, clip_low, clip_high, beta, mean);
    const dust_status st = check_policy(p, clip_low, clip_high, mean, workspace, ws_bytes);
    if (st != DUST_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        for (float* v : {total, kl_mean, clipped})
            if (v && cudaMemsetAsync(v, 0, sizeof(float) * static_cast<size_t>(S), s) != cudaSuccess)
                return DUST_ERR_CUDA;
        return DUST_OK;
    }
    return cuda_status(launch_policy(p, loss, total, kl_mean, clipped, S > 1 ? delta : nullptr, workspace, s));
}

dust_status dust_policy_loss_grad(const float* nll, const float* old, const float* ref,
                                  const float* advantages, int32_t per_token, const int32_t* seq_offsets,
                                  int64_t n_seq, const int32_t* targets, int64_t S, int64_t T,
                                  double clip_low, double clip_high, float beta, dust_mean mean,
                                  const float* gtotal, float* gnll, void* workspace, size_t ws_bytes,
                                  void* stream) {
    const PolicyProblem p = policy_problem(nll, old, ref, advantages, per_token, seq_offsets, n_seq, targets,
                                           S, T, clip_low, clip_high, beta, mean);
    const dust_status st = check_policy(p, clip_low, clip_high, mean, workspace, ws_bytes);
    if (st != DUST_OK || T == 0) return st;
    if (!gtotal || !gnll) return DUST_ERR_INVALID_ARG;
    return cuda_status(launch_policy_grad(p, gtotal, gnll, workspace, static_cast<cudaStream_t>(stream)));
}

dust_status dust_clip_grads_workspace(size_t* bytes, int64_t n) {
    if (!bytes || n < 0) return DUST_ERR_INVALID_ARG;
    if (n > kMaxGrads) return DUST_ERR_RANGE;
    *bytes = a256(clip_workspace_bytes());
    return DUST_OK;
}

dust_status dust_clip_grads(const dust_grad* grads, int64_t n, float max_norm, float* norm,
                            void* workspace, size_t ws_bytes, void* stream) {
    if (n < 0 || (n > 0 && !grads) || !norm || !(max_norm >= 0.0f)) return DUST_ERR_INVALID_ARG;
    if (n > kMaxGrads) return DUST_ERR_RANGE;
    bool outs = false, nulls = false;
    for (int64_t i = 0; i < n; ++i) {
        const dust_grad& g = grads[i];
        if (g.n < 0 || !value_dtype(g.dtype)) return DUST_ERR_INVALID_ARG;
        if (g.n > kMaxElems) return DUST_ERR_RANGE;
        if (g.n == 0) continue;
        if (!g.g || !aligned_to(g.g, g.dtype) || !aligned_to(g.out, g.dtype)) return DUST_ERR_INVALID_ARG;
        (g.out ? outs : nulls) = true;
    }
    if (outs) {
        const std::unique_ptr<Span[]> spans(new (std::nothrow) Span[static_cast<size_t>(2 * n)]);
        if (!spans) return DUST_ERR_CUDA;
        if (nulls || clip_overlaps(grads, n, spans.get())) return DUST_ERR_INVALID_ARG;
    }
    if (!ws_ok(workspace, ws_bytes, a256(clip_workspace_bytes()))) return DUST_ERR_WORKSPACE;
    return cuda_status(launch_clip(grads, n, max_norm, norm, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
