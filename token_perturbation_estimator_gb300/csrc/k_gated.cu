// The gated feed-forward block's first half, h = act(X Wg^T) (X Wu^T), and its
// gradients (include/dust.h gives the formulas): what is copied first, and the
// order of the launches. The products are k_gated_tc.cu's; a few rows go to
// k_gated_few.cu.
//
// Backward: g and u once more, as D = [dG dU] in bf16, then gX = D [Wg; Wu] and
// [gWg; gWu] = D^T X in one launch.
//
// fp32 operands, and bf16 ones whose rows do not start on 16 bytes, are first
// copied into the workspace, as three bf16 planes or padded rows; gh as padded
// rows of its own type. (777 rows, d 301, f 1003, fp32: gradients 50 us, of which
// copying 8, D 22, the products 30 and their slices' sums 7, each launch by
// itself.)
#include <algorithm>

#include "gated.cuh"

namespace dust {

namespace {

size_t a256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
int64_t up(int64_t x, int64_t by) { return (x + by - 1) / by * by; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Rows that are copied: into bf16 planes (1 or 3), or as they are.
struct CopyJob {
    const void* src;
    int64_t ld, n, d, dp;  // n rows of d values, dp apart in the copy, zero from d on
    int vec;               // rows can be read 16 bytes at a time
    void* dst;
    int planes;            // 0: as they are
    unsigned blocks;       // CTAs that work on it
};
struct CopyJobs {
    CopyJob job[4];
};

template <typename TX>
__device__ void copy_rows(const CopyJob& a, int64_t block) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(TX));
    const int lane = threadIdx.x & 31;
    for (int64_t i = block * 8 + (threadIdx.x >> 5); i < a.n; i += static_cast<int64_t>(a.blocks) * 8) {
        const TX* s = static_cast<const TX*>(a.src) + i * a.ld;
        for (int64_t c = lane * 8; c < a.dp; c += 256) {
            alignas(16) TX x[8];
            if (a.vec && c + 8 <= a.d) {
#pragma unroll
                for (int u = 0; u < 8 / kPer; ++u)
                    reinterpret_cast<uint4*>(x)[u] = reinterpret_cast<const uint4*>(s + c)[u];
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = c + k < a.d ? s[c + k] : TX(0.0f);
            }
            if (a.planes == 0) {
                TX* o = static_cast<TX*>(a.dst) + i * a.dp + c;
#pragma unroll
                for (int u = 0; u < 8 / kPer; ++u)
                    reinterpret_cast<uint4*>(o)[u] = reinterpret_cast<const uint4*>(x)[u];
                continue;
            }
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = to_f(x[k]);
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.dst) + i * a.dp + c;
            for (int p = 0; p < a.planes; ++p) {
                alignas(16) __nv_bfloat16 b[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    b[k] = __float2bfloat16_rn(v[k]);
                    // Not up to infinity; and of an infinity nothing is left.
                    if (__hisinf(b[k])) b[k] = __float2bfloat16_rz(v[k]);
                    v[k] = __hisinf(b[k]) ? 0.0f : v[k] - __bfloat162float(b[k]);
                }
                *reinterpret_cast<uint4*>(o + p * a.n * a.dp) = *reinterpret_cast<const uint4*>(b);
            }
        }
    }
}

template <typename TX>
__global__ void __launch_bounds__(256) k_gated_copy(const CopyJobs a) {
    pdl_wait();
    pdl_trigger();
    unsigned block = blockIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (block < a.job[j].blocks) {
            copy_rows<TX>(a.job[j], block);
            return;
        }
        block -= a.job[j].blocks;
    }
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

// Operands are sized as if copied, wherever they lie: the size must not
// depend on addresses. Only what a call needs is touched.
struct Space {
    __nv_bfloat16 *x, *g, *u, *D;
    unsigned char* gh;
    float *gx_acc, *gw_acc;
    GatedCuts cuts;
    size_t total;
};

Space carve(void* ws, const GatedProblem& p, bool grad) {
    const int64_t dp = up(p.d, 8), planes = p.bf16 ? 1 : 3;
    Carver c{static_cast<unsigned char*>(ws)};
    Space w = {};
    if (!grad && p.T <= kGatedFew) return w;
    w.x = c.take<__nv_bfloat16>(planes * p.T * dp);
    w.g = c.take<__nv_bfloat16>(planes * p.f * dp);
    w.u = c.take<__nv_bfloat16>(planes * p.f * dp);
    if (grad) {
        const int n = static_cast<int>(planes);
        w.gh = c.take<unsigned char>(p.T * up(p.f, 8) * (p.bf16 ? 2 : 4));
        w.D = c.take<__nv_bfloat16>(planes * up(p.T, kHeadTile) * 2 * gated_half(p.f));
        // As for all gradients, whichever are asked for.
        w.cuts = gated_cuts(p.T, p.d, p.f, n);
        w.gx_acc = c.take<float>(w.cuts.x > 1 ? gated_acc_floats(p.T, p.d, n, w.cuts.x) : 0);
        w.gw_acc = c.take<float>(w.cuts.w > 1 ? 2 * gated_acc_floats(p.f, p.d, n, w.cuts.w) : 0);
    }
    w.total = c.at;
    return w;
}

#define DUST_TRY(x)                             \
    do {                                        \
        const cudaError_t e_ = (x);             \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

CopyJob copy_job(const void* src, int64_t ld, int64_t n, int64_t d, bool bf16, void* dst, int planes) {
    const int64_t size = bf16 ? 2 : 4;
    return {src, ld, n, d, up(d, 8),
            (ld * size) % 16 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0, dst, planes,
            static_cast<unsigned>(std::min<int64_t>((n + 7) / 8, 152 * 8))};
}

// Rows that start on 16 bytes, no further apart than TMA allows.
bool direct(const void* p, int64_t ld, int64_t per) {
    return ld % per == 0 && ld < (int64_t(1) << 36) && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// The matrix as an operand: where it lies, or the copy that *job is to make.
Planes operand(const void* src, int64_t ld, int64_t n, int64_t d, bool bf16, __nv_bfloat16* copy,
               CopyJob* job) {
    if (bf16 && direct(src, ld, 8)) return {src, n, d, ld, 1};
    const int planes = bf16 ? 1 : 3;
    *job = copy_job(src, ld, n, d, bf16, copy, planes);
    return {copy, n, up(d, 8), up(d, 8), planes};
}

cudaError_t copy(const CopyJobs& jobs, bool bf16, cudaStream_t s) {
    unsigned blocks = 0;
    for (const CopyJob& j : jobs.job) blocks += j.blocks;
    if (blocks == 0) return cudaSuccess;
    return bf16 ? launch_pdl(k_gated_copy<__nv_bfloat16>, dim3(blocks), dim3(256), 0, s, jobs)
                : launch_pdl(k_gated_copy<float>, dim3(blocks), dim3(256), 0, s, jobs);
}

// The operands of g and u, and the copies they need.
GatedTiles tiles_for(const GatedProblem& p, const Space& w, CopyJobs* jobs) {
    GatedTiles t = {};
    t.X = operand(p.X, p.ld_x, p.T, p.d, p.bf16, w.x, &jobs->job[0]);
    t.Wg = operand(p.Wg, p.ld_wg, p.f, p.d, p.bf16, w.g, &jobs->job[1]);
    t.Wu = operand(p.Wu, p.ld_wu, p.f, p.d, p.bf16, w.u, &jobs->job[2]);
    t.T = p.T;
    t.d = p.d;
    t.f = p.f;
    t.act = p.act;
    return t;
}

}  // namespace

size_t gated_workspace_bytes(const GatedProblem& p) { return carve(nullptr, p, false).total; }
size_t gated_grad_workspace_bytes(const GatedProblem& p) { return carve(nullptr, p, true).total; }

cudaError_t launch_gated(const GatedProblem& p, void* h, int64_t ld_h, void* ws, cudaStream_t s) {
    ProfScope ps(kStageGated, s);
    if (p.T <= kGatedFew) return launch_gated_few(p, h, ld_h, s);
    const Space w = carve(ws, p, false);
    CopyJobs jobs = {};
    GatedTiles t = tiles_for(p, w, &jobs);
    DUST_TRY(copy(jobs, p.bf16, s));
    t.h = h;
    t.ld_h = ld_h;
    return launch_gated_tiles(t, s);
}

cudaError_t launch_gated_grad(const GatedProblem& p, const void* gh, int64_t ld_gh, bool accumulate,
                              void* gX, int64_t ld_gx, void* gWg, void* gWu, bool gW_bf16, void* ws,
                              cudaStream_t s) {
    ProfScope ps(kStageGated, s);
    const Space w = carve(ws, p, true);
    CopyJobs jobs = {};
    GatedTiles t = tiles_for(p, w, &jobs);
    t.gh = gh;
    t.ld_gh = ld_gh;
    if (!direct(gh, ld_gh, p.bf16 ? 8 : 4)) {
        jobs.job[3] = copy_job(gh, ld_gh, p.T, p.f, p.bf16, w.gh, 0);
        t.gh = w.gh;
        t.ld_gh = up(p.f, 8);
    }
    t.D = {w.D, up(p.T, kHeadTile), 2 * gated_half(p.f), 2 * gated_half(p.f), p.bf16 ? 1 : 3};
    DUST_TRY(copy(jobs, p.bf16, s));
    DUST_TRY(launch_gated_tiles(t, s));
    return launch_gated_products({t.X, t.Wg, t.Wu, t.D, p.T, p.d, p.f, gX, ld_gx, gWg, gWu, p.bf16,
                                  gW_bf16, accumulate, w.cuts, w.gx_acc, w.gw_acc}, s);
}

}  // namespace dust
