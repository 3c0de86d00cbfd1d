// Tensor-core products of the head's losses and gradients (tcgen05, sm_103a).
//
//   kLse     x = scale H E^T tile by tile, never stored: each row's partial
//            (maximum, sum of exponentials) per half tile, and its target's
//            logit;
//   kFactor  the same tiles again, as G = weight (exp(x - lse) - [target]),
//            rounded to bf16 (fp32 inputs: as three bf16 planes);
//   kMul     gH = G E and gE = G^T H, the tiles of both in one launch.
//
// A CTA pair (a cluster of two, cta_group::2) makes a 256-row tile of 256 (or
// 128) columns: each CTA keeps 128 rows' fp32 accumulators in its TMEM, twice,
// so that one tile's epilogue runs beside the next tile's products. Per step
// of 64 along the summed dimension each CTA loads its 128 rows of A and its
// half of B's columns: 32 KB for 256 x 256 x 64 products per pair, a third less than
// two CTAs would load on their own. Operands are used as they are stored:
// K-major where the summed dimension is contiguous (H, E for the logits; G
// for gH), MN-major where it is not (E for gH; G and H for gE); the same
// 64 x 64 boxes with the 128-byte swizzle serve both.
//
// fp32 inputs come as three bf16 planes whose sum is the value to 24 bits
// (each plane the bf16 rounding of what the ones before leave), and a product
// is six products of planes, smallest first; what is left out is below 2^-24
// of the product.
//
// Persistent: warp 0 loads (both CTAs), warp 1 issues the MMAs (rank 0 only),
// eight warps drain the accumulators, two per TMEM lane quarter. All waits are
// bounded and record DUST_ERR_TIMEOUT in the device status word.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "head.cuh"
#include "tc_common.cuh"

namespace dust {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {

constexpr int kStages = 6;
constexpr int kHalf = 128;                        // rows of A per CTA
constexpr int kBoxBytes = kHeadBox * kHeadBox * 2;
constexpr int kStageBytes = 4 * kBoxBytes;        // two boxes of A, two of B
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStageBuf = 32 * 32 * 2;            // 32 rows x 32 columns of G
constexpr int kStoreBufs = 2;
constexpr int kSmemBytes = kStages * kStageBytes + kEpiWarps * kStoreBufs * kStageBuf + 1024 + 512;
constexpr uint32_t kTmemCols = 512;               // two accumulators of 256 columns
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

enum Mode { kLse, kFactor, kMul };

struct Ctl {
    uint64_t full[kStages];
    uint64_t empty[kStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint64_t never;
    uint32_t tmem;
    int abort;
    int issued;
    int consumed;
};

// One product C[m][n] = sum over k A(m, k) B(n, k) of a launch.
struct Dims {
    int64_t m, n, k;
    int mt, nt;  // tiles
};

struct TcArgs {
    int64_t rows, d, n, v0;    // rows without a device count
    const HeadCounts* counts;
    int planes;                // 1, or 3 (six products)
    int bn;                    // tile columns
    int group;                 // row tiles that run together (logits)
    float scale;
    const int32_t* targets;    // kLse
    int64_t T;
    HeadPart* part;
    int64_t ld_part;
    float* picked;
    const HeadRow* info;       // kFactor
    int64_t g_cols;
    const int32_t* row_of;     // kMul
    unsigned char* gH;
    int64_t ld_gh;
    float* gh_acc;
    unsigned char* gE;
    int gh_bf16, ge_bf16, gh_vec, ge_vec, first, last, accumulate;
    int stall;
    unsigned int* status;
};

// Planes of A and B of the p-th product, the smallest products first.
__device__ __forceinline__ int plane_a(int planes, int p) {
    constexpr int a[6] = {2, 0, 1, 1, 0, 0};
    return planes == 1 ? 0 : a[p];
}
__device__ __forceinline__ int plane_b(int planes, int p) {
    constexpr int b[6] = {0, 2, 1, 0, 1, 0};
    return planes == 1 ? 0 : b[p];
}

// Where a tile lies: which product (0: logits or gH, 1: gE), its first row
// and column, and its steps along the summed dimension per pair of planes.
struct Tile {
    int job;
    int64_t m0, n0;
    int steps;
    int index;  // among the product's tiles
};

template <int MODE>
struct Plan {
    int64_t rows;
    int mt, nt;        // job 0
    int mt1, nt1;      // job 1 (kMul)
    int n0_tiles, n1_tiles, total;
    int steps0, steps1;
    bool one_first;

    __device__ Plan(const TcArgs& a) {
        rows = a.counts ? a.counts->rows : a.rows;
        const auto up = [](int64_t v, int64_t by) { return static_cast<int>((v + by - 1) / by); };
        if (MODE != kMul) {
            mt = up(rows, kHeadTile);
            nt = up(a.n, a.bn);
            steps0 = up(a.d, 64);
            n0_tiles = mt * nt;
            mt1 = nt1 = n1_tiles = steps1 = 0;
        } else {
            mt = a.gH ? up(rows, kHeadTile) : 0;
            nt = up(a.d, a.bn);
            steps0 = up(a.n, 64);
            n0_tiles = mt * nt;
            mt1 = a.gE ? up(a.n, kHeadTile) : 0;
            nt1 = nt;
            steps1 = up(rows, 64);
            n1_tiles = mt1 * nt1;
        }
        total = n0_tiles + n1_tiles;
        one_first = steps1 > steps0;  // the longer tiles start first
    }

    __device__ Tile at(const TcArgs& a, int t) const {
        Tile w;
        if (MODE != kMul) {
            // Groups of row tiles; inside one, rows fastest: the group's H
            // stays in L2 while E streams by once per group.
            const int per = a.group * nt;
            const int g = t / per, in = t - g * per;
            const int gm = min(a.group, mt - g * a.group);
            const int c = in / gm;
            w.job = 0;
            w.m0 = static_cast<int64_t>(g * a.group + (in - c * gm)) * kHeadTile;
            w.n0 = static_cast<int64_t>(c) * a.bn;
            w.steps = steps0;
            w.index = c;
        } else {
            const int firsts = one_first ? n1_tiles : n0_tiles;
            const bool job1 = (t < firsts) == one_first;
            const int i = t < firsts ? t : t - firsts;
            const int r = i / nt;  // columns fastest: a row block of G is read by neighbours
            w.job = job1 ? 1 : 0;
            w.m0 = static_cast<int64_t>(r) * kHeadTile;
            w.n0 = static_cast<int64_t>(i - r * nt) * a.bn;
            w.steps = job1 ? steps1 : steps0;
            w.index = i;
        }
        return w;
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ void st_shared_16(uint32_t addr, const uint32_t* v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3])
                 : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// Up to 32 consecutive values of a row, of which `n` lie inside the output.
__device__ __forceinline__ void store_row(unsigned char* row, int64_t col, const float (&v)[32],
                                          int n, bool bf16, bool vec, bool add) {
    if (bf16) {
        __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(row) + col;
        if (vec && n >= 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4*>(p)[i] =
                    make_uint4(pack2(v[8 * i], v[8 * i + 1]), pack2(v[8 * i + 2], v[8 * i + 3]),
                               pack2(v[8 * i + 4], v[8 * i + 5]), pack2(v[8 * i + 6], v[8 * i + 7]));
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n) p[i] = __float2bfloat16_rn(v[i]);
        }
    } else {
        float* p = reinterpret_cast<float*>(row) + col;
        if (vec && n >= 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float4 o = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                if (add) {
                    const float4 b = reinterpret_cast<const float4*>(p)[i];
                    o = make_float4(b.x + o.x, b.y + o.y, b.z + o.z, b.w + o.w);
                }
                reinterpret_cast<float4*>(p)[i] = o;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < n) p[i] = add ? p[i] + v[i] : v[i];
        }
    }
}

// Adds a block's columns to a row's running sum s of 2^(c v - m). m stays a
// whole number (the largest c v so far, rounded up), so that c v - m is
// rounded once, and the few times it grows s is scaled by a power of two.
template <bool FULL>
__device__ __forceinline__ void softmax_block(const float (&v)[32], int n, float c, float& m,
                                              float& s) {
    float top = v[0];
    if (c >= 0.0f) {
#pragma unroll
        for (int i = 1; i < 32; ++i)
            if (FULL || i < n) top = fmaxf(top, v[i]);
    } else {
#pragma unroll
        for (int i = 1; i < 32; ++i)
            if (FULL || i < n) top = fminf(top, v[i]);
    }
    const float nm = fmaxf(m, ceilf(c * top));
    const float base = nm == -INFINITY ? 0.0f : nm;
    float e0 = 0.0f, e1 = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        if (FULL || i < n) e0 += ex2(fmaf(c, v[i], -base));
        if (FULL || i + 1 < n) e1 += ex2(fmaf(c, v[i + 1], -base));
    }
    s = fmaf(s, ex2(m - base), e0 + e1);
    m = nm;
}

// Epilogue of one tile for one warp: rows 32 q + lane of this CTA's half,
// columns [h bn / 2, (h + 1) bn / 2).
template <int MODE, int PLANES>
struct Epilogue {
    const TcArgs& a;
    const CUtensorMap* tmG;
    unsigned char* bufs;  // this warp's store buffers
    uint32_t used = 0;

    __device__ Epilogue(const TcArgs& args, const CUtensorMap* g, unsigned char* b)
        : a(args), tmG(g), bufs(b) {}

    // What the row needs besides the accumulator; loaded before the wait.
    int64_t row;
    bool live;
    int32_t target;
    HeadRow info;
    int64_t out_row;

    __device__ void begin(const Tile& w, const Plan<MODE>& plan, uint32_t rank, int q, int lane) {
        row = w.m0 + rank * kHalf + 32 * q + lane;
        if (MODE == kLse) {
            live = row < plan.rows;
            target = live && a.targets ? a.targets[row % a.T] : -1;
        } else if (MODE == kFactor) {
            live = row < plan.rows;
            if (live) info = a.info[row];
            target = live ? info.target : -1;
        } else if (w.job == 0) {
            live = row < plan.rows;
            out_row = live && a.row_of ? a.row_of[row] : row;
        } else {
            live = row < a.n;
            out_row = row;
        }
    }

    __device__ void run(const Tile& w, uint32_t taddr, int h, int lane, uint32_t rank, int q,
                        float alpha, bool zero) {
        const int cols = a.bn / 2;
        if (MODE == kLse) {
            const float c = a.scale * kLog2e;
            const int32_t first = static_cast<int32_t>(w.n0) + h * cols;
            float m = -INFINITY, s = 0.0f;
            // Target relative to the warp's first column, if it has one there.
            const int32_t tv = target - static_cast<int32_t>(a.v0) - first;
            for (int b = 0; b < cols / 32; ++b) {
                float v[32];
                tc::tmem_ld_32x32(taddr + h * cols + 32 * b, v);
                const int left = static_cast<int>(a.n) - (first + 32 * b);  // columns that exist
                if (left <= 0) break;
                const int at = tv - 32 * b;
                if (live && at >= 0 && at < 32 && at < left) {
                    float x = 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) x = (i == at) ? v[i] : x;
                    a.picked[row] = a.scale * x;
                }
                if (left >= 32)
                    softmax_block<true>(v, 32, c, m, s);
                else
                    softmax_block<false>(v, left, c, m, s);
            }
            if (live) {
                const HeadPart p = {m, s};
                a.part[(2 * static_cast<int64_t>(w.index) + h) * a.ld_part + row] = p;
            }
        } else if (MODE == kFactor) {
            const float c = a.scale * kLog2e;
            const uint32_t swz = (lane >> 1) & 3;
            for (int b = 0; b < cols / 32; ++b) {
                float v[32];
                const int64_t col = w.n0 + h * cols + 32 * b;
                tc::tmem_ld_32x32(taddr + h * cols + 32 * b, v);
                const int left = static_cast<int>(a.n - col);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    // The logarithm in two parts: its rounding would be the
                    // same for the whole row.
                    float t = fmaf(c, v[i], -info.lse_hi);
                    if (PLANES == 3) t -= info.lse_lo;
                    const float e = info.weight * ex2(t);
                    v[i] = live && i < left ? e : 0.0f;
                }
                const int64_t tv = target - a.v0 - col;
                if (tv >= 0 && tv < 32) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (i == tv) v[i] -= info.weight;
                }
#pragma unroll
                for (int p = 0; p < PLANES; ++p) {
                    unsigned char* buf = bufs + (used % kStoreBufs) * kStageBuf;
                    if (used >= kStoreBufs) {
                        if (lane == 0) tc::bulk_wait_read<kStoreBufs - 1>();
                        __syncwarp();
                    }
                    const uint32_t dst = tc::smem_u32(buf) + lane * 64;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t pk[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x0 = v[8 * u + 2 * j], x1 = v[8 * u + 2 * j + 1];
                            pk[j] = pack2(x0, x1);
                            if (p + 1 < PLANES) {  // what this plane leaves
                                v[8 * u + 2 * j] = x0 - __uint_as_float(pk[j] << 16);
                                v[8 * u + 2 * j + 1] = x1 - __uint_as_float(pk[j] & 0xffff0000u);
                            }
                        }
                        st_shared_16(dst + ((u ^ swz) << 4), pk);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        // G is padded to whole tiles: every block lies inside.
                        tc::tma_store_3d(tmG, buf, static_cast<int32_t>(col),
                                         static_cast<int32_t>(w.m0 + rank * kHalf + 32 * q), p);
                        tc::bulk_commit();
                    }
                    ++used;
                }
            }
        } else {
            for (int b = 0; b < cols / 32; ++b) {
                float v[32];
                const int at = h * cols + 32 * b;
                const int64_t col = w.n0 + at;
                tc::tmem_ld_32x32(taddr + at, v);
                if (col >= a.d) break;
                const int n = a.d - col < 32 ? static_cast<int>(a.d - col) : 32;
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : alpha * v[i];
                if (w.job == 1) {
                    if (live)
                        store_row(a.gE + out_row * a.d * (a.ge_bf16 ? 2 : 4), col, v, n,
                                  a.ge_bf16, a.ge_vec, a.accumulate);
                    continue;
                }
                if (a.gh_acc) {
                    // Running sums in the order of the accumulator: four
                    // columns of all rows together.
                    const int in_tile = static_cast<int>(rank) * kHalf + 32 * q + lane;
                    float4* p = reinterpret_cast<float4*>(
                        a.gh_acc + static_cast<int64_t>(w.index) * kHeadTile * kHeadTile);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float4* e = p + (at / 4 + i) * kHeadTile + in_tile;
                        if (!a.first) {
                            const float4 o = *e;
                            v[4 * i] += o.x;
                            v[4 * i + 1] += o.y;
                            v[4 * i + 2] += o.z;
                            v[4 * i + 3] += o.w;
                        }
                        if (!a.last) *e = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    }
                    if (!a.last) continue;
                }
                if (live)
                    store_row(a.gH + out_row * a.ld_gh * (a.gh_bf16 ? 2 : 4), col, v, n, a.gh_bf16,
                              a.gh_vec, false);
            }
        }
    }
};

// Maps: kLse H, -, E, -; kFactor H, Hc, E, G; kMul G, E, H, Hc.
template <int MODE, int PLANES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_head_tc(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
              const __grid_constant__ CUtensorMap tm2, const __grid_constant__ CUtensorMap tm3,
              const __grid_constant__ TcArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* store_bufs = smem + kStages * kStageBytes;
    Ctl* ctl = reinterpret_cast<Ctl*>(store_bufs + kEpiWarps * kStoreBufs * kStageBuf);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = tc::cluster_rank_of_cta();
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&ctl->full[i], 1);
            tc::mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ctl->tfull[i], 1);
            tc::mbar_init(&ctl->tempty[i], 2 * kEpiWarps);
        }
        tc::mbar_init(&ctl->drain, 1);
        tc::mbar_init(&ctl->never, 1);
        ctl->abort = 0;
        ctl->issued = 0;
        ctl->consumed = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(&ctl->tmem, kTmemCols);
        tc::tmem_relinquish_pair();
    }
    tc::tc_fence_before();
    tc::cluster_barrier();  // barriers of both CTAs are set up
    tc::tc_fence_after();
    const uint32_t tmem = ctl->tmem;
    volatile int* abort_flag = &ctl->abort;
    pdl_wait();
    pdl_trigger();

    const Plan<MODE> plan(a);
    const int pairs = a.planes == 1 ? 1 : 6;
    const int b_boxes = a.bn / 128;  // per CTA
    // A tile's products take about 0.3 us per step: the waits for a whole
    // tile are given 2 us per step on top of the usual limit.
    const uint64_t tile_ns =
        tc::kWaitNs + 2000ull * static_cast<uint64_t>(pairs) * max(plan.steps0, plan.steps1);

    if (warp == 0) {
        if (lane == 0) {
            // The rows that take part are read where they lie unless some were left out.
            const bool compact = a.counts && a.rows != plan.rows;
            const CUtensorMap *A0, *B0, *A1 = nullptr, *B1 = nullptr;
            if (MODE == kMul) {
                A0 = &tm0; B0 = &tm1;                      // gH = G E
                A1 = &tm0; B1 = compact ? &tm3 : &tm2;     // gE = G^T H
            } else {
                A0 = compact ? &tm1 : &tm0;
                B0 = &tm2;
            }
            int it = 0;
            for (int t = cluster; t < plan.total && !*abort_flag; t += n_clusters) {
                const Tile w = plan.at(a, t);
                const CUtensorMap* ma = w.job ? A1 : A0;
                const CUtensorMap* mb = w.job ? B1 : B0;
                // Which operand has the summed dimension in rows.
                const bool a_mn = MODE == kMul && w.job == 1, b_mn = MODE == kMul;
                const int32_t am = static_cast<int32_t>(w.m0) + static_cast<int32_t>(rank) * kHalf;
                // E is whole: its rows of the piece start at v0.
                const int32_t v0 = static_cast<int32_t>(a.v0);
                const int32_t bn0 = static_cast<int32_t>(w.n0) +
                                    static_cast<int32_t>(rank) * (a.bn / 2) +
                                    (MODE == kMul ? 0 : v0);
                const int32_t b_k0 = MODE == kMul && w.job == 0 ? v0 : 0;
                for (int p = 0; p < pairs && !*abort_flag; ++p) {
                    const int pa = plane_a(a.planes, p), pb = plane_b(a.planes, p);
                    for (int k = 0; k < w.steps; ++k, ++it) {
                        const int st = it % kStages;
                        if (!tc::mbar_wait_cluster(&ctl->empty[st], ((it / kStages) & 1) ^ 1,
                                                   tile_ns) || *abort_flag) {
                            *abort_flag = 1;
                            break;
                        }
                        unsigned char* base = smem + st * kStageBytes;
                        const uint32_t bar = tc::at_rank(&ctl->full[st], 0);
                        if (rank == 0)
                            tc::mbar_arrive_expect_tx(&ctl->full[st], 2 * (2 + b_boxes) * kBoxBytes);
                        const int32_t kk = k * 64;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            tc::tma_load_3d_pair(base + u * kBoxBytes, ma, a_mn ? am + 64 * u : kk,
                                                 a_mn ? kk : am + 64 * u, pa, bar);
                        for (int u = 0; u < b_boxes; ++u)
                            tc::tma_load_3d_pair(base + (2 + u) * kBoxBytes, mb,
                                                 b_mn ? bn0 + 64 * u : kk,
                                                 b_mn ? b_k0 + kk : bn0 + 64 * u, pb, bar);
                    }
                }
            }
            ctl->issued = it;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            if (a.stall && !tc::mbar_wait(&ctl->never, 0)) *abort_flag = 1;
            int it = 0, j = 0;
            for (int t = cluster; t < plan.total && !*abort_flag; t += n_clusters, ++j) {
                const Tile w = plan.at(a, t);
                const int acc = j & 1;
                if (!tc::mbar_wait_cluster(&ctl->tempty[acc], ((j >> 1) & 1) ^ 1, tile_ns)) {
                    *abort_flag = 1;
                    break;
                }
                tc::tc_fence_after();
                const bool a_mn = MODE == kMul && w.job == 1, b_mn = MODE == kMul;
                const uint32_t idesc = tc::idesc_bf16(kHeadTile, a.bn, a_mn, b_mn);
                // Bytes from one 16-deep slice of a step to the next.
                const uint32_t a_step = a_mn ? 2048 : 32, b_step = b_mn ? 2048 : 32;
                const uint32_t a_lbo = a_mn ? kBoxBytes : 16, b_lbo = b_mn ? kBoxBytes : 16;
                const uint32_t dst = tmem + acc * 256;
                const int n = pairs * w.steps;
                for (int k = 0; k < n; ++k, ++it) {
                    const int st = it % kStages;
                    if (!tc::mbar_wait_cluster(&ctl->full[st], (it / kStages) & 1, tc::kWaitNs) ||
                        *abort_flag) {
                        *abort_flag = 1;
                        break;
                    }
                    tc::tc_fence_after();
                    const uint32_t sa = tc::smem_u32(smem + st * kStageBytes);
                    const uint32_t sb = sa + 2 * kBoxBytes;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        tc::mma_bf16_pair(dst, tc::sdesc_sw128(sa + u * a_step, a_lbo, 1024),
                                          tc::sdesc_sw128(sb + u * b_step, b_lbo, 1024), idesc,
                                          (k | u) != 0 ? 1u : 0u);
                    tc::mma_commit_pair(&ctl->empty[st]);
                }
                if (*abort_flag) break;
                tc::mma_commit_pair(&ctl->tfull[acc]);
            }
            ctl->consumed = it;
            if (*abort_flag) {
                // Everything issued so far has to be done before TMEM is freed.
                tc::mma_commit_pair(&ctl->drain);
                tc::mbar_wait_cluster(&ctl->drain, 0, tc::kWaitNs);
            }
        }
    } else {
        const int ew = warp - 2, q = warp & 3, h = ew >> 2;
        Epilogue<MODE, PLANES> epi(a, &tm3, store_bufs + ew * kStoreBufs * kStageBuf);
        const float alpha = MODE == kMul ? a.scale * a.counts->gmax : 0.0f;
        int j = 0;
        for (int t = cluster; t < plan.total; t += n_clusters, ++j) {
            const Tile w = plan.at(a, t);
            const int acc = j & 1;
            epi.begin(w, plan, rank, q, lane);
            const bool ok = tc::mbar_wait_cluster(&ctl->tfull[acc], (j >> 1) & 1, tile_ns);
            tc::tc_fence_after();
            if (!__all_sync(0xffffffffu, ok) || *abort_flag) {
                *abort_flag = 1;
                break;
            }
            epi.run(w, tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * 256, h, lane, rank, q,
                    alpha, w.steps == 0);
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive_at(tc::at_rank(&ctl->tempty[acc], 0));
        }
        if (MODE == kFactor) {
            if (lane == 0) tc::bulk_wait_all();
            __syncwarp();
        }
    }
    __syncwarp();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        // Let the loads already issued land (rank 0 sees both CTAs').
        if (rank == 0)
            for (int it = ctl->consumed; it < ctl->issued; ++it)
                tc::mbar_wait(&ctl->full[it % kStages], (it / kStages) & 1);
        atomicExch(a.status, 5u /* DUST_ERR_TIMEOUT */);
    }
    tc::tc_fence_before();
    __syncwarp();
    tc::cluster_barrier();  // neither CTA leaves while the other may signal it
    if (warp == 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// [planes][rows][cols] as a 3-D map of box_rows x box_cols boxes.
bool make_map(CUtensorMap* map, const Planes& p, uint32_t box_cols, uint32_t box_rows,
              CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.cols), static_cast<cuuint64_t>(p.rows),
                          static_cast<cuuint64_t>(p.planes)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.ld) * 2,
                             static_cast<cuuint64_t>(p.rows) * static_cast<cuuint64_t>(p.ld) * 2};
    cuuint32_t box[3] = {box_cols, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool operand_map(CUtensorMap* map, const Planes& p) {
    return make_map(map, p, kHeadBox, kHeadBox, CU_TENSOR_MAP_SWIZZLE_128B);
}

// CTA pairs that can be resident at once, for the kernel of a mode.
template <int MODE, int PLANES>
int max_clusters() {
    constexpr int kMaxDev = 64;
    static int cache[kMaxDev] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0) {
        const void* k = reinterpret_cast<const void*>(k_head_tc<MODE, PLANES>);
        if (ensure_smem_limit(k, kSmemBytes) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return 0;
        cache[dev] = n;
    }
    return cache[dev];
}

template <int MODE, int PLANES>
cudaError_t launch_tc(const CUtensorMap (&m)[4], TcArgs a, int64_t tiles, cudaStream_t s) {
    const int fit = max_clusters<MODE, PLANES>();
    if (fit <= 0) return cudaErrorUnknown;
    if (tiles <= 0) return cudaSuccess;
    if (tiles > (int64_t(1) << 30)) return cudaErrorInvalidValue;
    a.status = status_word();
    if (!a.status) return cudaErrorUnknown;
    a.stall = take_stall_injection() ? 1 : 0;
    const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, fit));
    return launch_pdl(k_head_tc<MODE, PLANES>, dim3(2 * clusters), dim3(kThreads), kSmemBytes, s,
                      m[0], m[1], m[2], m[3], a);
}

int64_t tiles_of(int64_t n, int64_t by) { return (n + by - 1) / by; }

// Row tiles that run together: half of the pairs that are resident, so that
// two columns of tiles are in flight.
constexpr int kGroup = 38;

}  // namespace

int head_loss_columns(int64_t rows, int64_t V) {
    (void)rows;
    (void)V;
    return 256;
}

cudaError_t launch_head_lse(const HeadLogits& h, cudaStream_t s) {
    CUtensorMap m[4];
    if (!operand_map(&m[0], h.H) || !operand_map(&m[2], h.E)) return cudaErrorInvalidValue;
    m[1] = m[0];
    m[3] = m[0];
    TcArgs a = {};
    a.rows = h.H.rows;
    a.d = h.H.cols;
    a.n = h.n;
    a.v0 = h.v0;
    a.planes = h.H.planes;
    a.bn = head_loss_columns(a.rows, a.n);
    a.group = kGroup;
    a.scale = h.scale;
    a.targets = h.targets;
    a.T = h.T;
    a.part = h.part;
    a.ld_part = h.ld_part;
    a.picked = h.picked;
    return launch_tc<kLse, 1>(m, a, tiles_of(a.rows, kHeadTile) * tiles_of(a.n, a.bn), s);
}

cudaError_t launch_head_factor(const HeadLogits& h, cudaStream_t s) {
    CUtensorMap m[4];
    if (!operand_map(&m[0], h.H) || !operand_map(&m[2], h.E) ||
        !make_map(&m[3], h.G, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return cudaErrorInvalidValue;
    m[1] = m[0];
    if (h.Hc.base && !operand_map(&m[1], h.Hc)) return cudaErrorInvalidValue;
    TcArgs a = {};
    a.rows = h.H.rows;
    a.d = h.H.cols;
    a.n = h.n;
    a.v0 = h.v0;
    a.counts = h.counts;
    a.planes = h.H.planes;
    a.bn = 256;
    a.group = kGroup;
    a.scale = h.scale;
    a.info = h.rows;
    const int64_t tiles = tiles_of(a.rows, kHeadTile) * tiles_of(a.n, a.bn);
    return a.planes == 1 ? launch_tc<kFactor, 1>(m, a, tiles, s)
                         : launch_tc<kFactor, 3>(m, a, tiles, s);
}

size_t head_acc_bytes(int64_t rows, int64_t d) {
    return sizeof(float) * kHeadTile * kHeadTile *
           static_cast<size_t>(tiles_of(rows, kHeadTile) * tiles_of(d, 128));
}

cudaError_t launch_head_products(const HeadProducts& h, cudaStream_t s) {
    CUtensorMap m[4];
    if (!operand_map(&m[0], h.G) || !operand_map(&m[1], h.E) || !operand_map(&m[2], h.H))
        return cudaErrorInvalidValue;
    m[3] = m[2];
    if (h.Hc.base && !operand_map(&m[3], h.Hc)) return cudaErrorInvalidValue;
    TcArgs a = {};
    a.rows = h.H.rows;
    a.d = h.d;
    a.n = h.n;
    a.v0 = h.v0;
    a.counts = h.counts;
    a.planes = h.G.planes;
    a.bn = h.d <= 128 ? 128 : 256;
    a.scale = h.scale;
    a.row_of = h.row_of;
    a.gH = static_cast<unsigned char*>(h.gH);
    a.ld_gh = h.ld_gh;
    a.gh_acc = h.gh_acc;
    a.gE = static_cast<unsigned char*>(h.gE);
    a.gh_bf16 = h.gh_bf16;
    a.ge_bf16 = h.ge_bf16;
    const auto vec = [](const void* p, int64_t ld, bool bf16) {
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * (bf16 ? 2 : 4) % 16 == 0;
    };
    a.gh_vec = vec(h.gH, h.ld_gh, h.gh_bf16);
    a.ge_vec = vec(h.gE, h.d, h.ge_bf16);
    a.first = h.first;
    a.last = h.last;
    a.accumulate = h.accumulate;
    const int64_t nt = tiles_of(a.d, a.bn);
    const int64_t tiles = (h.gH ? tiles_of(a.rows, kHeadTile) * nt : 0) +
                          (h.gE ? tiles_of(a.n, kHeadTile) * nt : 0);
    return launch_tc<kMul, 1>(m, a, tiles, s);
}

}  // namespace dust
