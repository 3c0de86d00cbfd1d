// Tensor-core products of the gated feed-forward block (tcgen05, sm_103a).
//
//   kUp    g = X Wg^T and u = X Wu^T tile by tile, never stored: h = act(g) u;
//   kBack  the same tiles again, as dG = gh u act'(g) and dU = gh act(g) beside
//          each other in D, rounded to bf16 (fp32: as three bf16 planes);
//   kMul   gX = D [Wg; Wu] and [gWg; gWu] = D^T X, the tiles of both in one
//          launch.
//
// The tiles, their stages and their pairs of CTAs are those of the head's
// products. What is particular: of a tile's columns the first half are gates
// and the second half the same units' ups. Rank 0's half of B comes from Wg and
// rank 1's from Wu, so that both accumulators of a unit lie in one thread of
// the epilogue, 128 (64) columns apart, and nothing but h (or D) is written.
//
// fp32 products load all three planes of a step together and take narrow
// tiles, whose largest product has an accumulator of its own; their sums are
// joined from runs of steps (pair_tile.cuh says why).
//
// Bound by the tensor pipe: kUp of 65536 rows, d 512, f 2048 takes 156 to 164 us
// alone, 1680 to 1760 TFLOP/s (84 % busy: 54 rounds of 8 steps), 185 in a long
// row of calls, under the power limit; the gradients of 8192 rows, d 2048, f
// 8192 868 to 1000 us, 1900 to 1650 TFLOP/s (80 % busy in kBack, whose gh and D
// are 400 MB, 98 % in kMul). With d 512 kBack takes 215 us for 65536 rows, where
// its products alone would take 143: gh and D, 800 MB, stand beside the
// operands' loads, and every step fewer in flight costs (5 steps 5 us, 4 45 us).
// fp32 (six products): 4096 rows, d 512, f 2048 74 us, gradients 237 to 243: the
// copies into planes 13, D's tiles 93 (49 % of the tensor pipe: the runs' joining
// and three planes of D in the epilogues), the products 134 (78 %).
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "gated.cuh"
#include "pair_tile.cuh"

namespace dust {

namespace {

enum Mode { kUp, kBack, kMul };

// Steps that fp32 products add up in TMEM at a time: half of the head's, as what
// the tensor cores cut off shows twice here, in g and u and in the products of D
// (439 rows, d 1568, squared ReLU: h 1.3e-6 off with 8 steps, 6.2e-7 with 4).
constexpr int kFewSteps = kRun / 2;

// Steps in flight; kBack's epilogue warps hold their part of gh as well.
template <int MODE> constexpr int kDepth = MODE == kBack ? kStages - 1 : kStages;
constexpr int kHeldBytes = 32 * 128;  // 32 rows of 64 bf16 units, or of 32 fp32 ones
template <int MODE> constexpr int smem_of() {
    return kDepth<MODE> * kStageBytes + 1024 +
           (MODE == kBack ? kStoreBytes + kEpiWarps * kHeldBytes : kEpiWarps * kTurnBuf);
}
static_assert(smem_of<kBack>() + 512 <= 227 * 1024 && smem_of<kUp>() + 512 <= 227 * 1024,
              "shared memory per CTA, barriers included");

struct TcArgs {
    int64_t T, d, f, fp;       // fp: columns of D per half
    int bn;                    // tile columns
    int group;                 // row tiles that run together (kUp, kBack)
    int act;
    OutRows h;                 // kUp
    OutRows gX, gW[2];         // kMul
    int halves, first_half;    // of gWg and gWu, those that are wanted
    float *gx_acc, *gw_acc;    // tiles of partial sums, by unit
    int cut0, cut1, accumulate;
    int stall;
    unsigned int* status;
};

// Where a unit of work lies: which product (0: g and u, or gX; 1: gWg or gWu),
// its first row (of `half`: a unit of the block), its first unit (kUp, kBack)
// or column, and its steps along the summed dimension.
struct Tile {
    int job, half;
    int64_t m0, n0;
    int k0, steps;
    int index;  // the unit of work (kMul)
};

__device__ __forceinline__ Tile uniform(const Tile& t) {
    Tile w;
    w.job = uniform(t.job);
    w.half = uniform(t.half);
    w.m0 = uniform(static_cast<int>(t.m0));
    w.n0 = uniform(static_cast<int>(t.n0));
    w.k0 = uniform(t.k0);
    w.steps = uniform(t.steps);
    w.index = t.index;
    return w;
}

template <int MODE>
struct Plan : Deal {
    int mt, nt;              // tiles of job 0
    int mw;                  // row tiles of one half of job 1
    int steps0, steps1;      // of a whole tile
    int half_steps;          // kMul: of either half of job 0's sums
    bool one_first;          // kMul: job 1's units are the longer ones
    Divider by_nt, by_group, by_gm, by_last;

    __device__ Plan(const TcArgs& a, int c, int n)
        : Deal(c, n), by_nt(1), by_group(1), by_gm(1), by_last(1) {
        mt = divide_up(a.T, kHeadTile);
        half_steps = divide_up(a.f, 64);
        mw = 0;
        one_first = false;
        if (MODE != kMul) {
            nt = divide_up(a.f, a.bn / 2);
            steps0 = divide_up(a.d, 64);
            steps1 = 0;
            total = mt * nt;
            by_group = Divider(a.group * nt);
            by_gm = Divider(a.group);
            by_last = Divider(mt % a.group);
        } else {
            nt = divide_up(a.d, a.bn);
            steps0 = 2 * half_steps;
            steps1 = divide_up(a.T, 64);
            mw = divide_up(a.f, kHeadTile);
            const int units0 = (a.gX.base ? mt : 0) * nt * a.cut0;
            const int units1 = a.halves * mw * nt * a.cut1;
            const int cost0 = max(1, divide_up(steps0, a.cut0));
            const int cost1 = max(1, divide_up(steps1, a.cut1));
            one_first = cost1 > cost0;
            deal(one_first ? units1 : units0, one_first ? units0 : units1, max(cost0, cost1),
                 min(cost0, cost1));
        }
        by_nt = Divider(nt);
    }

    // The i-th unit of this cluster, or -1.
    __device__ int unit(int i) const {
        if (MODE == kMul) return dealt(i);
        const int64_t t = cluster + static_cast<int64_t>(i) * clusters;
        return t < total ? static_cast<int>(t) : -1;
    }

    __device__ Tile at(const TcArgs& a, int t) const {
        Tile w;
        w.half = 0;
        if (MODE != kMul) {
            // Groups of row tiles; inside one, rows fastest: the group's rows of
            // X stay in L2 while the weights stream by once per group.
            int g, in, c, r;
            by_group(t, g, in);
            if ((g + 1) * a.group <= mt)
                by_gm(in, c, r);
            else
                by_last(in, c, r);
            w.job = 0;
            w.m0 = static_cast<int64_t>(g * a.group + r) * kHeadTile;
            w.n0 = static_cast<int64_t>(c) * (a.bn / 2);
            w.k0 = 0;
            w.steps = steps0;
            w.index = t;
        } else {
            const bool job1 = (t < longs) == one_first;
            const int i = t < longs ? t : t - longs;
            const int cut = job1 ? a.cut1 : a.cut0;
            const int steps = job1 ? steps1 : steps0;
            int tile = i;
            w.k0 = 0;
            w.steps = steps;
            if (cut > 1) {
                tile = i / cut;
                const int64_t part = i - tile * cut;
                w.k0 = static_cast<int>(steps * part / cut);
                w.steps = static_cast<int>(steps * (part + 1) / cut) - w.k0;
            }
            int r, c;  // columns fastest: a row block of D is read by neighbours
            by_nt(tile, r, c);
            w.job = job1 ? 1 : 0;
            if (job1) {
                w.half = a.first_half + (r >= mw ? 1 : 0);
                if (r >= mw) r -= mw;
            }
            w.m0 = static_cast<int64_t>(r) * kHeadTile;
            w.n0 = static_cast<int64_t>(c) * a.bn;
            w.index = i;
        }
        return w;
    }
};

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// As pack2, but the largest bf16 numbers where these round to infinity.
__device__ __forceinline__ uint32_t pack2_finite(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The sigmoid p of z, and exp(-z) as far as it is finite (so that p times it,
// what p leaves to 1, is a number where p is 0): by the special-function units where the result is
// rounded to bf16 (2^-22 off at z near 0, |z| 2^-24 further out), by expf and a
// division for fp32.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z, float& e) {
    const float x = EXACT ? expf(-z) : ex2(-1.4426950408889634f * z);
    e = fminf(x, 0x1p126f);
    return EXACT ? 1.0f / (1.0f + x) : rcp(1.0f + x);
}

// z of the tanh form: the gate's probability is the sigmoid of it.
__device__ __forceinline__ float gelu_z(float g) {
    constexpr float kB = 0.044715f, kC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    return kC * g * fmaf(kB * g, g, 1.0f);
}

// h = act(g) u, over g.
template <int ACT, bool EXACT>
__device__ __forceinline__ void forward(float (&g)[32], const float (&u)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        float e;
        if (ACT == DUST_ACT_RELU2) {
            const float r = max_nan(g[i], 0.0f);
            g[i] = r * r * u[i];
        } else {
            g[i] = g[i] * sigmoid<EXACT>(ACT == DUST_ACT_GELU ? gelu_z(g[i]) : g[i], e) * u[i];
        }
    }
}

// dG = gh u act'(g) over g, dU = gh act(g) over u.
template <int ACT, bool EXACT>
__device__ __forceinline__ void backward(float (&g)[32], float (&u)[32], const float (&gh)[32]) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float x = g[i];
        float act, slope;
        if (ACT == DUST_ACT_RELU2) {
            const float r = max_nan(x, 0.0f);
            act = r * r;
            slope = 2.0f * r;
        } else {
            float e, dz = x;
            const float p = sigmoid<EXACT>(ACT == DUST_ACT_GELU ? gelu_z(x) : x, e);
            if (ACT == DUST_ACT_GELU) {
                // Far out p (1 - p) is 0, and its factor has to stay finite there: all
                // of it at the nearer of x and 1e4.
                const float y = fminf(fmaxf(x, -1e4f), 1e4f);
                dz = y * (1.5957691216057308f * fmaf(3.0f * 0.044715f * y, y, 1.0f));
            }
            act = x * p;
            slope = fmaf(dz, p * (p * e), p);
        }
        g[i] = gh[i] * u[i] * slope;
        u[i] = gh[i] * act;
    }
}

template <bool EXACT>
__device__ __forceinline__ void forward_by(int act, float (&g)[32], const float (&u)[32]) {
    if (act == DUST_ACT_SILU) forward<DUST_ACT_SILU, EXACT>(g, u);
    else if (act == DUST_ACT_GELU) forward<DUST_ACT_GELU, EXACT>(g, u);
    else forward<DUST_ACT_RELU2, EXACT>(g, u);
}

template <bool EXACT>
__device__ __forceinline__ void backward_by(int act, float (&g)[32], float (&u)[32], const float (&gh)[32]) {
    if (act == DUST_ACT_SILU) backward<DUST_ACT_SILU, EXACT>(g, u, gh);
    else if (act == DUST_ACT_GELU) backward<DUST_ACT_GELU, EXACT>(g, u, gh);
    else backward<DUST_ACT_RELU2, EXACT>(g, u, gh);
}

// Epilogue of one unit of work for one warp: rows 32 q + lane of this CTA's
// half, and of the tile's units or columns the h-th half.
template <int MODE, int PLANES>
struct Epilogue {
    static constexpr bool kRuns = PLANES == 3;
    const TcArgs& a;
    const CUtensorMap *tmD, *tmGh;
    unsigned char* bufs;  // this warp's: kBack's store buffers, the others' 32 x 32 values
    unsigned char* held;  // kBack: this warp's part of gh
    uint64_t* landed;     // and its barrier
    uint32_t rank;
    int q, h, lane;
    uint32_t used = 0;
    uint32_t asked = 0, got = 0;  // kBack: parts of gh
    // A unit's sums over its runs of steps but the last, and whether there are
    // such: of kUp and kBack 32 gates and 32 ups, of kMul 64 columns.
    static constexpr int kSums = kRuns ? 64 : 1;
    float sum[kSums] = {};
    bool summed = false;

    __device__ int64_t row_of(const Tile& w) const { return w.m0 + rank * kHalf + 32 * q + lane; }

    // Whether any of this warp's 32 rows is wanted: of D, kMul sums over rows up
    // to the next multiple of 64.
    __device__ bool wanted(const Tile& w) const {
        const int64_t row = w.m0 + rank * kHalf + 32 * q;
        if (MODE == kMul) return row < (w.job == 1 ? a.f : a.T);
        return row < (MODE == kBack ? (a.T + 63) / 64 * 64 : a.T);
    }

    // The tile's b-th 32 units of this warp.
    __device__ int unit_of(int b) const { return h * (a.bn / 4) + 32 * b; }

    // Asks for this warp's rows and units of gh (zeros where there are none).
    // All lanes have read the last ones.
    __device__ void fetch(const Tile& w) {
        if (lane == 0) {
            tc::mbar_arrive_expect_tx(landed, kHeldBytes);
            tc::tma_load_2d(held, tmGh, static_cast<int32_t>(w.n0) + unit_of(0),
                            static_cast<int32_t>(row_of(w)), landed);
        }
        ++asked;
    }

    // Block b of what was asked for: a lane's row lies in 16-byte pieces that
    // the row's number permutes.
    __device__ void take(int b, float (&v)[32]) const {
        constexpr int kVecs = PLANES == 1 ? 4 : 8;
        const unsigned char* row = held + lane * 128;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const uint4 x = *reinterpret_cast<const uint4*>(row + (((b * kVecs + i) ^ (lane & 7)) << 4));
            const uint32_t r[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (PLANES == 1) {
                    v[(8 * i + 2 * k) % 32] = __uint_as_float(r[k] << 16);
                    v[(8 * i + 2 * k + 1) % 32] = __uint_as_float(r[k] & 0xffff0000u);
                } else {
                    v[4 * i + k] = __uint_as_float(r[k]);
                }
            }
        }
    }

    __device__ void up(const Tile& w, uint32_t taddr) {
        const int64_t row = row_of(w);
        const int32_t to = row < a.T ? static_cast<int32_t>(row) : -1;
#pragma unroll 1
        for (int b = 0; b < a.bn / 128; ++b) {
            const int c = unit_of(b);
            const int64_t unit = w.n0 + c;
            if (unit >= a.f) break;
            float g[32], u[32];
            whole_sum(taddr, c, 0, g);
            whole_sum(taddr, a.bn / 2 + c, 1, u);
            forward_by<PLANES == 3>(a.act, g, u);
            const int n = a.f - unit < 32 ? static_cast<int>(a.f - unit) : 32;
            store_block(tc::smem_u32(bufs), g, lane, to, a.h, unit, n, false);
        }
    }

    // `next`: the tile to ask for once this one's part of gh has been read.
    __device__ void back(const Tile& w, const Tile* next, uint32_t taddr) {
        const int64_t row = row_of(w);
        const int blocks = a.bn / 128;
#pragma unroll 1
        for (int b = 0; b < blocks; ++b) {
            const int c = unit_of(b);
            const int64_t unit = w.n0 + c;
            float g[32], u[32], gh[32];
            take(b, gh);
            if (b + 1 == blocks) {
                __syncwarp();
                if (next) fetch(*next);
            }
            if (unit >= (a.f + 63) / 64 * 64) continue;
            whole_sum(taddr, c, 0, g);
            whole_sum(taddr, a.bn / 2 + c, 1, u);
            backward_by<PLANES == 3>(a.act, g, u, gh);
            const int left = row < a.T ? static_cast<int>(min(a.f - unit, static_cast<int64_t>(32))) : 0;
            if (left < 32) {  // D is zero where there is no row or unit
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    g[i] = i < left ? g[i] : 0.0f;
                    u[i] = i < left ? u[i] : 0.0f;
                }
            }
            store_planes(g, static_cast<int32_t>(unit), static_cast<int32_t>(row - lane));
            store_planes(u, static_cast<int32_t>(a.fp + unit), static_cast<int32_t>(row - lane));
        }
    }

    // The same, once this warp's part of gh is there; false if it did not come.
    __device__ bool back_when_landed(const Tile& w, const Tile* next, uint32_t taddr, uint64_t limit_ns,
                                     volatile int* abort_flag) {
        if (!__all_sync(0xffffffffu, wait_or_abort(landed, got & 1, limit_ns, abort_flag))) {
            *abort_flag = 1;
            return false;
        }
        ++got;
        back(w, next, taddr);
        return true;
    }

    // The block's dG or dU as planes of D. One plane keeps 8 bits of them: D is an
    // operand of bf16 products. Beside gX's and the weights' own rounding (1.7e-3,
    // normwise) that makes their gradients 2.3e-3 off, and fp32 gWg and gWu 1.7e-3
    // (8192 rows, 2048 -> 8192: 2.55e-3 from what fp32 dG and dU give, rounded, of
    // which all but 0.5e-3 goes when those are rounded as here). A second plane
    // would double the products, which take two thirds of the time; fp32 inputs
    // have three.
    __device__ void store_planes(float (&v)[32], int32_t col, int32_t row0) {
        const uint32_t swz = (lane >> 1) & 3;
#pragma unroll
        for (int p = 0; p < PLANES; ++p) {
            unsigned char* buf = bufs + (used % kStoreBufs) * kStageBuf;
            if (used >= kStoreBufs) {
                if (lane == 0) tc::bulk_wait_read<kStoreBufs - 1>();
                __syncwarp();
            }
            const uint32_t dst = tc::smem_u32(buf) + lane * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t pk[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x0 = v[8 * i + 2 * j], x1 = v[8 * i + 2 * j + 1];
                    // The largest of several planes: not up to infinity, of which the
                    // others could not take anything back.
                    pk[j] = PLANES > 1 && p == 0 ? pack2_finite(x0, x1) : pack2(x0, x1);
                    if (p + 1 < PLANES) {  // what this plane leaves
                        v[8 * i + 2 * j] = x0 - __uint_as_float(pk[j] << 16);
                        v[8 * i + 2 * j + 1] = x1 - __uint_as_float(pk[j] & 0xffff0000u);
                    }
                }
                st_shared_16(dst + ((i ^ swz) << 4), pk);
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                // D is padded to whole tiles: every block lies inside.
                tc::tma_store_3d(tmD, buf, col, row0, p);
                tc::bulk_commit();
            }
            ++used;
        }
    }

    // Columns [at, at + 32) of the accumulators of a run of steps: both of them
    // for fp32. TMEM is read by whole warps at once: the lanes meet first.
    __device__ void accumulators(uint32_t taddr, int at, float (&v)[32]) const {
        __syncwarp();
        tc::tmem_ld_32x32(taddr + at, v);
        if (PLANES == 3) {
            float big[32];
            tc::tmem_ld_32x32(taddr + 128 + at, big);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += big[i];
        }
    }

    // The same of the unit's whole sum, after its last run; `part`: which of the
    // warp's two blocks of columns.
    __device__ void whole_sum(uint32_t taddr, int at, int part, float (&v)[32]) const {
        accumulators(taddr, at, v);
        if (kRuns && summed) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += part ? sum[(32 + i) % kSums] : sum[i % kSums];
        }
    }

    // Adds a run that is not the last to the unit's sums.
    __device__ void collect(uint32_t taddr, bool first) {
#pragma unroll
        for (int b = 0; b < kSums / 32; ++b) {
            float v[32];
            accumulators(taddr, MODE == kMul ? h * 64 + 32 * b : 64 * b + 32 * h, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                sum[(32 * b + i) % kSums] = first ? v[i] : sum[(32 * b + i) % kSums] + v[i];
        }
    }

    __device__ void product(const Tile& w, uint32_t taddr) {
        const int cols = a.bn / kShare;
        const bool job1 = w.job == 1, zero = w.steps == 0;
        float* acc = job1 ? a.gw_acc : a.gx_acc;
        const bool whole = (job1 ? a.cut1 : a.cut0) == 1;
        const OutRows& out = job1 ? a.gW[w.half] : a.gX;
        const int64_t row = row_of(w);
        const int32_t to = row < (job1 ? a.f : a.T) ? static_cast<int32_t>(row) : -1;
#pragma unroll 1
        for (int b = 0; b < cols / 32; ++b) {
            const int at = h * cols + 32 * b;
            const int64_t col = w.n0 + at;
            if (col >= a.d) break;
            float v[32];
            whole_sum(taddr, at, b & 1, v);
            const int n = a.d - col < 32 ? static_cast<int>(a.d - col) : 32;
            if (zero) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = 0.0f;
            }
            if (whole) {
                store_block(tc::smem_u32(bufs), v, lane, to, out, col, n, job1 && a.accumulate);
                continue;
            }
            // Partial sums lie as the accumulator has them: four columns of all
            // rows together.
            float4* p = reinterpret_cast<float4*>(acc + static_cast<int64_t>(w.index) * kSlotFloats) +
                        at / 4 * kHeadTile + static_cast<int>(rank) * kHalf + 32 * q + lane;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p[i * kHeadTile] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
    }
};

// Maps: kUp X, Wg, Wu, -, -; kBack X, Wg, Wu, D, gh; kMul D, Wg, Wu, X, -.
template <int MODE, int PLANES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_gated_tc(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
               const __grid_constant__ CUtensorMap tm2, const __grid_constant__ CUtensorMap tm3,
               const __grid_constant__ CUtensorMap tm4, const __grid_constant__ TcArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* store_bufs = smem + kDepth<MODE> * kStageBytes;
    __shared__ Ctl ctl_s;
    __shared__ uint64_t gh_landed[kEpiWarps];
    Ctl* ctl = &ctl_s;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(tc::cluster_rank_of_cta());
    const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kDepth<MODE>; ++i) {
            tc::mbar_init(&ctl->full[i], 1);
            tc::mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&ctl->tfull[i], 1);
            tc::mbar_init(&ctl->tempty[i], 2 * kEpiWarps);
        }
        for (int i = 0; i < kEpiWarps; ++i) tc::mbar_init(&gh_landed[i], 1);
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

    const Plan<MODE> plan(a, cluster, n_clusters);
    const int b_boxes = a.bn / 128;  // per CTA
    const int run = PLANES == 3 ? kFewSteps : 1 << 30;
    // A tile's products take about 0.3 us per step: the waits for a whole
    // tile are given 2 us per step on top of the usual limit.
    const uint64_t tile_ns = tc::kWaitNs + 2000ull * static_cast<uint64_t>(PLANES == 3 ? 6 : 1) *
                                               max(plan.steps0, plan.steps1);

    // Whole warps go through the steps of the loads and of the products, one
    // lane issues them: operands then lie in uniform registers.
    if (warp == 0) {
        const bool one = elect_one();
        const uint32_t full = tc::at_rank(&ctl->full[0], 0);
        const uint32_t bytes = 2 * (2 + b_boxes) * kBoxBytes;  // of a step, both CTAs
        int it = 0, st = 0;
        uint32_t parity = 1;
        bool stop = false;
        for (int j = 0, t; !stop && (t = uniform(plan.unit(j))) >= 0; ++j) {
            const Tile w = uniform(plan.at(a, t));
            const bool a_mn = MODE == kMul && w.job == 1, b_mn = MODE == kMul;
            const int32_t am = static_cast<int32_t>(w.m0) + static_cast<int32_t>(rank) * kHalf +
                               (a_mn ? w.half * static_cast<int32_t>(a.fp) : 0);
            // kUp and kBack: the same units of either matrix.
            const int32_t bn0 = static_cast<int32_t>(w.n0) +
                                (MODE == kMul ? static_cast<int32_t>(rank) * (a.bn / 2) : 0);
            for (int c = 0; c < w.steps && !stop; ++c) {
                const int k = w.k0 + c;
                int32_t ak = k * 64, bk = ak;
                const CUtensorMap* mb = MODE != kMul ? (rank == 0 ? &tm1 : &tm2) : w.job ? &tm3 : &tm1;
                if (MODE == kMul && w.job == 0 && k >= plan.half_steps) {
                    bk = (k - plan.half_steps) * 64;
                    ak = static_cast<int32_t>(a.fp) + bk;
                    mb = &tm2;
                }
                for (int i = 0; i < PLANES; ++i, ++it) {
                    const int p = PLANES - 1 - i;  // the smallest plane first
                    if (!warp_wait(&ctl->empty[st], parity, tile_ns, abort_flag)) {
                        *abort_flag = 1;
                        stop = true;
                        break;
                    }
                    unsigned char* base = smem + st * kStageBytes;
                    const uint32_t bar = full + st * 8;
                    if (one) {
                        if (rank == 0) tc::mbar_arrive_expect_tx(&ctl->full[st], bytes);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            tc::tma_load_3d_pair(base + u * kBoxBytes, &tm0, a_mn ? am + 64 * u : ak,
                                                 a_mn ? ak : am + 64 * u, p, bar);
                        tc::tma_load_3d_pair(base + 2 * kBoxBytes, mb, b_mn ? bn0 : bk, b_mn ? bk : bn0, p,
                                             bar);
                        if (b_boxes == 2)
                            tc::tma_load_3d_pair(base + 3 * kBoxBytes, mb, b_mn ? bn0 + 64 : bk,
                                                 b_mn ? bk : bn0 + 64, p, bar);
                    }
                    __syncwarp();
                    if (++st == kDepth<MODE>) {
                        st = 0;
                        parity ^= 1;
                    }
                }
            }
        }
        if (lane == 0) ctl->issued = it;
        // The last stages' releases land here, too, before the CTA may leave: they
        // come from the pair's first CTA, whenever their products are done.
        for (int i = 0; i < kDepth<MODE> && !stop; ++i) {
            if (!warp_wait(&ctl->empty[st], parity, tile_ns, abort_flag)) {
                *abort_flag = 1;
                stop = true;
            }
            if (++st == kDepth<MODE>) {
                st = 0;
                parity ^= 1;
            }
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool one = elect_one();
            bool stop = a.stall && !__all_sync(0xffffffffu, tc::mbar_wait(&ctl->never, 0));
            const uint32_t acc0 = uniform(tmem);
            int it = 0, st = 0;
            uint32_t parity = 0;
            const auto advance = [&] {
                ++it;
                if (++st == kDepth<MODE>) {
                    st = 0;
                    parity ^= 1;
                }
            };
            const auto landed = [&] { return warp_wait(&ctl->full[st], parity, tc::kWaitNs, abort_flag); };
            int t = uniform(plan.unit(0));
            Tile next = t >= 0 ? uniform(plan.at(a, t)) : Tile{};
            // Accumulators are filled in turn, one per run of steps of a unit.
            Tile w = next;
            for (int j = 0, i = 0, c = 0; !stop && (c > 0 || t >= 0); ++j) {
                if (c == 0) {
                    w = next;
                    // The next one's place is worked out before this one's steps.
                    t = uniform(plan.unit(++i));
                    if (t >= 0) next = uniform(plan.at(a, t));
                }
                const int acc = j & 1, steps = min(run, w.steps - c);
                if (!warp_wait(&ctl->tempty[acc], ((j >> 1) & 1) ^ 1, tile_ns, abort_flag)) {
                    stop = true;
                    break;
                }
                tc::tc_fence_after();
                const bool a_mn = MODE == kMul && w.job == 1, b_mn = MODE == kMul;
                const uint32_t idesc = tc::idesc_bf16(kHeadTile, a.bn, a_mn, b_mn);
                const uint32_t dst = acc0 + acc * 256;
                const Operand A = {tc::sdesc_sw128(tc::smem_u32(smem), a_mn ? kBoxBytes : 16, 1024),
                                   a_mn ? 2048u : 32u};
                const Operand B = {tc::sdesc_sw128(tc::smem_u32(smem + 2 * kBoxBytes),
                                                   b_mn ? kBoxBytes : 16, 1024),
                                   b_mn ? 2048u : 32u};
                for (int k = 0; k < steps; ++k) {
                    const int s2 = st;
                    stop = !landed();
                    if (stop) break;
                    advance();
                    if (PLANES == 1) {
                        tc::tc_fence_after();
                        if (one) {
                            issue_step(dst, A, s2, B, s2, idesc, k != 0);
                            tc::mma_commit_pair(&ctl->empty[s2]);
                        }
                        __syncwarp();
                        continue;
                    }
                    const int s1 = st;
                    stop = !landed();
                    if (stop) break;
                    advance();
                    const int s0 = st;
                    stop = !landed();
                    if (stop) break;
                    advance();
                    tc::tc_fence_after();
                    if (one) {
                        issue_step(dst, A, s2, B, s0, idesc, k != 0);
                        issue_step(dst, A, s0, B, s2, idesc, true);
                        tc::mma_commit_pair(&ctl->empty[s2]);
                        issue_step(dst, A, s1, B, s1, idesc, true);
                        issue_step(dst, A, s1, B, s0, idesc, true);
                        issue_step(dst, A, s0, B, s1, idesc, true);
                        tc::mma_commit_pair(&ctl->empty[s1]);
                        issue_step(dst + 128, A, s0, B, s0, idesc, k != 0);
                        tc::mma_commit_pair(&ctl->empty[s0]);
                    }
                    __syncwarp();
                }
                if (stop) break;
                if (one) tc::mma_commit_pair(&ctl->tfull[acc]);
                __syncwarp();
                c = w.steps - c > run ? c + run : 0;
            }
            if (one) {
                if (stop) *abort_flag = 1;
                ctl->consumed = it;
                if (stop) {
                    // Everything issued so far has to be done before TMEM is freed.
                    tc::mma_commit_pair(&ctl->drain);
                    tc::mbar_wait_for(&ctl->drain, 0, tc::kWaitNs);
                }
            }
            __syncwarp();
        }
    } else {
        const int ew = warp - 2, q = warp & 3, h = ew >> 2;
        constexpr int kOwn = MODE == kBack ? kStoreBufs * kStageBuf : kTurnBuf;
        Epilogue<MODE, PLANES> epi{a, &tm3, &tm4, store_bufs + kEpiWarps * kHeldBytes * (MODE == kBack) + ew * kOwn,
                                   store_bufs + ew * kHeldBytes, &gh_landed[ew], rank, q, h, lane};
        bool ok = true;
        int t = plan.unit(0);
        Tile w = t >= 0 ? plan.at(a, t) : Tile{};
        if (MODE == kBack && t >= 0 && epi.wanted(w)) epi.fetch(w);
        for (int i = 1, j = 0; ok && t >= 0; ++i) {
            const bool wanted = epi.wanted(w);
            t = plan.unit(i);
            const Tile next = t >= 0 ? plan.at(a, t) : Tile{};
            const bool next_wanted = t >= 0 && epi.wanted(next);
            for (int c = 0; ok && c >= 0; ++j) {  // runs of steps
                const int acc = j & 1;
                ok = __all_sync(0xffffffffu, wait_or_abort(&ctl->tfull[acc], (j >> 1) & 1, tile_ns,
                                                           abort_flag) && !*abort_flag);
                tc::tc_fence_after();
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                const bool last = w.steps - c <= run;
                const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * 256;
                if (wanted) {
                    if (PLANES == 3 && !last) {
                        epi.collect(taddr, c == 0);
                    } else {
                        epi.summed = c > 0;
                        if constexpr (MODE == kUp)
                            epi.up(w, taddr);
                        else if constexpr (MODE == kBack)
                            ok = epi.back_when_landed(w, next_wanted ? &next : nullptr, taddr, tile_ns,
                                                      abort_flag);
                        else
                            epi.product(w, taddr);
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_at(tc::at_rank(&ctl->tempty[acc], 0));
                c = last ? -1 : c + run;
            }
            if (MODE == kBack && ok && !wanted && next_wanted) epi.fetch(next);
            w = next;
        }
        if (MODE == kBack) {
            // A part of gh that was asked for and not used lands first.
            if (epi.asked != epi.got) tc::mbar_wait(&gh_landed[ew], epi.got & 1);
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
                tc::mbar_wait(&ctl->full[it % kDepth<MODE>], (it / kDepth<MODE>) & 1);
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

// The slices' partial sums added in order, into gX (t0 tiles) and gWg, gWu (t1
// tiles): a CTA takes 32 rows and 32 columns of a tile at a time.
__global__ void __launch_bounds__(256)
    k_gated_sum(const __grid_constant__ TcArgs a, int64_t t0, int64_t t1) {
    pdl_wait();
    pdl_trigger();
    const int nt = divide_up(a.d, a.bn), mw = divide_up(a.f, kHeadTile);
    const int per = 8 * (a.bn / 32);
    const int lane = threadIdx.x & 31, c4 = threadIdx.x >> 5;
    for (int64_t b = blockIdx.x; b < (t0 + t1) * per; b += gridDim.x) {
        const bool job = b >= t0 * per;
        const int64_t tile = b / per - (job ? t0 : 0);
        const int in = static_cast<int>(b % per);
        const int r = (in & 7) * 32 + lane, c = (in >> 3) * 32 + c4 * 4;
        int64_t rt = tile / nt;
        const int half = job ? a.first_half + (rt >= mw ? 1 : 0) : 0;
        if (job && rt >= mw) rt -= mw;
        const int64_t row = rt * kHeadTile + r, col = tile % nt * a.bn + c;
        if (row >= (job ? a.f : a.T) || col >= a.d) continue;
        const int cut = job ? a.cut1 : a.cut0;
        const float4* p = reinterpret_cast<const float4*>((job ? a.gw_acc : a.gx_acc) +
                                                          tile * cut * kSlotFloats) +
                          c / 4 * kHeadTile + r;
        float4 v = *p;
        for (int k = 1; k < cut; ++k) {
            const float4 u = p[static_cast<int64_t>(k) * (kSlotFloats / 4)];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        const float x[4] = {v.x, v.y, v.z, v.w};
        const OutRows& out = job ? a.gW[half] : a.gX;
        unsigned char* at = out.base + row * out.pitch;
        for (int i = 0; i < 4 && col + i < a.d; ++i) {
            if (out.bf16) {
                reinterpret_cast<__nv_bfloat16*>(at)[col + i] = __float2bfloat16_rn(x[i]);
            } else {
                float* o = reinterpret_cast<float*>(at) + col + i;
                *o = job && a.accumulate ? *o + x[i] : x[i];
            }
        }
    }
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
        const void* k = reinterpret_cast<const void*>(k_gated_tc<MODE, PLANES>);
        if (ensure_smem_limit(k, smem_of<MODE>()) != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem_of<MODE>();
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
cudaError_t launch_tc(const CUtensorMap (&m)[5], TcArgs a, int64_t tiles, cudaStream_t s) {
    const int fit = max_clusters<MODE, PLANES>();
    if (fit <= 0) return cudaErrorUnknown;
    if (tiles <= 0) return cudaSuccess;
    if (tiles > (int64_t(1) << 30)) return cudaErrorInvalidValue;
    a.status = status_word();
    if (!a.status) return cudaErrorUnknown;
    a.stall = take_stall_injection() ? 1 : 0;
    const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, fit));
    return launch_pdl(k_gated_tc<MODE, PLANES>, dim3(2 * clusters), dim3(kThreads), smem_of<MODE>(), s,
                      m[0], m[1], m[2], m[3], m[4], a);
}

// Rows of `cols` values that are written.
OutRows out_rows(void* p, int64_t ld, int64_t cols, bool bf16) {
    // The rows' length too: what follows it is not written.
    const int size = bf16 ? 2 : 4;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * size) |
                         static_cast<uintptr_t>(cols * size);
    int align = 16;
    while (align > size && at % align != 0) align /= 2;
    return OutRows{static_cast<unsigned char*>(p), ld * size, bf16, align};
}

// gh as 32 rows of 128 bytes at a time.
bool held_map(CUtensorMap* map, const GatedTiles& t) {
    auto fn = encode_fn();
    if (!fn) return false;
    const bool f32 = t.X.planes == 3;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.f), static_cast<cuuint64_t>(t.T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(t.ld_gh) * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, 32u}, estr[2] = {1, 1};
    return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void*>(t.gh), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_gated_tiles(const GatedTiles& t, cudaStream_t s) {
    CUtensorMap m[5];
    if (!operand_map(&m[0], t.X) || !operand_map(&m[1], t.Wg) || !operand_map(&m[2], t.Wu))
        return cudaErrorInvalidValue;
    m[3] = m[4] = m[0];
    const bool back = t.gh != nullptr;
    const int planes = t.X.planes;
    if (back && (!make_map(&m[3], t.D, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B) || !held_map(&m[4], t)))
        return cudaErrorInvalidValue;
    TcArgs a = {};
    a.T = t.T;
    a.d = t.d;
    a.f = t.f;
    a.fp = gated_half(t.f);
    a.bn = planes == 3 ? 128 : logit_columns(t.T, 2 * t.f);
    a.group = kGroup;
    a.act = t.act;
    if (!back) a.h = out_rows(t.h, t.ld_h, t.f, planes == 1);
    const int64_t tiles = tiles_of(t.T, kHeadTile) * tiles_of(t.f, a.bn / 2);
    if (planes == 1) return back ? launch_tc<kBack, 1>(m, a, tiles, s) : launch_tc<kUp, 1>(m, a, tiles, s);
    return back ? launch_tc<kBack, 3>(m, a, tiles, s) : launch_tc<kUp, 3>(m, a, tiles, s);
}

GatedCuts gated_cuts(int64_t T, int64_t d, int64_t f, int planes) {
    const int64_t nt = tiles_of(d, product_columns(d, planes));
    const Cuts c = cuts_of(tiles_of(T, kHeadTile) * nt, 2 * tiles_of(f, 64),
                           2 * tiles_of(f, kHeadTile) * nt, tiles_of(T, 64), planes);
    return {c.a, c.b};
}

int64_t gated_acc_floats(int64_t rows, int64_t d, int planes, int cut) {
    return tiles_of(rows, kHeadTile) * tiles_of(d, product_columns(d, planes)) * cut * kSlotFloats;
}

cudaError_t launch_gated_products(const GatedProducts& g, cudaStream_t s) {
    CUtensorMap m[5];
    if (!operand_map(&m[0], g.D) || !operand_map(&m[1], g.Wg) || !operand_map(&m[2], g.Wu) ||
        !operand_map(&m[3], g.X))
        return cudaErrorInvalidValue;
    m[4] = m[3];
    const int planes = g.D.planes;
    TcArgs a = {};
    a.T = g.T;
    a.d = g.d;
    a.f = g.f;
    a.fp = gated_half(g.f);
    a.bn = product_columns(g.d, planes);
    if (g.gX) a.gX = out_rows(g.gX, g.ld_gx, g.d, g.bf16);
    a.gW[0] = out_rows(g.gWg, g.d, g.d, g.gW_bf16);
    a.gW[1] = out_rows(g.gWu, g.d, g.d, g.gW_bf16);
    a.halves = (g.gWg ? 1 : 0) + (g.gWu ? 1 : 0);
    a.first_half = g.gWg ? 0 : 1;
    a.gx_acc = g.gx_acc;
    a.gw_acc = g.gw_acc;
    a.cut0 = g.cuts.x;
    a.cut1 = g.cuts.w;
    a.accumulate = g.accumulate;
    const int64_t nt = tiles_of(a.d, a.bn);
    const int64_t t0 = g.gX ? tiles_of(a.T, kHeadTile) * nt : 0;
    const int64_t t1 = a.halves * tiles_of(a.f, kHeadTile) * nt;
    const int64_t units = t0 * a.cut0 + t1 * a.cut1;
    const cudaError_t e = planes == 1 ? launch_tc<kMul, 1>(m, a, units, s) : launch_tc<kMul, 3>(m, a, units, s);
    const int64_t s0 = a.cut0 > 1 ? t0 : 0, s1 = a.cut1 > 1 ? t1 : 0;
    if (e != cudaSuccess || s0 + s1 == 0) return e;
    const int64_t blocks = std::min<int64_t>((s0 + s1) * 8 * (a.bn / 32), 152 * 8);
    return launch_pdl(k_gated_sum, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, s0, s1);
}

}  // namespace dust
