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
// is six products of planes; what is left out is below 2^-24 of the product.
// The logits take one pair of planes after another, the smallest products
// first; the gradients' products take all planes of a step together, the
// largest product in an accumulator of its own.
//
// Persistent: warp 0 loads (both CTAs), warp 1 issues the MMAs (rank 0 only),
// eight warps drain the accumulators, two per TMEM lane quarter. All waits are
// bounded and record DUST_ERR_TIMEOUT in the device status word.
//
// A step's products take 540 clocks of the tensor pipe, and for long the two
// issuing warps took longer: 560 to load (four boxes of 60 to 145 clocks, the
// flag of a failed wait read every step), 540 to issue. Going through the
// steps as whole warps, with operands in uniform registers, brought the logits
// of 16384 rows, d 512, V 32768 from 366 to 273 us.
//
// Bound by the tensor pipe (94 % busy at d 1024): the logits of 4096 rows, d
// 1024, V 32768 take 139 us, 1980 TFLOP/s; in long runs the power limit
// lowers the clock, and the gradients of 8192 rows (83 % taking part), d 2048,
// V 50257, their logits summed in runs, take 2.33 to 2.66 ms, 1800 to 1580
// TFLOP/s. fp32 (six products counted): the loss of 4096 rows, d 1024, V 32768
// 831 us, 1980 TFLOP/s; gradients 2760, 1790. Below d 384 the epilogue
// binds (2.6e12 exponentials a second, half of what the special-function units
// can do: two warps per scheduler), and fp32 gradients there HBM, by G's three
// planes.
#include <algorithm>
#include <mutex>

#include "f32x2.cuh"
#include "pair_tile.cuh"

namespace dust {

namespace {

enum Mode { kLse, kFactor, kMul };

template <int MODE> constexpr int smem_of() {
    return kStages * kStageBytes + 1024 +
           (MODE == kFactor ? kStoreBytes : kEpiWarps * kTurnBuf);
}
static_assert(smem_of<kFactor>() + 512 <= 227 * 1024 && smem_of<kLse>() + 512 <= 227 * 1024,
              "shared memory per CTA, barriers included");


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
    HeadPicks picks;
    const HeadRow* info;       // kFactor
    int64_t g_cols;
    const int32_t* row_of;     // kMul
    OutRows out0, out1;        // gH, gE
    float *gh_acc, *ge_acc;    // tiles of partial sums, by unit
    int first, last, accumulate;
    int cut0, cut1;            // slices of the summed dimension, gH and gE
    int joint;                 // kMul, fp32, narrow tiles: see launch_head_products
    int stall;
    unsigned int* status;
};

// Where a unit of work lies: which product (0: logits or gH, 1: gE), its
// first row and column, and its steps along the summed dimension (of every
// pair of planes).
struct Tile {
    int job;
    int64_t m0, n0;
    int k0, steps;
    int index;  // its column of tiles (logits), or the unit (kMul)
};

template <int MODE>
struct Plan : Deal {
    int64_t rows;
    int mt, nt;              // tiles of job 0
    int steps0, steps1;      // of a whole tile
    int units0, units1;
    bool one_first;          // kMul: gE's units are the longer ones
    Divider by_nt, by_group, by_gm, by_last;

    __device__ Plan(const TcArgs& a, int c, int n)
        : Deal(c, n), by_nt(1), by_group(1), by_gm(1), by_last(1) {
        rows = a.counts ? a.counts->rows : a.rows;
        nt = divide_up(MODE == kMul ? a.d : a.n, a.bn);
        by_nt = Divider(nt);
        if (MODE != kMul) {
            mt = divide_up(rows, kHeadTile);
            steps0 = divide_up(a.d, 64);
            steps1 = units1 = 0;
            units0 = mt * nt;
            one_first = false;
            total = units0;
            by_group = Divider(a.group * nt);
            by_gm = Divider(a.group);
            by_last = Divider(mt % a.group);
        } else {
            mt = a.out0.base ? divide_up(rows, kHeadTile) : 0;
            steps0 = divide_up(a.n, 64);
            steps1 = divide_up(rows, 64);
            units0 = mt * nt * a.cut0;
            units1 = (a.out1.base ? divide_up(a.n, kHeadTile) : 0) * nt * a.cut1;
            const int cost0 = max(1, divide_up(steps0, a.cut0));
            const int cost1 = max(1, divide_up(steps1, a.cut1));
            one_first = cost1 > cost0;
            deal(one_first ? units1 : units0, one_first ? units0 : units1, max(cost0, cost1),
                 min(cost0, cost1));
        }
    }

    // The i-th unit of this cluster, or -1.
    __device__ int unit(int i) const {
        if (MODE == kMul) return dealt(i);
        const int64_t t = cluster + static_cast<int64_t>(i) * clusters;
        return t < total ? static_cast<int>(t) : -1;
    }

    __device__ Tile at(const TcArgs& a, int t) const {
        Tile w;
        if (MODE != kMul) {
            // Groups of row tiles; inside one, rows fastest: the group's H
            // stays in L2 while E streams by once per group.
            int g, in, c, r;
            by_group(t, g, in);
            if ((g + 1) * a.group <= mt)
                by_gm(in, c, r);
            else
                by_last(in, c, r);
            w.job = 0;
            w.m0 = static_cast<int64_t>(g * a.group + r) * kHeadTile;
            w.n0 = static_cast<int64_t>(c) * a.bn;
            w.k0 = 0;
            w.steps = steps0;
            w.index = c;
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
            int r, c;  // columns fastest: a row block of G is read by neighbours
            by_nt(tile, r, c);
            w.job = job1 ? 1 : 0;
            w.m0 = static_cast<int64_t>(r) * kHeadTile;
            w.n0 = static_cast<int64_t>(c) * a.bn;
            w.index = i;
        }
        return w;
    }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

constexpr float kLog2e = 1.4426950408889634f;

// Adds a block's columns to a row's running sum s of 2^(c v - m). m stays a
// whole number (the largest c v so far, rounded up), so that c v - m is
// rounded once, and the few times it grows s is scaled by a power of two.
template <bool FULL>
__device__ __forceinline__ void softmax_block(const float (&v)[32], int n, float c, float& m,
                                              float& s) {
    // The largest c v, whichever sign c has.
    float top = -INFINITY;
    if (!FULL || c < 0.0f) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) top = fmaxf(top, c < 0.0f ? -v[i] : v[i]);
        if (c < 0.0f) top = -top;
    } else {
        float t[2] = {v[0], v[1]};
#pragma unroll
        for (int i = 2; i < 30; i += 4) {
            t[0] = max3(t[0], v[i], v[i + 1]);
            t[1] = max3(t[1], v[i + 2], v[i + 3]);
        }
        top = max3(fmaxf(t[0], t[1]), v[30], v[31]);
    }
    const float nm = fmaxf(m, ceilf(c * top));
    const float base = nm == -INFINITY ? 0.0f : nm;
    float sum;
    if (FULL) {
        float2 e[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        const float2 cc = {c, c}, bb = {-base, -base};
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float2 t = fma2(cc, make_float2(v[i], v[i + 1]), bb);
            t.x = ex2(t.x);
            t.y = ex2(t.y);
            e[(i >> 1) & 1] = add2(e[(i >> 1) & 1], t);
        }
        const float2 u = add2(e[0], e[1]);
        sum = u.x + u.y;
    } else {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) sum += ex2(fmaf(c, v[i], -base));
    }
    s = fmaf(s, ex2(m - base), sum);
    m = nm;
}

// What a row needs besides the accumulator; loaded a unit ahead.
struct RowOf {
    int64_t row;
    bool live;
    HeadRow info;      // kLse: the target alone
    int64_t out_row;
    int64_t list;      // with a teacher's entries: which list,
    int pick, picks_end;  // the next one here, their end,
    int2 entry, after; // the next one itself and the one after it
};

// Epilogue of one unit for one warp: rows 32 q + lane of this CTA's half,
// columns [h bn / 2, (h + 1) bn / 2).
template <int MODE, int PLANES, bool RUNS>
struct Epilogue {
    const TcArgs& a;
    const CUtensorMap* tmG;
    unsigned char* bufs;  // this warp's: kFactor's store buffers, the others' 32 x 32 values
    uint32_t rank;
    int q, h, lane;
    uint32_t used = 0;
    // A unit's sums over its runs of steps but the last (narrow tiles), and
    // whether there are such.
    static constexpr int kSums = RUNS ? 128 / kShare : 1;
    float sum[kSums] = {};
    bool summed = false;

    __device__ RowOf begin(const Tile& w, const Plan<MODE>& plan) const {
        RowOf o;
        o.row = w.m0 + rank * kHalf + 32 * q + lane;
        o.info.target = -1;
        o.out_row = o.row;
        o.pick = o.picks_end = 0;
        if (MODE == kLse) {
            o.live = o.row < plan.rows;
            if (o.live) {
                o.list = static_cast<uint32_t>(o.row) % static_cast<uint32_t>(a.T);
                if (a.targets) o.info.target = a.targets[o.list];
                if (a.picks.entries) find_picks(w, o);
            }
        } else if (MODE == kFactor) {
            o.live = o.row < plan.rows;
            if (o.live) o.info = a.info[o.row];
        } else if (w.job == 0) {
            o.live = o.row < plan.rows;
            if (o.live && a.row_of) o.out_row = a.row_of[o.row];
        } else {
            o.live = o.row < a.n;
        }
        return o;
    }

    // Where the row's entries among its columns start and end.
    __device__ void find_picks(const Tile& w, RowOf& o) const {
        const int bin = static_cast<int>((a.v0 + w.n0) / (a.bn / kShare)) + h;
        const uint16_t* at = a.picks.starts + o.list * (a.picks.bins + 1) + bin;
        o.pick = at[0];
        o.picks_end = at[1];
    }
    __device__ void first_picks(RowOf& o) const {
        const int2* at = a.picks.entries + o.list * a.picks.K + o.pick;
        if (o.pick < o.picks_end) o.entry = at[0];
        if (o.pick + 1 < o.picks_end) o.after = at[1];
    }
    // On to the next entry; the one after it is on its way meanwhile.
    __device__ void next_pick(RowOf& o) const {
        ++o.pick;
        o.entry = o.after;
        if (o.pick + 1 < o.picks_end) o.after = a.picks.entries[o.list * a.picks.K + o.pick + 1];
    }
    // The further steps of the loads ahead, each after what it needs has come:
    // an entry its place, and kFactor's places the row's number.
    __device__ void second(const Tile& w, RowOf& o) const {
        if (MODE == kLse) first_picks(o);
        if (MODE == kFactor && a.picks.entries && o.live) {
            o.list = o.info.target;
            find_picks(w, o);
        }
    }
    __device__ void third(RowOf& o) const {
        if (MODE == kFactor) first_picks(o);
    }

    // Whether any of this warp's 32 rows is wanted: kLse and kMul want those
    // that exist; of G, kMul sums over rows up to the next multiple of 64.
    __device__ bool wanted(const Tile& w, const Plan<MODE>& plan) const {
        const int64_t row = w.m0 + rank * kHalf + 32 * q;
        if (MODE == kMul) return row < (w.job == 1 ? a.n : plan.rows);
        return row < (MODE == kFactor ? (plan.rows + 63) / 64 * 64 : plan.rows);
    }

    __device__ void lse(const Tile& w, RowOf o, uint32_t taddr) {
        const int cols = a.bn / kShare;
        const float c = a.scale * kLog2e;
        const int32_t first = static_cast<int32_t>(w.n0) + h * cols;
        float m = -INFINITY, s = 0.0f;
        // Target relative to the warp's first column, if it has one there.
        const int32_t tv = o.info.target - static_cast<int32_t>(a.v0) - first;
        for (int b = 0; b < cols / 32; ++b) {
            float v[32];
            whole_sum(taddr, h * cols + 32 * b, v);
            const int left = static_cast<int>(a.n) - (first + 32 * b);  // columns that exist
            if (left <= 0) break;
            // Logits that are wanted by themselves, the target's and the
            // teacher's entries': the row's 32 through shared memory, where a
            // thread can choose among its own.
            const int at = tv - 32 * b;
            const int32_t past = first + 32 * b + 32;
            const bool pick = o.pick < o.picks_end && o.entry.x < past;
            if (pick || (o.live && at >= 0 && at < 32 && at < left)) {
                const uint32_t buf = tc::smem_u32(bufs) + lane * 128;
                const uint32_t swz = lane & 7;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    st_shared_16(buf + ((u ^ swz) << 4), reinterpret_cast<const uint32_t*>(v) + 4 * u);
                const auto logit = [&](int c) {
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(x)
                                 : "r"(buf + (((c >> 2) ^ swz) << 4) + (c & 3) * 4)
                                 : "memory");
                    return a.scale * x;
                };
                if (!pick) a.picked[o.row] = logit(at);
                while (o.pick < o.picks_end && o.entry.x < past) {
                    a.picks.student[o.row * a.picks.K + o.entry.y] = logit(o.entry.x - (past - 32));
                    next_pick(o);
                }
            }
            if (left >= 32)
                softmax_block<true>(v, 32, c, m, s);
            else
                softmax_block<false>(v, left, c, m, s);
        }
        if (o.live)
            a.part[(static_cast<int64_t>(w.index) * kShare + h) * a.ld_part + o.row] = {m, s};
    }

    __device__ void factor(const Tile& w, RowOf o, uint32_t taddr) {
        const int cols = a.bn / kShare;
        const float c = a.scale * kLog2e;
        const uint32_t swz = (lane >> 1) & 3;
        for (int b = 0; b < cols / 32; ++b) {
            float v[32];
            const int64_t col = w.n0 + h * cols + 32 * b;
            whole_sum(taddr, h * cols + 32 * b, v);
            const int left = static_cast<int>(a.n - col);
            const float2 cc = {c, c}, hi = {-o.info.lse_hi, -o.info.lse_hi};
            const float2 ww = {o.info.weight, o.info.weight};
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float2 t = fma2(cc, make_float2(v[i], v[i + 1]), hi);
                if (PLANES == 3) {
                    // The logarithm in two parts: its rounding would be the
                    // same for the whole row.
                    t.x -= o.info.lse_lo;
                    t.y -= o.info.lse_lo;
                }
                t.x = ex2(t.x);
                t.y = ex2(t.y);
                t = mul2(ww, t);
                v[i] = t.x;
                v[i + 1] = t.y;
            }
            if (!o.live || left < 32) {  // G is zero where there is no row or column
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = o.live && i < left ? v[i] : 0.0f;
            }
            const int64_t tv = a.picks.entries ? -1 : o.info.target - a.v0 - col;
            if (tv >= 0 && tv < 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (i == tv) v[i] -= o.info.weight;
            }
            const int32_t past = static_cast<int32_t>(a.v0 + col) + 32;
            const RowOf here = o;  // the block's entries, once more for every plane
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
                // The teacher's entries replace what the softmax gave.
                if (p > 0) o = here;
                while (o.pick < o.picks_end && o.entry.x < past) {
                    float g = o.info.weight * __int_as_float(o.entry.y);
#pragma unroll
                    for (int k = 0; k < p; ++k) g -= __bfloat162float(__float2bfloat16_rn(g));
                    const uint32_t c = static_cast<uint32_t>(o.entry.x - (past - 32));
                    const __nv_bfloat16 e = __float2bfloat16_rn(g);
                    asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + (((c >> 3) ^ swz) << 4) +
                                                                 (c & 7) * 2),
                                 "h"(*reinterpret_cast<const uint16_t*>(&e))
                                 : "memory");
                    next_pick(o);
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
    }

    // Columns [at, at + 32) of the accumulators of a run of steps: both of them
    // for fp32 products. TMEM is read by whole warps at once, and lanes come
    // here from places where they part (a row's own entries, a lane that
    // stores): they meet first.
    __device__ void accumulators(uint32_t taddr, int at, float (&v)[32]) const {
        __syncwarp();
        tc::tmem_ld_32x32(taddr + at, v);
        if (MODE == kMul && PLANES == 3) {
            float big[32];
            tc::tmem_ld_32x32(taddr + 128 + at, big);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += big[i];
        }
    }

    // Columns [at, at + 32) of the unit's whole sum, after its last run.
    __device__ void whole_sum(uint32_t taddr, int at, float (&v)[32]) const {
        accumulators(taddr, at, v);
        if (RUNS && summed) {
            const bool second = (at & 32) != 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += second ? sum[(32 + i) % kSums] : sum[i % kSums];
        }
    }

    // Adds a run that is not the last to the unit's sums.
    __device__ void collect(uint32_t taddr, bool first) {
        const int cols = a.bn / kShare;
#pragma unroll
        for (int b = 0; b < kSums / 32; ++b) {
            float v[32];
            accumulators(taddr, h * cols + 32 * b, v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                sum[(32 * b + i) % kSums] = first ? v[i] : sum[(32 * b + i) % kSums] + v[i];
        }
    }

    __device__ void product(const Tile& w, const RowOf& o, uint32_t taddr, float alpha) {
        const int cols = a.bn / kShare;
        const bool job1 = w.job == 1, zero = w.steps == 0;
        float* acc = job1 ? a.ge_acc : a.gh_acc;
        const bool add = !job1 && !a.first;
        // The result is whole here unless other slices or pieces add to it.
        const bool whole = job1 ? a.cut1 == 1 : a.cut0 == 1 && a.last;
        const OutRows& out = job1 ? a.out1 : a.out0;
        const int32_t to = o.live ? static_cast<int32_t>(o.out_row) : -1;
        const uint32_t buf = tc::smem_u32(bufs);
        // (Not unrolled: tiles of few rows' gradients spend their time here, and
        // four copies of it do not fit the instruction cache.)
#pragma unroll 1
        for (int at = h * cols; at < (h + 1) * cols; at += 32) {
            const int64_t col = w.n0 + at;
            if (col >= a.d) break;
            float v[32];
            whole_sum(taddr, at, v);
            const int n = a.d - col < 32 ? static_cast<int>(a.d - col) : 32;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = zero ? 0.0f : alpha * v[i];
            if (acc && (add || !whole)) {
                // Partial sums lie as the accumulator has them: four columns
                // of all rows together.
                float4* p = reinterpret_cast<float4*>(acc + static_cast<int64_t>(w.index) * kSlotFloats) +
                            at / 4 * kHeadTile + static_cast<int>(rank) * kHalf + 32 * q + lane;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (add) {
                        const float4 u = p[i * kHeadTile];
                        v[4 * i] += u.x;
                        v[4 * i + 1] += u.y;
                        v[4 * i + 2] += u.z;
                        v[4 * i + 3] += u.w;
                    }
                    if (!whole)
                        p[i * kHeadTile] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            if (whole)
                store_block(buf, v, lane, to, out, col, n, job1 && a.accumulate);
        }
    }
};

__device__ __forceinline__ Tile uniform(const Tile& t) {
    Tile w;
    w.job = uniform(t.job);
    w.m0 = uniform(static_cast<int>(t.m0));
    w.n0 = uniform(static_cast<int>(t.n0));
    w.k0 = uniform(t.k0);
    w.steps = uniform(t.steps);
    w.index = t.index;
    return w;
}

// Maps: kLse H, -, E, -; kFactor H, Hc, E, G; kMul G, E, H, Hc.
template <int MODE, int PLANES, bool RUNS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_head_tc(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
              const __grid_constant__ CUtensorMap tm2, const __grid_constant__ CUtensorMap tm3,
              const __grid_constant__ TcArgs a) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* store_bufs = smem + kStages * kStageBytes;
    __shared__ Ctl ctl_s;
    Ctl* ctl = &ctl_s;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = uniform(tc::cluster_rank_of_cta());
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

    const Plan<MODE> plan(a, cluster, n_clusters);
    const int pairs = a.planes == 1 ? 1 : 6;
    const int b_boxes = a.bn / 128;  // per CTA
    const int run = RUNS ? kRun : 1 << 30;
    // A tile's products take about 0.3 us per step: the waits for a whole
    // tile are given 2 us per step on top of the usual limit.
    const uint64_t tile_ns =
        tc::kWaitNs + 2000ull * static_cast<uint64_t>(pairs) * max(plan.steps0, plan.steps1);

    // The loads and the products are issued by one lane each, but the whole
    // warp goes through the steps with them: places, addresses and descriptors
    // are then the same in all lanes for the compiler too, which keeps them in
    // uniform registers. (In a branch of one lane, every operand of every
    // instruction was moved there first: 145 cycles a load, 57 a product.)
    if (warp == 0) {
        const bool one = elect_one();
        // The rows that take part are read where they lie unless some were left out.
        const bool compact = uniform(a.counts && a.rows != plan.rows) != 0;
        const uint32_t full = tc::at_rank(&ctl->full[0], 0);
        const uint32_t bytes = 2 * (2 + b_boxes) * kBoxBytes;  // of a step, both CTAs
        const CUtensorMap *A0, *B0, *A1 = nullptr, *B1 = nullptr;
        if (MODE == kMul) {
            A0 = &tm0; B0 = &tm1;                      // gH = G E
            A1 = &tm0; B1 = compact ? &tm3 : &tm2;     // gE = G^T H
        } else {
            A0 = compact ? &tm1 : &tm0;
            B0 = &tm2;
        }
        int it = 0, st = 0;
        uint32_t parity = 1;
        bool stop = false;
        for (int j = 0, t; !stop && (t = uniform(plan.unit(j))) >= 0; ++j) {
            const Tile w = uniform(plan.at(a, t));
            const CUtensorMap* ma = w.job ? A1 : A0;
            const CUtensorMap* mb = w.job ? B1 : B0;
            // Which operand has the summed dimension in rows.
            const bool a_mn = MODE == kMul && w.job == 1, b_mn = MODE == kMul;
            const int32_t am = static_cast<int32_t>(w.m0) + static_cast<int32_t>(rank) * kHalf;
            // E is whole: its rows of the piece start at v0.
            const int32_t v0 = static_cast<int32_t>(a.v0);
            const int32_t bn0 = static_cast<int32_t>(w.n0) +
                                static_cast<int32_t>(rank) * (a.bn / 2) + (MODE == kMul ? 0 : v0);
            const int32_t b_k0 = MODE == kMul && w.job == 0 ? v0 : 0;
            // Steps of one pair of planes after another, or the planes of
            // one step after another, the smallest first.
            for (int c = 0; c < w.steps && !stop; c += run) {
                for (int p = 0, n = min(run, w.steps - c); p < (a.joint ? n : pairs) && !stop; ++p) {
                    const int pa0 = pairs == 1 ? 0 : plane_a(p), pb0 = pairs == 1 ? 0 : plane_b(p);
                    for (int i = 0; i < (a.joint ? 3 : n); ++i, ++it) {
                        const int32_t kk = (w.k0 + c + (a.joint ? p : i)) * 64;
                        const int pa = a.joint ? 2 - i : pa0, pb = a.joint ? 2 - i : pb0;
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
                                tc::tma_load_3d_pair(base + u * kBoxBytes, ma, a_mn ? am + 64 * u : kk,
                                                     a_mn ? kk : am + 64 * u, pa, bar);
                            tc::tma_load_3d_pair(base + 2 * kBoxBytes, mb, b_mn ? bn0 : kk,
                                                 b_mn ? b_k0 + kk : bn0, pb, bar);
                            if (b_boxes == 2)
                                tc::tma_load_3d_pair(base + 3 * kBoxBytes, mb, b_mn ? bn0 + 64 : kk,
                                                     b_mn ? b_k0 + kk : bn0 + 64, pb, bar);
                        }
                        __syncwarp();
                        if (++st == kStages) {
                            st = 0;
                            parity ^= 1;
                        }
                    }
                }
            }
        }
        if (lane == 0) ctl->issued = it;
        // The last stages' releases land here, too, before the CTA may leave: they
        // come from the pair's first CTA, whenever their products are done.
        for (int i = 0; i < kStages && !stop; ++i) {
            if (!warp_wait(&ctl->empty[st], parity, tile_ns, abort_flag)) {
                *abort_flag = 1;
                stop = true;
            }
            if (++st == kStages) {
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
                if (++st == kStages) {
                    st = 0;
                    parity ^= 1;
                }
            };
            const auto loaded = [&] {
                return warp_wait(&ctl->full[st], parity, tc::kWaitNs, abort_flag);
            };
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
                const int n = a.joint ? steps : pairs * steps;
                for (int k = 0; k < n; ++k) {
                    const int s2 = st;
                    stop = !loaded();
                    if (stop) break;
                    advance();
                    if (!a.joint) {
                        tc::tc_fence_after();
                        if (one) {
                            issue_step(dst, A, s2, B, s2, idesc, k != 0);
                            tc::mma_commit_pair(&ctl->empty[s2]);
                        }
                        __syncwarp();
                        continue;
                    }
                    const int s1 = st;
                    stop = !loaded();
                    if (stop) break;
                    advance();
                    const int s0 = st;
                    stop = !loaded();
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
        constexpr int kOwn = MODE == kFactor ? kStoreBufs * kStageBuf : kTurnBuf;
        Epilogue<MODE, PLANES, RUNS> epi{a, &tm3, store_bufs + ew * kOwn, rank, q, h, lane};
        const float alpha = MODE == kMul ? a.scale * a.counts->gmax : 0.0f;
        int t = plan.unit(0);
        Tile w = t >= 0 ? plan.at(a, t) : Tile{};
        RowOf o = {};
        if (t >= 0) o = epi.begin(w, plan);
        epi.second(w, o);
        bool ok = true;
        for (int i = 1, j = 0; t >= 0 && ok; ++i) {
            epi.third(o);
            Tile next = w;
            RowOf next_o = {};
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
                if (last) {
                    // The next unit's rows are loaded beside this one's arithmetic.
                    t = plan.unit(i);
                    if (t >= 0) {
                        next = plan.at(a, t);
                        next_o = epi.begin(next, plan);
                    }
                }
                const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * 256;
                if (epi.wanted(w, plan)) {
                    if (RUNS && !last) {
                        epi.collect(taddr, c == 0);
                    } else {
                        epi.summed = c > 0;
                        if constexpr (MODE == kLse)
                            epi.lse(w, o, taddr);
                        else if constexpr (MODE == kFactor)
                            epi.factor(w, o, taddr);
                        else
                            epi.product(w, o, taddr, alpha);
                    }
                }
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive_at(tc::at_rank(&ctl->tempty[acc], 0));
                c = last ? -1 : c + run;
            }
            if (ok && t >= 0) epi.second(next, next_o);
            w = next;
            o = next_o;
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

// The slices' partial sums of the products added in order, into gH (t0 tiles)
// and gE (t1 tiles): a CTA takes 32 rows and 32 columns of a tile at a time.
__global__ void __launch_bounds__(256)
    k_head_sum(const __grid_constant__ TcArgs a, int64_t t0, int64_t t1) {
    pdl_wait();
    pdl_trigger();
    const int nt = static_cast<int>((a.d + a.bn - 1) / a.bn);
    const int per = 8 * (a.bn / 32);
    const int lane = threadIdx.x & 31, c4 = threadIdx.x >> 5;
    for (int64_t b = blockIdx.x; b < (t0 + t1) * per; b += gridDim.x) {
        const bool job = b >= t0 * per;
        const int64_t tile = b / per - (job ? t0 : 0);
        const int in = static_cast<int>(b % per);
        const int r = (in & 7) * 32 + lane, c = (in >> 3) * 32 + c4 * 4;
        const int64_t row = tile / nt * kHeadTile + r, col = tile % nt * a.bn + c;
        if (row >= (job ? a.n : a.counts->rows) || col >= a.d) continue;
        const int cut = job ? a.cut1 : a.cut0;
        const float4* p = reinterpret_cast<const float4*>((job ? a.ge_acc : a.gh_acc) +
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
        const OutRows& out = job ? a.out1 : a.out0;
        const int64_t to = !job && a.row_of ? a.row_of[row] : row;
        unsigned char* at = out.base + to * out.pitch;
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

cudaError_t launch_sum(const TcArgs& a, int64_t t0, int64_t t1, cudaStream_t s) {
    const int64_t blocks = std::min<int64_t>((t0 + t1) * 8 * (a.bn / 32), 152 * 8);
    return launch_pdl(k_head_sum, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a, t0, t1);
}

// CTA pairs that can be resident at once, for the kernel of a mode.
template <int MODE, int PLANES, bool RUNS>
int max_clusters() {
    constexpr int kMaxDev = 64;
    static int cache[kMaxDev] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return 0;
    std::lock_guard<std::mutex> lk(mu);
    if (cache[dev] == 0) {
        const void* k = reinterpret_cast<const void*>(k_head_tc<MODE, PLANES, RUNS>);
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

template <int MODE, int PLANES, bool RUNS>
cudaError_t launch_tc(const CUtensorMap (&m)[4], TcArgs a, int64_t tiles, cudaStream_t s) {
    const int fit = max_clusters<MODE, PLANES, RUNS>();
    if (fit <= 0) return cudaErrorUnknown;
    if (tiles <= 0) return cudaSuccess;
    if (tiles > (int64_t(1) << 30)) return cudaErrorInvalidValue;
    a.status = status_word();
    if (!a.status) return cudaErrorUnknown;
    a.stall = take_stall_injection() ? 1 : 0;
    const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, fit));
    return launch_pdl(k_head_tc<MODE, PLANES, RUNS>, dim3(2 * clusters), dim3(kThreads), smem_of<MODE>(), s,
                      m[0], m[1], m[2], m[3], a);
}

// Whether logits over d columns are summed in runs (kRun), in narrow tiles:
// about a sixth slower. (Normwise error of single logits, in one run and in
// runs of 8 steps: d 1024 1.0e-6 and 4.7e-7, d 2048 2.1e-6 and 4.8e-7, d 8192
// 9.1e-6 and 4.8e-7.) The loss and the gradient sum them alike, so that what is
// cut off is the same in lse and in x and cancels in exp(x - lse): of a token
// that the model is sure of, the target's entry of G is the small difference
// p - 1, and an error of x that lse does not share is an error of it in full
// (loss 1e-4, target's logit 30: gH was 0.8 to 1.4 off, by row, at d 2048, and
// 10 at d 8192, when the bf16 gradient alone summed in one run).
bool in_runs(int64_t d) { return d > 1024; }

}  // namespace

int head_columns(int64_t rows, int64_t n, int64_t d) {
    return in_runs(d) ? 128 : logit_columns(rows, n);
}

HeadCuts head_cuts(int64_t rows, int64_t n, int64_t d, int planes) {
    const int64_t nt = tiles_of(d, product_columns(d, planes));
    const Cuts c = cuts_of(tiles_of(rows, kHeadTile) * nt, tiles_of(n, 64), tiles_of(n, kHeadTile) * nt,
                           tiles_of(rows, 64), planes);
    return {c.a, c.b};
}

// The whole vocabulary if its G has at most 2^28 values over the planes (512
// MB), else pieces of whole tiles of that or less (four tiles at least): of
// the sizes down to half of it the one whose tiles leave the pairs idle
// least, by the steps of all pieces' rounds (16384 rows, d 512, V 32768:
// pieces of 8192 took 1282 us, of 16384 1208).
int64_t head_piece(int64_t rows, int64_t V, int64_t d, int planes) {
    constexpr int64_t kMost = int64_t(1) << 28, kLaunches = 50;  // two launches, in steps
    const int64_t mt = tiles_of(rows, kHeadTile), whole = tiles_of(V, kHeadTile);
    const int64_t cap = std::max<int64_t>(kMost / (mt * kHeadTile * planes) / kHeadTile, 4);
    if (whole <= cap) return whole * kHeadTile;
    const int64_t pairs = planes == 1 ? 1 : 6, nt = tiles_of(d, product_columns(d, planes));
    const int64_t logits = tiles_of(d, 64) * pairs + 3, c1 = tiles_of(rows, 64) * pairs + 4;
    const auto cost = [&](int64_t n) {  // of a piece of n tiles
        const int64_t c0 = n * (kHeadTile / 64) * pairs + 4, t0 = mt * nt, t1 = n * nt;
        // A quarter of a step per tile of gH: its running sums, read and written.
        return tiles_of(mt * n, kPairs) * logits + kLaunches + t0 / 4 +
               (c1 > c0 ? makespan(t1, c1, t0, c0) : makespan(t0, c0, t1, c1));
    };
    int64_t best = cap, least = -1;
    const int64_t by = std::max<int64_t>(1, cap / 64);
    for (int64_t n = cap; n >= (cap + 1) / 2; n -= by) {
        const int64_t full = whole / n, rest = whole % n;
        const int64_t c = full * cost(n) + (rest ? cost(rest) : 0);
        if (least < 0 || c < least) {
            least = c;
            best = n;
        }
    }
    return best * kHeadTile;
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
    a.bn = h.bn;
    a.group = kGroup;
    a.scale = h.scale;
    a.targets = h.targets;
    a.T = h.T;
    a.part = h.part;
    a.ld_part = h.ld_part;
    a.picked = h.picked;
    a.picks = h.picks;
    const int64_t tiles = tiles_of(a.rows, kHeadTile) * tiles_of(a.n, a.bn);
    return in_runs(a.d) ? launch_tc<kLse, 1, true>(m, a, tiles, s)
                        : launch_tc<kLse, 1, false>(m, a, tiles, s);
}

bool make_head_maps(HeadMaps* m, const Planes& H, const Planes& Hc, const Planes& E,
                    const Planes& G) {
    if (!operand_map(&m->H, H) || !operand_map(&m->E, E) || !operand_map(&m->G, G) ||
        !make_map(&m->G_store, G, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return false;
    m->Hc = m->H;
    return !Hc.base || operand_map(&m->Hc, Hc);
}

cudaError_t launch_head_factor(const HeadLogits& h, const HeadMaps& maps, cudaStream_t s) {
    const CUtensorMap m[4] = {maps.H, maps.Hc, maps.E, maps.G_store};
    TcArgs a = {};
    a.rows = h.H.rows;
    a.d = h.H.cols;
    a.n = h.n;
    a.v0 = h.v0;
    a.counts = h.counts;
    a.planes = h.H.planes;
    a.bn = h.bn;
    a.group = kGroup;
    a.scale = h.scale;
    a.picks = h.picks;
    a.info = h.rows;
    const int64_t tiles = tiles_of(a.rows, kHeadTile) * tiles_of(a.n, a.bn);
    if (a.planes == 1)
        return in_runs(a.d) ? launch_tc<kFactor, 1, true>(m, a, tiles, s)
                            : launch_tc<kFactor, 1, false>(m, a, tiles, s);
    return in_runs(a.d) ? launch_tc<kFactor, 3, true>(m, a, tiles, s)
                        : launch_tc<kFactor, 3, false>(m, a, tiles, s);
}

int64_t head_acc_floats(int64_t m, int64_t d, int planes, int cut) {
    return tiles_of(m, kHeadTile) * tiles_of(d, product_columns(d, planes)) * cut * kSlotFloats;
}

cudaError_t launch_head_products(const HeadProducts& h, const HeadMaps& maps, cudaStream_t s) {
    const CUtensorMap m[4] = {maps.G, maps.E, maps.H, maps.Hc};
    TcArgs a = {};
    a.rows = h.rows;
    a.d = h.d;
    a.n = h.n;
    a.v0 = h.v0;
    a.counts = h.counts;
    a.planes = h.planes;
    a.bn = product_columns(h.d, a.planes);
    // All planes of a step together: three loads of A and B serve its six
    // products, and G is read once from HBM instead of once per product (16384
    // rows, V 32768: d 64 2798 -> 2000 us, 1400 of them G's bytes; d 512, where
    // wide tiles did without, 6280 -> 5920). The smallest products are no longer
    // summed first; so the largest has an accumulator of its own, beside which
    // the others' rounding does not show. There is room for two of 128 columns.
    a.joint = a.planes == 3;
    a.scale = h.scale;
    a.row_of = h.row_of;
    a.gh_acc = h.gh_acc;
    a.ge_acc = h.ge_acc;
    a.cut0 = h.cuts.gh;
    a.cut1 = h.cuts.ge;
    const auto out = [&](void* p, int64_t ld, bool bf16) {
        // The rows' length too: what follows it is not written.
        const int size = bf16 ? 2 : 4;
        const uintptr_t at = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * size) |
                             static_cast<uintptr_t>(h.d * size);
        int align = 16;
        while (align > size && at % align != 0) align /= 2;
        return OutRows{static_cast<unsigned char*>(p), ld * size, bf16, align};
    };
    a.out0 = out(h.gH, h.ld_gh, h.gh_bf16);
    a.out1 = out(h.gE, h.d, h.ge_bf16);
    a.first = h.first;
    a.last = h.last;
    a.accumulate = h.accumulate;
    const int64_t nt = tiles_of(a.d, a.bn);
    const int64_t t0 = h.gH ? tiles_of(a.rows, kHeadTile) * nt : 0;
    const int64_t t1 = h.gE ? tiles_of(a.n, kHeadTile) * nt : 0;
    const int64_t units = t0 * a.cut0 + t1 * a.cut1;
    cudaError_t e = a.planes == 1 ? launch_tc<kMul, 1, false>(m, a, units, s)
                                  : launch_tc<kMul, 3, true>(m, a, units, s);
    const int64_t s0 = a.cut0 > 1 && h.last ? t0 : 0, s1 = a.cut1 > 1 ? t1 : 0;
    if (e == cudaSuccess && s0 + s1 > 0) e = launch_sum(a, s0, s1, s);
    return e;
}

}  // namespace dust
