// What the kernels that work on 256-row tiles by CTA pairs share (k_head_tc.cu,
// k_gated_tc.cu): stages of TMA boxes in shared memory, products of bf16
// operands or of three bf16 planes (fp32), waits that end, stores of tiles to
// rows of any alignment, and how units of work are dealt to the pairs.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "head.cuh"
#include "tc_common.cuh"

namespace dust {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

namespace {  // each kernel's translation unit has its own

inline int64_t tiles_of(int64_t n, int64_t by) { return (n + by - 1) / by; }

constexpr int kHalf = 128;                        // rows of A per CTA
constexpr int kBoxBytes = kHeadBox * kHeadBox * 2;
constexpr int kStageBytes = 4 * kBoxBytes;        // two boxes of A, two of B
constexpr int kEpiWarps = 8;
constexpr int kShare = kEpiWarps / 4;             // warps that share a TMEM lane quarter
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStageBuf = 32 * 32 * 2;            // 32 rows x 32 columns of bf16, to be stored by TMA
constexpr int kStoreBufs = 2;
constexpr int kStoreBytes = kEpiWarps * kStoreBufs * kStageBuf;
constexpr int kTurnBuf = 32 * 32 * 4;             // 32 rows x 32 columns of fp32
constexpr int kSlotFloats = kHeadTile * kHeadTile;  // a tile of partial sums
constexpr uint32_t kTmemCols = 512;               // two accumulators of 256 columns
constexpr int kStages = 6;                        // steps in flight

// Steps that fp32 products add up in TMEM at a time. The tensor cores cut a
// sum's last bits off instead of rounding them, so its error grows with the
// number of additions, not with its root; runs are joined in registers, rounded
// (4096 rows, d 512, V 16384, normwise error of gH: 1.9e-5 without runs, 1.3e-6
// with 16 steps, 6.8e-7 with 8, 4.1e-7 with 4, which takes 5 % longer where
// sums are short).
constexpr int kRun = 8;

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

// An output of the products: rows `pitch` bytes apart, whose starts and ends
// lie on multiples of `align` bytes (16 at most).
struct OutRows {
    unsigned char* base;
    int64_t pitch;
    int bf16, align;
};

// Planes of A and B of the p-th product, the smallest products first: (2, 0),
// (0, 2), (1, 1), (1, 0), (0, 1), (0, 0). In registers: a table in memory
// would be read per step.
__device__ __forceinline__ int plane_a(int p) { return 0x001102 >> (4 * p) & 15; }
__device__ __forceinline__ int plane_b(int p) { return 0x010120 >> (4 * p) & 15; }

// Division by a number that stays the same: a product and a correction (a
// division proper takes some forty instructions, and a tile's place takes
// several; with one step of products per tile that bound the kernel).
struct Divider {
    uint32_t d, inverse;
    __device__ explicit Divider(int n) : d(static_cast<uint32_t>(max(n, 1))) {
        inverse = d == 1 ? 0xffffffffu : static_cast<uint32_t>((1ull << 32) / d);
    }
    // a < 2^31: the product is 0 to 2 short of the quotient.
    __device__ __forceinline__ void operator()(int a, int& q, int& r) const {
        uint32_t u = __umulhi(static_cast<uint32_t>(a), inverse);
        uint32_t left = static_cast<uint32_t>(a) - u * d;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (left >= d) {
                left -= d;
                ++u;
            }
        q = static_cast<int>(u);
        r = static_cast<int>(left);
    }
};

__device__ __forceinline__ int divide_up(int64_t v, int by) {
    return static_cast<int>(static_cast<uint32_t>(v + by - 1) / static_cast<uint32_t>(by));
}

// Units of work of two lengths, dealt to the clusters: long units round robin,
// then the short ones to whoever is done first: the clusters from `high` on
// have one long unit less, and take `rounds` short ones each while the others
// finish; from there on everyone in turn. The units are numbered long ones
// first.
struct Deal {
    int cluster, clusters;
    int total = 0, longs = 0, mine = 0, high = 0, rounds = 0;

    __device__ Deal(int c, int n) : cluster(c), clusters(n) {}

    __device__ void deal(int n_long, int n_short, int c_long, int c_short) {
        total = n_long + n_short;
        longs = n_long;
        high = longs % clusters;
        mine = longs / clusters + (cluster < high ? 1 : 0);
        rounds = high == 0 ? 0 : divide_up(c_long, c_short);
    }

    // The i-th unit of this cluster, or -1.
    __device__ int dealt(int i) const {
        if (i < mine) return cluster + i * clusters;
        i -= mine;
        int64_t t;
        const int low = clusters - high;
        if (cluster >= high && i < rounds) {
            t = static_cast<int64_t>(i) * low + cluster - high;
        } else {
            if (cluster >= high) i -= rounds;
            t = static_cast<int64_t>(rounds) * low + static_cast<int64_t>(i) * clusters + cluster;
        }
        return t < total - longs ? longs + static_cast<int>(t) : -1;
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

__device__ __forceinline__ float4 ld_shared_4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Writes 32 columns from `col` of which `n` lie inside the output: a lane has
// a row's values v, and row `to` is its place (-1: none). They are turned
// around in shared memory (4 KB at buf, 16-byte pieces permuted by row), so
// that neighbouring lanes write neighbouring columns. With a row per lane,
// each store touched 32 lines: the gradients of 3 rows, d 898, V 16557, bf16,
// took 283 us then and 86 so (both on these tiles).
__device__ __forceinline__ void store_block(uint32_t buf, const float (&v)[32], int lane, int32_t to,
                                            const OutRows& out, int64_t col, int n, bool add) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u[4] = {__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                               __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
        st_shared_16(buf + lane * 128 + ((i ^ (lane & 7)) << 4), u);
    }
    __syncwarp();
    unsigned char* first = out.base + col * (out.bf16 ? 2 : 4);
    const auto at_row = [&](int r) -> unsigned char* {
        const int32_t at = __shfl_sync(0xffffffffu, to, r);
        return at < 0 ? nullptr : first + at * out.pitch;
    };
    // Everything that a few stores need is read before the first of them.
    if (out.align == 16 && !out.bf16) {
        const int c = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            float4* p[4];
            float4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 4 * (i + k) + (lane >> 3);
                p[k] = reinterpret_cast<float4*>(at_row(r));
                x[k] = ld_shared_4(buf + r * 128 + ((c ^ (r & 7)) << 4));
                if (4 * c >= n) p[k] = nullptr;
                if (add && p[k]) {
                    const float4 o = p[k][c];
                    x[k] = make_float4(o.x + x[k].x, o.y + x[k].y, o.z + x[k].z, o.w + x[k].w);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (p[k]) p[k][c] = x[k];
        }
    } else if (out.align == 16) {
        const int c = lane & 3;
        uint4* p[4];
        uint4 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = 8 * k + (lane >> 2);
            p[k] = reinterpret_cast<uint4*>(at_row(r));
            const float4 y = ld_shared_4(buf + r * 128 + (((2 * c) ^ (r & 7)) << 4));
            const float4 z = ld_shared_4(buf + r * 128 + (((2 * c + 1) ^ (r & 7)) << 4));
            x[k] = make_uint4(pack2(y.x, y.y), pack2(y.z, y.w), pack2(z.x, z.y), pack2(z.z, z.w));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (p[k] && 8 * c < n) p[k][c] = x[k];
    } else if (out.bf16 && out.align >= 4) {
        const int c = lane & 15;  // rows of an even number of values
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
            uint32_t* p[8];
            uint32_t x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = 2 * (i + k) + (lane >> 4);
                p[k] = reinterpret_cast<uint32_t*>(at_row(r));
                float lo, hi;
                asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                             : "=f"(lo), "=f"(hi)
                             : "r"(buf + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8)
                             : "memory");
                x[k] = pack2(lo, hi);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (p[k] && 2 * c < n) p[k][c] = x[k];
        }
    } else if (const int32_t row0 = __shfl_sync(0xffffffffu, to, 0);
               __all_sync(0xffffffffu, to < 0 || to == row0 + lane)) {
        // Neighbouring rows: the first `live` of them exist. No shuffles, one
        // running address (65 rows, d 129, V 1003, fp32: 44.8 -> 38.4 us).
        const int live = __popc(__ballot_sync(0xffffffffu, to >= 0));
        uint32_t at[8];  // by row mod 8
#pragma unroll
        for (int k = 0; k < 8; ++k) at[k] = buf + (((lane >> 2) ^ k) << 4) + (lane & 3) * 4;
        unsigned char* p = first + row0 * out.pitch + lane * (out.bf16 ? 2 : 4);
        const int rows = lane < n ? live : 0;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x[k]) : "r"(at[k] + (i + k) * 128) : "memory");
            if (add) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (i + k < rows) x[k] = *reinterpret_cast<const float*>(p + k * out.pitch) + x[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (i + k >= rows) continue;
                if (out.bf16) *reinterpret_cast<__nv_bfloat16*>(p + k * out.pitch) = __float2bfloat16_rn(x[k]);
                else *reinterpret_cast<float*>(p + k * out.pitch) = x[k];
            }
            p += 8 * out.pitch;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            unsigned char* p[8];
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = i + k;
                p[k] = at_row(r);
                asm volatile("ld.shared.f32 %0, [%1];"
                             : "=f"(x[k])
                             : "r"(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4)
                             : "memory");
                if (lane >= n) p[k] = nullptr;
                if (add && p[k]) x[k] = reinterpret_cast<const float*>(p[k])[lane] + x[k];
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!p[k]) continue;
                if (out.bf16) reinterpret_cast<__nv_bfloat16*>(p[k])[lane] = __float2bfloat16_rn(x[k]);
                else reinterpret_cast<float*>(p[k])[lane] = x[k];
            }
        }
    }
    __syncwarp();
}

// try_wait that may suspend the thread for up to hint ns.
__device__ __forceinline__ bool try_wait_hint(uint64_t* bar, uint32_t parity, uint32_t hint) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(hint)
        : "memory");
    return ok != 0;
}

// As mbar_wait_for, and false as soon as anyone in this CTA has given up. The
// flag is read while there is something to wait for, not on the way.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                              volatile int* abort_flag) {
    if (try_wait_hint(bar, parity, 100000)) return true;
    const uint64_t t0 = tc::globaltimer();
    while (true) {
        if (try_wait_hint(bar, parity, 100000)) return true;
        if (*abort_flag || tc::globaltimer() - t0 > limit_ns) return false;
    }
}

// The same for a whole warp, whose lanes all get the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns,
                                          volatile int* abort_flag) {
    if (__all_sync(0xffffffffu, try_wait_hint(bar, parity, 100000))) return true;
    const uint64_t t0 = tc::globaltimer();
    while (true) {
        if (__all_sync(0xffffffffu, try_wait_hint(bar, parity, 100000))) return true;
        const bool enough = *abort_flag || tc::globaltimer() - t0 > limit_ns;
        if (__any_sync(0xffffffffu, enough)) return false;
    }
}

// Lane 0's value, which the compiler then knows to be the same in all lanes.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// An operand in the stages: the descriptor of stage 0, and the bytes from one
// 16-deep slice of a step to the next.
struct Operand {
    uint64_t first;
    uint32_t slice;
};

// The products of one step: A of one stage, B of the same or another. (The
// address is the descriptor's lowest field and stays below its 14 bits.)
__device__ __forceinline__ void issue_step(uint32_t to, const Operand& A, int stage_a, const Operand& B,
                                           int stage_b, uint32_t idesc, bool add) {
    const uint64_t da = A.first + static_cast<uint32_t>(stage_a) * (kStageBytes >> 4);
    const uint64_t db = B.first + static_cast<uint32_t>(stage_b) * (kStageBytes >> 4);
#pragma unroll
    for (uint32_t u = 0; u < 4; ++u)
        tc::mma_bf16_pair(to, da + (u * A.slice >> 4), db + (u * B.slice >> 4), idesc,
                          add || u != 0 ? 1u : 0u);
}

// [planes][rows][cols] as a 3-D map of box_rows x box_cols boxes.
inline bool make_map(CUtensorMap* map, const Planes& p, uint32_t box_cols, uint32_t box_rows,
              CUtensorMapSwizzle swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.cols), static_cast<cuuint64_t>(p.rows),
                          static_cast<cuuint64_t>(p.planes)};
    // (One plane: its distance to the next is not used, but has a limit.)
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(p.ld) * 2,
                             static_cast<cuuint64_t>(p.planes == 1 ? 1 : p.rows) *
                                 static_cast<cuuint64_t>(p.ld) * 2};
    cuuint32_t box[3] = {box_cols, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.base), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool operand_map(CUtensorMap* map, const Planes& p) {
    return make_map(map, p, kHeadBox, kHeadBox, CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr int kPairs = 76;  // CTA pairs of a whole GPU, for the choices below

// When the last pair is done, in steps, if n_long units of c_long steps and
// then n_short of c_short are dealt as Deal does.
inline int64_t makespan(int64_t n_long, int64_t c_long, int64_t n_short, int64_t c_short) {
    const int64_t q = n_long / kPairs, high = n_long % kPairs, low = kPairs - high;
    const int64_t lo = q * c_long, hi = lo + (high ? c_long : 0);
    if (n_short == 0) return hi;
    const int64_t rounds = high ? tiles_of(c_long, c_short) : 0;
    if (n_short <= rounds * low) return std::max(hi, lo + tiles_of(n_short, low) * c_short);
    const int64_t rest = n_short - rounds * low, full = rest / kPairs, left = rest % kPairs;
    return std::max(high ? hi + (full + (left > 0)) * c_short : 0,
                    lo + (rounds + full + (left > high)) * c_short);
}

// Columns of the tiles of `rows` x `n` logits: 128 where that ends sooner,
// counted in rounds of the pairs. A narrow tile takes 0.58 of a wide one's time
// (16384 rows, d 1024, V 32768: 663 us in narrow tiles, 570 in wide ones), and
// 0.65 where d is 512 or less.
inline int logit_columns(int64_t rows, int64_t n) {
    const int64_t mt = tiles_of(rows, kHeadTile);
    const int64_t wide = tiles_of(mt * tiles_of(n, 256), kPairs) * 20;
    const int64_t narrow = tiles_of(mt * tiles_of(n, 128), kPairs) * 13;
    return narrow < wide ? 128 : 256;
}

// Columns of the tiles of the products: by what is computed past d; narrow in
// fp32, where a thread of the epilogue holds a unit's sums over its runs (kRun:
// 64 of them, where wide tiles would make 128; beside a block's values this
// takes all 168 registers that ten warps leave a thread, and 236 bytes are
// spilled), and TMEM two accumulators (see launch_head_products).
inline int product_columns(int64_t d, int planes) {
    return planes == 3 || tiles_of(d, 128) * 13 < tiles_of(d, 256) * 20 ? 128 : 256;
}

// Slices of the summed dimension of two products that are made in one launch,
// of ta tiles of steps_a steps and tb tiles of steps_b: 1 where whole tiles share
// the pairs evenly (within a quarter), else the pair of cuts that ends
// soonest, an epilogue being worth 4 steps of one product, and a cut product's
// partial sums and their adding up 12 steps and a third of one per unit.
struct Cuts { int a, b; };
inline Cuts cuts_of(int64_t ta, int64_t steps_a, int64_t tb, int64_t steps_b, int planes) {
    const int64_t pairs = planes == 1 ? 1 : 6;
    const int64_t t[2] = {ta, tb}, steps[2] = {steps_a, steps_b};
    const auto ends = [&](int64_t a, int64_t b) {
        const int64_t c0 = tiles_of(steps[0], a) * pairs + 4, c1 = tiles_of(steps[1], b) * pairs + 4;
        return c1 > c0 ? makespan(t[1] * b, c1, t[0] * a, c0) : makespan(t[0] * a, c0, t[1] * b, c1);
    };
    Cuts best = {1, 1};
    int64_t least = 3 * ends(1, 1);
    const int64_t even = (t[0] * steps[0] + t[1] * steps[1]) * pairs / kPairs;
    if (4 * least <= 3 * 5 * even) return best;
    constexpr int kCuts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 64};
    for (const int a : kCuts) {
        if (a > steps[0] || (a > 1 && t[0] * a > 4 * kPairs)) break;
        for (const int b : kCuts) {
            if (b > steps[1] || (b > 1 && t[1] * b > 4 * kPairs)) break;
            const int64_t e = 3 * ends(a, b) + (a > 1 ? 36 + t[0] * a : 0) +
                              (b > 1 ? 36 + t[1] * b : 0);
            if (e < least) {
                least = e;
                best = {a, b};
            }
        }
    }
    return best;
}

// Row tiles that run together: half of the pairs that are resident, so that
// two columns of tiles are in flight.
constexpr int kGroup = 38;

}  // namespace
}  // namespace dust
