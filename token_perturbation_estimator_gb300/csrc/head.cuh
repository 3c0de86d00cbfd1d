// Launch interfaces of the head's losses and gradients: k_head.cu (rows,
// reductions, the order of the steps) and k_head_tc.cu (tensor-core products).
#pragma once
#include <cuda.h>

#include "internal.cuh"

namespace dust {

// What each token is to be scored against: one target id (K = 1, no teacher),
// or K teacher entries.
struct HeadTargets {
    const int32_t* ids;     // [T][K]; outside [0, V): absent
    const float* teacher;   // [T][K] teacher logits, or null
    int64_t K;
    bool many;              // distillation
};

struct HeadProblem {
    const void* H;          // [S * T][d], row stride ld_h
    const void* E;          // [V][d], row stride ld_e
    int64_t ld_h, ld_e;
    bool bf16;
    int64_t S, T, d, V;
    HeadTargets tg;
    float scale;
};

size_t head_loss_workspace_bytes(const HeadProblem& p);
size_t head_grad_workspace_bytes(const HeadProblem& p);
// student: the picked logits [S * T][K] (distillation only).
cudaError_t launch_head_loss(const HeadProblem& p, float* loss, float* lse, float* student,
                             float* delta, void* ws, cudaStream_t s);
cudaError_t launch_head_grad(const HeadProblem& p, const float* lse, const float* student,
                             const float* gloss, bool accumulate, void* gH, int64_t ld_gh,
                             void* gE, bool gE_bf16, void* ws, cudaStream_t s);

// ---- tensor-core products (k_head_tc.cu) ----

// A bf16 matrix in 1 plane, or an fp32 one as 3 bf16 planes whose sum it is.
struct Planes {
    const void* base;
    int64_t rows, cols, ld;  // ld in elements, a multiple of 8; base 16-byte aligned
    int planes;              // planes follow one another, rows * ld elements apart
};

// One row that takes part in a gradient.
struct alignas(16) HeadRow {
    float lse_hi, lse_lo;  // lse log2(e), as a sum of two
    float weight;          // gloss over the largest |gloss|
    int32_t target;        // distillation: the row's number
};

struct HeadCounts {      // written on the device by the row pass
    int32_t rows;        // rows that take part
    float gmax;          // the largest |gloss| among them (1 if that is 0 or not finite)
};

constexpr int kHeadTile = 256;  // rows of a CTA pair's tile; its columns too, or half
constexpr int kHeadBox = 64;    // rows and columns of a TMA box

// The teacher's entries in order of their ids (absent ones left out), and
// where those of each half tile of columns start: for the loss of each token,
// for the gradient of each row.
struct HeadPicks {
    const int2* entries;    // [..][K]: id, and its place among the token's entries; or id, and
                            // exp(x - lse) - q as a float, the same for every entry of an id
    const uint16_t* starts; // [..][bins + 1]: the first entry of a half tile
    int bins;               // half tiles of the whole vocabulary
    int64_t K;
    float* student;         // [rows][K], written (loss)
};

// Partial softmax sums of one row over half a tile's columns: the largest
// logit rounded up to a whole number in units of log 2, and the sum of
// 2^(logit - that).
struct alignas(8) HeadPart { float m, s; };

struct HeadLogits {
    Planes H, E;         // [rows][d], [V][d]
    Planes Hc;           // the rows that take part (gradient), or base null
    int64_t v0, n;       // columns [v0, v0 + n) of the vocabulary
    int bn;              // columns of a tile: head_columns()
    float scale;
    HeadPicks picks;     // distillation, or entries null
    // forward
    const int32_t* targets;  // [T], or null
    int64_t T;
    HeadPart* part;      // [2 * column tiles][ld_part]
    int64_t ld_part;
    float* picked;       // [rows] scaled logits of the targets
    // gradient
    const HeadCounts* counts;
    const HeadRow* rows;
    Planes G;            // [rows rounded up to a tile][n rounded up to a tile]
};

// Columns of the tiles of logits for these sizes.
int head_columns(int64_t rows, int64_t n, int64_t d);

cudaError_t launch_head_lse(const HeadLogits& a, cudaStream_t s);

// ---- the loss and the gradients of a few rows (k_head_few.cu) ----
bool head_few(const HeadProblem& p);        // whether there are few enough
int head_few_parts(const HeadProblem& p);   // partial sums per row
cudaError_t launch_head_few(const HeadProblem& p, HeadPart* part, int64_t ld_part, float* picked,
                            float* student, cudaStream_t s);
int head_few_grad_rows(const HeadProblem& p);   // rows of E a CTA takes at a time (the picks' bins)
int head_few_grad_parts(const HeadProblem& p);  // parts of R d values
cudaError_t launch_head_few_grad(const HeadProblem& p, const HeadPicks& picks, const int32_t* alive,
                                 const float* lse, const float* gloss, bool accumulate, float* part,
                                 void* gH, int64_t ld_gh, void* gE, bool gE_bf16, cudaStream_t s);

// The tensor maps of a gradient's operands, made once per call.
struct HeadMaps {
    CUtensorMap H, Hc, E, G, G_store;
};
bool make_head_maps(HeadMaps* m, const Planes& H, const Planes& Hc, const Planes& E,
                    const Planes& G);
cudaError_t launch_head_factor(const HeadLogits& a, const HeadMaps& m, cudaStream_t s);

// Vocabulary rows of a piece of the gradients.
int64_t head_piece(int64_t rows, int64_t V, int64_t d, int planes);

// Slices of the summed dimension of each product, for the sizes of one piece.
struct HeadCuts { int gh, ge; };
HeadCuts head_cuts(int64_t rows, int64_t n, int64_t d, int planes);

// gH += alpha G E_piece and gE_piece = alpha G^T H, one launch; slices' sums
// are added up by one more.
struct HeadProducts {
    int64_t rows;        // all rows, whether they take part or not
    int planes;
    int64_t v0, n;       // vocabulary rows of the piece
    int64_t d;
    float scale;
    const HeadCounts* counts;
    const int32_t* row_of;  // original row of each row that takes part
    void* gH;            // or null
    int64_t ld_gh;
    bool gh_bf16;
    float* gh_acc;       // partial sums: across pieces, and of slices (else null)
    float* ge_acc;       // of slices (else null)
    HeadCuts cuts;
    bool first, last;    // piece
    void* gE;            // the piece's rows, or null
    bool ge_bf16, accumulate;
};
// Partial sums of a product of m rows and d columns.
int64_t head_acc_floats(int64_t m, int64_t d, int planes, int cut);
cudaError_t launch_head_products(const HeadProducts& a, const HeadMaps& m, cudaStream_t s);

}  // namespace dust
