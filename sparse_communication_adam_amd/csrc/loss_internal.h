// loss_internal.h - types shared by the host side of the loss and routing
// operators (loss_api.cpp) and their kernels (k_topk.hip, k_distill.hip,
// k_balance.hip, k_vocab.hip, k_expert.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "scape.h"

namespace scape {

// Errors and checks shared with scape_api.cpp.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);

// A matrix of logits: rows of `cols` elements, `ld` elements apart.
struct Logits {
    const void* z;
    int32_t dtype;
    int64_t rows, cols, ld;
};
inline int dtype_size(int32_t dtype) { return dtype == SCAPE_DTYPE_F32 ? 4 : 2; }

// ---------------------------------------------------------------------------
// Row kernels: workgroups of 256 threads take a row, or a part of one.  Fewer,
// fuller threads beat more: the work that each wave does once a row
// (reductions, the entries' terms) is about as much as 64 elements a lane cost.
constexpr int kRowThreads = 256;
// A kernel that holds the row in registers has at most 16 granules a thread (64
// registers, which leaves as many for the arithmetic at 4 waves per SIMD), and a
// form with 512 threads for twice the row.
constexpr int kHeldGranules = 16;
constexpr int kTopkCapacity = kRowThreads * kHeldGranules;
constexpr int kFusedCapacity = 2 * kTopkCapacity;
constexpr int kMaxSplits = 64;  // a lane of the joining wave for each part
static_assert((SCAPE_ROW_MAX_COLS / 4 + 2) / kTopkCapacity < kMaxSplits, "the longest row fits");

// Granules a row of `cols` elements can touch, whatever its alignment.
inline int64_t row_granules(int32_t dtype, int64_t cols) {
    const int n = 16 / dtype_size(dtype);
    return (cols + n - 1 + n - 1) / n;
}

// Workgroups a row is split over.
struct RowSplit {
    int32_t splits;
    int32_t per;  // granules of each part, a multiple of the unit asked for (the last one may have fewer)
};
// The distillation kernels' parts are cut at whole cells of their bitmap.
constexpr int kCellUnit = 4 * kRowThreads;
RowSplit topk_split(int32_t dtype, int64_t cols);
RowSplit distill_split(int32_t dtype, int64_t rows, int64_t cols);  // of the loss
RowSplit distill_grad_split(int32_t dtype, int64_t rows, int64_t cols);

// ---- k_topk.hip
constexpr int kTopkList = 2048;       // candidates a workgroup sorts in LDS (>= SCAPE_TOPK_MAX_K)
constexpr int kTopkSmallCols = 1024;  // rows that a wave or part of one holds
constexpr int kTopkSmallK = 32;
inline bool topk_small(int64_t cols, int32_t k) { return cols <= kTopkSmallCols && k <= kTopkSmallK; }
struct TopkArgs {
    Logits in;
    int32_t k;
    float scale, c2;  // c2 = scale * log2(e)
    void* val;
    int32_t* idx;
    float* lse;       // or NULL
    uint64_t* cand;   // splits > 1: [rows][splits][k] candidates, then
    float2* part;     // [rows][splits] (reference, sum)
    int32_t splits, per;
};
hipError_t launch_topk(hipStream_t s, const TopkArgs& a);

// ---- k_distill.hip
struct DistillArgs {
    Logits in;
    const void* t_val;
    int32_t t_dtype;
    const int32_t* t_idx;
    const float* t_lse;  // or NULL: renormalised over the entries
    int32_t k;
    float scale, c2;     // c2 = scale * log2(e)
    const float* weight; // or NULL
    const float* dloss;  // backward only, or NULL
    float* loss;
    float* stats;        // [rows][2]
    void* dz;            // or NULL
    int64_t ld_dz;
    float2* part;        // splits > 1: [rows][splits] (reference, sum)
    float2* anchor;      // [rows] the row's L as scale * x + y: for the gradient of the same call, which then
                         // depends on differences of logits only; NULL: from stats
    int32_t splits, per;
    int32_t grad_splits, grad_per;  // of k_distill_grad
};
hipError_t launch_distill_forward(hipStream_t s, const DistillArgs& a);
hipError_t launch_distill_backward(hipStream_t s, const DistillArgs& a);

// ---- k_balance.hip
constexpr int kForwardThreads = 1024, kBackwardThreads = 256;
constexpr int kBackwardBatch = 4;  // tokens a group has on their way
// Lanes that hold a token: with one granule each for up to four, then with
// eight elements each, so that a reduction over the lanes serves more of them;
// 64 may hold 16.
inline int balance_lanes(int32_t dtype, int64_t experts) {
    const int64_t n = 16 / dtype_size(dtype), g = (experts + n - 1) / n, e = (experts + 7) / 8;
    return g <= 1 ? 1 : g <= 4 ? 4 : e <= 8 ? 8 : e <= 16 ? 16 : e <= 32 ? 32 : 64;
}
// The tokens of a segment are cut into runs of `run` tokens, one workgroup
// each.  Segment s's runs start at slot offsets[s] / run + s: no two segments
// share a slot, and tokens / run + segments slots hold them all.
struct BalanceArgs {
    Logits in;             // rows: tokens, cols: experts
    const int32_t* idx;    // [tokens][k]
    int32_t k;
    const int32_t* offsets;  // [segments + 1], or NULL: one segment of all tokens
    int32_t segments;
    const uint8_t* mask;   // [tokens], or NULL
    int32_t score;
    float alpha;
    int32_t* counts;       // [segments][experts]
    float* psum;           // [segments][experts]
    int32_t* n_tok;        // [segments]
    float* loss;           // [segments], or NULL
    const float* dloss;    // backward only: [segments], or NULL
    void* dz;
    int64_t ld_dz;
    int32_t run, slots;
    bool whole;            // forward: a workgroup a segment, no runs
    float2* part;          // [slots][experts]: a run's sum of scores, and its count's bits
    int32_t* part_tok;     // [slots]
};
hipError_t launch_balance_forward(hipStream_t s, const BalanceArgs& a);
hipError_t launch_balance_loss(hipStream_t s, const int32_t* counts, const float* psum, const int32_t* n_tok,
                               int32_t segments, int32_t experts, int32_t k, float alpha, float* loss);
hipError_t launch_balance_backward(hipStream_t s, const BalanceArgs& a);

// ---- k_vocab.hip
constexpr int kSmallWords = 64, kSmallDims = 128;  // tiles of up to 128 tokens
constexpr int kVocabTops = 1024;                   // workgroups that look for the largest exponent
struct VocabRow {
    float f, lse2;  // P's factor (0: does not count), log-sum-exp in base 2
    int32_t label;
    float dh;       // dh's power of two
};
struct VocabArgs {
    const void* h;
    const void* w;
    int64_t ld_h, ld_w;
    int32_t dtype;
    int64_t rows, cols, dim;
    const int32_t* label;
    const float* weight;  // or NULL
    float scale, c2;      // c2 = scale * log2(e)
    int32_t tile_m, tile_n;    // words and tokens of a tile of the logits
    int32_t dh_tile;           // columns of a tile of dh; columns and words of one of dw
    uint32_t tiles_v, tiles_n;
    // forward
    float* loss;
    float* lse;           // backward: read only
    float2* part;         // [tiles_v][rows] (reference, sum), in base 2
    float* at_label;      // [rows] the label's product
    // backward
    const float* dloss;   // or NULL
    void* dh;             // or NULL
    void* dw;             // or NULL
    int64_t ld_dh, ld_dw;
    int64_t rows_pad;     // whole tiles of tokens
    int64_t piece;        // words of a piece
    int64_t ld_p, block_p;  // P: from a row to the next, and from 64 words to the next 64
    int64_t split_words;  // words of a split of dh's sum, a multiple of 64
    int32_t splits;
    VocabRow* row;        // [rows_pad]
    float* dw_scale;      // [1]
    int32_t* top;         // [kVocabTops] largest exponents (fp16)
    void* h_copy;         // [rows][dim]
    void* p;              // rows_pad x piece
    float* dh_sum;        // [splits][rows][dim]
};
hipError_t launch_vocab_loss(hipStream_t s, const VocabArgs& a);
hipError_t launch_vocab_grad(hipStream_t s, const VocabArgs& a);

// ---- k_expert.hip
constexpr int kMaxExperts = SCAPE_EXPERT_MAX;
struct SortArgs {
    const int32_t* idx;  // [choices]
    int64_t choices;
    int32_t experts, bits;  // bits: experts <= 2^bits
    int32_t run, blocks;    // choices of a block (a multiple of 256), and the blocks
    int32_t* offsets;       // [experts + 1]
    int32_t* row;           // [choices]
    uint32_t* counts;       // [blocks][experts]
};
hipError_t launch_expert_sort(hipStream_t s, const SortArgs& a);
struct MoveArgs {
    int32_t dtype;
    int64_t tokens, dim, rows;  // rows: of y
    int32_t k;
    const int32_t* row;    // [tokens][k]
    const void* x;         // gather: tokens' rows; gradient: dout
    int64_t ld_x;
    void* y;               // gather: written; combine: read; gradient: dy, or NULL
    int64_t ld_y;
    const void* y_in;      // gradient: y
    int64_t ld_y_in;
    void* out;             // combine
    int64_t ld_out;
    const float* weight;   // [tokens][k], or NULL
    float* dweight;        // [tokens][k], or NULL
};
hipError_t launch_expert_gather(hipStream_t s, const MoveArgs& a);
hipError_t launch_expert_combine(hipStream_t s, const MoveArgs& a);
hipError_t launch_expert_combine_back(hipStream_t s, const MoveArgs& a);

}  // namespace scape
