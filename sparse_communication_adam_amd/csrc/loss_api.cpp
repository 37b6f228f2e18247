// loss_api.cpp - host side of the loss and routing operators of
// include/scape.h: row top-k, distillation from a teacher's top logits, router
// balance loss, vocabulary loss, tokens to their experts and back.
// Arguments are validated here, before anything is launched; the operators
// hold no state and allocate nothing.
#include "loss_internal.h"

#include <cmath>
#include <initializer_list>

using namespace scape;

namespace scape {

namespace {
RowSplit split_evenly(int64_t granules, int64_t parts, int32_t unit) {
    const int64_t units = (granules + unit - 1) / unit, per = (units + parts - 1) / parts;
    return RowSplit{(int32_t)((units + per - 1) / per), (int32_t)(per * unit)};
}
// Parts of at least `least` granules while there are fewer than `fill` in all.
RowSplit split_to_fill(int64_t granules, int64_t rows, int64_t fill, int64_t least) {
    int64_t n = rows > 0 ? fill / rows : 1;
    if (n > granules / least) n = granules / least;
    if (n > kMaxSplits) n = kMaxSplits;
    return split_evenly(granules, n > 1 ? n : 1, kCellUnit);
}
}  // namespace

// The top-k holds a row in registers: up to 8192 granules in a workgroup of 512
// threads, a longer one in parts of up to 4096, each a workgroup of 256, and a
// merge (replayed, us, k = 64: 50304 bf16 in two parts and whole, 512 rows 24
// and 22, 4096 rows 91 and 95; 32000 f32 25 and 22, 98 and 92; 50257 f32 in
// parts of 4096 and of 8192, 512 rows 32 and 36, 4096 rows 157 and 180).  More
// parts than that never paid, not even for one row.
RowSplit topk_split(int32_t dtype, int64_t cols) {
    const int64_t g = row_granules(dtype, cols);
    return split_evenly(g, g <= kFusedCapacity ? 1 : (g + kTopkCapacity - 1) / kTopkCapacity, kRowThreads);
}

// The distillation streams a row of any length.  Cutting it costs the loss a
// join, so only the longest rows are cut, and only where there are fewer than
// the 256 CUs (replayed graphs, us, whole and cut: 7x131072 bf16, 16384
// granules, 19 and 20, 256 rows of them 22 and 28; 7x262144 f32 30 and 20).
RowSplit distill_split(int32_t dtype, int64_t rows, int64_t cols) {
    return split_to_fill(row_granules(dtype, cols), rows, 256, 16384);
}
// The gradient from the statistics has nothing to join; its parts reload the
// entries instead (64x131072 bf16 26 and 18; 16x262144 f32 60 and 18;
// 512x50304 f32, 12576 granules, 48 and 44, 1024 rows of them 85 and 85).
RowSplit distill_grad_split(int32_t dtype, int64_t rows, int64_t cols) {
    return split_to_fill(row_granules(dtype, cols), rows, 2048, 4096);
}

}  // namespace scape

namespace {

constexpr size_t kWorkspaceAlign = 16;
// A launch's threads are counted in 32 bits.
constexpr int64_t kMaxRowBlocks = (int64_t(1) << 32) / 512 - 1;
constexpr int64_t kMaxSmallRows = int64_t(1) << 25;
constexpr int64_t kMaxTokens = int64_t(1) << 30;
constexpr int64_t kMaxSegments = int64_t(1) << 21;
constexpr int64_t kMaxElements = int64_t(1) << 46;  // rows * ld: far beyond memory, far below 2^63

bool is_aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int check_dtype(int32_t dtype, const char* name) {
    if (dtype != SCAPE_DTYPE_F32 && dtype != SCAPE_DTYPE_BF16 && dtype != SCAPE_DTYPE_F16)
        return fail(SCAPE_ERR_INVALID_ARG, "%s: unknown type %d", name, dtype);
    return SCAPE_OK;
}

// A matrix argument: its pointer may be NULL only where it holds no row.
int check_matrix(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const char* name) {
    if (rows > 0 && !p) return fail(SCAPE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!is_aligned(p, dtype_size(dtype))) return fail(SCAPE_ERR_ALIGN, "%s must be aligned to its element", name);
    if (ld < cols) return fail(SCAPE_ERR_SHAPE, "%s: rows of %lld columns are %lld elements apart", name, (long long)cols,
                               (long long)ld);
    if (ld > kMaxElements || rows * (double)ld > (double)kMaxElements)
        return fail(SCAPE_ERR_SHAPE, "%s is too large", name);
    return SCAPE_OK;
}

int check_array(const void* p, size_t align, const char* name) {
    if (!p) return fail(SCAPE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!is_aligned(p, align)) return fail(SCAPE_ERR_ALIGN, "%s must be %zu-byte aligned", name, align);
    return SCAPE_OK;
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
    if (need == 0) return SCAPE_OK;
    if (!ws) return fail(SCAPE_ERR_INVALID_ARG, "workspace is NULL (%lld bytes needed)", (long long)need);
    if (have < need)
        return fail(SCAPE_ERR_SHAPE, "workspace has %lld bytes, needs %lld", (long long)have, (long long)need);
    if (!is_aligned(ws, kWorkspaceAlign)) return fail(SCAPE_ERR_ALIGN, "workspace must be %zu-byte aligned", kWorkspaceAlign);
    return SCAPE_OK;
}

// What an argument takes of memory: rows of `width` bytes, `pitch` apart (an
// array is one row).  No memory: p is NULL.
struct Extent {
    const void* p;
    int64_t rows, width, pitch;
    const char* name;
};
Extent matrix_of(const void* p, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, const char* name) {
    const int64_t size = dtype_size(dtype);
    return Extent{p, rows, cols * size, ld * size, name};
}
Extent array_of(const void* p, int64_t bytes, const char* name) { return Extent{p, 1, bytes, bytes, name}; }

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Whether two extents share a byte; columns of one buffer beside each other do not.
bool share(const Extent& a, const Extent& b) {
    if (!a.p || !b.p || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
    const int64_t d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);  // b's first byte as a counts
    if (d >= (a.rows - 1) * a.pitch + a.width || -d >= (b.rows - 1) * b.pitch + b.width) return false;
    if (a.rows > b.rows) return share(b, a);
    if (a.pitch == b.pitch && a.rows > 1) {
        // b's row t + i meets a's row i where -b.width < d + t pitch < a.width
        int64_t t = floor_div(-b.width - d, a.pitch) + 1;
        if (t < 1 - a.rows) t = 1 - a.rows;
        return t < b.rows && d + t * a.pitch < a.width;
    }
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t at = i * a.pitch - d;  // a's row as b counts
        int64_t j = floor_div(at - b.width, b.pitch) + 1;
        if (j < 0) j = 0;
        if (j < b.rows && j * b.pitch < at + a.width) return true;
    }
    return false;
}
int check_apart(const Extent& out, std::initializer_list<Extent> others) {
    for (const Extent& o : others)
        if (share(out, o)) return fail(SCAPE_ERR_INVALID_ARG, "%s overlaps %s", out.name, o.name);
    return SCAPE_OK;
}

float base2(float scale) { return (float)((double)scale * 1.44269504088896340736); }

int check_scale(float scale) {
    if (!(scale > 0.0f) || !std::isfinite(base2(scale)))
        return fail(SCAPE_ERR_INVALID_ARG, "scale must be positive and finite");
    return SCAPE_OK;
}

// Shapes of the row operators.
int check_rows(int64_t rows, int64_t cols, int32_t k, int32_t max_k) {
    if (rows < 0 || cols < 1) return fail(SCAPE_ERR_SHAPE, "rows must be >= 0 and cols >= 1");
    if (cols > SCAPE_ROW_MAX_COLS)
        return fail(SCAPE_ERR_SHAPE, "%lld columns exceed the maximum of %d", (long long)cols, SCAPE_ROW_MAX_COLS);
    if (k < 1 || k > max_k) return fail(SCAPE_ERR_SHAPE, "k must be in 1..%d (got %d)", max_k, k);
    return SCAPE_OK;
}
int check_blocks(int64_t rows, const RowSplit& sp) {
    if (rows > kMaxRowBlocks / sp.splits) return fail(SCAPE_ERR_SHAPE, "too many rows (%lld)", (long long)rows);
    return SCAPE_OK;
}


int topk_shape(int32_t dtype, int64_t rows, int64_t cols, int32_t k, RowSplit* sp) {
    int rc;
    if ((rc = check_dtype(dtype, "z"))) return rc;
    if ((rc = check_rows(rows, cols, k, SCAPE_TOPK_MAX_K))) return rc;
    if (k > cols) return fail(SCAPE_ERR_SHAPE, "k = %d exceeds the row's %lld columns", k, (long long)cols);
    *sp = RowSplit{1, 0};
    if (topk_small(cols, k)) {
        if (rows > kMaxSmallRows) return fail(SCAPE_ERR_SHAPE, "too many rows (%lld)", (long long)rows);
        return SCAPE_OK;
    }
    *sp = topk_split(dtype, cols);
    return check_blocks(rows, *sp);
}
int64_t topk_bytes(int64_t rows, int32_t k, const RowSplit& sp) {
    return sp.splits > 1 ? rows * sp.splits * ((int64_t)k * 8 + 8) : 0;
}

int distill_shape(int32_t dtype, int64_t rows, int64_t cols, int32_t k, RowSplit (*split)(int32_t, int64_t, int64_t),
                  RowSplit* sp) {
    int rc;
    if ((rc = check_dtype(dtype, "z"))) return rc;
    if ((rc = check_rows(rows, cols, k, SCAPE_DISTILL_MAX_K))) return rc;
    *sp = split(dtype, rows, cols);
    return check_blocks(rows, *sp);
}
// The parts' sums, and the anchors where the gradient is a launch of its own.
int64_t parts_bytes(int64_t rows, const RowSplit& sp) { return sp.splits > 1 ? rows * sp.splits * 8 : 0; }
int64_t distill_bytes(int64_t rows, const RowSplit& sp, bool grad) {
    return parts_bytes(rows, sp) + (grad && (sp.splits > 1 || sp.per > kFusedCapacity) ? rows * 8 : 0);
}

int distill_query(int32_t dtype, int64_t rows, int64_t cols, int32_t k, bool grad, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    RowSplit sp;
    if (int rc = distill_shape(dtype, rows, cols, k, distill_split, &sp)) return rc;
    *bytes = distill_bytes(rows, sp, grad);
    return SCAPE_OK;
}

int check_teacher(const scape_teacher* t, int64_t rows) {
    if (!t) return fail(SCAPE_ERR_INVALID_ARG, "teacher is NULL");
    int rc;
    if ((rc = check_dtype(t->dtype, "teacher->val"))) return rc;
    if (rows == 0) return SCAPE_OK;
    if ((rc = check_array(t->val, dtype_size(t->dtype), "teacher->val"))) return rc;
    if ((rc = check_array(t->idx, 4, "teacher->idx"))) return rc;
    if (t->lse && !is_aligned(t->lse, 4)) return fail(SCAPE_ERR_ALIGN, "teacher->lse must be 4-byte aligned");
    return SCAPE_OK;
}

int check_optional(const void* p, const char* name) {
    if (p && !is_aligned(p, 4)) return fail(SCAPE_ERR_ALIGN, "%s must be 4-byte aligned", name);
    return SCAPE_OK;
}

// Tokens of a run.  The forward pass joins a segment's runs in one workgroup,
// so it takes about a run for each CU.
int32_t forward_run(int64_t tokens) {
    constexpr int64_t kRuns = 256, kStep = 128;
    const int64_t r = (tokens + kRuns - 1) / kRuns;
    return (int32_t)(r <= kStep ? kStep : (r + kStep - 1) / kStep * kStep);
}
// The gradient has nothing to join: a run is one batch of a workgroup's groups
// (2^16 of them at most, then several).
int32_t backward_run(int32_t dtype, int64_t tokens, int32_t experts) {
    const int64_t batch = kBackwardThreads / balance_lanes(dtype, experts) * kBackwardBatch, n = tokens / (batch << 16) + 1;
    return (int32_t)(batch * n);
}
// Few logits: a workgroup a segment makes its sums and its loss in one launch
// (replayed, us, in runs and whole: 2000x8 in 7 segments 17 and 13, 1024x64 in
// one 16 and 14, 2048x64 in one 17 and 20).
bool whole_segments(int64_t tokens, int32_t experts) { return tokens * experts <= 65536; }

int balance_shape(int32_t dtype, int64_t tokens, int32_t experts, int32_t segments) {
    int rc;
    if ((rc = check_dtype(dtype, "logits"))) return rc;
    if (tokens < 0 || tokens > kMaxTokens) return fail(SCAPE_ERR_SHAPE, "tokens must be in 0..2^30");
    if (experts < 1 || experts > SCAPE_BALANCE_MAX_EXPERTS)
        return fail(SCAPE_ERR_SHAPE, "experts must be in 1..%d (got %d)", SCAPE_BALANCE_MAX_EXPERTS, experts);
    if (segments < 1 || segments > kMaxSegments) return fail(SCAPE_ERR_SHAPE, "segments must be in 1..2^21");
    return SCAPE_OK;
}
int check_choices(int64_t tokens, int32_t experts, int32_t k) {
    if (k < 1 || k > experts) return fail(SCAPE_ERR_SHAPE, "k must be in 1..experts (got %d)", k);
    if (tokens * k > INT32_MAX) return fail(SCAPE_ERR_SHAPE, "more than 2^31 - 1 choices");
    return SCAPE_OK;
}
int check_alpha(float alpha) {
    if (!std::isfinite(alpha)) return fail(SCAPE_ERR_INVALID_ARG, "alpha must be finite");
    return SCAPE_OK;
}
int check_router(int32_t score, const int32_t* offsets, int32_t segments) {
    if (score != SCAPE_SCORE_SOFTMAX && score != SCAPE_SCORE_SIGMOID)
        return fail(SCAPE_ERR_INVALID_ARG, "unknown score %d", score);
    if (!offsets && segments != 1) return fail(SCAPE_ERR_INVALID_ARG, "%d segments need offsets", segments);
    return check_optional(offsets, "offsets");
}
int64_t balance_bytes(int64_t tokens, int32_t experts, int32_t segments) {
    const int64_t slots = tokens / forward_run(tokens) + segments;
    return slots * (8 * (int64_t)experts + 4);
}

// ---- vocabulary loss
constexpr int64_t kMaxHeadLd = int64_t(1) << 21;  // a tile's offsets stay below 2^31 bytes

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Tokens of a tile: what holds few, and of many the size that wastes least.  A
// tile of 192 takes 4/5 of one of 256 (1536 tokens in 8 and in 6 tiles, us: loss of
// 50257x1024 bf16 159 and 147, of 131072x2048 f16 694 and 636, gradients 496 and
// 467, 2280 and 2173; 300 tokens of 50257x1024 50 and 55, 500 of them 72 and 59).
// How many CUs get a tile is not looked at: 129 to 256 tokens under fewer than
// 65536 words leave some idle.
int32_t vocab_tile(int64_t rows) {
    for (int32_t t = 16; t <= 128; t *= 2)
        if (rows <= t) return t;
    return (rows + 191) / 192 * 4 < (rows + 255) / 256 * 5 ? 192 : 256;
}

int vocab_shape(int32_t dtype, int64_t rows, int64_t cols, int64_t dim, VocabArgs* a) {
    if (dtype != SCAPE_DTYPE_BF16 && dtype != SCAPE_DTYPE_F16)
        return fail(SCAPE_ERR_INVALID_ARG, "the vocabulary loss takes bfloat16 or float16 (got type %d)", dtype);
    if (rows < 0 || rows > SCAPE_VOCAB_MAX_ROWS)
        return fail(SCAPE_ERR_SHAPE, "rows must be in 0..%d", SCAPE_VOCAB_MAX_ROWS);
    if (cols < 1 || cols > SCAPE_ROW_MAX_COLS) return fail(SCAPE_ERR_SHAPE, "cols must be in 1..%d", SCAPE_ROW_MAX_COLS);
    if (dim < 8 || dim > SCAPE_VOCAB_MAX_DIM || dim % 8)
        return fail(SCAPE_ERR_SHAPE, "dim must be a multiple of 8 in 8..%d (got %lld)", SCAPE_VOCAB_MAX_DIM, (long long)dim);
    a->dtype = dtype;
    a->rows = rows;
    a->cols = cols;
    a->dim = dim;
    a->tile_n = vocab_tile(rows);
    const bool small = a->tile_n <= 128;
    a->tile_m = small ? kSmallWords : 256;
    a->dh_tile = small ? kSmallDims : 256;
    a->tiles_v = (uint32_t)((cols + a->tile_m - 1) / a->tile_m);
    a->tiles_n = (uint32_t)((rows + a->tile_n - 1) / a->tile_n);
    a->rows_pad = (int64_t)a->tiles_n * a->tile_n;
    return SCAPE_OK;
}
// The pieces of the backward pass: P of one is at most 2^27 elements, but never
// less than 4096 words wide, so that dw has tiles for the CUs: above 32768 rows it
// is up to 4096 rows_pad elements (8 GB at the most rows).  P lies in blocks of
// 64 words, [words / 64][rows_pad][64], so that what a step of either product
// takes is one run of memory or four; fewer rows than a step's lie as rows.
// dh's sums are split over the words where its tiles leave CUs idle: the number
// of splits is the one with the least rounds of tiles on the CUs times a split's
// steps (and about 6 more for its start and its end), counting the splits'
// sums, which are written and read once more, at a step for each 8 MB.  Beside
// dw, in one launch (up to 64 tokens), there are 128 workgroups where the tiles
// divide them, three times as many where not.  bf16 gradient us with 128 and 384:
//   7 x 50257 x 256 26 and 28, 512 37 and 39, 768 50 and 53, 1024 64 and 67, 1536
//   115 and 107, 2048 150 and 134, 4096 295 and 287, 5120 369 and 354
//   64 x 32000 x 1024 46 and 49, 1536 68 and 75, 2048 95 and 103, 4096 178 and 190
// so it is right up to a width of 1024 but for 768, and for wider rows as the
// vocabulary has it; where it is not, it costs a tenth.  Alone dh takes as many
// workgroups as LDS holds.
void vocab_pieces(VocabArgs* a) {
    int64_t most = a->rows_pad ? (int64_t(1) << 27) / a->rows_pad / 256 * 256 : a->cols;
    if (most < 4096) most = 4096;
    const int64_t pieces = (a->cols + most - 1) / most;
    a->piece = round_up((a->cols + pieces - 1) / pieces, 256);
    a->ld_p = a->tile_n >= 64 ? 64 : a->piece;
    a->block_p = a->rows_pad * 64;
    const int64_t tiles = (a->dim + a->dh_tile - 1) / a->dh_tile * (a->tiles_n ? a->tiles_n : 1);
    const int64_t slots = a->tile_n <= 64 ? (128 % tiles == 0 ? 128 : 384) : a->tile_n <= 128 ? 512 : 256;
    int64_t best = INT64_MAX;
    for (int64_t n = 1; n <= 128 && (n == 1 || a->piece / n >= 256); ++n) {
        const int64_t words = round_up((a->piece + n - 1) / n, 64), splits = (a->piece + words - 1) / words;
        const int64_t cost = (tiles * splits + slots - 1) / slots * (words / 64 + 6) +
                             (splits > 1 ? splits * a->rows * a->dim * 8 / (int64_t(8) << 20) : 0);
        if (cost < best) {
            best = cost;
            a->split_words = words;
            a->splits = (int32_t)splits;
        }
    }
}
int64_t vocab_loss_bytes(const VocabArgs& a) {
    return a.rows * ((int64_t)a.tiles_v * 8 + 4);
}
// The workspace of the backward pass, each part a multiple of 16 bytes.
struct VocabParts {
    int64_t row, dw_scale, top, h_copy, p, dh_sum, all;
};
VocabParts vocab_parts(const VocabArgs& a) {
    VocabParts w;
    w.row = 0;
    w.dw_scale = w.row + a.rows_pad * (int64_t)sizeof(VocabRow);
    w.top = w.dw_scale + 16;
    w.h_copy = w.top + (a.dtype == SCAPE_DTYPE_F16 ? kVocabTops * 4 : 0);
    w.p = w.h_copy + a.rows * a.dim * 2;
    w.dh_sum = w.p + a.rows_pad * a.piece * 2;
    const bool summed = a.splits > 1 || a.piece < a.cols;  // else one launch writes dh itself
    w.all = a.rows ? w.dh_sum + (summed ? (int64_t)a.splits * a.rows * a.dim * 4 : 0) : 0;
    return w;
}

// A matrix that is moved 16 bytes at a time.
int check_wide(const void* p, int64_t rows, int64_t dim, int64_t ld, const char* name) {
    if (rows > 0 && !p) return fail(SCAPE_ERR_INVALID_ARG, "%s is NULL", name);
    if (!is_aligned(p, 16)) return fail(SCAPE_ERR_ALIGN, "%s must be 16-byte aligned", name);
    if (ld < dim) return fail(SCAPE_ERR_SHAPE, "%s: rows of %lld columns are %lld elements apart", name, (long long)dim,
                              (long long)ld);
    if (ld > kMaxHeadLd) return fail(SCAPE_ERR_SHAPE, "%s: rows are more than 2^21 elements apart", name);
    if (ld % 8) return fail(SCAPE_ERR_ALIGN, "%s: rows must be a multiple of 8 elements apart", name);
    return SCAPE_OK;
}
int vocab_head(const scape_head* h, VocabArgs* a) {
    if (!h) return fail(SCAPE_ERR_INVALID_ARG, "head is NULL");
    int rc;
    if ((rc = vocab_shape(h->dtype, h->rows, h->cols, h->dim, a))) return rc;
    if ((rc = check_wide(h->h, h->rows, h->dim, h->ld_h, "h"))) return rc;
    if ((rc = check_wide(h->w, h->cols, h->dim, h->ld_w, "w"))) return rc;
    if ((rc = check_scale(h->scale))) return rc;
    if (h->rows > 0 && (rc = check_array(h->label, 4, "label"))) return rc;
    if ((rc = check_optional(h->weight, "weight"))) return rc;
    a->h = h->h;
    a->w = h->w;
    a->ld_h = h->ld_h;
    a->ld_w = h->ld_w;
    a->label = h->label;
    a->weight = h->weight;
    a->scale = h->scale;
    a->c2 = base2(h->scale);
    return SCAPE_OK;
}

struct HeadExtents {
    Extent h, w, label, weight;
    explicit HeadExtents(const VocabArgs& a)
        : h(matrix_of(a.h, a.dtype, a.rows, a.dim, a.ld_h, "h")), w(matrix_of(a.w, a.dtype, a.cols, a.dim, a.ld_w, "w")),
          label(array_of(a.label, a.rows * 4, "label")), weight(array_of(a.weight, a.rows * 4, "weight")) {}
};

// ---- tokens to their experts
constexpr int64_t kMaxMoved = int64_t(1) << 25;     // tokens of a move: a wave each
constexpr int64_t kMaxMovedDim = int64_t(1) << 24;  // bytes in a row are counted in 32 bits

int sort_shape(int64_t tokens, int32_t k, int32_t experts, SortArgs* a) {
    if (experts < 1 || experts > SCAPE_EXPERT_MAX)
        return fail(SCAPE_ERR_SHAPE, "experts must be in 1..%d (got %d)", SCAPE_EXPERT_MAX, experts);
    if (tokens < 0 || tokens > kMaxTokens) return fail(SCAPE_ERR_SHAPE, "tokens must be in 0..2^30");
    if (k < 1) return fail(SCAPE_ERR_SHAPE, "k must be at least 1 (got %d)", k);
    if (tokens * k > INT32_MAX) return fail(SCAPE_ERR_SHAPE, "more than 2^31 - 1 choices");
    a->choices = tokens * k;
    a->experts = experts;
    a->bits = 0;
    while ((1 << a->bits) < experts) ++a->bits;
    // a block of 2048 choices; more where there would be over 512 of them
    int64_t run = 2048;
    if (a->choices > run * 512) run = round_up((a->choices + 511) / 512, 256);
    a->run = (int32_t)run;
    a->blocks = a->choices <= run ? 1 : (int32_t)((a->choices + run - 1) / run);
    return SCAPE_OK;
}
int64_t sort_bytes(const SortArgs& a) { return a.blocks > 1 ? (int64_t)a.blocks * a.experts * 4 : 0; }

int check_moves(int32_t dtype, int64_t tokens, int64_t dim, int64_t rows, int32_t k, const int32_t* row) {
    int rc;
    if ((rc = check_dtype(dtype, "the rows"))) return rc;
    if (tokens < 0 || tokens > kMaxMoved) return fail(SCAPE_ERR_SHAPE, "tokens must be in 0..2^25");
    if (dim < 1 || dim > kMaxMovedDim) return fail(SCAPE_ERR_SHAPE, "dim must be in 1..2^24");
    if (rows < 0) return fail(SCAPE_ERR_SHAPE, "rows must be >= 0");
    if (k < 1) return fail(SCAPE_ERR_SHAPE, "k must be at least 1 (got %d)", k);
    if (tokens * k > INT32_MAX) return fail(SCAPE_ERR_SHAPE, "more than 2^31 - 1 choices");
    if (tokens > 0 && (rc = check_array(row, 4, "row"))) return rc;
    return SCAPE_OK;
}

}  // namespace

extern "C" {

int scape_topk_rows_workspace(int32_t dtype, int64_t rows, int64_t cols, int32_t k, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    RowSplit sp;
    if (int rc = topk_shape(dtype, rows, cols, k, &sp)) return rc;
    *bytes = topk_bytes(rows, k, sp);
    return SCAPE_OK;
}

int scape_topk_rows(const void* z, int32_t dtype, int64_t rows, int64_t cols, int64_t ld, int32_t k, float scale,
                    void* val, int32_t* idx, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    RowSplit sp;
    int rc;
    if ((rc = topk_shape(dtype, rows, cols, k, &sp))) return rc;
    if ((rc = check_matrix(z, dtype, rows, cols, ld, "z"))) return rc;
    if ((rc = check_scale(scale))) return rc;
    if (rows == 0) return SCAPE_OK;
    if ((rc = check_array(val, dtype_size(dtype), "val"))) return rc;
    if ((rc = check_array(idx, 4, "idx"))) return rc;
    if ((rc = check_optional(lse, "lse"))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, topk_bytes(rows, k, sp)))) return rc;
    TopkArgs a{};
    a.in = Logits{z, dtype, rows, cols, ld};
    a.k = k;
    a.scale = scale;
    a.c2 = base2(scale);
    a.val = val;
    a.idx = idx;
    a.lse = lse;
    a.splits = sp.splits;
    a.per = sp.per;
    a.cand = static_cast<uint64_t*>(workspace);
    a.part = reinterpret_cast<float2*>(static_cast<uint64_t*>(workspace) + (sp.splits > 1 ? rows * sp.splits * k : 0));
    const hipError_t e = launch_topk((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "row top-k");
}

int scape_distill_workspace(int32_t dtype, int64_t rows, int64_t cols, int32_t k, int64_t* bytes) {
    return distill_query(dtype, rows, cols, k, true, bytes);
}

int scape_distill_loss_workspace(int32_t dtype, int64_t rows, int64_t cols, int32_t k, int64_t* bytes) {
    return distill_query(dtype, rows, cols, k, false, bytes);
}

int scape_distill_forward(const void* z, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                          const scape_teacher* teacher, float scale, const float* weight, float* loss, float* stats,
                          void* dz, int64_t ld_dz, void* workspace, int64_t workspace_bytes, void* stream) {
    RowSplit sp;
    int rc;
    if ((rc = check_teacher(teacher, rows))) return rc;
    if ((rc = distill_shape(dtype, rows, cols, teacher->k, distill_split, &sp))) return rc;
    if ((rc = check_matrix(z, dtype, rows, cols, ld, "z"))) return rc;
    if ((rc = check_scale(scale))) return rc;
    if (dz && (rc = check_matrix(dz, dtype, rows, cols, ld_dz, "dz"))) return rc;
    if (dz == z && dz && ld_dz != ld) return fail(SCAPE_ERR_SHAPE, "dz over z needs z's row distance");
    if (rows == 0) return SCAPE_OK;
    if ((rc = check_optional(weight, "weight"))) return rc;
    if ((rc = check_array(loss, 4, "loss"))) return rc;
    if ((rc = check_array(stats, 4, "stats"))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, distill_bytes(rows, sp, dz != nullptr)))) return rc;
    DistillArgs a{};
    a.in = Logits{z, dtype, rows, cols, ld};
    a.t_val = teacher->val;
    a.t_dtype = teacher->dtype;
    a.t_idx = teacher->idx;
    a.t_lse = teacher->lse;
    a.k = teacher->k;
    a.scale = scale;
    a.c2 = base2(scale);
    a.weight = weight;
    a.loss = loss;
    a.stats = stats;
    a.dz = dz;
    a.ld_dz = ld_dz;
    a.part = static_cast<float2*>(workspace);
    a.splits = sp.splits;
    a.per = sp.per;
    if (dz) {
        if (distill_bytes(rows, sp, true) > parts_bytes(rows, sp)) a.anchor = a.part + parts_bytes(rows, sp) / 8;
        if ((rc = distill_shape(dtype, rows, cols, teacher->k, distill_grad_split, &sp))) return rc;
        a.grad_splits = sp.splits;
        a.grad_per = sp.per;
    }
    const hipError_t e = launch_distill_forward((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "distillation loss");
}

int scape_distill_backward(const void* z, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                           const scape_teacher* teacher, float scale, const float* weight, const float* stats,
                           const float* dloss, void* dz, int64_t ld_dz, void* stream) {
    RowSplit sp;
    int rc;
    if ((rc = check_teacher(teacher, rows))) return rc;
    if ((rc = distill_shape(dtype, rows, cols, teacher->k, distill_grad_split, &sp))) return rc;
    if ((rc = check_matrix(z, dtype, rows, cols, ld, "z"))) return rc;
    if ((rc = check_scale(scale))) return rc;
    if ((rc = check_matrix(dz, dtype, rows, cols, ld_dz, "dz"))) return rc;
    if (dz == z && dz && ld_dz != ld) return fail(SCAPE_ERR_SHAPE, "dz over z needs z's row distance");
    if (rows == 0) return SCAPE_OK;
    if ((rc = check_optional(weight, "weight"))) return rc;
    if ((rc = check_array(stats, 4, "stats"))) return rc;
    if ((rc = check_optional(dloss, "dloss"))) return rc;
    DistillArgs a{};
    a.in = Logits{z, dtype, rows, cols, ld};
    a.t_val = teacher->val;
    a.t_dtype = teacher->dtype;
    a.t_idx = teacher->idx;
    a.t_lse = teacher->lse;
    a.k = teacher->k;
    a.scale = scale;
    a.c2 = base2(scale);
    a.weight = weight;
    a.dloss = dloss;
    a.stats = const_cast<float*>(stats);  // read only in this launch
    a.dz = dz;
    a.ld_dz = ld_dz;
    a.grad_splits = sp.splits;
    a.grad_per = sp.per;
    const hipError_t e = launch_distill_backward((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "distillation gradient");
}

int scape_balance_workspace(int64_t tokens, int32_t experts, int32_t segments, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    if (int rc = balance_shape(SCAPE_DTYPE_F32, tokens, experts, segments)) return rc;
    *bytes = balance_bytes(tokens, experts, segments);
    return SCAPE_OK;
}

int scape_balance_forward(const void* logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t ld,
                          const int32_t* idx, int32_t k, const int32_t* offsets, int32_t segments,
                          const uint8_t* mask, int32_t score, float alpha, int32_t* counts, float* psum,
                          int32_t* n_tok, float* loss, void* workspace, int64_t workspace_bytes, void* stream) {
    int rc;
    if ((rc = balance_shape(dtype, tokens, experts, segments))) return rc;
    if ((rc = check_choices(tokens, experts, k))) return rc;
    if ((rc = check_matrix(logits, dtype, tokens, experts, ld, "logits"))) return rc;
    if ((rc = check_router(score, offsets, segments))) return rc;
    if ((rc = check_alpha(alpha))) return rc;
    if (tokens > 0 && (rc = check_array(idx, 4, "idx"))) return rc;
    if ((rc = check_array(counts, 4, "counts"))) return rc;
    if ((rc = check_array(psum, 4, "psum"))) return rc;
    if ((rc = check_array(n_tok, 4, "n_tok"))) return rc;
    if ((rc = check_optional(loss, "loss"))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, balance_bytes(tokens, experts, segments)))) return rc;
    BalanceArgs a{};
    a.in = Logits{logits, dtype, tokens, experts, ld};
    a.idx = idx;
    a.k = k;
    a.offsets = offsets;
    a.segments = segments;
    a.mask = mask;
    a.score = score;
    a.alpha = alpha;
    a.counts = counts;
    a.psum = psum;
    a.n_tok = n_tok;
    a.loss = loss;
    a.whole = tokens > 0 && whole_segments(tokens, experts);
    a.run = forward_run(tokens);
    a.part = static_cast<float2*>(workspace);
    const int64_t slots = tokens / a.run + segments;
    a.part_tok = reinterpret_cast<int32_t*>(a.part + slots * experts);
    a.slots = (int32_t)(a.whole ? segments : slots);
    const hipError_t e = launch_balance_forward((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "balance loss");
}

int scape_balance_loss(const int32_t* counts, const float* psum, const int32_t* n_tok, int32_t segments,
                       int32_t experts, int32_t k, float alpha, float* loss, void* stream) {
    int rc;
    if ((rc = balance_shape(SCAPE_DTYPE_F32, 0, experts, segments))) return rc;
    if ((rc = check_choices(0, experts, k))) return rc;
    if ((rc = check_alpha(alpha))) return rc;
    if ((rc = check_array(counts, 4, "counts"))) return rc;
    if ((rc = check_array(psum, 4, "psum"))) return rc;
    if ((rc = check_array(n_tok, 4, "n_tok"))) return rc;
    if ((rc = check_array(loss, 4, "loss"))) return rc;
    const hipError_t e = launch_balance_loss((hipStream_t)stream, counts, psum, n_tok, segments, experts, k, alpha, loss);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "balance loss");
}

int scape_balance_backward(const void* logits, int32_t dtype, int64_t tokens, int32_t experts, int64_t ld, int32_t k,
                           const int32_t* offsets, int32_t segments, const uint8_t* mask, int32_t score, float alpha,
                           const int32_t* counts, const int32_t* n_tok, const float* dloss, void* dlogits,
                           int64_t ld_d, void* stream) {
    int rc;
    if ((rc = balance_shape(dtype, tokens, experts, segments))) return rc;
    if ((rc = check_choices(tokens, experts, k))) return rc;
    if ((rc = check_matrix(logits, dtype, tokens, experts, ld, "logits"))) return rc;
    if ((rc = check_matrix(dlogits, dtype, tokens, experts, ld_d, "dlogits"))) return rc;
    if (dlogits == logits && dlogits && ld_d != ld)
        return fail(SCAPE_ERR_SHAPE, "dlogits over logits needs the logits' row distance");
    if ((rc = check_router(score, offsets, segments))) return rc;
    if ((rc = check_alpha(alpha))) return rc;
    if (tokens == 0) return SCAPE_OK;
    if ((rc = check_array(counts, 4, "counts"))) return rc;
    if ((rc = check_array(n_tok, 4, "n_tok"))) return rc;
    if ((rc = check_optional(dloss, "dloss"))) return rc;
    BalanceArgs a{};
    a.in = Logits{logits, dtype, tokens, experts, ld};
    a.k = k;
    a.offsets = offsets;
    a.segments = segments;
    a.mask = mask;
    a.score = score;
    a.alpha = alpha;
    a.counts = const_cast<int32_t*>(counts);  // read only in this launch
    a.n_tok = const_cast<int32_t*>(n_tok);
    a.dloss = dloss;
    a.dz = dlogits;
    a.ld_dz = ld_d;
    a.run = backward_run(dtype, tokens, experts);
    a.slots = (int32_t)(tokens / a.run + segments);
    const hipError_t e = launch_balance_backward((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "balance gradient");
}

int scape_vocab_loss_workspace(int32_t dtype, int64_t rows, int64_t cols, int64_t dim, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    VocabArgs a{};
    if (int rc = vocab_shape(dtype, rows, cols, dim, &a)) return rc;
    *bytes = vocab_loss_bytes(a);
    return SCAPE_OK;
}

int scape_vocab_loss_forward(const scape_head* head, float* loss, float* lse, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    VocabArgs a{};
    int rc;
    if ((rc = vocab_head(head, &a))) return rc;
    if (a.rows == 0) return SCAPE_OK;
    if ((rc = check_array(loss, 4, "loss"))) return rc;
    if ((rc = check_array(lse, 4, "lse"))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, vocab_loss_bytes(a)))) return rc;
    const HeadExtents in(a);
    const Extent to = array_of(loss, a.rows * 4, "loss"), to_lse = array_of(lse, a.rows * 4, "lse");
    const Extent ws = array_of(workspace, vocab_loss_bytes(a), "workspace");
    if ((rc = check_apart(to, {to_lse, ws, in.h, in.w, in.label}))) return rc;
    if (loss != a.weight && (rc = check_apart(to, {in.weight}))) return rc;
    if ((rc = check_apart(to_lse, {ws, in.h, in.w, in.label, in.weight}))) return rc;
    if ((rc = check_apart(ws, {in.h, in.w, in.label, in.weight}))) return rc;
    a.loss = loss;
    a.lse = lse;
    a.part = static_cast<float2*>(workspace);
    a.at_label = reinterpret_cast<float*>(a.part + a.rows * a.tiles_v);
    const hipError_t e = launch_vocab_loss((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "vocabulary loss");
}

int scape_vocab_grad_workspace(int32_t dtype, int64_t rows, int64_t cols, int64_t dim, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    VocabArgs a{};
    if (int rc = vocab_shape(dtype, rows, cols, dim, &a)) return rc;
    vocab_pieces(&a);
    *bytes = vocab_parts(a).all;
    return SCAPE_OK;
}

int scape_vocab_loss_backward(const scape_head* head, const float* lse, const float* dloss, void* dh, int64_t ld_dh,
                              void* dw, int64_t ld_dw, void* workspace, int64_t workspace_bytes, void* stream) {
    VocabArgs a{};
    int rc;
    if ((rc = vocab_head(head, &a))) return rc;
    if (dh && (rc = check_wide(dh, a.rows, a.dim, ld_dh, "dh"))) return rc;
    if (dw && (rc = check_wide(dw, a.cols, a.dim, ld_dw, "dw"))) return rc;
    if (a.rows > 0 && (rc = check_array(lse, 4, "lse"))) return rc;
    if ((rc = check_optional(dloss, "dloss"))) return rc;
    if (!dw && (!dh || a.rows == 0)) return SCAPE_OK;
    vocab_pieces(&a);
    const VocabParts w = vocab_parts(a);
    if ((rc = check_workspace(workspace, workspace_bytes, w.all))) return rc;
    const HeadExtents in(a);
    const Extent from_lse = array_of(lse, a.rows * 4, "lse"), from_dloss = array_of(dloss, a.rows * 4, "dloss");
    const Extent to_h = matrix_of(dh, a.dtype, a.rows, a.dim, ld_dh, "dh"), to_w = matrix_of(dw, a.dtype, a.cols, a.dim, ld_dw, "dw");
    const Extent scratch = array_of(workspace, w.all, "workspace");
    if ((rc = check_apart(to_h, {to_w, scratch, in.h, in.w, in.label, in.weight, from_lse, from_dloss}))) return rc;
    if ((rc = check_apart(to_w, {scratch, in.h, in.w, in.label, in.weight, from_lse, from_dloss}))) return rc;
    if ((rc = check_apart(scratch, {in.h, in.w, in.label, in.weight, from_lse, from_dloss}))) return rc;
    char* const ws = static_cast<char*>(workspace);
    a.lse = const_cast<float*>(lse);  // read only in these launches
    a.dloss = dloss;
    a.dh = dh;
    a.dw = dw;
    a.ld_dh = ld_dh;
    a.ld_dw = ld_dw;
    if (a.rows > 0) {
        a.row = reinterpret_cast<VocabRow*>(ws + w.row);
        a.dw_scale = reinterpret_cast<float*>(ws + w.dw_scale);
        a.top = reinterpret_cast<int32_t*>(ws + w.top);
        a.h_copy = ws + w.h_copy;
        a.p = ws + w.p;
        a.dh_sum = reinterpret_cast<float*>(ws + w.dh_sum);
    }
    const hipError_t e = launch_vocab_grad((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "vocabulary loss gradient");
}

int scape_expert_sort_workspace(int64_t tokens, int32_t k, int32_t experts, int64_t* bytes) {
    if (!bytes) return fail(SCAPE_ERR_INVALID_ARG, "bytes is NULL");
    SortArgs a{};
    if (int rc = sort_shape(tokens, k, experts, &a)) return rc;
    *bytes = sort_bytes(a);
    return SCAPE_OK;
}

int scape_expert_sort(const int32_t* idx, int64_t tokens, int32_t k, int32_t experts, int32_t* offsets, int32_t* row,
                      void* workspace, int64_t workspace_bytes, void* stream) {
    SortArgs a{};
    int rc;
    if ((rc = sort_shape(tokens, k, experts, &a))) return rc;
    if (tokens > 0 && (rc = check_array(idx, 4, "idx"))) return rc;
    if ((rc = check_array(offsets, 4, "offsets"))) return rc;
    if (tokens > 0 && (rc = check_array(row, 4, "row"))) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, sort_bytes(a)))) return rc;
    const Extent from = array_of(idx, a.choices * 4, "idx"), to = array_of(row, a.choices * 4, "row");
    const Extent first = array_of(offsets, ((int64_t)experts + 1) * 4, "offsets"), ws = array_of(workspace, sort_bytes(a), "workspace");
    if (row != idx && (rc = check_apart(to, {from}))) return rc;  // in place a wave reads its choices before their places are written
    if ((rc = check_apart(first, {from, to, ws}))) return rc;
    if ((rc = check_apart(ws, {from, to}))) return rc;
    a.idx = idx;
    a.offsets = offsets;
    a.row = row;
    a.counts = static_cast<uint32_t*>(workspace);
    const hipError_t e = launch_expert_sort((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "expert sort");
}

int scape_expert_gather(const void* x, int32_t dtype, int64_t tokens, int64_t dim, int64_t ld_x, const int32_t* row,
                        int32_t k, void* y, int64_t rows, int64_t ld_y, void* stream) {
    int rc;
    if ((rc = check_moves(dtype, tokens, dim, rows, k, row))) return rc;
    if ((rc = check_matrix(x, dtype, tokens, dim, ld_x, "x"))) return rc;
    if ((rc = check_matrix(y, dtype, rows, dim, ld_y, "y"))) return rc;
    if (tokens == 0 || rows == 0) return SCAPE_OK;
    if ((rc = check_apart(matrix_of(y, dtype, rows, dim, ld_y, "y"),
                          {matrix_of(x, dtype, tokens, dim, ld_x, "x"), array_of(row, tokens * k * 4, "row")})))
        return rc;
    MoveArgs a{};
    a.dtype = dtype;
    a.tokens = tokens;
    a.dim = dim;
    a.rows = rows;
    a.k = k;
    a.row = row;
    a.x = x;
    a.ld_x = ld_x;
    a.y = y;
    a.ld_y = ld_y;
    const hipError_t e = launch_expert_gather((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "expert gather");
}

int scape_expert_combine(const void* y, int32_t dtype, int64_t rows, int64_t dim, int64_t ld_y, const int32_t* row,
                         const float* weight, int64_t tokens, int32_t k, void* out, int64_t ld_out, void* stream) {
    int rc;
    if ((rc = check_moves(dtype, tokens, dim, rows, k, row))) return rc;
    if ((rc = check_matrix(y, dtype, rows, dim, ld_y, "y"))) return rc;
    if ((rc = check_matrix(out, dtype, tokens, dim, ld_out, "out"))) return rc;
    if ((rc = check_optional(weight, "weight"))) return rc;
    if (tokens == 0) return SCAPE_OK;
    if ((rc = check_apart(matrix_of(out, dtype, tokens, dim, ld_out, "out"),
                          {matrix_of(y, dtype, rows, dim, ld_y, "y"), array_of(row, tokens * k * 4, "row"),
                           array_of(weight, tokens * k * 4, "weight")})))
        return rc;
    MoveArgs a{};
    a.dtype = dtype;
    a.tokens = tokens;
    a.dim = dim;
    a.rows = rows;
    a.k = k;
    a.row = row;
    a.weight = weight;
    a.y = const_cast<void*>(y);  // read only in this launch
    a.ld_y = ld_y;
    a.out = out;
    a.ld_out = ld_out;
    const hipError_t e = launch_expert_combine((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "expert combine");
}

int scape_expert_combine_backward(const void* y, int32_t dtype, int64_t rows, int64_t dim, int64_t ld_y,
                                  const int32_t* row, const float* weight, const void* dout, int64_t ld_dout,
                                  int64_t tokens, int32_t k, void* dy, int64_t ld_dy, float* dweight, void* stream) {
    int rc;
    if ((rc = check_moves(dtype, tokens, dim, rows, k, row))) return rc;
    if (dweight && (rc = check_matrix(y, dtype, rows, dim, ld_y, "y"))) return rc;
    if ((rc = check_matrix(dout, dtype, tokens, dim, ld_dout, "dout"))) return rc;
    if (dy && (rc = check_matrix(dy, dtype, rows, dim, ld_dy, "dy"))) return rc;
    if (dy && dy == y && ld_dy != ld_y) return fail(SCAPE_ERR_SHAPE, "dy over y needs y's row distance");
    if ((rc = check_optional(weight, "weight"))) return rc;
    if ((rc = check_optional(dweight, "dweight"))) return rc;
    if (tokens == 0 || (!dy && !dweight)) return SCAPE_OK;
    const Extent from = matrix_of(dweight ? y : nullptr, dtype, rows, dim, ld_y, "y");  // else it is not read
    const Extent from_out = matrix_of(dout, dtype, tokens, dim, ld_dout, "dout"), places = array_of(row, tokens * k * 4, "row");
    const Extent gates = array_of(weight, tokens * k * 4, "weight"), to_gates = array_of(dweight, tokens * k * 4, "dweight");
    const Extent to = matrix_of(dy, dtype, rows, dim, ld_dy, "dy");
    if (dy != y && (rc = check_apart(to, {from}))) return rc;
    if ((rc = check_apart(to, {from_out, places, gates, to_gates}))) return rc;
    if ((rc = check_apart(to_gates, {from, from_out, places, gates}))) return rc;
    MoveArgs a{};
    a.dtype = dtype;
    a.tokens = tokens;
    a.dim = dim;
    a.rows = rows;
    a.k = k;
    a.row = row;
    a.weight = weight;
    a.x = dout;
    a.ld_x = ld_dout;
    a.y = dy;
    a.ld_y = ld_dy;
    a.y_in = y;
    a.ld_y_in = ld_y;
    a.dweight = dweight;
    const hipError_t e = launch_expert_combine_back((hipStream_t)stream, a);
    return e == hipSuccess ? SCAPE_OK : hip_fail(e, "expert combine gradient");
}

}  // extern "C"
