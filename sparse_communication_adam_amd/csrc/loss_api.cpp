// loss_api.cpp - host side of the loss operators of include/scape.h: row
// top-k, distillation from a teacher's top logits, router balance loss.
// Arguments are validated here, before anything is launched; the operators
// hold no state and allocate nothing.
#include "loss_internal.h"

#include <cmath>

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

}  // extern "C"
