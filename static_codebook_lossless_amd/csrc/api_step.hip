// C-ABI entry points of the norm, dropout and log-probability operators:
// argument checks and HIP error mapping.  The kernels live in norm.hip,
// dropout.hip and logprob.hip.
#include "checks.h"

using namespace pc::checks;

namespace {

constexpr size_t kMaxPicked = 64;  // tokens and alternatives of a row: a lane each

bool mask_ok(const pc_mask *m) {
    return m->p >= 0.0 && m->p <= 1.0 && aligned(m->d_random, 8);
}

// The sum has x's type, or 32 bits.
bool sum_type_ok(int dtype, int sum_dtype) { return is_dtype(dtype) && (sum_dtype == dtype || sum_dtype == PC_F32); }

bool in_place_ok(const void *a, size_t lda, int ta, const void *b, size_t ldb, int tb) {
    return a != b || (lda == ldb && ta == tb);
}

bool scale_ok(float s) { return s >= 0x1p-64f && s <= 0x1p64f; }

bool tokens_ok(const void *tokens, int token_bytes, size_t n) {
    if (token_bytes != 4 && token_bytes != 8) return false;
    return n == 0 || (tokens && aligned(tokens, token_bytes));
}

// Rows of logits: the launches count them, and their stretches, in 32 bits.
bool logits_size_ok(uint64_t rows, uint64_t vocab) {
    return size_ok(rows, vocab) && rows * ((vocab + 1023) / 1024) < (1ull << 31);
}

}  // namespace

extern "C" {

pc_status pc_dropout(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, const pc_mask *mask,
                     void *d_out, size_t ld_out, void *stream) {
    if (!is_dtype(dtype) || !mask || !mask_ok(mask)) return PC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PC_OK;
    if (!plain_ok(d_x, dtype, cols, ldx) || !plain_ok(d_out, dtype, cols, ld_out)) return PC_ERR_INVALID_ARG;
    if (!in_place_ok(d_x, ldx, 0, d_out, ld_out, 0)) return PC_ERR_INVALID_ARG;
    if (!size_ok(rows, cols) || !span_ok(rows, ldx) || !span_ok(rows, ld_out)) return PC_ERR_UNSUPPORTED;
    return map_hip(pc::launch_dropout(d_x, dtype, rows, cols, ldx, mask, d_out, ld_out,
                                      static_cast<hipStream_t>(stream)));
}

pc_status pc_rmsnorm_store(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, const void *d_res,
                           int sum_dtype, size_t ld_res, const pc_mask *mask, const void *d_weight, int weight_dtype,
                           float eps, void *d_sum, size_t ld_sum, int format, uint8_t *d_sym, uint8_t *d_scale,
                           uint64_t *d_counts, void *d_y, int y_dtype, size_t ld_y, int y_stored, float *d_rstd,
                           void *stream) {
    if (!sum_type_ok(dtype, sum_dtype) || (d_weight && !is_dtype(weight_dtype)) || (d_y && !is_dtype(y_dtype)))
        return PC_ERR_INVALID_ARG;
    if (!d_res && sum_dtype != dtype) return PC_ERR_INVALID_ARG;
    if (mask && !mask_ok(mask)) return PC_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || eps > 3.402823466e38f) return PC_ERR_INVALID_ARG;
    if ((d_sym != nullptr) != (d_scale != nullptr) || (d_sym && !is_format(format))) return PC_ERR_INVALID_ARG;
    if ((d_counts || (d_y && y_stored)) && !d_sym) return PC_ERR_INVALID_ARG;
    if (d_sum && !d_res && !mask) return PC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PC_OK;
    if (!plain_ok(d_x, dtype, cols, ldx) || (d_res && !plain_ok(d_res, sum_dtype, cols, ld_res)) ||
        (d_weight && !plain_ok(d_weight, weight_dtype, cols, cols)) ||
        (d_sum && !plain_ok(d_sum, sum_dtype, cols, ld_sum)) || (d_y && !plain_ok(d_y, y_dtype, cols, ld_y)))
        return PC_ERR_INVALID_ARG;
    if (!aligned(d_counts, 8) || !aligned(d_rstd, 4)) return PC_ERR_INVALID_ARG;
    if (d_sum && (!in_place_ok(d_sum, ld_sum, sum_dtype, d_x, ldx, dtype) ||
                  !in_place_ok(d_sum, ld_sum, sum_dtype, d_res, ld_res, sum_dtype)))
        return PC_ERR_INVALID_ARG;
    if (d_y && (!in_place_ok(d_y, ld_y, y_dtype, d_x, ldx, dtype) ||
                !in_place_ok(d_y, ld_y, y_dtype, d_res, ld_res, sum_dtype) || d_y == d_sum))
        return PC_ERR_INVALID_ARG;
    const void *others[] = {d_x, d_res, d_weight, d_sum, d_y, d_counts};
    for (const void *p : others)
        if (p && (p == d_sym || p == d_scale || p == d_rstd)) return PC_ERR_INVALID_ARG;
    if ((d_weight && (d_weight == d_sum || d_weight == d_y)) || (d_sym && (d_sym == d_scale || d_sym == (void *)d_rstd)) ||
        (d_scale && d_scale == (void *)d_rstd))
        return PC_ERR_INVALID_ARG;
    if (!size_ok(rows, cols) || !span_ok(rows, ldx) || (d_res && !span_ok(rows, ld_res)) ||
        (d_sum && !span_ok(rows, ld_sum)) || (d_y && !span_ok(rows, ld_y)))
        return PC_ERR_UNSUPPORTED;
    pc::RmsNorm c = {};
    c.x = d_x;
    c.res = d_res;
    c.weight = d_weight;
    c.sum = d_sum;
    c.y = d_y;
    c.sym = d_sym;
    c.scale = d_scale;
    c.counts = d_counts;
    c.rstd = d_rstd;
    c.mask = mask;
    c.rows = rows;
    c.cols = cols;
    c.ldx = ldx;
    c.ld_res = ld_res;
    c.ld_sum = ld_sum;
    c.ld_y = ld_y;
    c.dtype = dtype;
    c.sum_dtype = sum_dtype;
    c.weight_dtype = weight_dtype;
    c.y_dtype = y_dtype;
    c.format = format;
    c.y_stored = y_stored != 0;
    c.eps = eps;
    return map_hip(pc::launch_rmsnorm_store(c, static_cast<hipStream_t>(stream)));
}

size_t pc_rmsnorm_backward_workspace_bytes(size_t rows, size_t cols) {
    if (rows == 0 || cols == 0 || !size_ok(rows, cols)) return 0;
    return pc::rmsnorm_backward_workspace(rows, cols);
}

pc_status pc_rmsnorm_backward(const void *d_dy, int dtype, size_t rows, size_t cols, size_t ld_dy, const void *d_sum,
                              int sum_dtype, size_t ld_sum, const pc_q8 *stored_sum, const void *d_weight,
                              int weight_dtype, const float *d_rstd, const void *d_dsum, size_t ld_dsum,
                              const pc_mask *mask, void *d_dres, size_t ld_dres, void *d_dx, size_t ld_dx,
                              void *d_dweight, int dweight_dtype, int accumulate, void *d_ws, size_t ws_bytes,
                              void *stream) {
    if (!sum_type_ok(dtype, sum_dtype) || (d_weight && !is_dtype(weight_dtype)) ||
        (d_dweight && !is_dtype(dweight_dtype)))
        return PC_ERR_INVALID_ARG;
    if (mask && !mask_ok(mask)) return PC_ERR_INVALID_ARG;
    if ((d_sum != nullptr) && stored_sum) return PC_ERR_INVALID_ARG;
    if (stored_sum && (stored_sum->rows != rows || stored_sum->cols != cols || !is_format(stored_sum->format)))
        return PC_ERR_INVALID_ARG;
    if (cols == 0 || (rows == 0 && (accumulate || !d_dweight))) return PC_OK;
    if (d_dweight && (d_dweight == d_weight || !plain_ok(d_dweight, dweight_dtype, cols, cols))) return PC_ERR_INVALID_ARG;
    if (rows) {
        if (!plain_ok(d_dy, dtype, cols, ld_dy) || (d_weight && !plain_ok(d_weight, weight_dtype, cols, cols)) ||
            !d_rstd || !aligned(d_rstd, 4))
            return PC_ERR_INVALID_ARG;
        if (stored_sum ? !stored_ok(stored_sum) : !plain_ok(d_sum, sum_dtype, cols, ld_sum))
            return PC_ERR_INVALID_ARG;
        if ((d_dsum && !plain_ok(d_dsum, sum_dtype, cols, ld_dsum)) ||
            (d_dres && !plain_ok(d_dres, sum_dtype, cols, ld_dres)) ||
            (d_dx && !plain_ok(d_dx, dtype, cols, ld_dx)))
            return PC_ERR_INVALID_ARG;
        // in the place of an input's row, element by element, or in none
        const struct { const void *p; size_t ld; int type; } rows_in[] = {
            {d_dy, ld_dy, dtype}, {d_sum, ld_sum, sum_dtype}, {d_dsum, ld_dsum, sum_dtype}};
        for (const auto &in : rows_in) {
            if ((d_dres && !in_place_ok(d_dres, ld_dres, sum_dtype, in.p, in.ld, in.type)) ||
                (d_dx && !in_place_ok(d_dx, ld_dx, dtype, in.p, in.ld, in.type)))
                return PC_ERR_INVALID_ARG;
            if (d_dweight && d_dweight == in.p) return PC_ERR_INVALID_ARG;
        }
        const void *others[] = {d_weight, d_rstd, stored_sum ? stored_sum->sym : nullptr,
                                stored_sum ? stored_sum->scale : nullptr};
        for (const void *in : others)
            if (in && (d_dres == in || d_dx == in || d_dweight == in)) return PC_ERR_INVALID_ARG;
        if (d_dweight && (d_dweight == d_dres || d_dweight == d_dx)) return PC_ERR_INVALID_ARG;
        if (d_dres && d_dres == d_dx && (mask || sum_dtype != dtype || ld_dres != ld_dx)) return PC_ERR_INVALID_ARG;
    }
    if (!size_ok(rows, cols) || !size_ok(1, cols) ||
        (rows && (!span_ok(rows, ld_dy) || (d_sum && !span_ok(rows, ld_sum)) ||
                  (stored_sum && (!span_ok(rows, stored_sum->ld_sym) || !span_ok(rows, stored_sum->ld_scale))) ||
                  (d_dsum && !span_ok(rows, ld_dsum)) || (d_dres && !span_ok(rows, ld_dres)) ||
                  (d_dx && !span_ok(rows, ld_dx)))))
        return PC_ERR_UNSUPPORTED;
    const size_t need = d_dweight ? pc_rmsnorm_backward_workspace_bytes(rows, cols) : 0;
    if (need) {
        if (!d_ws || !aligned(d_ws, 16)) return PC_ERR_INVALID_ARG;
        if (ws_bytes < need) return PC_ERR_CAPACITY;
    }
    pc::RmsNormGrad c = {};
    c.dy = d_dy;
    c.sum = d_sum;
    c.d_sum = d_dsum;
    c.weight = d_weight;
    c.stored = stored_sum;
    c.rstd = d_rstd;
    c.d_res = d_dres;
    c.d_x = d_dx;
    c.d_weight = d_dweight;
    c.ws = d_ws;
    c.mask = mask;
    c.rows = rows;
    c.cols = cols;
    c.ld_dy = ld_dy;
    c.ld_sum = ld_sum;
    c.ld_d_sum = ld_dsum;
    c.ld_d_res = ld_dres;
    c.ld_d_x = ld_dx;
    c.dtype = dtype;
    c.sum_dtype = sum_dtype;
    c.weight_dtype = weight_dtype;
    c.d_weight_dtype = dweight_dtype;
    c.accumulate = accumulate != 0;
    return map_hip(pc::launch_rmsnorm_backward(c, static_cast<hipStream_t>(stream)));
}

size_t pc_logprobs_workspace_bytes(size_t rows, size_t vocab, size_t top, int dtype) {
    if (rows == 0 || vocab == 0 || top > kMaxPicked || top > vocab || !is_dtype(dtype) || !logits_size_ok(rows, vocab))
        return 0;
    return pc::logprobs_workspace(rows, vocab, (uint32_t)top, dtype);
}

pc_status pc_logprobs(const void *d_logits, int dtype, size_t rows, size_t vocab, size_t ld, float scale,
                      const void *d_tokens, int token_bytes, size_t n_tokens, int64_t padding, float *d_logp,
                      size_t top, int64_t *d_top_index, float *d_top_logp, float *d_stats, uint32_t *d_status,
                      void *d_ws, size_t ws_bytes, void *stream) {
    if (!is_dtype(dtype) || !scale_ok(scale) || !tokens_ok(rows ? d_tokens : nullptr, token_bytes, rows ? n_tokens : 0))
        return PC_ERR_INVALID_ARG;
    if (rows == 0) return PC_OK;
    if (vocab == 0 || top > vocab || !plain_ok(d_logits, dtype, vocab, ld)) return PC_ERR_INVALID_ARG;
    if (n_tokens && (!d_logp || !aligned(d_logp, 4))) return PC_ERR_INVALID_ARG;
    if (top && (!d_top_index || !d_top_logp || !aligned(d_top_index, 8) || !aligned(d_top_logp, 4)))
        return PC_ERR_INVALID_ARG;
    if (!aligned(d_stats, 4) || !aligned(d_status, 4)) return PC_ERR_INVALID_ARG;
    if (n_tokens > kMaxPicked || top > kMaxPicked || !logits_size_ok(rows, vocab) || !span_ok(rows, ld))
        return PC_ERR_UNSUPPORTED;
    const size_t need = pc_logprobs_workspace_bytes(rows, vocab, top, dtype);
    if (need) {
        if (!d_ws || !aligned(d_ws, 16)) return PC_ERR_INVALID_ARG;
        if (ws_bytes < need) return PC_ERR_CAPACITY;
    }
    pc::LogProbs c = {};
    c.logits = d_logits;
    c.tokens = d_tokens;
    c.logp = d_logp;
    c.top_logp = d_top_logp;
    c.stats = d_stats;
    c.top_index = d_top_index;
    c.status = d_status;
    c.ws = d_ws;
    c.rows = rows;
    c.vocab = vocab;
    c.ld = ld;
    c.padding = padding;
    c.n_tokens = (uint32_t)n_tokens;
    c.top = (uint32_t)top;
    c.dtype = dtype;
    c.token_bytes = token_bytes;
    c.scale = scale;
    return map_hip(pc::launch_logprobs(c, static_cast<hipStream_t>(stream)));
}

pc_status pc_logprobs_backward(const void *d_logits, int dtype, size_t rows, size_t vocab, size_t ld, float scale,
                               const float *d_stats, const void *d_tokens, int token_bytes, size_t n_tokens,
                               int64_t padding, const float *d_dlogp, const float *d_dentropy, void *d_dlogits,
                               size_t ld_out, void *stream) {
    if (!is_dtype(dtype) || !scale_ok(scale) || !tokens_ok(rows ? d_tokens : nullptr, token_bytes, rows ? n_tokens : 0))
        return PC_ERR_INVALID_ARG;
    if (rows == 0) return PC_OK;
    if (vocab == 0 || !plain_ok(d_logits, dtype, vocab, ld) || !plain_ok(d_dlogits, dtype, vocab, ld_out))
        return PC_ERR_INVALID_ARG;
    if (!in_place_ok(d_logits, ld, 0, d_dlogits, ld_out, 0)) return PC_ERR_INVALID_ARG;
    if (!d_stats || !aligned(d_stats, 4) || !aligned(d_dlogp, 4) || !aligned(d_dentropy, 4)) return PC_ERR_INVALID_ARG;
    if (n_tokens && !d_dlogp) return PC_ERR_INVALID_ARG;
    if (d_dlogits == d_stats || (n_tokens && (d_dlogits == d_tokens || d_dlogits == d_dlogp)) || d_dlogits == d_dentropy)
        return PC_ERR_INVALID_ARG;
    if (n_tokens > kMaxPicked || !logits_size_ok(rows, vocab) || !span_ok(rows, ld) || !span_ok(rows, ld_out))
        return PC_ERR_UNSUPPORTED;
    pc::LogProbsGrad c = {};
    c.logits = d_logits;
    c.tokens = d_tokens;
    c.stats = d_stats;
    c.d_logp = d_dlogp;
    c.d_entropy = d_dentropy;
    c.d_logits = d_dlogits;
    c.rows = rows;
    c.vocab = vocab;
    c.ld = ld;
    c.ld_out = ld_out;
    c.padding = padding;
    c.n_tokens = (uint32_t)n_tokens;
    c.dtype = dtype;
    c.token_bytes = token_bytes;
    c.scale = scale;
    return map_hip(pc::launch_logprobs_backward(c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
