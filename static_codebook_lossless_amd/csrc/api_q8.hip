// C-ABI entry points of the stored-tensor and embedding operators: argument
// checks and HIP error mapping.  The kernels live in q8.hip, wgrad.hip and
// embed.hip.
#include "checks.h"

using namespace pc::checks;

extern "C" {

pc_status pc_q8_store(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, int format, uint8_t *d_sym,
                      uint8_t *d_scale, uint64_t *d_counts, void *stream) {
    if (!is_dtype(dtype) || !is_format(format)) return PC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PC_OK;
    if (!plain_ok(d_x, dtype, cols, ldx) || !d_sym || !d_scale) return PC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_counts) & 7) return PC_ERR_INVALID_ARG;
    if (!size_ok(rows, cols) || !span_ok(rows, ldx)) return PC_ERR_UNSUPPORTED;
    return map_hip(pc::launch_q8_store(d_x, dtype, rows, cols, ldx, format, d_sym, d_scale, d_counts,
                                       static_cast<hipStream_t>(stream)));
}

pc_status pc_q8_load(const pc_q8 *q, void *d_out, int dtype, size_t ld_out, void *stream) {
    if (!q || !is_dtype(dtype) || !is_format(q->format)) return PC_ERR_INVALID_ARG;
    if (q->rows == 0 || q->cols == 0) return PC_OK;
    if (!stored_ok(q) || !plain_ok(d_out, dtype, q->cols, ld_out)) return PC_ERR_INVALID_ARG;
    if (!size_ok(q->rows, q->cols) || !span_ok(q->rows, ld_out) || !span_ok(q->rows, q->ld_sym) ||
        !span_ok(q->rows, q->ld_scale))
        return PC_ERR_UNSUPPORTED;
    return map_hip(pc::launch_q8_load(q, d_out, dtype, ld_out, static_cast<hipStream_t>(stream)));
}

pc_status pc_q8_glu_backward(const void *d_dh, int dtype, size_t ld_dh, const pc_q8 *gate, const pc_q8 *up,
                             int activation, void *d_gate, size_t ld_gate, void *d_up, size_t ld_up, void *d_h,
                             size_t ld_h, void *stream) {
    if (!gate || !is_dtype(dtype) || !is_format(gate->format)) return PC_ERR_INVALID_ARG;
    if (activation < PC_ACT_SILU || activation > PC_ACT_GELU_TANH) return PC_ERR_INVALID_ARG;
    const size_t rows = gate->rows, cols = gate->cols;
    if (up && (up->rows != rows || up->cols != cols || up->format != gate->format)) return PC_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return PC_OK;
    if (!plain_ok(d_dh, dtype, cols, ld_dh) || !stored_ok(gate) || !plain_ok(d_gate, dtype, cols, ld_gate))
        return PC_ERR_INVALID_ARG;
    if ((up != nullptr) != (d_up != nullptr)) return PC_ERR_INVALID_ARG;
    if (up && (!stored_ok(up) || !plain_ok(d_up, dtype, cols, ld_up))) return PC_ERR_INVALID_ARG;
    if (d_h && !plain_ok(d_h, dtype, cols, ld_h)) return PC_ERR_INVALID_ARG;
    if (d_gate == d_dh && ld_gate != ld_dh) return PC_ERR_INVALID_ARG;
    if (!size_ok(rows, cols) || !span_ok(rows, ld_dh) || !span_ok(rows, ld_gate) || !span_ok(rows, gate->ld_sym) ||
        !span_ok(rows, gate->ld_scale) || (d_h && !span_ok(rows, ld_h)) ||
        (up && (!span_ok(rows, ld_up) || !span_ok(rows, up->ld_sym) || !span_ok(rows, up->ld_scale))))
        return PC_ERR_UNSUPPORTED;
    return map_hip(pc::launch_q8_glu_backward(d_dh, dtype, ld_dh, gate, up, activation, d_gate, ld_gate, d_up, ld_up,
                                              d_h, ld_h, static_cast<hipStream_t>(stream)));
}

size_t pc_q8_weight_grad_workspace_bytes(size_t rows, size_t n_out, size_t n_in, int dy_dtype) {
    if (!is_dtype(dy_dtype) || rows == 0 || n_out == 0 || n_in == 0 || !size_ok(n_out, n_in) ||
        !size_ok(rows, n_out) || !size_ok(rows, n_in))
        return 0;
    return pc::wgrad_workspace(rows, n_out, n_in, dy_dtype);
}

pc_status pc_q8_weight_grad(const void *d_dy, int dy_dtype, size_t ld_dy, size_t n_out, const pc_q8 *x, void *d_dw,
                            int dw_dtype, size_t ld_dw, int accumulate, void *d_ws, size_t ws_bytes, void *stream) {
    if (!x || !is_dtype(dy_dtype) || !is_dtype(dw_dtype) || !is_format(x->format)) return PC_ERR_INVALID_ARG;
    const size_t rows = x->rows, n_in = x->cols;
    if (n_out == 0 || n_in == 0 || (rows == 0 && accumulate)) return PC_OK;
    if (!plain_ok(d_dw, dw_dtype, n_in, ld_dw)) return PC_ERR_INVALID_ARG;
    if (rows && (!plain_ok(d_dy, dy_dtype, n_out, ld_dy) || !stored_ok(x))) return PC_ERR_INVALID_ARG;
    if (!size_ok(n_out, n_in) || !size_ok(rows, n_out) || !size_ok(rows, n_in) || !span_ok(n_out, ld_dw) ||
        !pc::wgrad_fits(rows, n_out, n_in, dy_dtype) ||
        (rows && (!span_ok(rows, ld_dy) || !span_ok(rows, x->ld_sym) || !span_ok(rows, x->ld_scale))))
        return PC_ERR_UNSUPPORTED;
    if (rows && (ld_dy >= kMaxDistance || x->ld_sym >= kMaxDistance || x->ld_scale >= kMaxDistance))
        return PC_ERR_UNSUPPORTED;
    const size_t need = pc_q8_weight_grad_workspace_bytes(rows, n_out, n_in, dy_dtype);
    if (need) {
        if (!d_ws || (reinterpret_cast<uintptr_t>(d_ws) & 15)) return PC_ERR_INVALID_ARG;
        if (ws_bytes < need) return PC_ERR_CAPACITY;
    }
    return map_hip(pc::launch_q8_weight_grad(d_dy, dy_dtype, ld_dy, n_out, x, d_dw, dw_dtype, ld_dw, accumulate != 0,
                                             d_ws, static_cast<hipStream_t>(stream)));
}

static pc_status embed_checked(const void *d_tokens, int token_bytes, size_t n, const void *d_table,
                               const uint8_t *codes, int kind, size_t vocab, size_t dim, size_t ld_table,
                               size_t ld_codes, float scale, void *d_out, int out_dtype, size_t ld_out,
                               uint32_t *d_status, void *stream) {
    if ((token_bytes != 4 && token_bytes != 8) || !is_dtype(out_dtype)) return PC_ERR_INVALID_ARG;
    if (n == 0 || dim == 0) return PC_OK;
    if (!d_tokens || (reinterpret_cast<uintptr_t>(d_tokens) & (token_bytes - 1))) return PC_ERR_INVALID_ARG;
    if (!plain_ok(d_out, out_dtype, dim, ld_out)) return PC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(d_status) & 3) return PC_ERR_INVALID_ARG;
    if (!size_ok(n, dim) || !span_ok(n, ld_out) || !span_ok(vocab, ld_table) || !span_ok(vocab, ld_codes))
        return PC_ERR_UNSUPPORTED;
    return map_hip(pc::launch_embed(d_tokens, token_bytes, n, d_table, codes, kind, vocab, dim, ld_table, ld_codes,
                                    scale, d_out, out_dtype, ld_out, d_status, static_cast<hipStream_t>(stream)));
}

pc_status pc_embed(const void *d_tokens, int token_bytes, size_t n, const void *d_table, int table_dtype,
                   size_t vocab, size_t dim, size_t ld_table, float scale, void *d_out, int out_dtype, size_t ld_out,
                   uint32_t *d_status, void *stream) {
    if (!is_dtype(table_dtype)) return PC_ERR_INVALID_ARG;
    if (n && dim && vocab && !plain_ok(d_table, table_dtype, dim, ld_table)) return PC_ERR_INVALID_ARG;
    return embed_checked(d_tokens, token_bytes, n, d_table, nullptr, table_dtype, vocab, dim, ld_table, 0, scale,
                         d_out, out_dtype, ld_out, d_status, stream);
}

pc_status pc_embed_q8(const void *d_tokens, int token_bytes, size_t n, const pc_q8 *table, float scale, void *d_out,
                      int out_dtype, size_t ld_out, uint32_t *d_status, void *stream) {
    if (!table || !is_format(table->format)) return PC_ERR_INVALID_ARG;
    if (n && table->rows && table->cols && !stored_ok(table)) return PC_ERR_INVALID_ARG;
    return embed_checked(d_tokens, token_bytes, n, table->sym, table->scale, 4 + table->format, table->rows,
                         table->cols, table->ld_sym, table->ld_scale, scale, d_out, out_dtype, ld_out, d_status,
                         stream);
}

static bool embed_backward_size_ok(size_t n, size_t dim, size_t vocab) {
    return n < kMaxWidth && vocab <= kMaxWidth && size_ok(n, dim) && size_ok(vocab, dim) &&
           pc::embed_backward_fits(n, dim, vocab);
}

size_t pc_embed_backward_workspace_bytes(size_t n, size_t dim, size_t vocab) {
    if (dim == 0 || vocab == 0 || !embed_backward_size_ok(n, dim, vocab)) return 0;
    return pc::embed_backward_workspace(n, dim, vocab);
}

pc_status pc_embed_backward(const void *d_dy, int dy_dtype, size_t ld_dy, const void *d_tokens, int token_bytes,
                            size_t n, size_t dim, size_t vocab, int64_t padding, float scale, void *d_grad,
                            int grad_dtype, size_t ld_grad, int accumulate, void *d_ws, size_t ws_bytes,
                            void *stream) {
    if ((token_bytes != 4 && token_bytes != 8) || !is_dtype(dy_dtype) || !is_dtype(grad_dtype))
        return PC_ERR_INVALID_ARG;
    if (dim == 0 || vocab == 0 || (n == 0 && accumulate)) return PC_OK;
    if (!plain_ok(d_grad, grad_dtype, dim, ld_grad)) return PC_ERR_INVALID_ARG;
    if (n && (!plain_ok(d_dy, dy_dtype, dim, ld_dy) || !d_tokens ||
              (reinterpret_cast<uintptr_t>(d_tokens) & (token_bytes - 1))))
        return PC_ERR_INVALID_ARG;
    if (!embed_backward_size_ok(n, dim, vocab) || !span_ok(vocab, ld_grad) || (n && !span_ok(n, ld_dy)))
        return PC_ERR_UNSUPPORTED;
    const size_t need = pc_embed_backward_workspace_bytes(n, dim, vocab);
    if (need) {
        if (!d_ws || (reinterpret_cast<uintptr_t>(d_ws) & 15)) return PC_ERR_INVALID_ARG;
        if (ws_bytes < need) return PC_ERR_CAPACITY;
    }
    return map_hip(pc::launch_embed_backward(d_dy, dy_dtype, ld_dy, d_tokens, token_bytes, (uint32_t)n, dim, vocab,
                                             padding, scale, d_grad, grad_dtype, ld_grad, accumulate != 0, d_ws,
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
