// Internal declarations of libpc.so (device helpers and kernel launchers).
// Target: CDNA4 (gfx950), wave64.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pc.h"

namespace pc {

constexpr uint32_t kWave = 64;
constexpr uint32_t kSub = PC_SUBSTREAM;  // symbols per decode sub-stream
constexpr uint32_t kPeek = PC_MAX_LEN;   // bits looked at per codeword
constexpr size_t kMaxChunk = (size_t)1 << 24;
// decode: sub-stream indices, and an index plus 256, stay below 2^32
constexpr uint64_t kMaxDecodeSubstreams = 0xFFFFFF00ull;

// Byte offsets inside pc_codebook (checked by static_asserts in codebook.cpp).
constexpr uint32_t kOffLength = 32;
constexpr uint32_t kOffCode = 288;
constexpr uint32_t kOffDecSym = 800;
constexpr uint32_t kOffQlcBits = 8992;
constexpr uint32_t kOffQlcStart = 9000;
constexpr uint32_t kOffSymOfRank = 9272;

// ---------------------------------------------------------------------------
// wave64 helpers
// ---------------------------------------------------------------------------

template <int CTRL, int ROW_MASK = 0xF>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    // Lanes whose DPP source is outside the pattern (or whose row is masked
    // off) receive 0.
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false);
}

// Inclusive prefix sum over the 64 lanes of a wave (row shifts inside rows
// of 16, then the row broadcasts of lane 15 and lane 31).
__device__ __forceinline__ uint32_t wave_incl_scan(uint32_t v) {
    v += dpp_u32<0x111>(v);        // row_shr:1
    v += dpp_u32<0x112>(v);        // row_shr:2
    v += dpp_u32<0x114>(v);        // row_shr:4
    v += dpp_u32<0x118>(v);        // row_shr:8
    v += dpp_u32<0x142, 0xA>(v);   // row_bcast:15 -> rows 1 and 3
    v += dpp_u32<0x143, 0xC>(v);   // row_bcast:31 -> rows 2 and 3
    return v;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

__device__ __forceinline__ uint64_t wave_min_u64(uint64_t v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        uint64_t o = __shfl_xor(v, m, 64);
        v = o < v ? o : v;
    }
    return v;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) {
        uint64_t o = __shfl_xor(v, m, 64);
        v = o > v ? o : v;
    }
    return v;
}

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 16-byte load of data read once (non-temporal: not kept in the caches).
__device__ __forceinline__ uint4 load_stream16(const void *p) {
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint32_t uniform(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    uint32_t lo = uniform((uint32_t)v), hi = uniform((uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}

// ---------------------------------------------------------------------------
// Launchers (defined in the .hip files, called from api.hip).
// ---------------------------------------------------------------------------

// max_polls: polls of the cross-chunk scan's bounded wait before it gives up
// and writes PC_ERR_TIMEOUT to *status (which the launch first zeroes).
constexpr uint32_t kDefaultWaitPolls = 1u << 20;

hipError_t launch_encode(const pc_codebook *cb, const uint8_t *in, uint64_t n, uint32_t chunk,
                         uint32_t *payload, uint32_t *chunk_bits, uint64_t *cwo, uint32_t *sub_off,
                         uint64_t *ws, uint32_t *status, uint32_t max_polls, hipStream_t stream);

enum DecodeMode { kDecodeLut12 = 0, kDecodeQlc = 1 };

hipError_t launch_decode(int mode, const pc_codebook *cb, const uint32_t *payload, uint64_t payload_words,
                         const uint32_t *chunk_bits, const uint64_t *cwo, const uint32_t *sub_off,
                         uint64_t n, uint32_t chunk, uint8_t *out, uint32_t *status, hipStream_t stream);

hipError_t launch_histogram(const uint8_t *in, uint64_t n, uint64_t *counts, hipStream_t stream);

hipError_t launch_q8_store(const void *x, int dtype, uint64_t rows, uint64_t cols, uint64_t ldx, int format,
                           uint8_t *sym, uint8_t *scale, uint64_t *counts, hipStream_t stream);

hipError_t launch_q8_load(const pc_q8 *q, void *out, int dtype, uint64_t ld_out, hipStream_t stream);

hipError_t launch_q8_glu_backward(const void *dh, int dtype, uint64_t ld_dh, const pc_q8 *gate, const pc_q8 *up,
                                  int act, void *d_gate, uint64_t ld_gate, void *d_up, uint64_t ld_up, void *h,
                                  uint64_t ld_h, hipStream_t stream);

bool wgrad_fits(uint64_t t, uint64_t n, uint64_t k, int dy_dtype);
uint64_t wgrad_workspace(uint64_t t, uint64_t n, uint64_t k, int dy_dtype);
hipError_t launch_q8_weight_grad(const void *dy, int dtype, uint64_t ld_dy, uint64_t n_out, const pc_q8 *x, void *dw,
                                 int dw_dtype, uint64_t ld_dw, bool accumulate, void *ws, hipStream_t stream);

// kind: a pc_dtype, or 4 + a pc_q8_format for a stored table (then with codes).
hipError_t launch_embed(const void *tokens, int token_bytes, uint64_t n, const void *table, const uint8_t *codes,
                        int kind, uint64_t vocab, uint64_t dim, uint64_t ld_table, uint64_t ld_codes, float scale,
                        void *out, int out_dtype, uint64_t ld_out, uint32_t *status, hipStream_t stream);

// Whether the launches of this size are possible.
bool embed_backward_fits(uint64_t n, uint64_t dim, uint64_t vocab);
uint64_t embed_backward_workspace(uint64_t n, uint64_t dim, uint64_t vocab);
hipError_t launch_embed_backward(const void *dy, int dtype, uint64_t ld_dy, const void *tokens, int token_bytes,
                                 uint32_t n, uint64_t dim, uint64_t vocab, int64_t padding, float scale, void *grad,
                                 int grad_dtype, uint64_t ld_grad, bool accumulate, void *ws, hipStream_t stream);

// Arguments of the norm's entries; dtypes are pc_dtypes, NULL what is not wanted.
struct RmsNorm {
    const void *x, *res, *weight;
    void *sum, *y;
    uint8_t *sym, *scale;
    uint64_t *counts;
    float *rstd;
    const pc_mask *mask;
    uint64_t rows, cols, ldx, ld_res, ld_sum, ld_y;
    int dtype, sum_dtype, weight_dtype, y_dtype, format, y_stored;
    float eps;
};
hipError_t launch_rmsnorm_store(const RmsNorm &c, hipStream_t stream);

struct RmsNormGrad {
    const void *dy, *sum, *d_sum, *weight;
    const pc_q8 *stored;  // in place of sum
    const float *rstd;
    void *d_res, *d_x, *d_weight, *ws;
    const pc_mask *mask;
    uint64_t rows, cols, ld_dy, ld_sum, ld_d_sum, ld_d_res, ld_d_x;
    int dtype, sum_dtype, weight_dtype, d_weight_dtype, accumulate;
};
uint64_t rmsnorm_backward_workspace(uint64_t rows, uint64_t cols);
hipError_t launch_rmsnorm_backward(const RmsNormGrad &c, hipStream_t stream);

hipError_t launch_dropout(const void *x, int dtype, uint64_t rows, uint64_t cols, uint64_t ldx, const pc_mask *mask,
                          void *out, uint64_t ld_out, hipStream_t stream);

struct LogProbs {
    const void *logits, *tokens;
    float *logp, *top_logp, *stats;
    int64_t *top_index;
    uint32_t *status;
    void *ws;
    uint64_t rows, vocab, ld;
    int64_t padding;
    uint32_t n_tokens, top;
    int dtype, token_bytes;
    float scale;
};
uint64_t logprobs_workspace(uint64_t rows, uint64_t vocab, uint32_t top, int dtype);
hipError_t launch_logprobs(const LogProbs &c, hipStream_t stream);

struct LogProbsGrad {
    const void *logits, *tokens;
    const float *stats, *d_logp, *d_entropy;
    void *d_logits;
    uint64_t rows, vocab, ld, ld_out;
    int64_t padding;
    uint32_t n_tokens;
    int dtype, token_bytes;
    float scale;
};
hipError_t launch_logprobs_backward(const LogProbsGrad &c, hipStream_t stream);

}  // namespace pc
