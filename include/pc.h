/*
 * pc.h -- fixed-codebook ("single-stage") prefix coding of 8-bit tensors on
 * AMD Instinct MI355X (gfx950).  C ABI of libpc.so.
 *
 * Method
 *   "Single-Stage Huffman Encoder for ML Compression" (abstract): a Huffman
 *   code is normally built per message (frequency analysis, codebook
 *   generation, codebook sent with the data).  The single-stage encoder
 *   instead uses one fixed codebook derived from the average distribution of
 *   previous batches, so the run-time work is only the symbol-to-codeword
 *   mapping and nothing but the codewords is transmitted.
 *   "Quad Length Codes for Lossless Compression of e4m3" (abstract, Tables 1
 *   and 2): the second codebook kind -- a 3-bit prefix names one of 8 areas,
 *   and area a carries a fixed-width b_a-bit index into the symbols ranked by
 *   descending probability (code length 3 + b_a).
 *
 * Alphabet 256 (one byte per symbol: e4m3 or int8).  Code lengths are 1..12
 * bits.  All integers are little-endian.
 *
 * Container (the pages define none; this is the library's format)
 *   - The input of n symbols is cut into chunks of `chunk` symbols (a
 *     multiple of 256, at most 2^24; the last chunk may be short).  Each chunk
 *     is an independent bitstream: its codewords concatenated, most
 *     significant bit first; stream bit j is bit (31 - j%32) of 32-bit word
 *     j/32; the chunk is zero-padded to a whole word.
 *   - payload: the chunks' words back to back; chunk c starts at word
 *     chunk_word_offset[c]; chunk_word_offset[num_chunks] is the total.
 *   - chunk_bits[c]: exact unpadded bit count of chunk c.
 *   - sub_off: for every chunk c and j = 0 .. ceil(len_c/256)-1, the bit
 *     offset (relative to chunk c's first bit) of the chunk's symbol 256*j.
 *     Flattened in chunk order; entry j = 0 is always 0.  This side index
 *     lets the decoder run one independent 256-symbol sub-stream per lane.
 *   Nothing of the codebook travels with the data: encoder and decoder must
 *   use the same pc_codebook (compare codebook_id).
 *
 * Errors
 *   Every entry point returns a pc_status synchronously for argument, size
 *   and launch errors.  Device entry points are asynchronous on `stream` (a
 *   hipStream_t; NULL is the default stream).  Data-dependent decode errors
 *   are reported through a device status word (see pc_decode).
 *
 * Stored tensors ("Q8") and the operators of a training step that use them
 *   The bytes the coder takes come from somewhere and go somewhere: the
 *   second half of this file stores a tensor of a training step as e4m3 or
 *   int8 symbols with one power-of-two scale for every 32 columns (the
 *   symbols are what pc_encode codes and pc_histogram counts), and uses the
 *   symbols, as pc_decode gives them back, in the backward pass and as an
 *   embedding table.  The last part has what stands between the products of
 *   such a step: the norm of a residual block, which stores its output, dropout
 *   from a counter, and the loss (log probabilities of given tokens, the
 *   entropy and the logits' gradient).
 *
 * Memory
 *   The library never allocates.  Every buffer belongs to the caller; device
 *   pointers must stay valid until the stream has executed the call.
 */
#ifndef PC_H
#define PC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PC_ALPHABET 256
#define PC_MAX_LEN 12
#define PC_SUBSTREAM 256
#define PC_QLC_AREAS 8
#define PC_CODEBOOK_MAGIC 0x31424350u /* "PCB1" */
#define PC_CODEBOOK_VERSION 1u

typedef enum pc_status {
    PC_OK = 0,
    PC_ERR_INVALID_ARG = 1, /* a pointer, size, alignment or enum is invalid */
    PC_ERR_UNSUPPORTED = 2, /* valid request the library cannot serve */
    PC_ERR_CAPACITY = 3,    /* an output or workspace buffer is too small */
    PC_ERR_CORRUPT = 4,     /* data do not form a valid container (decode) */
    PC_ERR_HIP = 5,         /* the HIP runtime reported an error */
    PC_ERR_TIMEOUT = 6      /* a bounded device wait gave up (encode); outputs invalid */
} pc_status;

typedef enum pc_codebook_kind {
    PC_CODEBOOK_HUFFMAN = 0, /* canonical, package-merge length-limited to 12 bits */
    PC_CODEBOOK_QLC = 1      /* Quad Length Code: 3-bit area + fixed-width index */
} pc_codebook_kind;

/*
 * The codebook: a flat, position-independent blob (9536 bytes).  Build it on
 * the host with pc_codebook_build, copy it to device memory once, and pass
 * the device copy to pc_encode / pc_decode.  Layout is fixed (offsets in
 * bytes): header 0, length 32, code 288, dec_sym 800, dec_len 4896,
 * qlc_bits 8992, qlc_start 9000, rank_of 9016, sym_of_rank 9272.
 */
typedef struct pc_codebook {
    uint32_t magic;          /* PC_CODEBOOK_MAGIC */
    uint32_t version;        /* PC_CODEBOOK_VERSION */
    uint32_t kind;           /* pc_codebook_kind */
    uint32_t max_len;        /* longest code length in use (<= 12) */
    uint32_t codebook_id;    /* FNV-1a 32 over kind (4 bytes), length[256], qlc_bits[8] */
    uint32_t complete;       /* 1 when the Kraft sum is exactly 1 */
    uint32_t reserved[2];
    uint8_t length[256];     /* code length of every byte value, 1..12 */
    uint16_t code[256];      /* code value, right-aligned (MSB first on the wire) */
    uint8_t dec_sym[4096];   /* 12-bit peek (next 12 stream bits) -> symbol */
    uint8_t dec_len[4096];   /* 12-bit peek -> code length; 0 = no codeword */
    uint8_t qlc_bits[8];     /* QLC: index width of each area (zeros for Huffman) */
    uint16_t qlc_start[8];   /* QLC: first rank of each area */
    uint8_t rank_of[256];    /* QLC: rank (descending count) of each byte value */
    uint8_t sym_of_rank[256];/* QLC: byte value of each rank */
    uint8_t pad[8];
} pc_codebook;

/* Human-readable name of a status code (static storage; library-defined). */
const char *pc_status_string(int status);

/*
 * Build a fixed codebook on the host.  Pure, deterministic, thread-safe.
 *
 * counts: the pooled histogram of previous batches ("Single-Stage Huffman
 *   Encoder for ML Compression", abstract: the average distribution of
 *   previous data batches; pooling equal-size batches by summing counts is
 *   proportional to averaging their PMFs).
 * kind = PC_CODEBOOK_HUFFMAN: weights max(count,1) (every byte stays
 *   codable), package-merge length-limited to 12 bits (on equal weight a leaf
 *   precedes a package; leaves ordered by (weight, byte value)), then
 *   canonical codes in (length, byte value) order.  qlc_bits must be NULL.
 * kind = PC_CODEBOOK_QLC: qlc_bits[a] (0..9) is the index width of area a
 *   ("Quad Length Codes for Lossless Compression of e4m3", Tables 1 and 2);
 *   the areas must cover 256 ranks (sum 2^b >= 256).  Ranks order bytes by descending count, equal counts
 *   by lower byte value; the byte of rank r in area a gets code
 *   (a << b_a) | (r - start_a) of length 3 + b_a.
 * Returns PC_ERR_INVALID_ARG for NULL pointers, an unknown kind, or bad
 * QLC widths; `out` is fully written on PC_OK.
 */
pc_status pc_codebook_build(const uint64_t counts[256], int kind, const uint8_t qlc_bits[8],
                            pc_codebook *out);

/*
 * Host check of a codebook blob (magic, version, lengths, tables).  The
 * pages define no codebook format ("Single-Stage Huffman Encoder for ML
 * Compression", abstract, only requires that encoder and decoder hold the
 * same precomputed codebook); this checks the library's own layout above.
 */
pc_status pc_codebook_validate(const pc_codebook *cb);

/*
 * Choose QLC area widths for a histogram: the 8 widths (each 0..9, areas
 * covering 256 ranks) that minimise sum(count * (3 + b_area(rank))) over the
 * ranked histogram, by dynamic programming over contiguous rank ranges --
 * "Quad Length Codes for Lossless Compression of e4m3" (abstract) notes
 * that the scheme adapts to the distribution.  Ties keep the
 * lexicographically smallest width vector.  Host only.
 */
pc_status pc_qlc_optimal_bits(const uint64_t counts[256], uint8_t bits_out[8]);

/*
 * How well a fixed codebook fits a batch (host, pure).  For the byte
 * histogram `counts` of the batch:
 *   *avg_bits = sum(count * length) / sum(count): the payload bits per
 *               symbol the codebook spends on that batch;
 *   *entropy  = the batch's Shannon entropy, -sum(p log2 p), in bits per
 *               symbol: the bound a code built for the batch itself
 *               approaches.
 * The single-stage codebook is built once from earlier batches ("Single-
 * Stage Huffman Encoder for ML Compression", abstract), so avg_bits -
 * entropy measures how far the batches have drifted from it; the Shannonic
 * page ("Shannonic: Efficient Entropy-Optimal Compression for ML
 * Workloads", key observation 1) expects static tables to be refreshed when
 * the distribution drifts.  A caller rebuilds (pc_codebook_build on the
 * pooled counts of recent batches) once the gap passes its threshold.
 * An all-zero histogram gives 0 and 0.  PC_ERR_INVALID_ARG for NULL
 * pointers or a blob that fails pc_codebook_validate.
 */
pc_status pc_codebook_fit(const pc_codebook *cb, const uint64_t counts[256], double *avg_bits, double *entropy);

/*
 * Code lengths of the per-shard comparator (host, pure).  "Single-Stage
 * Huffman Encoder for ML Compression" (abstract) measures the fixed codebook
 * against Huffman codes built for each shard from its own statistics (the
 * three-stage scheme: count, build, send the codebook).  This returns that
 * code for one shard's histogram: package-merge limited to 12 bits over the
 * byte values that occur (count > 0), with the same tie rules as
 * pc_codebook_build; an absent byte value gets length 0 (no codeword), a
 * histogram with one byte value gives it length 1, an all-zero histogram
 * gives all zeros.  Unlike pc_codebook_build, counts are not floored: a
 * shard's own code never has to code a byte it does not contain.
 *   lengths_out[256]   written in full on PC_OK.
 * PC_ERR_INVALID_ARG for NULL pointers.
 */
pc_status pc_shard_code_lengths(const uint64_t counts[256], uint8_t lengths_out[256]);

/*
 * Size queries (host, pure) of the container above, which is the library's
 * own (the pages define no container).  chunk must be a valid chunk size,
 * else 0.  The payload bound uses the 12-bit length limit (PC_MAX_LEN).
 */
size_t pc_num_chunks(size_t n, size_t chunk);          /* ceil(n / chunk) */
size_t pc_num_substreams(size_t n, size_t chunk);      /* sum over chunks of ceil(len_c / 256) */
size_t pc_max_payload_words(size_t n, size_t chunk);   /* sum over chunks of ceil(12 len_c / 32) */
size_t pc_encode_workspace_bytes(size_t n, size_t chunk);  /* 8 (1 + chunks), + 4 per 64 KiB of full
                                                          chunks for chunks of several 64 KiB (rounded up to 8) */

/*
 * Encode n symbols (device, asynchronous on `stream`): every byte becomes
 * its codeword from the fixed codebook and the codewords are concatenated
 * ("Single-Stage Huffman Encoder for ML Compression", abstract: symbol to
 * codeword mapping with one precomputed codebook; "Quad Length Codes for
 * Lossless Compression of e4m3", abstract, for the QLC codewords), chunk by
 * chunk into the container described above.
 *   d_cb       device copy of a pc_codebook.
 *   d_in       n input bytes, 16-byte aligned.
 *   chunk      symbols per chunk: multiple of 256, 256 <= chunk <= 2^24.
 *   d_payload  >= pc_max_payload_words(n, chunk) words (capacity is checked
 *              against that bound, so encoding can never overflow), 16-byte
 *              aligned.  Exactly chunk_word_offset[num_chunks] words are
 *              written.
 *   d_chunk_bits          [num_chunks] u32
 *   d_chunk_word_offset   [num_chunks + 1] u64 (exclusive prefix of words)
 *   d_sub_off             [pc_num_substreams(n, chunk)] u32
 *   d_ws, ws_bytes        scratch of at least pc_encode_workspace_bytes,
 *              8-byte aligned; its contents need no initialisation.
 *   d_status   one u32 in device memory (4-byte aligned).  The call first
 *              sets it to 0 on the stream, then to PC_ERR_TIMEOUT if the
 *              cross-chunk scan gave up waiting for an earlier workgroup's
 *              word count (see pc_encode_set_wait_limit); the outputs are
 *              then invalid.  Read it after the stream has executed the call.
 * n = 0 writes chunk_word_offset[0] = 0, *d_status = 0 and nothing else.
 * Calls that share a workspace must be ordered on one stream.  More than
 * 2^31 - 1 chunks: PC_ERR_UNSUPPORTED.
 */
pc_status pc_encode(const pc_codebook *d_cb, const uint8_t *d_in, size_t n, size_t chunk,
                    uint32_t *d_payload, size_t payload_capacity_words,
                    uint32_t *d_chunk_bits, uint64_t *d_chunk_word_offset, uint32_t *d_sub_off,
                    void *d_ws, size_t ws_bytes, uint32_t *d_status, void *stream);

/*
 * pc_encode for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same
 * arguments, outputs, status word and errors as pc_encode, without the
 * workspace: the cross-chunk scan's ticket and descriptors live in a static
 * device array of the library (8 MiB + 8 bytes per GPU, held until the
 * process ends), so the call allocates nothing.  At most 2^20 chunks per
 * call, and pc_encode_workspace_bytes(n, chunk) at most that array's size
 * (PC_ERR_CAPACITY beyond; it binds for chunks of several 64 KiB, which
 * keep one u32 per 64 KiB in the array).  Every call on one GPU shares that GPU's
 * array and clears it first on its stream: calls that overlap on one GPU
 * (several streams, or host threads) race and must be serialised by the
 * caller, e.g. by issuing them on one stream.
 */
pc_status pc_encode_noalloc(const pc_codebook *d_cb, const uint8_t *d_in, size_t n, size_t chunk,
                            uint32_t *d_payload, size_t payload_capacity_words,
                            uint32_t *d_chunk_bits, uint64_t *d_chunk_word_offset, uint32_t *d_sub_off,
                            uint32_t *d_status, void *stream);

/*
 * Bound of the encoder's one device-side wait (host, process-wide; returns
 * the previous bound).  The pages describe no GPU encoder; this library's
 * chunks learn their output offsets from a single-pass scan in which a
 * workgroup waits until the workgroups of all earlier chunks have published
 * their word counts.  Every wave of that wait polls at most `polls` times,
 * then gives up and reports PC_ERR_TIMEOUT through pc_encode's d_status
 * instead of waiting on.  The default (polls = 0 restores it) is 2^20 polls,
 * about a second: far beyond a correct run's wait, short enough that a
 * workgroup held up by other work on a time-sliced GPU ends in an error
 * rather than a hang.  Small limits make give-ups frequent (the tests use 1
 * to exercise the report); each call reads the bound when it is made.
 */
uint32_t pc_encode_set_wait_limit(uint32_t polls);

/*
 * Decode n symbols (device, asynchronous on `stream`) with the generic
 * engine: one lane per 256-symbol sub-stream, one 12-bit peek per codeword
 * through the dec_sym/dec_len tables held in LDS.  Works for both codebook
 * kinds.  The decoder holds the same fixed codebook as the encoder, so no
 * table travels with the data ("Single-Stage Huffman Encoder for ML
 * Compression", abstract); one table lookup per codeword instead of a
 * bit-by-bit tree walk is the decoding-speed concern of "Quad Length Codes
 * for Lossless Compression of e4m3" (abstract).
 *   d_payload, payload_words   the payload (16-byte aligned) and its length;
 *              no word at or past payload_words is ever read.
 *   d_chunk_bits, d_chunk_word_offset, d_sub_off   as written by pc_encode.
 *   d_out      n output bytes, 16-byte aligned; nothing outside [0, n) is
 *              written.
 *   d_status   one u32 in device memory.  The caller zeroes it before the
 *              call; the decoder sets it to PC_ERR_CORRUPT when the
 *              container is inconsistent (chunk_word_offset steps that differ
 *              from ceil(chunk_bits/32) or run past payload_words, a chunk
 *              whose first sub-stream does not start at bit 0, a bit pattern
 *              that is no codeword, or a sub-stream that does not end exactly
 *              where the next one starts / at chunk_bits).  On such an error
 *              d_out holds unspecified bytes.
 * 2^32 - 256 or more sub-streams (n of about 2^40 and up, past one GPU's
 * memory): PC_ERR_UNSUPPORTED.
 */
pc_status pc_decode(const pc_codebook *d_cb, const uint32_t *d_payload, size_t payload_words,
                    const uint32_t *d_chunk_bits, const uint64_t *d_chunk_word_offset,
                    const uint32_t *d_sub_off, size_t n, size_t chunk, uint8_t *d_out,
                    uint32_t *d_status, void *stream);

/*
 * Decode a QLC-coded stream the way "Quad Length Codes for Lossless
 * Compression of e4m3" (abstract) describes its decoder: read the 3-bit
 * area number, read that area's fixed-width index, map the rank to the
 * symbol through the 256-entry table.  Same arguments, container
 * and error rules as pc_decode; d_cb must be a PC_CODEBOOK_QLC codebook
 * (PC_ERR_CORRUPT in *d_status otherwise).
 */
pc_status pc_decode_qlc(const pc_codebook *d_cb, const uint32_t *d_payload, size_t payload_words,
                        const uint32_t *d_chunk_bits, const uint64_t *d_chunk_word_offset,
                        const uint32_t *d_sub_off, size_t n, size_t chunk, uint8_t *d_out,
                        uint32_t *d_status, void *stream);

/*
 * Byte histogram on the device: d_counts[s] += number of bytes equal to s in
 * d_in[0, n).  Accumulates, so pooling previous batches is repeated calls on
 * the same d_counts (256 u64, 8-byte aligned).  d_in needs no alignment.
 * The pooled histogram of previous batches is what the fixed codebook is
 * built from ("Single-Stage Huffman Encoder for ML Compression", abstract:
 * the average distribution of previous data batches).
 */
pc_status pc_histogram(const uint8_t *d_in, size_t n, uint64_t *d_counts, void *stream);

/*
 * Measurement helper, not part of the coding method: copies `bytes` bytes
 * from d_src to d_dst with the 16-byte non-temporal loads and stores the
 * coder kernels use, so that the HBM bytes hardware counters report for this
 * known transfer (read `bytes`, write `bytes`) can calibrate the counts
 * taken on the coder kernels.  Both pointers 16-byte aligned device memory,
 * bytes a multiple of 16 (PC_ERR_INVALID_ARG otherwise); asynchronous on
 * `stream`; bytes == 0 does nothing.
 */
pc_status pc_traffic_probe(const void *d_src, void *d_dst, size_t bytes, void *stream);

/* ------------------------------------------------------------------------
 * Tensors stored in 8 bits, and the operators that use them
 *
 * A stored tensor ("Q8") of rows x cols elements is
 *   sym    one byte per element, rows of cols bytes; row r starts at
 *          sym + r * ld_sym.  Dense (ld_sym == cols) it is the byte string
 *          that pc_encode takes.
 *   scale  one code per group of 32 columns (the last group of a row may be
 *          short); row r starts at scale + r * ld_scale.
 * The element in row r and column c stands for
 *          element(sym[r][c]) * 2^(scale[r][c / 32] - 127),
 * element() being OCP E4M3FN or int8 two's complement.  A byte that stands
 * for no number (0x7F and 0xFF in e4m3, 0x80 in int8) reads as NaN.  Powers
 * of two keep stored values exact in bf16 and f32, so the matrix instructions
 * multiply them without rounding them again.  Scale codes run from 1 to 254;
 * pc_q8_store writes 10 to 249, under which only 2^128 and more, as infinity,
 * leaves the range of bf16 and f32.
 *
 * Tensors of plain numbers are f32, f16 or bf16, rows of unit stride and a
 * row distance `ld` in elements that may exceed the width; pointers need the
 * alignment of their element only.  All arithmetic is in 32 bits, rounded
 * once to the output's type.  Inputs and outputs must not overlap unless an
 * entry says so.  Every entry is asynchronous on `stream`, allocates
 * nothing, keeps nothing between calls, and gives the same bits every time.
 * ------------------------------------------------------------------------ */

#define PC_Q8_GROUP 32

typedef enum pc_dtype { PC_F32 = 0, PC_F16 = 1, PC_BF16 = 2 } pc_dtype;

typedef enum pc_q8_format {
    PC_Q8_E4M3 = 0, /* largest magnitude 448 */
    PC_Q8_INT8 = 1  /* -127 .. 127 */
} pc_q8_format;

typedef enum pc_activation {
    PC_ACT_SILU = 0,     /* x / (1 + exp(-x)) */
    PC_ACT_GELU = 1,     /* x Phi(x), Phi the normal distribution function */
    PC_ACT_GELU_TANH = 2 /* x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) */
} pc_activation;

/* A stored tensor in device memory, as an argument (the struct itself is host memory, read during the call). */
typedef struct pc_q8 {
    const uint8_t *sym;
    const uint8_t *scale;
    uint64_t rows, cols;
    uint64_t ld_sym;   /* >= cols */
    uint64_t ld_scale; /* >= ceil(cols / 32) */
    int32_t format;    /* pc_q8_format */
    int32_t reserved;  /* 0 */
} pc_q8;

/*
 * Store a tensor in 8 bits.  For each group of 32 columns of a row, with a
 * the largest finite magnitude in it and M the format's (448 or 127):
 *   k = the smallest integer >= -117 with a <= M 2^k  (-117 where a is 0)
 *   sym = x 2^-k rounded to the nearest element, ties to even;  code = k + 127
 * so no finite value saturates.  Magnitudes from 248 * 2^120 on (e4m3; int8:
 * above 127 * 2^121, and from it on beside such a one), the largest finite
 * f32 and bf16 among them, round to 2^128 and so read back as infinity.
 * Infinities and NaN take no part in a and become 0x7F (e4m3) or 0x80 (int8),
 * which read back as NaN.
 *   d_x       rows x cols, row distance ldx.
 *   d_sym     rows * cols bytes, dense.
 *   d_scale   rows * ceil(cols / 32) bytes, dense.
 *   d_counts  NULL, or 256 u64 (8-byte aligned) to which the histogram of
 *             the symbols is added, as pc_histogram would, in the same pass:
 *             the statistics a codebook is built from.
 * rows == 0 or cols == 0 does nothing.  cols is below 2^31.
 */
pc_status pc_q8_store(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, int format,
                      uint8_t *d_sym, uint8_t *d_scale, uint64_t *d_counts, void *stream);

/* Read a stored tensor back: d_out (rows x cols, row distance ld_out) = the values, rounded to dtype. */
pc_status pc_q8_load(const pc_q8 *q, void *d_out, int dtype, size_t ld_out, void *stream);

/*
 * Backward pass of an activation whose inputs were stored.  With g and u the
 * stored gate and up values and dh the gradient of h:
 *   h = act(g) u,   d_gate = dh u act'(g),   d_up = dh act(g);
 * with up == NULL (an activation without a gate)  h = act(g), d_gate = dh act'(g).
 *   d_dh     rows x cols, as are the outputs; all of one dtype, each with a
 *            row distance of its own.  d_gate may be d_dh itself (same ld).
 *   gate, up stored tensors of that size and of one format; to read gate and
 *            up out of one tensor that holds them side by side, point into it.
 *   d_up     NULL exactly where up is NULL.
 *   d_h      NULL, or receives h (for the weight gradient of what follows).
 */
pc_status pc_q8_glu_backward(const void *d_dh, int dtype, size_t ld_dh, const pc_q8 *gate, const pc_q8 *up,
                             int activation, void *d_gate, size_t ld_gate, void *d_up, size_t ld_up, void *d_h,
                             size_t ld_h, void *stream);

/*
 * Weight gradient of a projection whose input x was stored:
 *   dW[n][k] = sum over rows t of dy[t][n] x[t][k]   (+ dW[n][k] where accumulate)
 *   d_dy      x->rows x n_out, row distance ld_dy.
 *   d_dw      n_out x x->cols, row distance ld_dw, f32, f16 or bf16.
 * Products are exact and sums are in 32 bits: stored values and bf16
 * gradients go into bf16 matrix instructions as they are; f16 and f32
 * gradients go in as two and three bf16 terms that add up to them (two and
 * three times the operations; of f32 gradients below 2^-110 what lies below
 * 2^-133, bf16's smallest step, is lost).
 *   d_ws, ws_bytes  scratch of pc_q8_weight_grad_workspace_bytes (which may
 *             be 0, then d_ws may be NULL), 16-byte aligned.
 * x->rows == 0: dW = 0, or stays where accumulate.  PC_ERR_UNSUPPORTED: row
 * distances of dy and x of 2^24 elements and more, and a dW of 2^24 - 7 tiles
 * of 128 x 128 (256 x 256 where those are 160 and dy is bf16) and more.
 */
size_t pc_q8_weight_grad_workspace_bytes(size_t rows, size_t n_out, size_t n_in, int dy_dtype);
pc_status pc_q8_weight_grad(const void *d_dy, int dy_dtype, size_t ld_dy, size_t n_out, const pc_q8 *x, void *d_dw,
                            int dw_dtype, size_t ld_dw, int accumulate, void *d_ws, size_t ws_bytes, void *stream);

/*
 * Embedding lookup: out[t] = scale * table[token[t]].
 *   d_tokens  n tokens, 4 or 8 bytes each (token_bytes), signed.
 *   d_table   vocab x dim, row distance ld_table; pc_embed_q8 takes a stored
 *             table (vocab = table->rows, dim = table->cols).
 *   d_out     n x dim, row distance ld_out.
 *   d_status  NULL, or one u32 that the caller has zeroed: a token outside
 *             [0, vocab) sets it to PC_ERR_INVALID_ARG.  Its row of the
 *             output is 0 either way.
 */
pc_status pc_embed(const void *d_tokens, int token_bytes, size_t n, const void *d_table, int table_dtype,
                   size_t vocab, size_t dim, size_t ld_table, float scale, void *d_out, int out_dtype,
                   size_t ld_out, uint32_t *d_status, void *stream);
pc_status pc_embed_q8(const void *d_tokens, int token_bytes, size_t n, const pc_q8 *table, float scale, void *d_out,
                      int out_dtype, size_t ld_out, uint32_t *d_status, void *stream);

/*
 * Gradient of the embedding table:
 *   grad[v] = scale * sum over t with token[t] == v of dy[t]   (+ grad[v] where accumulate)
 * Tokens are sorted first and each row is summed in the order of its tokens,
 * in blocks whose sizes depend on the call's sizes alone, so the result has the same
 * bits every time.  Rows without a token become 0 (stay, where accumulate).
 * Tokens outside [0, vocab) and tokens equal to `padding` (-1: none) add
 * nothing.
 *   d_dy      n x dim, row distance ld_dy.
 *   d_grad    vocab x dim, row distance ld_grad.
 *   d_ws, ws_bytes  scratch of pc_embed_backward_workspace_bytes (0 for few
 *             tokens, then d_ws may be NULL), 16-byte aligned.
 * Limits: with b = ceil(n / 32) ceil(dim / 512) (ceil(n / 8) in place of
 * ceil(n / 32) where n ceil(dim / 512) is at most 32768), b - ceil(dim / 512)
 * below 2^24 and b + vocab at most 2^26 - 4; n x dim and vocab x dim of at
 * most 2^36 - 4096 elements each, dim counted in whole 32s.  Beyond them
 * PC_ERR_UNSUPPORTED, and 0 bytes of workspace.
 */
size_t pc_embed_backward_workspace_bytes(size_t n, size_t dim, size_t vocab);
pc_status pc_embed_backward(const void *d_dy, int dy_dtype, size_t ld_dy, const void *d_tokens, int token_bytes,
                            size_t n, size_t dim, size_t vocab, int64_t padding, float scale, void *d_grad,
                            int grad_dtype, size_t ld_grad, int accumulate, void *d_ws, size_t ws_bytes,
                            void *stream);

/* ------------------------------------------------------------------------
 * What a step does between its products: dropout, the norm with the
 * residual's addition and an output in 8 bits, and log probabilities
 * ------------------------------------------------------------------------ */

/*
 * A dropout mask.  It is stored nowhere: whether element (r, c) of a tensor
 * is dropped follows from its place, the seed and the offset alone, so a
 * backward pass makes the same mask again.
 *   Numbers: Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
 *   numbers: as easy as 1, 2, 3", 2011) with the counter (c / 8, r, low word,
 *   high word of the offset) and the seed's low and high word as the key.  Of
 *   its four words, column c takes the low (c even) or high (c odd) 16 bits of
 *   word (c mod 8) / 2; the element is dropped, whatever it holds, where they
 *   are below T = 65536 p rounded to a whole number (ties to even).  The
 *   others are multiplied by 65536 / (65536 - T).
 *   p         0 (nothing is dropped) to 1 (everything is).
 *   d_random  NULL, or two u64 in device memory (8-byte aligned): the seed, in
 *             place of `seed`, and a number added to `offset` modulo 2^64.  A
 *             captured graph reads them anew at each replay; they stay as they
 *             are until the backward pass that takes the mask again has run.
 * Calls that shall not share a mask differ in seed or offset.  The struct is host memory, read during the call.
 */
typedef struct pc_mask {
    double p;
    uint64_t seed, offset;
    const uint64_t *d_random;
} pc_mask;

/* out = mask(x): rows x cols of one dtype, each with its row distance; d_out may be d_x (same ld).  cols is below 2^31. */
pc_status pc_dropout(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, const pc_mask *mask,
                     void *d_out, size_t ld_out, void *stream);

/*
 * Root-mean-square norm of a residual block's input, stored in 8 bits:
 *   h = res + mask(x), rounded to sum_dtype
 *   rstd = (mean of h^2 over the row + eps)^-1/2
 *   y = h rstd weight
 *   d_x      rows x cols of dtype, row distance ldx.
 *   d_res    NULL (no residual: then sum_dtype is dtype), or rows x cols of sum_dtype: dtype or PC_F32.
 *   mask     NULL, or the dropout of x.
 *   d_weight NULL (1), or cols numbers of weight_dtype.
 *   eps      positive and finite.
 *   d_sum    NULL, or receives h; may be d_res, or d_x where the types agree (same ld).  NULL without d_res and mask (h is x).
 *   d_sym, d_scale  NULL, or receive y as pc_q8_store would store it, dense;
 *            d_counts as there (NULL without d_sym).  What is stored is y
 *            from h in 64 bits, rounded once; what f32 cannot hold counts as infinite.
 *   d_y      NULL, or receives y rounded to y_dtype (from 32 bits, which have y
 *            to 3.1 2^-24 of it or 2^-126); where y_stored, the stored values in
 *            its place, as pc_q8_load gives them (needs d_sym).  May be d_x or
 *            d_res of its type (same ld).
 *   d_rstd   NULL, or receives rows f32.
 * No output overlaps an input or another output but for what is said here.
 * Squares are summed in 64 bits.  A row that holds an infinity has rstd 0, one
 * that holds NaN has rstd NaN.  cols is below 2^31; cols == 0 writes nothing, rstd neither.
 */
pc_status pc_rmsnorm_store(const void *d_x, int dtype, size_t rows, size_t cols, size_t ldx, const void *d_res,
                           int sum_dtype, size_t ld_res, const pc_mask *mask, const void *d_weight, int weight_dtype,
                           float eps, void *d_sum, size_t ld_sum, int format, uint8_t *d_sym, uint8_t *d_scale,
                           uint64_t *d_counts, void *d_y, int y_dtype, size_t ld_y, int y_stored, float *d_rstd,
                           void *stream);

/*
 * Backward pass of pc_rmsnorm_store.  With n = h rstd and g = dy weight:
 *   d = rstd (g - n mean(g n)) + dsum
 *   d_res = d,  d_x = mask(d),  d_weight = sum over the rows of dy n  (+ d_weight where accumulate)
 *   d_dy     rows x cols of dtype, the gradient of y.
 *   d_sum    h, rows x cols of sum_dtype (dtype or PC_F32); or NULL, and
 *   stored_sum  h as it was stored, in its place.
 *   d_rstd   rows f32, as the forward pass gave them.
 *   d_dsum   NULL, or the gradient that reaches h on the residual's way, of sum_dtype.
 *   mask     NULL, or the forward pass's.
 *   d_dres   NULL, or receives d in sum_dtype.
 *   d_dx     NULL, or receives mask(d) in dtype.  Each of the two may be one of d_dy, d_sum and
 *            d_dsum of its type (same ld); no output overlaps an input otherwise, or another output.
 *   d_dweight  NULL, or receives cols numbers of dweight_dtype (no other argument's memory); each
 *            is summed in 32 bits in an order that depends on the sizes alone.
 *   d_ws, ws_bytes  scratch of pc_rmsnorm_backward_workspace_bytes (0 for few
 *            rows, then d_ws may be NULL), 16-byte aligned; not needed without d_dweight.
 * Computed in 32 bits: an n below 2^-126 (a small h in a row of large ones) is off by 2^-150.
 * rows == 0: d_weight = 0, or stays where accumulate.
 */
size_t pc_rmsnorm_backward_workspace_bytes(size_t rows, size_t cols);
pc_status pc_rmsnorm_backward(const void *d_dy, int dtype, size_t rows, size_t cols, size_t ld_dy, const void *d_sum,
                              int sum_dtype, size_t ld_sum, const pc_q8 *stored_sum, const void *d_weight,
                              int weight_dtype, const float *d_rstd, const void *d_dsum, size_t ld_dsum,
                              const pc_mask *mask, void *d_dres, size_t ld_dres, void *d_dx, size_t ld_dx,
                              void *d_dweight, int dweight_dtype, int accumulate, void *d_ws, size_t ws_bytes,
                              void *stream);

/*
 * Log probabilities of rows of logits.  With z = scale x:
 *   logp[j] = z[token[j]] - ln sum exp z,   entropy = - sum p ln p,  p = exp(logp)
 *   d_logits  rows x vocab, row distance ld.  -infinity marks a token that cannot be chosen.
 *   scale     2^-64 to 2^64: the inverse temperature.
 *   d_tokens  rows x n_tokens (at most 64) of 4 or 8 bytes each, signed, dense: one or more for each row.
 *   d_logp    rows x n_tokens f32 (NULL where n_tokens is 0).  A token equal to `padding` or outside [0, vocab) gets 0.
 *   top       0 to 64, at most vocab: the largest logits of each row,
 *             in descending order, equal ones by their index (NaN counts as
 *             -infinity): d_top_index rows x top i64, d_top_logp f32.
 *   d_stats   NULL, or rows x 4 f32 for the backward pass and the caller: the
 *             row's largest logit, ln sum exp(z - scale largest), the entropy, and ln sum exp z.
 *   d_status  NULL, or one u32 that the caller has zeroed: a token outside
 *             [0, vocab) other than `padding` sets it to PC_ERR_INVALID_ARG.
 *   d_ws, ws_bytes  scratch of pc_logprobs_workspace_bytes (which may be 0,
 *             then d_ws may be NULL), 16-byte aligned.
 * A row that is -infinity throughout has nothing to choose: log probabilities
 * -infinity, entropy 0.  A row that holds NaN or +infinity: NaN.
 * PC_ERR_UNSUPPORTED: more than 64 tokens or alternatives, and rows x
 * ceil(vocab / 1024) of 2^31 and more.
 */
size_t pc_logprobs_workspace_bytes(size_t rows, size_t vocab, size_t top, int dtype);
pc_status pc_logprobs(const void *d_logits, int dtype, size_t rows, size_t vocab, size_t ld, float scale,
                      const void *d_tokens, int token_bytes, size_t n_tokens, int64_t padding, float *d_logp,
                      size_t top, int64_t *d_top_index, float *d_top_logp, float *d_stats, uint32_t *d_status,
                      void *d_ws, size_t ws_bytes, void *stream);

/*
 * Gradient of the logits, from those of the log probabilities and of the entropy:
 *   dlogits[v] = scale (sum over j with token[j] == v of dlogp[j]
 *                       - p[v] (sum over j of dlogp[j] + dentropy (ln p[v] + entropy)))
 *   d_logits, scale, d_tokens, padding  as in the forward pass; d_stats what it gave.
 *   d_dlogp   rows x n_tokens f32 (NULL where n_tokens is 0).  Of a token
 *             equal to `padding` or outside the vocabulary it is not used.
 *   d_dentropy  NULL, or rows f32.
 *   d_dlogits rows x vocab of the logits' dtype; may be d_logits (same ld), and overlaps no other input.
 * Probabilities below 2^-126 count as 0.  Rows whose given gradients are all 0
 * get zeros, whatever their logits; so do rows that are -infinity throughout.
 */
pc_status pc_logprobs_backward(const void *d_logits, int dtype, size_t rows, size_t vocab, size_t ld, float scale,
                               const float *d_stats, const void *d_tokens, int token_bytes, size_t n_tokens,
                               int64_t padding, const float *d_dlogp, const float *d_dentropy, void *d_dlogits,
                               size_t ld_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PC_H */
