// Weight gradient of a projection whose input was stored in 8 bits:
//   dW[n][k] = sum over t of dy[t][n] x[t][k].
//
// A matrix product whose long axis t is the row axis of both operands.  Tiles
// of 64 rows lie in LDS as they lie in memory, in bf16 (x's symbols are exact
// there, as the scales are powers of two), and the transposing LDS reads hand
// every lane the consecutive t of one column that the matrix instruction
// takes.
//
// Large tiles are bound by the matrix cores at the clock they hold: 4096 rows,
// 11008 x 4096 from e4m3 and bf16 into f32 take 317-326 us (1.13-1.17 PFLOP/s;
// under the profiler, of few passes, 333-354); the matrix instructions alone,
// without loads and LDS, take 305 us, as 688 tiles are 2.7 rounds of 256 CUs.
// A library product of the same shape with x already in bf16 takes 379 us.
// int8 takes 500 us: its symbols need 4.5 vector instructions each, e4m3's half
// a one, and the one wave of a SIMD issues them between its matrix
// instructions (matrix cores busy 34% of the time, e4m3 59%).  11007 x 4095
// takes 411 us: rows of odd alignment cost 37 of the 90 more, the tile at the
// operands' end (accumulators through 476 bytes of scratch a lane) and the
// guarded epilogue the others.
// Small tiles with a long t (32768 rows, 320 x 1000) take 44 us from e4m3 and
// 50 from int8, and 6 us to join their slices.  No unit is full there (matrix
// cores 31 and 26%, LDS 40 and 34%, vector issue 16 and 44%): the two waves of
// a SIMD stand 42% of their time at waits for loads, LDS and barriers, and the
// 24 tiles read the operands 2.2 times (116 of 52 MiB).
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace pc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kThreads = 256;
constexpr uint32_t kStep = 64;  // rows t of one LDS tile

// dy as sums of bf16 terms: bf16 is its own, f16 (11 bits) needs two of 8
// bits, f32 (24 bits) three.
template <int DT> constexpr uint32_t kTerms = DT == PC_BF16 ? 1 : DT == PC_F16 ? 2 : 3;

// Term `WHICH` of v, as the upper half of an f32: v cut off to 8 bits, then
// what is left, which 32 bits hold exactly.  Infinity and NaN are their own
// first term and leave 0.
template <uint32_t WHICH>
__device__ __forceinline__ uint32_t term_bits(float v) {
    const uint32_t u = as_u32(__builtin_canonicalizef(v));  // a NaN's upper half is one too
    if constexpr (WHICH == 0) {
        return u;
    } else {
        const float rest = v - as_f32(u & 0xFFFF0000u);
        return term_bits<WHICH - 1>(__builtin_isfinite(v) ? rest : 0.0f);
    }
}

// Memory as the hardware's bounds-checked buffer: a load that starts at or
// past its end reads 0.  `window` walks down the rows of an operand, a tile
// at a time; `left`: bytes from there to the operand's last element.
typedef __amdgpu_buffer_rsrc_t Buffer;
struct Window {
    uint64_t at, step;
    int64_t left;

    __device__ __forceinline__ Window(const void *p, uint64_t row, uint64_t before, uint64_t rows, uint64_t width)
        : at(reinterpret_cast<uint64_t>(p) + before), step(kStep * row),
          left(rows ? (int64_t)((rows - 1) * row + width) : 0) {}
    __device__ __forceinline__ Buffer buffer() const {
        const int32_t high = (int32_t)(left >> 32);
        const uint32_t bytes = high < 0 ? 0u : high > 0 ? 0xFFFFFFFFu : (uint32_t)left;
        return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(at), 0, (int)bytes, 0x00020000);
    }
    __device__ __forceinline__ void down(uint32_t tiles = 1) {
        at += tiles * step;
        left -= (int64_t)(tiles * step);
    }
};

// A lane's pieces of a tile as loaded, P of them: 8 elements of dy, or 16
// symbols of x and their scale code.
template <int DT, uint32_t P> struct RawDy {
    static constexpr uint32_t kWords = DT == PC_F32 ? 2 : 1;
    u32x4 w[P][kWords];

    __device__ __forceinline__ void load(Buffer b, uint32_t at, uint32_t step) {
#pragma unroll
        for (uint32_t p = 0; p < P; ++p)
#pragma unroll
            for (uint32_t k = 0; k < kWords; ++k)
                w[p][k] = __builtin_amdgcn_raw_buffer_load_b128(b, at + p * step + 16 * k, 0, 0);
    }
    // the first n elements of piece p, each by itself
    __device__ __forceinline__ void load_single(uint32_t p, Buffer b, uint32_t at, uint32_t n) {
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {
            if constexpr (DT == PC_F32) {
                w[p][c / 4][c % 4] = c < n ? __builtin_amdgcn_raw_buffer_load_b32(b, at + 4 * c, 0, 0) : 0u;
            } else {
                const uint32_t e = c < n ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, at + 2 * c, 0, 0) : 0u;
                w[p][0][c / 2] = c % 2 ? w[p][0][c / 2] | e << 16 : e;
            }
        }
    }
    // piece p's term in bf16
    template <uint32_t WHICH>
    __device__ __forceinline__ u32x4 piece(uint32_t p) const {
        if constexpr (DT == PC_BF16) {
            return w[p][0];
        } else {
            u32x4 out;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float a, b;
                if constexpr (DT == PC_F16) {
                    const uint32_t u = w[p][0][k];
                    const f16x2 h = __builtin_bit_cast(f16x2, u);
                    a = (float)h[0];
                    b = (float)h[1];
                } else {
                    a = as_f32(w[p][k / 2][(2 * k) % 4]);
                    b = as_f32(w[p][k / 2][(2 * k) % 4 + 1]);
                }
                out[k] = __builtin_amdgcn_perm(term_bits<WHICH>(b), term_bits<WHICH>(a), 0x07060302u);
            }
            return out;
        }
    }
};

template <int FMT, uint32_t P> struct RawX {
    u32x4 w[P];
    uint32_t code[P];

    __device__ __forceinline__ void load(Buffer b, uint32_t at, uint32_t step, Buffer codes, uint32_t code_at,
                                         uint32_t code_step) {
#pragma unroll
        for (uint32_t p = 0; p < P; ++p) {
            w[p] = __builtin_amdgcn_raw_buffer_load_b128(b, at + p * step, 0, 0);
            code[p] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(codes, code_at + p * code_step, 0, 0);
        }
    }
    __device__ __forceinline__ void load_single(uint32_t p, Buffer b, uint32_t at, uint32_t n) {
        w[p] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (uint32_t c = 0; c < 16; ++c)
            if (c < n)
                w[p][c / 4] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(b, at + c, 0, 0) << (8 * (c % 4));
    }
    // half h of piece p in bf16
    __device__ __forceinline__ u32x4 piece(uint32_t p, uint32_t h) const {
        const float s = scale_of(code[p]);
        u32x4 out;
        if constexpr (FMT == PC_Q8_E4M3) {
#pragma unroll
            for (uint32_t k = 0; k < 2; ++k) {
                out[2 * k] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[p][2 * h + k], s, false));
                out[2 * k + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[p][2 * h + k], s, true));
            }
        } else {
            // without branches, in the middle of the products
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) {
                const uint32_t u = w[p][2 * h + k / 2] >> (16 * (k % 2));
                float lo = (float)(int)(int8_t)(u & 0xFFu), hi = (float)(int)(int8_t)((u >> 8) & 0xFFu);
                lo = lo == -128.0f ? __builtin_nanf("") : lo;
                hi = hi == -128.0f ? __builtin_nanf("") : hi;
                out[k] = __builtin_amdgcn_perm(as_u32(hi * s), as_u32(lo * s), 0x07060302u);
            }
        }
        return out;
    }
};

// Rows in LDS are bf16, without padding; a row's 64-byte chunks (32 columns,
// a fragment's) change places with the row, by its last two bits, so that the
// four rows that a transposing read takes together lie in different banks.
__device__ __forceinline__ uint32_t swizzled(uint32_t unit, uint32_t row) { return unit ^ (row & 3) << 2; }  // 16-byte units

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;

// Transposing read: of 16 lanes, lane i points at 4 columns of row i / 4 (of
// 4), columns 4 (i % 4) .. of 16; lane j gets column j of the 4 rows.
__device__ __forceinline__ bf16x4 read_transposed(const void *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (lds_bf16x4 *)(__attribute__((address_space(3))) void *)const_cast<void *>(p));
}

struct Shape {
    uint64_t t, n, k;  // rows, n_out, n_in
    uint64_t ld_dy, ld_sym, ld_scale, ld_out;
    uint32_t slice;    // LDS tiles of one slice of t
    uint32_t tiles_n, tiles_k;
};

// Workgroups go to the eight dies in turn, each with an L2 of its own: a die
// gets a run of consecutive tiles of the order below, in which 8 tiles along k
// come before the next along n, so that the 32 tiles a die works on at a time
// read about 4 strips of dy and 8 of x.  The grid is a multiple of 8; tiles
// past the last have n >= tiles_n.
struct Tile {
    uint32_t n, k;
};
__device__ __forceinline__ Tile tile_of(const Shape &s, uint32_t block, uint32_t blocks) {
    const uint32_t o = block % 8 * (blocks / 8) + block / 8;
    const uint32_t band = o / (s.tiles_n * 8), in_band = o % (s.tiles_n * 8);
    const uint32_t left = s.tiles_k - min(s.tiles_k, band * 8), width = min(left, 8u);  // the last band may be narrower
    if (width == 0) return {s.tiles_n, 0};
    return {in_band / width, band * 8 + in_band % width};
}

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The order of a phase's instructions (16 products of a wave): the LDS reads
// of the next phase first, two behind every matrix instruction, then V vector
// instructions, W LDS writes and L loads spread over the others, so that the
// matrix cores never wait for a run of other work.
template <uint32_t M, uint32_t V, uint32_t W, uint32_t L, bool LOADS_FIRST = false>
__device__ __forceinline__ void interleave() {
    if constexpr (M == 16) {
#pragma unroll
        for (uint32_t m = 0; m < 16; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                            // matrix
            if (m < 8) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                 // LDS read
            if (L && (m < 8) == LOADS_FIRST) __builtin_amdgcn_sched_group_barrier(0x020, L / 8, 0);
            if (V && m >= 8) __builtin_amdgcn_sched_group_barrier(0x002, V / 8, 0);
            if (W && m >= 8) __builtin_amdgcn_sched_group_barrier(0x200, W / 8, 0);       // LDS write
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Three phases as one where the pieces take much vector work (int8): 8 vector
// instructions behind each of the 48 matrix instructions.  As above, only for
// the large tiles, which f16 and f32 gradients do not take.
template <uint32_t M>
__device__ __forceinline__ void interleave_three() {
    if constexpr (M == 16) {
#pragma unroll
        for (uint32_t m = 0; m < 48; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, 8, 0);
            if (m % 3 == 2) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
            if (m >= 32) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

template <int DT, int FMT, bool RAGGED, uint32_t WN, uint32_t WK, uint32_t FN, uint32_t FK>
__global__ __launch_bounds__(WN *WK *kWave, FN * FK == 16 ? 1 : 2) void wgrad_kernel(const typename Plain<DT>::type *__restrict__ dy,
                                                                 const uint8_t *__restrict__ sym,
                                                                 const uint8_t *__restrict__ scale, Shape s,
                                                                 void *__restrict__ out, int out_dtype, uint32_t add) {
    constexpr uint32_t BN = WN * FN * 32, BK = WK * FK * 32, NT = WN * WK * kWave;
    constexpr uint32_t kElem = sizeof(typename Plain<DT>::type);
    constexpr uint32_t UN = BN / 8, UK = BK / 8;                            // 16-byte units of a row in LDS
    constexpr uint32_t PY = kStep * UN / NT, PX = kStep * UK / 2 / NT;      // pieces of a lane
    constexpr uint32_t RY = NT / UN, RX = NT / (UK / 2);                    // rows between them
    static_assert(RY % 4 == 0 && RX % 4 == 0, "a lane's pieces lie in rows of the same last two bits");
    __shared__ u32x4 ly[2][kStep * UN];
    __shared__ u32x4 lx[2][kStep * UK];
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
    const uint32_t wn = wave / WK, wk = wave % WK;
    const Tile tile = tile_of(s, blockIdx.x, gridDim.x);
    if (tile.n >= s.tiles_n) return;
    const uint64_t n0 = (uint64_t)tile.n * BN, k0 = (uint64_t)tile.k * BK;
    const uint32_t all = (uint32_t)((s.t + kStep - 1) / kStep);
    const uint32_t first = min(all, blockIdx.y * s.slice), tiles = min(all - first, s.slice);

    const uint32_t yc = tid % UN, yt = tid / UN, xc = tid % (UK / 2), xt = tid / (UK / 2);  // first pieces
    const uint32_t y_row = (uint32_t)s.ld_dy * kElem, x_row = (uint32_t)s.ld_sym, c_row = (uint32_t)s.ld_scale;
    const uint32_t y_at = yt * y_row + yc * 8 * kElem, x_at = xt * x_row + xc * 16, c_at = xt * c_row + xc / 2;
    RawDy<DT, PY> ry;
    RawX<FMT, PX> rx;

    // The operands from this slice's first row on.  Loads run ahead of the
    // products, past the slice's end, within the tensor; what they bring from
    // there is not multiplied.
    const uint64_t t_first = (uint64_t)first * kStep, rows = s.t > t_first ? s.t - t_first : 0;
    const uint64_t c0 = k0 / kGroup;
    const Window y0(dy + n0, y_row, t_first * y_row, rows, (s.n - n0) * kElem);
    const Window x0(sym + k0, x_row, t_first * x_row, rows, s.k - k0);
    const Window q0(scale + c0, c_row, t_first * c_row, rows, (s.k + kGroup - 1) / kGroup - c0);
    Window yw = y0, xw = x0, qw = q0;
    auto load_dy = [&]() {
        ry.load(yw.buffer(), y_at, RY * y_row);
        yw.down();
    };
    auto load_x = [&]() {
        rx.load(xw.buffer(), x_at, RX * x_row, qw.buffer(), c_at, RX * c_row);
        xw.down();
        qw.down();
    };
    auto put_dy = [&](auto which, uint32_t buf) {
        u32x4 *to = ly[buf] + yt * UN + swizzled(yc, yt);
#pragma unroll
        for (uint32_t p = 0; p < PY; ++p) to[p * RY * UN] = ry.template piece<decltype(which)::value>(p);
    };
    auto put_x = [&](uint32_t buf) {
        u32x4 *to = lx[buf] + xt * UK + swizzled(2 * xc, xt);
#pragma unroll
        for (uint32_t p = 0; p < PX; ++p)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) to[p * RX * UK + h] = rx.piece(p, h);
    };
    f32x16 acc[FN][FK];
#pragma unroll
    for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j) acc[i][j] = f32x16{0};

    if (tiles) {
        // a lane's place in the transposing reads: row q (of 4) of the half
        // wave's 8, columns 16 (lane / 16 % 2) + 4 (lane % 4) of the fragment's 32
        const uint32_t q = lane % 16 / 4, row = lane / 32 * 8 + q, within = lane / 16 % 2 * 32 + lane % 4 * 8;
        uint32_t a_at[FN], b_at[FK];  // bytes
#pragma unroll
        for (uint32_t i = 0; i < FN; ++i) a_at[i] = row * UN * 16 + ((wn * FN + i) ^ q) * 64 + within;
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j) b_at[j] = row * UK * 16 + ((wk * FK + j) ^ q) * 64 + within;
        bf16x8 fa[2][FN], fb[2][FK];
        auto fragment = [&](const u32x4 *tile, uint32_t at, uint32_t units) {
            const char *p = reinterpret_cast<const char *>(tile) + at;
            return __builtin_shufflevector(read_transposed(p), read_transposed(p + 4 * units * 16), 0, 1, 2, 3, 4, 5, 6, 7);
        };
        auto read = [&](uint32_t which, uint32_t buf, uint32_t kk) {
#pragma unroll
            for (uint32_t i = 0; i < FN; ++i) fa[which][i] = fragment(ly[buf] + kk * 16 * UN, a_at[i], UN);
#pragma unroll
            for (uint32_t j = 0; j < FK; ++j) fb[which][j] = fragment(lx[buf] + kk * 16 * UK, b_at[j], UK);
        };
        auto multiply = [&](uint32_t which) {
#pragma unroll
            for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
                for (uint32_t j = 0; j < FK; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[which][i], fb[which][j], acc[i][j], 0, 0, 0);
        };
        // Multiplies tile i out of its LDS buffer, puts tile i + 1 into the other
        // one and loads tile i + 2 (a second tile on its way in registers gained
        // nothing: 55 against 52 us for 320 x 1000 of 32768 rows).  The barrier
        // stands before the last quarter of the products: by then the other
        // waves' pieces of tile i + 1 are in LDS, and its first fragments arrive
        // behind those products.
        auto step = [&](auto which, uint32_t i) {
            constexpr uint32_t M = FN * FK;
            constexpr bool kFewVector = FMT == PC_Q8_E4M3 && kTerms<DT> == 1;
            const uint32_t buf = i & 1;
            read(1, buf, 1);
            put_dy(which, buf ^ 1);
            multiply(0);
            if (kFewVector) interleave<M, 0, 8, 0>();
            load_dy();
            read(0, buf, 2);
            put_x(buf ^ 1);
            multiply(1);
            if (kFewVector) interleave<M, 32, 8, 8, true>();
            load_x();
            read(1, buf, 3);
            multiply(0);
            if (kFewVector) interleave<M, 0, 0, 8>();
            else interleave_three<M>();
            lds_barrier();
            read(0, buf ^ 1, 0);
            multiply(1);
            interleave<M, 0, 0, 0>();
        };
        // Widths that are no multiple of a piece: a piece that sticks out of the
        // tensor's last row may lose the elements that are inside, as its load
        // crosses the end.  The tiles that can hold one (the last, and the one
        // before where rows are shorter than a piece) are done by themselves.
        const uint32_t apart = !RAGGED || rows > (uint64_t)tiles * kStep + 16 ? 0
                               : rows + kStep > (uint64_t)tiles * kStep + 16 ? 1
                                                                             : 2;
        const uint32_t whole = tiles - min(tiles, apart);
        auto pass = [&](auto which) {
            yw = y0;
            xw = x0;
            qw = q0;
            if (!RAGGED || whole) {
                load_dy();
                load_x();
                put_dy(which, 0);
                put_x(0);
                load_dy();
                load_x();
                lds_barrier();
                read(0, 0, 0);
#pragma unroll 1
                for (uint32_t i = 0; i < whole; ++i) step(which, i);
            }
            if constexpr (RAGGED) {
#pragma unroll 1
                for (uint32_t i = whole; i < tiles; ++i) {
                    yw = y0;
                    xw = x0;
                    qw = q0;
                    yw.down(i);
                    xw.down(i);
                    qw.down(i);
                    const Window ye = yw, xe = xw;
                    load_dy();
                    load_x();
                    const uint64_t cy = n0 + yc * 8, cx = k0 + xc * 16;
                    if (cy < s.n && cy + 8 > s.n) {
#pragma unroll
                        for (uint32_t p = 0; p < PY; ++p) {
                            const uint32_t at = y_at + p * RY * y_row;
                            if (at < ye.left && at + 8 * kElem > ye.left)
                                ry.load_single(p, ye.buffer(), at, (uint32_t)(s.n - cy));
                        }
                    }
                    if (cx < s.k && cx + 16 > s.k) {
#pragma unroll
                        for (uint32_t p = 0; p < PX; ++p) {
                            const uint32_t at = x_at + p * RX * x_row;
                            if (at < xe.left && at + 16 > xe.left)
                                rx.load_single(p, xe.buffer(), at, (uint32_t)(s.k - cx));
                        }
                    }
                    lds_barrier();  // the other waves' reads of the last tile
                    put_dy(which, 0);
                    put_x(0);
                    lds_barrier();
#pragma unroll
                    for (uint32_t kk = 0; kk < kStep / 16; ++kk) {
                        read(0, 0, kk);
                        multiply(0);
                    }
                }
            }
        };
        pass(std::integral_constant<uint32_t, 0>());
        if constexpr (kTerms<DT> > 1) {
            lds_barrier();  // the other waves' reads of the last tile
            pass(std::integral_constant<uint32_t, 1>());
        }
        if constexpr (kTerms<DT> > 2) {
            lds_barrier();
            pass(std::integral_constant<uint32_t, 2>());
        }
    }

    // Accumulating tiles take the guarded way, one load and store after the
    // other: 4096 rows to 11008 x 4096 638 us against 321, 2048 to 4096 x 4096
    // 136 against 67.
    const bool inside = n0 + BN <= s.n && k0 + BK <= s.k && !add;
    auto write = [&](auto o) {
        typedef typename Plain<decltype(o)::value>::type T;
        // a slice's partial sums (one slice: the output), at the wave's first row and column, the same for all lanes
        T *base = static_cast<T *>(out) + (uint64_t)blockIdx.y * s.n * s.k + (n0 + wn * FN * 32) * s.ld_out + k0 +
                  wk * FK * 32;
        const uint32_t below = lane / 32 * 4;
        const uint64_t at = below * s.ld_out + lane % 32;
        if (inside) {
            // 128 bytes a row and half wave.  A large result in f32 streams past
            // the caches (352 -> 342 us); partial sums, which only the small
            // tiles leave, are read next.
#pragma unroll
            for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
                for (uint32_t v = 0; v < 16; ++v) {
                    T *p = base + (i * 32 + v / 4 * 8 + v % 4) * s.ld_out + at;
#pragma unroll
                    for (uint32_t j = 0; j < FK; ++j) {
                        if constexpr (decltype(o)::value == PC_F32 && FN * FK == 16) {
                            const float value = acc[i][j][v];
                            __builtin_nontemporal_store(value, p + j * 32);
                        } else {
                            p[j * 32] = (T)acc[i][j][v];
                        }
                    }
                }
            return;
        }
#pragma unroll
        for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
            for (uint32_t v = 0; v < 16; ++v) {
                const uint32_t r = i * 32 + v / 4 * 8 + v % 4;
                if (n0 + wn * FN * 32 + r + below >= s.n) continue;
                T *p = base + r * s.ld_out + at;
#pragma unroll
                for (uint32_t j = 0; j < FK; ++j)
                    if (k0 + (wk * FK + j) * 32 + lane % 32 < s.k)
                        p[j * 32] = (T)(acc[i][j][v] + (add ? widen(p[j * 32]) : 0.0f));
            }
    };
    with_dtype(out_dtype, write);
}

// Joins the slices' partial sums: four neighbours of the dense partial sums in
// a lane, a quarter of the slices in each of the four waves, in their order,
// the loads for 8 of them in flight together.
template <int ODT>
__global__ __launch_bounds__(kThreads) void join_kernel(const float *__restrict__ part, uint32_t slices, uint64_t n,
                                                        uint64_t k, uint64_t ld_out,
                                                        typename Plain<ODT>::type *__restrict__ out, uint32_t add) {
    constexpr uint32_t kAhead = 8, kShares = kThreads / kWave;
    typedef typename Plain<ODT>::type T;
    __shared__ f32x4 sums[kShares][kWave];
    const uint32_t lane = threadIdx.x % kWave, share = threadIdx.x / kWave;
    const uint64_t all = n * k, i = ((uint64_t)blockIdx.x * kWave + lane) * 4;
    const uint32_t have = count_before(all, i, 4);
    const uint32_t each = (slices + kShares - 1) / kShares, first = min(slices, share * each);
    const uint32_t end = min(slices, first + each);
    f32x4 sum = {0, 0, 0, 0};
    for (uint32_t s0 = first; s0 < end; s0 += kAhead) {
        f32x4 v[kAhead];
#pragma unroll
        for (uint32_t a = 0; a < kAhead; ++a) {
            const float *p = part + min(s0 + a, end - 1) * all;
            if (have == 4) {
                typedef f32x4 any __attribute__((aligned(4)));
                v[a] = *reinterpret_cast<const any *>(p + i);
            } else {
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) v[a][j] = j < have ? p[i + j] : 0.0f;
            }
        }
#pragma unroll
        for (uint32_t a = 0; a < kAhead; ++a)
            if (s0 + a < end) sum += v[a];
    }
    sums[share][lane] = sum;
    __syncthreads();
    if (share) return;
#pragma unroll
    for (uint32_t w = 1; w < kShares; ++w) sum += sums[w][lane];
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        if (j >= have) continue;
        T *p = out + (i + j) / k * ld_out + (i + j) % k;
        *p = (T)(sum[j] + (add ? widen(*p) : 0.0f));
    }
}

// Tiles of 256 x 256 (a wave's 128 x 128 part reads the least from LDS for
// each product) where there are enough of them for most of the 256 CUs, else of
// 128 x 128, two workgroups to a CU: 2048 rows to 4096 x 4096 take 65 us in
// large tiles and 81 in small ones, to 4096 x 2816 (176 large tiles) 54 and 59,
// to 2048 x 4096 (128 large tiles) 51 and 41.  Fewer small tiles than CUs share
// t in slices of at least 8 LDS tiles: 512 x 512 of 8192 rows takes 18 us so
// and 22 us in slices of 4, of 512 rows 12 and 16; 64 x 64 of 65536 rows 43 us,
// in slices of 4 62 us, of 2 104 us (of 16384 rows 20, 20 and 30); 32 x 1024 of
// 65536 rows 34 us in all three.  f16 and f32 gradients, of twice and three
// times the products, keep to the small tiles.
uint64_t tiles_of(uint64_t n, uint64_t k, uint32_t side) { return ((n + side - 1) / side) * ((k + side - 1) / side); }

struct Plan {
    uint32_t side, slices, slice;
};

Plan plan_of(uint64_t t, uint64_t n, uint64_t k, int dtype) {
    Plan p;
    const uint64_t steps = (t + kStep - 1) / kStep;
    p.side = dtype == PC_BF16 && tiles_of(n, k, 256) >= 160 ? 256 : 128;
    const uint64_t tiles = tiles_of(n, k, p.side);
    p.slices = 1;
    if (p.side == 128 && tiles < 256 && steps >= 16) p.slices = (uint32_t)std::min<uint64_t>(512 / tiles, steps / 8);
    p.slice = (uint32_t)((steps + p.slices - 1) / p.slices);
    return p;
}

}  // namespace

uint64_t wgrad_workspace(uint64_t t, uint64_t n, uint64_t k, int dtype) {
    const Plan p = plan_of(t, n, k, dtype);
    return p.slices > 1 ? (uint64_t)p.slices * n * k * 4 : 0;
}

// The launch takes a workgroup for every tile, a multiple of 8 of them, and fewer than 2^24.
bool wgrad_fits(uint64_t t, uint64_t n, uint64_t k, int dtype) {
    return tiles_of(n, k, plan_of(t, n, k, dtype).side) + 7 < 1ull << 24;
}

hipError_t launch_q8_weight_grad(const void *dy, int dtype, uint64_t ld_dy, uint64_t n_out, const pc_q8 *x, void *dw,
                                 int dw_dtype, uint64_t ld_dw, bool accumulate, void *ws, hipStream_t stream) {
    const uint64_t t = x->rows, n = n_out, k = x->cols;
    const Plan p = plan_of(t, n, k, dtype);
    const bool split = p.slices > 1;
    const Shape s = {t, n, k, ld_dy, x->ld_sym, x->ld_scale, split ? k : ld_dw, p.slice,
                     (uint32_t)((n + p.side - 1) / p.side), (uint32_t)((k + p.side - 1) / p.side)};
    const dim3 grid((s.tiles_n * s.tiles_k + 7) / 8 * 8, p.slices);
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto launch = [&](auto kern) {
            hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, stream, static_cast<const typename Plain<DT>::type *>(dy),
                               x->sym, x->scale, s, split ? ws : dw, split ? (int)PC_F32 : dw_dtype,
                               (uint32_t)(accumulate && !split));
        };
        auto by_side = [&](auto f, auto r) {
            constexpr int FMT = decltype(f)::value;
            constexpr bool RAGGED = decltype(r)::value;
            if constexpr (DT == PC_BF16) {
                if (p.side == 256) return launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 4, 4>);
            }
            launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 2, 2>);
        };
        auto by_format = [&](auto r) {
            if (x->format == PC_Q8_E4M3) by_side(std::integral_constant<int, PC_Q8_E4M3>(), r);
            else by_side(std::integral_constant<int, PC_Q8_INT8>(), r);
        };
        if (n % 8 || k % 16) by_format(std::true_type());
        else by_format(std::false_type());
    });
    if (split)
        with_dtype(dw_dtype, [&](auto o) {
            constexpr int ODT = decltype(o)::value;
            hipLaunchKernelGGL(join_kernel<ODT>, dim3((uint32_t)((n * k + 4 * kWave - 1) / (4 * kWave))), dim3(kThreads), 0,
                               stream, static_cast<const float *>(ws), p.slices, n, k, ld_dw,
                               static_cast<typename Plain<ODT>::type *>(dw), (uint32_t)accumulate);
        });
    return hipGetLastError();
}

}  // namespace pc
