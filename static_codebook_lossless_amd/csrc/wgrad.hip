// Weight gradient of a projection whose input was stored in 8 bits:
//   dW[n][k] = sum over t of dy[t][n] x[t][k].
//
// A matrix product whose long axis t is the row axis of both operands.  Tiles
// of 64 rows lie in LDS as they lie in memory, in bf16 (x's symbols are exact
// there, as the scales are powers of two), and the transposing LDS reads hand
// every lane the consecutive t of one column that the matrix instruction
// takes.
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

// Term `which` of v, as the upper half of an f32: v cut off to 8 bits, then
// what is left, which 32 bits hold exactly.  Infinity and NaN are their own
// first term and leave 0.
__device__ __forceinline__ float cut(float v) {
    const uint32_t u = as_u32(v), special = (u & 0x7FFFFFFFu) > 0x7F800000u ? 0x400000u : 0u;  // NaN stays NaN
    return as_f32((u | special) & 0xFFFF0000u);
}
__device__ __forceinline__ float left(float v, float first) {
    return (as_u32(v) & 0x7F800000u) == 0x7F800000u ? 0.0f : v - first;
}
__device__ __forceinline__ uint32_t term_bits(float v, uint32_t which) {
    float t = cut(v);
    for (uint32_t i = 0; i < which; ++i) {
        v = left(v, t);
        t = cut(v);
    }
    return as_u32(t);
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
    __device__ __forceinline__ void down() {
        at += step;
        left -= (int64_t)step;
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
    // piece p in bf16
    __device__ __forceinline__ u32x4 piece(uint32_t p, uint32_t which) const {
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
                out[k] = __builtin_amdgcn_perm(term_bits(b, which), term_bits(a, which), 0x07060302u);
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
            float v[8];
            const u32x2 u = {w[p][2 * h], w[p][2 * h + 1]};
            // one multiply-add a symbol where 128 times the scale is a number and no symbol NaN
            const uint32_t a = u[0] ^ 0x80808080u, b = u[1] ^ 0x80808080u;
            const bool nan = (((a - 0x01010101u) & ~a) | ((b - 0x01010101u) & ~b)) & 0x80808080u;
            if (nan || code[p] > 247) {
                unit_values<FMT>(u, s, v);
            } else {
                const float down = -128.0f * s;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k] = __builtin_fmaf((float)((a >> (8 * k)) & 0xFFu), s, down);
                    v[4 + k] = __builtin_fmaf((float)((b >> (8 * k)) & 0xFFu), s, down);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                out[k] = __builtin_amdgcn_perm(as_u32(v[2 * k + 1]), as_u32(v[2 * k]), 0x07060302u);
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

// SETS: tiles on their way in registers.
template <int DT, int FMT, bool RAGGED, uint32_t WN, uint32_t WK, uint32_t FN, uint32_t FK, uint32_t SETS>
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
    const uint32_t steps = tiles * kTerms<DT>;

    const uint32_t yc = tid % UN, yt = tid / UN, xc = tid % (UK / 2), xt = tid / (UK / 2);  // first pieces
    const uint32_t y_row = (uint32_t)s.ld_dy * kElem, x_row = (uint32_t)s.ld_sym, c_row = (uint32_t)s.ld_scale;
    const uint32_t y_at = yt * y_row + yc * 8 * kElem, x_at = xt * x_row + xc * 16, c_at = xt * c_row + xc / 2;
    RawDy<DT, PY> ry[SETS];
    RawX<FMT, PX> rx[SETS];

    // The operands from this slice's first row on.  Loads run ahead of the
    // products, past the slice's end, within the tensor; what they bring from
    // there is not multiplied.
    const uint64_t t_first = (uint64_t)first * kStep, rows = s.t > t_first ? s.t - t_first : 0;
    const uint64_t c0 = k0 / kGroup;
    const Window y0(dy + n0, y_row, t_first * y_row, rows, (s.n - n0) * kElem);
    const Window x0(sym + k0, x_row, t_first * x_row, rows, s.k - k0);
    const Window q0(scale + c0, c_row, t_first * c_row, rows, (s.k + kGroup - 1) / kGroup - c0);
    Window yw = y0, xw = x0, qw = q0;
    uint32_t y_tile = 0, x_tile = 0;  // for gradients of several terms, which read dy and x once for each
    auto load_dy = [&](RawDy<DT, PY> &r) {
        r.load(yw.buffer(), y_at, RY * y_row);
        yw.down();
        if (kTerms<DT> > 1 && ++y_tile == tiles) {
            y_tile = 0;
            yw = y0;
        }
    };
    auto load_x = [&](RawX<FMT, PX> &r) {
        r.load(xw.buffer(), x_at, RX * x_row, qw.buffer(), c_at, RX * c_row);
        xw.down();
        qw.down();
        if (kTerms<DT> > 1 && ++x_tile == tiles) {
            x_tile = 0;
            xw = x0;
            qw = q0;
        }
    };
    // A piece that sticks out of the tensor's last row (widths that are no
    // multiple of a piece): its load may have dropped elements that are inside.
    // Only the last tiles of t meet one.
    auto mend = [&](RawDy<DT, PY> &y, RawX<FMT, PX> &x, uint32_t i) {
        if constexpr (!RAGGED) return;
        const uint64_t t0 = (uint64_t)(kTerms<DT> == 1 ? i : i % tiles) * kStep;
        if (i >= steps || rows - t0 >= kStep + 16) return;
        const uint64_t cy = n0 + yc * 8, cx = k0 + xc * 16;
        if (cy < s.n && cy + 8 > s.n) {
            Window w = y0;
            w.at += t0 * y_row;
            w.left -= (int64_t)(t0 * y_row);
#pragma unroll
            for (uint32_t p = 0; p < PY; ++p) {
                const uint32_t at = y_at + p * RY * y_row;
                if (at < w.left && at + 8 * kElem > w.left) y.load_single(p, w.buffer(), at, (uint32_t)(s.n - cy));
            }
        }
        if (cx < s.k && cx + 16 > s.k) {
            Window w = x0;
            w.at += t0 * x_row;
            w.left -= (int64_t)(t0 * x_row);
#pragma unroll
            for (uint32_t p = 0; p < PX; ++p) {
                const uint32_t at = x_at + p * RX * x_row;
                if (at < w.left && at + 16 > w.left) x.load_single(p, w.buffer(), at, (uint32_t)(s.k - cx));
            }
        }
    };
    auto put_dy = [&](const RawDy<DT, PY> &r, uint32_t i) {
        u32x4 *to = ly[i & 1] + yt * UN + swizzled(yc, yt);
#pragma unroll
        for (uint32_t p = 0; p < PY; ++p) to[p * RY * UN] = r.piece(p, kTerms<DT> == 1 ? 0 : i / tiles);
    };
    auto put_x = [&](const RawX<FMT, PX> &r, uint32_t i) {
        u32x4 *to = lx[i & 1] + xt * UK + swizzled(2 * xc, xt);
#pragma unroll
        for (uint32_t p = 0; p < PX; ++p)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h) to[p * RX * UK + h] = r.piece(p, h);
    };

    f32x16 acc[FN][FK];
#pragma unroll
    for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j) acc[i][j] = f32x16{0};

    if (steps) {
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
        // Multiplies tile i out of its LDS buffer, puts tile i + 1 (register set
        // R) into the other one and loads tile i + 1 + SETS.  The barrier stands
        // before the last quarter of the products: by then the other waves'
        // pieces of tile i + 1 are in LDS, and its first fragments arrive behind
        // those products.
        auto step = [&](auto set, uint32_t i) {
            constexpr uint32_t R = decltype(set)::value, M = FN * FK;
            const uint32_t buf = i & 1;
            mend(ry[R], rx[R], i + 1);
            read(1, buf, 1);
            put_dy(ry[R], i + 1);
            multiply(0);
            interleave<M, 0, 8, 0>();
            load_dy(ry[R]);
            read(0, buf, 2);
            put_x(rx[R], i + 1);
            multiply(1);
            interleave<M, 32, 8, 8, true>();
            load_x(rx[R]);
            read(1, buf, 3);
            multiply(0);
            interleave<M, 0, 0, 8>();
            lds_barrier();
            read(0, buf ^ 1, 0);
            multiply(1);
            interleave<M, 0, 0, 0>();
        };
        auto run = [&](auto self, auto set, uint32_t i) {
            constexpr uint32_t R = decltype(set)::value;
            if (R && i >= steps) return;
            step(std::integral_constant<uint32_t, (R + 1) % SETS>(), i);
            if constexpr (R + 1 < SETS) self(self, std::integral_constant<uint32_t, R + 1>(), i + 1);
        };
        // tile 0 goes to LDS, tiles 1 .. SETS to the sets 1, .., SETS - 1, 0
        load_dy(ry[0]);
        load_x(rx[0]);
#pragma unroll
        for (uint32_t r = 1; r < SETS; ++r) {
            load_dy(ry[r]);
            load_x(rx[r]);
        }
        mend(ry[0], rx[0], 0);
        put_dy(ry[0], 0);
        put_x(rx[0], 0);
        load_dy(ry[0]);
        load_x(rx[0]);
        lds_barrier();
        read(0, 0, 0);
#pragma unroll 1
        for (uint32_t i = 0; i < steps; i += SETS) run(run, std::integral_constant<uint32_t, 0>(), i);
    }

    auto write = [&](auto o) {
        typedef typename Plain<decltype(o)::value>::type T;
        T *base = static_cast<T *>(out) + (uint64_t)blockIdx.y * s.n * s.k;  // a slice's partial sums (one slice: the output)
#pragma unroll
        for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
            for (uint32_t v = 0; v < 16; ++v) {
                const uint64_t n = n0 + (wn * FN + i) * 32 + v / 4 * 8 + lane / 32 * 4 + v % 4;
                if (n >= s.n) continue;
#pragma unroll
                for (uint32_t j = 0; j < FK; ++j) {
                    const uint64_t k = k0 + (wk * FK + j) * 32 + lane % 32;
                    T *p = base + n * s.ld_out + k;
                    if (k < s.k) *p = (T)(acc[i][j][v] + (add ? widen(*p) : 0.0f));
                }
            }
    };
    with_dtype(out_dtype, write);
}

// Joins the slices' partial sums, in their order.
template <int ODT>
__global__ __launch_bounds__(kThreads) void join_kernel(const float *__restrict__ part, uint32_t slices, uint64_t n,
                                                        uint64_t k, uint64_t ld_out,
                                                        typename Plain<ODT>::type *__restrict__ out, uint32_t add) {
    const uint64_t i = (uint64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n * k) return;
    float v = 0.0f;
    for (uint32_t s = 0; s < slices; ++s) v += part[s * n * k + i];
    typename Plain<ODT>::type *p = out + i / k * ld_out + i % k;
    *p = (typename Plain<ODT>::type)(v + (add ? widen(*p) : 0.0f));
}

// Tile sides: 256 (a wave's 128 x 128 part reads the least from LDS for each
// product), or 128 where that leaves workgroup slots empty.
uint64_t tiles_of(uint64_t n, uint64_t k, uint32_t side) { return ((n + side - 1) / side) * ((k + side - 1) / side); }

struct Plan {
    uint32_t side, slices, slice;
};

Plan plan_of(uint64_t t, uint64_t n, uint64_t k) {
    Plan p;
    const uint64_t steps = (t + kStep - 1) / kStep;
    p.side = tiles_of(n, k, 256) >= 192 ? 256 : 128;
    const uint64_t tiles = tiles_of(n, k, p.side);
    p.slices = 1;
    if (tiles < 256 && steps >= 8) p.slices = (uint32_t)std::min<uint64_t>(512 / tiles, steps / 4);
    p.slice = (uint32_t)((steps + p.slices - 1) / p.slices);
    return p;
}

}  // namespace

uint64_t wgrad_workspace(uint64_t t, uint64_t n, uint64_t k, int) {
    const Plan p = plan_of(t, n, k);
    return p.slices > 1 ? (uint64_t)p.slices * n * k * 4 : 0;
}

hipError_t launch_q8_weight_grad(const void *dy, int dtype, uint64_t ld_dy, uint64_t n_out, const pc_q8 *x, void *dw,
                                 int dw_dtype, uint64_t ld_dw, bool accumulate, void *ws, hipStream_t stream) {
    const uint64_t t = x->rows, n = n_out, k = x->cols;
    const Plan p = plan_of(t, n, k);
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
            p.side == 256 ? launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 4, 4, 1>)
                          : launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 2, 2, 2>);
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
            hipLaunchKernelGGL(join_kernel<ODT>, dim3((uint32_t)((n * k + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                               stream, static_cast<const float *>(ws), p.slices, n, k, ld_dw,
                               static_cast<typename Plain<ODT>::type *>(dw), (uint32_t)accumulate);
        });
    return hipGetLastError();
}

}  // namespace pc
