// Weight gradient of a projection whose input was stored in 8 bits:
//   dW[n][k] = sum over t of dy[t][n] x[t][k].
//
// A matrix product whose long axis t is the row axis of both operands.  The
// matrix instruction wants 8 consecutive t of one column in a lane, so a lane
// loads blocks of 8 rows by 8 columns, turns x's symbols into bf16 (exact:
// the scales are powers of two), transposes the block with byte permutes and
// writes it to LDS as eight 16-byte pieces, one for each column.
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace pc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kThreads = 256;
constexpr uint32_t kStep = 64;               // rows t of one LDS tile
constexpr uint32_t kBlocks = kStep / 8;      // blocks of 8 rows in it

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
// past `bytes` reads 0.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer make_buffer(const void *p, uint64_t bytes) {
    const uint64_t at = uniform64(reinterpret_cast<uint64_t>(p));
    const uint32_t most = uniform((uint32_t)min(bytes, (uint64_t)0xFFFFFFFFu));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void *>(at), 0, (int)most, 0x00020000);
}

// A block of 8 rows of 8 columns as loaded: rows of 8 elements of dy, or of
// 8 symbols of x with the rows' scale codes.
template <int DT> struct RawDy {
    static constexpr uint32_t kWords = DT == PC_F32 ? 2 : 1;
    u32x4 w[8][kWords];

    __device__ __forceinline__ void load(Buffer b, uint32_t at, uint32_t row) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (uint32_t k = 0; k < kWords; ++k)
                w[i][k] = __builtin_amdgcn_raw_buffer_load_b128(b, at + i * row + 16 * k, 0, 0);
    }
    // the first n elements of row i, each by itself
    __device__ __forceinline__ void load_single(int i, Buffer b, uint32_t at, uint32_t n) {
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {
            if constexpr (DT == PC_F32) {
                w[i][c / 4][c % 4] = c < n ? __builtin_amdgcn_raw_buffer_load_b32(b, at + 4 * c, 0, 0) : 0u;
            } else {
                const uint32_t e = c < n ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(b, at + 2 * c, 0, 0) : 0u;
                w[i][0][c / 2] = c % 2 ? w[i][0][c / 2] | e << 16 : e;
            }
        }
    }
    // bf16 pairs of row i
    __device__ __forceinline__ void words(int i, uint32_t which, uint32_t out[4]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (DT == PC_BF16) {
                out[k] = w[i][0][k];
            } else {
                float a, b;
                if constexpr (DT == PC_F16) {
                    const uint32_t u = w[i][0][k];
                    const f16x2 h = __builtin_bit_cast(f16x2, u);
                    a = (float)h[0];
                    b = (float)h[1];
                } else {
                    a = as_f32(w[i][(2 * k) / 4][(2 * k) % 4]);
                    b = as_f32(w[i][(2 * k) / 4][(2 * k) % 4 + 1]);
                }
                out[k] = __builtin_amdgcn_perm(term_bits(b, which), term_bits(a, which), 0x07060302u);
            }
        }
    }
};

template <int FMT> struct RawX {
    u32x2 w[8];
    uint32_t code[8];

    __device__ __forceinline__ void load(Buffer b, uint32_t at, uint32_t row, Buffer codes, uint32_t code_at,
                                         uint32_t code_row) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            w[i] = __builtin_amdgcn_raw_buffer_load_b64(b, at + i * row, 0, 0);
            code[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(codes, code_at + i * code_row, 0, 0);
        }
    }
    __device__ __forceinline__ void load_single(int i, Buffer b, uint32_t at, uint32_t n) {
        w[i] = u32x2{0, 0};
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c)
            if (c < n) w[i][c / 4] |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(b, at + c, 0, 0) << (8 * (c % 4));
    }
    __device__ __forceinline__ void words(int i, uint32_t, uint32_t out[4]) const {
        const float s = scale_of(code[i]);
        if constexpr (FMT == PC_Q8_E4M3) {
            out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][0], s, false));
            out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][0], s, true));
            out[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][1], s, false));
            out[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i][1], s, true));
        } else {
            float v[8];
            unit_values<FMT>(w[i], s, v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                out[k] = __builtin_amdgcn_perm(as_u32(v[2 * k + 1]), as_u32(v[2 * k]), 0x07060302u);
        }
    }
};

// A block in LDS: eight 16-byte pieces, one for each column with its 8 rows,
// `distance` pieces apart.
template <class RAW>
__device__ __forceinline__ void put_transposed(const RAW &r, uint32_t which, u32x4 *to, uint32_t distance) {
    uint32_t w[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) r.words(i, which, w[i]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        u32x4 even, odd;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            even[i] = __builtin_amdgcn_perm(w[2 * i + 1][c], w[2 * i][c], 0x05040100u);
            odd[i] = __builtin_amdgcn_perm(w[2 * i + 1][c], w[2 * i][c], 0x07060302u);
        }
        to[(2 * c) * distance] = even;
        to[(2 * c + 1) * distance] = odd;
    }
}

// Where a tile of B columns keeps its pieces: block l of 8 columns is one
// lane's, and the pieces of its column c lie at c * (B / 8) + l, so that
// neighbouring lanes write, and later read, neighbouring pieces.  A wave with
// F fragments of 32 columns takes the columns c of its share of every block;
// its fragment j, lane r has column c = column_in_block(j, r) of block r % (B / 8),
// so that a lane's fragments are neighbouring columns of the result.
template <uint32_t B, uint32_t F>
__device__ __forceinline__ uint32_t column_in_block(uint32_t wave, uint32_t j, uint32_t r) {
    return wave * (F * 256 / B) + r / (B / 8) * F + j;
}

struct Shape {
    uint64_t t, n, k;  // rows, n_out, n_in
    uint64_t ld_dy, ld_sym, ld_scale, ld_out;
    uint32_t slice;    // LDS tiles of one slice of t
    uint32_t tiles_n, tiles_k;
};

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The order of a step's instructions up to its barrier: between two matrix
// instructions (of a step's three quarters of M each) a share of everything
// else, so that the matrix cores never wait for a run of other work.
template <uint32_t M>
__device__ __forceinline__ void interleave() {
    if constexpr (M == 16) {
#pragma unroll
        for (uint32_t m = 0; m < 3 * M; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                    // matrix
            if (m % M < 8) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                     // LDS read
            __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);                                    // vector
            if (m >= 4 && m % 2 == 1 && m < 40) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);  // LDS write
            if (m >= 20 && m < 28) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);             // load
            if (m >= 40) __builtin_amdgcn_sched_group_barrier(0x020, 2, 0);
        }
    }
}
template <uint32_t M, uint32_t R>
__device__ __forceinline__ void interleave_tail() {
    if constexpr (M == 16) {
#pragma unroll
        for (uint32_t m = 0; m < R; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, M - R, 0);
    }
}

template <int DT, int FMT, bool RAGGED, uint32_t WN, uint32_t WK, uint32_t FN, uint32_t FK>
__global__ __launch_bounds__(WN *WK *kWave, 1) void wgrad_kernel(const typename Plain<DT>::type *__restrict__ dy,
                                                                 const uint8_t *__restrict__ sym,
                                                                 const uint8_t *__restrict__ scale, Shape s,
                                                                 void *__restrict__ out, int out_dtype, uint32_t add) {
    constexpr uint32_t BN = WN * FN * 32, BK = WK * FK * 32, NT = WN * WK * kWave;
    constexpr uint32_t kElem = sizeof(typename Plain<DT>::type);
    // blocks of the two tiles: one of each for every lane, or one for every lane of either half
    constexpr bool kBoth = kBlocks * BN / 8 == NT && kBlocks * BK / 8 == NT;
    static_assert(kBoth || (kBlocks * BN / 8 == NT / 2 && kBlocks * BK / 8 == NT / 2), "blocks");
    __shared__ u32x4 ly[2][kBlocks * BN];
    __shared__ u32x4 lx[2][kBlocks * BK];
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
    const uint32_t wn = wave / WK, wk = wave % WK;
    const uint64_t n0 = (uint64_t)(blockIdx.x / s.tiles_k) * BN, k0 = (uint64_t)(blockIdx.x % s.tiles_k) * BK;
    const uint32_t all = (uint32_t)((s.t + kStep - 1) / kStep);
    const uint32_t first = min(all, blockIdx.y * s.slice), tiles = min(all - first, s.slice);
    const uint32_t steps = tiles * kTerms<DT>;

    const bool has_dy = kBoth || wave < WN * WK / 2, has_x = kBoth || !has_dy;
    const uint32_t b = kBoth ? tid : tid % (NT / 2);
    const uint32_t yl = b % (BN / 8), yt = b / (BN / 8), xl = b % (BK / 8), xt = b / (BK / 8);
    const uint32_t y_row = (uint32_t)s.ld_dy * kElem, x_row = (uint32_t)s.ld_sym, c_row = (uint32_t)s.ld_scale;
    const uint32_t y_at = yt * 8 * y_row + yl * 8 * kElem, x_at = xt * 8 * x_row + xl * 8;
    const uint32_t c_at = xt * 8 * c_row + xl / kUnitsPerGroup;
    RawDy<DT> ry;
    RawX<FMT> rx;

    // Rows from tile i's first to the tensor's last; none past the last tile.
    auto rows_of = [&](uint32_t i, uint64_t &t0) -> uint64_t {
        t0 = (uint64_t)(first + (kTerms<DT> == 1 ? i : i % tiles)) * kStep;
        return i < steps ? s.t - t0 : 0;
    };
    // Loads tile i (past the last: zeros) into registers.
    auto load_dy = [&](uint32_t i) {
        uint64_t t0;
        const uint64_t rows = rows_of(i, t0), bytes = rows * y_row - (s.ld_dy - (s.n - n0)) * kElem;
        if (has_dy) ry.load(make_buffer(dy + t0 * s.ld_dy + n0, rows ? bytes : 0), y_at, y_row);
    };
    auto load_x = [&](uint32_t i) {
        uint64_t t0;
        const uint64_t rows = rows_of(i, t0), bytes = rows * x_row - (s.ld_sym - (s.k - k0));
        const uint64_t code_bytes = rows * c_row - (s.ld_scale - ((s.k + kGroup - 1) / kGroup - k0 / kGroup));
        if (has_x)
            rx.load(make_buffer(sym + t0 * s.ld_sym + k0, rows ? bytes : 0), x_at, x_row,
                    make_buffer(scale + t0 * s.ld_scale + k0 / kGroup, rows ? code_bytes : 0), c_at, c_row);
    };
    // A block that sticks out of the tensor's last row (widths that are no
    // multiple of 8): its load may have dropped elements that are inside.
    // Only the last tiles of t meet one.
    auto mend = [&](uint32_t i) {
        if constexpr (!RAGGED) return;
        uint64_t t0;
        const uint64_t rows = rows_of(i, t0);
        if (rows == 0 || rows >= kStep + 8) return;
        const uint64_t cy = n0 + yl * 8, cx = k0 + xl * 8;
        if (has_dy && cy < s.n && cy + 8 > s.n) {
            const uint64_t bytes = ((rows - 1) * s.ld_dy + (s.n - n0)) * kElem;
            const Buffer buf = make_buffer(dy + t0 * s.ld_dy + n0, bytes);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t at = y_at + r * y_row;
                if (at < bytes && at + 8 * kElem > bytes) ry.load_single(r, buf, at, (uint32_t)(s.n - cy));
            }
        }
        if (has_x && cx < s.k && cx + 8 > s.k) {
            const uint64_t bytes = (rows - 1) * s.ld_sym + (s.k - k0);
            const Buffer buf = make_buffer(sym + t0 * s.ld_sym + k0, bytes);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const uint32_t at = x_at + r * x_row;
                if (at < bytes && at + 8 > bytes) rx.load_single(r, buf, at, (uint32_t)(s.k - cx));
            }
        }
    };
    auto put_dy = [&](uint32_t i, uint32_t buf) {
        if (has_dy) put_transposed(ry, kTerms<DT> == 1 ? 0 : i / tiles, ly[buf] + yt * BN + yl, BN / 8);
    };
    auto put_x = [&](uint32_t buf) {
        if (has_x) put_transposed(rx, 0, lx[buf] + xt * BK + xl, BK / 8);
    };

    f32x16 acc[FN][FK];
#pragma unroll
    for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j) acc[i][j] = f32x16{0};

    if (steps) {
        const uint32_t r = lane % 32, half = lane / 32;
        uint32_t a_at[FN], b_at[FK];
#pragma unroll
        for (uint32_t i = 0; i < FN; ++i)
            a_at[i] = half * BN + column_in_block<BN, FN>(wn, i, r) * (BN / 8) + r % (BN / 8);
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j)
            b_at[j] = half * BK + column_in_block<BK, FK>(wk, j, r) * (BK / 8) + r % (BK / 8);
        bf16x8 fa[2][FN], fb[2][FK];
        auto read = [&](uint32_t which, uint32_t buf, uint32_t kk) {
#pragma unroll
            for (uint32_t i = 0; i < FN; ++i) fa[which][i] = __builtin_bit_cast(bf16x8, ly[buf][a_at[i] + kk * 2 * BN]);
#pragma unroll
            for (uint32_t j = 0; j < FK; ++j) fb[which][j] = __builtin_bit_cast(bf16x8, lx[buf][b_at[j] + kk * 2 * BK]);
        };
        auto multiply = [&](uint32_t which) {
#pragma unroll
            for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
                for (uint32_t j = 0; j < FK; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[which][i], fb[which][j], acc[i][j], 0, 0, 0);
        };
        // Multiplies tile i out of LDS buffer P, puts tile i + 1 into the other
        // one and loads tile i + 2.  The barrier stands before the last quarter
        // of the products: by then the other waves' pieces of tile i + 1 are
        // in LDS, and its first fragments arrive behind those products.
        auto step = [&](auto parity, uint32_t i) {
            constexpr uint32_t P = decltype(parity)::value, Q = P ^ 1;
            mend(i + 1);
            read(1, P, 1);
            put_dy(i + 1, Q);
            multiply(0);
            load_dy(i + 2);
            read(0, P, 2);
            put_x(Q);
            multiply(1);
            load_x(i + 2);
            read(1, P, 3);
            multiply(0);
            interleave<FN * FK>();
            lds_barrier();
            read(0, Q, 0);
            multiply(1);
            interleave_tail<FN * FK, FN + FK>();
        };
        load_dy(0);
        load_x(0);
        mend(0);
        put_dy(0, 0);
        put_x(0);
        load_dy(1);
        load_x(1);
        lds_barrier();
        read(0, 0, 0);
        for (uint32_t i = 0; i < steps; i += 2) {
            step(std::integral_constant<uint32_t, 0>(), i);
            if (i + 1 < steps) step(std::integral_constant<uint32_t, 1>(), i + 1);
        }
    }

    const uint32_t r0 = lane % 32;
    const uint64_t k = k0 + r0 % (BK / 8) * 8 + column_in_block<BK, FK>(wk, 0, r0);
    auto write = [&](auto o) {
        typedef typename Plain<decltype(o)::value>::type T;
        T *base = static_cast<T *>(out) + (uint64_t)blockIdx.y * s.n * s.k;  // a slice's partial sums (one slice: the output)
#pragma unroll
        for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
            for (uint32_t v = 0; v < 16; ++v) {
                const uint32_t r = v / 4 * 8 + lane / 32 * 4 + v % 4;
                const uint64_t n = n0 + r % (BN / 8) * 8 + column_in_block<BN, FN>(wn, i, r);
                if (n >= s.n) continue;
                T *p = base + n * s.ld_out + k;
                if (k + FK <= s.k && !add) {
                    typedef T vec __attribute__((ext_vector_type(FK)));
                    typedef vec any __attribute__((aligned(sizeof(T))));
                    vec u;
#pragma unroll
                    for (uint32_t j = 0; j < FK; ++j) u[j] = (T)acc[i][j][v];
                    *reinterpret_cast<any *>(p) = u;
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < FK; ++j)
                        if (k + j < s.k) p[j] = (T)(acc[i][j][v] + (add ? widen(p[j]) : 0.0f));
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
    const dim3 grid(s.tiles_n * s.tiles_k, p.slices);
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
            p.side == 256 ? launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 4, 4>)
                          : launch(wgrad_kernel<DT, FMT, RAGGED, 2, 2, 2, 2>);
        };
        auto by_format = [&](auto r) {
            if (x->format == PC_Q8_E4M3) by_side(std::integral_constant<int, PC_Q8_E4M3>(), r);
            else by_side(std::integral_constant<int, PC_Q8_INT8>(), r);
        };
        if (n % 8 || k % 8) by_format(std::true_type());
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
