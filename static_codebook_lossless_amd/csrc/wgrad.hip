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

template <int DT> struct RawUnit { u32x4 w; };
template <> struct RawUnit<PC_F32> { u32x4 w, w2; };

template <int DT>
__device__ __forceinline__ void load_raw(const typename Plain<DT>::type *p, uint32_t n, RawUnit<DT> &r) {
    if (n == kUnit) {
        if constexpr (DT == PC_F32) {
            r.w = *reinterpret_cast<const u32x4_any4 *>(p);
            r.w2 = *reinterpret_cast<const u32x4_any4 *>(p + 4);
        } else {
            r.w = *reinterpret_cast<const u32x4_any2 *>(p);
        }
        return;
    }
    if constexpr (DT == PC_F32) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
            r.w[i] = i < n ? as_u32(p[i]) : 0u;
            r.w2[i] = 4 + i < n ? as_u32(p[4 + i]) : 0u;
        }
    } else {
        const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
            r.w[i] = (2 * i < n ? q[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)q[2 * i + 1] << 16 : 0u);
    }
}

// The four words (bf16 pairs) of a row's 8 columns.
template <int DT>
__device__ __forceinline__ void to_bf16(const RawUnit<DT> &r, uint32_t which, uint32_t w[4]) {
    if constexpr (DT == PC_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = r.w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            if constexpr (DT == PC_F16) {
                const uint32_t u = r.w[i];
                const f16x2 h = __builtin_bit_cast(f16x2, u);
                a = (float)h[0];
                b = (float)h[1];
            } else {
                a = as_f32(i < 2 ? r.w[2 * (i % 2)] : r.w2[2 * (i % 2)]);
                b = as_f32(i < 2 ? r.w[2 * (i % 2) + 1] : r.w2[2 * (i % 2) + 1]);
            }
            w[i] = __builtin_amdgcn_perm(term_bits(b, which), term_bits(a, which), 0x07060302u);
        }
    }
}

template <int FMT>
__device__ __forceinline__ void to_bf16(u32x2 s, float scale, uint32_t w[4]) {
    if constexpr (FMT == PC_Q8_E4M3) {
        w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s[0], scale, false));
        w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s[0], scale, true));
        w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s[1], scale, false));
        w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(s[1], scale, true));
    } else {
        float v[8];
        unit_values<FMT>(s, scale, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(as_u32(v[2 * i + 1]), as_u32(v[2 * i]), 0x07060302u);
    }
}

// 8 rows of 8 columns (bf16 pairs along the columns) to eight 16-byte pieces
// of 8 rows, written to LDS `distance` pieces apart.
__device__ __forceinline__ void put_transposed(const uint32_t w[8][4], u32x4 *to, uint32_t distance) {
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

// Column of the piece at place p of a tile of B columns: pieces are placed so
// that neighbouring lanes, which hold neighbouring blocks of 8 columns, write
// neighbouring pieces.
template <uint32_t B>
__device__ __forceinline__ uint32_t column_at(uint32_t p) {
    return (p % (B / 8)) * 8 + p / (B / 8);
}

struct Shape {
    uint64_t t, n, k;       // rows, n_out, n_in
    uint64_t ld_dy, ld_out;
    uint64_t slice;         // rows of one slice of t (a multiple of kStep)
    uint32_t tiles_n, tiles_k;
};

template <int DT, int FMT, int ODT, uint32_t WN, uint32_t WK, uint32_t FN, uint32_t FK>
__global__ __launch_bounds__(kThreads) void wgrad_kernel(const typename Plain<DT>::type *__restrict__ dy,
                                                         const uint8_t *__restrict__ sym,
                                                         const uint8_t *__restrict__ scale, uint64_t ld_sym,
                                                         uint64_t ld_scale, Shape s,
                                                         typename Plain<ODT>::type *__restrict__ out, uint32_t add) {
    constexpr uint32_t BN = WN * FN * 32, BK = WK * FK * 32;
    static_assert(WN * WK * kWave == kThreads, "waves");
    __shared__ u32x4 ly[kStep / 8 * BN];
    __shared__ u32x4 lx[kStep / 8 * BK];
    const uint32_t tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const uint32_t wn = wave / WK, wk = wave % WK;
    const uint32_t tile = blockIdx.x;
    const uint64_t n0 = (uint64_t)(tile / s.tiles_k) * BN, k0 = (uint64_t)(tile % s.tiles_k) * BK;
    const uint64_t t_begin = (uint64_t)blockIdx.y * s.slice, t_end = min(s.t, t_begin + s.slice);
    out += (uint64_t)blockIdx.y * s.n * s.k;  // a slice's own partial sums (one slice: the output)

    f32x16 acc[FN][FK];
#pragma unroll
    for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
        for (uint32_t j = 0; j < FK; ++j) acc[i][j] = f32x16{0};

    for (uint32_t which = 0; which < kTerms<DT>; ++which) {
        for (uint64_t t0 = t_begin; t0 < t_end; t0 += kStep) {
            __syncthreads();
            for (uint32_t b = tid; b < kStep / 8 * BN / 8; b += kThreads) {
                const uint32_t tb = b / (BN / 8), l = b % (BN / 8);
                const uint64_t c = n0 + l * 8;
                const uint32_t n = c < s.n ? (uint32_t)min((uint64_t)8, s.n - c) : 0;
                uint32_t w[8][4];
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    RawUnit<DT> r = {};
                    const uint64_t t = t0 + tb * 8 + i;
                    if (n && t < t_end) load_raw<DT>(dy + t * s.ld_dy + c, n, r);
                    to_bf16<DT>(r, which, w[i]);
                }
                put_transposed(w, ly + tb * BN + l, BN / 8);
            }
            for (uint32_t b = tid; b < kStep / 8 * BK / 8; b += kThreads) {
                const uint32_t tb = b / (BK / 8), l = b % (BK / 8);
                const uint64_t c = k0 + l * 8;
                const uint32_t n = c < s.k ? (uint32_t)min((uint64_t)8, s.k - c) : 0;
                uint32_t w[8][4];
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) {
                    u32x2 q = {0, 0};
                    uint32_t code = 127;
                    const uint64_t t = t0 + tb * 8 + i;
                    if (n && t < t_end) {
                        q = load_symbols(sym + t * ld_sym + c, n);
                        code = scale[t * ld_scale + c / kGroup];
                    }
                    to_bf16<FMT>(q, scale_of(code), w[i]);
                }
                put_transposed(w, lx + tb * BK + l, BK / 8);
            }
            __syncthreads();
#pragma unroll
            for (uint32_t kk = 0; kk < kStep / 16; ++kk) {
                bf16x8 a[FN], b[FK];
                const uint32_t tb = kk * 2 + lane / 32;
#pragma unroll
                for (uint32_t i = 0; i < FN; ++i)
                    a[i] = __builtin_bit_cast(bf16x8, ly[tb * BN + (wn * FN + i) * 32 + lane % 32]);
#pragma unroll
                for (uint32_t j = 0; j < FK; ++j)
                    b[j] = __builtin_bit_cast(bf16x8, lx[tb * BK + (wk * FK + j) * 32 + lane % 32]);
#pragma unroll
                for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
                    for (uint32_t j = 0; j < FK; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
            }
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < FN; ++i)
#pragma unroll
        for (uint32_t v = 0; v < 16; ++v) {
            const uint32_t r = v / 4 * 8 + lane / 32 * 4 + v % 4;
            const uint64_t n = n0 + column_at<BN>((wn * FN + i) * 32 + r);
            if (n >= s.n) continue;
#pragma unroll
            for (uint32_t j = 0; j < FK; ++j) {
                const uint64_t k = k0 + column_at<BK>((wk * FK + j) * 32 + lane % 32);
                if (k >= s.k) continue;
                typename Plain<ODT>::type *p = out + n * s.ld_out + k;
                const float old = add ? widen(*p) : 0.0f;
                *p = (typename Plain<ODT>::type)(acc[i][j][v] + old);
            }
        }
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

constexpr uint32_t kTileN = 128, kTileK = 128;

uint32_t slices_of(uint64_t t, uint64_t n, uint64_t k) {
    const uint64_t tiles = ((n + kTileN - 1) / kTileN) * ((k + kTileK - 1) / kTileK);
    const uint64_t steps = (t + kStep - 1) / kStep;
    if (tiles >= 256 || steps < 8) return 1;
    return (uint32_t)std::min<uint64_t>(512 / tiles, steps / 4);
}

}  // namespace

uint64_t wgrad_workspace(uint64_t t, uint64_t n, uint64_t k, int) {
    const uint32_t slices = slices_of(t, n, k);
    return slices > 1 ? (uint64_t)slices * n * k * 4 : 0;
}

hipError_t launch_q8_weight_grad(const void *dy, int dtype, uint64_t ld_dy, uint64_t n_out, const pc_q8 *x, void *dw,
                                 int dw_dtype, uint64_t ld_dw, bool accumulate, void *ws, hipStream_t stream) {
    const uint64_t t = x->rows, n = n_out, k = x->cols;
    const uint32_t slices = slices_of(t, n, k);
    Shape s = {t, n, k, ld_dy, slices > 1 ? k : ld_dw, 0, (uint32_t)((n + kTileN - 1) / kTileN),
               (uint32_t)((k + kTileK - 1) / kTileK)};
    const uint64_t steps = (t + kStep - 1) / kStep;
    s.slice = (steps + slices - 1) / slices * kStep;
    const dim3 grid(s.tiles_n * s.tiles_k, slices);
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        with_dtype(slices > 1 ? (int)PC_F32 : dw_dtype, [&](auto o) {
            constexpr int ODT = decltype(o)::value;
            auto launch = [&](auto kern) {
                hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, stream,
                                   static_cast<const typename Plain<DT>::type *>(dy), x->sym, x->scale, x->ld_sym,
                                   x->ld_scale, s, static_cast<typename Plain<ODT>::type *>(slices > 1 ? ws : dw),
                                   (uint32_t)(accumulate && slices == 1));
            };
            x->format == PC_Q8_E4M3 ? launch(wgrad_kernel<DT, PC_Q8_E4M3, ODT, 2, 2, 2, 2>)
                                    : launch(wgrad_kernel<DT, PC_Q8_INT8, ODT, 2, 2, 2, 2>);
        });
    });
    if (slices > 1)
        with_dtype(dw_dtype, [&](auto o) {
            constexpr int ODT = decltype(o)::value;
            hipLaunchKernelGGL(join_kernel<ODT>, dim3((uint32_t)((n * k + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                               stream, static_cast<const float *>(ws), slices, n, k, ld_dw,
                               static_cast<typename Plain<ODT>::type *>(dw), (uint32_t)accumulate);
        });
    return hipGetLastError();
}

}  // namespace pc
