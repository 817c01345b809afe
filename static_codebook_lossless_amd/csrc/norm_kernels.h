// Root-mean-square norm with what a residual block does around it: dropout of
// the block's output, the residual's addition, the norm, and the norm's output
// stored in 8 bits; and the backward pass of all of that.
//
//   h = round(res + mask(x)),  r = (mean(h^2) + eps)^-1/2,  y = h r w
//   d = r (g - n mean(g n)) + d_sum,  g = dy w,  n = h r
//   d_res = d,  d_x = mask(d),  d_w = sum over rows of dy n
#pragma once

#include <type_traits>

#include "norm.h"

namespace pc {
namespace {

constexpr uint32_t kMaxWaves = kMaxThreads / kWave;

// Histogram copies of the counting form, as in the store.
constexpr uint32_t kCopies = 8;
constexpr uint32_t kCopyStride = 257;
constexpr uint32_t kBins = kMaxWaves * kCopies * kCopyStride;

// 8 elements of a type known at run time.
struct AnyUnit { u32x4 w[2]; };

__device__ __forceinline__ AnyUnit load_any(int kind, const void *p, uint64_t at, uint32_t n) {
    AnyUnit r = {};
    if (kind == PC_F32) {
        const RawUnit<PC_F32> u = load_raw<PC_F32>(static_cast<const float *>(p) + at, n);
        r.w[0] = u.w[0];
        r.w[1] = u.w[1];
    } else {  // both 16-bit types load alike
        r.w[0] = load_raw<PC_F16>(static_cast<const _Float16 *>(p) + at, n).w[0];
    }
    return r;
}

__device__ __forceinline__ void widen_any(int kind, const AnyUnit &r, float v[8]) {
    if (kind == PC_F32) {
        RawUnit<PC_F32> u;
        u.w[0] = r.w[0];
        u.w[1] = r.w[1];
        widen_unit<PC_F32>(u, v);
    } else if (kind == PC_F16) {
        RawUnit<PC_F16> u;
        u.w[0] = r.w[0];
        widen_unit<PC_F16>(u, v);
    } else {
        RawUnit<PC_BF16> u;
        u.w[0] = r.w[0];
        widen_unit<PC_BF16>(u, v);
    }
}

__device__ __forceinline__ void store_any(int kind, void *p, uint64_t at, uint32_t n, const float v[8]) {
    if (kind == PC_F32) store_unit<PC_F32>(static_cast<float *>(p) + at, n, v);
    else if (kind == PC_F16) store_unit<PC_F16>(static_cast<_Float16 *>(p) + at, n, v);
    else store_unit<PC_BF16>(static_cast<__bf16 *>(p) + at, n, v);
}

template <int DT>
__device__ __forceinline__ float rounded(float v) {
    return widen((typename Plain<DT>::type)v);
}

// How many of a unit's places lie before the row's end.  WHOLE: widths are
// multiples of 8, so all or none, and the code for parts of a unit is left out
// (with it a kernel takes half as many registers more).
template <bool WHOLE>
__device__ __forceinline__ uint32_t places(uint32_t cols, uint32_t col) {
    if constexpr (WHOLE) return col < cols ? kUnit : 0;
    else return count_before(cols, col, kUnit);
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) { return v + as_f32(dpp_u32<CTRL>(as_u32(v))); }

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    const u32x2 o = {dpp_u32<CTRL>(u[0]), dpp_u32<CTRL>(u[1])};
    return v + __builtin_bit_cast(double, o);
}

// v of the lane 16 further on, or back, in a half of the wave: of two registers
// that hold the same, odd rows of 16 lanes of one change places with even ones
// of the other.
__device__ __forceinline__ uint32_t other_row(uint32_t v) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
}

__device__ __forceinline__ float other_row(float v) { return as_f32(other_row(as_u32(v))); }

__device__ __forceinline__ double other_row(double v) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{other_row(u[0]), other_row(u[1])});
}

__device__ __forceinline__ float from_lane(float v, int lane) {
    return as_f32((uint32_t)__builtin_amdgcn_readlane((int)as_u32(v), lane));
}

__device__ __forceinline__ double from_lane(double v, int lane) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    const u32x2 o = {(uint32_t)__builtin_amdgcn_readlane((int)u[0], lane),
                     (uint32_t)__builtin_amdgcn_readlane((int)u[1], lane)};
    return __builtin_bit_cast(double, o);
}

// The lanes that share a row: a part of a wave (SUB of 16 or 32) or whole waves
// (SUB of 64, a.team lanes).
template <uint32_t SUB>
struct Team {
    uint32_t lanes, waves, at, index, count;  // at: the lane's place; index: the team's in the workgroup
    __device__ __forceinline__ explicit Team(uint32_t team) {
        const uint32_t tid = threadIdx.x;
        lanes = SUB < kWave ? SUB : team;
        waves = lanes / kWave;
        if constexpr (SUB < kWave) {
            index = tid / SUB;
            at = tid % SUB;
        } else {
            index = uniform(tid / kWave) / waves;
            at = tid - index * lanes;
        }
        count = blockDim.x / lanes;
    }
};

// The sum over a team, the same in all its lanes.  `part` alternates between
// two areas from call to call, so one barrier a call is enough: what a call
// writes was last read before the barrier of the call between.
template <uint32_t SUB, class T>
__device__ __forceinline__ T team_sum(const Team<SUB> &team, T v, T *part) {
    v = dpp_add<0xB1>(v);   // the neighbour in the pair
    v = dpp_add<0x4E>(v);   // the other pair
    v = dpp_add<0x141>(v);  // the other half of 8
    v = dpp_add<0x140>(v);  // the other half of 16
    if constexpr (SUB == 16) return v;
    if constexpr (SUB == 32) return v + other_row(v);
    v = (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
    if (team.waves == 1) return v;
    if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
    __syncthreads();
    const uint32_t first = team.index * team.waves;
    T s = part[first];
    for (uint32_t i = 1; i < team.waves; ++i) s += part[first + i];
    return s;
}

// Hides from the compiler what is in registers, so that it widens the elements
// anew after a wait and does not keep them wide meanwhile.
template <class V>
__device__ __forceinline__ void forget(V &v) { asm volatile("" : "+v"(v)); }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

// r = (mean + eps)^-1/2.  Squares are summed in 64 bits, where those of all
// 32-bit numbers fit; a vector instruction takes as long as in 32 bits.  The
// hardware's estimate has 23 bits, which a Newton step doubles.
__device__ __forceinline__ double rstd_of(const NormArgs &a, double squares) {
    const double m = squares * a.per_col + a.eps, r = __builtin_amdgcn_rsq(m);
    return m == __builtin_inf() ? 0.0 : r * (1.5 - 0.5 * m * r * r);
}

// A number as 32 bits hold it, with an odd last bit where they do not hold all
// of it: rounding that to fewer bits rounds the number itself.
__device__ __forceinline__ float rounded_to_odd(double v) {
    const float s = (float)v;
    const double rest = v - (double)s;
    uint32_t u = as_u32(s);
    if (rest != 0.0 && !(u & 1) && s != 0.0f && (u & 0x7F800000u) != 0x7F800000u) u += (rest > 0.0) == (s > 0.0f) ? 1 : -1;
    return as_f32(u);
}

template <int DT>
__device__ __forceinline__ RawUnit<DT> to_raw(const float v[8]) {
    RawUnit<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == PC_F32 ? 8 : 4); ++i) {
        if constexpr (DT == PC_F32) {
            r.w[i / 4][i % 4] = as_u32(v[i]);
        } else {
            typedef typename Plain<DT>::type t2 __attribute__((ext_vector_type(2)));
            const f32x2 f = {v[2 * i], v[2 * i + 1]};
            r.w[0][i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, t2));
        }
    }
    return r;
}

// The first n (1..8) elements of a unit as they are.
template <int DT>
__device__ __forceinline__ void store_raw(typename Plain<DT>::type *p, uint32_t n, const RawUnit<DT> &r) {
    float v[8];
    widen_unit<DT>(r, v);
    store_unit<DT>(p, n, v);
}

// h of a unit, as the sum's type holds it.
template <int DT, int RT>
__device__ __forceinline__ RawUnit<RT> block_sum(const NormArgs &a, const MaskKey &key, const RawUnit<DT> &x,
                                                 const RawUnit<RT> &res, uint64_t row, uint32_t col) {
    float h[8];
    widen_unit<DT>(x, h);
    if (a.mask.below) drop_unit(a.mask, key, row, col, h);
    if (a.res) {
        float r[8];
        widen_unit<RT>(res, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
    return to_raw<RT>(h);
}

// `again` forms the unit's h and weights once more: they are not kept for the
// few units that need them.
//
// y is (h r) w in 32 bits, off by 3.1 2^-24, as long as r and h r are normal
// numbers.  r of a row above 2^126 has fewer digits, and a small h in a row of
// large ones leaves h r below 2^-126, off by 2^-150, and y by that times the
// weight (FAINT: no sum in f16 has either).  Units where it could be seen are
// formed in 64 bits: from a weight of 2^24 on, which makes it 2^-126, and for
// what is stored from one of 1 on where the group's scale is small (at those
// above kFaintCode it is at most 2^-34 of the scale, which `unsure` covers
// beside the 3.1 2^-24).
constexpr float kNormal = 0x1p-126f, kFaintWeight = 0x1p24f;
constexpr uint32_t kFaintCode = 34;

template <bool COUNT, bool FAINT, class AGAIN>
__device__ __forceinline__ void norm_unit(const NormArgs &a, uint64_t row, uint32_t col, uint32_t n, double rstd,
                                          const float w[8], const float h[8], uint32_t *bins, AGAIN &&again) {
    float y[8];
    const float r = (float)rstd;
    float heavy = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = h[i] * r * w[i];
        heavy = fmaxf(heavy, fabsf(w[i]));
    }
    const bool faint = FAINT && (heavy > kFaintWeight || r < kNormal), above_1 = FAINT && heavy > 1.0f;
    const bool plain = a.y && !a.y_stored && n, e4m3 = a.format == PC_Q8_E4M3;
    if (plain) store_any(a.y_kind, a.y, row * a.ld_y + col, n, y);
    // y is off by 3.1 2^-24 at most; where that could change what is stored (one unit of
    // a wave in 150 or so), the wave forms it again in 64 bits, so that nothing but
    // the rounding to 8 bits shows
    bool unsure = faint;
    uint32_t code = 0;
    u32x2 s = {0, 0};
    if (a.sym) {
        bool may;
        s = e4m3 ? to_stored<PC_Q8_E4M3, true>(y, code, &may) : to_stored<PC_Q8_INT8, true>(y, code, &may);
        unsure |= may || (above_1 && code <= kFaintCode);
    }
    if (__ballot(unsure)) {
        float h2[8], w2[8];
        again(h2, w2);
        double v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (double)h2[i] * rstd * (double)w2[i];
        if (faint && plain) {  // once more, over the first
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (float)v[i];
            store_any(a.y_kind, a.y, row * a.ld_y + col, n, y);
        }
        if (a.sym) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = rounded_to_odd(v[i]);
            s = e4m3 ? to_stored<PC_Q8_E4M3>(y, code) : to_stored<PC_Q8_INT8>(y, code);
        }
    }
    if (!a.sym) return;
    if (n) {
        store_symbols(a.sym + row * a.cols + col, n, s);
        if (col % kGroup == 0) a.scale[row * a.groups + col / kGroup] = (uint8_t)code;
        if (a.y && a.y_stored) {
            float v[8];
            if (e4m3) unit_values<PC_Q8_E4M3>(s, scale_of(code), v);
            else unit_values<PC_Q8_INT8>(s, scale_of(code), v);
            store_any(a.y_kind, a.y, row * a.ld_y + col, n, v);
        }
    }
    if constexpr (COUNT) {
#pragma unroll
        for (uint32_t i = 0; i < kUnit; ++i)
            if (i < n) atomicAdd(&bins[(s[i / 4] >> (8 * (i % 4))) & 0xFF], 1u);
    }
}

// A team takes a row into its registers, so that x, the residual and the mask's
// numbers are read and formed once.  U units a lane; LONG: rows of more than
// team * U units, read in turns.  8192 x 8192 bf16 with a residual and a mask,
// to e4m3 and the stored y: 102-103 us, 5.9 TB/s beside vector work in 84% of the
// cycles; 8192 x 4096 without the mask, to e4m3 and y: 57 us, 5.3 TB/s.  Bounds
// on waves for the registers are not asked for: the compiler then spills (150 us).
template <int DT, int RT, int U, uint32_t SUB, bool COUNT, bool LONG, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ double part[2][kMaxWaves];
    __shared__ uint32_t all_bins[COUNT ? kBins : 1];
    const uint32_t tid = threadIdx.x;
    const Team<SUB> team(a.team);
    const TX *x = static_cast<const TX *>(a.x);
    const TR *res = static_cast<const TR *>(a.res);
    TR *sum = static_cast<TR *>(a.sum);
    uint32_t *bins = all_bins;
    if constexpr (COUNT) {
        for (uint32_t i = tid; i < kBins; i += blockDim.x) all_bins[i] = 0;
        __syncthreads();
        bins += (tid / kWave * kCopies + (tid % kWave) / (kWave / kCopies)) * kCopyStride;
    }
    MaskKey key = {};
    if (a.mask.below) key = mask_key(a.mask);
    uint32_t turn = 0;
    for (uint64_t row0 = (uint64_t)blockIdx.x * team.count; row0 < a.rows;
         row0 += (uint64_t)gridDim.x * team.count, turn ^= 1) {
        const uint64_t row = row0 + team.index;
        const uint32_t cols = row < a.rows ? a.cols : 0;
        auto column = [&](uint32_t base, uint32_t j) {
            uint32_t col = (base + j * team.lanes + team.at) * kUnit;
            forget(col);  // addresses are formed where they are used, not kept
            if constexpr (!LONG) __builtin_assume(col <= U * kMaxThreads * kUnit);  // 32-bit offsets
            return col;
        };
        // h of U units from column unit `base` on; their squares' sum
        RawUnit<RT> h[U];
        auto head = [&](uint32_t base, bool write) {
            RawUnit<DT> rx[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = column(base, j);
                rx[j] = load_raw<DT, STREAM>(x + row * a.ldx + col, places<WHOLE>(cols, col));
            }
            if (a.res) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint32_t col = column(base, j);
                    h[j] = load_raw<RT, STREAM>(res + row * a.ld_res + col, places<WHOLE>(cols, col));
                }
            }
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = column(base, j), n = places<WHOLE>(cols, col);
                h[j] = block_sum<DT, RT>(a, key, rx[j], h[j], row, col);
                if (write && n) store_raw<RT>(sum + row * a.ld_sum + col, n, h[j]);
                float v[8];
                widen_unit<RT>(h[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) s += (double)v[i] * (double)v[i];
                if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);
            }
            return s;
        };
        auto tail = [&](uint32_t base, double rstd) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = column(base, j), n = places<WHOLE>(cols, col);
                float w[8], v[8];
                auto form = [&](float v[8], float w[8]) {
                    uint32_t at = col;
                    forget(at);
                    if (a.weight) {
                        widen_any(a.weight_kind, load_any(a.weight_kind, a.weight, at, n), w);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
                    }
                    forget(h[j].w[0]);
                    if constexpr (RT == PC_F32) forget(h[j].w[1]);
                    widen_unit<RT>(h[j], v);
                };
                form(v, w);
                norm_unit<COUNT, RT != PC_F16>(a, row, col, n, rstd, w, v, bins, form);
                if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);  // one unit's registers at a time
            }
        };
        if constexpr (!LONG) {
            const double own = head(0, sum != nullptr);
            const double rstd = rstd_of(a, team_sum(team, own, part[turn]));
            if (team.at == 0 && cols && a.rstd) a.rstd[row] = (float)rstd;
            tail(0, rstd);
        } else {
            // the last units' group of 4 lanes stays whole
            const uint32_t units = (a.cols + kGroup - 1) / kGroup * kUnitsPerGroup;
            double own = 0.0;
            for (uint32_t base = 0; base < units; base += U * team.lanes) own += head(base, sum != nullptr);
            const double rstd = rstd_of(a, team_sum(team, own, part[turn]));
            if (team.at == 0 && cols && a.rstd) a.rstd[row] = (float)rstd;
            for (uint32_t base = 0; base < units; base += U * team.lanes) {
                if (sum) {  // the sum may have taken an input's place: it is read back by the lanes that wrote it
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        const uint32_t col = column(base, j);
                        h[j] = load_raw<RT>(sum + row * a.ld_sum + col, places<WHOLE>(cols, col));
                    }
                } else {
                    head(base, false);
                }
                tail(base, rstd);
            }
        }
    }
    if constexpr (COUNT) {
        __syncthreads();
        if (tid < 256) {
            uint64_t s = 0;
            for (uint32_t c = 0; c < kMaxWaves * kCopies; ++c) s += all_bins[c * kCopyStride + tid];
            if (s) atomicAdd(reinterpret_cast<unsigned long long *>(&a.counts[tid]), (unsigned long long)s);
        }
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

template <int RT, bool STORED> struct KeptUnit { RawUnit<RT> raw; };
template <int RT> struct KeptUnit<RT, true> { u32x2 sym; uint32_t code; };

template <int RT, bool STORED, bool STREAM>
__device__ __forceinline__ KeptUnit<RT, STORED> load_kept(const GradArgs &a, uint64_t row, uint32_t col, uint32_t n) {
    KeptUnit<RT, STORED> k = {};
    if constexpr (STORED) {
        if (n) {
            k.sym = load_symbols(a.sym + row * a.ld_sym + col, n);
            k.code = a.scale[row * a.ld_scale + col / kGroup];
        }
    } else {
        k.raw = load_raw<RT, STREAM>(static_cast<const typename Plain<RT>::type *>(a.sum) + row * a.ld_sum + col, n);
    }
    return k;
}

template <int RT, bool STORED>
__device__ __forceinline__ void widen_kept(const GradArgs &a, const KeptUnit<RT, STORED> &k, float h[8]) {
    if constexpr (STORED) {
        if (a.format == PC_Q8_E4M3) unit_values<PC_Q8_E4M3>(k.sym, scale_of(k.code), h);
        else unit_values<PC_Q8_INT8>(k.sym, scale_of(k.code), h);
    } else {
        widen_unit<RT>(k.raw, h);
    }
}

__device__ __forceinline__ void load_weights(const GradArgs &a, uint32_t col, uint32_t n, float w[8]) {
    if (a.weight) {
        widen_any(a.weight_kind, load_any(a.weight_kind, a.weight, col, n), w);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    }
}

// The gradients of a unit, written.
template <int DT, int RT>
__device__ __forceinline__ void grad_unit(const GradArgs &a, const MaskKey &key, uint64_t row, uint32_t col, uint32_t n,
                                          float rstd, float mean, const float g[8], const float norm[8],
                                          const RawUnit<RT> &d_sum) {
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = rstd * (g[i] - norm[i] * mean);
    if (a.d_sum) {
        float s[8];
        widen_unit<RT>(d_sum, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += s[i];
    }
    if (!n) return;
    if (a.d_res) store_unit<RT>(static_cast<typename Plain<RT>::type *>(a.d_res) + row * a.ld_d_res + col, n, d);
    if (a.d_x) {
        if (a.mask.below) drop_unit(a.mask, key, row, col, d);
        store_unit<DT>(static_cast<typename Plain<DT>::type *>(a.d_x) + row * a.ld_d_x + col, n, d);
    }
}

template <int RT, bool STORED>
__device__ __forceinline__ void forget_kept(KeptUnit<RT, STORED> &k) {
    if constexpr (STORED) {
        forget(k.sym);
    } else {
        forget(k.raw.w[0]);
        if constexpr (RT == PC_F32) forget(k.raw.w[1]);
    }
}

// A team takes every (grid * teams)th row and sums the weight's gradient over
// them in its registers; the next row's tensors are on their way while a row
// is worked on.  A workgroup's teams join their sums in LDS, in order.  8192 x
// 8192 bf16, the sum in e4m3, with a mask: 102-109 us, 5.7-6.1 TB/s with the partial
// sums' 16 MiB, vector work in 59% of the cycles.
template <int DT, int RT, int U, uint32_t SUB, bool STORED, bool STREAM, bool WHOLE>
__device__ __forceinline__ void grad_rows(const GradArgs &a, uint32_t blocks) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ float part[2][kMaxWaves];
    __shared__ float sums[U == 1 ? kGradThreads * kUnit : 1];
    const Team<SUB> team(a.team);
    const uint64_t step = (uint64_t)blocks * team.count;
    const TX *dy = static_cast<const TX *>(a.dy);
    const TR *d_sum = static_cast<const TR *>(a.d_sum);
    MaskKey key = {};
    if (a.mask.below) key = mask_key(a.mask);
    struct Row {
        RawUnit<DT> dy[U];
        KeptUnit<RT, STORED> kept[U];
        RawUnit<RT> d_sum[U];
        float rstd;
    };
    auto column = [&](uint32_t j) {
        uint32_t col = (j * team.lanes + team.at) * kUnit;
        forget(col);  // addresses are formed where they are used, not kept
        __builtin_assume(col <= U * kMaxThreads * kUnit);  // 32-bit offsets
        return col;
    };
    auto load = [&](uint64_t row, Row &r) {
        const uint32_t cols = row < a.rows ? a.cols : 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t col = column(j), n = places<WHOLE>(cols, col);
            r.dy[j] = load_raw<DT, STREAM>(dy + row * a.ld_dy + col, n);
            r.kept[j] = load_kept<RT, STORED, STREAM>(a, row, col, n);
            r.d_sum[j] = load_raw<RT, STREAM>(d_sum + row * a.ld_d_sum + col, a.d_sum ? n : 0);
        }
        r.rstd = cols ? a.rstd[row] : 0.0f;
    };
    float w[U][8], dw[U][8];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t col = column(j);
        load_weights(a, col, places<WHOLE>(a.cols, col), w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    }
    uint64_t row0 = (uint64_t)blockIdx.x * team.count;
    uint32_t turn = 0;
    Row r;
    load(row0 + team.index, r);
    for (; row0 < a.rows; row0 += step, turn ^= 1) {
        const uint64_t row = row0 + team.index;
        const uint32_t cols = row < a.rows ? a.cols : 0;
        Row next;
        load(row + step, next);
        float along = 0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float g[8], norm[8];
            widen_unit<DT>(r.dy[j], g);
            widen_kept<RT, STORED>(a, r.kept[j], norm);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float gn = g[i] * (norm[i] * r.rstd);
                dw[j][i] += gn;
                along += gn * w[j][i];
            }
            if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);
        }
        const float mean = team_sum(team, along, part[turn]) * a.per_col;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t col = column(j);
            float g[8], norm[8];
            forget(r.dy[j].w[0]);
            if constexpr (DT == PC_F32) forget(r.dy[j].w[1]);
            forget_kept(r.kept[j]);
            widen_unit<DT>(r.dy[j], g);
            widen_kept<RT, STORED>(a, r.kept[j], norm);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                norm[i] *= r.rstd;
                g[i] *= w[j][i];
            }
            grad_unit<DT, RT>(a, key, row, col, places<WHOLE>(cols, col), r.rstd, mean, g, norm, r.d_sum[j]);
            if constexpr (U > 1) __builtin_amdgcn_sched_barrier(0);
        }
        r = next;
    }
    if (!a.partial) return;
    if constexpr (U == 1) {  // larger rows have a workgroup each
        if (team.count > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[threadIdx.x * kUnit + i] = dw[0][i];
            __syncthreads();
            if (team.index) return;
            for (uint32_t k = 1; k < team.count; ++k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[0][i] += sums[(k * team.lanes + team.at) * kUnit + i];
            }
        }
    }
    float *to = a.partial + (uint64_t)blockIdx.x * a.ld_partial;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t col = column(j), n = places<WHOLE>(a.cols, col);
        if (n) store_unit<PC_F32>(to + col, n, dw[j]);
    }
}

template <int DT, int RT, int U, uint32_t SUB, bool STORED, bool STREAM, bool WHOLE>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_kernel(GradArgs a) {
    grad_rows<DT, RT, U, SUB, STORED, STREAM, WHOLE>(a, gridDim.x);
}

// The weight's gradient of 64 columns: 8 lanes side by side hold them, the
// workgroup's groups of 8 lanes take the rows in turns.
template <int DT, int RT, bool STORED>
__device__ __forceinline__ void grad_columns(const GradArgs &a, uint32_t block) {
    constexpr uint32_t kSide = kOnceColumns / kUnit;
    __shared__ float sums[kMaxThreads * kUnit];
    const uint32_t tid = threadIdx.x, groups = blockDim.x / kSide, parts = blockDim.x / kWave;
    const uint32_t col = (block * kSide + tid % kSide) * kUnit, n = count_before(a.cols, col, kUnit);
    float dw[8] = {};
#pragma unroll 4
    for (uint64_t row = tid / kSide; row < a.rows; row += groups) {
        float g[8], norm[8];
        load_unit<DT>(static_cast<const typename Plain<DT>::type *>(a.dy) + row * a.ld_dy + col, n, g);
        widen_kept<RT, STORED>(a, load_kept<RT, STORED, false>(a, row, col, n), norm);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += g[i] * (norm[i] * rstd);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[tid * kUnit + i] = dw[i];
    __syncthreads();
    // a lane to a column, the waves share the groups; then the waves' sums in order
    const uint32_t lane = tid % kWave, wave = tid / kWave;
    float s = 0.0f;
    for (uint32_t g = wave; g < groups; g += parts) s += sums[g * kOnceColumns + lane];
    __syncthreads();
    sums[tid] = s;
    __syncthreads();
    const uint32_t at = block * kOnceColumns + lane;
    if (wave || at >= a.cols) return;
    for (uint32_t p = 1; p < parts; ++p) s += sums[p * kWave + lane];
    with_dtype(a.d_weight_kind, [&](auto d) {
        typedef typename Plain<decltype(d)::value>::type T;
        T *out = static_cast<T *>(a.d_weight) + at;
        if (a.accumulate) s += widen(*out);
        *out = (T)s;
    });
}

// Few rows in one launch: some workgroups take rows, the others columns, which
// need nothing of each other: the weight's gradient reads dy and the sum again,
// but has no partial sums, and the call no second launch and no workspace (128
// x 2048 bf16 with the host's share: 14.9 us, in one launch 10.6; on the device 7.2
// and 5.0).
template <int DT, int RT, bool STORED>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_once_kernel(GradArgs a) {
    if (blockIdx.x < a.row_blocks) grad_rows<DT, RT, 1, kWave, STORED, false, false>(a, a.row_blocks);
    else grad_columns<DT, RT, STORED>(a, blockIdx.x - a.row_blocks);
}

// Rows of more units than a workgroup's registers hold, read twice (2048 x 40000
// bf16 with the weight's gradient: 233 us, at one reading's bytes 2.8 TB/s; 4096 x
// 16384 with an f32 sum: 305 us, 3.5 TB/s).
template <int DT, int RT, bool STORED>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_long_kernel(GradArgs a) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ float part[2][kMaxWaves];
    const uint32_t tid = threadIdx.x;
    const Team<kWave> team(kMaxThreads);
    const TX *dy = static_cast<const TX *>(a.dy);
    const TR *d_sum = static_cast<const TR *>(a.d_sum);
    MaskKey key = {};
    if (a.mask.below) key = mask_key(a.mask);
    uint32_t turn = 0;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const float rstd = a.rstd[row];
        auto unit = [&](uint32_t col, uint32_t n, float g[8], float norm[8]) {
            float w[8];
            load_unit<DT>(dy + row * a.ld_dy + col, n, g);
            widen_kept<RT, STORED>(a, load_kept<RT, STORED, false>(a, row, col, n), norm);
            load_weights(a, col, n, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                norm[i] *= rstd;
                g[i] *= w[i];
            }
        };
        float along = 0.0f;
        for (uint32_t col = tid * kUnit; col < a.cols; col += kMaxThreads * kUnit) {
            float g[8], norm[8];
            unit(col, count_before(a.cols, col, kUnit), g, norm);
#pragma unroll
            for (int i = 0; i < 8; ++i) along += g[i] * norm[i];
        }
        const float mean = team_sum(team, along, part[turn]) * a.per_col;
        for (uint32_t col = tid * kUnit; col < a.cols; col += kMaxThreads * kUnit) {
            const uint32_t n = count_before(a.cols, col, kUnit);
            float g[8], norm[8];
            unit(col, n, g, norm);
            const RawUnit<RT> s = load_raw<RT>(d_sum + row * a.ld_d_sum + col, a.d_sum ? n : 0);
            grad_unit<DT, RT>(a, key, row, col, n, rstd, mean, g, norm, s);
        }
    }
}

// The weight's gradient of such rows: a wave holds 512 columns and takes every
// (slices * 4)th row.

template <int DT, int RT, bool STORED>
__global__ __launch_bounds__(kColumnThreads) void norm_weight_kernel(GradArgs a) {
    const uint32_t wave = uniform(threadIdx.x / kWave), col = (blockIdx.x * kWave + threadIdx.x % kWave) * kUnit;
    const uint32_t n = count_before(a.cols, col, kUnit), first = blockIdx.y * kColumnWaves + wave;
    float dw[8] = {};
    for (uint64_t row = first; row < a.rows; row += (uint64_t)gridDim.y * kColumnWaves) {
        const float rstd = a.rstd[row];
        float g[8], norm[8];
        load_unit<DT>(static_cast<const typename Plain<DT>::type *>(a.dy) + row * a.ld_dy + col, n, g);
        widen_kept<RT, STORED>(a, load_kept<RT, STORED, false>(a, row, col, n), norm);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += g[i] * (norm[i] * rstd);
    }
    if (n) store_unit<PC_F32>(a.partial + first * a.ld_partial + col, n, dw);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

template <int DT, int RT>
hipError_t launch_norm(const NormArgs &a, const NormPlan &p, hipStream_t stream) {
    auto launch = [&](auto k) { hipLaunchKernelGGL(k, dim3(p.blocks), dim3(p.threads), 0, stream, a); };
    if (a.counts) {
        if (p.is_long) launch(norm_kernel<DT, RT, 4, kWave, true, true, false, false>);
        else if (p.per == 2) launch(norm_kernel<DT, RT, 2, kWave, true, false, false, false>);
        else launch(norm_kernel<DT, RT, 1, kWave, true, false, false, false>);
    } else if (p.is_long) {
        launch(norm_kernel<DT, RT, 4, kWave, false, true, false, false>);
    } else if (!p.whole) {
        if (p.per == 2) launch(norm_kernel<DT, RT, 2, kWave, false, false, false, false>);
        else launch(norm_kernel<DT, RT, 1, kWave, false, false, false, false>);
    } else if (p.per == 4) {
        if (p.streams) launch(norm_kernel<DT, RT, 4, kWave, false, false, true, true>);
        else launch(norm_kernel<DT, RT, 4, kWave, false, false, false, true>);
    } else if (p.per == 2) {
        if (p.streams) launch(norm_kernel<DT, RT, 2, kWave, false, false, true, true>);
        else launch(norm_kernel<DT, RT, 2, kWave, false, false, false, true>);
    } else {
        if (a.team == 16) launch(norm_kernel<DT, RT, 1, 16, false, false, false, true>);
        else if (a.team == 32) launch(norm_kernel<DT, RT, 1, 32, false, false, false, true>);
        else launch(norm_kernel<DT, RT, 1, kWave, false, false, false, true>);
    }
    return hipGetLastError();
}

template <int DT, int RT, bool STORED>
void launch_grad(const GradArgs &a, const GradPlan &p, hipStream_t stream) {
    auto launch = [&](auto k, dim3 grid, uint32_t threads) { hipLaunchKernelGGL(k, grid, dim3(threads), 0, stream, a); };
    const dim3 grid(p.blocks);
    if (p.once) {
        if (!p.columns_first) {
            launch(norm_grad_once_kernel<DT, RT, STORED>, grid, p.threads);
            return;
        }
        const auto k = norm_grad_once_kernel<DT, RT, STORED>;
        GradArgs columns = a;
        columns.row_blocks = 0;
        hipLaunchKernelGGL(k, dim3(p.blocks - a.row_blocks), dim3(p.threads), 0, stream, columns);
        launch(k, dim3(a.row_blocks), p.threads);
        return;
    }
    if (p.per == 0) {
        // before d_x, which may take dy's place
        if (a.partial) launch(norm_weight_kernel<DT, RT, STORED>, dim3(p.column_blocks, p.slices), kColumnThreads);
        if (a.d_res || a.d_x) launch(norm_grad_long_kernel<DT, RT, STORED>, grid, p.threads);
        return;
    }
    if (p.per == 2) {
        if constexpr (DT != PC_F32 && RT != PC_F32) {
            if (!p.whole) launch(norm_grad_kernel<DT, RT, 2, kWave, STORED, false, false>, grid, p.threads);
            else if (p.streams) launch(norm_grad_kernel<DT, RT, 2, kWave, STORED, true, true>, grid, p.threads);
            else launch(norm_grad_kernel<DT, RT, 2, kWave, STORED, false, true>, grid, p.threads);
        }
    } else if (!p.whole) {
        launch(norm_grad_kernel<DT, RT, 1, kWave, STORED, false, false>, grid, p.threads);
    } else if (p.team == 16) {
        launch(norm_grad_kernel<DT, RT, 1, 16, STORED, false, true>, grid, p.threads);
    } else if (p.team == 32) {
        launch(norm_grad_kernel<DT, RT, 1, 32, STORED, false, true>, grid, p.threads);
    } else if (p.streams) {
        launch(norm_grad_kernel<DT, RT, 1, kWave, STORED, true, true>, grid, p.threads);
    } else {
        launch(norm_grad_kernel<DT, RT, 1, kWave, STORED, false, true>, grid, p.threads);
    }
}

template <int DT, int RT>
hipError_t launch_norm_grad(const GradArgs &a, const GradPlan &p, hipStream_t stream) {
    if (a.sym) launch_grad<DT, RT, true>(a, p, stream);
    else launch_grad<DT, RT, false>(a, p, stream);
    return hipGetLastError();
}

}  // namespace
}  // namespace pc
