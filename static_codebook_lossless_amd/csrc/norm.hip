// Root-mean-square norm with what a residual block does around it: dropout of
// the block's output, the residual's addition, the norm, and the norm's output
// stored in 8 bits; and the backward pass of all of that.
//
//   h = round(res + mask(x)),  r = (mean(h^2) + eps)^-1/2,  y = h r w
//   d = r (g - n mean(g n)) + d_sum,  g = dy w,  n = h r
//   d_res = d,  d_x = mask(d),  d_w = sum over rows of dy n
#include <algorithm>
#include <type_traits>

#include "random.h"

namespace pc {
namespace {

constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kMaxWaves = kMaxThreads / kWave;

// Histogram copies of the counting form, as in the store.
constexpr uint32_t kCopies = 8;
constexpr uint32_t kCopyStride = 257;
constexpr uint32_t kBins = kMaxWaves * kCopies * kCopyStride;
constexpr uint32_t kCountBlocks = 256;

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

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) { return v + as_f32(dpp_u32<CTRL>(as_u32(v))); }

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
    const u32x2 u = __builtin_bit_cast(u32x2, v);
    const u32x2 o = {dpp_u32<CTRL>(u[0]), dpp_u32<CTRL>(u[1])};
    return v + __builtin_bit_cast(double, o);
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

// The sum over a wave, the same in every lane.
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
    v = dpp_add<0xB1>(v);   // the neighbour in the pair
    v = dpp_add<0x4E>(v);   // the other pair
    v = dpp_add<0x141>(v);  // the other half of 8
    v = dpp_add<0x140>(v);  // the other half of 16
    return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}

// The sum over a row's team of waves.  `part` alternates between two areas
// from call to call, so one barrier a call is enough: what a call writes was
// last read before the barrier of the call between.
template <class T>
__device__ __forceinline__ T team_sum(T v, T *part, uint32_t wave, uint32_t team_waves) {
    v = wave_sum(v);
    if (team_waves == 1) return v;
    if (threadIdx.x % kWave == 0) part[wave] = v;
    __syncthreads();
    const uint32_t first = wave / team_waves * team_waves;
    T s = part[first];
    for (uint32_t i = 1; i < team_waves; ++i) s += part[first + i];
    return s;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------

struct NormArgs {
    const void *x, *res, *weight;
    void *sum, *y;
    uint8_t *sym, *scale;
    uint64_t *counts;
    float *rstd;
    uint64_t rows, ldx, ld_res, ld_sum, ld_y;
    uint32_t cols, groups;
    uint32_t team;  // lanes to a row: a power of two from 64 to the workgroup's
    int weight_kind, y_kind, format, y_stored;
    double eps, per_col;  // per_col: 1 / cols
    MaskArg mask;
};

// r = (mean + eps)^-1/2.  Squares are summed in 64 bits, where those of all
// 32-bit numbers fit; a vector instruction takes as long as in 32 bits.  The
// hardware's estimate has 23 bits, which a Newton step doubles.
__device__ __forceinline__ float rstd_of(const NormArgs &a, double squares) {
    const double m = squares * a.per_col + a.eps, r = __builtin_amdgcn_rsq(m);
    return m == __builtin_inf() ? 0.0f : (float)(r * (1.5 - 0.5 * m * r * r));
}

// h of a unit, as the sum's type holds it.
template <int DT, int RT>
__device__ __forceinline__ void block_sum(const NormArgs &a, const MaskKey &key, const RawUnit<DT> &x,
                                          const RawUnit<RT> &res, uint64_t row, uint32_t col, float h[8]) {
    widen_unit<DT>(x, h);
    if (a.mask.below) drop_unit(a.mask, key, row, col, h);
    if (a.res) {
        float r[8];
        widen_unit<RT>(res, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] += r[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = rounded<RT>(h[i]);
}

template <bool COUNT>
__device__ __forceinline__ void norm_unit(const NormArgs &a, uint64_t row, uint32_t col, uint32_t n, float rstd,
                                          const float w[8], const float h[8], uint32_t *bins) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
    if (a.y && !a.y_stored && n) store_any(a.y_kind, a.y, row * a.ld_y + col, n, y);
    if (!a.sym) return;
    auto store = [&](auto f) {
        constexpr int FMT = decltype(f)::value;
        uint32_t code;
        const u32x2 s = to_stored<FMT>(y, code);
        if (n) {
            store_symbols(a.sym + row * a.cols + col, n, s);
            if (col % kGroup == 0) a.scale[row * a.groups + col / kGroup] = (uint8_t)code;
            if (a.y && a.y_stored) {
                float v[8];
                unit_values<FMT>(s, scale_of(code), v);
                store_any(a.y_kind, a.y, row * a.ld_y + col, n, v);
            }
        }
        if constexpr (COUNT) {
#pragma unroll
            for (uint32_t i = 0; i < kUnit; ++i)
                if (i < n) atomicAdd(&bins[(s[i / 4] >> (8 * (i % 4))) & 0xFF], 1u);
        }
    };
    if (a.format == PC_Q8_E4M3) store(std::integral_constant<int, PC_Q8_E4M3>());
    else store(std::integral_constant<int, PC_Q8_INT8>());
}

// U units a lane; LONG: rows of more than team * U units, read in turns.
template <int DT, int RT, int U, bool COUNT, bool LONG>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ double part[2][kMaxWaves];
    __shared__ uint32_t all_bins[COUNT ? kBins : 1];
    const uint32_t tid = threadIdx.x, wave = uniform(tid / kWave), team_waves = a.team / kWave;
    const uint32_t at = tid & (a.team - 1), teams = blockDim.x / a.team;
    const TX *x = static_cast<const TX *>(a.x);
    const TR *res = static_cast<const TR *>(a.res);
    TR *sum = static_cast<TR *>(a.sum);
    uint32_t *bins = all_bins;
    if constexpr (COUNT) {
        for (uint32_t i = tid; i < kBins; i += blockDim.x) all_bins[i] = 0;
        __syncthreads();
        bins += (wave * kCopies + (tid % kWave) / (kWave / kCopies)) * kCopyStride;
    }
    MaskKey key = {};
    if (a.mask.below) key = mask_key(a.mask);
    uint32_t turn = 0;
    for (uint64_t row0 = (uint64_t)blockIdx.x * teams; row0 < a.rows; row0 += (uint64_t)gridDim.x * teams, turn ^= 1) {
        const uint64_t row = row0 + wave / team_waves;
        const uint32_t cols = row < a.rows ? a.cols : 0;
        // h of U units from column unit `base` on; their square's sum
        float h[U][8];
        auto head = [&](uint32_t base, bool write) {
            RawUnit<DT> rx[U];
            RawUnit<RT> rr[U];
            uint32_t n[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = (base + j * a.team + at) * kUnit;
                n[j] = count_before(cols, col, kUnit);
                rx[j] = load_raw<DT>(x + row * a.ldx + col, n[j]);
            }
            if (a.res) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint32_t col = (base + j * a.team + at) * kUnit;
                    rr[j] = load_raw<RT>(res + row * a.ld_res + col, n[j]);
                }
            }
            double s = 0.0;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = (base + j * a.team + at) * kUnit;
                block_sum<DT, RT>(a, key, rx[j], rr[j], row, col, h[j]);
                if (write && n[j]) store_unit<RT>(sum + row * a.ld_sum + col, n[j], h[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) s += (double)h[j][i] * (double)h[j][i];
            }
            return s;
        };
        auto weights = [&](uint32_t base, AnyUnit w[U]) {
            if (!a.weight) return;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = (base + j * a.team + at) * kUnit;
                w[j] = load_any(a.weight_kind, a.weight, col, count_before(cols, col, kUnit));
            }
        };
        auto tail = [&](uint32_t base, float rstd, const AnyUnit raw[U]) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const uint32_t col = (base + j * a.team + at) * kUnit;
                float w[8];
                if (a.weight) {
                    widen_any(a.weight_kind, raw[j], w);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
                }
                norm_unit<COUNT>(a, row, col, count_before(cols, col, kUnit), rstd, w, h[j], bins);
            }
        };
        AnyUnit w[U] = {};
        if constexpr (!LONG) {
            const double own = head(0, sum != nullptr);
            weights(0, w);
            const float rstd = rstd_of(a, team_sum(own, part[turn], wave, team_waves));
            if (at == 0 && cols && a.rstd) a.rstd[row] = rstd;
            tail(0, rstd, w);
        } else {
            // the last units' group of 4 lanes stays whole
            const uint32_t units = (a.cols + kGroup - 1) / kGroup * kUnitsPerGroup;
            double own = 0.0;
            for (uint32_t base = 0; base < units; base += U * a.team) own += head(base, sum != nullptr);
            const float rstd = rstd_of(a, team_sum(own, part[turn], wave, team_waves));
            if (at == 0 && cols && a.rstd) a.rstd[row] = rstd;
            for (uint32_t base = 0; base < units; base += U * a.team) {
                weights(base, w);
                if (sum) {  // the sum may have taken an input's place: it is read back by the lanes that wrote it
#pragma unroll
                    for (int j = 0; j < U; ++j) {
                        const uint32_t col = (base + j * a.team + at) * kUnit;
                        widen_unit<RT>(load_raw<RT>(sum + row * a.ld_sum + col, count_before(cols, col, kUnit)), h[j]);
                    }
                } else {
                    head(base, false);
                }
                tail(base, rstd, w);
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

struct GradArgs {
    const void *dy, *sum, *d_sum, *weight;
    const uint8_t *sym, *scale;  // the sum in its stored form, in place of `sum`
    const float *rstd;
    void *d_res, *d_x;
    float *partial;  // [teams of all workgroups][ld_partial], or nullptr
    uint64_t rows, ld_dy, ld_sum, ld_sym, ld_scale, ld_d_sum, ld_d_res, ld_d_x, ld_partial;
    uint32_t cols, team;
    int weight_kind, format;
    float per_col;  // 1 / cols
    MaskArg mask;
};

template <int RT, bool STORED> struct KeptUnit { RawUnit<RT> raw; };
template <int RT> struct KeptUnit<RT, true> { u32x2 sym; uint32_t code; };

template <int RT, bool STORED>
__device__ __forceinline__ KeptUnit<RT, STORED> load_kept(const GradArgs &a, uint64_t row, uint32_t col, uint32_t n) {
    KeptUnit<RT, STORED> k = {};
    if constexpr (STORED) {
        if (n) {
            k.sym = load_symbols(a.sym + row * a.ld_sym + col, n);
            k.code = a.scale[row * a.ld_scale + col / kGroup];
        }
    } else {
        k.raw = load_raw<RT>(static_cast<const typename Plain<RT>::type *>(a.sum) + row * a.ld_sum + col, n);
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

// A team takes every (grid * teams)th row and sums the weight's gradient over
// them in its registers; the next row's tensors are on their way while a row
// is worked on.
template <int DT, int RT, int U, bool STORED>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_kernel(GradArgs a) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ float part[2][kMaxWaves];
    const uint32_t tid = threadIdx.x, wave = uniform(tid / kWave), team_waves = a.team / kWave;
    const uint32_t at = tid & (a.team - 1), teams = blockDim.x / a.team;
    const uint64_t step = (uint64_t)gridDim.x * teams;
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
    auto load = [&](uint64_t row, Row &r) {
        const uint32_t cols = row < a.rows ? a.cols : 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t col = (j * a.team + at) * kUnit, n = count_before(cols, col, kUnit);
            r.dy[j] = load_raw<DT>(dy + row * a.ld_dy + col, n);
            r.kept[j] = load_kept<RT, STORED>(a, row, col, n);
            r.d_sum[j] = load_raw<RT>(d_sum + row * a.ld_d_sum + col, a.d_sum ? n : 0);
        }
        r.rstd = cols ? a.rstd[row] : 0.0f;
    };
    float w[U][8], dw[U][8];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const uint32_t col = (j * a.team + at) * kUnit;
        load_weights(a, col, count_before(a.cols, col, kUnit), w[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
    }
    uint64_t row0 = (uint64_t)blockIdx.x * teams;
    uint32_t turn = 0;
    Row r;
    load(row0 + wave / team_waves, r);
    for (; row0 < a.rows; row0 += step, turn ^= 1) {
        const uint64_t row = row0 + wave / team_waves;
        const uint32_t cols = row < a.rows ? a.cols : 0;
        Row next;
        load(row + step, next);
        float g[U][8], norm[U][8], along = 0.0f;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            widen_unit<DT>(r.dy[j], g[j]);
            widen_kept<RT, STORED>(a, r.kept[j], norm[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                norm[j][i] *= r.rstd;
                dw[j][i] += g[j][i] * norm[j][i];
                g[j][i] *= w[j][i];
                along += g[j][i] * norm[j][i];
            }
        }
        const float mean = team_sum(along, part[turn], wave, team_waves) * a.per_col;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t col = (j * a.team + at) * kUnit;
            grad_unit<DT, RT>(a, key, row, col, count_before(cols, col, kUnit), r.rstd, mean, g[j], norm[j],
                              r.d_sum[j]);
        }
        r = next;
    }
    if (a.partial) {
        float *to = a.partial + ((uint64_t)blockIdx.x * teams + wave / team_waves) * a.ld_partial;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t col = (j * a.team + at) * kUnit, n = count_before(a.cols, col, kUnit);
            if (n) store_unit<PC_F32>(to + col, n, dw[j]);
        }
    }
}

// Rows of more units than a workgroup's registers hold, read twice.
template <int DT, int RT, bool STORED>
__global__ __launch_bounds__(kMaxThreads) void norm_grad_long_kernel(GradArgs a) {
    typedef typename Plain<DT>::type TX;
    typedef typename Plain<RT>::type TR;
    __shared__ float part[2][kMaxWaves];
    const uint32_t tid = threadIdx.x, wave = uniform(tid / kWave), team_waves = a.team / kWave;
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
            widen_kept<RT, STORED>(a, load_kept<RT, STORED>(a, row, col, n), norm);
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
        const float mean = team_sum(along, part[turn], wave, team_waves) * a.per_col;
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
constexpr uint32_t kColumnThreads = 256;
constexpr uint32_t kColumnWaves = kColumnThreads / kWave;

template <int DT, int RT, bool STORED>
__global__ __launch_bounds__(kColumnThreads) void norm_weight_kernel(GradArgs a) {
    const uint32_t wave = uniform(threadIdx.x / kWave), col = (blockIdx.x * kWave + threadIdx.x % kWave) * kUnit;
    const uint32_t n = count_before(a.cols, col, kUnit), first = blockIdx.y * kColumnWaves + wave;
    float dw[8] = {};
    for (uint64_t row = first; row < a.rows; row += (uint64_t)gridDim.y * kColumnWaves) {
        const float rstd = a.rstd[row];
        float g[8], norm[8];
        load_unit<DT>(static_cast<const typename Plain<DT>::type *>(a.dy) + row * a.ld_dy + col, n, g);
        widen_kept<RT, STORED>(a, load_kept<RT, STORED>(a, row, col, n), norm);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] += g[i] * (norm[i] * rstd);
    }
    if (n) store_unit<PC_F32>(a.partial + first * a.ld_partial + col, n, dw);
}

// The sums of `parts` rows of partial sums, 64 columns to a workgroup: its
// waves take every 16th row and their sums are added in order.
template <int DT>
__global__ __launch_bounds__(kMaxThreads) void norm_join_kernel(const float *__restrict__ partial, uint64_t ld,
                                                                uint32_t parts, uint32_t cols, int accumulate,
                                                                typename Plain<DT>::type *__restrict__ out) {
    __shared__ float sums[kMaxWaves][kWave];
    const uint32_t lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    for (uint32_t first = blockIdx.x * kWave; first < cols; first += gridDim.x * kWave) {
        const uint32_t col = first + lane;
        float s = 0.0f;
        if (col < cols) {
#pragma unroll 4
            for (uint32_t i = wave; i < parts; i += kMaxWaves) s += partial[i * ld + col];
        }
        sums[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && col < cols) {
            float t = sums[0][lane];
            for (uint32_t i = 1; i < kMaxWaves; ++i) t += sums[i][lane];
            if (accumulate) t += widen(out[col]);
            out[col] = (typename Plain<DT>::type)t;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

uint32_t units_of(uint64_t cols) { return (uint32_t)((cols + kGroup - 1) / kGroup * kUnitsPerGroup); }

// The smallest team (a power of two of lanes, whole waves) of `per` units a lane.
uint32_t team_for(uint32_t units, uint32_t per) {
    uint32_t team = kWave;
    while (team < kMaxThreads && team * per < units) team *= 2;
    return team;
}

// Calls f with the compile-time types of x and of the sum: the sum's is x's own or f32.
template <class F>
void with_types(int x, int sum, F &&f) {
    with_dtype(x, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        if (sum == DT) f(d, d);
        else if constexpr (DT != PC_F32) f(d, std::integral_constant<int, PC_F32>());
    });
}

struct GradPlan {
    uint32_t per, team, threads, blocks;  // per == 0: long rows
    uint32_t parts;                       // rows of partial sums
    uint32_t column_blocks, slices;       // of the long rows' weight gradient
};

GradPlan plan_grad(uint64_t rows, uint64_t cols) {
    GradPlan p = {};
    const uint32_t units = units_of(cols);
    p.per = units <= kMaxThreads ? 1 : units <= 2 * kMaxThreads ? 2 : 0;
    if (p.per) {
        p.team = team_for(units, p.per);
        p.threads = std::max(p.team, 256u);
        const uint32_t teams = p.threads / p.team;
        p.blocks = (uint32_t)std::min<uint64_t>((rows + teams - 1) / teams, 256 * (kMaxThreads / p.threads));
        p.parts = p.blocks * teams;
    } else {
        p.team = p.threads = kMaxThreads;
        p.blocks = (uint32_t)std::min<uint64_t>(rows, 512);
        p.column_blocks = (units + kWave - 1) / kWave;
        const uint64_t wanted = std::max<uint64_t>(1, 1024 / p.column_blocks);
        p.slices = (uint32_t)std::min<uint64_t>(wanted, (rows + kColumnWaves - 1) / kColumnWaves);
        p.parts = p.slices * kColumnWaves;
    }
    return p;
}

uint64_t partial_width(uint64_t cols) { return (cols + 3) / 4 * 4; }

}  // namespace

hipError_t launch_rmsnorm_store(const RmsNorm &c, hipStream_t stream) {
    NormArgs a = {};
    a.x = c.x;
    a.res = c.res;
    a.weight = c.weight;
    a.sum = c.sum;
    a.y = c.y;
    a.sym = c.sym;
    a.scale = c.scale;
    a.counts = c.counts;
    a.rstd = c.rstd;
    a.rows = c.rows;
    a.ldx = c.ldx;
    a.ld_res = c.ld_res;
    a.ld_sum = c.ld_sum;
    a.ld_y = c.ld_y;
    a.cols = (uint32_t)c.cols;
    a.groups = (uint32_t)((c.cols + kGroup - 1) / kGroup);
    a.weight_kind = c.weight_dtype;
    a.y_kind = c.y_dtype;
    a.format = c.format;
    a.y_stored = c.y_stored;
    a.eps = c.eps;
    a.per_col = 1.0 / (double)c.cols;
    a.mask = mask_arg(c.mask);
    const uint32_t units = units_of(c.cols);
    const bool count = c.counts != nullptr;
    uint32_t per = 2;
    bool is_long = false;
    if (units <= kWave || c.rows <= 512) per = 1;
    if (units > per * kMaxThreads) per = 2;
    if (units > per * kMaxThreads) {
        per = 4;
        is_long = units > per * kMaxThreads;
    }
    a.team = team_for(units, per);
    const uint32_t threads = count ? kMaxThreads : std::max(a.team, 256u), teams = threads / a.team;
    const uint64_t wanted = (c.rows + teams - 1) / teams, most = count ? kCountBlocks : (1u << 22) - 1;
    const dim3 grid((uint32_t)std::min(wanted, most));
    with_types(c.dtype, c.sum_dtype, [&](auto d, auto r) {
        constexpr int DT = decltype(d)::value, RT = decltype(r)::value;
        auto launch = [&](auto k) { hipLaunchKernelGGL(k, grid, dim3(threads), 0, stream, a); };
        if (count) {
            if (is_long) launch(norm_kernel<DT, RT, 4, true, true>);
            else if (per == 4) launch(norm_kernel<DT, RT, 4, true, false>);
            else if (per == 2) launch(norm_kernel<DT, RT, 2, true, false>);
            else launch(norm_kernel<DT, RT, 1, true, false>);
        } else {
            if (is_long) launch(norm_kernel<DT, RT, 4, false, true>);
            else if (per == 4) launch(norm_kernel<DT, RT, 4, false, false>);
            else if (per == 2) launch(norm_kernel<DT, RT, 2, false, false>);
            else launch(norm_kernel<DT, RT, 1, false, false>);
        }
    });
    return hipGetLastError();
}

uint64_t rmsnorm_backward_workspace(uint64_t rows, uint64_t cols) {
    return (uint64_t)plan_grad(rows, cols).parts * partial_width(cols) * sizeof(float);
}

hipError_t launch_rmsnorm_backward(const RmsNormGrad &c, hipStream_t stream) {
    const GradPlan p = plan_grad(c.rows, c.cols);
    GradArgs a = {};
    a.dy = c.dy;
    a.sum = c.sum;
    a.ld_sum = c.ld_sum;
    if (c.stored) {
        a.sym = c.stored->sym;
        a.scale = c.stored->scale;
        a.ld_sym = c.stored->ld_sym;
        a.ld_scale = c.stored->ld_scale;
        a.format = c.stored->format;
    }
    a.d_sum = c.d_sum;
    a.weight = c.weight;
    a.weight_kind = c.weight_dtype;
    a.rstd = c.rstd;
    a.d_res = c.d_res;
    a.d_x = c.d_x;
    a.partial = c.d_weight ? static_cast<float *>(c.ws) : nullptr;
    a.rows = c.rows;
    a.ld_dy = c.ld_dy;
    a.ld_d_sum = c.ld_d_sum;
    a.ld_d_res = c.ld_d_res;
    a.ld_d_x = c.ld_d_x;
    a.ld_partial = partial_width(c.cols);
    a.cols = (uint32_t)c.cols;
    a.team = p.team;
    a.per_col = (float)(1.0 / (double)c.cols);
    a.mask = mask_arg(c.mask);
    if (c.rows) {
        with_types(c.dtype, c.sum_dtype, [&](auto d, auto r) {
            constexpr int DT = decltype(d)::value, RT = decltype(r)::value;
            auto by_kept = [&](auto s) {
                constexpr bool STORED = decltype(s)::value;
                auto launch = [&](auto k, dim3 grid, uint32_t threads) {
                    hipLaunchKernelGGL(k, grid, dim3(threads), 0, stream, a);
                };
                if (p.per == 1) {
                    launch(norm_grad_kernel<DT, RT, 1, STORED>, dim3(p.blocks), p.threads);
                } else if (p.per == 2) {
                    launch(norm_grad_kernel<DT, RT, 2, STORED>, dim3(p.blocks), p.threads);
                } else {
                    // before d_x, which may take dy's place
                    if (a.partial)
                        launch(norm_weight_kernel<DT, RT, STORED>, dim3(p.column_blocks, p.slices), kColumnThreads);
                    if (a.d_res || a.d_x)
                        launch(norm_grad_long_kernel<DT, RT, STORED>, dim3(p.blocks), p.threads);
                }
            };
            if (c.stored) by_kept(std::true_type());
            else by_kept(std::false_type());
        });
    }
    if (c.d_weight) {
        const dim3 grid((uint32_t)std::min<uint64_t>((c.cols + kWave - 1) / kWave, 1u << 16));
        with_dtype(c.d_weight_dtype, [&](auto d) {
            constexpr int DT = decltype(d)::value;
            hipLaunchKernelGGL(norm_join_kernel<DT>, grid, dim3(kMaxThreads), 0, stream, a.partial, a.ld_partial,
                               c.rows ? p.parts : 0, (uint32_t)c.cols, c.accumulate,
                               static_cast<typename Plain<DT>::type *>(c.d_weight));
        });
    }
    return hipGetLastError();
}

}  // namespace pc
