// Storing a tensor as 8-bit symbols with one power-of-two scale for every 32
// columns, reading it back, and the backward pass of an activation whose
// inputs were stored.
//
// All three read and write every byte once and compute little: they are
// bound by HBM.  A lane handles 8 columns (16 bytes of a 16-bit type, 8
// symbols), so four neighbouring lanes hold a group, and the largest
// magnitude of a group costs two DPP exchanges and no LDS.  Tensors whose rows
// lie end to end in whole groups count as one row and need no division.
//
// Measured at 4096 x 16384 bf16 (a device copy reaches 5.2 TB/s): store 33 us
// (6.1 TB/s), with the histogram 49 us, load 29 us (6.8 TB/s), the backward
// pass of gate and up in one tensor with h 109 us on the device, 115 through
// the binding (5.9 TB/s).  In f32: load of 4096 x 8192 27 us (6.2 TB/s; 38 us
// alone, when no part of the output is in the memory-side cache), that
// backward pass of 2048 x 16384 115 us (5.2 TB/s).  Small calls (store of 32 x
// 2048) take 3.7 us on the device and 10 us through the binding.
#include <algorithm>
#include <type_traits>

#include "q8.h"

namespace pc {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kPerLane = 4;  // units per lane
constexpr uint32_t kTile = kThreads * kPerLane;

// ---------------------------------------------------------------------------
// store
// ---------------------------------------------------------------------------

// Histogram of the symbols in LDS, as in the byte histogram but with 8 copies
// per wave, 257 words apart, added to the caller's counts at the end.  One
// workgroup of 16 waves fills a CU: the sums at the end cost 15 ns for every
// workgroup, as they meet at the same 256 addresses.  64 Mi bf16 elements:
// two workgroups of 4 waves and 16 copies 89 us, four of 4 and 8 copies 67 us,
// the same with the next tile's loads ahead 60 us, one of 16 waves 51 us (4
// copies: 60 us).
constexpr uint32_t kCopies = 8;
constexpr uint32_t kCopyStride = 257;
constexpr uint32_t kCountThreads = 1024;
constexpr uint32_t kBins = kCountThreads / kWave * kCopies * kCopyStride;
constexpr uint32_t kCountBlocks = 256;
constexpr uint32_t kCountPerLane = 2;

// PER units in a lane; the next tile's are loaded while a tile is stored and
// counted (a counting workgroup takes many tiles, the others one).
template <int DT, int FMT, bool COUNT>
__global__ __launch_bounds__(COUNT ? kCountThreads : kThreads) void store_kernel(const typename Plain<DT>::type *__restrict__ x, Units units,
                                                         uint64_t ldx, uint64_t ld_sym, uint64_t ld_scale,
                                                         uint8_t *__restrict__ sym, uint8_t *__restrict__ scale,
                                                         uint64_t *__restrict__ counts) {
    constexpr uint32_t THREADS = COUNT ? kCountThreads : kThreads, PER = COUNT ? kCountPerLane : kPerLane;
    constexpr uint32_t kTileUnits = THREADS * PER;
    __shared__ uint32_t bins[COUNT ? kBins : 1];
    const uint32_t tid = threadIdx.x;
    uint32_t *my = bins;
    struct Unit {
        RawUnit<DT> raw;
        uint64_t row, col;
        uint32_t n;
    };
    auto load = [&](uint64_t base, Unit u[PER]) {
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) {
            const uint32_t local = j * THREADS + tid;
            u[j].n = 0;
            u[j].row = u[j].col = 0;
            if (base + local < units.total) {
                find_unit(units, base, local, u[j].row, u[j].col);
                // a short group's last units may hold no column at all
                u[j].n = count_before(units.cols, u[j].col, kUnit);
            }
            u[j].raw = load_raw<DT>(x + u[j].row * ldx + u[j].col, u[j].n);
        }
    };
    auto store = [&](const Unit &u) {
        float v[8];
        widen_unit<DT>(u.raw, v);
        uint32_t code;
        const u32x2 w = to_stored<FMT>(v, code);
        if (u.n) {
            store_symbols(sym + u.row * ld_sym + u.col, u.n, w);
            if (u.col % kGroup == 0) scale[u.row * ld_scale + u.col / kGroup] = (uint8_t)code;
        }
        if constexpr (COUNT) {
            if (u.n == kUnit) {
#pragma unroll
                for (uint32_t i = 0; i < kUnit; ++i) atomicAdd(&my[(w[i / 4] >> (8 * (i % 4))) & 0xFF], 1u);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < kUnit; ++i)
                    if (i < u.n) atomicAdd(&my[(w[i / 4] >> (8 * (i % 4))) & 0xFF], 1u);
            }
        }
    };
    Unit u[PER];
    uint64_t base = (uint64_t)blockIdx.x * kTileUnits;
    load(base, u);
    if constexpr (!COUNT) {
#pragma unroll
        for (uint32_t j = 0; j < PER; ++j) store(u[j]);
    } else {
        for (uint32_t i = tid; i < kBins; i += THREADS) bins[i] = 0;
        __syncthreads();
        my += ((tid / kWave) * kCopies + (tid % kWave) / (kWave / kCopies)) * kCopyStride;
        for (; base < units.total; base += (uint64_t)gridDim.x * kTileUnits) {
            Unit next[PER];
            load(base + (uint64_t)gridDim.x * kTileUnits, next);
#pragma unroll
            for (uint32_t j = 0; j < PER; ++j) store(u[j]);
#pragma unroll
            for (uint32_t j = 0; j < PER; ++j) u[j] = next[j];
        }
        __syncthreads();
        // four threads a bin, a quarter of the copies each
        constexpr uint32_t kShare = THREADS / 256;
        uint32_t s = 0;
        for (uint32_t c = tid / 256; c < THREADS / kWave * kCopies; c += kShare) s += bins[c * kCopyStride + tid % 256];
        __syncthreads();
        bins[tid] = s;
        __syncthreads();
        if (tid < 256) {
            uint64_t sum = 0;
#pragma unroll
            for (uint32_t c = 0; c < kShare; ++c) sum += bins[c * 256 + tid];
            if (sum) atomicAdd(reinterpret_cast<unsigned long long *>(&counts[tid]), (unsigned long long)sum);
        }
    }
}

// ---------------------------------------------------------------------------
// load
// ---------------------------------------------------------------------------

// Two units a lane: four leave a small tensor too few workgroups (1021 x 5001
// in f32: 9.0 us, with two 8.4), one costs large ones a little (64 Mi in bf16:
// 30.3 us, with two 29.4).
constexpr uint32_t kLoadPerLane = 2;
constexpr uint32_t kLoadTile = kThreads * kLoadPerLane;

template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void load_kernel(const uint8_t *__restrict__ sym,
                                                        const uint8_t *__restrict__ scale, uint64_t ld_sym,
                                                        uint64_t ld_scale, Units units, uint64_t ld_out,
                                                        typename Plain<DT>::type *__restrict__ out) {
    const uint64_t base = (uint64_t)blockIdx.x * kLoadTile;
    u32x2 w[kLoadPerLane];
    uint32_t code[kLoadPerLane], n[kLoadPerLane];
    uint64_t row[kLoadPerLane], col[kLoadPerLane];
#pragma unroll
    for (uint32_t j = 0; j < kLoadPerLane; ++j) {
        const uint32_t local = j * kThreads + threadIdx.x;
        n[j] = 0;
        if (base + local < units.total) {
            find_unit(units, base, local, row[j], col[j]);
            n[j] = count_before(units.cols, col[j], kUnit);
        }
        if (n[j]) {
            w[j] = load_symbols(sym + row[j] * ld_sym + col[j], n[j]);
            code[j] = scale[row[j] * ld_scale + col[j] / kGroup];
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kLoadPerLane; ++j) {
        if (!n[j]) continue;
        float v[8];
        unit_values<FMT>(w[j], scale_of(code[j]), v);
        store_unit<DT>(out + row[j] * ld_out + col[j], n[j], v);
    }
}

// ---------------------------------------------------------------------------
// gated activation, backward
// ---------------------------------------------------------------------------

constexpr float kLog2E = 1.44269504088896340736f;

// p = 1 / (1 + exp(-z)) and q = p (1 - p), both from w = exp(-|z|) <= 1, so
// that neither end loses its digits: with r = 1 / (1 + w), p is r or w r, and
// q = w r^2.  NaN for NaN.
__device__ __forceinline__ void sigmoid(float z, float &p, float &q) {
    const float w = __builtin_amdgcn_exp2f(-kLog2E * __builtin_fabsf(z));
    const float r = __builtin_amdgcn_rcpf(1.0f + w), t = w * r;
    p = z < 0.0f ? t : r;
    q = t * r;
}

// y = act(g), d = act'(g).
//   SiLU:  y = g p(g),  d = p + g p (1 - p), p the sigmoid.
//   GELU by the normal distribution function P and its density f:
//     y = g P(g),  d = P(g) + g f(g),
//   with the tail 1 - P(|g|) = exp(-g^2 / 2) R(t), t = 1 / (1 + 0.31 |g|): it
//   shares the exponential with the density.  R is t times a polynomial of
//   degree 9, the minimax one of the relative error (1.2e-8) on 0 <= |g| <= 30
//   by Remez exchange in 64 bits, so small values of the tail keep their digits.
//   Five terms (Abramowitz and Stegun 7.1.26) bound only the absolute error:
//   twice the error of 32-bit arithmetic near 0, 0.3% of y at g = -6, and the
//   same time (4096 x 16384 bf16 with h: 114-115 us).  g has 8 bits at most, so
//   its square is exact.
//   The tanh form by  (1 + tanh z) / 2 = p(2 z):
//     y = g p,  d = p + g p (1 - p) z',  z' = 2 sqrt(2/pi) (1 + 3 c g^2).
// Beyond |g| = 30 both GELU forms are 0 or the identity in 32 bits; g is held
// there inside them, so that no product of 0 and infinity arises.
template <int ACT>
__device__ __forceinline__ void activation(float g, float &y, float &d) {
    if constexpr (ACT == PC_ACT_SILU) {
        float p, q;
        sigmoid(g, p, q);
        y = g * p;
        d = p + g * q;
    } else {
        float b = g > 30.0f ? 30.0f : g;  // NaN stays
        b = b < -30.0f ? -30.0f : b;
        if constexpr (ACT == PC_ACT_GELU) {
            const float e = __builtin_amdgcn_exp2f(-0.5f * kLog2E * (b * b));
            const float t = __builtin_amdgcn_rcpf(1.0f + 0.31f * __builtin_fabsf(b));
            float poly = -0.0208458804f;
            poly = poly * t + 0.103536583f;
            poly = poly * t - 0.183982273f;
            poly = poly * t + 0.119086217f;
            poly = poly * t - 0.0342832404f;
            poly = poly * t + 0.0719690451f;
            poly = poly * t + 0.0850876055f;
            poly = poly * t + 0.112106008f;
            poly = poly * t + 0.123653373f;
            poly = poly * t + 0.123672557f;
            const float tail = e * t * poly;
            const float p = b < 0.0f ? tail : 1.0f - tail;
            y = g * p;
            d = p + b * e * 0.39894228040143267794f;
        } else {
            constexpr float a = 1.59576912160573071176f, c = 0.044715f;
            const float s = b * b;
            float p, q;
            sigmoid(a * b * (1.0f + c * s), p, q);
            y = g * p;
            d = p + b * q * (a * (1.0f + 3.0f * c * s));
        }
    }
}

struct StoredArg {
    const uint8_t *sym, *scale;
    uint64_t ld_sym, ld_scale;
};

constexpr uint32_t kGluPerLane = 2;
constexpr uint32_t kGluTile = kThreads * kGluPerLane;

template <int DT, int FMT, int ACT>
__global__ __launch_bounds__(kThreads) void glu_kernel(const typename Plain<DT>::type *dh, uint64_t ld_dh,
                                                       StoredArg gate, StoredArg up, Units units,
                                                       typename Plain<DT>::type *d_gate, uint64_t ld_gate,
                                                       typename Plain<DT>::type *__restrict__ d_up, uint64_t ld_up,
                                                       typename Plain<DT>::type *__restrict__ h, uint64_t ld_h) {
    const uint64_t base = (uint64_t)blockIdx.x * kGluTile;
    float dv[kGluPerLane][8];
    u32x2 gw[kGluPerLane], uw[kGluPerLane];
    uint32_t gc[kGluPerLane], uc[kGluPerLane], n[kGluPerLane];
    uint64_t row[kGluPerLane], col[kGluPerLane];
#pragma unroll
    for (uint32_t j = 0; j < kGluPerLane; ++j) {
        const uint32_t local = j * kThreads + threadIdx.x;
        n[j] = 0;
        if (base + local < units.total) {
            find_unit(units, base, local, row[j], col[j]);
            n[j] = count_before(units.cols, col[j], kUnit);
        }
        if (n[j]) {
            const uint64_t r = row[j], c = col[j];
            load_unit<DT>(dh + r * ld_dh + c, n[j], dv[j]);
            gw[j] = load_symbols(gate.sym + r * gate.ld_sym + c, n[j]);
            gc[j] = gate.scale[r * gate.ld_scale + c / kGroup];
            if (up.sym) {
                uw[j] = load_symbols(up.sym + r * up.ld_sym + c, n[j]);
                uc[j] = up.scale[r * up.ld_scale + c / kGroup];
            }
        }
    }
#pragma unroll
    for (uint32_t j = 0; j < kGluPerLane; ++j) {
        if (!n[j]) continue;
        const uint64_t r = row[j], c = col[j];
        float g[8], u[8], dg[8], du[8], hv[8];
        unit_values<FMT>(gw[j], scale_of(gc[j]), g);
        if (up.sym) {
            unit_values<FMT>(uw[j], scale_of(uc[j]), u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) u[i] = 1.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y, d;
            activation<ACT>(g[i], y, d);
            dg[i] = dv[j][i] * u[i] * d;
            du[i] = dv[j][i] * y;
            hv[i] = y * u[i];
        }
        store_unit<DT>(d_gate + r * ld_gate + c, n[j], dg);
        if (d_up) store_unit<DT>(d_up + r * ld_up + c, n[j], du);
        if (h) store_unit<DT>(h + r * ld_h + c, n[j], hv);
    }
}

StoredArg stored(const pc_q8 *q) {
    if (!q) return {nullptr, nullptr, 0, 0};
    return {q->sym, q->scale, q->ld_sym, q->ld_scale};
}

bool dense(const pc_q8 *q) { return q->ld_sym == q->cols && q->ld_scale * kGroup == q->cols; }

}  // namespace

hipError_t launch_q8_store(const void *x, int dtype, uint64_t rows, uint64_t cols, uint64_t ldx, int format,
                           uint8_t *sym, uint8_t *scale, uint64_t *counts, hipStream_t stream) {
    const Units units = make_units(rows, cols, ldx == cols);
    const uint64_t groups = (cols + kGroup - 1) / kGroup;
    const uint64_t tile = counts ? kCountThreads * kCountPerLane : kTile, tiles = (units.total + tile - 1) / tile;
    const dim3 grid((uint32_t)(counts ? std::min<uint64_t>(tiles, kCountBlocks) : tiles));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        typedef const typename Plain<DT>::type *P;
        auto launch = [&](auto k) {
            hipLaunchKernelGGL(k, grid, dim3(counts ? kCountThreads : kThreads), 0, stream, static_cast<P>(x), units, ldx, cols, groups, sym,
                               scale, counts);
        };
        if (format == PC_Q8_E4M3)
            counts ? launch(store_kernel<DT, PC_Q8_E4M3, true>) : launch(store_kernel<DT, PC_Q8_E4M3, false>);
        else
            counts ? launch(store_kernel<DT, PC_Q8_INT8, true>) : launch(store_kernel<DT, PC_Q8_INT8, false>);
    });
    return hipGetLastError();
}

hipError_t launch_q8_load(const pc_q8 *q, void *out, int dtype, uint64_t ld_out, hipStream_t stream) {
    const Units units = make_units(q->rows, q->cols, dense(q) && ld_out == q->cols);
    const dim3 grid((uint32_t)((units.total + kLoadTile - 1) / kLoadTile));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        auto launch = [&](auto k) {
            hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, stream, q->sym, q->scale, q->ld_sym, q->ld_scale, units,
                               ld_out, static_cast<typename Plain<DT>::type *>(out));
        };
        q->format == PC_Q8_E4M3 ? launch(load_kernel<DT, PC_Q8_E4M3>) : launch(load_kernel<DT, PC_Q8_INT8>);
    });
    return hipGetLastError();
}

hipError_t launch_q8_glu_backward(const void *dh, int dtype, uint64_t ld_dh, const pc_q8 *gate, const pc_q8 *up,
                                  int act, void *d_gate, uint64_t ld_gate, void *d_up, uint64_t ld_up, void *h,
                                  uint64_t ld_h, hipStream_t stream) {
    const uint64_t cols = gate->cols;
    const bool whole = ld_dh == cols && dense(gate) && ld_gate == cols && (!up || (dense(up) && ld_up == cols)) &&
                       (!h || ld_h == cols);
    const Units units = make_units(gate->rows, cols, whole);
    const dim3 grid((uint32_t)((units.total + kGluTile - 1) / kGluTile));
    with_dtype(dtype, [&](auto d) {
        constexpr int DT = decltype(d)::value;
        typedef typename Plain<DT>::type T;
        auto launch = [&](auto k) {
            hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, stream, static_cast<const T *>(dh), ld_dh, stored(gate),
                               stored(up), units, static_cast<T *>(d_gate), ld_gate, static_cast<T *>(d_up), ld_up,
                               static_cast<T *>(h), ld_h);
        };
        auto by_act = [&](auto f) {
            constexpr int FMT = decltype(f)::value;
            if (act == PC_ACT_SILU) launch(glu_kernel<DT, FMT, PC_ACT_SILU>);
            else if (act == PC_ACT_GELU) launch(glu_kernel<DT, FMT, PC_ACT_GELU>);
            else launch(glu_kernel<DT, FMT, PC_ACT_GELU_TANH>);
        };
        if (gate->format == PC_Q8_E4M3) by_act(std::integral_constant<int, PC_Q8_E4M3>());
        else by_act(std::integral_constant<int, PC_Q8_INT8>());
    });
    return hipGetLastError();
}

}  // namespace pc
