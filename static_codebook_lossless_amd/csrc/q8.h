// Device helpers of the stored-tensor operators: 8 consecutive elements of a
// row at a time, in the plain types and in the 8-bit form.
#pragma once

#include <type_traits>

#include "pc_internal.h"

namespace pc {

constexpr uint32_t kGroup = PC_Q8_GROUP;  // columns per scale code
constexpr uint32_t kUnit = 8;             // columns one lane handles at a time
constexpr uint32_t kUnitsPerGroup = kGroup / kUnit;
constexpr uint32_t kMinCode = 10;         // 2^-117: the smallest element (2^-9 in e4m3) stays a normal number

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Rows may start anywhere an element may: vectors of a smaller alignment
// than their size, which the hardware loads and stores in one instruction.
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));

template <int DT> struct Plain;
template <> struct Plain<PC_F32> { typedef float type; };
template <> struct Plain<PC_F16> { typedef _Float16 type; };
template <> struct Plain<PC_BF16> { typedef __bf16 type; };

__device__ __forceinline__ float as_f32(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t as_u32(float f) { return __builtin_bit_cast(uint32_t, f); }

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
__device__ __forceinline__ float widen(__bf16 v) { return as_f32((uint32_t)__builtin_bit_cast(uint16_t, v) << 16); }

// How many of the `most` places from `at` on lie before `end`.  The difference
// is one that is valid for every `at`:  of  at < end ? min(end - at, most) : 0
// the compiler forms the minimum ahead of the test, takes at <= end as given
// from there on, and drops other clamps that this would make needless (loads
// then ran past the end of rows).
template <class T>
__device__ __forceinline__ uint32_t count_before(T end, T at, uint32_t most) {
    const T past = at > end ? at : end, left = past - at;
    return left < most ? (uint32_t)left : most;
}

// n (0..8) elements as loaded; the others 0.
template <int DT> struct RawUnit { u32x4 w[DT == PC_F32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ RawUnit<DT> load_raw(const typename Plain<DT>::type *p, uint32_t n) {
    RawUnit<DT> r = {};
    if (n == kUnit) {
        if constexpr (DT == PC_F32) {
            r.w[0] = *reinterpret_cast<const u32x4_any4 *>(p);
            r.w[1] = *reinterpret_cast<const u32x4_any4 *>(p + 4);
        } else {
            r.w[0] = *reinterpret_cast<const u32x4_any2 *>(p);
        }
    } else if (n) {
#pragma unroll
        for (uint32_t i = 0; i < kUnit; ++i)
            if (i < n) {
                if constexpr (DT == PC_F32) r.w[i / 4][i % 4] = as_u32(p[i]);
                else r.w[0][i / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, p[i]) << (16 * (i % 2));
            }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void widen_unit(const RawUnit<DT> &r, float v[8]) {
    if constexpr (DT == PC_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = as_f32(r.w[i / 4][i % 4]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = r.w[0][i];
            if constexpr (DT == PC_BF16) {
                v[2 * i] = as_f32(u << 16);
                v[2 * i + 1] = as_f32(u & 0xFFFF0000u);
            } else {
                const f16x2 h = __builtin_bit_cast(f16x2, u);
                v[2 * i] = (float)h[0];
                v[2 * i + 1] = (float)h[1];
            }
        }
    }
}

// n (1..8) elements at p as f32; the others 0.
template <int DT>
__device__ __forceinline__ void load_unit(const typename Plain<DT>::type *p, uint32_t n, float v[8]) {
    widen_unit<DT>(load_raw<DT>(p, n), v);
}

// A vector store at an address of a smaller alignment; STREAM: the caches need
// not keep it.
template <uint32_t ALIGN, bool STREAM, class V>
__device__ __forceinline__ void put(void *p, V v) {
    typedef V any __attribute__((aligned(ALIGN)));
    if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<any *>(p));
    else *static_cast<any *>(p) = v;
}

// The first n (1..8) values of v, rounded to the type, at p.  16-bit types,
// whose lanes write 16 bytes side by side, stream past the caches (64 MiB read
// back in bf16: 34.8 -> 30.2 us, a lookup of 256 MiB: 89 -> 56 us, no
// difference at 16 MiB); in f32 the two halves of a lane lie 32 bytes apart
// and would each be written as part of a line (27.6 -> 52.7 us).
template <int DT>
__device__ __forceinline__ void store_unit(typename Plain<DT>::type *p, uint32_t n, const float v[8]) {
    typedef typename Plain<DT>::type T;
    if (n == kUnit) {
        if constexpr (DT == PC_F32) {
            u32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = as_u32(v[i]);
                b[i] = as_u32(v[4 + i]);
            }
            *reinterpret_cast<u32x4_any4 *>(p) = a;
            *reinterpret_cast<u32x4_any4 *>(p + 4) = b;
        } else {
            typedef T t2 __attribute__((ext_vector_type(2)));
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x2 f = {v[2 * i], v[2 * i + 1]};
                a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, t2));
            }
            put<2, true>(p, a);
        }
    } else {
#pragma unroll
        for (uint32_t i = 0; i < kUnit; ++i)
            if (i < n) p[i] = (T)v[i];
    }
}

// n (1..8) symbols at p, in the bytes of a pair of words; the others 0.
__device__ __forceinline__ u32x2 load_symbols(const uint8_t *p, uint32_t n) {
    if (n == kUnit) return *reinterpret_cast<const u32x2_any *>(p);
    u32x2 w = {0, 0};
#pragma unroll
    for (uint32_t i = 0; i < kUnit; ++i)
        if (i < n) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
    return w;
}

__device__ __forceinline__ void store_symbols(uint8_t *p, uint32_t n, u32x2 w) {
    if (n == kUnit) {
        *reinterpret_cast<u32x2_any *>(p) = w;
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < kUnit; ++i)
        if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
}

// 2^(code - 127) for codes 1..254.
__device__ __forceinline__ float scale_of(uint32_t code) { return as_f32(code << 23); }

// The values of 8 symbols.  int8: the byte with its sign bit turned over is
// the element plus 128.
template <int FMT>
__device__ __forceinline__ void unit_values(u32x2 w, float scale, float v[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if constexpr (FMT == PC_Q8_E4M3) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], false);
            const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[k], true);
            v[4 * k] = lo[0] * scale;
            v[4 * k + 1] = lo[1] * scale;
            v[4 * k + 2] = hi[0] * scale;
            v[4 * k + 3] = hi[1] * scale;
        } else {
            const uint32_t u = w[k] ^ 0x80808080u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[4 * k + i] = ((float)((u >> (8 * i)) & 0xFFu) - 128.0f) * scale;
            // a byte of u is 0 exactly where the symbol is 0x80
            if ((u - 0x01010101u) & ~u & 0x80808080u) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (((u >> (8 * i)) & 0xFFu) == 0) v[4 * k + i] = __builtin_nanf("");
            }
        }
    }
}

// Division of t < 2^31 by a number fixed before the launch.
struct Divider {
    uint32_t d, magic, shift;
    explicit Divider(uint32_t by = 1) : d(by), magic(0), shift(0) {
        while ((1ull << shift) < by) ++shift;
        magic = (uint32_t)((((1ull << shift) - by) << 32) / by + 1);
    }
    __device__ __forceinline__ uint32_t over(uint32_t t) const { return (__umulhi(t, magic) + t) >> shift; }
};

// The units of a rows x cols tensor, each row's count rounded up to whole
// groups.  A tensor whose rows all lie end to end in whole groups is one row.
struct Units {
    uint64_t total, cols;
    Divider per_row;
    uint32_t flat;
};

inline Units make_units(uint64_t rows, uint64_t cols, bool dense) {
    Units u;
    const uint64_t per = (cols + kGroup - 1) / kGroup * kUnitsPerGroup;
    u.flat = dense && cols % kGroup == 0;
    u.total = rows * per;
    u.cols = u.flat ? rows * cols : cols;
    u.per_row = Divider(u.flat ? 1u : (uint32_t)per);
    return u;
}

// Row and first column of unit base + local (base the same for all lanes).
__device__ __forceinline__ void find_unit(const Units &u, uint64_t base, uint32_t local, uint64_t &row, uint64_t &col) {
    if (u.flat) {
        row = 0;
        col = (base + local) * kUnit;
        return;
    }
    const uint32_t d = u.per_row.d;
    uint64_t r0;
    uint32_t c0;
    if ((base >> 32) == 0) {
        r0 = (uint32_t)base / d;
        c0 = (uint32_t)base % d;
    } else {
        r0 = base / d;
        c0 = (uint32_t)(base % d);
    }
    const uint32_t t = c0 + local, q = u.per_row.over(t);
    row = r0 + q;
    col = (uint64_t)(t - q * d) * kUnit;
}

// Calls f with a compile-time dtype; false for an unknown one.
template <class F>
__host__ __device__ inline bool with_dtype(int dtype, F &&f) {
    switch (dtype) {
        case PC_F32: f(std::integral_constant<int, PC_F32>()); return true;
        case PC_F16: f(std::integral_constant<int, PC_F16>()); return true;
        case PC_BF16: f(std::integral_constant<int, PC_BF16>()); return true;
    }
    return false;
}

}  // namespace pc
