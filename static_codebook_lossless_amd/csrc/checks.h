// Argument checks that the entry points of the tensor operators share.
#pragma once

#include "pc_internal.h"

namespace pc {
namespace checks {

// A launch has fewer than 2^24 workgroups of 256 lanes; the smallest tile is
// 512 units of 8 columns.
constexpr uint64_t kMaxGroups = (1ull << 24) - 1;
constexpr uint64_t kMaxWidth = 1ull << 31;
constexpr uint64_t kMaxDistance = 1ull << 24;  // weight gradient: offsets inside a tile of 64 rows stay below 2^32 bytes
constexpr uint64_t kMaxElements = 1ull << 47;  // beyond any memory; keeps sizes below 64 bits

inline bool is_dtype(int d) { return d == PC_F32 || d == PC_F16 || d == PC_BF16; }
inline bool is_format(int f) { return f == PC_Q8_E4M3 || f == PC_Q8_INT8; }

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// rows x cols elements of a dtype at p, row distance ld.
inline bool plain_ok(const void *p, int dtype, size_t cols, size_t ld) {
    return p && ld >= cols && aligned(p, dtype == PC_F32 ? 4 : 2);
}

inline bool stored_ok(const pc_q8 *q) {
    return q->sym && q->scale && q->ld_sym >= q->cols && q->ld_scale >= (q->cols + 31) / 32;
}

inline bool size_ok(uint64_t rows, uint64_t cols) {
    if (cols >= kMaxWidth) return false;
    if (cols == 0 || rows == 0) return true;
    const uint64_t padded = (cols + 31) / 32 * 32;
    return rows <= kMaxElements / padded && (rows * (padded / 8) + 511) / 512 <= kMaxGroups;
}

// The distance from a tensor's first to its last row fits 63 bits in bytes.
inline bool span_ok(uint64_t rows, uint64_t ld) { return rows == 0 || ld <= (1ull << 60) / rows; }

inline pc_status map_hip(hipError_t e) { return e == hipSuccess ? PC_OK : PC_ERR_HIP; }

}  // namespace checks
}  // namespace pc
