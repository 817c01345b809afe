// Arguments and launch plans of the norm's kernels (norm_kernels.h), which are
// compiled for one pair of types at a time (norm_f32.hip and so on: together
// they would take minutes), and launched from norm.hip.
#pragma once

#include "random.h"

namespace pc {

constexpr uint32_t kMaxThreads = 1024;
constexpr uint32_t kCountBlocks = 256;  // workgroups of the counting form
constexpr uint32_t kGradThreads = 256;
constexpr uint32_t kOnceColumns = 64;  // of a workgroup, where rows and columns share a launch
constexpr uint32_t kColumnThreads = 256;  // weight gradient of long rows
constexpr uint32_t kColumnWaves = kColumnThreads / kWave;

struct NormArgs {
    const void *x, *res, *weight;
    void *sum, *y;
    uint8_t *sym, *scale;
    uint64_t *counts;
    float *rstd;
    uint64_t rows, ldx, ld_res, ld_sum, ld_y;
    uint32_t cols, groups;
    uint32_t team;  // lanes to a row: whole waves, or 16 or 32 of one
    int weight_kind, y_kind, format, y_stored;
    double eps, per_col;  // per_col: 1 / cols
    MaskArg mask;
};

struct GradArgs {
    const void *dy, *sum, *d_sum, *weight;
    const uint8_t *sym, *scale;  // the sum in its stored form, in place of `sum`
    const float *rstd;
    void *d_res, *d_x;
    float *partial;  // partial sums, [GradPlan::parts][ld_partial] (a row for each workgroup, or for each wave where rows are long), or nullptr
    uint64_t rows, ld_dy, ld_sum, ld_sym, ld_scale, ld_d_sum, ld_d_res, ld_d_x, ld_partial;
    uint32_t cols, team;
    int weight_kind, format;
    float per_col;  // 1 / cols
    MaskArg mask;
    // rows and columns in one launch
    void *d_weight;
    int d_weight_kind, accumulate;
    uint32_t row_blocks;
};

// How a call is split, by rules on sizes alone (norm.hip).
struct NormPlan {
    uint32_t per, threads, blocks;
    bool whole, is_long, streams;
};

struct GradPlan {
    uint32_t per, team, threads, blocks;  // per == 0: long rows
    uint32_t parts;                       // rows of partial sums
    uint32_t column_blocks, slices;       // of the long rows' weight gradient
    bool whole, streams, once;            // once: blocks for rows and for columns in one launch
    bool columns_first;                   // of these, the columns' in a launch before: the rows' write what they read
};


// Launches for x of type DT and a sum of type RT.
template <int DT, int RT>
hipError_t norm_forward(const NormArgs &a, const NormPlan &p, hipStream_t stream);
template <int DT, int RT>
hipError_t norm_backward(const GradArgs &a, const GradPlan &p, hipStream_t stream);

}  // namespace pc
