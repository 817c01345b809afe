// Root-mean-square norm with what a residual block does around it: dropout of
// the block's output, the residual's addition, the norm, and the norm's output
// stored in 8 bits; and the backward pass of all of that.
//
//   h = round(res + mask(x)),  r = (mean(h^2) + eps)^-1/2,  y = h r w
//   d = r (g - n mean(g n)) + d_sum,  g = dy w,  n = h r
//   d_res = d,  d_x = mask(d),  d_w = sum over rows of dy n
#include <algorithm>

#include "norm.h"

namespace pc {
namespace {

// The sums of `parts` rows of partial sums, 16 columns to a workgroup: its 64
// groups of 16 lanes take every 64th row, and their sums are added in order.
constexpr uint32_t kJoinColumns = 16;
constexpr uint32_t kJoinGroups = kMaxThreads / kJoinColumns;

template <int DT>
__global__ __launch_bounds__(kMaxThreads) void norm_join_kernel(const float *__restrict__ partial, uint64_t ld,
                                                                uint32_t parts, uint32_t cols, int accumulate,
                                                                typename Plain<DT>::type *__restrict__ out) {
    __shared__ float sums[kJoinGroups][kJoinColumns];
    const uint32_t lane = threadIdx.x % kJoinColumns, group = threadIdx.x / kJoinColumns;
    for (uint32_t first = blockIdx.x * kJoinColumns; first < cols; first += gridDim.x * kJoinColumns) {
        const uint32_t col = first + lane;
        float s = 0.0f;
        if (col < cols) {
#pragma unroll 4
            for (uint32_t i = group; i < parts; i += kJoinGroups) s += partial[i * ld + col];
        }
        sums[group][lane] = s;
        __syncthreads();
        if (group == 0 && col < cols) {
            float t = sums[0][lane];
            for (uint32_t i = 1; i < kJoinGroups; ++i) t += sums[i][lane];
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

// The lanes of a row with `per` units each: whole waves, or 16 or 32 with one unit each.
uint32_t team_for(uint32_t units, uint32_t per, bool parts_of_waves) {
    const uint32_t lanes = (units + per - 1) / per;
    if (parts_of_waves && per == 1 && lanes <= 16) return 16;
    if (parts_of_waves && per == 1 && lanes <= 32) return 32;
    return std::min(kMaxThreads, (lanes + kWave - 1) / kWave * kWave);
}

// The lanes of a workgroup of whole teams: `most`, or a little less, where teams are small.
uint32_t lanes_for(uint32_t team, uint32_t most) { return std::max(team, most / team * team); }

// Inputs of so many bytes, which the memory-side cache does not hold, stream
// past the caches.  Forward, 8192 x 8192 bf16 with a mask (256 MiB): 111 us,
// streamed 106; 8192 x 4096: 52.7 and 53.5; 8192 x 2048: 26.0 and 30.8.
// Backward, 8192 x 8192 with the sum in e4m3: 100 and 97 us; 8192 x 4096 (192
// MiB): 49.5 and 55.4.
constexpr uint64_t kStreamBytes = 256ull << 20;

uint64_t size_of(int dtype) { return dtype == PC_F32 ? 4 : 2; }

// Units a lane: one for rows of a wave, then two (8192 x 4096 bf16: 52.7 us,
// with one 58.4, with four 54.4), four where the workgroup would be over 1024
// lanes, and for streamed rows from half of that on (8192 x 8192 with a mask:
// 104 us, with two 106).  Counting and ragged widths make do with two; longer
// rows are read twice.
NormPlan plan_norm(const RmsNorm &c, uint32_t &team) {
    NormPlan p = {};
    const uint32_t units = units_of(c.cols);
    const bool count = c.counts != nullptr;
    p.whole = c.cols % kUnit == 0 && !count;
    p.streams = c.rows * c.cols * (size_of(c.dtype) + (c.res ? size_of(c.sum_dtype) : 0)) >= kStreamBytes;
    p.per = units <= kWave ? 1 : 2;
    if (p.whole && (units > 2 * kMaxThreads || (p.streams && units >= kMaxThreads))) p.per = 4;
    p.is_long = units > p.per * kMaxThreads;
    team = team_for(units, p.is_long ? 4 : p.per, p.whole);
    p.threads = lanes_for(team, count ? kMaxThreads : 256);
    const uint64_t teams = p.threads / team, wanted = (c.rows + teams - 1) / teams;
    p.blocks = (uint32_t)std::min<uint64_t>(wanted, count ? kCountBlocks : (1u << 22) - 1);
    return p;
}

// One unit a lane; two where the workgroup would be over 1024 lanes, and for
// streamed rows from half of that on (8192 x 8192 bf16 with the sum in e4m3:
// 87 us, with one 97); f32 has no registers for two (4096 x 8192: 109 and 200
// us), so its rows of over 8192 columns are read twice.  Workgroups for 1024
// lanes on every CU: more of them have more partial sums to write and join
// (8192 x 4096: 49.5, 57.0 and 62.8 us for one, two and four times as many).
GradPlan plan_grad(uint64_t rows, uint64_t cols, bool f32, uint64_t bytes) {
    GradPlan p = {};
    const uint32_t units = units_of(cols);
    p.whole = cols % kUnit == 0;
    p.streams = bytes >= kStreamBytes;
    p.per = 1;
    if (!f32 && (units > kMaxThreads || (p.streams && units >= kMaxThreads))) p.per = 2;
    if (units > p.per * kMaxThreads) p.per = 0;
    if (p.per) {
        p.team = team_for(units, p.per, p.whole);
        p.threads = p.per == 1 ? lanes_for(p.team, kGradThreads) : p.team;
        const uint64_t teams = p.threads / p.team, wanted = (rows + teams - 1) / teams;
        const uint32_t on_a_cu = std::max(1u, (kMaxThreads + p.threads / 2) / p.threads);
        p.blocks = (uint32_t)std::min<uint64_t>(wanted, 256 * on_a_cu);
        p.parts = p.blocks;
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

// Rows and columns in one launch, by sizes alone.  bf16, in one launch and in two,
// on the device with inputs from HBM (as a captured step has it) and with the host's
// share of an eager pass: 128 x 2048 5.0 and 7.2, 10.6 and 14.9 us; 512 x 8192 15.5 and
// 17.2, 15.1 and 16.9; 512 x 4096 10.2 and 16.6, 10.8 and 16.3; 512 x 1024 11.6 and 7.4,
// 11.3 and 14.8: narrow rows gain with the host's share alone.  Beyond the rule one launch
// is the slower one: 1024 x 1024 on the device 15.1 and 8.6, 2048 x 2048 39 and 17.
constexpr uint64_t kOnceRows = 512, kOnceElements = 1ull << 22;

bool once_fits(uint64_t rows, uint64_t cols) {
    return rows <= kOnceRows && rows * cols <= kOnceElements && units_of(cols) <= kMaxThreads;
}

// The same plan for one launch; the columns' workgroups come after the rows'.
GradPlan plan_once(uint64_t rows, uint64_t cols, uint32_t &row_blocks) {
    GradPlan p = {};
    p.once = true;
    p.per = 1;
    p.team = team_for(units_of(cols), 1, false);
    p.threads = lanes_for(p.team, kGradThreads);
    const uint64_t teams = p.threads / p.team;
    row_blocks = (uint32_t)((rows + teams - 1) / teams);
    p.blocks = row_blocks + (uint32_t)((cols + kOnceColumns - 1) / kOnceColumns);
    return p;
}

uint64_t partial_width(uint64_t cols) { return (cols + 3) / 4 * 4; }

}  // namespace

hipError_t launch_rmsnorm_store(const RmsNorm &c, hipStream_t stream) {
    NormArgs a = {};
    const NormPlan p = plan_norm(c, a.team);
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
    const bool wide = c.sum_dtype == PC_F32;
    if (c.dtype == PC_F32) return norm_forward<PC_F32, PC_F32>(a, p, stream);
    if (c.dtype == PC_F16)
        return wide ? norm_forward<PC_F16, PC_F32>(a, p, stream) : norm_forward<PC_F16, PC_F16>(a, p, stream);
    return wide ? norm_forward<PC_BF16, PC_F32>(a, p, stream) : norm_forward<PC_BF16, PC_BF16>(a, p, stream);
}

uint64_t rmsnorm_backward_workspace(uint64_t rows, uint64_t cols) {
    if (once_fits(rows, cols)) return 0;
    // the largest of any types'
    uint32_t parts = 0;
    for (int f32 = 0; f32 < 2; ++f32)
        for (int streams = 0; streams < 2; ++streams)
            parts = std::max(parts, plan_grad(rows, cols, f32, streams ? kStreamBytes : 0).parts);
    return (uint64_t)parts * partial_width(cols) * sizeof(float);
}

hipError_t launch_rmsnorm_backward(const RmsNormGrad &c, hipStream_t stream) {
    const uint64_t kept = c.stored ? 1 : size_of(c.sum_dtype), d_sum = c.d_sum ? size_of(c.sum_dtype) : 0;
    GradArgs a = {};
    const bool once = c.d_weight && c.rows && once_fits(c.rows, c.cols);
    GradPlan p = once ? plan_once(c.rows, c.cols, a.row_blocks)
                      : plan_grad(c.rows, c.cols, c.sum_dtype == PC_F32,
                                  c.rows * c.cols * (size_of(c.dtype) + kept + d_sum));
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
    a.partial = c.d_weight && !once ? static_cast<float *>(c.ws) : nullptr;
    a.d_weight = c.d_weight;
    a.d_weight_kind = c.d_weight_dtype;
    a.accumulate = c.accumulate;
    a.rows = c.rows;
    a.ld_dy = c.ld_dy;
    a.ld_d_sum = c.ld_d_sum;
    a.ld_d_res = c.ld_d_res;
    a.ld_d_x = c.ld_d_x;
    a.ld_partial = partial_width(c.cols);
    a.cols = (uint32_t)c.cols;
    a.team = p.team;
    p.columns_first = (c.d_x && (c.d_x == c.sum || c.d_x == c.dy)) || (c.d_res && (c.d_res == c.sum || c.d_res == c.dy));
    a.per_col = (float)(1.0 / (double)c.cols);
    a.mask = mask_arg(c.mask);
    if (c.rows) {
        const bool wide = c.sum_dtype == PC_F32;
        hipError_t e;
        if (c.dtype == PC_F32)
            e = norm_backward<PC_F32, PC_F32>(a, p, stream);
        else if (c.dtype == PC_F16)
            e = wide ? norm_backward<PC_F16, PC_F32>(a, p, stream) : norm_backward<PC_F16, PC_F16>(a, p, stream);
        else
            e = wide ? norm_backward<PC_BF16, PC_F32>(a, p, stream) : norm_backward<PC_BF16, PC_BF16>(a, p, stream);
        if (e != hipSuccess) return e;
    }
    if (c.d_weight && !once) {
        const dim3 grid((uint32_t)std::min<uint64_t>((c.cols + kJoinColumns - 1) / kJoinColumns, 1u << 16));
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
