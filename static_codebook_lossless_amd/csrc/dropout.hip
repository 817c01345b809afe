// Dropout: out = mask(x), the mask made from a counter in the kernel.  Its
// backward pass is the same call on the gradient.  One call of the generator
// serves the 8 columns of a lane's unit.  4096 x 16384 bf16: 46-47 us, 5.8 TB/s,
// which memory bounds (vector work 59%); 64 x 2048: 3.2 us, a launch's own time.
#include "random.h"

namespace pc {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kPerLane = 2;  // units per lane
constexpr uint32_t kTile = kThreads * kPerLane;

template <int DT>
__global__ __launch_bounds__(kThreads) void dropout_kernel(const typename Plain<DT>::type *x, uint64_t ldx, Units units,
                                                           MaskArg mask, typename Plain<DT>::type *out,
                                                           uint64_t ld_out) {
    const uint64_t base = (uint64_t)blockIdx.x * kTile;
    const MaskKey key = mask_key(mask);
    RawUnit<DT> raw[kPerLane];
    uint32_t n[kPerLane];
    uint64_t row[kPerLane], col[kPerLane];
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        const uint32_t local = j * kThreads + threadIdx.x;
        n[j] = 0;
        row[j] = col[j] = 0;
        if (base + local < units.total) {
            find_unit(units, base, local, row[j], col[j]);
            n[j] = count_before(units.cols, col[j], kUnit);
        }
        raw[j] = load_raw<DT>(x + row[j] * ldx + col[j], n[j]);
    }
#pragma unroll
    for (uint32_t j = 0; j < kPerLane; ++j) {
        if (!n[j]) continue;
        float v[8];
        widen_unit<DT>(raw[j], v);
        drop_unit(mask, key, row[j], (uint32_t)col[j], v);
        store_unit<DT>(out + row[j] * ld_out + col[j], n[j], v);
    }
}

}  // namespace

hipError_t launch_dropout(const void *x, int dtype, uint64_t rows, uint64_t cols, uint64_t ldx, const pc_mask *mask,
                          void *out, uint64_t ld_out, hipStream_t stream) {
    const Units units = make_units(rows, cols, false);  // the mask goes by row and column
    const dim3 grid((uint32_t)((units.total + kTile - 1) / kTile));
    with_dtype(dtype, [&](auto d) {
        typedef typename Plain<decltype(d)::value>::type T;
        hipLaunchKernelGGL(dropout_kernel<decltype(d)::value>, grid, dim3(kThreads), 0, stream,
                           static_cast<const T *>(x), ldx, units, mask_arg(mask), static_cast<T *>(out), ld_out);
    });
    return hipGetLastError();
}

}  // namespace pc
