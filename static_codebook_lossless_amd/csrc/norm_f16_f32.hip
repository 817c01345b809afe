// The norm's kernels for x in f16 and a sum in f32.
#include "norm_kernels.h"

namespace pc {

template <>
hipError_t norm_forward<PC_F16, PC_F32>(const NormArgs &a, const NormPlan &p, hipStream_t stream) {
    return launch_norm<PC_F16, PC_F32>(a, p, stream);
}

template <>
hipError_t norm_backward<PC_F16, PC_F32>(const GradArgs &a, const GradPlan &p, hipStream_t stream) {
    return launch_norm_grad<PC_F16, PC_F32>(a, p, stream);
}

}  // namespace pc
