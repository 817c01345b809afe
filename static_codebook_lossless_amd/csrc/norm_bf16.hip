// The norm's kernels for x in bf16 and a sum in bf16.
#include "norm_kernels.h"

namespace pc {

template <>
hipError_t norm_forward<PC_BF16, PC_BF16>(const NormArgs &a, const NormPlan &p, hipStream_t stream) {
    return launch_norm<PC_BF16, PC_BF16>(a, p, stream);
}

template <>
hipError_t norm_backward<PC_BF16, PC_BF16>(const GradArgs &a, const GradPlan &p, hipStream_t stream) {
    return launch_norm_grad<PC_BF16, PC_BF16>(a, p, stream);
}

}  // namespace pc
