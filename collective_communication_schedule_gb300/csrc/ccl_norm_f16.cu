// The norm's kernels for rows of f16.
#include "ccl_norm_kernels.cuh"

namespace ccl {
namespace tensor {

const NormKernels& norm_kernels_f16_f16()
{
    static const NormKernels k = norm_kernels_of<CCL_F16, CCL_F16>();
    return k;
}
const NormKernels& norm_kernels_f16_f32()
{
    static const NormKernels k = norm_kernels_of<CCL_F16, CCL_F32>();
    return k;
}

}  // namespace tensor
}  // namespace ccl
