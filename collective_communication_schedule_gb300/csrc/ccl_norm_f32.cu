// The norm's kernels for rows of f32.
#include "ccl_norm_kernels.cuh"

namespace ccl {
namespace tensor {

const NormKernels& norm_kernels_f32_f32()
{
    static const NormKernels k = norm_kernels_of<CCL_F32, CCL_F32>();
    return k;
}

}  // namespace tensor
}  // namespace ccl
