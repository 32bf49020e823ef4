// The norm's kernels for rows of bf16.
#include "ccl_norm_kernels.cuh"

namespace ccl {
namespace tensor {

const NormKernels& norm_kernels_bf16_bf16()
{
    static const NormKernels k = norm_kernels_of<CCL_BF16, CCL_BF16>();
    return k;
}
const NormKernels& norm_kernels_bf16_f32()
{
    static const NormKernels k = norm_kernels_of<CCL_BF16, CCL_F32>();
    return k;
}

}  // namespace tensor
}  // namespace ccl
