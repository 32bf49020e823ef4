// The norm's kernels for rows of bf16.
#include "ccl_norm_kernels.cuh"

namespace ccl {
namespace tensor {

const NormKernels& norm_kernels_bf16_bf16() { return norm_kernels_of<CCL_BF16, CCL_BF16>(); }
const NormKernels& norm_kernels_bf16_f32() { return norm_kernels_of<CCL_BF16, CCL_F32>(); }

}  // namespace tensor
}  // namespace ccl
