// The norm's kernels for rows of f16.
#include "ccl_norm_kernels.cuh"

namespace ccl {
namespace tensor {

const NormKernels& norm_kernels_f16_f16() { return norm_kernels_of<CCL_F16, CCL_F16>(); }
const NormKernels& norm_kernels_f16_f32() { return norm_kernels_of<CCL_F16, CCL_F32>(); }

}  // namespace tensor
}  // namespace ccl
