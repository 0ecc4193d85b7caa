// zccl_norm_backward_f32_f32.cu -- the backward norm kernels of a residual and a block of these types.
#include "zccl_norm_backward.cuh"

namespace zccl {
template NormKernel norm_backward_kernel_for<float, float>(const Shape&, bool, bool, bool, uint32_t*);
}  // namespace zccl
