// zccl_norm_f32_f32.cu -- the forward norm kernels of a residual and a block of these types.
#include "zccl_norm_forward.cuh"

namespace zccl {
template NormKernel norm_kernel_for<float, float>(const Shape&, bool, bool, bool, uint32_t*);
}  // namespace zccl
