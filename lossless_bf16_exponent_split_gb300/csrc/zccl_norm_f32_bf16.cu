// zccl_norm_f32_bf16.cu -- the forward norm kernels of a residual and a block of these types.
#include "zccl_norm_forward.cuh"

namespace zccl {
template NormKernel norm_kernel_for<float, __nv_bfloat16>(const Shape&, bool, bool, bool, uint32_t*);
}  // namespace zccl
