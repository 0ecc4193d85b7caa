// zccl_norm_bf16_f32.cu -- the forward norm kernels of a residual and a block of these types.
#include "zccl_norm_forward.cuh"

namespace zccl {
template NormKernel norm_kernel_for<__nv_bfloat16, float>(const Shape&, bool, bool, bool, uint32_t*);
}  // namespace zccl
