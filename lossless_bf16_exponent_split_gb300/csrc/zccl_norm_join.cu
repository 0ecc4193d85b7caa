// zccl_norm_join.cu -- a backward pass's launch, and the kernel that adds the workers'
// sums of the weights' and the gate's gradients up.
#include "zccl_norm.h"

namespace zccl {

namespace {

// Adds the partial sums up: blockIdx.y = 0, 1 a weight's, 2 + i those of a gate row that
// several workers have parts of: gate row i (kByRow), or the one that goes on behind
// worker i's rows.
constexpr uint32_t kJoinRows = 32;  // partial sums of a column that are added side by side

template <bool kByRow>
__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(NormArgs a, int weight_dtype)
{
    __shared__ float red[kJoinRows][33];
    pdl_wait();
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const uint32_t lane = threadIdx.x & 31, sub = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, job = blockIdx.y;
    float sum = 0.0f;
    void* out;
    int dtype = weight_dtype;
    uint64_t at = col;
    if (job < 2) {
        out = job == 0 ? a.grad_weight : a.grad_post_weight;
        if (out == nullptr) return;
        const float* p = a.sums + job * pitch + col;
        if (col < a.hidden)
#pragma unroll 8
            for (uint32_t g = sub; g < a.groups; g += kJoinRows) sum += p[g * kWeightSlots * pitch];
    } else {
        uint64_t gate_row = job - 2;
        if (!kByRow) {
            const uint64_t next = first_row(a.rows, a.workers, job - 2 + 1);
            gate_row = (next - 1) / a.gate_span;
        }
        const uint64_t begin = gate_row * a.gate_span, end = begin + a.gate_span < a.rows ? begin + a.gate_span : a.rows;
        const uint32_t from = worker_of(a.rows, a.workers, begin), to = worker_of(a.rows, a.workers, end - 1);
        if (from == to || (!kByRow && from != job - 2)) return;  // the worker's own, or another's to add up
        if (col < a.hidden)
#pragma unroll 4
            for (uint32_t w = from + sub; w <= to; w += kJoinRows)
                sum += a.parts[((uint64_t)w * kGateSlots + (w == from ? kSlotBehind : kSlotBefore)) * pitch + col];
        out = a.grad_gate;
        dtype = a.gate.dtype;
        at += gate_row * a.hidden;
    }
    red[sub][lane] = sum;
    __syncthreads();
    if (sub != 0 || col >= a.hidden) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) sum += red[i][lane];
    if (dtype == ZCCL_BF16)
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(sum);
    else
        static_cast<float*>(out)[at] = sum;
}

cudaError_t launch_join(const NormArgs& a, int weight_dtype, cudaStream_t stream)
{
    const bool gate = a.grad_gate != nullptr && a.gate_span > 1 && a.workers > 1;
    if (a.grad_weight == nullptr && a.grad_post_weight == nullptr && !gate) return cudaSuccess;
    const uint64_t gate_rows = (a.rows + a.gate_span - 1) / a.gate_span;
    const bool by_row = gate_rows < a.workers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.hidden + 31) / 32, !gate ? 2 : by_row ? 2 + (uint32_t)gate_rows : 2 + a.workers - 1);
    cfg.blockDim = dim3(32 * kJoinRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, by_row ? norm_join_kernel<true> : norm_join_kernel<false>, a, weight_dtype);
}

}  // namespace

zccl_status_t launch_norm_backward(NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec, cudaStream_t stream)
{
    const Shape s = norm_shape(a.hidden, a.rows, vec && x_dtype == ZCCL_BF16 && dtype == ZCCL_BF16);
    a.workers = s.workers;
    a.groups = s.grid / s.ctas;
    a.parts = a.sums + (uint64_t)a.groups * kWeightSlots * ((a.hidden + 7) / 8 * 8);
    const bool post = a.post, drop = a.drop.below > 0 && a.grad_y != nullptr;
    uint32_t thread_bytes = 0;
    const NormKernel kernel =
        x_dtype == ZCCL_BF16
            ? (dtype == ZCCL_BF16 ? norm_backward_kernel_for<__nv_bfloat16, __nv_bfloat16>(s, vec, post, drop, &thread_bytes)
                                  : norm_backward_kernel_for<__nv_bfloat16, float>(s, vec, post, drop, &thread_bytes))
            : (dtype == ZCCL_BF16 ? norm_backward_kernel_for<float, __nv_bfloat16>(s, vec, post, drop, &thread_bytes)
                                  : norm_backward_kernel_for<float, float>(s, vec, post, drop, &thread_bytes));
    const uint32_t threads = s.warps * 32;
    const size_t smem = s.team == kLong ? 0 : threads * thread_bytes + kTeamRed * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (smem > 48 << 10) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = s.team == kClusterTeam ? launch_clusters(kernel, s.grid, threads, smem, s.ctas, stream, a)
                                   : launch_dependent(kernel, s.grid, threads, smem, stream, a);
    if (e == cudaSuccess) e = launch_join(a, weight_dtype, stream);
    return launched(e);
}

}  // namespace zccl
