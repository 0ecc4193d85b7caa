// zccl_norm_join.cu -- a backward pass's launch, and the kernel that adds the workers'
// sums of the weights' and the gate's gradients up.
#include "zccl_norm.h"

namespace zccl {

namespace {

// The workers that have parts of a gate row.
struct Sharers {
    uint32_t from, to;
};
__device__ __forceinline__ Sharers sharers(const NormArgs& a, uint32_t gate_row)
{
    const uint32_t begin = gate_row * a.gate_span, end = begin + a.gate_span < a.rows ? begin + a.gate_span : a.rows;
    return {worker_of(a.rows, a.workers, begin), worker_of(a.rows, a.workers, end - 1)};
}

template <typename T>
__device__ __forceinline__ void store_as(void* p, int dtype, uint64_t at, T v)
{
    if (dtype == ZCCL_BF16)
        static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[at] = v;
}

// Adds the partial sums of 4 kLanes columns up: blockIdx.y = 0, 1 a weight's, 2 + i those
// of gate row i.  kLanes lanes hold a row's columns, so that a thread has few rows, all
// of them on their way at once; fewer where there are few columns, for more CTAs.
constexpr uint32_t kJoinThreads = 1024;

template <int kLanes>
__global__ void __launch_bounds__(kJoinThreads) norm_join_kernel(NormArgs a, int weight_dtype)
{
    constexpr uint32_t kRows = kJoinThreads / kLanes, kCols = 4 * kLanes, kWarps = kJoinThreads / 32;
    __shared__ float red[kWarps][kCols + 1];
    pdl_wait();
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, job = blockIdx.y;
    const uint32_t col = blockIdx.x * kCols + lane % kLanes * 4, first = threadIdx.x / kLanes;
    float4 sum = make_float4(0, 0, 0, 0);
    const auto add = [&](const float* p) {
        const float4 v = *reinterpret_cast<const float4*>(p + col);
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    };
    void* out = a.grad_gate;
    int dtype = a.gate.dtype;
    uint64_t at = 0;
    if (job < 2) {
        out = job == 0 ? a.grad_weight : a.grad_post_weight;
        dtype = weight_dtype;
        if (out == nullptr) return;
        if (col < pitch)
#pragma unroll 8
            for (uint32_t g = first; g < a.groups; g += kRows) add(a.sums + ((uint64_t)g * kWeightSlots + job) * pitch);
    } else {
        const Sharers s = sharers(a, job - 2);
        if (s.from == s.to) return;  // its worker's own
        if (col < pitch)
#pragma unroll 8
            for (uint32_t w = s.from + first; w <= s.to; w += kRows)
                add(a.parts + ((uint64_t)w * kGateSlots + (w == s.from ? kSlotBehind : kSlotBefore)) * pitch);
        at = (uint64_t)(job - 2) * a.hidden;
    }
#pragma unroll
    for (int o = 16; o >= kLanes; o /= 2) {
        sum.x += __shfl_xor_sync(0xFFFFFFFFu, sum.x, o);
        sum.y += __shfl_xor_sync(0xFFFFFFFFu, sum.y, o);
        sum.z += __shfl_xor_sync(0xFFFFFFFFu, sum.z, o);
        sum.w += __shfl_xor_sync(0xFFFFFFFFu, sum.w, o);
    }
    if (lane < kLanes) {
        float* p = &red[warp][lane * 4];
        p[0] = sum.x, p[1] = sum.y, p[2] = sum.z, p[3] = sum.w;
    }
    __syncthreads();
    // a warp a column
    if (warp >= kCols) return;
    float v = red[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const uint32_t c = blockIdx.x * kCols + warp;
    if (lane == 0 && c < a.hidden) store_as(out, dtype, at + c, v);
}

// With more gate rows than workers a gate row has parts of two or three workers: a thread
// a column of the one that goes on behind worker blockIdx.y's rows.
__global__ void __launch_bounds__(256) norm_join_gates_kernel(NormArgs a)
{
    pdl_wait();
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const uint32_t col = blockIdx.x * 256 + threadIdx.x, w = blockIdx.y;
    const uint32_t gate_row = (first_row(a.rows, a.workers, w + 1) - 1) / a.gate_span;
    const Sharers s = sharers(a, gate_row);
    if (s.from != w || s.to == w || col >= a.hidden) return;
    float sum = a.parts[((uint64_t)w * kGateSlots + kSlotBehind) * pitch + col];
    for (uint32_t i = w + 1; i <= s.to; ++i) sum += a.parts[((uint64_t)i * kGateSlots + kSlotBefore) * pitch + col];
    store_as(a.grad_gate, a.gate.dtype, (uint64_t)gate_row * a.hidden + col, sum);
}

template <typename... Args>
cudaError_t launch_2d(void (*kernel)(Args...), dim3 grid, uint32_t threads, cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What is to be added up: weights' sums, gate rows' parts.
bool joins_weights(const NormArgs& a) { return a.grad_weight != nullptr || a.grad_post_weight != nullptr; }
bool joins_gates(const NormArgs& a) { return a.grad_gate != nullptr && a.gate_span > 1 && a.workers > 1; }

cudaError_t launch_join(const NormArgs& a, int weight_dtype, cudaStream_t stream)
{
    const uint32_t gate_rows = (a.rows - 1) / a.gate_span + 1;
    const bool by_row = joins_gates(a) && gate_rows < a.workers;
    if (joins_gates(a) && !by_row) {
        const cudaError_t e = launch_2d(norm_join_gates_kernel, dim3((a.hidden + 255) / 256, a.workers - 1), 256, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (!joins_weights(a) && !by_row) return cudaSuccess;
    // 32 columns a CTA, fewer where that makes less than 128 of them
    const uint32_t jobs = by_row ? 2 + gate_rows : 2;
    const uint32_t lanes = a.hidden * jobs >= 128 * 32 ? 8 : a.hidden * jobs >= 128 * 16 ? 4 : 2;
    return launch_2d(lanes == 8 ? norm_join_kernel<8> : lanes == 4 ? norm_join_kernel<4> : norm_join_kernel<2>,
                     dim3((a.hidden + 4 * lanes - 1) / (4 * lanes), jobs), kJoinThreads, stream, a, weight_dtype);
}

}  // namespace

zccl_status_t launch_norm_backward(NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec, cudaStream_t stream)
{
    const Shape s = norm_shape(a.hidden, a.rows, size_of(x_dtype) + size_of(dtype), vec, true);
    a.workers = s.workers;
    a.groups = s.grid / s.ctas;
    a.parts = a.sums + (uint64_t)a.groups * kWeightSlots * ((a.hidden + 7) / 8 * 8);
    const bool post = a.post, drop = a.drop.below > 0 && a.grad_y != nullptr;
    uint32_t warp_bytes = 0;
    const NormKernel kernel =
        x_dtype == ZCCL_BF16
            ? (dtype == ZCCL_BF16 ? norm_backward_kernel_for<__nv_bfloat16, __nv_bfloat16>(s, vec, post, drop, &warp_bytes)
                                  : norm_backward_kernel_for<__nv_bfloat16, float>(s, vec, post, drop, &warp_bytes))
            : (dtype == ZCCL_BF16 ? norm_backward_kernel_for<float, __nv_bfloat16>(s, vec, post, drop, &warp_bytes)
                                  : norm_backward_kernel_for<float, float>(s, vec, post, drop, &warp_bytes));
    const uint32_t threads = s.warps * 32;
    const size_t smem = s.team == kLong ? 0 : s.warps * warp_bytes + kTeamBytes;
    a.joined = joins_weights(a) || joins_gates(a);
    cudaError_t e = launch_teams(kernel, s, threads, smem, stream, a);
    if (e == cudaSuccess && a.joined) e = launch_join(a, weight_dtype, stream);
    return launched(e);
}

}  // namespace zccl
