// zccl_norm.h -- arguments of the norm kernels, and how a backward pass's rows are
// shared out.
#pragma once

#include "zccl_rows.cuh"

namespace zccl {

constexpr uint64_t kMaxNormHidden = 65536;

struct NormArgs {
    const void* x;       // forward: the residual; backward: the stored r (with grad_h)
    const void* y;       // nullptr: no join (forward), not read (backward)
    uint64_t x_stride, y_stride;
    Vector weight, post_weight, gate;
    uint64_t gate_stride, gate_span;
    uint64_t rows;
    uint32_t hidden;
    int post;
    float inv_hidden, eps;
    float factor;        // scale, times the dropout's gain
    DropArgs drop;
    void* r;             // forward
    void* h;
    // backward
    const void* grad_r;
    const void* grad_h;
    uint64_t grad_r_stride, grad_h_stride;
    void* grad_x;
    void* grad_y;
    void* grad_weight;
    void* grad_post_weight;
    void* grad_gate;
    float* sums;         // workspace: [workers][kSlots][hidden]
    uint32_t workers;
};

// A backward pass's rows are shared out over workers, each a run of neighbouring
// rows.  A worker keeps its sums of the weights' gradients over its rows, and of
// the gate's over the rows of a gate row.  Gate rows that lie within a worker's
// rows it finishes itself; of the first and the last one it has only a part, maybe.
enum { kSlotWeight = 0, kSlotPost = 1, kSlotGateFirst = 2, kSlotGateLast = 3, kSlots = 4 };

// The first row of worker w.
__host__ __device__ inline uint64_t first_row(uint64_t rows, uint32_t workers, uint32_t w)
{
    const uint64_t base = rows / workers, more = rows - base * workers;
    return base * w + (w < more ? w : more);
}
// The worker of a row.
__host__ __device__ inline uint32_t worker_of(uint64_t rows, uint32_t workers, uint64_t row)
{
    const uint64_t base = rows / workers, more = rows - base * workers, large = more * (base + 1);
    return (uint32_t)(row < large ? row / (base + 1) : more + (row - large) / base);
}

// The most workers that a workspace has room for: two to four a SM, fewer for rows so
// long that their sums would take more than 100 MB.
constexpr uint32_t kMaxWorkers = 608;
inline uint32_t norm_workers(uint64_t hidden, uint64_t rows)
{
    uint64_t n = kMaxWorkers * 8192ull / hidden;
    n = n < kMaxWorkers ? n : kMaxWorkers;
    n = n < rows ? n : rows;
    return (uint32_t)(n > 0 ? n : 1);
}

// Sums N values over a CTA of `warps` warps, the same way in every thread; `red` holds
// 2 * 32 * N floats, whose halves take turns by `turn`.
template <int N>
__device__ __forceinline__ void cta_sum(float (&s)[N], float* red, uint32_t& turn)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
    if (warps == 1) return;
    float* at = red + turn * 32 * N;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) at[i * 32 + warp] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = lane < warps ? at[i * 32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
    }
}

// What the block's output is multiplied by before it joins (scale, gate, the
// dropout's gain), and which of the lane's eight values stay.
template <bool kVec>
__device__ __forceinline__ uint32_t join_factors(float (&k)[8], const NormArgs& a, uint64_t offset, uint64_t row,
                                                 uint32_t tile)
{
    load_vector<kVec>(k, a.gate, a.gate.p != nullptr ? row / a.gate_span * a.gate_stride : 0, tile, a.hidden);
#pragma unroll
    for (int j = 0; j < 8; ++j) k[j] *= a.factor;
    return a.drop.below > 0 ? kept_piece<kVec>(a.drop, offset, (uint32_t)row, tile) : 0xFFu;
}

zccl_status_t launch_norm(const NormArgs& a, int x_dtype, int dtype, bool vec, cudaStream_t stream);
zccl_status_t launch_norm_backward(const NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec,
                                   cudaStream_t stream);

}  // namespace zccl
