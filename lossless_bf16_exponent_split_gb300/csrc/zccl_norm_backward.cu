// zccl_norm_backward.cu -- gradients of the join of a block's output with the
// residual and of the norms around it.
//
// With a row's rho = rsqrt(mean r^2 + eps), eta = rsqrt(mean y^2 + eps), k = the
// join's factor (0 where dropped), w and p the two weights:
//   d    = dr + rho (dh w - r c),     c  = rho^2 mean(dh w r)      the gradient of x
//   dy   = eta (k d p - y c'),        c' = eta^2 mean(k d p y)     (k d without post)
//   dw  += dh r rho, dp += k d y eta, dgate += (k / gate) d N(y)
// c' needs d, but its sum is that of three others, mean(k d p y) = mean(k p y dr) +
// rho (mean(k p y dh w) - c mean(k p y r)): all six sums of a row are taken at once.
#include "zccl_norm.h"

namespace zccl {

namespace {

constexpr int kSums = 6;

// The sums of a piece: r^2, dh w r, y^2, and k p y times dr, dh w and r.
__device__ __forceinline__ void add_sums(float (&s)[kSums], const float (&r)[8], const float (&hw)[8], const float (&up)[8],
                                         const float (&y)[8], const float (&kp)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float q = kp[j] * y[j];
        s[0] = fmaf(r[j], r[j], s[0]);
        s[1] = fmaf(hw[j], r[j], s[1]);
        s[2] = fmaf(y[j], y[j], s[2]);
        s[3] = fmaf(q, up[j], s[3]);
        s[4] = fmaf(q, hw[j], s[4]);
        s[5] = fmaf(q, r[j], s[5]);
    }
}

struct RowFactors {
    float rho, c, eta, cy;
};
__device__ __forceinline__ RowFactors row_factors(const NormArgs& a, const float (&s)[kSums])
{
    RowFactors f{0.0f, 0.0f, 1.0f, 0.0f};
    if (a.grad_h != nullptr) {
        f.rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
        f.c = s[1] * a.inv_hidden * f.rho * f.rho;
    }
    if (a.post) {
        f.eta = rsqrtf(s[2] * a.inv_hidden + a.eps);
        f.cy = (s[3] + f.rho * (s[4] - f.c * s[5])) * a.inv_hidden * f.eta * f.eta;
    }
    return f;
}

template <typename T, bool kVec>
__device__ __forceinline__ void load_or_zero(float (&v)[8], const void* p, uint64_t first, uint32_t tile, uint32_t hidden)
{
    if (p != nullptr) {
        load8<T, kVec>(v, static_cast<const T*>(p) + first, tile, hidden);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
}

template <bool kVec>
__device__ __forceinline__ void add_to(float* p, float (&v)[8], bool first, uint32_t tile, uint32_t hidden)
{
    if (!first) {
        float o[8];
        load8<float, kVec>(o, p, tile, hidden);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += o[j];
    }
    store8<float, kVec>(p, v, tile, hidden);
}

// Writes a gate row's gradient, of its own type.
template <bool kVec>
__device__ __forceinline__ void store_gate(const NormArgs& a, uint64_t gate_row, float (&v)[8], uint32_t tile)
{
    if (a.gate.dtype == ZCCL_BF16)
        store8<__nv_bfloat16, kVec>(static_cast<__nv_bfloat16*>(a.grad_gate) + gate_row * a.hidden, v, tile, a.hidden);
    else
        store8<float, kVec>(static_cast<float*>(a.grad_gate) + gate_row * a.hidden, v, tile, a.hidden);
}

// A CTA a worker; its rows are read once for the sums and once for the gradients, and
// the sums over rows stay in the workspace: any size.
template <typename Tx, typename Ty, bool kVec>
__global__ void norm_backward_long_kernel(NormArgs a)
{
    __shared__ float red[2 * 32 * kSums];
    uint32_t turn = 0;
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t warp = threadIdx.x >> 5, step = blockDim.x / 32 * kTile, wk = blockIdx.x;
    const uint64_t lo = first_row(a.rows, a.workers, wk), hi = first_row(a.rows, a.workers, wk + 1);
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    float* sums = a.sums + wk * kSlots * pitch;
    const bool join = a.grad_y != nullptr;
    for (uint64_t t = lo; t < hi; ++t) {
        const uint64_t gate_row = t / a.gate_span;
        float s[kSums] = {};
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            float r[8], hw[8], up[8], y[8], kp[8], w[8];
            load_or_zero<Tx, kVec>(r, a.x, t * a.x_stride, tile, a.hidden);
            load_or_zero<Ty, kVec>(hw, a.grad_h, t * a.grad_h_stride, tile, a.hidden);
            load_or_zero<Tx, kVec>(up, a.grad_r, t * a.grad_r_stride, tile, a.hidden);
            load_or_zero<Ty, kVec>(y, a.y, t * a.y_stride, tile, a.hidden);
            load_vector<kVec>(w, a.weight, 0, tile, a.hidden);
#pragma unroll
            for (int j = 0; j < 8; ++j) hw[j] *= w[j];
            const uint32_t kept = join_factors<kVec>(kp, a, offset, t, tile);
            load_vector<kVec>(w, a.post_weight, 0, tile, a.hidden);
#pragma unroll
            for (int j = 0; j < 8; ++j) kp[j] = (kept >> j) & 1u ? kp[j] * w[j] : 0.0f;
            add_sums(s, r, hw, up, y, kp);
        }
        cta_sum<kSums>(s, red, turn);
        const RowFactors f = row_factors(a, s);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            float r[8], dh[8], d[8], y[8], k[8], w[8], v[8];
            load_or_zero<Tx, kVec>(r, a.x, t * a.x_stride, tile, a.hidden);
            load_or_zero<Ty, kVec>(dh, a.grad_h, t * a.grad_h_stride, tile, a.hidden);
            load_or_zero<Tx, kVec>(d, a.grad_r, t * a.grad_r_stride, tile, a.hidden);
            load_vector<kVec>(w, a.weight, 0, tile, a.hidden);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] += f.rho * (dh[j] * w[j] - r[j] * f.c);
                v[j] = d[j];
            }
            if (a.grad_x != nullptr) store8<Tx, kVec>(static_cast<Tx*>(a.grad_x) + t * a.hidden, v, tile, a.hidden);
            if (a.grad_weight != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = dh[j] * (r[j] * f.rho);
                add_to<kVec>(sums + kSlotWeight * pitch, v, t == lo, tile, a.hidden);
            }
            if (!join) continue;
            load_or_zero<Ty, kVec>(y, a.y, t * a.y_stride, tile, a.hidden);
            const uint32_t kept = join_factors<kVec>(k, a, offset, t, tile);
            load_vector<kVec>(w, a.post_weight, 0, tile, a.hidden);
            if (a.grad_gate != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (kept >> j) & 1u ? a.factor * d[j] * (y[j] * f.eta * w[j]) : 0.0f;
                if (a.gate_span == 1) {
                    store_gate<kVec>(a, gate_row, v, tile);
                } else {
                    // of the worker's first gate row, or of a later one
                    const bool first = gate_row == lo / a.gate_span;
                    const uint64_t end = (gate_row + 1) * a.gate_span;
                    add_to<kVec>(sums + (first ? kSlotGateFirst : kSlotGateLast) * pitch, v,
                                 t == lo || t == gate_row * a.gate_span, tile, a.hidden);
                    if (!first && t + 1 == end && t + 1 < hi) store_gate<kVec>(a, gate_row, v, tile);
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = (kept >> j) & 1u ? k[j] * d[j] : 0.0f;
            if (a.grad_post_weight != nullptr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = k[j] * (y[j] * f.eta);
                add_to<kVec>(sums + kSlotPost * pitch, v, t == lo, tile, a.hidden);
            }
            if (a.post)
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] = f.eta * (k[j] * w[j] - y[j] * f.cy);
            store8<Ty, kVec>(static_cast<Ty*>(a.grad_y) + t * a.hidden, k, tile, a.hidden);
        }
    }
}

// Adds the workers' sums up: blockIdx.y = 0, 1 a weight's, 2 + 2 w + l those of the
// first (l = 0) or last (l = 1) gate row of worker w, where w is the first of the workers
// that share it.
constexpr int kJoinRows = 32;  // partial sums of a column that are added side by side

__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(NormArgs a, int weight_dtype)
{
    __shared__ float red[kJoinRows][33];
    pdl_wait();
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const uint32_t lane = threadIdx.x & 31, sub = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    uint32_t begin = 0, end = a.workers, job = blockIdx.y;
    uint64_t gate_row = 0;
    void* out = nullptr;
    int dtype = weight_dtype;
    if (job < 2) {
        out = job == 0 ? a.grad_weight : a.grad_post_weight;
        if (out == nullptr) return;
    } else {
        const uint32_t w = (job - 2) / 2, last = (job - 2) % 2;
        const uint64_t lo = first_row(a.rows, a.workers, w), hi = first_row(a.rows, a.workers, w + 1);
        const uint64_t g_lo = lo / a.gate_span, g_hi = (hi - 1) / a.gate_span;
        gate_row = last ? g_hi : g_lo;
        if (last && g_hi == g_lo) return;                            // one gate row: its first
        if (!last && gate_row * a.gate_span < lo) return;            // begun by an earlier worker
        uint64_t stop = (gate_row + 1) * a.gate_span;
        stop = stop < a.rows ? stop : a.rows;
        begin = w;
        end = worker_of(a.rows, a.workers, stop - 1) + 1;
        out = a.grad_gate;
        dtype = a.gate.dtype;
    }
    float sum = 0.0f;
    if (col < a.hidden)
        for (uint32_t w = begin + sub; w < end; w += kJoinRows) {
            uint32_t slot = job;
            if (job >= 2) slot = first_row(a.rows, a.workers, w) / a.gate_span == gate_row ? kSlotGateFirst : kSlotGateLast;
            sum += a.sums[((uint64_t)w * kSlots + slot) * pitch + col];
        }
    red[sub][lane] = sum;
    __syncthreads();
    if (sub != 0 || col >= a.hidden) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) sum += red[i][lane];
    const uint64_t at = (job >= 2 ? gate_row * a.hidden : 0) + col;
    if (dtype == ZCCL_BF16)
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(sum);
    else
        static_cast<float*>(out)[at] = sum;
}

cudaError_t launch_join(const NormArgs& a, int weight_dtype, cudaStream_t stream)
{
    const bool gate = a.grad_gate != nullptr && a.gate_span > 1;
    if (a.grad_weight == nullptr && a.grad_post_weight == nullptr && !gate) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.hidden + 31) / 32, gate ? 2 + 2 * a.workers : 2);
    cfg.blockDim = dim3(32 * kJoinRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_join_kernel, a, weight_dtype);
}

template <typename Tx, typename Ty>
cudaError_t launch_backward_as(const NormArgs& a, bool vec, cudaStream_t stream)
{
    const uint32_t tiles = (a.hidden + kTile - 1) / kTile, threads = 32 * (tiles < 16 ? tiles : 16);
    return launch_dependent(vec ? norm_backward_long_kernel<Tx, Ty, true> : norm_backward_long_kernel<Tx, Ty, false>,
                            a.workers, threads, 0, stream, a);
}

}  // namespace

zccl_status_t launch_norm_backward(const NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec,
                                   cudaStream_t stream)
{
    cudaError_t e;
    if (x_dtype == ZCCL_BF16)
        e = dtype == ZCCL_BF16 ? launch_backward_as<__nv_bfloat16, __nv_bfloat16>(a, vec, stream)
                               : launch_backward_as<__nv_bfloat16, float>(a, vec, stream);
    else
        e = dtype == ZCCL_BF16 ? launch_backward_as<float, __nv_bfloat16>(a, vec, stream)
                               : launch_backward_as<float, float>(a, vec, stream);
    if (e == cudaSuccess) e = launch_join(a, weight_dtype, stream);
    return launched(e);
}

}  // namespace zccl
