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
    float* sums = a.sums + wk * kWeightSlots * pitch;
    float* parts = a.parts + wk * kGateSlots * pitch;
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
                const uint64_t begin = gate_row * a.gate_span, end = begin + a.gate_span;
                if (a.gate_span > 1)
                    add_to<kVec>(parts + (begin < lo ? kSlotBefore : kSlotBehind) * pitch, v, t == lo || t == begin, tile, a.hidden);
                if (begin >= lo && (t + 1 == end || t + 1 == a.rows)) store_gate<kVec>(a, gate_row, v, tile);
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

// A team a worker.  Weights and the join's factors of the lane's columns are kept in
// shared memory, the sums over rows in registers.  While a gate stays the same the sums
// of p's and of the gate's gradient are the same up to a factor of each column,
//   e = sum of (kept) d y eta:   dp += scale gate e,   dgate = scale p e
// so one sum serves both, and is taken out when the gate changes.
template <typename Tx, typename Ty, bool kVec, int kTeam>
__global__ void __launch_bounds__(kTeam == kWarpTeam ? kWarpsPerCta * 32 : kTeamWarps * 32, kTeam == kWarpTeam ? 2 : 1) norm_backward_kernel(NormArgs a)
{
    extern __shared__ float4 smem[];
    uint32_t turn = 0;
    const uint32_t warp = threadIdx.x >> 5, threads = blockDim.x;
    // eight values of each thread's own, by name
    enum { kW, kP, kK, kDp, kOwn };
    const auto put = [&](int name, const float (&v)[8]) {
        smem[(2 * name) * threads + threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
        smem[(2 * name + 1) * threads + threadIdx.x] = make_float4(v[4], v[5], v[6], v[7]);
    };
    const auto get = [&](int name, float (&v)[8]) {
        const float4 x = smem[(2 * name) * threads + threadIdx.x], y = smem[(2 * name + 1) * threads + threadIdx.x];
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    };
    float* const red = reinterpret_cast<float*>(smem + 2 * kOwn * threads);
    uint32_t worker = blockIdx.x, tile = warp * kTile;
    if (kTeam == kWarpTeam) worker = blockIdx.x * kWarpsPerCta + warp, tile = 0;
    if (kTeam == kClusterTeam) {
        uint32_t ctas;
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
        worker = blockIdx.x / ctas;
        tile = (cluster_rank() * (threads / 32) + warp) * kTile;
    }
    pdl_wait();
    if (kTeam == kClusterTeam) cluster_sync();  // the others' shared memory is there
    const uint64_t offset = drop_offset(a.drop);
    const uint64_t lo = worker < a.workers ? first_row(a.rows, a.workers, worker) : 0;
    const uint64_t hi = worker < a.workers ? first_row(a.rows, a.workers, worker + 1) : 0;
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const bool join = a.grad_y != nullptr;
    float dw[8] = {}, e[8] = {};
    {
        float v[8];
        load_vector<kVec>(v, a.weight, 0, tile, a.hidden);
        put(kW, v);
        load_vector<kVec>(v, a.post_weight, 0, tile, a.hidden);
        put(kP, v);
        put(kDp, dw);
    }
    Piece<Tx, kVec> pr, pu;
    Piece<Ty, kVec> ph, py;
    const auto load = [&](uint64_t t) {
        if (a.x != nullptr) pr.load(static_cast<const Tx*>(a.x) + t * a.x_stride, tile, a.hidden);
        if (a.grad_h != nullptr) ph.load(static_cast<const Ty*>(a.grad_h) + t * a.grad_h_stride, tile, a.hidden);
        if (a.grad_r != nullptr) pu.load(static_cast<const Tx*>(a.grad_r) + t * a.grad_r_stride, tile, a.hidden);
        if (a.y != nullptr) py.load(static_cast<const Ty*>(a.y) + t * a.y_stride, tile, a.hidden);
    };
    // what is not there stays zero
    pr.zero(), pu.zero(), ph.zero(), py.zero();
    if (lo < hi) load(lo);
    uint64_t gate_row = lo / a.gate_span, gate_end = lo;  // where the gate changes
    const auto take_out = [&](uint64_t t) {
        float v[8], o[8];
        get(kK, v);
        get(kDp, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(v[j], e[j], o[j]);
        put(kDp, o);
        if (a.grad_gate == nullptr) return;
        get(kP, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= a.factor * e[j];
        const uint64_t begin = gate_row * a.gate_span;
        if (begin >= lo && (t == begin + a.gate_span || t == a.rows))
            store_gate<kVec>(a, gate_row, v, tile);
        else
            store8<float, kVec>(a.parts + (worker * kGateSlots + (begin < lo ? kSlotBefore : kSlotBehind)) * pitch, v, tile, a.hidden);
    };
    for (uint64_t t = lo; t < hi; ++t) {
        float r[8], dh[8], d[8], y[8];
        pr.get(r), ph.get(dh), pu.get(d), py.get(y);
        if (t + 1 < hi) load(t + 1);
        if (join && t == gate_end) {
            if (t > lo) {
                take_out(t);
                ++gate_row;
            }
            gate_end = a.gate.p != nullptr ? (gate_row + 1) * a.gate_span : a.rows;
            float k[8];
            load_vector<kVec>(k, a.gate, gate_row * a.gate_stride, tile, a.hidden);
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] *= a.factor, e[j] = 0.0f;
            put(kK, k);
        }
        const uint32_t kept = a.drop.below > 0 && join ? kept_piece<kVec>(a.drop, offset, (uint32_t)t, tile) : 0xFFu;
        float s[kSums] = {};
        if (a.grad_h != nullptr) {
            float w[8];
            get(kW, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                s[0] = fmaf(r[j], r[j], s[0]);
                s[1] = fmaf(dh[j] * w[j], r[j], s[1]);
            }
        }
        if (a.post) {
            float w[8], k[8], p[8];
            get(kW, w), get(kK, k), get(kP, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float q = (kept >> j) & 1u ? k[j] * p[j] * y[j] : 0.0f;
                s[2] = fmaf(y[j], y[j], s[2]);
                s[3] = fmaf(q, d[j], s[3]);
                s[4] = fmaf(q, dh[j] * w[j], s[4]);
                s[5] = fmaf(q, r[j], s[5]);
            }
        }
        RowFactors f{0.0f, 0.0f, 1.0f, 0.0f};
        if (a.grad_h != nullptr || a.post) {
            team_sum<kSums, kTeam>(s, red, turn);
            f = row_factors(a, s);
        }
        float v[8];
        if (a.grad_h != nullptr) {
            float w[8];
            get(kW, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] += f.rho * (dh[j] * w[j] - r[j] * f.c);
                dw[j] = fmaf(dh[j], r[j] * f.rho, dw[j]);
            }
        }
        if (a.grad_x != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = d[j];
            store8<Tx, kVec>(static_cast<Tx*>(a.grad_x) + t * a.hidden, v, tile, a.hidden);
        }
        if (!join) continue;
        float k[8];
        get(kK, k);
        if (a.y != nullptr) {
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] += (kept >> j) & 1u ? d[j] * (y[j] * f.eta) : 0.0f;
        }
        if (a.post) {
            float p[8];
            get(kP, p);
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = f.eta * (((kept >> j) & 1u ? k[j] * d[j] * p[j] : 0.0f) - y[j] * f.cy);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) k[j] = (kept >> j) & 1u ? k[j] * d[j] : 0.0f;
        }
        store8<Ty, kVec>(static_cast<Ty*>(a.grad_y) + t * a.hidden, k, tile, a.hidden);
    }
    if (join && lo < hi && a.y != nullptr) take_out(hi);
    pdl_launch_dependents();
    // the weights' sums: of a CTA's warps where each is a team
    float dp[8];
    get(kDp, dp);
    if (kTeam == kWarpTeam) {
        put(kW, dw);
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float sum[8] = {};
            for (uint32_t i = 0; i < kWarpsPerCta; ++i) {
                const int name = n == 0 ? kW : kDp;
                const float4 x = smem[(2 * name) * threads + threadIdx.x + 32 * i];
                const float4 z = smem[(2 * name + 1) * threads + threadIdx.x + 32 * i];
                sum[0] += x.x, sum[1] += x.y, sum[2] += x.z, sum[3] += x.w, sum[4] += z.x, sum[5] += z.y, sum[6] += z.z, sum[7] += z.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) (n == 0 ? dw : dp)[j] = sum[j];
        }
    }
    const uint64_t group = kTeam == kWarpTeam ? blockIdx.x : worker;
    if (a.grad_weight != nullptr) store8<float, kVec>(a.sums + (group * kWeightSlots + kSlotWeight) * pitch, dw, tile, a.hidden);
    if (a.grad_post_weight != nullptr)
        store8<float, kVec>(a.sums + (group * kWeightSlots + kSlotPost) * pitch, dp, tile, a.hidden);
}

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

using NormKernel = void (*)(NormArgs);

template <typename Tx, typename Ty, bool kVec>
NormKernel backward_for(Team team)
{
    return team == kWarpTeam  ? norm_backward_kernel<Tx, Ty, kVec, kWarpTeam>
           : team == kCtaTeam ? norm_backward_kernel<Tx, Ty, kVec, kCtaTeam>
           : team == kLong    ? norm_backward_long_kernel<Tx, Ty, kVec>
                              : norm_backward_kernel<Tx, Ty, kVec, kClusterTeam>;
}
template <typename Tx>
NormKernel backward_for(int dtype, bool vec, Team team)
{
    if (dtype == ZCCL_BF16) return vec ? backward_for<Tx, __nv_bfloat16, true>(team) : backward_for<Tx, __nv_bfloat16, false>(team);
    return vec ? backward_for<Tx, float, true>(team) : backward_for<Tx, float, false>(team);
}

constexpr uint32_t kSmWarps = 16;  // of a backward pass: 128 registers a thread

}  // namespace

// Of each group of teams the weights' sums, of each worker its parts of gate rows.
uint64_t norm_backward_bytes(uint64_t hidden, uint64_t rows)
{
    const Shape s = norm_shape(hidden, rows, kSmWarps);
    const uint64_t groups = s.grid / s.ctas, pitch = (hidden + 7) / 8 * 8;
    return (groups * kWeightSlots + (uint64_t)s.workers * kGateSlots) * pitch * sizeof(float);
}

zccl_status_t launch_norm_backward(NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec, cudaStream_t stream)
{
    const Shape s = norm_shape(a.hidden, a.rows, kSmWarps);
    a.workers = s.workers;
    a.groups = s.grid / s.ctas;
    a.parts = a.sums + (uint64_t)a.groups * kWeightSlots * ((a.hidden + 7) / 8 * 8);
    const NormKernel kernel = x_dtype == ZCCL_BF16 ? backward_for<__nv_bfloat16>(dtype, vec, s.team)
                                                   : backward_for<float>(dtype, vec, s.team);
    const uint32_t threads = s.warps * 32;
    const size_t smem = s.team == kLong ? 0 : threads * 4 * 8 * sizeof(float) + kTeamRed * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (smem > 48 << 10) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = s.team == kClusterTeam ? launch_clusters(kernel, s.grid, threads, smem, s.ctas, stream, a)
                                   : launch_dependent(kernel, s.grid, threads, smem, stream, a);
    if (e == cudaSuccess) e = launch_join(a, weight_dtype, stream);
    return launched(e);
}

}  // namespace zccl
