// zccl_norm.cu -- the join of a block's output with the residual and the norm of
// the next block's input, and the host side of both directions.
#include <cmath>

#include "zccl_norm.h"

namespace zccl {

namespace {

// A CTA a row, read once for each of its sums: any size.
template <typename Tx, typename Ty, bool kVec>
__global__ void norm_long_kernel(NormArgs a)
{
    __shared__ float red[2 * 32];
    uint32_t turn = 0;
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t warp = threadIdx.x >> 5, step = blockDim.x / 32 * kTile;
    for (uint64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const Tx* x = static_cast<const Tx*>(a.x) + t * a.x_stride;
        const Ty* y = static_cast<const Ty*>(a.y) + t * a.y_stride;
        Tx* r = static_cast<Tx*>(a.r) + t * a.hidden;
        float eta[1] = {0.0f}, rho[1] = {0.0f};
        if (a.y != nullptr && a.post) {
            for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
                float v[8];
                load8<Ty, kVec>(v, y, tile, a.hidden);
#pragma unroll
                for (int j = 0; j < 8; ++j) eta[0] = fmaf(v[j], v[j], eta[0]);
            }
            cta_sum<1>(eta, red, turn);
            eta[0] = rsqrtf(eta[0] * a.inv_hidden + a.eps);
        }
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            float v[8];
            load8<Tx, kVec>(v, x, tile, a.hidden);
            if (a.y != nullptr) {
                float b[8], k[8];
                load8<Ty, kVec>(b, y, tile, a.hidden);
                const uint32_t kept = join_factors<kVec>(k, a, offset, t, tile);
                if (a.post) {
                    float w[8];
                    load_vector<kVec>(w, a.post_weight, 0, tile, a.hidden);
#pragma unroll
                    for (int j = 0; j < 8; ++j) b[j] = b[j] * eta[0] * w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = (kept >> j) & 1u ? fmaf(k[j], b[j], v[j]) : v[j];
                store8<Tx, kVec>(r, v, tile, a.hidden);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) rho[0] = fmaf(v[j], v[j], rho[0]);
        }
        if (a.h == nullptr) continue;
        cta_sum<1>(rho, red, turn);
        rho[0] = rsqrtf(rho[0] * a.inv_hidden + a.eps);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            float v[8], w[8];
            load8<Tx, kVec>(v, a.y != nullptr ? r : x, tile, a.hidden);
            load_vector<kVec>(w, a.weight, 0, tile, a.hidden);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * rho[0] * w[j];
            store8<Ty, kVec>(static_cast<Ty*>(a.h) + t * a.hidden, v, tile, a.hidden);
        }
    }
}

// A team a worker: a row is read once and stays in registers, with the next one on its
// way; weights and the gate stay there too.
template <typename Tx, typename Ty, bool kVec, int kTeam>
__global__ void __launch_bounds__(kTeam == kWarpTeam ? kWarpsPerCta * 32 : kTeamWarps * 32) norm_kernel(NormArgs a)
{
    __shared__ float red[kTeam == kWarpTeam ? 1 : kTeamRed];
    uint32_t turn = 0;
    const uint32_t warp = threadIdx.x >> 5;
    uint32_t worker = blockIdx.x, tile = warp * kTile;
    if (kTeam == kWarpTeam) worker = blockIdx.x * kWarpsPerCta + warp, tile = 0;
    if (kTeam == kClusterTeam) {
        uint32_t ctas;
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
        worker = blockIdx.x / ctas;
        tile = (cluster_rank() * (blockDim.x / 32) + warp) * kTile;
    }
    pdl_wait();
    if (kTeam == kClusterTeam) cluster_sync();  // the others' shared memory is there
    if (kTeam == kWarpTeam && worker >= a.workers) return;
    const uint64_t offset = drop_offset(a.drop);
    const uint64_t lo = first_row(a.rows, a.workers, worker), hi = first_row(a.rows, a.workers, worker + 1);
    const bool join = a.y != nullptr;
    Piece<Tx, kVec> px;
    Piece<Ty, kVec> py;
    const auto load = [&](uint64_t t) {
        px.load(static_cast<const Tx*>(a.x) + t * a.x_stride, tile, a.hidden);
        if (join) py.load(static_cast<const Ty*>(a.y) + t * a.y_stride, tile, a.hidden);
    };
    py.zero();
    load(lo);
    float w[8], k[8];
    load_vector<kVec>(w, a.weight, 0, tile, a.hidden);
    uint64_t gate_end = lo;  // where the gate changes
    for (uint64_t t = lo; t < hi; ++t) {
        float x[8], y[8];
        px.get(x), py.get(y);
        if (t + 1 < hi) load(t + 1);
        float s[1] = {0.0f};
        if (join) {
            if (t == gate_end) {
                // the join's factor of each column, with the weight of the norm after the block
                const uint64_t row = t / a.gate_span;
                float p[8];
                load_vector<kVec>(k, a.gate, a.gate.p != nullptr ? row * a.gate_stride : 0, tile, a.hidden);
                load_vector<kVec>(p, a.post_weight, 0, tile, a.hidden);
#pragma unroll
                for (int j = 0; j < 8; ++j) k[j] = k[j] * a.factor * p[j];
                gate_end = a.gate.p != nullptr ? (row + 1) * a.gate_span : a.rows;
            }
            const uint32_t kept = a.drop.below > 0 ? kept_piece<kVec>(a.drop, offset, (uint32_t)t, tile) : 0xFFu;
            float eta = 1.0f;
            if (a.post) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] = fmaf(y[j], y[j], s[0]);
                team_sum<1, kTeam>(s, red, turn);
                eta = rsqrtf(s[0] * a.inv_hidden + a.eps);
                s[0] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = (kept >> j) & 1u ? fmaf(k[j], y[j] * eta, x[j]) : x[j];
            store8<Tx, kVec>(static_cast<Tx*>(a.r) + t * a.hidden, x, tile, a.hidden);
        }
        if (a.h == nullptr) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) s[0] = fmaf(x[j], x[j], s[0]);
        team_sum<1, kTeam>(s, red, turn);
        const float rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] * rho * w[j];
        store8<Ty, kVec>(static_cast<Ty*>(a.h) + t * a.hidden, x, tile, a.hidden);
    }
}

using NormKernel = void (*)(NormArgs);

template <typename Tx, typename Ty, bool kVec>
NormKernel norm_for(Team team)
{
    return team == kWarpTeam  ? norm_kernel<Tx, Ty, kVec, kWarpTeam>
           : team == kCtaTeam ? norm_kernel<Tx, Ty, kVec, kCtaTeam>
           : team == kLong    ? norm_long_kernel<Tx, Ty, kVec>
                              : norm_kernel<Tx, Ty, kVec, kClusterTeam>;
}
template <typename Tx>
NormKernel norm_for(int dtype, bool vec, Team team)
{
    if (dtype == ZCCL_BF16) return vec ? norm_for<Tx, __nv_bfloat16, true>(team) : norm_for<Tx, __nv_bfloat16, false>(team);
    return vec ? norm_for<Tx, float, true>(team) : norm_for<Tx, float, false>(team);
}

constexpr uint32_t kSmWarps = 16;

bool dtype_ok(int dtype) { return dtype == ZCCL_BF16 || dtype == ZCCL_F32; }
uint64_t size_of(int dtype) { return dtype == ZCCL_BF16 ? 2 : 4; }

// The configuration and what both directions share; *drop_ok false: refused.
bool norm_config(const zccl_norm_t* c, int x_dtype, int dtype, const void* d_weight, const void* d_post_weight,
                 int weight_dtype, const void* d_gate, int gate_dtype, uint64_t gate_stride, uint64_t gate_span,
                 uint64_t rows, uint64_t offset, const uint64_t* d_offset, NormArgs* a)
{
    if (c == nullptr || c->hidden == 0 || c->hidden > ZCCL_MAX_NORM_HIDDEN || !(c->eps > 0.0f) || !std::isfinite(c->eps) ||
        !std::isfinite(c->scale) || !drop_args(c->dropout, c->seed, offset, d_offset, &a->drop) || !dtype_ok(x_dtype) ||
        !dtype_ok(dtype) || !dtype_ok(weight_dtype) || !dtype_ok(gate_dtype) || rows >= (1ull << 31) ||
        gate_span == 0 || gate_stride >= kMaxElems || !is_aligned(d_weight, size_of(weight_dtype)) ||
        !is_aligned(d_post_weight, size_of(weight_dtype)) || !is_aligned(d_gate, size_of(gate_dtype)) ||
        (d_post_weight != nullptr && !c->post))
        return false;
    a->weight = {d_weight, weight_dtype};
    a->post_weight = {d_post_weight, weight_dtype};
    a->gate = {d_gate, gate_dtype};
    a->gate_stride = gate_stride;
    a->gate_span = gate_span;
    a->rows = rows;
    a->hidden = (uint32_t)c->hidden;
    a->post = c->post != 0;
    a->inv_hidden = 1.0f / (float)c->hidden;
    a->eps = c->eps;
    a->factor = c->scale * (a->drop.below > 0 ? a->drop.gain : 1.0f);
    return true;
}

// Whether rows of this type, `stride` elements apart, all begin on 16 bytes.
bool on_16(const void* p, int dtype, uint64_t stride, uint64_t rows)
{
    return is_aligned(p, 16) && (p == nullptr || rows <= 1 || stride * size_of(dtype) % 16 == 0);
}

}  // namespace

zccl_status_t launch_norm(NormArgs& a, int x_dtype, int dtype, bool vec, cudaStream_t stream)
{
    const Shape s = norm_shape(a.hidden, a.rows, kSmWarps);
    a.workers = s.workers;
    const NormKernel kernel =
        x_dtype == ZCCL_BF16 ? norm_for<__nv_bfloat16>(dtype, vec, s.team) : norm_for<float>(dtype, vec, s.team);
    return launched(s.team == kClusterTeam ? launch_clusters(kernel, s.grid, s.warps * 32, 0, s.ctas, stream, a)
                                           : launch_dependent(kernel, s.grid, s.warps * 32, 0, stream, a));
}

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_residual_norm(const zccl_norm_t* cfg, const void* d_x, int x_dtype, uint64_t x_stride,
                                 const void* d_y, int dtype, uint64_t y_stride, const void* d_weight,
                                 const void* d_post_weight, int weight_dtype, const void* d_gate, int gate_dtype,
                                 uint64_t gate_stride, uint64_t gate_span, uint64_t rows, uint64_t offset,
                                 const uint64_t* d_offset, void* d_r, void* d_h, cudaStream_t stream)
{
    NormArgs a{};
    if (!norm_config(cfg, x_dtype, dtype, d_weight, d_post_weight, weight_dtype, d_gate, gate_dtype, gate_stride, gate_span,
                     rows, offset, d_offset, &a) ||
        x_stride >= kMaxElems || y_stride >= kMaxElems)
        return ZCCL_ERR_INVALID_ARG;
    if (rows == 0) return ZCCL_OK;
    const uint64_t xs = size_of(x_dtype), ys = size_of(dtype);
    if (!good_ptr(d_x, xs) || !is_aligned(d_y, ys) || !is_aligned(d_h, ys) || (d_y == nullptr) != (d_r == nullptr) ||
        !is_aligned(d_r, xs) || (d_y == nullptr && (d_h == nullptr || d_gate != nullptr || d_post_weight != nullptr)) ||
        (d_weight != nullptr && d_h == nullptr) || (rows > 1 && d_r == d_x && x_stride != a.hidden))
        return ZCCL_ERR_INVALID_ARG;
    a.x = d_x;
    a.y = d_y;
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.r = d_r;
    a.h = d_h;
    const bool vec = a.hidden % 8 == 0 && on_16(d_x, x_dtype, x_stride, rows) && on_16(d_y, dtype, y_stride, rows) &&
                     on_16(d_r, x_dtype, 0, 1) && on_16(d_h, dtype, 0, 1) && on_16(d_weight, weight_dtype, 0, 1) &&
                     on_16(d_post_weight, weight_dtype, 0, 1) && on_16(d_gate, gate_dtype, gate_stride, rows);
    return launch_norm(a, x_dtype, dtype, vec, stream);
}

zccl_status_t zccl_residual_norm_workspace_bytes(uint64_t hidden, uint64_t rows, uint64_t* bytes)
{
    if (bytes == nullptr || hidden == 0 || hidden > ZCCL_MAX_NORM_HIDDEN || rows >= (1ull << 31)) return ZCCL_ERR_INVALID_ARG;
    *bytes = norm_backward_bytes(hidden, rows);
    return ZCCL_OK;
}

zccl_status_t zccl_residual_norm_backward(const zccl_norm_t* cfg, const void* d_grad_r, uint64_t grad_r_stride,
                                          const void* d_grad_h, uint64_t grad_h_stride, const void* d_r, int x_dtype,
                                          uint64_t r_stride, const void* d_y, int dtype, uint64_t y_stride,
                                          const void* d_weight, const void* d_post_weight, int weight_dtype,
                                          const void* d_gate, int gate_dtype, uint64_t gate_stride,
                                          uint64_t gate_span, uint64_t rows, uint64_t offset,
                                          const uint64_t* d_offset, void* d_grad_x, void* d_grad_y,
                                          void* d_grad_weight, void* d_grad_post_weight, void* d_grad_gate, void* d_ws,
                                          uint64_t ws_bytes, cudaStream_t stream)
{
    NormArgs a{};
    if (!norm_config(cfg, x_dtype, dtype, d_weight, d_post_weight, weight_dtype, d_gate, gate_dtype, gate_stride, gate_span,
                     rows, offset, d_offset, &a) ||
        grad_r_stride >= kMaxElems || grad_h_stride >= kMaxElems || r_stride >= kMaxElems || y_stride >= kMaxElems)
        return ZCCL_ERR_INVALID_ARG;
    const uint64_t xs = size_of(x_dtype), ys = size_of(dtype), ws = size_of(weight_dtype);
    const bool join = d_grad_y != nullptr;
    if (!is_aligned(d_grad_weight, ws) || !is_aligned(d_grad_post_weight, ws) || !is_aligned(d_grad_gate, size_of(gate_dtype)) ||
        (d_grad_weight != nullptr && (d_weight == nullptr)) || (d_grad_post_weight != nullptr && d_post_weight == nullptr) ||
        (d_grad_gate != nullptr && d_gate == nullptr))
        return ZCCL_ERR_INVALID_ARG;
    if (rows == 0) {
        // sums over no rows; a gate has no rows either
        for (void* p : {d_grad_weight, d_grad_post_weight})
            if (p != nullptr && cudaMemsetAsync(p, 0, a.hidden * ws, stream) != cudaSuccess) return ZCCL_ERR_CUDA;
        return ZCCL_OK;
    }
    const bool reads_y = join && (a.post || d_grad_gate != nullptr);
    if ((d_grad_r == nullptr && d_grad_h == nullptr) || !is_aligned(d_grad_r, xs) || !is_aligned(d_grad_h, ys) ||
        (d_grad_h != nullptr && !good_ptr(d_r, xs)) || (d_grad_h == nullptr && d_weight != nullptr) ||
        (reads_y && !good_ptr(d_y, ys)) || !is_aligned(d_grad_x, xs) || !is_aligned(d_grad_y, ys) ||
        (!join && (d_gate != nullptr || d_post_weight != nullptr)) ||
        (d_grad_x == nullptr && !join && d_grad_weight == nullptr))
        return ZCCL_ERR_INVALID_ARG;
    uint64_t need = 0;
    zccl_residual_norm_workspace_bytes(a.hidden, rows, &need);
    if (!good_ptr(d_ws, 16)) return ZCCL_ERR_INVALID_ARG;
    if (ws_bytes < need) return ZCCL_ERR_BUFFER_TOO_SMALL;
    a.post = a.post && join;
    a.x = d_grad_h != nullptr ? d_r : nullptr;
    a.y = reads_y ? d_y : nullptr;
    a.x_stride = r_stride;
    a.y_stride = y_stride;
    a.grad_r = d_grad_r;
    a.grad_h = d_grad_h;
    a.grad_r_stride = grad_r_stride;
    a.grad_h_stride = grad_h_stride;
    a.grad_x = d_grad_x;
    a.grad_y = d_grad_y;
    a.grad_weight = d_grad_weight;
    a.grad_post_weight = d_grad_post_weight;
    a.grad_gate = d_grad_gate;
    a.sums = static_cast<float*>(d_ws);
    const bool vec = a.hidden % 8 == 0 && on_16(a.x, x_dtype, r_stride, rows) && on_16(a.y, dtype, y_stride, rows) &&
                     on_16(d_grad_r, x_dtype, grad_r_stride, rows) && on_16(d_grad_h, dtype, grad_h_stride, rows) &&
                     on_16(d_grad_x, x_dtype, 0, 1) && on_16(d_grad_y, dtype, 0, 1) && on_16(d_weight, weight_dtype, 0, 1) &&
                     on_16(d_post_weight, weight_dtype, 0, 1) && on_16(d_gate, gate_dtype, gate_stride, rows) &&
                     on_16(d_grad_gate, gate_dtype, 0, 1);
    return launch_norm_backward(a, x_dtype, dtype, weight_dtype, vec, stream);
}

}  // extern "C"
