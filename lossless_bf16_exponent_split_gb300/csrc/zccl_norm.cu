// zccl_norm.cu -- the join of a block's output with the residual and the norm of
// the next block's input, and the host side of both directions.
#include <cmath>

#include "zccl_norm.h"

namespace zccl {

namespace {

// A CTA a row, read once for each of its sums: any size.
template <typename Tx, typename Ty, bool kVec>
__global__ void __launch_bounds__(kTeamWarps * 32) norm_long_kernel(NormArgs a)
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
        float eta = 1.0f;
        float2 sum = twice(0.0f);
        if (a.y != nullptr && a.post) {
            for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
                const Eight v = load8<Ty, kVec>(y, tile, a.hidden);
                dot(sum, v, v);
            }
            float s[1] = {sum.x + sum.y};
            cta_sum<1>(s, red, turn);
            eta = rsqrtf(s[0] * a.inv_hidden + a.eps);
            sum = twice(0.0f);
        }
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            Eight v = load8<Tx, kVec>(x, tile, a.hidden);
            if (a.y != nullptr) {
                const Eight k = mul(join_factors<kVec>(a, t, tile), load_vector<kVec>(a.post_weight, 0, tile, a.hidden));
                const Eight b = mul(load8<Ty, kVec>(y, tile, a.hidden), eta);
                v = where_kept<kVec>(join_kept<kVec>(a, offset, t, tile), fma(k, b, v), v);
                v = store8<Tx, kVec>(r, v, tile, a.hidden);
            }
            dot(sum, v, v);
        }
        if (a.h == nullptr) continue;
        float s[1] = {sum.x + sum.y};
        cta_sum<1>(s, red, turn);
        const float rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            const Eight v = mul(load8<Tx, kVec>(a.y != nullptr ? r : x, tile, a.hidden), rho);
            store8<Ty, kVec>(static_cast<Ty*>(a.h) + t * a.hidden, mul(v, load_vector<kVec>(a.weight, 0, tile, a.hidden)), tile,
                             a.hidden);
        }
    }
}

// A team a worker: a row is read once and stays in registers, with the next one on its
// way; weights and the gate stay there too.
template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces>
__global__ void __launch_bounds__(kTeam == kWarpTeam ? kWarpsPerCta * 32 : kTeamWarps * 32, kTeam == kWarpTeam ? 2 : 1)
    norm_kernel(NormArgs a)
{
    __shared__ float red[kTeam == kWarpTeam ? 1 : kTeamRed];
    uint32_t turn = 0;
    pdl_wait();
    const Place at = place<kTeam>();
    if (kTeam == kWarpTeam && at.worker >= a.workers) return;
    const uint64_t offset = drop_offset(a.drop);
    const uint64_t lo = first_row(a.rows, a.workers, at.worker), hi = first_row(a.rows, a.workers, at.worker + 1);
    const bool join = a.y != nullptr;
    Piece<Tx, kVec> px[kPieces];
    Piece<Ty, kVec> py[kPieces] = {};
    const auto load = [&](uint64_t t) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            px[n].load(static_cast<const Tx*>(a.x) + t * a.x_stride, at.tile(n), a.hidden);
            if (join) py[n].load(static_cast<const Ty*>(a.y) + t * a.y_stride, at.tile(n), a.hidden);
        }
    };
    load(lo);
    Eight w[kPieces], k[kPieces];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) w[n] = load_vector<kVec>(a.weight, 0, at.tile(n), a.hidden);
    uint64_t gate_end = lo;  // where the gate changes
    for (uint64_t t = lo; t < hi; ++t) {
        Eight x[kPieces], y[kPieces];
#pragma unroll
        for (int n = 0; n < kPieces; ++n) x[n] = px[n].get(), y[n] = py[n].get();
        if (t + 1 < hi) load(t + 1);
        if (join) {
            if (t == gate_end) {
                // the join's factor of each column, with the weight of the norm after the block
#pragma unroll
                for (int n = 0; n < kPieces; ++n)
                    k[n] = mul(join_factors<kVec>(a, t, at.tile(n)), load_vector<kVec>(a.post_weight, 0, at.tile(n), a.hidden));
                gate_end = a.gate.p != nullptr ? (t / a.gate_span + 1) * a.gate_span : a.rows;
            }
            if (a.post) {
                float2 sum = twice(0.0f);
#pragma unroll
                for (int n = 0; n < kPieces; ++n) dot(sum, y[n], y[n]);
                float s[1] = {sum.x + sum.y};
                team_sum<1, kTeam>(s, red, turn);
                const float eta = rsqrtf(s[0] * a.inv_hidden + a.eps);
#pragma unroll
                for (int n = 0; n < kPieces; ++n) y[n] = mul(y[n], eta);
            }
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                x[n] = where_kept<kVec>(join_kept<kVec>(a, offset, t, at.tile(n)), fma(k[n], y[n], x[n]), x[n]);
                x[n] = store8<Tx, kVec>(static_cast<Tx*>(a.r) + t * a.hidden, x[n], at.tile(n), a.hidden);
            }
        }
        if (a.h == nullptr) continue;
        float2 sum = twice(0.0f);
#pragma unroll
        for (int n = 0; n < kPieces; ++n) dot(sum, x[n], x[n]);
        float s[1] = {sum.x + sum.y};
        team_sum<1, kTeam>(s, red, turn);
        const float rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
#pragma unroll
        for (int n = 0; n < kPieces; ++n)
            store8<Ty, kVec>(static_cast<Ty*>(a.h) + t * a.hidden, mul(mul(x[n], rho), w[n]), at.tile(n), a.hidden);
    }
}

using NormKernel = void (*)(NormArgs);

template <typename Tx, typename Ty, bool kVec>
NormKernel norm_for(const Shape& s)
{
    constexpr int kMost = kVec && sizeof(Tx) == 2 && sizeof(Ty) == 2 ? 2 : 1;
    if (s.team == kWarpTeam) return norm_kernel<Tx, Ty, kVec, kWarpTeam, 1>;
    if (s.team == kLong) return norm_long_kernel<Tx, Ty, kVec>;
    if (s.pieces == 1) return s.team == kCtaTeam ? norm_kernel<Tx, Ty, kVec, kCtaTeam, 1> : norm_kernel<Tx, Ty, kVec, kClusterTeam, 1>;
    return s.team == kCtaTeam ? norm_kernel<Tx, Ty, kVec, kCtaTeam, kMost> : norm_kernel<Tx, Ty, kVec, kClusterTeam, kMost>;
}
template <typename Tx>
NormKernel norm_for(int dtype, bool vec, const Shape& s)
{
    if (dtype == ZCCL_BF16) return vec ? norm_for<Tx, __nv_bfloat16, true>(s) : norm_for<Tx, __nv_bfloat16, false>(s);
    return vec ? norm_for<Tx, float, true>(s) : norm_for<Tx, float, false>(s);
}

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
    const Shape s = norm_shape(a.hidden, a.rows, vec && x_dtype == ZCCL_BF16 && dtype == ZCCL_BF16);
    a.workers = s.workers;
    const NormKernel kernel = x_dtype == ZCCL_BF16 ? norm_for<__nv_bfloat16>(dtype, vec, s) : norm_for<float>(dtype, vec, s);
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
    const uint64_t narrow = norm_backward_bytes(norm_shape(hidden, rows, true), hidden);
    const uint64_t wide = norm_backward_bytes(norm_shape(hidden, rows, false), hidden);
    *bytes = narrow > wide ? narrow : wide;  // whatever the types
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
