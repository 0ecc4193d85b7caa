// zccl_norm.cu -- the host side of the join of a block's output with the residual and
// of the norms around it, both directions.
#include <cmath>

#include "zccl_norm.h"

namespace zccl {

namespace {

bool dtype_ok(int dtype) { return dtype == ZCCL_BF16 || dtype == ZCCL_F32; }

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
    a->gate_span = (uint32_t)(gate_span < rows ? gate_span : rows > 0 ? rows : 1);
    a->rows = (uint32_t)rows;
    a->hidden = (uint32_t)c->hidden;
    a->post = c->post != 0;
    a->inv_hidden = 1.0f / (float)c->hidden;
    a->eps = c->eps;
    a->scale = c->scale;
    a->gain = a->drop.below > 0 ? a->drop.gain : 1.0f;
    a->factor = a->scale * a->gain;
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
    const Shape s = norm_shape(a.hidden, a.rows, size_of(x_dtype) + size_of(dtype), vec, false);
    a.workers = s.workers;
    const bool post = a.post && a.y != nullptr, drop = a.drop.below > 0;
    uint32_t warp_bytes = 0;
    const NormKernel kernel = x_dtype == ZCCL_BF16
                                  ? (dtype == ZCCL_BF16 ? norm_kernel_for<__nv_bfloat16, __nv_bfloat16>(s, vec, post, drop, &warp_bytes)
                                                        : norm_kernel_for<__nv_bfloat16, float>(s, vec, post, drop, &warp_bytes))
                                  : (dtype == ZCCL_BF16 ? norm_kernel_for<float, __nv_bfloat16>(s, vec, post, drop, &warp_bytes)
                                                        : norm_kernel_for<float, float>(s, vec, post, drop, &warp_bytes));
    return launched(launch_teams(kernel, s, s.warps * 32, s.team == kLong ? 0 : s.warps * warp_bytes, stream, a));
}

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_residual_norm(const zccl_norm_t* cfg, const void* d_x, int x_dtype, uint64_t x_stride,
                                 const void* d_y, int dtype, uint64_t y_stride, const void* d_weight,
                                 const void* d_post_weight, int weight_dtype, const void* d_gate, int gate_dtype,
                                 uint64_t gate_stride, uint64_t gate_span, uint64_t rows, uint64_t offset,
                                 const uint64_t* d_offset, void* d_r, void* d_h, uint32_t* d_status,
                                 cudaStream_t stream)
{
    NormArgs a{};
    if (!norm_config(cfg, x_dtype, dtype, d_weight, d_post_weight, weight_dtype, d_gate, gate_dtype, gate_stride, gate_span,
                     rows, offset, d_offset, &a) ||
        x_stride >= kMaxElems || y_stride >= kMaxElems || !is_aligned(d_status, 4))
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
    a.status = d_status;
    const bool vec = a.hidden % 8 == 0 && on_16(d_x, x_dtype, x_stride, rows) && on_16(d_y, dtype, y_stride, rows) &&
                     on_16(d_r, x_dtype, 0, 1) && on_16(d_h, dtype, 0, 1) && on_16(d_weight, weight_dtype, 0, 1) &&
                     on_16(d_post_weight, weight_dtype, 0, 1) && on_16(d_gate, gate_dtype, gate_stride, rows);
    return launch_norm(a, x_dtype, dtype, vec, stream);
}

zccl_status_t zccl_residual_norm_workspace_bytes(uint64_t hidden, uint64_t rows, uint64_t* bytes)
{
    if (bytes == nullptr || hidden == 0 || hidden > ZCCL_MAX_NORM_HIDDEN || rows >= (1ull << 31)) return ZCCL_ERR_INVALID_ARG;
    *bytes = 0;  // the most, whatever the types
    for (uint32_t of_values = 4; of_values <= 8; of_values += 2)
        for (const bool vec : {false, true}) {
            const uint64_t need = norm_backward_bytes(norm_shape(hidden, rows, of_values, vec, true), hidden);
            if (need > *bytes) *bytes = need;
        }
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
                                          uint64_t ws_bytes, uint32_t* d_status, cudaStream_t stream)
{
    NormArgs a{};
    if (!norm_config(cfg, x_dtype, dtype, d_weight, d_post_weight, weight_dtype, d_gate, gate_dtype, gate_stride, gate_span,
                     rows, offset, d_offset, &a) ||
        grad_r_stride >= kMaxElems || grad_h_stride >= kMaxElems || r_stride >= kMaxElems || y_stride >= kMaxElems ||
        !is_aligned(d_status, 4))
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
    a.status = d_status;
    const bool vec = a.hidden % 8 == 0 && on_16(a.x, x_dtype, r_stride, rows) && on_16(a.y, dtype, y_stride, rows) &&
                     on_16(d_grad_r, x_dtype, grad_r_stride, rows) && on_16(d_grad_h, dtype, grad_h_stride, rows) &&
                     on_16(d_grad_x, x_dtype, 0, 1) && on_16(d_grad_y, dtype, 0, 1) && on_16(d_weight, weight_dtype, 0, 1) &&
                     on_16(d_post_weight, weight_dtype, 0, 1) && on_16(d_gate, gate_dtype, gate_stride, rows) &&
                     on_16(d_grad_gate, gate_dtype, 0, 1);
    return launch_norm_backward(a, x_dtype, dtype, weight_dtype, vec, stream);
}

}  // extern "C"
