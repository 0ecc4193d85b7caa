// zccl_fp8_host.cu -- the C ABI of the block-scaled e4m3 layers: argument
// checks, the workspace's layout and the choice of kernels.
#include "zccl_fp8.cuh"

using namespace zccl;

namespace {

constexpr uint64_t kMaxDim = 1ull << 24;        // one extent of a product
constexpr uint64_t kMaxBoxRows = 1ull << 31;    // operand rows of 128 codes, a TMA coordinate

bool sizes_ok(uint64_t rows, uint64_t k, uint64_t n, uint32_t groups)
{
    return groups >= 1 && groups <= kMaxGroupsFp8 && k >= 1 && n >= 1 && k < kMaxDim && n < kMaxDim &&
           rows < (1ull << 31) && blocks_of(k) * rows < kMaxBoxRows && blocks_of(n) * rows < kMaxBoxRows &&
           groups * blocks_of(k) * n < kMaxBoxRows && groups * blocks_of(n) * k < kMaxBoxRows &&
           (rows / kFp8Block + groups) * (k > n ? k : n) < kMaxBoxRows;
}

bool float_type(int t) { return t == ZCCL_BF16 || t == ZCCL_F32; }
uintptr_t size_of(int t) { return t == ZCCL_BF16 ? 2 : 4; }

// A workspace begins with the counters of a call's products: two tickets, then those of a product's parts.
constexpr uint64_t kCountersAt = 256;
constexpr uint64_t kTicketBytes = kCountersAt + 4 * kJoinCounters;
static_assert(kTicketBytes % 256 == 0, "what follows is aligned");

// Rows of `cols` values quantised by row.
struct RowsLayout {
    uint64_t q, scale, end;
};
RowsLayout rows_layout(uint64_t at, uint64_t rows, uint64_t cols)
{
    RowsLayout l;
    l.q = at;
    l.scale = l.q + blocks_of(cols) * rows * kFp8Block;
    l.end = round_up(l.scale + 4 * blocks_of(cols) * rows, 256);
    return l;
}

// The same quantised along the rows of each group.
uint64_t token_blocks(uint64_t rows, uint32_t groups) { return rows / kFp8Block + groups; }
RowsLayout tokens_layout(uint64_t at, uint64_t rows, uint64_t cols, uint32_t groups)
{
    RowsLayout l;
    l.q = at;
    l.scale = l.q + token_blocks(rows, groups) * cols * kFp8Block;
    l.end = round_up(l.scale + 4 * token_blocks(rows, groups) * cols, 256);
    return l;
}

// y = x times the transpose of the packed weight [groups][n][k].  x nullptr: x is
// quantised in the workspace already.  parts: room for part_bytes().
zccl_status_t linear(const void* x, int dtype, uint64_t stride, uint64_t rows, uint64_t k, const uint8_t* weight, uint64_t n,
                     uint32_t groups, const int32_t* offsets, void* out, int out_dtype, uint8_t* ws, uint8_t* parts,
                     uint32_t* status, int sms, cudaStream_t stream)
{
    const float* sb = reinterpret_cast<const float*>(weight + weight_code_bytes(groups, n, k));
    const RowsLayout l = rows_layout(kTicketBytes, rows, k);
    QuantArgs q{};
    q.x = x;
    q.stride = stride;
    q.rows = (uint32_t)rows;
    q.cols = (uint32_t)k;
    q.q = ws + l.q;
    q.scale = reinterpret_cast<float*>(ws + l.scale);
    q.ticket = reinterpret_cast<uint32_t*>(ws);
    const uint32_t split = matmul_split(rows, n, k, groups);
    q.counters = split > 1 ? reinterpret_cast<uint32_t*>(ws + kCountersAt) : nullptr;
    if (x != nullptr && launch_quantize_rows(q, dtype, sms, stream) != cudaSuccess) return ZCCL_ERR_CUDA;
    MatmulArgs m{};
    m.a = q.q;
    m.sa = q.scale;
    m.b = weight;
    m.sb = sb;
    m.offsets = offsets;
    m.rows = (uint32_t)rows;
    m.n = (uint32_t)n;
    m.KB = (uint32_t)blocks_of(k);
    m.G = groups;
    m.out = out;
    m.out_f32 = out_dtype == ZCCL_F32;
    m.ticket = reinterpret_cast<uint32_t*>(ws);
    m.split = split;
    m.counters = reinterpret_cast<uint32_t*>(ws + kCountersAt);
    m.parts = reinterpret_cast<float*>(parts);
    m.status = status;
    return launched(takes_small(rows, n, k, groups, sms) ? launch_small(m, sms, stream) : launch_matmul(m, sms, stream));
}

}  // namespace

extern "C" {

zccl_status_t zccl_fp8_weight_bytes(uint32_t groups, uint64_t n, uint64_t k, uint64_t* bytes)
{
    if (bytes == nullptr || !sizes_ok(0, k, n, groups)) return ZCCL_ERR_INVALID_ARG;
    *bytes = weight_bytes(groups, n, k);
    return ZCCL_OK;
}

zccl_status_t zccl_fp8_weight_quantize(const void* d_w, int dtype, uint32_t groups, uint64_t n, uint64_t k, void* d_weight,
                                       void* d_weight_t, cudaStream_t stream)
{
    if (!sizes_ok(0, k, n, groups) || !float_type(dtype) || !good_ptr(d_w, size_of(dtype)) ||
        (d_weight == nullptr && d_weight_t == nullptr) || !is_aligned(d_weight, 16) || !is_aligned(d_weight_t, 16) ||
        groups * blocks_of(n) * blocks_of(k) >= (1ull << 31))
        return ZCCL_ERR_INVALID_ARG;
    PackArgs p{};
    p.w = d_w;
    p.G = groups;
    p.n = (uint32_t)n;
    p.k = (uint32_t)k;
    p.packed = reinterpret_cast<uint8_t*>(d_weight);
    p.packed_t = reinterpret_cast<uint8_t*>(d_weight_t);
    return launched(launch_pack(p, dtype, stream));
}

zccl_status_t zccl_fp8_weight_pack(const void* d_codes, const float* d_scale, uint32_t groups, uint64_t n, uint64_t k,
                                   void* d_weight, void* d_weight_t, cudaStream_t stream)
{
    if (!sizes_ok(0, k, n, groups) || d_codes == nullptr || !good_ptr(d_scale, 4) ||
        (d_weight == nullptr && d_weight_t == nullptr) || !is_aligned(d_weight, 16) || !is_aligned(d_weight_t, 16) ||
        groups * blocks_of(n) * blocks_of(k) >= (1ull << 31))
        return ZCCL_ERR_INVALID_ARG;
    PackArgs p{};
    p.codes = reinterpret_cast<const uint8_t*>(d_codes);
    p.scale = d_scale;
    p.G = groups;
    p.n = (uint32_t)n;
    p.k = (uint32_t)k;
    p.packed = reinterpret_cast<uint8_t*>(d_weight);
    p.packed_t = reinterpret_cast<uint8_t*>(d_weight_t);
    return launched(launch_pack(p, ZCCL_F32, stream));
}

zccl_status_t zccl_fp8_linear_workspace_bytes(uint64_t rows, uint64_t k, uint64_t n, uint32_t groups, int backward,
                                              uint64_t* bytes)
{
    if (bytes == nullptr || !sizes_ok(rows, k, n, groups)) return ZCCL_ERR_INVALID_ARG;
    if (!backward) {
        *bytes = rows_layout(kTicketBytes, rows, k).end + part_bytes(matmul_split(rows, n, k, groups));
    } else {
        const RowsLayout dy = rows_layout(kTicketBytes, rows, n), dyt = tokens_layout(dy.end, rows, n, groups);
        const uint32_t split = matmul_split(rows, k, n, groups), split_w = wgrad_split(rows, n, k, groups);
        *bytes = tokens_layout(dyt.end, rows, k, groups).end + part_bytes(split > split_w ? split : split_w);
    }
    return ZCCL_OK;
}

zccl_status_t zccl_fp8_linear(const void* d_x, int dtype, uint64_t stride, uint64_t rows, uint64_t k, const void* d_weight,
                              uint64_t n, uint32_t groups, const int32_t* d_offsets, void* d_out, int out_dtype,
                              void* d_ws, uint64_t ws_bytes, uint32_t* d_status, cudaStream_t stream)
{
    if (!sizes_ok(rows, k, n, groups) || !float_type(dtype) || !float_type(out_dtype) || stride >= kMaxElems ||
        (d_offsets == nullptr && groups != 1) || !is_aligned(d_offsets, 4) || !is_aligned(d_status, 4) ||
        !good_ptr(d_weight, 16) || !good_ptr(d_ws, 16))
        return ZCCL_ERR_INVALID_ARG;
    uint64_t need = 0;
    zccl_fp8_linear_workspace_bytes(rows, k, n, groups, 0, &need);
    if (ws_bytes < need) return ZCCL_ERR_BUFFER_TOO_SMALL;
    if (rows == 0) return ZCCL_OK;
    if (!good_ptr(d_x, size_of(dtype)) || !good_ptr(d_out, size_of(out_dtype))) return ZCCL_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return ZCCL_ERR_CUDA;
    uint8_t* ws = reinterpret_cast<uint8_t*>(d_ws);
    return linear(d_x, dtype, stride, rows, k, reinterpret_cast<const uint8_t*>(d_weight), n, groups, d_offsets, d_out,
                  out_dtype, ws, ws + rows_layout(kTicketBytes, rows, k).end, d_status, sms, stream);
}

zccl_status_t zccl_fp8_linear_backward(const void* d_grad, const void* d_x, int dtype, uint64_t grad_stride,
                                       uint64_t x_stride, uint64_t rows, uint64_t k, const void* d_weight_t, uint64_t n,
                                       uint32_t groups, const int32_t* d_offsets, void* d_grad_x, void* d_grad_w,
                                       int out_dtype, void* d_ws, uint64_t ws_bytes, uint32_t* d_status,
                                       cudaStream_t stream)
{
    if (!sizes_ok(rows, k, n, groups) || !float_type(dtype) || !float_type(out_dtype) || grad_stride >= kMaxElems ||
        x_stride >= kMaxElems || (d_offsets == nullptr && groups != 1) || !is_aligned(d_offsets, 4) ||
        !is_aligned(d_status, 4) || !good_ptr(d_ws, 16) || (d_grad_x != nullptr && !good_ptr(d_weight_t, 16)) ||
        !is_aligned(d_grad_x, size_of(out_dtype)) || !is_aligned(d_grad_w, size_of(out_dtype)))
        return ZCCL_ERR_INVALID_ARG;
    uint64_t need = 0;
    zccl_fp8_linear_workspace_bytes(rows, k, n, groups, 1, &need);
    if (ws_bytes < need) return ZCCL_ERR_BUFFER_TOO_SMALL;
    if (rows > 0 && (!good_ptr(d_grad, size_of(dtype)) || (d_grad_w != nullptr && !good_ptr(d_x, size_of(dtype)))))
        return ZCCL_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return ZCCL_ERR_CUDA;
    uint8_t* ws = reinterpret_cast<uint8_t*>(d_ws);
    const RowsLayout dy = rows_layout(kTicketBytes, rows, n), dyt = tokens_layout(dy.end, rows, n, groups),
                     xt = tokens_layout(dyt.end, rows, k, groups);
    QuantArgs q{};
    q.rows = (uint32_t)rows;
    q.offsets = d_offsets;
    q.G = groups;
    q.x = d_grad;
    q.stride = grad_stride;
    q.cols = (uint32_t)n;
    q.q = ws + dyt.q;
    q.scale = reinterpret_cast<float*>(ws + dyt.scale);
    const bool both = d_grad_w != nullptr && d_grad_x != nullptr && rows > 0 && quantizes_both(q, dtype);
    if (both) {
        q.q_rows = ws + dy.q;
        q.scale_rows = reinterpret_cast<float*>(ws + dy.scale);
        q.ticket = reinterpret_cast<uint32_t*>(ws);  // the product of the rows' gradient
        if (matmul_split(rows, k, n, groups) > 1) q.counters = reinterpret_cast<uint32_t*>(ws + kCountersAt);
    }
    if (d_grad_w != nullptr && rows > 0 && launch_quantize_tokens(q, dtype, sms, stream) != cudaSuccess)
        return ZCCL_ERR_CUDA;
    if (d_grad_x != nullptr && rows > 0) {
        const zccl_status_t st =
            linear(both ? nullptr : d_grad, dtype, grad_stride, rows, n, reinterpret_cast<const uint8_t*>(d_weight_t), k,
                   groups, d_offsets, d_grad_x, out_dtype, ws, ws + xt.end, d_status, sms, stream);
        if (st != ZCCL_OK) return st;
    }
    if (d_grad_w == nullptr) return ZCCL_OK;
    QuantArgs r = q;
    r.x = d_x;
    r.stride = x_stride;
    r.cols = (uint32_t)k;
    r.q = ws + xt.q;
    r.scale = reinterpret_cast<float*>(ws + xt.scale);
    r.q_rows = nullptr;
    const uint32_t split = wgrad_split(rows, n, k, groups);
    r.counters = split > 1 ? reinterpret_cast<uint32_t*>(ws + kCountersAt) : nullptr;
    r.ticket = reinterpret_cast<uint32_t*>(ws) + 32;
    if (launch_quantize_tokens(r, dtype, sms, stream) != cudaSuccess) return ZCCL_ERR_CUDA;
    WgradArgs w{};
    w.a = q.q;
    w.sa = q.scale;
    w.b = r.q;
    w.sb = r.scale;
    w.offsets = d_offsets;
    w.rows = (uint32_t)rows;
    w.m = (uint32_t)n;
    w.n = (uint32_t)k;
    w.G = groups;
    w.blocks = (uint32_t)token_blocks(rows, groups);
    w.out = d_grad_w;
    w.out_f32 = out_dtype == ZCCL_F32;
    w.ticket = reinterpret_cast<uint32_t*>(ws) + 32;
    w.split = split;
    w.counters = reinterpret_cast<uint32_t*>(ws + kCountersAt);
    w.parts = reinterpret_cast<float*>(ws + xt.end);
    w.status = d_status;
    return launched(launch_wgrad(w, sms, stream));
}

}  // extern "C"
