// zccl_combine.cu -- the experts' rows weighted and added back into their
// tokens' rows, and the gradients of the rows and of the weights.
//
// Both are bound by HBM.  Forward: 2 T K H bytes read and 2 T H written; a
// thread owns up to four 16-byte pieces of a token's row and has eight pieces in
// flight, of as many slots' rows as there are.  Backward: 2 T K H read and as many
// written (the token's gradient row comes from L1/L2 for all but one of its K
// slots); a warp owns one slot, for short rows fewer lanes of it do, so the dot
// product needs no other warp.  16384 tokens, 8
// slots, hidden 2048: forward 93 us (6.5 TB/s), backward 178 us (6.4 TB/s).
#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr int kThreads = 256;

struct CombineArgs {
    const uint16_t* y;
    uint64_t rows;
    uint32_t pieces;  // 16-byte pieces of a row
    const int32_t* pos;
    const float* weights;
    uint64_t tokens;
    uint32_t K;
    uint16_t* out;
    // backward
    const uint16_t* grad_out;
    const int32_t* total;
    uint16_t* grad_y;
    float* grad_weights;
    uint32_t lanes;   // threads of a token (forward) or a slot
};

__device__ __forceinline__ void add_piece(float (&acc)[8], float w, const uint4& v)
{
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc[2 * i] = fmaf(w, bf16_lo(q[i]), acc[2 * i]);
        acc[2 * i + 1] = fmaf(w, bf16_hi(q[i]), acc[2 * i + 1]);
    }
}

// `lanes` threads (a power of two up to 256) own a token; each has kPieces pieces
// of kSlots rows in flight.
template <int kSlots, int kPieces>
__global__ void __launch_bounds__(kThreads) combine_kernel(CombineArgs a)
{
    pdl_wait();
    const uint32_t sub = threadIdx.x / a.lanes, at = threadIdx.x - sub * a.lanes;
    const uint64_t t = (uint64_t)blockIdx.x * (kThreads / a.lanes) + sub;
    if (t >= a.tokens) return;
    const int32_t* pos = a.pos + t * a.K;
    const float* weights = a.weights != nullptr ? a.weights + t * a.K : nullptr;
    for (uint32_t c0 = at; c0 < a.pieces; c0 += a.lanes * kPieces) {
        float acc[kPieces][8] = {};
        for (uint32_t k0 = 0; k0 < a.K; k0 += kSlots) {
            // the places first: a load behind each would wait for it
            int32_t row[kSlots];
            float w[kSlots];
#pragma unroll
            for (uint32_t k = 0; k < kSlots; ++k) {
                row[k] = k0 + k < a.K ? pos[k0 + k] : -1;
                w[k] = weights == nullptr ? 1.0f : k0 + k < a.K ? weights[k0 + k] : 0.0f;
            }
            uint4 v[kSlots][kPieces];
#pragma unroll
            for (uint32_t k = 0; k < kSlots; ++k) {
                const bool there = row[k] >= 0 && (uint64_t)row[k] < a.rows;
                if (!there) w[k] = 0.0f;
#pragma unroll
                for (uint32_t j = 0; j < kPieces; ++j) {
                    const uint32_t c = c0 + j * a.lanes;
                    v[k][j] = there && c < a.pieces ? ld_once(reinterpret_cast<const uint4*>(a.y) + (uint64_t)row[k] * a.pieces + c)
                                                    : make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (uint32_t k = 0; k < kSlots; ++k)
#pragma unroll
                for (uint32_t j = 0; j < kPieces; ++j) add_piece(acc[j], w[k], v[k][j]);
        }
#pragma unroll
        for (uint32_t j = 0; j < kPieces; ++j)
            if (c0 + j * a.lanes < a.pieces)
                reinterpret_cast<uint4*>(a.out)[t * a.pieces + c0 + j * a.lanes] =
                    make_uint4(pack_bf16(acc[j][0], acc[j][1]), pack_bf16(acc[j][2], acc[j][3]), pack_bf16(acc[j][4], acc[j][5]),
                               pack_bf16(acc[j][6], acc[j][7]));
    }
}

// kLanes threads (0: `lanes`, a power of two below 32) own a slot, and a row of
// grad_y.
template <uint32_t kLanes>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(CombineArgs a)
{
    pdl_wait();
    const uint32_t lanes = kLanes > 0 ? kLanes : a.lanes;
    const uint32_t at = threadIdx.x % lanes;
    const uint64_t i = (uint64_t)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    const bool slot = i < a.tokens * a.K;
    const int32_t row = slot ? a.pos[i] : -1;
    float dot = 0.0f;
    if (row >= 0 && (uint64_t)row < a.rows) {
        const float w = a.weights != nullptr ? a.weights[i] : 1.0f;
        const uint4* up = reinterpret_cast<const uint4*>(a.grad_out) + (i / a.K) * a.pieces;
        const uint4* y = reinterpret_cast<const uint4*>(a.y) + (uint64_t)row * a.pieces;
        uint4* gy = reinterpret_cast<uint4*>(a.grad_y) + (uint64_t)row * a.pieces;
        constexpr int kFlight = 4;
        for (uint32_t c0 = at; c0 < a.pieces; c0 += lanes * kFlight) {
            uint4 g[kFlight], v[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const uint32_t c = c0 + lanes * u;
                const bool in = c < a.pieces;
                g[u] = in ? up[c] : make_uint4(0, 0, 0, 0);
                v[u] = in && a.y != nullptr ? ld_once(y + c) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < kFlight; ++u) {
                const uint32_t gq[4] = {g[u].x, g[u].y, g[u].z, g[u].w}, vq[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float lo = bf16_lo(gq[q]), hi = bf16_hi(gq[q]);
                    dot = fmaf(lo, bf16_lo(vq[q]), dot);
                    dot = fmaf(hi, bf16_hi(vq[q]), dot);
                    o[q] = pack_bf16(w * lo, w * hi);
                }
                if (c0 + lanes * u < a.pieces) __stcs(gy + c0 + lanes * u, make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
    __syncwarp();
    for (uint32_t o = a.lanes / 2; o > 0; o /= 2) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
    if (at == 0 && slot && a.grad_weights != nullptr) a.grad_weights[i] = dot;
    // rows that no slot points to
    if (a.total != nullptr && i < a.rows && (int64_t)i >= (int64_t)*a.total) {
        uint4* gy = reinterpret_cast<uint4*>(a.grad_y) + i * a.pieces;
        for (uint32_t c = at; c < a.pieces; c += lanes) gy[c] = make_uint4(0, 0, 0, 0);
    }
}

// The smallest power of two up to `most` that is at least n.
uint32_t lanes_for(uint32_t n, uint32_t most)
{
    uint32_t lanes = 1;
    while (lanes < most && lanes < n) lanes *= 2;
    return lanes;
}

bool combine_sizes_ok(uint64_t rows, uint64_t hidden, uint64_t tokens, uint32_t top_k)
{
    return top_k >= 1 && top_k <= ZCCL_MAX_TOP_K && tokens < (1ull << 31) / top_k && rows < (1ull << 31) &&
           hidden % 8 == 0 && hidden < (1ull << 24) && rows * hidden < kMaxElems && tokens * hidden < kMaxElems;
}

}  // namespace

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_combine(const uint16_t* d_y, uint64_t rows, uint64_t hidden, const int32_t* d_pos,
                           const float* d_weights, uint64_t tokens, uint32_t top_k, uint16_t* d_out,
                           cudaStream_t stream)
{
    if (!combine_sizes_ok(rows, hidden, tokens, top_k) || !is_aligned(d_weights, 4)) return ZCCL_ERR_INVALID_ARG;
    if (tokens == 0 || hidden == 0) return ZCCL_OK;
    if ((rows > 0 && d_y == nullptr) || !is_aligned(d_y, 16) || !good_ptr(d_pos, 4) || !good_ptr(d_out, 16))
        return ZCCL_ERR_INVALID_ARG;
    CombineArgs a{};
    a.y = d_y;
    a.rows = rows;
    a.pieces = (uint32_t)(hidden / 8);
    a.pos = d_pos;
    a.weights = d_weights;
    a.tokens = tokens;
    a.K = top_k;
    a.out = d_out;
    // Eight pieces in flight in a thread, of as many slots as there are up to eight: with eight slots' places and one
    // piece for any K, 16384 tokens with one slot, hidden 4096, took 95 us, now 44;
    // two slots, 1024: 27 and 18.
    const uint32_t in_flight = top_k == 1 ? 4 : top_k == 2 ? 4 : top_k <= 4 ? 2 : 1;
    a.lanes = lanes_for((a.pieces + in_flight - 1) / in_flight, kThreads);
    void (*kernel)(CombineArgs) = top_k == 1   ? combine_kernel<1, 4>
                                  : top_k == 2 ? combine_kernel<2, 4>
                                  : top_k <= 4 ? combine_kernel<4, 2>
                                               : combine_kernel<8, 1>;
    const uint32_t per_cta = kThreads / a.lanes;
    return launched(launch_dependent(kernel, (uint32_t)((tokens + per_cta - 1) / per_cta), kThreads, 0, stream, a));
}

zccl_status_t zccl_combine_backward(const uint16_t* d_grad_out, const uint16_t* d_y, uint64_t rows, uint64_t hidden,
                                    const int32_t* d_pos, const float* d_weights, const int32_t* d_total,
                                    uint64_t tokens, uint32_t top_k, uint16_t* d_grad_y, float* d_grad_weights,
                                    cudaStream_t stream)
{
    if (!combine_sizes_ok(rows, hidden, tokens, top_k) || !is_aligned(d_weights, 4) || !is_aligned(d_total, 4) ||
        !is_aligned(d_y, 16) || !is_aligned(d_grad_y, 16) || !is_aligned(d_grad_weights, 4) ||
        (d_grad_weights != nullptr && rows > 0 && hidden > 0 && d_y == nullptr))
        return ZCCL_ERR_INVALID_ARG;
    if (tokens > 0 && (!good_ptr(d_pos, 4) || (hidden > 0 && !good_ptr(d_grad_out, 16)))) return ZCCL_ERR_INVALID_ARG;
    if (rows > 0 && hidden > 0 && d_grad_y == nullptr) return ZCCL_ERR_INVALID_ARG;
    const uint64_t slots = tokens * top_k, items = slots > rows ? slots : rows;
    if (items == 0) return ZCCL_OK;
    CombineArgs a{};
    a.y = d_grad_weights != nullptr ? d_y : nullptr;
    a.rows = rows;
    a.pieces = (uint32_t)(hidden / 8);
    a.pos = d_pos;
    a.weights = d_weights;
    a.tokens = tokens;
    a.K = top_k;
    a.grad_out = d_grad_out;
    a.total = d_total;
    a.grad_y = d_grad_y;
    a.grad_weights = d_grad_weights;
    // a warp a slot, and fewer lanes for short rows: 16384 tokens of 8 slots, hidden 64, took 43 us with a
    // warp, 15 with a lane a piece, 8 with a lane four pieces
    a.lanes = lanes_for((a.pieces + 3) / 4, 32);
    const uint32_t per_cta = kThreads / a.lanes;
    return launched(launch_dependent(a.lanes == 32 ? combine_backward_kernel<32> : combine_backward_kernel<0>,
                                     (uint32_t)((items + per_cta - 1) / per_cta), kThreads, 0, stream, a));
}

}  // extern "C"
