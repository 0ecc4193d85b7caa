// zccl_dropout.cu -- dropout whose mask is recomputed from its counter.
#include <cmath>

#include "zccl_rows.cuh"

namespace zccl {

namespace {

constexpr int kDropWarps = 8;

struct DropoutArgs {
    const void* x;
    uint64_t stride;
    uint64_t rows;
    uint32_t cols, tiles;  // tiles of a row
    DropArgs drop;
    void* out;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kDropWarps * 32) dropout_kernel(DropoutArgs a)
{
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint64_t total = a.rows * a.tiles, step = (uint64_t)gridDim.x * kDropWarps;
    for (uint64_t i = (uint64_t)blockIdx.x * kDropWarps + (threadIdx.x >> 5); i < total; i += step) {
        const uint64_t row = i / a.tiles;
        const uint32_t tile = (uint32_t)(i - row * a.tiles) * kTile;
        float v[8];
        load8<T, kVec>(v, static_cast<const T*>(a.x) + row * a.stride, tile, a.cols);
        const uint32_t kept = kept_piece<kVec>(a.drop, offset, (uint32_t)row, tile);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (kept >> j) & 1u ? v[j] * a.drop.gain : 0.0f;
        store8<T, kVec>(static_cast<T*>(a.out) + row * a.cols, v, tile, a.cols);
    }
}

template <typename T>
cudaError_t launch_dropout(const DropoutArgs& a, int sms, cudaStream_t stream)
{
    const uint64_t warps = a.rows * a.tiles, ctas = (warps + kDropWarps - 1) / kDropWarps, most = (uint64_t)sms * 64;
    const bool vec = a.cols % 8 == 0 && a.stride * sizeof(T) % 16 == 0 && is_aligned(a.x, 16) && is_aligned(a.out, 16);
    return launch_dependent(vec ? dropout_kernel<T, true> : dropout_kernel<T, false>, (uint32_t)(ctas < most ? ctas : most),
                            kDropWarps * 32, 0, stream, a);
}

}  // namespace

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_dropout(const void* d_x, int dtype, uint64_t stride, uint64_t rows, uint64_t cols, float p,
                           uint64_t seed, uint64_t offset, const uint64_t* d_offset, void* d_out, cudaStream_t stream)
{
    DropoutArgs a{};
    const uintptr_t size = dtype == ZCCL_BF16 ? 2 : 4;
    if ((dtype != ZCCL_BF16 && dtype != ZCCL_F32) || rows >= (1ull << 32) || cols >= (1ull << 24) ||
        rows * cols >= kMaxElems || stride >= kMaxElems || !drop_args(p, seed, offset, d_offset, &a.drop))
        return ZCCL_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return ZCCL_OK;
    if (!good_ptr(d_x, size) || !good_ptr(d_out, size) || (rows > 1 && d_x == d_out && stride != cols))
        return ZCCL_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (sms == 0) return ZCCL_ERR_CUDA;
    a.x = d_x;
    a.stride = stride;
    a.rows = rows;
    a.cols = (uint32_t)cols;
    a.tiles = (uint32_t)((cols + kTile - 1) / kTile);
    a.out = d_out;
    return launched(dtype == ZCCL_BF16 ? launch_dropout<__nv_bfloat16>(a, sms, stream) : launch_dropout<float>(a, sms, stream));
}

}  // extern "C"
