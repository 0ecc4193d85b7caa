// zccl_dropout.cu -- dropout whose mask is recomputed from its counter.
//
// Ten rounds of the generator give eight values' bits: about 80 instructions for eight
// values with their comparisons, half of what the machine issues while HBM moves them in
// BF16.  131072 x 1024 in BF16: 90 us (5.9 TB/s, 88 % of measured); 8191 x 2047 in 32 bits,
// whose rows begin anywhere: 22 us (6.1 TB/s); the same in BF16 23 us, bound by its 16-bit
// loads and stores.
#include <cmath>

#include "zccl_rows.cuh"

namespace zccl {

namespace {

constexpr int kDropWarps = 8;
constexpr int kDropCtas = 3;  // of an SM

struct DropoutArgs {
    const void* x;
    uint64_t stride;
    uint64_t rows;
    uint32_t cols, tiles;  // tiles of a row
    uint32_t step;         // rows that the warps take at a time
    DropArgs drop;
    void* out;
};

// A warp keeps its place in the rows and goes from row to row, kRows of them on their
// way at a time.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kDropWarps * 32, kDropCtas) dropout_kernel(DropoutArgs a)
{
    constexpr int kRows = sizeof(T) == 2 ? 4 : 2;
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t warp = blockIdx.x * kDropWarps + (threadIdx.x >> 5);
    const uint32_t tile = warp % a.tiles * kTile;
    const uint64_t first = warp / a.tiles;
    if (first >= a.step) return;
    for (uint64_t row = first; row < a.rows; row += kRows * a.step) {
        Piece<T, kVec> p[kRows];
#pragma unroll
        for (int n = 0; n < kRows; ++n)
            if (row + n * a.step < a.rows) p[n].load(static_cast<const T*>(a.x) + (row + n * a.step) * a.stride, tile, a.cols);
#pragma unroll
        for (int n = 0; n < kRows; ++n) {
            const uint64_t at = row + n * a.step;
            if (at >= a.rows) break;
            const Kept<kVec> kept = kept_piece<kVec>(a.drop, offset, (uint32_t)at, tile);
            store8<T, kVec>(static_cast<T*>(a.out) + at * a.cols, where_kept<kVec>(kept, mul(p[n].get(), a.drop.gain)), tile, a.cols);
        }
    }
}

// Narrow rows: a lane has a block of eight columns, and a warp as many rows as its lanes
// have blocks for (100000 x 8 2.0 us, 16 with a warp a row).
constexpr uint32_t kNarrow = 128;  // columns

template <typename T, bool kVec>
__global__ void __launch_bounds__(kDropWarps * 32) dropout_narrow_kernel(DropoutArgs a)
{
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t lane = threadIdx.x & 31, blocks = (a.cols + 7) / 8, rows = 32 / blocks, sub = lane / blocks;
    const uint32_t block = lane - sub * blocks, col = block * 8;
    const uint64_t first = ((uint64_t)blockIdx.x * kDropWarps + (threadIdx.x >> 5)) * rows + sub;
    if (sub >= rows) return;
    for (uint64_t row = first; row < a.rows; row += a.step) {
        const T* x = static_cast<const T*>(a.x) + row * a.stride + col;
        T* out = static_cast<T*>(a.out) + row * a.cols + col;
        const Kept<true> kept = kept_block(a.drop, offset, (uint32_t)row, block);
        if (kVec) {
            store_near(out, where_kept<true>(kept, mul(load_near(x), a.drop.gain)));
        } else {
            Eight v = all_eight(0.0f);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < a.cols) v[j] = to_float<T>(x[j]);
            v = where_kept<true>(kept, mul(v, a.drop.gain));
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (col + j < a.cols) out[j] = from_float<T>(v[j]);
        }
    }
}

template <typename T>
cudaError_t launch_dropout(DropoutArgs& a, int sms, cudaStream_t stream)
{
    const bool vec = a.cols % 8 == 0 && a.stride * sizeof(T) % 16 == 0 && is_aligned(a.x, 16) && is_aligned(a.out, 16);
    if (a.cols <= kNarrow) {
        const uint64_t per_cta = kDropWarps * (32 / ((a.cols + 7) / 8)), ctas = (a.rows + per_cta - 1) / per_cta, most = (uint64_t)sms * 8;
        const uint32_t grid = (uint32_t)(ctas < most ? ctas : most);
        a.step = (uint32_t)(grid * per_cta);
        return launch_dependent(vec ? dropout_narrow_kernel<T, true> : dropout_narrow_kernel<T, false>, grid, kDropWarps * 32, 0,
                                stream, a);
    }
    // as many rows at a time as the machine holds: tiles < 2^16, so the CTAs for one row are fewer than 2^13
    const uint64_t most = (uint64_t)sms * kDropCtas * kDropWarps / a.tiles;
    a.step = (uint32_t)(a.rows < most ? a.rows : most > 0 ? most : 1);
    const uint64_t ctas = ((uint64_t)a.step * a.tiles + kDropWarps - 1) / kDropWarps;
    return launch_dependent(vec ? dropout_kernel<T, true> : dropout_kernel<T, false>, (uint32_t)ctas,
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
