// zccl_fp8_small.cu -- products of block-scaled e4m3 weights with few rows: a
// serving step's.
//
// With few rows a group the weights' bytes are all the work, so the kernel is
// built to stream them: a warp reads 16 weight rows of a block (2 KB, straight
// to registers in the layout of the 16 x 8 x 32 matrix instruction: the order
// of the values along the reduction axis is free as long as both operands share
// it), and the eight warps of a CTA split the reduction and add up in shared
// memory.  The rows are quantised on the fly, in registers, so a call is one
// launch.  The products are exact in the instruction; sums are fp32.
#include "zccl_fp8.cuh"

namespace zccl {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kTileRows = 16;  // weight rows of an item

__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 values of a row from column c on, zeros past its end or without a row.
template <typename T, bool kVec>
__device__ __forceinline__ void load16(const T* row, uint32_t c, uint32_t cols, bool on, float (&v)[16])
{
    if (kVec) {
        constexpr int kLoads = 16 * sizeof(T) / 16, kPer = 16 / kLoads;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool in = on && c + i * kPer < cols;
            const uint4 p = in ? *(reinterpret_cast<const uint4*>(row + c) + i) : make_uint4(0, 0, 0, 0);
            const uint32_t q[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (sizeof(T) == 2) {
                    v[i * 8 + 2 * j] = bf16_lo(q[j]);
                    v[i * 8 + 2 * j + 1] = bf16_hi(q[j]);
                } else {
                    v[i * 4 + j] = __uint_as_float(q[j]);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = on && c + i < cols ? to_float<T>(row[c + i]) : 0.0f;
    }
}

template <typename T, bool kVec, int kNT>
__global__ void __launch_bounds__(kThreads) small_kernel(SmallArgs a)
{
    constexpr uint32_t kChunk = 8 * kNT;  // rows of an item
    __shared__ float sums[kWarps][kNT * 4][32];
    __shared__ uint32_t prefix[kMaxGroupsFp8 + 1];
    pdl_wait();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, q = lane & 3;
    group_prefix(a.offsets, a.rows, a.G, kChunk, 0x7FFFFFFFu, prefix);
    __syncthreads();
    const uint32_t tiles = (a.n + kTileRows - 1) / kTileRows, nbs = (uint32_t)blocks_of(a.n);
    const uint64_t items = (uint64_t)prefix[a.G] * tiles;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t chunk = (uint32_t)(it / tiles), n0 = (uint32_t)(it % tiles) * kTileRows;
        const uint32_t g = group_at(prefix, a.G, chunk);
        uint32_t lo, hi;
        group_rows(a.offsets, a.rows, g, &lo, &hi);
        const uint32_t r0 = lo + (chunk - prefix[g]) * kChunk, count = min(kChunk, hi - r0);
        const uint32_t na = min(n0 + gq, a.n - 1), nb = min(n0 + gq + 8, a.n - 1);
        const float* sb = a.sb + ((uint64_t)g * nbs + n0 / kFp8Block) * a.KB;
        float acc[kNT][4] = {};
#pragma unroll 2
        for (uint32_t kb = warp; kb < a.KB; kb += kWarps) {
            const uint8_t* base = a.b + ((uint64_t)g * a.KB + kb) * a.n * kFp8Block + q * 16;
            const uint4 wa0 = ld_once(reinterpret_cast<const uint4*>(base + (uint64_t)na * kFp8Block));
            const uint4 wa1 = ld_once(reinterpret_cast<const uint4*>(base + (uint64_t)na * kFp8Block + 64));
            const uint4 wb0 = ld_once(reinterpret_cast<const uint4*>(base + (uint64_t)nb * kFp8Block));
            const uint4 wb1 = ld_once(reinterpret_cast<const uint4*>(base + (uint64_t)nb * kFp8Block + 64));
            const float sw = sb[kb];
#pragma unroll
            for (int t = 0; t < kNT; ++t) {
                const uint32_t r = t * 8 + gq;
                const bool on = r < count;
                const T* row = reinterpret_cast<const T*>(a.x) + (uint64_t)(r0 + (on ? r : 0)) * a.stride;
                float v0[16], v1[16], amax = 0.0f;
                load16<T, kVec>(row, kb * kFp8Block + q * 16, a.K, on, v0);
                load16<T, kVec>(row, kb * kFp8Block + q * 16 + 64, a.K, on, v1);
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(v0[i]), fabsf(v1[i])));
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
                float scale, f;
                block_scale(amax, &scale, &f);
                uint32_t x0[4], x1[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x0[i] = e4m3x4(v0[4 * i] * f, v0[4 * i + 1] * f, v0[4 * i + 2] * f, v0[4 * i + 3] * f);
                    x1[i] = e4m3x4(v1[4 * i] * f, v1[4 * i + 1] * f, v1[4 * i + 2] * f, v1[4 * i + 3] * f);
                }
                float d[4] = {};
                mma_16x8x32(d, wa0.x, wb0.x, wa0.y, wb0.y, x0[0], x0[1]);
                mma_16x8x32(d, wa0.z, wb0.z, wa0.w, wb0.w, x0[2], x0[3]);
                mma_16x8x32(d, wa1.x, wb1.x, wa1.y, wb1.y, x1[0], x1[1]);
                mma_16x8x32(d, wa1.z, wb1.z, wa1.w, wb1.w, x1[2], x1[3]);
                // the instruction's columns are rows 2 q and 2 q + 1 of x
                const float s0 = sw * __shfl_sync(0xFFFFFFFFu, scale, 8 * q);
                const float s1 = sw * __shfl_sync(0xFFFFFFFFu, scale, 8 * q + 4);
                acc[t][0] = fmaf(d[0], s0, acc[t][0]);
                acc[t][1] = fmaf(d[1], s1, acc[t][1]);
                acc[t][2] = fmaf(d[2], s0, acc[t][2]);
                acc[t][3] = fmaf(d[3], s1, acc[t][3]);
            }
        }
#pragma unroll
        for (int t = 0; t < kNT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[warp][t * 4 + i][lane] = acc[t][i];
        __syncthreads();
        for (uint32_t o = threadIdx.x; o < kChunk * kTileRows; o += kThreads) {
            const uint32_t t = o / kTileRows, n = o % kTileRows;
            const uint32_t i = (t / 8) * 4 + (n / 8) * 2 + (t & 1), l = (n % 8) * 4 + (t % 8) / 2;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += sums[w][i][l];
            if (t < count && n0 + n < a.n) {
                const uint64_t at = (uint64_t)(r0 + t) * a.n + n0 + n;
                if (a.out_f32)
                    reinterpret_cast<float*>(a.out)[at] = sum;
                else
                    reinterpret_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(sum);
            }
        }
        __syncthreads();
    }
    // rows outside every group
    if (a.offsets != nullptr) {
        const int32_t t = ld_l2(a.offsets + a.G);
        const uint64_t tail = t < 0 ? 0u : min((uint32_t)t, a.rows), n = (uint64_t)a.rows * a.n;
        for (uint64_t i = tail * a.n + blockIdx.x * kThreads + threadIdx.x; i < n; i += (uint64_t)gridDim.x * kThreads) {
            if (a.out_f32)
                reinterpret_cast<float*>(a.out)[i] = 0.0f;
            else
                reinterpret_cast<uint16_t*>(a.out)[i] = 0;
        }
    }
}

template <typename T, bool kVec>
cudaError_t small_as(const SmallArgs& a, int sms, cudaStream_t stream)
{
    // rows an item takes: the mean rows of a group, rounded up to 8, 16 or 32
    const uint32_t mean = (a.rows + a.G - 1) / a.G;
    const uint32_t chunk = mean <= 8 ? 8 : mean <= 16 ? 16 : 32;
    const uint64_t items = ((uint64_t)a.rows / chunk + a.G) * ((a.n + kTileRows - 1) / kTileRows);
    const uint64_t most = (uint64_t)sms * 4;
    const uint32_t grid = (uint32_t)(items < most ? items : most);
    if (chunk == 8) return launch_dependent(small_kernel<T, kVec, 1>, grid, kThreads, 0, stream, a);
    if (chunk == 16) return launch_dependent(small_kernel<T, kVec, 2>, grid, kThreads, 0, stream, a);
    return launch_dependent(small_kernel<T, kVec, 4>, grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_small(const SmallArgs& a, int dtype, int sms, cudaStream_t stream)
{
    const uint32_t values = dtype == ZCCL_BF16 ? 8 : 4;
    const bool vec = a.K % values == 0 && a.stride % values == 0 && is_aligned(a.x, 16);
    if (dtype == ZCCL_BF16)
        return vec ? small_as<__nv_bfloat16, true>(a, sms, stream) : small_as<__nv_bfloat16, false>(a, sms, stream);
    return vec ? small_as<float, true>(a, sms, stream) : small_as<float, false>(a, sms, stream);
}

}  // namespace zccl
