// zccl_fp8_small.cu -- products of block-scaled e4m3 weights with few rows: a
// serving step's.
//
// With few rows a group the weights' bytes are all the work, so the kernel is
// built to stream them: a warp reads 16 weight rows of a block (2 KB, straight
// to registers in the layout of the 16 x 8 x 32 matrix instruction: the order
// of the values along the reduction axis is free as long as both operands share
// it) and multiplies them with 8 rows of x, or two or four times as many.  Where
// there are too few such pieces for the GPU's warps, up to eight warps split the
// reduction and add up in shared memory.  Products are exact in the instruction;
// sums are fp32, in an order that depends on the sizes only.
//
// The instruction's e4m3 operands are converted in the integer pipe, which bounds
// the kernel from 16 rows on; one row through 14336 x 4096 (n x k) takes 12.9 us
// with the quantisation (2.0 us alone) that it starts beside, 264 rows through 64
// experts of 1024 x 2048 28.7 us after theirs (4.4 TB/s).  With two and four eights
// of rows a warp the register caps spill (188 and 40 bytes a thread).
// Measured and left out: the weights through a ring in shared memory (bulk copies
// and these instructions, or TMA and the tensor memory's, every CTA with an equal
// piece of all the blocks): 10 % less for the 64 experts, 15 % more for one row.
#include "zccl_fp8.cuh"

namespace zccl {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr uint32_t kTileRows = 16;  // weight rows of a warp
constexpr uint32_t kEarly = 4;      // blocks of a warp that are asked for while x is quantised
constexpr int kFlight = 2;          // blocks in flight in a warp; with three CTAs an SM enough to fill the memory's latency

__device__ __forceinline__ void mma_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Consecutive bytes to L2 (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// `split` warps (1, 2, 4 or 8) share a warp's weight rows.
template <typename T, int kNT>
__global__ void __launch_bounds__(kThreads, kNT == 4 ? 2 : 3) small_kernel(MatmulArgs a, uint32_t split)
{
    constexpr uint32_t kChunk = 8 * kNT;  // rows of x
    __shared__ float sums[kWarps][kNT * 4][32];
    __shared__ uint32_t prefix[kMaxGroupsFp8 + 1];
    __shared__ uint2 range[kMaxGroupsFp8];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, q = lane & 3;
    // The kernel before this one quantises x.  It lets this one start once everything before it is done, so the
    // groups' table and the weights can be read; x and its scales, and anything written, come after the wait.
    group_prefix(a.offsets, a.rows, a.G, kChunk, 0x7FFFFFFFu, prefix);
    for (uint32_t g = threadIdx.x; g < a.G; g += kThreads) group_rows(a.offsets, a.rows, g, &range[g].x, &range[g].y);
    __syncthreads();
    const uint32_t nbs = (uint32_t)blocks_of(a.n), wide = kWarps / split * kTileRows;  // weight rows of a CTA
    const uint32_t tiles = (a.n + wide - 1) / wide, first = warp % split;
    const uint64_t items = (uint64_t)prefix[a.G] * tiles;
    if (blockIdx.x < items) {  // the first weights to L2 meanwhile, a lane a block (1 to 2 us less a call)
        const uint32_t chunk = blockIdx.x / tiles, g = group_at(prefix, a.G, chunk), kb = first + lane * split;
        const uint32_t n0 = (blockIdx.x - chunk * tiles) * wide + warp / split * kTileRows;
        if (lane < kEarly && kb < a.KB && n0 < a.n)
            prefetch_l2(a.b + (((uint64_t)g * a.KB + kb) * a.n + n0) * kFp8Block, min(kTileRows, a.n - n0) * kFp8Block);
    }
    pdl_wait();
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t chunk = (uint32_t)(it / tiles);
        const uint32_t n0 = (uint32_t)(it - (uint64_t)chunk * tiles) * wide + warp / split * kTileRows;
        const uint32_t g = group_at(prefix, a.G, chunk);
        const uint32_t r0 = range[g].x + (chunk - prefix[g]) * kChunk, count = min(kChunk, range[g].y - r0);
        float acc[kNT][4] = {};
        if (n0 < a.n) {
            // lanes past the weight's or x's last row read that row and drop the result
            const uint8_t* const wa = a.b + ((uint64_t)g * a.KB * a.n + min(n0 + gq, a.n - 1)) * kFp8Block + q * 16;
            const uint8_t* const wb = a.b + ((uint64_t)g * a.KB * a.n + min(n0 + gq + 8, a.n - 1)) * kFp8Block + q * 16;
            const float* const sb = a.sb + ((uint64_t)g * nbs + n0 / kFp8Block) * a.KB;
            const uint64_t wstep = (uint64_t)a.n * kFp8Block, xstep = (uint64_t)a.rows * kFp8Block;
            for (uint32_t kb0 = first; kb0 < a.KB; kb0 += kFlight * split) {
                uint4 w[kFlight][4], x[kFlight][kNT][2];
                float s[kFlight][kNT][2], sw[kFlight];
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    const uint32_t kb = min(kb0 + f * split, a.KB - 1);
                    w[f][0] = ld_once(reinterpret_cast<const uint4*>(wa + kb * wstep));
                    w[f][1] = ld_once(reinterpret_cast<const uint4*>(wa + kb * wstep + 64));
                    w[f][2] = ld_once(reinterpret_cast<const uint4*>(wb + kb * wstep));
                    w[f][3] = ld_once(reinterpret_cast<const uint4*>(wb + kb * wstep + 64));
                }
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    const uint32_t kb = min(kb0 + f * split, a.KB - 1);
                    sw[f] = kb0 + f * split < a.KB ? sb[kb] : 0.0f;  // a block too many adds nothing
#pragma unroll
                    for (int t = 0; t < kNT; ++t) {
                        const uint8_t* xr = a.a + kb * xstep + (uint64_t)(r0 + min(t * 8 + gq, count - 1)) * kFp8Block + q * 16;
                        x[f][t][0] = *reinterpret_cast<const uint4*>(xr);
                        x[f][t][1] = *reinterpret_cast<const uint4*>(xr + 64);
                        // the instruction's columns are rows 2 q and 2 q + 1
                        const float* xs = a.sa + (uint64_t)kb * a.rows + r0;
                        s[f][t][0] = xs[min(t * 8 + 2 * q, count - 1)];
                        s[f][t][1] = xs[min(t * 8 + 2 * q + 1, count - 1)];
                    }
                }
#pragma unroll
                for (int f = 0; f < kFlight; ++f) {
                    if (kb0 + f * split >= a.KB) break;
#pragma unroll
                    for (int t = 0; t < kNT; ++t) {
                        const uint4 x0 = x[f][t][0], x1 = x[f][t][1];
                        float d[4] = {};
                        mma_16x8x32(d, w[f][0].x, w[f][2].x, w[f][0].y, w[f][2].y, x0.x, x0.y);
                        mma_16x8x32(d, w[f][0].z, w[f][2].z, w[f][0].w, w[f][2].w, x0.z, x0.w);
                        mma_16x8x32(d, w[f][1].x, w[f][3].x, w[f][1].y, w[f][3].y, x1.x, x1.y);
                        mma_16x8x32(d, w[f][1].z, w[f][3].z, w[f][1].w, w[f][3].w, x1.z, x1.w);
                        const float s0 = s[f][t][0] * sw[f], s1 = s[f][t][1] * sw[f];
                        acc[t][0] = fmaf(d[0], s0, acc[t][0]);
                        acc[t][1] = fmaf(d[1], s1, acc[t][1]);
                        acc[t][2] = fmaf(d[2], s0, acc[t][2]);
                        acc[t][3] = fmaf(d[3], s1, acc[t][3]);
                    }
                }
            }
        }
        if (split > 1) {
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) sums[warp][t * 4 + i][lane] = acc[t][i];
            __syncthreads();
            if (first == 0)
#pragma unroll
                for (int t = 0; t < kNT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        for (uint32_t w = 1; w < split; ++w) acc[t][i] += sums[warp + w][t * 4 + i][lane];
            __syncthreads();
        }
        if (first == 0)
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t r = t * 8 + 2 * q + (i & 1), n = n0 + gq + 8 * (i >> 1);
                    if (r < count && n < a.n) reinterpret_cast<T*>(a.out)[(uint64_t)(r0 + r) * a.n + n] = from_float<T>(acc[t][i]);
                }
    }
    // rows outside every group
    if (a.offsets != nullptr) {
        const int32_t t = ld_l2(a.offsets + a.G);
        const uint64_t tail = t < 0 ? 0u : min((uint32_t)t, a.rows), n = (uint64_t)a.rows * a.n;
        for (uint64_t i = tail * a.n + blockIdx.x * kThreads + threadIdx.x; i < n; i += (uint64_t)gridDim.x * kThreads)
            reinterpret_cast<T*>(a.out)[i] = from_float<T>(0.0f);
    }
}

template <typename T, int kNT>
cudaError_t small_as(const MatmulArgs& a, int sms, cudaStream_t stream)
{
    constexpr int kPerSm = kNT == 4 ? 2 : 3;
    // warps at work: at least 16 an SM, by splitting the reduction where the weight rows (of every group that can
    // have rows) do not give that many (twice as many measured slower: 12.9 us against 11.6 for one row through
    // 4096 x 14336, 29.1 against 28.3 for 264 rows through 64 experts).
    const uint64_t groups = a.rows < a.G ? a.rows : a.G, pieces = groups * ((a.n + kTileRows - 1) / kTileRows);
    uint32_t split = 1;
    while (split < kWarps && split < a.KB && pieces * split < (uint64_t)sms * 16) split *= 2;
    const uint32_t wide = kWarps / split * kTileRows;
    const uint64_t items = ((uint64_t)a.rows / (8 * kNT) + a.G) * ((a.n + wide - 1) / wide), most = (uint64_t)sms * kPerSm;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((uint32_t)(items < most ? items : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, small_kernel<T, kNT>, a, split);
}

// Rows a warp takes, in eights: the mean rows of a group, rounded up.
uint32_t row_tiles(uint64_t rows, uint32_t groups)
{
    const uint64_t mean = (rows + groups - 1) / groups;
    return mean <= 8 ? 1 : mean <= 16 ? 2 : 4;
}

template <typename T>
cudaError_t small_typed(const MatmulArgs& a, int sms, cudaStream_t stream)
{
    const uint32_t nt = row_tiles(a.rows, a.G);
    return nt == 1 ? small_as<T, 1>(a, sms, stream) : nt == 2 ? small_as<T, 2>(a, sms, stream) : small_as<T, 4>(a, sms, stream);
}

}  // namespace

// The two products by what a block of the reduction costs, in ps.  This one:
// 23, 38 or 54 a weight row and chunk of 8, 16 or 32 rows of x (the conversion
// of e4m3 operands bounds it), and some groups have a chunk more than the mean
// says.  The other: 0.55 us a round of its tiles (less in parts, and 5 us a call
// to join them), or 25 ps a weight row, the memory's time.  Measured, this one
// and the other, in us a call (n x k):
//   14336 x 4096, 1 group: 1 row 12.9, 25.5; 8 rows 13.4, 21.8; 32 rows 36.8, 21.3
//   4096 x 4096, 1 group: 1 row 7.1, 18.0; 32 rows 13.3, 16.1; 48 rows 22.5, 17.2
//   4096 x 4096, 8 groups: 8 rows 21.1, 29.1; 64 rows 34.1, 29.8; 256 rows 83.8, 30.4
//   1024 x 2048, 64 groups: 64 rows 19.8, 28.7; 256 rows 30.8, 31.4; 768 rows 45.7, 32.8
bool takes_small(uint64_t rows, uint64_t n, uint64_t k, uint32_t groups, int sms)
{
    if (rows > 32ull * groups) return false;
    const uint32_t nt = row_tiles(rows, groups);
    const uint64_t active = rows < groups ? rows : groups;
    const uint64_t chunks = groups == 1 ? (rows + 8 * nt - 1) / (8 * nt) : active + rows / 32;
    const uint64_t here = chunks * n * (nt == 1 ? 23 : nt == 2 ? 38 : 54);
    const uint64_t rounds = (active * ((n + 255) / 256) + sms - 1) / sms, by_bytes = active * n * 25;
    const uint32_t split = matmul_split(rows, n, k, groups);
    const uint64_t by_tiles = rounds * 550000 / split + (split > 1 ? 5000000 / blocks_of(k) : 0);
    return here <= (by_tiles > by_bytes ? by_tiles : by_bytes);
}

cudaError_t launch_small(const MatmulArgs& a, int sms, cudaStream_t stream)
{
    return a.out_f32 ? small_typed<float>(a, sms, stream) : small_typed<__nv_bfloat16>(a, sms, stream);
}

}  // namespace zccl
