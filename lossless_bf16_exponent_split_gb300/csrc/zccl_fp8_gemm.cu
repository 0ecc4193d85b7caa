// zccl_fp8_gemm.cu -- products of block-scaled e4m3 operands on the tensor
// cores, by groups of rows.
//
//   y[r][n]  = sum over blocks b of sa[b][r] sw[n / 128][b] (qa[b][r] . qw[b][n])
//   dw[m][n] = sum over a group's token blocks t of sa[t][m] sb[t][n] (qa[t][m] . qb[t][n])
//
// Persistent CTAs, one per SM, each 128 x 256 of an output at a time.  Warp 0
// fills a ring of operand stages by TMA, warp 1 issues the matrix instructions
// of a block of 128 (4 of 128 x 256 x 32) into one of two accumulators in
// tensor memory, and two warpgroups take each finished block out of tensor
// memory, scale it and add it to the sums in their registers: the scales change
// from block to block, so a sum cannot stay in tensor memory.  A block costs
// the tensor cores 512 cycles and each of the two warpgroups 128 x 128
// multiply-adds (half of them as packed pairs), so the additions hide behind
// the next block's products.
#include <atomic>
#include <cuda.h>

#include "zccl_fp8.cuh"
#include "zccl_tcgen05.cuh"

namespace zccl {

namespace {

constexpr uint32_t kTileM = 128;
constexpr uint32_t kTileN = 256;
constexpr uint32_t kStages = 4;
constexpr uint32_t kABytes = kTileM * kFp8Block, kBBytes = kTileN * kFp8Block;
constexpr uint32_t kThreads = 384;     // warps 0..3: load, issue, two idle; 4..11: two warpgroups that add
constexpr uint32_t kTmemColumns = 2 * kTileN;
constexpr uint32_t kBandRows = 8;      // tiles of a band share their weight columns in L2
// registers: 384 threads x 168 at launch = 128 x 40 + 256 x 232
constexpr int kRegsFew = 40, kRegsMany = 232;

struct TileArgs {
    const float* sa;
    const float* sb;
    const int32_t* offsets;
    uint32_t rows, m, n, KB, G, blocks;
    void* out;
    int out_f32;
    uint32_t* status;
};

struct Smem {
    uint64_t full[kStages], empty[kStages], done[2], taken[2], drain;
    uint32_t tmem, failed;
    uint32_t prefix[kMaxGroupsFp8 + 1];
    alignas(16) float col[2][2][128];  // weight gradient: column scales of a block, by warpgroup
};
constexpr uint32_t kSmemBytes = 1024 + kStages * (kABytes + kBBytes) + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "fits the shared memory of a CTA");

// One output tile.
struct Tile {
    uint32_t g, m0, n0;    // group, first row (of the output) and column
    uint32_t row_end;      // rows of the tile end here
    uint32_t blocks;       // blocks of the reduction
    uint32_t a0, a_step;   // operand rows: a0 + block * a_step
    uint32_t b0, b_step;
};

// kWgrad = false: tiles of group g are its blocks of 128 rows (prefix) by
// columns; the blocks after the last group's are the rows outside every group.
// kWgrad = true: every group has the same tiles; prefix counts token blocks.
template <bool kWgrad>
__device__ __forceinline__ uint32_t tile_count(const TileArgs& a, const uint32_t* prefix, uint32_t tail0)
{
    const uint32_t nt = (a.n + kTileN - 1) / kTileN;
    if (kWgrad) return a.G * ((a.m + kTileM - 1) / kTileM) * nt;
    return (prefix[a.G] + (a.rows - tail0 + kTileM - 1) / kTileM) * nt;
}

template <bool kWgrad>
__device__ __forceinline__ Tile tile_at(const TileArgs& a, const uint32_t* prefix, uint32_t tail0, uint32_t t)
{
    const uint32_t nt = (a.n + kTileN - 1) / kTileN;
    Tile c;
    uint32_t mt, i, lo = 0;
    if (kWgrad) {
        mt = (a.m + kTileM - 1) / kTileM;
        c.g = t / (mt * nt);
        i = t - c.g * mt * nt;
        c.blocks = prefix[c.g + 1] - prefix[c.g];
        c.row_end = a.m;
    } else {
        uint32_t mb = t / nt;
        if (mb < prefix[a.G]) {
            c.g = group_at(prefix, a.G, mb);
            mt = prefix[c.g + 1] - prefix[c.g];
            i = t - prefix[c.g] * nt;
            group_rows(a.offsets, a.rows, c.g, &lo, &c.row_end);
            c.blocks = a.KB;
        } else {  // rows outside every group: zeros
            c.g = 0;
            mt = (a.rows - tail0 + kTileM - 1) / kTileM;
            i = t - prefix[a.G] * nt;
            lo = tail0;
            c.row_end = a.rows;
            c.blocks = 0;
        }
    }
    // bands of 8 tile rows, column by column within a band
    const uint32_t band = i / (kBandRows * nt), in_band = i - band * kBandRows * nt;
    const uint32_t height = min(kBandRows, mt - band * kBandRows);
    const uint32_t col = in_band / height;
    c.m0 = lo + (band * kBandRows + in_band - col * height) * kTileM;
    c.n0 = col * kTileN;
    if (kWgrad) {
        c.a_step = a.m;
        c.b_step = a.n;
        c.a0 = prefix[c.g] * a.m + c.m0;
        c.b0 = prefix[c.g] * a.n + c.n0;
    } else {
        c.a_step = a.rows;
        c.b_step = a.n;
        c.a0 = c.m0;
        c.b0 = c.g * a.KB * a.n + c.n0;
    }
    return c;
}

// Waits for a phase; on timeout the CTA's roles all give up.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, Smem* s, uint32_t* status)
{
    if (mbar_try_wait(bar, phase)) return true;
    if (mbar_wait(bar, phase)) return true;
    *(volatile uint32_t*)&s->failed = 1;
    report(status, ZCCL_ERR_TIMEOUT);
    return false;
}

// 64 sums of a row's 128 columns from column n on (pairs acc[0..63]) to the output.
template <typename T>
__device__ __forceinline__ void store_row(T* row, uint32_t n, uint32_t n_end, const uint64_t (&acc)[64])
{
    constexpr uint32_t kVec = 16 / sizeof(T);
    const bool vec = ((uintptr_t)(row + n) & 15) == 0;
#pragma unroll
    for (uint32_t i = 0; i < 128; i += kVec) {
        if (vec && n + i + kVec <= n_end) {
            uint4 v;
            if (sizeof(T) == 2)
                v = make_uint4(pack_bf16(pair_lo(acc[i / 2]), pair_hi(acc[i / 2])),
                               pack_bf16(pair_lo(acc[i / 2 + 1]), pair_hi(acc[i / 2 + 1])),
                               pack_bf16(pair_lo(acc[i / 2 + 2 < 64 ? i / 2 + 2 : 63]), pair_hi(acc[i / 2 + 2 < 64 ? i / 2 + 2 : 63])),
                               pack_bf16(pair_lo(acc[i / 2 + 3 < 64 ? i / 2 + 3 : 63]), pair_hi(acc[i / 2 + 3 < 64 ? i / 2 + 3 : 63])));
            else
                v = make_uint4((uint32_t)acc[i / 2], (uint32_t)(acc[i / 2] >> 32), (uint32_t)acc[i / 2 + 1],
                               (uint32_t)(acc[i / 2 + 1] >> 32));
            *reinterpret_cast<uint4*>(row + n + i) = v;
        } else {
#pragma unroll
            for (uint32_t j = 0; j < kVec; ++j)
                if (n + i + j < n_end)
                    row[n + i + j] = from_float<T>((i + j) & 1 ? pair_hi(acc[(i + j) / 2]) : pair_lo(acc[(i + j) / 2]));
        }
    }
}

template <bool kWgrad>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, TileArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    Smem* s = reinterpret_cast<Smem*>(ring + kStages * (kABytes + kBBytes));
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&s->done[i], 1);
            mbar_init(&s->taken[i], 8);
        }
        mbar_init(&s->drain, 1);
        s->failed = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&s->tmem, kTmemColumns);
        tmem_release_permit();
    }
    pdl_wait();
    group_prefix(a.offsets, a.rows, a.G, kTileM, kWgrad ? a.blocks : 0x7FFFFFFFu, s->prefix);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s->tmem;
    uint32_t tail0 = a.rows;
    if (!kWgrad && a.offsets != nullptr) {
        const int32_t t = ld_l2(a.offsets + a.G);
        tail0 = t < 0 ? 0u : min((uint32_t)t, a.rows);
    }
    const uint32_t tiles = tile_count<kWgrad>(a, s->prefix, tail0);

    if (warp < 4) {
        regs_fewer<kRegsFew>();
        if (warp == 0 && lane == 0) {
            // ---- operand tiles into the ring
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
                for (uint32_t b = 0; b < c.blocks; ++b) {
                    if (!(ok = wait_phase(&s->empty[stage], phase ^ 1, s, a.status))) break;
                    uint8_t* at = ring + stage * (kABytes + kBBytes);
                    mbar_arrive_expect_tx(&s->full[stage], kABytes + kBBytes);
                    tma_load_2d(at, &map_a, 0, (int32_t)(c.a0 + b * c.a_step), &s->full[stage]);
                    tma_load_2d(at + kABytes, &map_b, 0, (int32_t)(c.b0 + b * c.b_step), &s->full[stage]);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
            }
            // the CTA may end only once the ring is its own again: every stage read, and after a timeout at
            // least every load landed
            for (uint32_t i = 0; i < kStages; ++i) {
                if (ok) {
                    ok = wait_phase(&s->empty[stage], phase ^ 1, s, a.status);
                } else {
                    mbar_wait(&s->full[stage], phase ^ 1, kSpinTimeoutNs / 8);
                }
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        } else if (warp == 1 && lane == 0) {
            // ---- matrix instructions
            uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
            bool ok = true;
            constexpr uint32_t idesc = instr_desc(kTileM, kTileN);
            for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
                for (uint32_t b = 0; b < c.blocks; ++b) {
                    if (!(ok = wait_phase(&s->taken[buf], buf_phase ^ 1, s, a.status))) break;
                    if (!(ok = wait_phase(&s->full[stage], phase, s, a.status))) break;
                    tc_fence_after();
                    const uint32_t at = smem_addr(ring + stage * (kABytes + kBBytes));
                    const uint64_t da = smem_desc(at), db = smem_desc(at + kABytes);
#pragma unroll
                    for (uint32_t k = 0; k < kFp8Block / 32; ++k)
                        mma_e4m3(tmem + buf * kTileN, da + 2 * k, db + 2 * k, idesc, k > 0);
                    mma_commit(&s->empty[stage]);
                    mma_commit(&s->done[buf]);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                    if (++buf == 2) buf = 0, buf_phase ^= 1;
                }
            }
            if (!ok) {  // the accumulators are freed below: let the instructions issued so far end
                mma_commit(&s->drain);
                mbar_wait(&s->drain, 0);
            }
        }
    } else {
        regs_more<kRegsMany>();
        // ---- sums: warpgroup wg has columns 128 wg .. 128 wg + 127, warp w of it lanes 32 w .. 32 w + 31
        const uint32_t wg = (warp - 4) >> 2, sub = warp & 3, tid = threadIdx.x & 127;
        const uint32_t taddr = tmem + ((sub * 32) << 16) + wg * 128;
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;
        for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
            const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
            const uint32_t row = c.m0 + sub * 32 + lane, n = c.n0 + wg * 128;
            const uint32_t safe_row = min(row, (kWgrad ? a.m : a.rows) - 1);
            const float* pa = a.sa + (kWgrad ? (uint64_t)s->prefix[c.g] * a.m : 0) + safe_row;
            const uint64_t pa_step = kWgrad ? a.m : a.rows;
            const float* pb;
            uint64_t pb_step;
            if (kWgrad) {  // a column's scale, one per thread, shared through smem
                pb = a.sb + (uint64_t)s->prefix[c.g] * a.n + min(n + tid, a.n - 1);
                pb_step = a.n;
            } else {
                const uint32_t nbs = (uint32_t)blocks_of(a.n);
                pb = a.sb + ((uint64_t)c.g * nbs + min(n / kFp8Block, nbs - 1)) * a.KB;
                pb_step = 1;
            }
            uint64_t acc[64];
#pragma unroll
            for (int i = 0; i < 64; ++i) acc[i] = 0;
            float next_a = 0.0f, next_b = 0.0f;
            if (c.blocks > 0) next_a = *pa, next_b = *pb;
            for (uint32_t b = 0; b < c.blocks; ++b) {
                const float sa = kWgrad ? next_a : next_a * next_b;
                if (kWgrad) {
                    s->col[wg][b & 1][tid] = next_b;
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory");
                }
                if (b + 1 < c.blocks) next_a = pa[(b + 1) * pa_step], next_b = pb[(b + 1) * pb_step];
                // after a timeout the loops run out without waiting, so that the warpgroup's barriers stay in step
                if (ok) ok = wait_phase(&s->done[buf], buf_phase, s, a.status);
                tc_fence_after();
                const uint64_t sa2 = pair(__float_as_uint(sa), __float_as_uint(sa));
                const uint32_t from = taddr + buf * kTileN;
                uint32_t r[2][32];
                tmem_load32(from, r[0]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_wait32(r[q & 1]);
                    if (q < 3) tmem_load32(from + 32 * (q + 1), r[(q + 1) & 1]);
                    if (q == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&s->taken[buf]);
                    }
                    if (kWgrad) {
                        const float4* col = reinterpret_cast<const float4*>(&s->col[wg][b & 1][32 * q]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = col[i];
                            const uint64_t f0 = pair(__float_as_uint(f.x), __float_as_uint(f.y));
                            const uint64_t f1 = pair(__float_as_uint(f.z), __float_as_uint(f.w));
                            // the scales first: their product overflows only where the sum does
                            acc[16 * q + 2 * i] = fma_pair(pair(r[q & 1][4 * i], r[q & 1][4 * i + 1]), mul_pair(f0, sa2),
                                                           acc[16 * q + 2 * i]);
                            acc[16 * q + 2 * i + 1] = fma_pair(pair(r[q & 1][4 * i + 2], r[q & 1][4 * i + 3]),
                                                               mul_pair(f1, sa2), acc[16 * q + 2 * i + 1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            acc[16 * q + i] = fma_pair(pair(r[q & 1][2 * i], r[q & 1][2 * i + 1]), sa2, acc[16 * q + i]);
                    }
                }
                if (++buf == 2) buf = 0, buf_phase ^= 1;
            }
            if (ok && row < c.row_end && n < a.n) {
                const uint64_t at = ((kWgrad ? (uint64_t)c.g * a.m : 0) + row) * a.n;
                if (a.out_f32)
                    store_row<float>(reinterpret_cast<float*>(a.out) + at, n, a.n, acc);
                else
                    store_row<__nv_bfloat16>(reinterpret_cast<__nv_bfloat16*>(a.out) + at, n, a.n, acc);
            }
            __syncwarp();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_free(tmem, kTmemColumns);
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeTiled encoder()
{
    static std::atomic<void*> known{nullptr};
    void* f = known.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        known.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// Rows of 128 codes; a box is `box` of them, swizzled.  Boxes that reach past
// the last row read zeros there.
bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box)
{
    const EncodeTiled encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {kFp8Block, rows};
    const cuuint64_t strides[1] = {kFp8Block};
    const cuuint32_t boxes[2] = {kFp8Block, box};
    const cuuint32_t steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kWgrad>
cudaError_t launch_tiles(const TileArgs& a, const uint8_t* qa, uint64_t rows_a, const uint8_t* qb, uint64_t rows_b,
                         uint64_t most_tiles, int sms, cudaStream_t stream)
{
    CUtensorMap map_a, map_b;
    if (!make_map(&map_a, qa, rows_a, kTileM) || !make_map(&map_b, qb, rows_b, kTileN)) return cudaErrorUnknown;
    const cudaError_t e =
        cudaFuncSetAttribute(gemm_kernel<kWgrad>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((uint32_t)(most_tiles < (uint64_t)sms ? most_tiles : (uint64_t)sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gemm_kernel<kWgrad>, map_a, map_b, a);
}

}  // namespace

cudaError_t launch_matmul(const MatmulArgs& m, int sms, cudaStream_t stream)
{
    TileArgs a{};
    a.sa = m.sa;
    a.sb = m.sb;
    a.offsets = m.offsets;
    a.rows = m.rows;
    a.m = m.rows;
    a.n = m.n;
    a.KB = m.KB;
    a.G = m.G;
    a.out = m.out;
    a.out_f32 = m.out_f32;
    a.status = m.status;
    const uint64_t most = (blocks_of(m.rows) + m.G) * ((m.n + kTileN - 1) / kTileN);
    return launch_tiles<false>(a, m.a, (uint64_t)m.KB * m.rows, m.b, (uint64_t)m.G * m.KB * m.n, most, sms, stream);
}

cudaError_t launch_wgrad(const WgradArgs& w, int sms, cudaStream_t stream)
{
    TileArgs a{};
    a.sa = w.sa;
    a.sb = w.sb;
    a.offsets = w.offsets;
    a.rows = w.rows;
    a.m = w.m;
    a.n = w.n;
    a.G = w.G;
    a.blocks = w.blocks;
    a.out = w.out;
    a.out_f32 = w.out_f32;
    a.status = w.status;
    const uint64_t most = (uint64_t)w.G * ((w.m + kTileM - 1) / kTileM) * ((w.n + kTileN - 1) / kTileN);
    return launch_tiles<true>(a, w.a, (uint64_t)w.blocks * w.m, w.b, (uint64_t)w.blocks * w.n, most, sms, stream);
}

}  // namespace zccl
