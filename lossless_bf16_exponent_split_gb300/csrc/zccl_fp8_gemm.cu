// zccl_fp8_gemm.cu -- products of block-scaled e4m3 operands on the tensor
// cores, by groups of rows.
//
//   y[r][n]  = sum over blocks b of sa[b][r] sw[n / 128][b] (qa[b][r] . qw[b][n])
//   dw[m][n] = sum over a group's token blocks t of sa[t][m] sb[t][n] (qa[t][m] . qb[t][n])
//
// Persistent CTAs, one per SM, each 128 x 256 of an output at a time.  Warp 0
// fills a ring of operand stages by TMA; warp 1 issues the matrix instructions
// of a block of 128 (4 of 128 x 256 x 32) into one of two accumulators in
// tensor memory (one warp issues them all: a version with two warps taking turns
// faulted now and then in a CTA's first blocks); two warpgroups take each
// finished block out of tensor memory, scale it and add it to the sums in their
// registers: the scales change from block to block, so a sum cannot stay in
// tensor memory.  A block is 512 cycles of the tensor cores; issuing it takes
// 200, a commit 120 and the waits 100, so there is one commit, and the first
// warp that adds gives the stage back.  What bounds the kernel are the
// warpgroups: 128 columns a thread out of tensor memory and 128 multiply-adds a
// block are 300 issue cycles of a scheduler, and every wait that is not straight
// code adds to them, so a warp waits once a block (the scales arrive on the
// barrier of the block's products) and asks for the next block before it has
// added the last columns of this one.  Warp 3 brings the scales by asynchronous
// copies, blocks ahead.  A finished tile leaves through shared memory, so that
// a store covers whole sectors: stored from the registers, one row a thread, a
// tile took 6000 cycles.
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
constexpr uint32_t kScaleSlots = 6;
constexpr uint32_t kScaleLag = 4;      // a block's scales are reported this many blocks after their copies are issued
constexpr uint32_t kOutBytes = 64;     // bytes of a staged output row
constexpr uint32_t kOutPitch = kOutBytes + 16;  // 16 more, against bank conflicts
constexpr uint32_t kThreads = 384;     // warps 0..3: load, issue, idle, scales; 4..11: two warpgroups that add
constexpr uint32_t kTmemColumns = 2 * kTileN;
constexpr uint32_t kBandRows = 8;      // tiles of a band share their weight columns in L2
// registers: 384 threads x 168 at launch = 128 x 104 + 256 x 200; with another split, or
// wider pieces out of tensor memory, registers spill, and a spilled register's
// reload misses the little L1 that is left: it cost a block 1000 cycles
constexpr int kRegsFew = 104, kRegsMany = 200;

struct TileArgs {
    const float* sa;
    const float* sb;
    const int32_t* offsets;
    uint32_t rows, m, n, KB, G, blocks;
    void* out;
    uint32_t* status;
};

struct Smem {
    alignas(16) uint8_t out[8][32 * kOutPitch];        // by warp: 32 rows of a finished tile
    alignas(16) float row_scale[kScaleSlots][kTileM];
    alignas(16) float col_scale[kScaleSlots][kTileN];  // weight gradient: by column; else one per 128 columns
    uint64_t full[kStages], empty[kStages], done[2], taken[2], drain;
    uint32_t tmem;
    uint32_t prefix[kMaxGroupsFp8 + 1];
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

// Waits for a phase, a whole warp at once: the vote makes the result uniform,
// so that no lane can leave the others behind.  Reading the timer takes longer
// than a phase, so the timed wait comes after many untimed tries.  After a
// timeout the CTA's roles run out without waiting for one another.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, uint32_t* status)
{
#pragma unroll 1
    for (uint32_t i = 0; i < 1024; ++i)
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, phase))) return true;
    const uint64_t t0 = globaltimer();
#pragma unroll 1
    for (;;) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, phase))) return true;
        if (__any_sync(0xFFFFFFFFu, globaltimer() - t0 > kSpinTimeoutNs)) break;
    }
    report(status, ZCCL_ERR_TIMEOUT);
    return false;
}

// Waits for two phases: one vote and no taken branch where both are there.
__device__ __forceinline__ bool wait_both(uint64_t* bar0, uint32_t phase0, uint64_t* bar1, uint32_t phase1, uint32_t* status)
{
    const bool t0 = mbar_try_wait(bar0, phase0), t1 = mbar_try_wait(bar1, phase1);
    if (__builtin_expect(__all_sync(0xFFFFFFFFu, t0 && t1), 1)) return true;
    return wait_phase(bar0, phase0, status) && wait_phase(bar1, phase1, status);
}

// The sums of a warp's 32 rows x 128 columns (lane = row, columns acc[0..127])
// to the output rows at out, columns n..n_end, `rows` of them inside the
// output, through the warp's staging buffer.
template <typename T>
__device__ __forceinline__ void store_rows(uint8_t* buf, T* out, uint64_t pitch, uint32_t rows, uint32_t n, uint32_t n_end,
                                           const float (&acc)[128])
{
    constexpr uint32_t kCols = kOutBytes / sizeof(T);  // columns of a staged row
    constexpr uint32_t kPer = 16 / sizeof(T);    // columns of a store
    const uint32_t lane = threadIdx.x & 31;
    const bool vec = ((uintptr_t)out & 15) == 0 && (pitch * sizeof(T)) % 16 == 0;
#pragma unroll
    for (uint32_t h = 0; h < 128; h += kCols) {
#pragma unroll
        for (uint32_t i = 0; i < kCols; i += kPer) {
            const float* x = &acc[h + i];
            uint4 v;
            if (sizeof(T) == 2)
                v = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4 % kPer], x[5 % kPer]),
                               pack_bf16(x[6 % kPer], x[7 % kPer]));
            else
                v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            *reinterpret_cast<uint4*>(buf + lane * kOutPitch + i * sizeof(T)) = v;
        }
        __syncwarp();
        if (vec) {  // an end of the output within a store is impossible: its width is a multiple of kPer
            const uint32_t r0 = lane >> 2, c = (lane & 3) * kPer;
            T* to = out + r0 * pitch + n + h + c;
            const uint8_t* from = buf + r0 * kOutPitch + c * sizeof(T);
            const bool in = n + h + c < n_end;
#pragma unroll
            for (uint32_t r = 0; r < 32; r += 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(from + r * kOutPitch);
                if (in && r0 + r < rows) *reinterpret_cast<uint4*>(to + r * pitch) = v;
            }
        } else {  // a value at a time, consecutive lanes consecutive columns
#pragma unroll 1
            for (uint32_t i = lane; i < 32 * kCols; i += 32) {
                const uint32_t r = i / kCols, j = i % kCols;
                if (r < rows && n + h + j < n_end)
                    out[r * pitch + n + h + j] = *reinterpret_cast<const T*>(buf + r * kOutPitch + j * sizeof(T));
            }
        }
        __syncwarp();
    }
}

// Four bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy4_async(float* dst, const float* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// Lane 0 arrives, without a branch.
__device__ __forceinline__ void arrive_lane0(uint64_t* bar, uint32_t lane)
{
    asm volatile("{\n .reg .pred p;\n setp.eq.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(smem_addr(bar)),
                 "r"(lane)
                 : "memory");
}

template <bool kWgrad, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, TileArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* ring = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Smem* s = reinterpret_cast<Smem*>(ring + kStages * (kABytes + kBBytes));
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&s->done[i], 1 + 32);  // the products' commit, and the warp that brought the scales
            mbar_init(&s->taken[i], 8);
        }
        mbar_init(&s->drain, 1);
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
        if (warp == 0) {
            // ---- operand tiles into the ring
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
                for (uint32_t b = 0; b < c.blocks; ++b) {
                    if (!(ok = wait_phase(&s->empty[stage], phase ^ 1, a.status))) break;
                    if (lane == 0) {
                        uint8_t* at = ring + stage * (kABytes + kBBytes);
                        mbar_arrive_expect_tx(&s->full[stage], kABytes + kBBytes);
                        tma_load_2d(at, &map_a, 0, (int32_t)(c.a0 + b * c.a_step), &s->full[stage]);
                        tma_load_2d(at + kABytes, &map_b, 0, (int32_t)(c.b0 + b * c.b_step), &s->full[stage]);
                    }
                    __syncwarp();
                    if (++stage == kStages) stage = 0, phase ^= 1;
                }
            }
            // the CTA may end only once the ring is its own again: every stage read, and after a timeout at
            // least every load landed
            for (uint32_t i = 0; i < kStages; ++i) {
                if (ok) {
                    ok = wait_phase(&s->empty[stage], phase ^ 1, a.status);
                } else {
                    mbar_wait(&s->full[stage], phase ^ 1, kSpinTimeoutNs / 8);
                    __syncwarp();
                }
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        } else if (warp == 1) {
            // ---- matrix instructions
            uint32_t count = 0;
            bool ok = true;
            constexpr uint32_t idesc = instr_desc(kTileM, kTileN);
            for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const uint32_t end = count + tile_at<kWgrad>(a, s->prefix, tail0, t).blocks;
                for (; count < end; ++count) {
                    const uint32_t stage = count % kStages, buf = count & 1;
                    if (!(ok = wait_both(&s->taken[buf], ((count >> 1) & 1) ^ 1, &s->full[stage], (count / kStages) & 1,
                                         a.status)))
                        break;
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t at = smem_addr(ring) + stage * (kABytes + kBBytes);
                        const uint64_t da = smem_desc(at), db = smem_desc(at + kABytes);
#pragma unroll
                        for (uint32_t k = 0; k < kFp8Block / 32; ++k)
                            mma_e4m3(tmem + buf * kTileN, da + 2 * k, db + 2 * k, idesc, k > 0);
                        mma_commit(&s->done[buf]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // the accumulators are freed below: let the instructions issued so far end
                if (lane == 0) mma_commit(&s->drain);
                __syncwarp();
                mbar_wait(&s->drain, 0);
                __syncwarp();
            }
        } else if (warp == 3) {
            // ---- scales: 32 threads, four rows and (weight gradient) eight columns each.  A block's slot is free
            // once the block six before it was taken; its scales are reported four blocks later, when the block two
            // before it is done with the barrier.
            uint32_t count = 0, slot = 0;
            bool ok = true;
            for (uint32_t t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
                const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
                const uint32_t last = (kWgrad ? a.m : a.rows) - 1, nbs = (uint32_t)blocks_of(a.n);
                const float* row = a.sa + (kWgrad ? (uint64_t)s->prefix[c.g] * a.m : 0);
                const float* col = kWgrad ? a.sb + (uint64_t)s->prefix[c.g] * a.n
                                          : a.sb + ((uint64_t)c.g * nbs + min(c.n0 / kFp8Block + lane, nbs - 1)) * a.KB;
                for (uint32_t b = 0; b < c.blocks; ++b, ++count) {
                    if (count >= kScaleSlots) {
                        const uint32_t old = count - kScaleSlots;
                        if (!(ok = wait_phase(&s->taken[old & 1], (old >> 1) & 1, a.status))) break;
                    }
#pragma unroll
                    for (uint32_t j = lane; j < kTileM; j += 32) copy4_async(&s->row_scale[slot][j], row + min(c.m0 + j, last));
                    row += kWgrad ? a.m : a.rows;
                    if (kWgrad) {
#pragma unroll
                        for (uint32_t j = lane; j < kTileN; j += 32)
                            copy4_async(&s->col_scale[slot][j], col + min(c.n0 + j, a.n - 1));
                        col += a.n;
                    } else {
                        if (lane < kTileN / kFp8Block) copy4_async(&s->col_scale[slot][lane], col);
                        ++col;
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (++slot == kScaleSlots) slot = 0;
                    if (count >= kScaleLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kScaleLag) : "memory");
                        const uint32_t ready = count - kScaleLag;
                        if (ready >= 2 && !(ok = wait_phase(&s->done[ready & 1], ((ready >> 1) & 1) ^ 1, a.status))) break;
                        mbar_arrive(&s->done[ready & 1]);
                    }
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            for (uint32_t ready = count > kScaleLag ? count - kScaleLag : 0; ok && ready < count; ++ready) {
                if (ready >= 2 && !(ok = wait_phase(&s->done[ready & 1], ((ready >> 1) & 1) ^ 1, a.status))) break;
                mbar_arrive(&s->done[ready & 1]);
            }
        }
    } else {
        regs_more<kRegsMany>();
        // ---- sums: warpgroup wg has columns 128 wg .. 128 wg + 127, warp w of it lanes 32 w .. 32 w + 31
        const uint32_t wg = (warp - 4) >> 2, sub = warp & 3;
        const uint32_t taddr = tmem + ((sub * 32) << 16) + wg * 128;
        uint32_t count = 0, slot = 0;
        bool ok = true;      // after a timeout the loops run out without waiting
        bool there = false;  // whether the next block is known to be done
        for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
            const Tile c = tile_at<kWgrad>(a, s->prefix, tail0, t);
            float acc[128];
#pragma unroll
            for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
#pragma unroll 1
            for (uint32_t b = 0; b < c.blocks; ++b) {
                const uint32_t buf = count & 1;
                if (__builtin_expect(!there && ok, 0)) ok = wait_phase(&s->done[buf], (count >> 1) & 1, a.status);
                // the products are done, so their stage is free
                if (warp == 4) arrive_lane0(&s->empty[count % kStages], lane);
                ++count;
                __syncwarp();
                tc_fence_after();
                const uint32_t from = taddr + buf * kTileN;
                uint32_t r[2][16];
                tmem_load16(from, r[0]);
                float sa = s->row_scale[slot][sub * 32 + lane];
                if (!kWgrad) sa *= s->col_scale[slot][wg];
                bool next = false;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    tmem_wait16(r[q & 1]);
                    if (q < 7) tmem_load16(from + 16 * (q + 1), r[(q + 1) & 1]);
                    if (q == 6) next = mbar_try_wait(&s->done[count & 1], (count >> 1) & 1);
                    if (q == 7 && !kWgrad) {
                        tc_fence_before();
                        __syncwarp();
                        arrive_lane0(&s->taken[buf], lane);
                    }
                    if (kWgrad) {
                        const float4* col = reinterpret_cast<const float4*>(&s->col_scale[slot][wg * 128 + 16 * q]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = col[i];
                            // the scales first: their product overflows only where the sum does
                            const float x[4] = {f.x * sa, f.y * sa, f.z * sa, f.w * sa};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                acc[16 * q + 4 * i + j] =
                                    fmaf(__uint_as_float(r[q & 1][4 * i + j]), x[j], acc[16 * q + 4 * i + j]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[16 * q + i] = fmaf(__uint_as_float(r[q & 1][i]), sa, acc[16 * q + i]);
                    }
                }
                if (kWgrad) {  // the column scales are read to the end
                    tc_fence_before();
                    __syncwarp();
                    arrive_lane0(&s->taken[buf], lane);
                }
                there = __all_sync(0xFFFFFFFFu, next);
                if (++slot == kScaleSlots) slot = 0;
            }
            const uint32_t row = c.m0 + sub * 32, n = c.n0 + wg * 128;
            if (ok && row < c.row_end && n < a.n) {
                const uint64_t at = ((kWgrad ? (uint64_t)c.g * a.m : 0) + row) * a.n;
                store_rows(s->out[warp - 4], reinterpret_cast<T*>(a.out) + at, a.n, c.row_end - row, n, a.n, acc);
            }
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

template <bool kWgrad, typename T>
cudaError_t launch_tiles(const TileArgs& a, const uint8_t* qa, uint64_t rows_a, const uint8_t* qb, uint64_t rows_b,
                         uint64_t most_tiles, int sms, cudaStream_t stream)
{
    CUtensorMap map_a, map_b;
    if (!make_map(&map_a, qa, rows_a, kTileM) || !make_map(&map_b, qb, rows_b, kTileN)) return cudaErrorUnknown;
    const cudaError_t e =
        cudaFuncSetAttribute(gemm_kernel<kWgrad, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
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
    return cudaLaunchKernelEx(&cfg, gemm_kernel<kWgrad, T>, map_a, map_b, a);
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
    a.status = m.status;
    const uint64_t most = (blocks_of(m.rows) + m.G) * ((m.n + kTileN - 1) / kTileN);
    const auto launch = m.out_f32 ? launch_tiles<false, float> : launch_tiles<false, __nv_bfloat16>;
    return launch(a, m.a, (uint64_t)m.KB * m.rows, m.b, (uint64_t)m.G * m.KB * m.n, most, sms, stream);
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
    a.status = w.status;
    const uint64_t most = (uint64_t)w.G * ((w.m + kTileM - 1) / kTileM) * ((w.n + kTileN - 1) / kTileN);
    const auto launch = w.out_f32 ? launch_tiles<true, float> : launch_tiles<true, __nv_bfloat16>;
    return launch(a, w.a, (uint64_t)w.blocks * w.m, w.b, (uint64_t)w.blocks * w.n, most, sms, stream);
}

}  // namespace zccl
