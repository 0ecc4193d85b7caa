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
// faulted now and then in a CTA's first blocks); warp 2 draws the tiles by
// ticket; warp 3 brings the scales by asynchronous copies, two blocks ahead.  Two
// warpgroups take each finished block out of tensor memory, scale it and add it
// to the sums in their registers: the scales change from block to block, so a sum
// cannot stay in tensor memory.
//
// A block is 512 cycles of the tensor cores; it takes 890 to 940 here.  The two
// sides of it, in cycles, 112 blocks a tile, in a build that reads the clock: with
// the additions left out and the accumulator given back at once 924, with three
// quarters of the weight operand's loads left out 911, with both 772, as it is
// 937.  So the adding warps and the way of the operands (48 KB a block) are about
// equally long, and neither alone is the bound: an adding warp finds the next
// block done when it asks, before the last columns of this one, in 24 to 30 % of
// the blocks.  In the weight gradient it does in 72 %: a column's scale is its own
// there, a packed multiplication and a packed multiply-add a column pair (512
// issue cycles a block with two warps a scheduler), and the accumulator goes back
// after all of them, so the adding warps are the bound.  Their block: 128 columns
// a thread come out of tensor memory in pieces of 32, each waited for alone (a
// wait is for all of a warp's loads), with the additions of the piece before under
// it.  What was measured on the way: packed additions leave the issue slots that
// the issuing warp needs (with single ones a block took 1800 cycles); a warp waits
// once a block, on one barrier that the products and the scales share; 16 adding
// warps of 64 columns take 1010 to 1090 cycles, pieces of 64 columns 2 % more than
// of 32.  Between a tile's last additions and the next tile's first are 2000 to
// 3400 cycles, 1100 to 1700 of them storing through shared memory and by TMA
// (stored from the registers, one row a thread, 6000).
//
// 4096 x 4096 x 14336 (m, n, k) 204 us, 2.36 PFLOP/s; 131072 rows through 64 experts
// of 1024 x 2048 234 us, 2.35; the weight gradient of 4096 rows by 14336 x 4096
// 245 us, 1.96.
#include <atomic>
#include <cuda.h>

#include "zccl_fp8.cuh"
#include "zccl_tcgen05.cuh"

namespace zccl {

namespace {

constexpr uint32_t kTileM = 128;
constexpr uint32_t kTileN = 256;
constexpr uint32_t kStages = 3;
constexpr uint32_t kABytes = kTileM * kFp8Block, kBBytes = kTileN * kFp8Block;
constexpr uint32_t kScaleSlots = 4;
constexpr uint32_t kScaleLag = 2;      // a block's scales are reported this many blocks after their copies are issued
constexpr uint32_t kSumWarps = 8;      // warps that add, two to 32 rows of a tile
constexpr uint32_t kSumCols = 128;     // columns of one of them
constexpr uint32_t kThreads = 128 + 32 * kSumWarps;  // warps 0..3: load, issue, schedule, scales; then those that add
constexpr uint32_t kTmemColumns = 2 * kTileN;
constexpr uint32_t kBandRows = 8;      // tiles of a band share their weight columns in L2
// registers: 384 threads x 168 at launch = 128 x 56 + 256 x 224
constexpr int kRegsFew = 56, kRegsMany = 224;

struct TileArgs {
    const float* sa;
    const float* sb;
    const int32_t* offsets;
    uint32_t rows, m, n, KB, G, blocks;
    void* out;
    int tma_out;           // whether the output has a tensor map
    uint32_t* ticket;      // tiles given out so far
    uint32_t split;        // parts of a tile's reduction
    uint32_t* counters;    // by tile and adding warp: parts that are done
    float* parts;          // by tile, part and adding warp: its sums, by column and lane
    uint32_t* status;
};

// One output tile, as the scheduling warp hands it to the others.
struct alignas(16) Tile {
    uint32_t m0, n0;       // first row (of the output, within its group for a weight gradient) and column
    uint32_t row_end;      // rows of the tile end here
    uint32_t blocks;       // blocks of the reduction; kNoTile: there are no more tiles
    uint32_t a0, b0;       // first operand rows
    uint32_t sa0, sb0;     // first scales
    uint32_t g;            // group
    uint32_t join;         // tile, of those that are cut into parts
    uint32_t part, pad;
};
constexpr uint32_t kNoTile = 0xFFFFFFFFu;
constexpr uint32_t kTileSlots = 4;
constexpr uint32_t kTileReaders = 3 + kSumWarps;  // warps that read a tile

struct Smem {
    alignas(1024) uint8_t out[kSumWarps][2][32 * 128];  // by warp, twice: 32 rows of 128 bytes of a finished tile, swizzled
    alignas(16) float row_scale[kScaleSlots][kTileM];
    alignas(16) float col_scale[kScaleSlots][kTileN];  // weight gradient: by column; else one per 128 columns
    Tile tile[kTileSlots];
    uint64_t full[kStages], empty[kStages], told[kTileSlots], read[kTileSlots], done[2], drain;
    uint32_t tmem;
    uint32_t prefix[kMaxGroupsFp8 + 1];
    uint16_t order[kMaxGroupsFp8];  // weight gradient: the groups by their blocks, most first
};
constexpr uint32_t kSmemBytes = 1024 + kStages * (kABytes + kBBytes) + sizeof(Smem);
static_assert(kSmemBytes <= 232448, "fits the shared memory of a CTA");

// kWgrad = false: tiles of group g are its blocks of 128 rows (prefix) by
// columns; the blocks after the last group's are the rows outside every group.
// kWgrad = true: every group has the same tiles; prefix counts token blocks.
template <bool kWgrad>
__device__ __forceinline__ uint32_t tile_count(const TileArgs& a, const uint32_t* prefix, uint32_t tail0, uint32_t split)
{
    const uint32_t nt = (a.n + kTileN - 1) / kTileN;
    if (kWgrad) return a.G * ((a.m + kTileM - 1) / kTileM) * nt * split;
    return (prefix[a.G] * split + (a.rows - tail0 + kTileM - 1) / kTileM) * nt;
}

template <bool kWgrad>
__device__ __forceinline__ Tile tile_at(const TileArgs& a, const uint32_t* prefix, const uint16_t* order, uint32_t tail0,
                                        uint32_t split, uint32_t t)
{
    const uint32_t nt = (a.n + kTileN - 1) / kTileN;
    Tile c;
    uint32_t mt, i, lo = 0, kb0 = 0;
    if (kWgrad) {
        mt = (a.m + kTileM - 1) / kTileM;
        c.join = t / split;
        c.part = t - c.join * split;
        c.g = c.join / (mt * nt);
        i = c.join - c.g * mt * nt;
        c.g = order[c.g];
        const uint32_t blocks = prefix[c.g + 1] - prefix[c.g];
        kb0 = c.part * blocks / split;
        c.blocks = (c.part + 1) * blocks / split - kb0;
        c.row_end = a.m;
    } else {
        const uint32_t whole = t / split, mb = whole / nt;
        if (mb < prefix[a.G]) {
            c.join = whole;
            c.part = t - whole * split;
            kb0 = c.part * a.KB / split;
            t = whole;
            c.g = group_at(prefix, a.G, mb);
            mt = prefix[c.g + 1] - prefix[c.g];
            i = t - prefix[c.g] * nt;
            group_rows(a.offsets, a.rows, c.g, &lo, &c.row_end);
            c.blocks = (c.part + 1) * a.KB / split - kb0;
        } else {  // rows outside every group: zeros
            c.g = 0;
            mt = (a.rows - tail0 + kTileM - 1) / kTileM;
            i = t - prefix[a.G] * split * nt;
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
        c.sa0 = (prefix[c.g] + kb0) * a.m;
        c.sb0 = (prefix[c.g] + kb0) * a.n;
        c.a0 = c.sa0 + c.m0;
        c.b0 = c.sb0 + c.n0;
    } else {
        c.sa0 = kb0 * a.rows;
        c.sb0 = c.g * (uint32_t)blocks_of(a.n) * a.KB + kb0;
        c.a0 = c.sa0 + c.m0;
        c.b0 = (c.g * a.KB + kb0) * a.n + c.n0;
    }
    return c;
}

// Waits for a phase, a whole warp at once: the vote makes the result uniform,
// so that no lane can leave the others behind.  The clock is read every 256
// tries only, and the loop is short: the waits are inlined in many places, and
// the kernel's code has to stay in the instruction cache.  After a timeout the
// CTA's roles run out without waiting for one another.
constexpr int64_t kWaitCycles = 2000000000;  // about a second

__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t phase, uint32_t* status)
{
    const int64_t t0 = clock64();
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, phase))) return true;
        if ((i & 255) == 255 && __any_sync(0xFFFFFFFFu, clock64() - t0 > kWaitCycles)) break;
    }
    report(status, ZCCL_ERR_TIMEOUT);
    return false;
}

// The sums of a warp's 32 rows x 128 columns (lane = row) to the output, from
// row `row` (of `rows` inside the output, counted from there) and column n on,
// through the warp's two staging buffers, two pieces of 128 bytes a row at a time
// (one fence for both): rows of 128 bytes whose 16-byte pieces are XOR-swizzled
// with the row.  A whole box goes by one asynchronous TMA store that runs beside
// the next tile (all CTAs end their tiles together: stored by the threads, a
// tile's 64 KB took 4000 cycles); cut rows go by the threads.
template <typename T>
__device__ __forceinline__ void store_rows(uint8_t (&bufs)[2][32 * 128], const CUtensorMap* map, int tma, T* out,
                                           uint64_t row, uint32_t rows, uint32_t n, uint32_t n_end,
                                           const float (&acc)[kSumCols])
{
    constexpr uint32_t kCols = 128 / sizeof(T);  // columns of a staged row
    constexpr uint32_t kPer = 16 / sizeof(T);    // columns of a piece
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (uint32_t h0 = 0; h0 < kSumCols; h0 += 2 * kCols) {
        if (n + h0 >= n_end) break;
        const bool two = n + h0 + kCols < n_end;
        if (lane == 0) bulk_wait_read0();  // the buffers' last stores
        __syncwarp();
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) {
            if (t == 1 && !two) break;
#pragma unroll
            for (uint32_t p = 0; p < 8; ++p) {
                const float* x = &acc[h0 + t * kCols + p * kPer];
                uint4 v;
                if (sizeof(T) == 2)
                    v = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4 % kPer], x[5 % kPer]),
                                   pack_bf16(x[6 % kPer], x[7 % kPer]));
                else
                    v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
                *reinterpret_cast<uint4*>(bufs[t] + lane * 128 + ((p ^ (lane & 7)) * 16)) = v;
            }
        }
        if (tma && rows >= 32) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(map, bufs[0], (int32_t)(n + h0), (int32_t)row);
                if (two) tma_store_2d(map, bufs[1], (int32_t)(n + h0 + kCols), (int32_t)row);
                bulk_commit();
            }
            continue;
        }
        __syncwarp();
#pragma unroll 1
        for (uint32_t t = 0; t < (two ? 2 : 1); ++t) {
            const uint32_t h = h0 + t * kCols;
            const uint8_t* buf = bufs[t];
            if (tma) {  // cut rows, in whole pieces: the output's width is a multiple of a piece's
                const uint32_t p = lane & 7;
                T* to = out + (row + (lane >> 3)) * n_end + n + h + p * kPer;
#pragma unroll 1
                for (uint32_t r = lane >> 3; r < 32; r += 4, to += 4 * (uint64_t)n_end)
                    if (r < rows && n + h + p * kPer < n_end)
                        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(buf + r * 128 + ((p ^ (r & 7)) * 16));
            } else {  // a value at a time, consecutive lanes consecutive columns
                const uint32_t cols = min(kCols, n_end - n - h);
                T* to = out + row * n_end + n + h;
#pragma unroll 4
                for (uint32_t i = lane; i < 32 * kCols; i += 32) {
                    const uint32_t r = i / kCols, j = i % kCols;
                    if (r < rows && j < cols)
                        to[(uint64_t)r * n_end + j] =
                            reinterpret_cast<const T*>(buf + r * 128 + (((j / kPer) ^ (r & 7)) * 16))[j % kPer];
                }
            }
        }
    }
}

// The end of a part of a tile: the warp's sums go to memory; the last warp to
// come, by the counter, takes those of all parts, added in the parts' order, and
// returns true.
__device__ __forceinline__ bool join_parts(const TileArgs& a, const Tile& c, uint32_t split, uint32_t warp, uint32_t lane,
                                           float (&acc)[kSumCols])
{
    constexpr uint32_t kPart = kSumCols * 32;
    float* at = a.parts + ((uint64_t)c.join * split * kSumWarps + warp) * kPart + lane;
#pragma unroll
    for (uint32_t i = 0; i < kSumCols; ++i) __stcg(at + (uint64_t)c.part * kSumWarps * kPart + i * 32, acc[i]);
    __syncwarp();
    uint32_t before = 0;
    if (lane == 0) before = atom_inc_acq_rel(a.counters + c.join * kSumWarps + warp, split - 1);
    if (__shfl_sync(0xFFFFFFFFu, before, 0) != split - 1) return false;
    __syncwarp();
#pragma unroll
    for (uint32_t i = 0; i < kSumCols; ++i) acc[i] = __ldcg(at + i * 32);
#pragma unroll 1
    for (uint32_t p = 1; p < split; ++p) {
        at += kSumWarps * kPart;
#pragma unroll
        for (uint32_t i = 0; i < kSumCols; ++i) acc[i] += __ldcg(at + i * 32);
    }
    return true;
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ float lds_f32(uint32_t a)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}

// Four bytes to shared memory, asynchronously.
__device__ __forceinline__ void copy4_async(float* dst, const float* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// Lane 0 arrives, without a branch.
__device__ __forceinline__ void arrive_lane0(uint32_t bar, uint32_t lane)
{
    asm volatile("{\n .reg .pred p;\n setp.eq.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(bar),
                 "r"(lane)
                 : "memory");
}

// The next tile, copied out of its slot by a whole warp; false at the end (or
// after a timeout).
__device__ __forceinline__ bool next_tile(Smem* s, uint32_t* k, Tile* c, uint32_t lane, uint32_t* status)
{
    const uint32_t slot = *k % kTileSlots;
    if (!wait_phase(&s->told[slot], (*k / kTileSlots) & 1, status)) return false;
    *c = s->tile[slot];
    __syncwarp();
    arrive_lane0(smem_addr(&s->read[slot]), lane);
    ++*k;
    return c->blocks != kNoTile;
}

template <bool kWgrad, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_out, TileArgs a)
{
    extern __shared__ uint8_t raw[];
    uint8_t* ring = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
    Smem* s = reinterpret_cast<Smem*>(ring + kStages * (kABytes + kBBytes));
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(&s->full[i], 1 + kSumWarps);  // the operands, and the accumulator's release
            mbar_init(&s->empty[i], 1);
        }
        for (uint32_t i = 0; i < kTileSlots; ++i) {
            mbar_init(&s->told[i], 1);
            mbar_init(&s->read[i], kTileReaders);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(&s->done[i], 1 + 32);  // the products' commit, and the warp that brought the scales
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
    if (kWgrad) {
        for (uint32_t g = threadIdx.x; g < a.G; g += kThreads) {
            const uint32_t mine = s->prefix[g + 1] - s->prefix[g];
            uint32_t before = 0;
            for (uint32_t h = 0; h < a.G; ++h) {
                const uint32_t other = s->prefix[h + 1] - s->prefix[h];
                before += other > mine || (other == mine && h < g) ? 1u : 0u;
            }
            s->order[before] = (uint16_t)g;
        }
        __syncthreads();
    }
    const uint32_t tmem = s->tmem;
    // there is room for kJoinParts; what the host reckoned with may be less than the groups' blocks
    const uint32_t row_tiles = kWgrad ? a.G * ((a.m + kTileM - 1) / kTileM) : s->prefix[a.G];
    const uint32_t split = row_tiles * ((a.n + kTileN - 1) / kTileN) * a.split > kJoinParts ? 1 : a.split;

    if (warp < 4) {
        regs_fewer<kRegsFew>();
        Tile c;
        uint32_t k = 0;
        bool ok = true;
        if (warp == 0) {
            // ---- operand tiles into the ring
            const uint32_t a_step = kWgrad ? a.m : a.rows, b_step = a.n;
            uint32_t stage = 0, phase = 0;
            while (ok && next_tile(s, &k, &c, lane, a.status)) {
                for (uint32_t b = 0; b < c.blocks; ++b) {
                    if (!(ok = wait_phase(&s->empty[stage], phase ^ 1, a.status))) break;
                    if (lane == 0) {
                        uint8_t* at = ring + stage * (kABytes + kBBytes);
                        mbar_arrive_expect_tx(&s->full[stage], kABytes + kBBytes);
                        tma_load_2d(at, &map_a, 0, (int32_t)(c.a0 + b * a_step), &s->full[stage]);
                        tma_load_2d(at + kABytes, &map_b, 0, (int32_t)(c.b0 + b * b_step), &s->full[stage]);
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
            // ---- matrix instructions.  What the warp does between two blocks has to fit beside those it has
            // queued, so it waits on one barrier: a block's operands and its accumulator's release arrive together
            constexpr uint32_t idesc = instr_desc(kTileM, kTileN);
            const uint64_t desc0 = smem_desc(smem_addr(ring));
            uint32_t stage = 0, phase = 0, buf = 0;
            while (ok && next_tile(s, &k, &c, lane, a.status)) {
                const uint32_t blocks = __shfl_sync(0xFFFFFFFFu, c.blocks, 0);
#pragma unroll 1
                for (uint32_t b = 0; b < blocks; ++b) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(&s->full[stage], phase)) &&
                        !(ok = wait_phase(&s->full[stage], phase, a.status)))
                        break;
                    tc_fence_after();
                    const uint64_t da = desc0 + stage * ((kABytes + kBBytes) >> 4);
                    mma_block_e4m3(tmem + buf * kTileN, da, da + (kABytes >> 4), idesc, &s->done[buf], &s->empty[stage]);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                    buf ^= 1;
                }
            }
            if (!ok) {  // the accumulators are freed below: let the instructions issued so far end
                mma_commit(&s->drain);
                mbar_wait(&s->drain, 0);
                __syncwarp();
            }
        } else if (warp == 2) {
            // ---- the tiles, by ticket: a CTA that is done early takes more of them, and a weight gradient's
            // longest tiles go first.  A ticket is drawn while the tile before it waits for its slot.
            uint32_t tail0 = a.rows;
            if (!kWgrad && a.offsets != nullptr) {
                const int32_t t = ld_l2(a.offsets + a.G);
                tail0 = t < 0 ? 0u : min((uint32_t)t, a.rows);
            }
            const uint32_t tiles = tile_count<kWgrad>(a, s->prefix, tail0, split);
            uint32_t t = lane == 0 ? atomicAdd(a.ticket, 1u) : 0u;
            for (;; ++k) {
                const uint32_t slot = k % kTileSlots, now = __shfl_sync(0xFFFFFFFFu, t, 0);
                if (now < tiles) {
                    if (lane == 0) t = atomicAdd(a.ticket, 1u);
                    c = tile_at<kWgrad>(a, s->prefix, s->order, tail0, split, now);
                } else {
                    c.blocks = kNoTile;
                }
                if (!wait_phase(&s->read[slot], ((k / kTileSlots) & 1) ^ 1, a.status)) break;
                if (lane == 0) s->tile[slot] = c;
                __syncwarp();
                arrive_lane0(smem_addr(&s->told[slot]), lane);
                if (now >= tiles) break;
            }
        } else {
            // ---- scales: 32 threads, four rows and (weight gradient) eight columns each.  A block's slot is free
            // once the block four before it was taken, which the barrier of the block two before it says; that block's
            // own scales, which have landed by then, are reported first.  A tile without blocks reports what is left:
            // the sums of a tile before it must not wait for blocks that are more tiles away than there are slots
            const uint32_t last = (kWgrad ? a.m : a.rows) - 1, nbs = (uint32_t)blocks_of(a.n);
            uint32_t count = 0, told = 0, stage = 0, phase = 0;  // blocks asked for, and reported
            auto report_next = [&] {
                if (!wait_phase(&s->full[stage], phase, a.status)) return false;
                mbar_arrive(&s->done[told & 1]);
                ++told;
                if (++stage == kStages) stage = 0, phase ^= 1;
                return true;
            };
            auto report_all = [&] {
                asm volatile("cp.async.wait_all;" ::: "memory");
                while (ok && told < count) ok = report_next();
            };
            while (ok && next_tile(s, &k, &c, lane, a.status)) {
                if (c.blocks == 0) report_all();
                const float* row = a.sa + c.sa0;
                const float* col = a.sb + c.sb0 + (kWgrad ? 0 : min(c.n0 / kFp8Block + lane, nbs - 1) * a.KB);
#pragma unroll 1
                for (uint32_t b = 0; b < c.blocks; ++b, ++count) {
                    const uint32_t slot = count % kScaleSlots;
                    if (count - told >= kScaleLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(kScaleLag - 1) : "memory");
                        if (!(ok = report_next())) break;
                    }
#pragma unroll
                    for (uint32_t j = 0; j < kTileM; j += 32)
                        copy4_async(&s->row_scale[slot][lane + j], row + min(c.m0 + lane + j, last));
                    row += kWgrad ? a.m : a.rows;
                    if (kWgrad) {
#pragma unroll
                        for (uint32_t j = 0; j < kTileN; j += 32)
                            copy4_async(&s->col_scale[slot][lane + j], col + min(c.n0 + lane + j, a.n - 1));
                        col += a.n;
                    } else {
                        if (lane < kTileN / kFp8Block) copy4_async(&s->col_scale[slot][lane], col);
                        ++col;
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                }
            }
            report_all();
        }
    } else {
        regs_more<kRegsMany>();
        // ---- sums: warpgroup wg has columns 128 wg .. 128 wg + 127, warp w of it lanes 32 w .. 32 w + 31
        const uint32_t wg = (warp - 4) >> 2, sub = warp & 3;
        const uint32_t taddr = tmem + ((sub * 32) << 16) + wg * kSumCols;
        const uint32_t done = smem_addr(&s->done[0]);
        // where its scales are, and the barriers of the next blocks in turn
        const uint32_t rows_at = smem_addr(&s->row_scale[0][sub * 32 + lane]), block_at = smem_addr(&s->col_scale[0][wg]);
        // a row's scale, times that of its 128 columns if they have one
        auto scale_of = [&](uint32_t block) {
            const uint32_t slot = block % kScaleSlots;
            const float r = lds_f32(rows_at + slot * (kTileM * 4));
            return kWgrad ? r : r * lds_f32(block_at + slot * (kTileN * 4));
        };
        uint32_t free0 = smem_addr(&s->full[2 % kStages]), free1 = smem_addr(&s->full[3 % kStages]),
                 free2 = smem_addr(&s->full[4 % kStages]);
        static_assert(kStages == 3, "three barriers take turns");
        uint32_t k = 0, count = 0;
        bool ok = true;
        Tile c;
        arrive_lane0(smem_addr(&s->full[0]), lane);  // both accumulators are free for the first two blocks
        arrive_lane0(smem_addr(&s->full[1]), lane);
        uint32_t r[2][32];   // pieces of 32 columns, one on its way while the other is added
        bool there = false;  // whether the next block is known to be done and its first piece is on its way
        float sa = 0.0f;
        while (ok && next_tile(s, &k, &c, lane, a.status)) {
            float acc[kSumCols];
#pragma unroll
            for (uint32_t i = 0; i < kSumCols; ++i) acc[i] = 0.0f;
#pragma unroll 1
            for (uint32_t b = 0; b < c.blocks; ++b) {
                const uint32_t from = taddr + (count & 1) * kTileN;
                if (!there) {
                    if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(&s->done[count & 1], (count >> 1) & 1)) &&
                        !(ok = wait_phase(&s->done[count & 1], (count >> 1) & 1, a.status)))
                        break;
                    tc_fence_after();
                    tmem_load32(from, r[0]);
                    sa = scale_of(count);
                }
                const uint32_t slot = count % kScaleSlots;
                const float now = sa;
                ++count;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    tmem_wait32(r[q & 1]);
                    if (q < 3) tmem_load32(from + 32 * (q + 1), r[(q + 1) & 1]);
                    if (q == 3) {
                        if (!kWgrad) {
                            tc_fence_before();
                            __syncwarp();
                            arrive_lane0(free0, lane);
                        }
                        // the next block (of whatever tile), if it is done, before the last columns of this one
                        there = __all_sync(0xFFFFFFFFu, mbar_test_wait(done + 8 * (count & 1), (count >> 1) & 1));
                        if (there) {
                            tc_fence_after();
                            tmem_load32(taddr + (count & 1) * kTileN, r[0]);
                            sa = scale_of(count);
                        }
                    }
                    if (kWgrad) {
                        const float4* col = reinterpret_cast<const float4*>(&s->col_scale[slot][wg * kSumCols + 32 * q]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 f = col[i];
                            // the scales first, as the definition has it: their product is finite for blocks whose
                            // largest magnitudes' product is below 2^145
                            const float2 x0 = mul2(f.x, f.y, now), x1 = mul2(f.z, f.w, now);
                            float* to = &acc[32 * q + 4 * i];
                            const uint32_t* from_r = &r[q & 1][4 * i];
                            fma2(to[0], to[1], __uint_as_float(from_r[0]), __uint_as_float(from_r[1]), x0.x, x0.y);
                            fma2(to[2], to[3], __uint_as_float(from_r[2]), __uint_as_float(from_r[3]), x1.x, x1.y);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            fma2(acc[32 * q + i], acc[32 * q + i + 1], __uint_as_float(r[q & 1][i]),
                                 __uint_as_float(r[q & 1][i + 1]), now, now);
                    }
                }
                if (kWgrad) {  // the column scales are read to the end
                    tc_fence_before();
                    __syncwarp();
                    arrive_lane0(free0, lane);
                }
                const uint32_t first = free0;
                free0 = free1;
                free1 = free2;
                free2 = first;
            }
            const uint32_t row = c.m0 + sub * 32, n = c.n0 + wg * kSumCols;
            if (ok && row < c.row_end && n < a.n &&
                (split == 1 || (!kWgrad && c.blocks == 0) || join_parts(a, c, split, warp - 4, lane, acc)))
                store_rows(s->out[warp - 4], &map_out, a.tma_out, reinterpret_cast<T*>(a.out),
                           (kWgrad ? (uint64_t)c.g * a.m : 0) + row, c.row_end - row, n, a.n, acc);
        }
        if (lane == 0) bulk_wait0();
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

// A matrix of `rows` rows of `cols` elements, contiguous; a box is 128 bytes of
// each of `box` rows, swizzled.  Boxes that reach past the matrix read zeros
// there and write nothing.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, uint32_t size, const void* base, uint64_t cols, uint64_t rows,
              uint32_t box)
{
    const EncodeTiled encode = encoder();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols * size};
    const cuuint32_t boxes[2] = {128 / size, box};
    const cuuint32_t steps[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <bool kWgrad, typename T>
cudaError_t launch_tiles(TileArgs a, const uint8_t* qa, uint64_t rows_a, const uint8_t* qb, uint64_t rows_b,
                         uint64_t rows_out, uint64_t most_tiles, int sms, cudaStream_t stream)
{
    CUtensorMap map_a, map_b, map_out = {};
    if (!make_map(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, qa, kFp8Block, rows_a, kTileM) ||
        !make_map(&map_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, qb, kFp8Block, rows_b, kTileN))
        return cudaErrorUnknown;
    // the TMA wants rows that begin on 16 bytes, and coordinates in 31 bits
    a.tma_out = (uint64_t)a.n * sizeof(T) % 16 == 0 && is_aligned(a.out, 16) && rows_out < (1ull << 31);
    if (a.tma_out && !make_map(&map_out, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                               sizeof(T), a.out, a.n, rows_out, 32))
        return cudaErrorUnknown;
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
    return cudaLaunchKernelEx(&cfg, gemm_kernel<kWgrad, T>, map_a, map_b, map_out, a);
}

}  // namespace

// Parts of the reduction where the tiles are too few for the SMs (152 of them: a
// number of its own, so that a workspace's size is the same on any device).
// Joining costs about 5 us, so it wants 24 blocks, 8 a part at least: 48 rows by
// 4096 x 14336 (n x k) 28 us in four parts and 55 whole, by 4096 x 4096 17.2 and
// 19.6, by 1024 x 2048 (16 blocks) 14.3 and 13.2.  Eight parts: 29.6 and 21.3 for
// the first two.
static uint32_t split_of(uint64_t tiles, uint64_t blocks)
{
    if (tiles == 0 || blocks < 24) return 1;
    uint64_t split = 152 / tiles < 4 ? 152 / tiles : 4;
    if (split > blocks / 8) split = blocks / 8;
    return split < 2 ? 1 : (uint32_t)split;
}

uint32_t matmul_split(uint64_t rows, uint64_t n, uint64_t k, uint32_t groups)
{
    const uint64_t active = rows < groups ? rows : groups, by_rows = (rows + kTileM - 1) / kTileM;
    return split_of((active > by_rows ? active : by_rows) * ((n + kTileN - 1) / kTileN), blocks_of(k));
}

// The mean group's blocks stand for those of all.
uint32_t wgrad_split(uint64_t rows, uint64_t m, uint64_t n, uint32_t groups)
{
    return split_of(groups * ((m + kTileM - 1) / kTileM) * ((n + kTileN - 1) / kTileN), rows / kFp8Block / groups);
}

uint64_t part_bytes(uint32_t split) { return split > 1 ? (uint64_t)kJoinParts * kTileM * kTileN * 4 : 0; }

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
    a.ticket = m.ticket;
    a.split = m.split;
    a.counters = m.counters;
    a.parts = m.parts;
    a.status = m.status;
    const uint64_t most = (blocks_of(m.rows) + m.G) * ((m.n + kTileN - 1) / kTileN) * m.split;
    const auto launch = m.out_f32 ? launch_tiles<false, float> : launch_tiles<false, __nv_bfloat16>;
    return launch(a, m.a, (uint64_t)m.KB * m.rows, m.b, (uint64_t)m.G * m.KB * m.n, m.rows, most, sms, stream);
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
    a.ticket = w.ticket;
    a.split = w.split;
    a.counters = w.counters;
    a.parts = w.parts;
    a.status = w.status;
    const uint64_t most = (uint64_t)w.G * ((w.m + kTileM - 1) / kTileM) * ((w.n + kTileN - 1) / kTileN) * w.split;
    const auto launch = w.out_f32 ? launch_tiles<true, float> : launch_tiles<true, __nv_bfloat16>;
    return launch(a, w.a, (uint64_t)w.blocks * w.m, w.b, (uint64_t)w.blocks * w.n, (uint64_t)w.G * w.m, most, sms, stream);
}

}  // namespace zccl
