// zccl_dispatch.cu -- the rows of the tokens in expert order, and the segment
// table that the batched compression reads.
//
// A stable counting sort of the T * K slots by expert.  The slots are cut into
// tiles of whole tokens, one per CTA.  Few slots: one kernel, every CTA counts
// all slots itself.  Many: a first kernel counts each tile's slots per expert,
// at most a tile per SM, and its last CTA turns the counts into places (no CTA waits
// for another); in the second kernel several CTAs share a tile, each counts the
// slots of the tile before its own, ranks those and moves the rows.  A token's
// row is read once and stored K times.  Slots without an expert sort last and
// store zeros, so every row is written exactly once.
//
// Bound by HBM: 2 T H bytes read, 2 T K H written.  16384 tokens, 8 slots, hidden
// 2048: 100 us a call (6.1 TB/s).
#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr uint32_t kMoveThreads = 256;
constexpr uint32_t kCountThreads = 512;
constexpr uint32_t kFlight = 4;  // pieces of rows in flight in a thread
constexpr uint32_t kMoveWarps = kMoveThreads / 32;
// Up to this many slots every CTA counts them all itself.  Measured so and with
// the counting kernel, in us: top 8 of 64, hidden 2048, 4096 slots 6.0 and 9.5, 16384:
// 15.5 and 17.5, 32768: 33.8 and 30.1; top 8 of 256, hidden 256, 16384: 7.9 and 9.6,
// 32768: 12.4 and 10.8.
constexpr uint64_t kSmallSlots = 24576;
constexpr uint64_t kTileSlots = 2048;  // a counted tile has at least these, so that its last CTA has few counts to add up
// A counted tile's rows are moved by CTAs that store about this much each, but by
// no more than 64 (more, smaller CTAs end closer together: 100 us for the
// all-to-all's rows, 104 with four times as much each, 120 with four CTAs a tile).
constexpr uint64_t kSubBytes = 65536;
constexpr uint32_t kSubTiles = 64;

struct DispatchArgs {
    const int32_t* idx;
    uint64_t tokens;
    uint32_t E, K;
    const uint16_t* x;
    uint64_t stride;
    uint32_t pieces;  // 16-byte pieces of a row
    uint64_t hidden;
    uint16_t* rows;
    int32_t* pos;
    int32_t* counts;
    int32_t* offsets;
    zccl_segment_t* segs;
    uint64_t capacity;
    uint8_t* streams;
    uint32_t tiles;        // tiles that are counted
    uint32_t tile_tokens;  // tokens of a tile
    uint32_t sub_tokens;   // tokens of a CTA that moves rows
    uint32_t subs;         // CTAs that move a counted tile's rows
    uint32_t* ticket;      // CTAs of the counting kernel that are done
    int32_t* base;         // [tiles][E + 1]: a tile's count of an expert's slots, then its first row
};

__device__ __forceinline__ uint32_t bucket_of(int32_t e, uint32_t E) { return (uint32_t)e < E ? (uint32_t)e : E; }

// Exclusive prefix sum of v[0..n), in place, by warp 0 (n <= 513); v[n] must
// not be read.  Ends with no barrier.
__device__ void scan_warp0(int32_t* v, uint32_t n)
{
    if (threadIdx.x >= 32) return;
    const uint32_t per = (n + 31) / 32, lo = min(n, threadIdx.x * per), hi = min(n, lo + per);
    int32_t sum = 0;
    for (uint32_t i = lo; i < hi; ++i) sum += v[i];
    int32_t run = (int32_t)warp_scan((uint64_t)sum) - sum;
    for (uint32_t i = lo; i < hi; ++i) {
        const int32_t c = v[i];
        v[i] = run;
        run += c;
    }
}

// The outputs about the experts as wholes, by one CTA: first[0..E] are the
// experts' first rows (first[E]: the rows in all).
__device__ void write_tables(const DispatchArgs& a, const int32_t* first)
{
    for (uint32_t e = threadIdx.x; e <= a.E; e += blockDim.x) {
        a.offsets[e] = first[e];
        if (e < a.E) a.counts[e] = first[e + 1] - first[e];
    }
    if (a.segs == nullptr || threadIdx.x >= 32) return;
    // the streams' places: a prefix sum of their largest sizes
    const uint32_t n = 2 * a.E, per = (n + 31) / 32;
    const uint32_t lo = min(n, threadIdx.x * per), hi = min(n, lo + per);
    uint64_t run = 0;
    for (int pass = 0; pass < 2; ++pass) {
        uint64_t sum = 0;
        for (uint32_t i = lo; i < hi; ++i) {
            const uint32_t e = i / 2;
            const uint64_t begin = (uint64_t)first[e], count = (uint64_t)(first[e + 1] - first[e]);
            const uint64_t fixed = count < a.capacity ? count : a.capacity;
            const uint64_t row = i & 1 ? begin + fixed : begin, rows = i & 1 ? count - fixed : fixed;
            const uint64_t values = rows * a.hidden, bytes = stream_bytes_of(values, values);
            if (pass == 1)
                a.segs[i] = zccl_segment_t{a.rows + row * a.hidden, values, a.streams + run + sum, bytes};
            sum += round_up(bytes, 128);
        }
        if (pass == 0) run = warp_scan(sum) - sum;
    }
}

// Counts each tile's slots per expert; the last CTA done makes the counts
// places, a thread an expert, 32 tiles' counts in flight (a warp an expert, with
// shuffles, took 10 us for 64 experts and 28 for 512).
__global__ void __launch_bounds__(kCountThreads) dispatch_count_kernel(DispatchArgs a)
{
    __shared__ int32_t count[ZCCL_MAX_EXPERTS + 2];
    __shared__ uint32_t order;
    pdl_wait();
    const uint32_t tid = threadIdx.x, B = a.E + 1;
    for (uint32_t e = tid; e < B; e += kCountThreads) count[e] = 0;
    __syncthreads();
    const uint64_t lo = (uint64_t)blockIdx.x * a.tile_tokens * a.K;
    const uint64_t hi = min((uint64_t)(blockIdx.x + 1) * a.tile_tokens, a.tokens) * a.K;
    for (uint64_t i = lo + tid; i < hi; i += kCountThreads) atomicAdd(&count[bucket_of(a.idx[i], a.E)], 1);
    __syncthreads();
    for (uint32_t e = tid; e < B; e += kCountThreads) a.base[blockIdx.x * B + e] = count[e];
    __threadfence();
    __syncthreads();
    if (tid == 0) order = atom_inc_acq_rel(a.ticket, a.tiles - 1);  // wraps to 0 for the next call
    __syncthreads();
    if (order != a.tiles - 1) return;
    __threadfence();
    for (uint32_t e = tid; e < B; e += kCountThreads) {
        int32_t* at = a.base + e;
        int32_t run = 0;
        constexpr uint32_t kAhead = 32;
        for (uint32_t t0 = 0; t0 < a.tiles; t0 += kAhead) {
            int32_t c[kAhead];
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) c[j] = t0 + j < a.tiles ? ld_l2(at + (t0 + j) * B) : 0;
#pragma unroll
            for (uint32_t j = 0; j < kAhead; ++j) {
                if (t0 + j < a.tiles) at[(t0 + j) * B] = run;
                run += c[j];
            }
        }
        count[e] = run;
    }
    __syncthreads();
    scan_warp0(count, a.E + 1);
    __syncthreads();
    write_tables(a, count);
}

// Ranks a CTA's slots and moves their rows.  kSmall: the CTA counts all slots
// and those before its own itself (the counting kernel did not run).
template <bool kSmall>
__global__ void __launch_bounds__(kMoveThreads) dispatch_move_kernel(DispatchArgs a)
{
    extern __shared__ int32_t smem[];
    const uint32_t B = a.E + 1;                     // buckets
    int32_t* first = smem;                          // [B] next row of each bucket
    int32_t* place = first + B;                     // [kMoveThreads] row of a slot, negative: store zeros at ~row
    int32_t* by_warp = place + kMoveThreads;        // [kMoveWarps][B]
    pdl_wait();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t counted = blockIdx.x / a.subs;  // the tile that was counted
    const uint64_t tile = (uint64_t)counted * a.tile_tokens;
    const uint64_t lo = kSmall ? (uint64_t)blockIdx.x * a.sub_tokens
                               : min(tile + (uint64_t)(blockIdx.x % a.subs) * a.sub_tokens, a.tokens);
    const uint64_t hi = min(kSmall ? lo + a.sub_tokens : min(lo + a.sub_tokens, tile + a.tile_tokens), a.tokens);
    if (kSmall) {
        int32_t* all = by_warp;
        int32_t* before = by_warp + B + 1;
        for (uint32_t e = tid; e < B; e += kMoveThreads) all[e] = 0, before[e] = 0;
        __syncthreads();
        for (uint64_t i = tid; i < a.tokens * a.K; i += kMoveThreads) {
            const uint32_t e = bucket_of(a.idx[i], a.E);
            atomicAdd(&all[e], 1);
            if (i < lo * a.K) atomicAdd(&before[e], 1);
        }
        __syncthreads();
        scan_warp0(all, B);
        __syncthreads();
        for (uint32_t e = tid; e < B; e += kMoveThreads) first[e] = all[e] + before[e];
        if (blockIdx.x == 0) write_tables(a, all);
        __syncthreads();
    } else {
        for (uint32_t e = tid; e < B; e += kMoveThreads)
            first[e] = ld_l2(a.base + counted * B + e) + ld_l2(a.offsets + e);
        __syncthreads();
        for (uint64_t i = tile * a.K + tid; i < lo * a.K; i += kMoveThreads) atomicAdd(&first[bucket_of(a.idx[i], a.E)], 1);
        __syncthreads();
    }
    const uint32_t step = kMoveThreads / a.K;  // whole tokens of a round
    for (uint64_t t0 = lo; t0 < hi; t0 += step) {
        const uint32_t tokens = (uint32_t)min((uint64_t)step, hi - t0), slots = tokens * a.K;
        for (uint32_t i = tid; i < kMoveWarps * B; i += kMoveThreads) by_warp[i] = 0;
        __syncthreads();
        const uint32_t e = tid < slots ? bucket_of(a.idx[t0 * a.K + tid], a.E) : B;
        const uint32_t peers = __match_any_sync(0xFFFFFFFFu, e);
        const uint32_t rank = __popc(peers & ((1u << lane) - 1u));
        if (tid < slots && rank == 0) by_warp[warp * B + e] = __popc(peers);
        __syncthreads();
        const uint32_t warps = (slots + 31) / 32;
        for (uint32_t b = tid; b < B; b += kMoveThreads) {
            int32_t run = first[b];
            for (uint32_t w = 0; w < warps; ++w) {
                const int32_t c = by_warp[w * B + b];
                by_warp[w * B + b] = run;
                run += c;
            }
            first[b] = run;
        }
        __syncthreads();
        if (tid < slots) {
            const int32_t row = by_warp[warp * B + e] + (int32_t)rank;
            a.pos[t0 * a.K + tid] = e < a.E ? row : -1;
            place[tid] = e < a.E ? row : ~row;
        }
        __syncthreads();
        if (a.x != nullptr) {
            const uint32_t total = tokens * a.pieces;
            for (uint32_t p0 = tid; p0 < total; p0 += kFlight * kMoveThreads) {
                uint4 v[kFlight];
                uint32_t t[kFlight], c[kFlight];
#pragma unroll
                for (uint32_t f = 0; f < kFlight; ++f) {
                    const uint32_t p = min(p0 + f * kMoveThreads, total - 1);
                    t[f] = p / a.pieces;
                    c[f] = p - t[f] * a.pieces;
                    v[f] = ld_once(reinterpret_cast<const uint4*>(a.x + (t0 + t[f]) * a.stride) + c[f]);
                }
#pragma unroll
                for (uint32_t f = 0; f < kFlight; ++f)
                    if (p0 + f * kMoveThreads < total)
                        for (uint32_t k = 0; k < a.K; ++k) {
                            const int32_t row = place[t[f] * a.K + k];
                            uint4* dst = reinterpret_cast<uint4*>(a.rows) + (uint64_t)(row < 0 ? ~row : row) * a.pieces + c[f];
                            __stcs(dst, row < 0 ? make_uint4(0, 0, 0, 0) : v[f]);
                        }
            }
        }
        __syncthreads();
    }
}

struct DispatchPlan {
    uint32_t tiles, tile_tokens, sub_tokens, subs, ctas;
    bool small;
};

// Few slots: a CTA for a token, or for as many as make two CTAs per SM.  Many:
// counted tiles, one per SM at most, each moved by several CTAs.
DispatchPlan dispatch_plan(uint64_t tokens, uint32_t top_k, uint64_t hidden, int sms)
{
    DispatchPlan p{};
    p.small = tokens * top_k <= kSmallSlots;
    const uint64_t full = (tokens * top_k + kTileSlots - 1) / kTileSlots;
    const uint64_t most = p.small ? (uint64_t)sms * 2 : full < (uint64_t)sms ? full : (uint64_t)sms;
    p.tile_tokens = (uint32_t)((tokens + most - 1) / most);
    if (p.tile_tokens == 0) p.tile_tokens = 1;
    p.tiles = (uint32_t)((tokens + p.tile_tokens - 1) / p.tile_tokens);
    if (p.tiles == 0) p.tiles = 1;
    uint64_t sub = kSubBytes / (2 * top_k * hidden + 1) + 1;
    const uint32_t least = (p.tile_tokens + kSubTiles - 1) / kSubTiles;
    if (sub < least) sub = least;
    p.sub_tokens = p.small || sub > p.tile_tokens ? p.tile_tokens : (uint32_t)sub;
    p.subs = p.small ? 1 : (p.tile_tokens + p.sub_tokens - 1) / p.sub_tokens;
    p.ctas = p.tiles * p.subs;
    return p;
}

bool dispatch_sizes_ok(uint64_t tokens, uint32_t experts, uint32_t top_k)
{
    return experts >= 1 && experts <= ZCCL_MAX_EXPERTS && top_k >= 1 && top_k <= ZCCL_MAX_TOP_K &&
           tokens < (1ull << 31) / top_k;
}

}  // namespace

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_dispatch_workspace_bytes(uint64_t tokens, uint32_t experts, uint32_t top_k, uint64_t* bytes)
{
    if (bytes == nullptr || !dispatch_sizes_ok(tokens, experts, top_k)) return ZCCL_ERR_INVALID_ARG;
    // for any device: the tile count never passes the token count or this bound
    const uint64_t tiles = tokens < 1024 ? (tokens ? tokens : 1) : 1024;
    *bytes = round_up(256 + 4ull * (experts + 1) * tiles, 256);
    return ZCCL_OK;
}

uint64_t zccl_dispatch_stream_bytes(uint64_t rows, uint64_t hidden, uint32_t experts)
{
    // each stream: a header, slots rounded up to 1024 (11 bits each), escapes rounded up to 128, its place to 128
    const uint64_t n = rows * hidden, streams = 2ull * experts;
    return round_up(n + n * 11 / 8 + streams * (kHeaderBytes + kTailGrain * 11 / 8 + 3 * 128), 128);
}

zccl_status_t zccl_dispatch(const int32_t* d_idx, uint64_t tokens, uint32_t experts, uint32_t top_k,
                            const uint16_t* d_x, uint64_t stride, uint64_t hidden, uint16_t* d_rows, int32_t* d_pos,
                            int32_t* d_counts, int32_t* d_offsets, zccl_segment_t* d_segs, uint64_t capacity,
                            void* d_streams, uint64_t stream_bytes, void* d_ws, uint64_t ws_bytes,
                            cudaStream_t stream)
{
    if (!dispatch_sizes_ok(tokens, experts, top_k) || hidden >= (1ull << 24) || hidden % 8 != 0 || stride % 8 != 0 ||
        stride >= kMaxElems || tokens * top_k * hidden >= kMaxElems)
        return ZCCL_ERR_INVALID_ARG;
    if (!good_ptr(d_counts, 4) || !good_ptr(d_offsets, 4) || !good_ptr(d_ws, 16)) return ZCCL_ERR_INVALID_ARG;
    if (tokens > 0 && (!good_ptr(d_idx, 4) || !good_ptr(d_pos, 4))) return ZCCL_ERR_INVALID_ARG;
    const bool move = d_x != nullptr && hidden > 0 && tokens > 0;
    if (move && (!is_aligned(d_x, 16) || !good_ptr(d_rows, 16))) return ZCCL_ERR_INVALID_ARG;
    if (d_segs != nullptr) {
        if (!is_aligned(d_segs, 8) || !good_ptr(d_streams, 16) || !is_aligned(d_rows, 16) ||
            (d_rows == nullptr && tokens * hidden > 0))
            return ZCCL_ERR_INVALID_ARG;
        if (stream_bytes < zccl_dispatch_stream_bytes(tokens * top_k, hidden, experts)) return ZCCL_ERR_BUFFER_TOO_SMALL;
    }
    uint64_t need = 0;
    zccl_dispatch_workspace_bytes(tokens, experts, top_k, &need);
    if (ws_bytes < need) return ZCCL_ERR_BUFFER_TOO_SMALL;
    const int sms = sm_count();
    if (sms == 0) return ZCCL_ERR_CUDA;
    const DispatchPlan p = dispatch_plan(tokens, top_k, move ? hidden : 0, sms < 512 ? sms : 512);
    DispatchArgs a{};
    a.idx = d_idx;
    a.tokens = tokens;
    a.E = experts;
    a.K = top_k;
    a.x = move ? d_x : nullptr;
    a.stride = stride;
    a.pieces = (uint32_t)(hidden / 8);
    a.hidden = hidden;
    a.rows = d_rows;
    a.pos = d_pos;
    a.counts = d_counts;
    a.offsets = d_offsets;
    a.segs = d_segs;
    a.capacity = capacity;
    a.streams = reinterpret_cast<uint8_t*>(d_streams);
    a.tiles = p.tiles;
    a.tile_tokens = p.tile_tokens;
    a.sub_tokens = p.sub_tokens;
    a.subs = p.subs;
    a.ticket = reinterpret_cast<uint32_t*>(d_ws);
    a.base = reinterpret_cast<int32_t*>((uint8_t*)d_ws + 256);
    const size_t smem = sizeof(int32_t) * ((experts + 1) + kMoveThreads + (size_t)(kMoveWarps + 1) * (experts + 1));
    auto kernel = p.small ? dispatch_move_kernel<true> : dispatch_move_kernel<false>;
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return ZCCL_ERR_CUDA;
    if (!p.small) {
        const cudaError_t e = launch_dependent(dispatch_count_kernel, p.tiles, kCountThreads, 0, stream, a);
        if (e != cudaSuccess) return ZCCL_ERR_CUDA;
    }
    return launched(launch_dependent(kernel, p.ctas, kMoveThreads, smem, stream, a));
}

}  // extern "C"
