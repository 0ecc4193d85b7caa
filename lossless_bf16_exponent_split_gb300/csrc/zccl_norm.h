// zccl_norm.h -- arguments of the norm kernels, and how a backward pass's rows are
// shared out.
#pragma once

#include "zccl_rows.cuh"

namespace zccl {

struct NormArgs {
    const void* x;       // forward: the residual; backward: the stored r (with grad_h)
    const void* y;       // nullptr: no join (forward), not read (backward)
    uint64_t x_stride, y_stride;
    Vector weight, post_weight, gate;
    uint64_t gate_stride;
    uint32_t gate_span;  // at most `rows`, which are below 2^31
    uint32_t rows;
    uint32_t hidden;
    int post;
    float inv_hidden, eps;
    float scale, gain;   // of the join, and of its dropout (1 without)
    float factor;        // their product
    DropArgs drop;
    uint32_t* status;
    void* r;             // forward
    void* h;
    // backward
    const void* grad_r;
    const void* grad_h;
    uint64_t grad_r_stride, grad_h_stride;
    void* grad_x;
    void* grad_y;
    void* grad_weight;
    void* grad_post_weight;
    void* grad_gate;
    float* sums;         // workspace: weights' sums of each group (a CTA's or a cluster's teams), then gates' parts
    float* parts;
    uint32_t groups, workers;
    int joined;          // the kernel that adds them up follows
};

inline uint32_t size_of(int dtype) { return dtype == ZCCL_BF16 ? 2 : 4; }

// Rows are shared out over workers, each a run of neighbouring rows.  In a backward
// pass a worker keeps its sums of the weights' gradients over its rows, and of the
// gate's over the rows of a gate row.  A gate row that lies within a worker's rows it
// finishes itself; of one that began before its rows, or goes on behind them, it has a
// part.
enum { kSlotWeight = 0, kSlotPost = 1, kWeightSlots = 2 };  // sums of the weights: [groups][2][pitch]
enum { kSlotBefore = 0, kSlotBehind = 1, kGateSlots = 2 };  // parts of gate rows: [workers][2][pitch]

// The first row of worker w.
__host__ __device__ inline uint32_t first_row(uint32_t rows, uint32_t workers, uint32_t w)
{
    const uint32_t base = rows / workers, more = rows - base * workers;
    return base * w + (w < more ? w : more);
}
// The worker of a row.
__host__ __device__ inline uint32_t worker_of(uint32_t rows, uint32_t workers, uint32_t row)
{
    const uint32_t base = rows / workers, more = rows - base * workers, large = more * (base + 1);
    return row < large ? row / (base + 1) : more + (row - large) / base;
}

// How a row is held: by a warp (a tile at most), by the warps of a CTA, by those of a
// cluster's CTAs, or (kLong) read several times by a CTA; by half a warp or a quarter
// (rows on 16 bytes of up to 128 and 64 values), whose rows a warp goes through at once.
enum Team { kWarpTeam = 0, kCtaTeam = 1, kClusterTeam = 2, kLong = 3, kHalfTeam = 4, kQuarterTeam = 5 };
template <int kTeam>
constexpr uint32_t team_lanes = kTeam == kHalfTeam ? 16 : kTeam == kQuarterTeam ? 8 : 32;  // of a warp
template <int kTeam>
constexpr bool in_warp = kTeam == kWarpTeam || team_lanes<kTeam> < 32;
constexpr uint32_t kTeamWarps = 16;    // the most of a CTA
constexpr uint32_t kMoreWarps = 20;    // of an SM, where 16 are not a whole number of teams
constexpr uint32_t kMaxCluster = 4;    // CTAs
constexpr uint32_t kWarpsPerCta = 8;   // of warps that are teams

// Room for the sums of a team's warps, whose halves take turns, and a barrier of each
// half: a warp may put its sums of the next row while another still takes up those of
// this one; those of the row after it only when all have put the next row's, which they
// do after they have taken up this one's.
constexpr uint32_t kTeamRed = 2 * kTeamWarps * kMaxCluster * 8;
constexpr uint32_t kTeamBytes = kTeamRed * 4 + 16;

struct Shape {
    Team team;
    uint32_t pieces;   // tiles of a warp: 1 or 2
    uint32_t warps;    // of a CTA
    uint32_t ctas;     // of a row
    uint32_t workers;  // teams
    uint32_t grid;     // CTAs
};

// The SMs are taken as 152, each with 16 warps (128 registers a thread); forward, where a
// warp has one tile, 24 (80 registers).  `bytes`: of a value of x and one of y.  Where both
// have two a warp can hold two tiles: two are better (a row costs a warp about as much as
// two tiles do) where they come out even, in gradients from four tiles on (512 columns 55 us
// with one, 68 with two; 1024 with post and dropout 79, 69); of rows that begin anywhere from
// four, in gradients six, and not where that makes clusters of four of them (gradients: 500
// columns 48 us with one tile, 57 with two; 4095 54, 48; 10001 75, 59; 16383 61, 72.
// Forward, with post and dropout: 1001 columns 45 us, 40; 4095 55, 44; 8191 64, 51).
inline Shape norm_shape(uint64_t hidden, uint64_t rows, uint32_t bytes, bool vec, bool backward)
{
    constexpr uint32_t kSms = 152;
    const uint32_t tiles = (uint32_t)((hidden + kTile - 1) / kTile);
    const bool many = vec ? tiles > (backward ? 2 : 1) : tiles > (backward ? 5 : 3) && tiles <= 60;
    const uint32_t pieces = bytes == 4 && many && (tiles % 2 == 0 || tiles > 8) ? 2 : 1, units = (tiles + pieces - 1) / pieces;
    // a cluster's CTA holds three rows in shared memory: 15 warps of two 16-bit tiles, or 16 of one tile
    const uint32_t alone = 16, most = pieces == 2 ? 15 : 16, sm_warps = !backward && pieces == 1 ? 24 : 16;
    Shape s{};
    const auto at_most_rows = [&](uint64_t n) { return (uint32_t)(n < rows ? n : rows > 0 ? rows : 1); };
    if (tiles <= 1) {
        const uint32_t of_warp = !vec || hidden > 128 ? 1 : hidden > 64 ? 2 : 4;  // teams
        s = {of_warp == 4 ? kQuarterTeam : of_warp == 2 ? kHalfTeam : kWarpTeam, 1, kWarpsPerCta, 1, at_most_rows(kSms * sm_warps * of_warp), 0};
        s.grid = (s.workers + kWarpsPerCta * of_warp - 1) / (kWarpsPerCta * of_warp);
    } else if (units <= most * kMaxCluster && tiles <= kTeamWarps * kMaxCluster) {
        s.ctas = units <= alone ? 1 : units <= 2 * most ? 2 : 4;
        // 9 or 10 warps leave a third of an SM empty, three clusters' CTAs of 5 do not: 5120 columns forward 48.7 us,
        // 52.4 with 10 warps; not so the gradients (64.8 and 63.0), with three rows in shared memory
        if (!backward && (units == 9 || units == 10)) s.ctas = 2;
        s.team = s.ctas > 1 ? kClusterTeam : kCtaTeam;
        s.pieces = pieces;
        s.warps = (units + s.ctas - 1) / s.ctas;
        // clusters of four do not fill every group of SMs: 36 of 38 are taken
        uint32_t sm_ctas = sm_warps / s.warps;
        // one team more, of warps with one tile, where 16 warps are not a whole number of them: 32-bit residual, BF16
        // block, 2560 columns 45.0 us with 20 warps, 55.9 with 10; 1280 44.2 and 46.9.  All in 32 bits their rows would
        // take the shared memory that L1 has: 1280 columns 65 us, 54.5; rows that begin anywhere gain from a second team only
        // (2305 columns 61.9 and 64.9, 1300 62.7 and 59.1)
        if (backward && pieces == 1 && s.ctas == 1 && bytes < 8 && sm_ctas * s.warps < 16 && (vec || sm_ctas == 1)) sm_ctas = kMoreWarps / s.warps;
        s.workers = at_most_rows((uint64_t)(s.ctas == 4 ? 144 : kSms) * sm_ctas / s.ctas);
        s.grid = s.workers * s.ctas;
    } else {
        // gradients' sums stay in the workspace: fewer workers for longer rows (forward alike, where nothing asks for it)
        s = {kLong, 1, kTeamWarps, 1, at_most_rows(kSms * 16384 / hidden * 2), 0};
        s.grid = s.workers;
    }
    return s;
}

// N values, rounded up to a power of two: that many lanes of a warp hold one each.
template <int N>
constexpr int kValues = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : 8;

// Sums N values (N <= 8) over each L lanes: while a lane holds several it keeps half of them
// in a step, so that nine exchanges do for all eight of a warp.  Lanes L / kValues * i and
// up hold value i then.
template <int N, int L>
__device__ __forceinline__ float warp_sums(const float (&s)[N])
{
    constexpr int H = kValues<N>;
    const uint32_t lane = threadIdx.x & 31;
    float v[H];
#pragma unroll
    for (int i = 0; i < H; ++i) v[i] = i < N ? s[i] : 0.0f;
    int o = L / 2;
#pragma unroll
    for (int h = H / 2; h > 0; h /= 2, o /= 2) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float keep = upper ? v[i + h] : v[i], give = upper ? v[i] : v[i + h];
            v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
#pragma unroll
    for (int x = L / H / 2; x > 0; x /= 2) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], x);
    return v[0];
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_ctas()
{
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Sends v to the same place of CTA `rank` of the cluster, where its arrival counts on the
// same barrier.
__device__ __forceinline__ void send(float* p, uint64_t* bar, uint32_t rank, float v)
{
    uint32_t at, to;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_addr(bar)), "r"(rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at), "r"(__float_as_uint(v)), "r"(to)
                 : "memory");
}
// Bounded wait for what the cluster sends; false if it did not come.
__device__ __forceinline__ bool wait_sent(uint64_t* bar, uint32_t parity)
{
    const auto there = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            " selp.u32 %0, 1, 0, p;\n}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (there()) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1;; ++it) {
        if (there()) return true;
        if ((it & 15) == 0 && globaltimer() - t0 > kSpinTimeoutNs) return false;
    }
}

// A warp's worker, and its neighbouring tiles of a row.  Of teams that share a warp, each
// lane's: tiles then begin (modulo 2^32) where the team's first lane has column 0.
struct Place {
    uint32_t worker, first;
    __device__ __forceinline__ uint32_t tile(int n) const { return first + n * kTile; }
};
template <int kTeam, int kPieces>
__device__ __forceinline__ Place place()
{
    const uint32_t warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (in_warp<kTeam>) {
        const uint32_t team = (threadIdx.x & 31) / team_lanes<kTeam>;
        return {(blockIdx.x * kWarpsPerCta + warp) * (32 / team_lanes<kTeam>) + team, 0u - team * team_lanes<kTeam> * 8};
    }
    if (kTeam == kCtaTeam) return {blockIdx.x, warp * kPieces * kTile};
    const uint32_t ctas = cluster_ctas();
    return {blockIdx.x / ctas, (cluster_rank() * warps + warp) * kPieces * kTile};
}

// Where a warp's rows lo..hi-1 end: of teams that share it, where those of the one with most
// would.
template <int kTeam>
__device__ __forceinline__ uint32_t last_step(uint32_t lo, uint32_t hi)
{
    return team_lanes<kTeam> == 32 ? hi : lo + __reduce_max_sync(0xFFFFFFFFu, hi - lo);
}

// Sums N values (N <= 8) over a team, the same way in every thread, in steps: a warp's
// own sums (warp_sums), which it puts where all of the team find them, and, after a wait
// for all warps', the taking up of them.  A cluster's warps send theirs to each of its
// CTAs, which wait for the bytes to arrive: a cluster barrier would also wait for every
// store to global memory.
template <int N, int kTeam>
struct TeamSum {
    static constexpr int H = kValues<N>, kLanes = team_lanes<kTeam> / H;
    static constexpr int kRounds = ((int)kTeamWarps * (kTeam == kClusterTeam ? (int)kMaxCluster : 1) * H + 31) / 32;
    float* const red;
    uint64_t* const bar;
    uint32_t* const status;
    uint32_t turn = 0, parity = 0;
    float mine = 0.0f;   // of a team within a warp
    bool lost = false;   // a wait ran out: no other is begun, and all sums are NaN
    const uint32_t all;  // values of the team's warps
    __device__ __forceinline__ TeamSum(void* smem, uint32_t* status)
        : red(static_cast<float*>(smem)), bar(reinterpret_cast<uint64_t*>(red + kTeamRed)), status(status),
          all((blockDim.x >> 5) * (kTeam == kClusterTeam ? cluster_ctas() : 1) * H)
    {
        if (kTeam != kClusterTeam) return;
        if (threadIdx.x == 0) {
            mbar_init(bar, 1);
            mbar_init(bar + 1, 1);
            fence_mbar_init();
        }
        cluster_sync();
    }
    // Before the kernel ends: no CTA leaves while another may still send to it.
    __device__ __forceinline__ void close()
    {
        if (kTeam == kClusterTeam) cluster_sync();
    }

    // v: what warp_sums gave.
    __device__ __forceinline__ void put(float v)
    {
        const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float* at = red + turn * (kTeamRed / 2) + lane / kLanes;
        if (in_warp<kTeam>) mine = v;
        if (kTeam == kCtaTeam && lane % kLanes == 0) at[warp * H] = v;
        if (kTeam == kClusterTeam) {
            if (threadIdx.x == 0) mbar_arrive_expect_tx(bar + turn, all * 4);
            // the lanes that hold a value take a CTA each
            if (lane % kLanes < cluster_ctas()) send(at + (cluster_rank() * (blockDim.x >> 5) + warp) * H, bar + turn, lane % kLanes, v);
            __syncwarp();
        }
        turn ^= 1;
    }
    __device__ __forceinline__ void wait()
    {
        if (kTeam == kCtaTeam) __syncthreads();
        if (kTeam == kClusterTeam) {
            if (!lost && !wait_sent(bar + (turn ^ 1), parity)) lost = true;
            parity ^= turn ^ 1;  // both halves have been used
        }
    }
    __device__ __forceinline__ void take(float (&s)[N])
    {
        const uint32_t lane = threadIdx.x & 31;
        float v = mine;
        if (!in_warp<kTeam>) {
            const float* at = red + (turn ^ 1) * (kTeamRed / 2) + lane;
            v = 0.0f;
#pragma unroll
            for (int i = 0; i < kRounds; ++i)
                if (kTeam == kClusterTeam ? i * 32 < all : true) v += i * 32 + lane < all ? at[i * 32] : 0.0f;
            if (kTeam == kClusterTeam && __any_sync(0xFFFFFFFFu, lost)) {
                v = __uint_as_float(0x7FC00000u);
                if (lane == 0) report(status, ZCCL_ERR_TIMEOUT);
            }
#pragma unroll
            for (int o = 16; o >= H; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = N == 1 ? v : __shfl_sync(0xFFFFFFFFu, v, in_warp<kTeam> ? i * kLanes : i, team_lanes<kTeam>);
    }
    __device__ __forceinline__ void operator()(float (&s)[N])
    {
        put(warp_sums<N, team_lanes<kTeam>>(s));
        wait();
        take(s);
    }
};

// Sums N values over a CTA, the same way in every thread; `red` holds
// 2 * 32 * N floats, whose halves take turns by `turn`.
template <int N>
__device__ __forceinline__ void cta_sum(float (&s)[N], float* red, uint32_t& turn)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
    if (warps == 1) return;
    float* at = red + turn * 32 * N;
    turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) at[i * 32 + warp] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = lane < warps ? at[i * 32 + lane] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) s[i] += __shfl_xor_sync(0xFFFFFFFFu, s[i], o);
    }
}

// Of each group of teams the weights' sums, of each worker its parts of gate rows.
inline uint64_t norm_backward_bytes(const Shape& s, uint64_t hidden)
{
    return ((uint64_t)(s.grid / s.ctas) * kWeightSlots + (uint64_t)s.workers * kGateSlots) * ((hidden + 7) / 8 * 8) * sizeof(float);
}

// What the block's output is multiplied by before it joins (scale, gate, the
// dropout's gain).
template <bool kVec>
__device__ __forceinline__ Eight join_factors(const NormArgs& a, uint32_t row, uint32_t tile)
{
    const uint64_t at = a.gate.p != nullptr ? (uint64_t)(row / a.gate_span) * a.gate_stride : 0;
    return mul(mul(load_vector<kVec>(a.gate, at, tile, a.hidden), a.scale), a.gain);
}
// Asks for the gate's part of the lane's tile, to be loaded when its first row comes.
template <bool kVec>
__device__ __forceinline__ void prefetch_gate(const NormArgs& a, uint32_t row, uint32_t tile)
{
    const uint32_t c = column<kVec>(tile, 0);
    if (a.gate.p == nullptr || c >= a.hidden) return;
    const uint64_t at = ((uint64_t)(row / a.gate_span) * a.gate_stride + c) * (a.gate.dtype == ZCCL_BF16 ? 2 : 4);
    asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const char*>(a.gate.p) + at));
}
// Which of the lane's values of it stay.
template <bool kVec>
__device__ __forceinline__ Kept<kVec> join_kept(const NormArgs& a, uint64_t offset, uint32_t row, uint32_t tile)
{
    return a.drop.below > 0 ? kept_piece<kVec>(a.drop, offset, row, tile) : kept_all<kVec>();
}

using NormKernel = void (*)(NormArgs);
// The kernels of a pair of types; warp_bytes: shared memory of a warp.
template <typename Tx, typename Ty>
NormKernel norm_kernel_for(const Shape& s, bool vec, bool post, bool drop, uint32_t* warp_bytes);
template <typename Tx, typename Ty>
NormKernel norm_backward_kernel_for(const Shape& s, bool vec, bool post, bool drop, uint32_t* warp_bytes);

zccl_status_t launch_norm(NormArgs& a, int x_dtype, int dtype, bool vec, cudaStream_t stream);
zccl_status_t launch_norm_backward(NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec, cudaStream_t stream);

// The most shared memory that a CTA may be launched with, beside a TeamSum's of its own (the
// forward kernels have one).
constexpr int kMostSmem = (227 << 10) - (int)kTeamBytes;

// Launches `kernel` as launch_dependent does, in clusters where a row has several CTAs.
inline cudaError_t launch_teams(NormKernel kernel, const Shape& s, uint32_t threads, size_t smem, cudaStream_t stream,
                                const NormArgs& a)
{
    if (smem + kTeamBytes > 48 << 10) {
        // the limit is the kernel's and not the launch's: always the same one, as another thread may be about to
        // launch the same kernel for longer rows
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return e;
    }
    if (s.team != kClusterTeam) return launch_dependent(kernel, s.grid, threads, smem, stream, a);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s.grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = s.ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace zccl
