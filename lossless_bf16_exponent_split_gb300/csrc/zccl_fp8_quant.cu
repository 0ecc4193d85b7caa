// zccl_fp8_quant.cu -- activations and weights as block-scaled e4m3 codes.
//
// A block's codes are rne(x * (448 * (1 / amax))) with scale amax / 448.  Rows: a
// block is 128 values of a row, quantised by half a warp, so the maximum is
// four shuffles.  Along the rows: a block is one column of 128 rows of a
// group; a CTA takes 128 x 128 values, keeps them in registers between the
// maximum and the conversion, and exchanges the axes of the codes in shared
// memory.  All are bound by HBM: each value is read once (2 bytes for BF16)
// and written once (1 byte).  131072 x 2048 BF16 by rows: 125 us, 6.5 TB/s; 4096 x
// 14336 along the rows and by rows in one pass: 53 us, 4.4 TB/s (the exchange and
// 7 waves of tiles), 4096 x 4096 along the rows alone 12 us.  Weights are read a
// value at a time, whatever their extents: 64 x 1024 x 2048 fp32 105 us (6.4 TB/s),
// 124 with the exchanged form, BF16 243 and 261, codes 231.
#include "zccl_fp8.cuh"

namespace zccl {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerWarp = 8;  // rows in flight in a warp

// The counters of the product that follows (every earlier use of them is over).
__device__ __forceinline__ void zero_counters(const QuantArgs& a)
{
    if (blockIdx.x != 0) return;
    if (threadIdx.x == 0 && a.ticket != nullptr) *a.ticket = 0;
    if (a.counters != nullptr)
        for (uint32_t i = threadIdx.x; i < kJoinCounters; i += kThreads) a.counters[i] = 0;
}

// Eight values of a row from column c on; zeros past the row's end.  kVec (fp32;
// BF16 rows that allow it have a kernel of their own): the eight are 16-byte
// aligned and either all in the row or all past it.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* row, uint32_t c, uint32_t cols, float (&v)[8])
{
    if constexpr (kVec) {
        static_assert(sizeof(T) == 4, "fp32");
        if (c >= cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
            return;
        }
        const uint4 a = ld_once(reinterpret_cast<const uint4*>(row + c));
        const uint4 b = ld_once(reinterpret_cast<const uint4*>(row + c) + 1);
        const uint32_t q[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(q[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? to_float<T>(row[c + i]) : 0.0f;
    }
}

// A warp takes 8 rows and two neighbouring blocks; consecutive warps take
// consecutive pairs of blocks of the same rows.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantArgs a)
{
    pdl_wait();
    pdl_launch_dependents();  // the product may start: what it reads before its own wait was there before this kernel
    zero_counters(a);
    const uint32_t lane = threadIdx.x & 31, half = lane >> 4, i8 = (lane & 15) * 8;
    const uint32_t nb = (uint32_t)blocks_of(a.cols), pairs = (nb + 1) / 2;
    const uint64_t items = (uint64_t)pairs * ((a.rows + kRowsPerWarp - 1) / kRowsPerWarp);
    const uint64_t step = (uint64_t)gridDim.x * (kThreads / 32);
    for (uint64_t it = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
        const uint32_t r0 = (uint32_t)(it / pairs) * kRowsPerWarp, b = (uint32_t)(it % pairs) * 2 + half;
        const uint32_t c = b * kFp8Block + i8;
        float v[kRowsPerWarp][8];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r)
            load8<T, kVec>(reinterpret_cast<const T*>(a.x) + (uint64_t)min(r0 + r, a.rows - 1) * a.stride, c, a.cols, v[r]);
        float mine = 0.0f;
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            float amax = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[r][i]));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            float scale, f;
            block_scale(amax, &scale, &f);
            if ((lane & 15) == r) mine = scale;
            if (b < nb && r0 + r < a.rows) {
                const uint2 q = make_uint2(e4m3x4(v[r][0] * f, v[r][1] * f, v[r][2] * f, v[r][3] * f),
                                           e4m3x4(v[r][4] * f, v[r][5] * f, v[r][6] * f, v[r][7] * f));
                *reinterpret_cast<uint2*>(a.q + ((uint64_t)b * a.rows + r0 + r) * kFp8Block + i8) = q;
            }
        }
        const uint32_t r = lane & 15;
        if (r < kRowsPerWarp && b < nb && r0 + r < a.rows) a.scale[(uint64_t)b * a.rows + r0 + r] = mine;
    }
}

// Largest magnitudes of BF16 pairs.
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t mag_pair(uint32_t a) { return a & 0x7FFF7FFFu; }
__device__ __forceinline__ float max_of_pair(uint32_t a) { return fmaxf(bf16_lo(a), bf16_hi(a)); }

// Maxima of kRows pairs over kLanes = 2 kRows neighbouring lanes, by halves: in
// each step a lane gives away the rows that its partner keeps, so kRows
// exchanges do for kRows rows.  Ends with row owned_row(lane) in each lane.
template <int kRows>
__device__ __forceinline__ uint32_t max_rows(uint32_t (&m)[kRows], uint32_t lane)
{
#pragma unroll
    for (int n = kRows / 2; n > 0; n /= 2) {
        const bool upper = (lane & (2 * n)) != 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint32_t give = upper ? m[i] : m[i + n], keep = upper ? m[i + n] : m[i];
            m[i] = max_pair(keep, __shfl_xor_sync(0xFFFFFFFFu, give, 2 * n));
        }
    }
    return max_pair(m[0], __shfl_xor_sync(0xFFFFFFFFu, m[0], 1));
}
template <int kRows>
__device__ __forceinline__ uint32_t owned_row(uint32_t lane) { return (lane / 2) % kRows; }
// The lane, among the 2 kRows, that owns a row.
__device__ __forceinline__ constexpr uint32_t owner_of(uint32_t row) { return 2 * row; }

// BF16 rows in 16-byte pieces: as quantize_rows_kernel, with the values kept as
// they are read and the division done once a row (92 instructions a row of 256
// values and half the bandwidth before).
__global__ void __launch_bounds__(kThreads) quantize_rows_bf16_kernel(QuantArgs a)
{
    pdl_wait();
    pdl_launch_dependents();  // the product may start: what it reads before its own wait was there before this kernel
    zero_counters(a);
    const uint32_t lane = threadIdx.x & 31, half = lane >> 4, i8 = (lane & 15) * 8;
    const uint32_t nb = (uint32_t)blocks_of(a.cols), pairs = (nb + 1) / 2;
    const uint32_t groups = (a.rows + kRowsPerWarp - 1) / kRowsPerWarp;
    const uint32_t warps = gridDim.x * (kThreads / 32);
    // consecutive warps take consecutive pairs of blocks of the same rows
    const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const uint32_t step_g = warps / pairs, step_p = warps % pairs;
    uint32_t g = w / pairs, p = w % pairs;
    while (g < groups) {
        const uint32_t r0 = g * kRowsPerWarp, b = 2 * p + half, c = b * kFp8Block + i8;
        uint4 v[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r)
            v[r] = c < a.cols ? ld_once(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) +
                                                                       (uint64_t)min(r0 + r, a.rows - 1) * a.stride + c))
                              : make_uint4(0, 0, 0, 0);
        uint32_t m[kRowsPerWarp];
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r)
            m[r] = max_pair(max_pair(mag_pair(v[r].x), mag_pair(v[r].y)), max_pair(mag_pair(v[r].z), mag_pair(v[r].w)));
        float scale, factor;
        block_scale(max_of_pair(max_rows<kRowsPerWarp>(m, lane)), &scale, &factor);
        const uint32_t own = r0 + owned_row<kRowsPerWarp>(lane);
        if ((lane & 1) == 0 && b < nb && own < a.rows) a.scale[(uint64_t)b * a.rows + own] = scale;
        uint8_t* q = a.q + ((uint64_t)b * a.rows + r0) * kFp8Block + i8;
#pragma unroll
        for (int r = 0; r < kRowsPerWarp; ++r) {
            const float f = __shfl_sync(0xFFFFFFFFu, factor, (lane & 16) + owner_of(r));
            if (b < nb && r0 + r < a.rows)
                *reinterpret_cast<uint2*>(q + r * kFp8Block) =
                    make_uint2(e4m3x4(bf16_lo(v[r].x) * f, bf16_hi(v[r].x) * f, bf16_lo(v[r].y) * f, bf16_hi(v[r].y) * f),
                               e4m3x4(bf16_lo(v[r].z) * f, bf16_hi(v[r].z) * f, bf16_lo(v[r].w) * f, bf16_hi(v[r].w) * f));
        }
        g += step_g;
        p += step_p;
        if (p >= pairs) p -= pairs, ++g;
    }
}

// Four values of a row from column c on.  kVec (fp32): aligned to four values.
template <typename T, bool kVec>
__device__ __forceinline__ void load4(const T* row, uint32_t c, uint32_t cols, bool on, float (&v)[4])
{
    if constexpr (kVec) {
        static_assert(sizeof(T) == 4, "fp32");
        if (!on || c >= cols) {
            v[0] = v[1] = v[2] = v[3] = 0.0f;
        } else {
            const float4 q = *reinterpret_cast<const float4*>(row + c);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = on && c + i < cols ? to_float<T>(row[c + i]) : 0.0f;
    }
}

// 128 x 128 codes with their axes exchanged: thread (part, lane) holds, for
// rows 16 part .. 16 part + 15, the codes of columns 4 lane .. 4 lane + 3 (one
// word a row).  Column c's 128 bytes go to 16-byte places XOR-swizzled with its
// word, so both the writes and the reads are conflict-free.
__device__ __forceinline__ void exchange_store(const uint32_t (&w)[16], uint8_t* tile, uint32_t lane, uint32_t part)
{
    uint32_t col[4][4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {  // four rows' words -> the same four columns' words
        const uint32_t a = w[4 * g], b = w[4 * g + 1], c = w[4 * g + 2], d = w[4 * g + 3];
        const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
        const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
        col[0][g] = __byte_perm(ab0, cd0, 0x5410);
        col[1][g] = __byte_perm(ab0, cd0, 0x7632);
        col[2][g] = __byte_perm(ab1, cd1, 0x5410);
        col[3][g] = __byte_perm(ab1, cd1, 0x7632);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint4*>(tile + (4 * lane + j) * 128 + ((part ^ (lane & 7)) * 16)) =
            make_uint4(col[j][0], col[j][1], col[j][2], col[j][3]);
}

// The exchanged tile to 128-byte rows at dst (rows_left of them).
__device__ __forceinline__ void exchange_out(const uint8_t* tile, uint8_t* dst, uint32_t rows_left)
{
    for (uint32_t i = threadIdx.x; i < 128 * 8; i += kThreads) {
        const uint32_t row = i / 8, chunk = i % 8;
        if (row < rows_left)
            *reinterpret_cast<uint4*>(dst + (uint64_t)row * 128 + chunk * 16) =
                *reinterpret_cast<const uint4*>(tile + row * 128 + ((chunk ^ ((row >> 2) & 7)) * 16));
    }
}

// Blocks along the rows of each group: q [blocks][cols][128], scale [blocks][cols].
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quantize_tokens_kernel(QuantArgs a)
{
    __shared__ __align__(16) uint8_t tile[128 * 128];
    __shared__ float4 top[8][32];
    __shared__ uint32_t prefix[kMaxGroupsFp8 + 1];
    __shared__ uint2 range[kMaxGroupsFp8];
    pdl_wait();
    pdl_launch_dependents();  // the product may start: what it reads before its own wait was there before this kernel
    zero_counters(a);
    const uint32_t lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    group_prefix(a.offsets, a.rows, a.G, kFp8Block, (uint32_t)(a.rows / kFp8Block + a.G), prefix);
    for (uint32_t g = threadIdx.x; g < a.G; g += kThreads) group_rows(a.offsets, a.rows, g, &range[g].x, &range[g].y);
    __syncthreads();
    const uint32_t tiles = (uint32_t)blocks_of(a.cols);
    const uint64_t items = (uint64_t)prefix[a.G] * tiles;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t tb = (uint32_t)(it / tiles), c = (uint32_t)(it % tiles) * kFp8Block + 4 * lane;
        const uint32_t g = group_at(prefix, a.G, tb);
        const uint32_t lo = range[g].x, hi = range[g].y;
        const uint32_t r0 = lo + (tb - prefix[g]) * kFp8Block + 16 * part;
        float v[16][4], m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < 16; ++r)
            load4<T, kVec>(reinterpret_cast<const T*>(a.x) + (uint64_t)(r0 + r) * a.stride, c, a.cols, r0 + r < hi, v[r]);
#pragma unroll
        for (int r = 0; r < 16; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) m[j] = fmaxf(m[j], fabsf(v[r][j]));
        top[part][lane] = make_float4(m[0], m[1], m[2], m[3]);
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const float4 o = top[p][lane];
            m[0] = fmaxf(m[0], o.x), m[1] = fmaxf(m[1], o.y), m[2] = fmaxf(m[2], o.z), m[3] = fmaxf(m[3], o.w);
        }
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float scale;
            block_scale(m[j], &scale, &f[j]);
            if (part == 0 && c + j < a.cols) a.scale[(uint64_t)tb * a.cols + c + j] = scale;
        }
        uint32_t w[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) w[r] = e4m3x4(v[r][0] * f[0], v[r][1] * f[1], v[r][2] * f[2], v[r][3] * f[3]);
        exchange_store(w, tile, lane, part);
        __syncthreads();
        const uint32_t c0 = (uint32_t)(it % tiles) * kFp8Block;
        exchange_out(tile, a.q + ((uint64_t)tb * a.cols + c0) * kFp8Block, a.cols - c0);
    }
}

// The same for BF16 in 8-byte pieces, the values kept as they are read.  kRows:
// also the blocks along each row (q_rows, scale_rows, as quantize_rows_kernel
// makes them), so that a gradient is read once for both its uses; the rows
// outside every group get none.
template <bool kRows>
__global__ void __launch_bounds__(kThreads, kRows ? 3 : 4) quantize_tokens_bf16_kernel(QuantArgs a)
{
    __shared__ __align__(16) uint8_t tile[128 * 128];
    __shared__ uint2 top[8][32];
    __shared__ uint32_t prefix[kMaxGroupsFp8 + 1];
    __shared__ uint2 range[kMaxGroupsFp8];
    pdl_wait();
    pdl_launch_dependents();  // the product may start: what it reads before its own wait was there before this kernel
    zero_counters(a);
    const uint32_t lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    group_prefix(a.offsets, a.rows, a.G, kFp8Block, (uint32_t)(a.rows / kFp8Block + a.G), prefix);
    for (uint32_t g = threadIdx.x; g < a.G; g += kThreads) group_rows(a.offsets, a.rows, g, &range[g].x, &range[g].y);
    __syncthreads();
    const uint32_t tiles = (uint32_t)blocks_of(a.cols);
    const uint64_t items = (uint64_t)prefix[a.G] * tiles;
    for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const uint32_t tb = (uint32_t)(it / tiles), cb = (uint32_t)(it - (uint64_t)tb * tiles), c = cb * kFp8Block + 4 * lane;
        const uint32_t g = group_at(prefix, a.G, tb);
        const uint32_t lo = range[g].x, hi = range[g].y;
        const uint32_t r0 = lo + (tb - prefix[g]) * kFp8Block + 16 * part;
        const uint16_t* x = reinterpret_cast<const uint16_t*>(a.x) + (uint64_t)r0 * a.stride + c;
        uint2 v[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
            v[r] = r0 + r < hi && c < a.cols ? *reinterpret_cast<const uint2*>(x + r * a.stride) : make_uint2(0, 0);
        uint2 m = make_uint2(0, 0);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            m.x = max_pair(m.x, mag_pair(v[r].x));
            m.y = max_pair(m.y, mag_pair(v[r].y));
        }
        top[part][lane] = m;
        if (kRows) {
            uint32_t mr[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) mr[r] = max_pair(mag_pair(v[r].x), mag_pair(v[r].y));
            float scale, factor;
            block_scale(max_of_pair(max_rows<16>(mr, lane)), &scale, &factor);
            const uint32_t own = r0 + owned_row<16>(lane);
            if ((lane & 1) == 0 && own < hi) a.scale_rows[(uint64_t)cb * a.rows + own] = scale;
            uint8_t* q = a.q_rows + ((uint64_t)cb * a.rows + r0) * kFp8Block + 4 * lane;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float f = __shfl_sync(0xFFFFFFFFu, factor, owner_of(r));
                if (r0 + r < hi)
                    *reinterpret_cast<uint32_t*>(q + r * kFp8Block) =
                        e4m3x4(bf16_lo(v[r].x) * f, bf16_hi(v[r].x) * f, bf16_lo(v[r].y) * f, bf16_hi(v[r].y) * f);
            }
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const uint2 o = top[p][lane];
            m.x = max_pair(m.x, o.x);
            m.y = max_pair(m.y, o.y);
        }
        const float mag[4] = {bf16_lo(m.x), bf16_hi(m.x), bf16_lo(m.y), bf16_hi(m.y)};
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float scale;
            block_scale(mag[j], &scale, &f[j]);
            if (part == 0 && c + j < a.cols) a.scale[(uint64_t)tb * a.cols + c + j] = scale;
        }
        uint32_t w[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
            w[r] = e4m3x4(bf16_lo(v[r].x) * f[0], bf16_hi(v[r].x) * f[1], bf16_lo(v[r].y) * f[2], bf16_hi(v[r].y) * f[3]);
        exchange_store(w, tile, lane, part);
        __syncthreads();
        exchange_out(tile, a.q + ((uint64_t)tb * a.cols + cb * kFp8Block) * kFp8Block, a.cols - cb * kFp8Block);
    }
}

// One 128 x 128 block of a weight: quantised (w) or taken as it is (codes,
// scale), into the packed weight and the one with exchanged axes.
template <typename T>
__global__ void __launch_bounds__(kThreads) pack_kernel(PackArgs a)
{
    __shared__ __align__(16) uint8_t tile[128 * 128];
    __shared__ float top[8];
    pdl_wait();
    const uint32_t lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const uint32_t nbs = (uint32_t)blocks_of(a.n), kbs = (uint32_t)blocks_of(a.k);
    const uint32_t kb = blockIdx.x % kbs, nb = blockIdx.x / kbs % nbs, g = blockIdx.x / kbs / nbs;
    const uint32_t n0 = nb * kFp8Block, k0 = kb * kFp8Block, c = k0 + 4 * lane;
    const uint64_t sidx = ((uint64_t)g * nbs + nb) * kbs + kb, sidx_t = ((uint64_t)g * kbs + kb) * nbs + nb;
    uint32_t w[16];
    float scale;
    if (a.w != nullptr) {
        float v[16][4], m = 0.0f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t n = n0 + 16 * part + r;
            load4<T, false>(reinterpret_cast<const T*>(a.w) + ((uint64_t)g * a.n + n) * a.k, c, a.k, n < a.n, v[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(v[r][j]));
        }
        m = warp_max(m);
        if (lane == 0) top[part] = m;
        __syncthreads();
#pragma unroll
        for (int p = 0; p < 8; ++p) m = fmaxf(m, top[p]);
        float f;
        block_scale(m, &scale, &f);
#pragma unroll
        for (int r = 0; r < 16; ++r) w[r] = e4m3x4(v[r][0] * f, v[r][1] * f, v[r][2] * f, v[r][3] * f);
    } else {
        scale = a.scale[sidx];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t n = n0 + 16 * part + r;
            const uint8_t* row = a.codes + ((uint64_t)g * a.n + n) * a.k;
            w[r] = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n < a.n && c + j < a.k) w[r] |= (uint32_t)row[c + j] << (8 * j);
        }
    }
    if (a.packed != nullptr) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const uint32_t n = n0 + 16 * part + r;
            if (n < a.n)
                *reinterpret_cast<uint32_t*>(a.packed + (((uint64_t)g * kbs + kb) * a.n + n) * kFp8Block + 4 * lane) = w[r];
        }
        if (threadIdx.x == 0) reinterpret_cast<float*>(a.packed + weight_code_bytes(a.G, a.n, a.k))[sidx] = scale;
    }
    if (a.packed_t != nullptr) {
        exchange_store(w, tile, lane, part);
        __syncthreads();
        exchange_out(tile, a.packed_t + (((uint64_t)g * nbs + nb) * a.k + k0) * kFp8Block, a.k - k0);
        if (threadIdx.x == 0) reinterpret_cast<float*>(a.packed_t + weight_code_bytes(a.G, a.k, a.n))[sidx_t] = scale;
    }
}

// Whether rows can be read `values` at a time.
template <typename T>
bool vectored(const QuantArgs& a, uint32_t values)
{
    return a.cols % values == 0 && is_aligned(a.x, values * sizeof(T) < 16 ? values * sizeof(T) : 16) &&
           a.stride % values == 0;
}

uint32_t capped(uint64_t ctas, int sms, int per_sm)
{
    const uint64_t most = (uint64_t)sms * per_sm;
    return (uint32_t)(ctas < most ? ctas : most);
}

template <typename T>
cudaError_t quantize_rows_as(const QuantArgs& a, int sms, cudaStream_t stream)
{
    const uint64_t warps = (blocks_of(a.cols) + 1) / 2 * ((a.rows + kRowsPerWarp - 1) / kRowsPerWarp);
    const uint32_t grid = capped((warps + kThreads / 32 - 1) / (kThreads / 32), sms, 16);
    void (*kernel)(QuantArgs) = quantize_rows_kernel<T, false>;
    if (vectored<T>(a, 8)) {
        if constexpr (sizeof(T) == 2)
            kernel = quantize_rows_bf16_kernel;
        else
            kernel = quantize_rows_kernel<T, true>;
    }
    return launch_dependent(kernel, grid, kThreads, 0, stream, a);
}

template <typename T>
cudaError_t quantize_tokens_as(const QuantArgs& a, int sms, cudaStream_t stream)
{
    const uint64_t tiles = (a.rows / kFp8Block + a.G) * blocks_of(a.cols);
    void (*kernel)(QuantArgs) = quantize_tokens_kernel<T, false>;
    int per_sm = 2;
    if (vectored<T>(a, 4)) {
        if constexpr (sizeof(T) == 2) {
            kernel = a.q_rows != nullptr ? quantize_tokens_bf16_kernel<true> : quantize_tokens_bf16_kernel<false>;
            per_sm = a.q_rows != nullptr ? 3 : 4;
        } else {
            kernel = quantize_tokens_kernel<T, true>;
        }
    }
    return launch_dependent(kernel, capped(tiles, sms, per_sm), kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantArgs& a, int dtype, int sms, cudaStream_t stream)
{
    return dtype == ZCCL_BF16 ? quantize_rows_as<__nv_bfloat16>(a, sms, stream) : quantize_rows_as<float>(a, sms, stream);
}

cudaError_t launch_quantize_tokens(const QuantArgs& a, int dtype, int sms, cudaStream_t stream)
{
    return dtype == ZCCL_BF16 ? quantize_tokens_as<__nv_bfloat16>(a, sms, stream)
                              : quantize_tokens_as<float>(a, sms, stream);
}

bool quantizes_both(const QuantArgs& a, int dtype) { return dtype == ZCCL_BF16 && vectored<__nv_bfloat16>(a, 4); }

cudaError_t launch_pack(const PackArgs& a, int dtype, cudaStream_t stream)
{
    const uint32_t grid = (uint32_t)((uint64_t)a.G * blocks_of(a.n) * blocks_of(a.k));
    return dtype == ZCCL_BF16 ? launch_dependent(pack_kernel<__nv_bfloat16>, grid, kThreads, 0, stream, a)
                              : launch_dependent(pack_kernel<float>, grid, kThreads, 0, stream, a);
}

}  // namespace zccl
