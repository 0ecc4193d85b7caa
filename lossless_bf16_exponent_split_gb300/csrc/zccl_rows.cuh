// zccl_rows.cuh -- rows by pieces of eight values a lane, and the dropout's bits:
// shared by the norm and dropout kernels.
//
// A warp holds a tile of 256 columns of a row.  Where rows begin on 16 bytes
// (kVec) a lane's eight values are neighbours, moved 16 bytes at a time; else
// they are 32 columns apart, so that a warp's accesses stay whole lines whatever
// the rows' alignment.
#pragma once

#include "zccl_ops.cuh"

namespace zccl {

constexpr uint32_t kTile = 256;  // columns of a warp

template <bool kVec>
__device__ __forceinline__ uint32_t column(uint32_t tile, int j)
{
    const uint32_t lane = threadIdx.x & 31;
    return kVec ? tile + lane * 8 + j : tile + j * 32 + lane;
}

// Eight values of a lane as four pairs: most arithmetic on them is two at a time.
struct Eight {
    float2 v[4];
    __device__ __forceinline__ float& operator[](int j) { return j & 1 ? v[j / 2].y : v[j / 2].x; }
    __device__ __forceinline__ float operator[](int j) const { return j & 1 ? v[j / 2].y : v[j / 2].x; }
};
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ Eight all_eight(float x) { return {{twice(x), twice(x), twice(x), twice(x)}}; }
// a b, a s, a b + c, a s + c
__device__ __forceinline__ Eight mul(const Eight& a, const Eight& b)
{
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __fmul2_rn(a.v[i], b.v[i]);
    return o;
}
__device__ __forceinline__ Eight mul(const Eight& a, float s) { return mul(a, all_eight(s)); }
// a b + c with both operations rounded: products of two values an instruction would be
// fused with the addition.
__device__ __forceinline__ Eight mul_then_add(const Eight& a, const Eight& b, const Eight& c)
{
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o.v[i] = __fadd2_rn(make_float2(__fmul_rn(a.v[i].x, b.v[i].x), __fmul_rn(a.v[i].y, b.v[i].y)), c.v[i]);
    return o;
}
__device__ __forceinline__ Eight fma(const Eight& a, const Eight& b, const Eight& c)
{
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = __ffma2_rn(a.v[i], b.v[i], c.v[i]);
    return o;
}
__device__ __forceinline__ Eight fma(const Eight& a, float s, const Eight& c) { return fma(a, all_eight(s), c); }
// The sum of products, added to a pair.
__device__ __forceinline__ void dot(float2& s, const Eight& a, const Eight& b)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __ffma2_rn(a.v[i], b.v[i], s);
}

__device__ __forceinline__ Eight widen(const uint4& q)
{
    return {{make_float2(bf16_lo(q.x), bf16_hi(q.x)), make_float2(bf16_lo(q.y), bf16_hi(q.y)),
             make_float2(bf16_lo(q.z), bf16_hi(q.z)), make_float2(bf16_lo(q.w), bf16_hi(q.w))}};
}

// Eight neighbours on 16 bytes.
__device__ __forceinline__ Eight load_near(const __nv_bfloat16* p) { return widen(*reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ Eight load_near(const float* p)
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
__device__ __forceinline__ uint4 round_eight(const Eight& v)
{
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_near(__nv_bfloat16* p, const Eight& v) { *reinterpret_cast<uint4*>(p) = round_eight(v); }
__device__ __forceinline__ void store_near(float* p, const Eight& v)
{
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A lane's eight values of a tile as they are held in memory, to be widened later.
template <typename T, bool kVec>
struct Piece;
template <>
struct Piece<__nv_bfloat16, true> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* row, uint32_t tile, uint32_t cols)
    {
        const uint32_t c = column<true>(tile, 0);
        q = c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ Eight get() const { return widen(q); }
};
template <>
struct Piece<__nv_bfloat16, false> {
    uint4 q;
    __device__ __forceinline__ void load(const __nv_bfloat16* row, uint32_t tile, uint32_t cols)
    {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + column<false>(tile, 0);
        uint32_t w[8];
        if (tile + kTile <= cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = p[32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = column<false>(tile, j) < cols ? p[32 * j] : 0;
        }
        q = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    __device__ __forceinline__ Eight get() const { return widen(q); }
};
template <bool kVec>
struct Piece<float, kVec> {
    Eight v;
    __device__ __forceinline__ void load(const float* row, uint32_t tile, uint32_t cols)
    {
        if (kVec) {
            const uint32_t c = column<true>(tile, 0);
            v = c < cols ? load_near(row + c) : all_eight(0.0f);
        } else if (tile + kTile <= cols) {
            const float* p = row + column<false>(tile, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = p[32 * j];
        } else {
            const float* p = row + column<false>(tile, 0);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = column<false>(tile, j) < cols ? p[32 * j] : 0.0f;
        }
    }
    __device__ __forceinline__ Eight get() const { return v; }
};

template <typename T, bool kVec>
__device__ __forceinline__ Eight load8(const T* row, uint32_t tile, uint32_t cols)
{
    Piece<T, kVec> p;
    p.load(row, tile, cols);
    return p.get();
}

// Stores v rounded to T; what was stored.
template <typename T, bool kVec>
__device__ __forceinline__ Eight store8(T* row, const Eight& v, uint32_t tile, uint32_t cols)
{
    if (sizeof(T) == 2) {
        const uint4 q = round_eight(v);
        if (kVec) {
            const uint32_t c = column<true>(tile, 0);
            if (c < cols) *reinterpret_cast<uint4*>(row + c) = q;
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            uint16_t* p = reinterpret_cast<uint16_t*>(row) + column<false>(tile, 0);
            if (tile + kTile <= cols) {
#pragma unroll
                for (int j = 0; j < 8; ++j) p[32 * j] = (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (column<false>(tile, j) < cols) p[32 * j] = (uint16_t)(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
            }
        }
        return widen(q);
    }
    if (kVec) {
        const uint32_t c = column<true>(tile, 0);
        if (c < cols) store_near(reinterpret_cast<float*>(row + c), v);
    } else {
        float* p = reinterpret_cast<float*>(row) + column<false>(tile, 0);
        if (tile + kTile <= cols) {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[32 * j] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (column<false>(tile, j) < cols) p[32 * j] = v[j];
        }
    }
    return v;
}

// A vector of weights or a gate's row, of either type; all ones where there is none.
struct Vector {
    const void* p;
    int dtype;
};
template <bool kVec>
__device__ __forceinline__ Eight load_vector(const Vector& a, uint64_t first, uint32_t tile, uint32_t cols)
{
    if (a.p == nullptr) return all_eight(1.0f);
    if (a.dtype == ZCCL_BF16) return load8<__nv_bfloat16, kVec>(static_cast<const __nv_bfloat16*>(a.p) + first, tile, cols);
    return load8<float, kVec>(static_cast<const float*>(a.p) + first, tile, cols);
}

// ---- dropout ----------------------------------------------------------------
struct DropArgs {
    uint32_t below;      // of 2^16: how many of an element's values drop it; 0: no dropout
    float gain;          // 1 / (1 - below / 2^16)
    uint32_t key[10][2]; // of each round
    uint64_t offset;
    const uint64_t* more;  // device: added to the offset
};

inline bool drop_args(float p, uint64_t seed, uint64_t offset, const uint64_t* more, DropArgs* d)
{
    if (!(p >= 0.0f && p <= 1.0f) || !is_aligned(more, 8)) return false;
    const double below = floor((double)p * 65536.0 + 0.5);
    d->below = (uint32_t)below;
    d->gain = below < 65536.0 ? (float)(1.0 / (1.0 - below / 65536.0)) : 0.0f;
    for (uint32_t r = 0; r < 10; ++r) {
        d->key[r][0] = (uint32_t)seed + r * 0x9E3779B9u;
        d->key[r][1] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
    }
    d->offset = offset;
    d->more = more;
    return true;
}

__device__ __forceinline__ uint64_t drop_offset(const DropArgs& d)
{
    return d.offset + (d.more != nullptr ? *d.more : 0);
}

// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): ten rounds, in each the two
// even words are multiplied out to 64 bits by a constant, and the halves take each
// other's places with the odd words and the round's key.
__device__ __forceinline__ uint4 philox(uint4 c, const DropArgs& d)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ d.key[r][0], (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ d.key[r][1], (uint32_t)a);
    }
    return c;
}

// Which of a lane's eight values stay: the 16 bits of two at a time are compared.
template <bool kVec>
struct Kept;
template <>
struct Kept<true> {
    uint4 w;
    uint32_t below;  // in the upper half
    // of values 2 i and 2 i + 1
    __device__ __forceinline__ void pair(int i, bool* lo, bool* hi) const
    {
        const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
        *lo = x << 16 >= below;
        *hi = x >= below;
    }
};
template <>
struct Kept<false> {
    uint32_t bits;
    __device__ __forceinline__ void pair(int i, bool* lo, bool* hi) const
    {
        *lo = (bits >> (2 * i)) & 1u;
        *hi = (bits >> (2 * i + 1)) & 1u;
    }
};

// The bits of the eight columns from 8 block on.
__device__ __forceinline__ Kept<true> kept_block(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t block)
{
    Kept<true> k;
    k.w = philox(make_uint4(block, row, (uint32_t)offset, (uint32_t)(offset >> 32)), d);
    k.below = d.below << 16;
    if (d.below == 65536) k.w = make_uint4(0, 0, 0, 0), k.below = 1;  // nothing stays
    return k;
}

// Which of the lane's values of a tile stay.  The lanes hold a block each; where a
// lane's columns are 32 apart their bits come from the lanes that have them, so all
// lanes take part.
template <bool kVec>
__device__ __forceinline__ Kept<kVec> kept_piece(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t tile);
template <>
__device__ __forceinline__ Kept<true> kept_piece<true>(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t tile)
{
    return kept_block(d, offset, row, column<true>(tile, 0) / 8);
}
template <>
__device__ __forceinline__ Kept<false> kept_piece<false>(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t tile)
{
    const uint32_t lane = threadIdx.x & 31;
    const Kept<true> mine = kept_block(d, offset, row, tile / 8 + lane);
    uint32_t block = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bool lo, hi;
        mine.pair(i, &lo, &hi);
        block |= (lo ? 1u << (2 * i) : 0u) | (hi ? 2u << (2 * i) : 0u);
    }
    Kept<false> k{0};
#pragma unroll
    for (int j = 0; j < 8; ++j) k.bits |= ((__shfl_sync(0xFFFFFFFFu, block, j * 4 + lane / 8) >> (lane % 8)) & 1u) << j;
    return k;
}
// All stay.
template <bool kVec>
__device__ __forceinline__ Kept<kVec> kept_all();
template <>
__device__ __forceinline__ Kept<true> kept_all<true>() { return {make_uint4(0, 0, 0, 0), 0}; }
template <>
__device__ __forceinline__ Kept<false> kept_all<false>() { return {0xFFu}; }

template <bool kVec>
__device__ __forceinline__ Eight where_kept(const Kept<kVec>& k, const Eight& a, const Eight& b)
{
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bool lo, hi;
        k.pair(i, &lo, &hi);
        o.v[i] = make_float2(lo ? a.v[i].x : b.v[i].x, hi ? a.v[i].y : b.v[i].y);
    }
    return o;
}
template <bool kVec>
__device__ __forceinline__ Eight where_kept(const Kept<kVec>& k, const Eight& a)
{
    return where_kept<kVec>(k, a, all_eight(0.0f));
}

}  // namespace zccl
