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

__device__ __forceinline__ void widen(float (&v)[8], const uint4& q)
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
}

// A piece as it is held in memory, to be widened later: eight values of T (kVec) or
// their widened form.
template <typename T, bool kVec>
struct Piece {
    float v[8];
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
    __device__ __forceinline__ void load(const T* row, uint32_t tile, uint32_t cols)
    {
        if (kVec) {
            const uint32_t c = column<true>(tile, 0);
            if (c < cols) {
                const float4* p = reinterpret_cast<const float4*>(row + c);
                const float4 a = p[0], b = p[1];
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t c = column<false>(tile, j);
                v[j] = c < cols ? to_float<T>(row[c]) : 0.0f;
            }
        }
    }
    __device__ __forceinline__ void get(float (&o)[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = v[j];
    }
};
template <>
struct Piece<__nv_bfloat16, true> {
    uint4 q;
    __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const __nv_bfloat16* row, uint32_t tile, uint32_t cols)
    {
        const uint32_t c = column<true>(tile, 0);
        q = c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&o)[8]) const { widen(o, q); }
};

template <typename T, bool kVec>
__device__ __forceinline__ void load8(float (&v)[8], const T* row, uint32_t tile, uint32_t cols)
{
    Piece<T, kVec> p;
    p.load(row, tile, cols);
    p.get(v);
}

// Rounds v to T, leaves in v what was stored, and stores it.
template <typename T, bool kVec>
__device__ __forceinline__ void store8(T* row, float (&v)[8], uint32_t tile, uint32_t cols)
{
    if (kVec) {
        const uint32_t c = column<true>(tile, 0);
        if (sizeof(T) == 2) {
            const uint4 q = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
            if (c < cols) *reinterpret_cast<uint4*>(row + c) = q;
            widen(v, q);
        } else if (c < cols) {
            float4* p = reinterpret_cast<float4*>(row + c);
            p[0] = make_float4(v[0], v[1], v[2], v[3]);
            p[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t c = column<false>(tile, j);
            const T t = from_float<T>(v[j]);
            if (c < cols) row[c] = t;
            v[j] = to_float<T>(t);
        }
    }
}

// A vector of weights or a gate's row, of either type; all ones where there is none.
struct Vector {
    const void* p;
    int dtype;
};
template <bool kVec>
__device__ __forceinline__ void load_vector(float (&v)[8], const Vector& a, uint64_t first, uint32_t tile, uint32_t cols)
{
    if (a.p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    } else if (a.dtype == ZCCL_BF16) {
        load8<__nv_bfloat16, kVec>(v, static_cast<const __nv_bfloat16*>(a.p) + first, tile, cols);
    } else {
        load8<float, kVec>(v, static_cast<const float*>(a.p) + first, tile, cols);
    }
}

// ---- dropout ----------------------------------------------------------------
struct DropArgs {
    uint32_t below;  // of 2^16: how many of an element's values drop it; 0: no dropout
    float gain;      // 1 / (1 - below / 2^16)
    uint32_t key[2];
    uint64_t offset;
    const uint64_t* more;  // device: added to the offset
};

inline bool drop_args(float p, uint64_t seed, uint64_t offset, const uint64_t* more, DropArgs* d)
{
    if (!(p >= 0.0f && p <= 1.0f) || !is_aligned(more, 8)) return false;
    const double below = floor((double)p * 65536.0 + 0.5);
    d->below = (uint32_t)below;
    d->gain = below < 65536.0 ? (float)(1.0 / (1.0 - below / 65536.0)) : 0.0f;
    d->key[0] = (uint32_t)seed;
    d->key[1] = (uint32_t)(seed >> 32);
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
// other's places with the odd words and the key, which moves on by a constant.
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1)
{
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c.x * 0xD2511F53u, b = (uint64_t)c.z * 0xCD9E8D57u;
        c = make_uint4((uint32_t)(b >> 32) ^ c.y ^ k0, (uint32_t)b, (uint32_t)(a >> 32) ^ c.w ^ k1, (uint32_t)a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return c;
}

// Which of the eight columns of a block (bit j: column 8 block + j) of a row stay.
__device__ __forceinline__ uint32_t kept_block(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t block)
{
    const uint4 u = philox(make_uint4(block, row, (uint32_t)offset, (uint32_t)(offset >> 32)), d.key[0], d.key[1]);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t kept = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        kept |= ((w[i] & 0xFFFFu) >= d.below ? 1u << (2 * i) : 0u) | ((w[i] >> 16) >= d.below ? 2u << (2 * i) : 0u);
    return kept;
}

// Which of the lane's eight values of a tile stay (bit j: its j-th).  The lanes hold
// a block each; where a lane's columns are 32 apart their bits come from the lanes
// that have them, so all lanes take part.
template <bool kVec>
__device__ __forceinline__ uint32_t kept_piece(const DropArgs& d, uint64_t offset, uint32_t row, uint32_t tile)
{
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t block = kept_block(d, offset, row, tile / 8 + lane);
    if (kVec) return block;
    uint32_t kept = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        kept |= ((__shfl_sync(0xFFFFFFFFu, block, j * 4 + lane / 8) >> (lane % 8)) & 1u) << j;
    return kept;
}

}  // namespace zccl
