// zccl_norm_feed.cuh -- the norm kernels' rows on their way from memory.
#pragma once

#include "zccl_norm.h"

namespace zccl {

// A worker's rows: x and y of the row at hand and of those behind it; backward r (as x),
// dh (as y), dr and y (as x1, y1).  What the call does not have reads as zero.
// kStages: rows in shared memory, or 0 for one in registers.
// Rows on 16 bytes may come by asynchronous copies into places of the thread's own, so that
// no thread waits for another's and no registers are held.  A lane's addresses move on
// from row to row; what it copies lies at constant distances from them.  16-bit values go
// past L1, of which the rows in shared memory leave little (gradients of 4096 x 14336 94
// us, 117 through it); a lane's two parts of 32-bit values share sectors, which L1 keeps for
// the second (2048 columns 56 us, 85 past it).
template <bool kPast, int kTo, int kFrom>
__device__ __forceinline__ void copy_16(uint32_t to, const char* from, uint32_t bytes)
{
    if (kPast)
        asm volatile("cp.async.cg.shared.global [%0+%3], [%1+%4], 16, %2;" ::"r"(to), "l"(from), "r"(bytes), "n"(kTo), "n"(kFrom) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0+%3], [%1+%4], 16, %2;" ::"r"(to), "l"(from), "r"(bytes), "n"(kTo), "n"(kFrom) : "memory");
}
template <typename Tx, typename Ty, bool kVec, int kPieces, int kStages, bool kBackward>
struct Feed {
    static_assert(kVec, "rows on 16 bytes");
    static constexpr int kX = sizeof(Tx) / 2, kY = sizeof(Ty) / 2, kAll = (kX + kY) * (kBackward ? 2 : 1);  // 16-byte parts of a piece
    static constexpr uint32_t kWarpBytes = kStages * kPieces * kAll * 512;
    static constexpr uint32_t kStage = kPieces * kAll * 32;  // 16-byte parts of a warp's stage
    const uint4* const mine;  // a warp's parts, 32 lanes each, one behind the other
    uint32_t to;              // the stage that the next row goes to
    uint32_t asked = 0;
    const char *x, *y, *x1, *y1;
    uint32_t bytes[kPieces];  // 16, or 0 where a piece lies behind the row's end
    __device__ __forceinline__ Feed(uint4* warp_smem, const NormArgs& a, const Place& place, uint32_t t)
        : mine(warp_smem + (threadIdx.x & 31)), to(smem_addr(warp_smem + (threadIdx.x & 31)))
    {
        for (uint32_t i = 0; i < kStages * kStage; i += 32) warp_smem[i + (threadIdx.x & 31)] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int n = 0; n < kPieces; ++n) bytes[n] = column<true>(place.tile(n), 0) < a.hidden ? 16 : 0;
        const uint64_t c = bytes[0] > 0 ? column<true>(place.tile(0), 0) : 0;
        x = static_cast<const char*>(a.x) + (t * a.x_stride + c) * sizeof(Tx);
        if (kBackward) {
            y = static_cast<const char*>(a.grad_h) + (t * a.grad_h_stride + c) * sizeof(Ty);
            x1 = static_cast<const char*>(a.grad_r) + (t * a.grad_r_stride + c) * sizeof(Tx);
            y1 = static_cast<const char*>(a.y) + (t * a.y_stride + c) * sizeof(Ty);
        } else {
            y = static_cast<const char*>(a.y) + (t * a.y_stride + c) * sizeof(Ty);
        }
    }
    template <typename T, int kPart>
    __device__ __forceinline__ void copy(const char*& from, uint64_t stride)
    {
        copy_piece<T, kPart, 0>(from);
        if constexpr (kPieces == 2) copy_piece<T, kPart, 1>(from);
        from += stride * sizeof(T);
    }
    template <typename T, int kPart, int n>
    __device__ __forceinline__ void copy_piece(const char* from)
    {
        copy_16<sizeof(T) == 2, (n * kAll + kPart) * 512, n * (int)(kTile * sizeof(T))>(to, from, bytes[n]);
        if constexpr (sizeof(T) == 4) copy_16<false, (n * kAll + kPart + 1) * 512, n * (int)(kTile * sizeof(T)) + 16>(to, from, bytes[n]);
    }
    // Asks for the next row (there: it is one of the worker's).
    __device__ __forceinline__ void ask(const NormArgs& a, const Place&, bool there)
    {
        if (there) {
            if constexpr (kBackward) {
                if (a.grad_h != nullptr) {
                    copy<Tx, 0>(x, a.x_stride);
                    copy<Ty, kX>(y, a.grad_h_stride);
                }
                if (a.grad_r != nullptr) copy<Tx, kX + kY>(x1, a.grad_r_stride);
                if (a.y != nullptr) copy<Ty, 2 * kX + kY>(y1, a.y_stride);
            } else {
                copy<Tx, 0>(x, a.x_stride);
                if (a.y != nullptr) copy<Ty, kX>(y, a.y_stride);
            }
        }
        const bool last = asked + 1 == kStages;
        asked = last ? 0 : asked + 1;
        to = last ? to - (kStages - 1) * kStage * 16 : to + kStage * 16;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Until all but the last kLater rows that were asked for are there.
    template <int kLater>
    __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLater) : "memory");
    }
    struct Row {
        const uint4* at;
        template <typename T>
        __device__ __forceinline__ Eight read(int n, int part) const
        {
            const uint4* p = at + (n * kAll + part) * 32;
            if (sizeof(T) == 2) return widen(*p);
            const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 32);
            return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
        }
        __device__ __forceinline__ Eight x(int n) const { return read<Tx>(n, 0); }
        __device__ __forceinline__ Eight y(int n) const { return read<Ty>(n, kX); }
        __device__ __forceinline__ Eight x1(int n) const { return read<Tx>(n, kX + kY); }
        __device__ __forceinline__ Eight y1(int n) const { return read<Ty>(n, 2 * kX + kY); }
    };
    // The row that was asked for before the last `later` ones.
    __device__ __forceinline__ Row row(uint32_t later) const
    {
        const uint32_t stage = asked + kStages - 1 - later;
        return {mine + (stage >= kStages ? stage - kStages : stage) * kStage};
    }
};

// Rows that begin anywhere: 32-bit values a lane's own ones by one, 16-bit ones by the
// words that hold them, from the one that holds a tile's first value on.  A value then is
// a half of a word later in a row that begins in the middle of one, and another lane may
// have copied it.
template <typename T>
constexpr uint32_t kLooseBytes = sizeof(T) == 4 ? 1024 : 528;  // of a tile: 256 values, or 129 words
template <int kTo, int kFrom>
__device__ __forceinline__ void copy_4(uint32_t to, const char* from, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0+%3], [%1+%4], 4, %2;" ::"r"(to), "l"(from), "r"(bytes), "n"(kTo), "n"(kFrom) : "memory");
}
template <typename Tx, typename Ty, int kPieces, int kStages, bool kBackward>
struct Feed<Tx, Ty, false, kPieces, kStages, kBackward> {
    static constexpr int kX = kLooseBytes<Tx>, kY = kLooseBytes<Ty>, kAll = (kX + kY) * (kBackward ? 2 : 1), kStage = kAll * kPieces;
    static constexpr uint32_t kWarpBytes = kStages * kStage;
    const char* const mine;  // the warp's stages
    uint32_t asked = 0;      // the stage that the next row goes to
    uint32_t shifts = 0;     // of each stage four bits: whether x, y, x1, y1 begin in the middle of a word
    const char *x, *y, *x1, *y1;  // the first tile of the row that is asked for next
    const uint32_t left;          // columns of the row from the tile on
    __device__ __forceinline__ Feed(uint4* warp_smem, const NormArgs& a, const Place& place, uint32_t t)
        : mine(reinterpret_cast<const char*>(warp_smem)), left(place.tile(0) < a.hidden ? a.hidden - place.tile(0) : 0)
    {
        for (uint32_t i = threadIdx.x & 31; i < kWarpBytes / 16; i += 32) warp_smem[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
        const uint64_t c = left > 0 ? place.tile(0) : 0;
        x = static_cast<const char*>(a.x) + (t * a.x_stride + c) * sizeof(Tx);
        if (kBackward) {
            y = static_cast<const char*>(a.grad_h) + (t * a.grad_h_stride + c) * sizeof(Ty);
            x1 = static_cast<const char*>(a.grad_r) + (t * a.grad_r_stride + c) * sizeof(Tx);
            y1 = static_cast<const char*>(a.y) + (t * a.y_stride + c) * sizeof(Ty);
        } else {
            y = static_cast<const char*>(a.y) + (t * a.y_stride + c) * sizeof(Ty);
        }
    }
    template <typename T, int kPart, int kBit>
    __device__ __forceinline__ void copy(const char*& from, uint64_t stride)
    {
        const uint32_t lane = threadIdx.x & 31, shift = sizeof(T) == 4 ? 0 : (uint32_t)(reinterpret_cast<uint64_t>(from) >> 1) & 1u;
        const uint32_t to = smem_addr(mine) + asked * kStage + kPart + lane * 4;
        const char* p = from - 2 * shift + lane * 4;  // (the first word's other half is not looked at)
        copy_piece<T>(to, p, shift, left);
        if constexpr (kPieces == 2) copy_piece<T>(to + kAll, p + kTile * sizeof(T), shift, left > kTile ? left - kTile : 0);
        if (sizeof(T) == 2) {
            const uint32_t at = 4 * asked + kBit;
            shifts = (shifts & ~(1u << at)) | shift << at;
        }
        from += stride * sizeof(T);
    }
    template <typename T>
    static __device__ __forceinline__ void copy_piece(uint32_t to, const char* p, uint32_t shift, uint32_t left)
    {
        const uint32_t lane = threadIdx.x & 31;
        if constexpr (sizeof(T) == 4) {
            const auto all = [&](auto size) {
                copy_4<0, 0>(to, p, size(0)), copy_4<128, 128>(to, p, size(1)), copy_4<256, 256>(to, p, size(2));
                copy_4<384, 384>(to, p, size(3)), copy_4<512, 512>(to, p, size(4)), copy_4<640, 640>(to, p, size(5));
                copy_4<768, 768>(to, p, size(6)), copy_4<896, 896>(to, p, size(7));
            };
            if (left >= kTile)
                all([](uint32_t) { return 4u; });
            else
                all([&](uint32_t j) { return j * 32 + lane < left ? 4u : 0u; });
        } else {
            const auto all = [&](auto size) {
                copy_4<0, 0>(to, p, size(lane)), copy_4<128, 128>(to, p, size(32 + lane));
                copy_4<256, 256>(to, p, size(64 + lane)), copy_4<384, 384>(to, p, size(96 + lane));
            };
            if (left >= kTile) {
                all([](uint32_t) { return 4u; });
                if (lane == 0 && shift) copy_4<512, 512>(to, p, 2);
            } else {
                const uint32_t halves = left > 0 ? shift + left : 0;  // those of the words that are wanted
                all([&](uint32_t word) { return 2 * word + 1 < halves ? 4u : 2 * word < halves ? 2u : 0u; });
            }
        }
    }
    // Asks for the next row (there: it is one of the worker's).
    __device__ __forceinline__ void ask(const NormArgs& a, const Place&, bool there)
    {
        __syncwarp();  // all lanes have read the stage's last row
        if (there) {
            if constexpr (kBackward) {
                if (a.grad_h != nullptr) {
                    copy<Tx, 0, 0>(x, a.x_stride);
                    copy<Ty, kX, 1>(y, a.grad_h_stride);
                }
                if (a.grad_r != nullptr) copy<Tx, kX + kY, 2>(x1, a.grad_r_stride);
                if (a.y != nullptr) copy<Ty, 2 * kX + kY, 3>(y1, a.y_stride);
            } else {
                copy<Tx, 0, 0>(x, a.x_stride);
                if (a.y != nullptr) copy<Ty, kX, 1>(y, a.y_stride);
            }
        }
        asked = asked + 1 == kStages ? 0 : asked + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Until all but the last kLater rows that were asked for are there.
    template <int kLater>
    __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kLater) : "memory");
        __syncwarp();
    }
    struct Row {
        const char* at;
        uint32_t shifts;
        template <typename T>
        __device__ __forceinline__ Eight read(int n, int part, int bit) const
        {
            const uint32_t lane = threadIdx.x & 31;
            Eight v;
            if (sizeof(T) == 4) {
                const float* p = reinterpret_cast<const float*>(at + n * kAll + part) + lane;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = p[32 * j];
            } else {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(at + n * kAll + part) + lane + ((shifts >> bit) & 1u);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float((uint32_t)p[32 * j] << 16);
            }
            return v;
        }
        __device__ __forceinline__ Eight x(int n) const { return read<Tx>(n, 0, 0); }
        __device__ __forceinline__ Eight y(int n) const { return read<Ty>(n, kX, 1); }
        __device__ __forceinline__ Eight x1(int n) const { return read<Tx>(n, kX + kY, 2); }
        __device__ __forceinline__ Eight y1(int n) const { return read<Ty>(n, 2 * kX + kY, 3); }
    };
    // The row that was asked for before the last `later` ones.
    __device__ __forceinline__ Row row(uint32_t later) const
    {
        const uint32_t back = asked + kStages - 1 - later, stage = back >= kStages ? back - kStages : back;
        return {mine + stage * kStage, shifts >> (4 * stage)};
    }
};

// Forward, rows of two tiles a warp come into registers: the row that is read, and the
// next one.
template <typename Tx, typename Ty, int kPieces>
struct Feed<Tx, Ty, true, kPieces, 0, false> {
    static constexpr uint32_t kWarpBytes = 0;
    struct Row {
        Piece<Tx, true> px[kPieces];
        Piece<Ty, true> py[kPieces];
        __device__ __forceinline__ Eight x(int n) const { return px[n].get(); }
        __device__ __forceinline__ Eight y(int n) const { return py[n].get(); }
    };
    Row next;
    const Tx* x;  // the row that is asked for next
    const Ty* y;
    __device__ __forceinline__ Feed(uint4*, const NormArgs& a, const Place&, uint32_t t)
        : next{}, x(static_cast<const Tx*>(a.x) + t * a.x_stride), y(static_cast<const Ty*>(a.y) + t * a.y_stride)
    {
    }
    __device__ __forceinline__ void ask(const NormArgs& a, const Place& place, bool there)
    {
        if (!there) return;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            next.px[n].load(x, place.tile(n), a.hidden);
            if (a.y != nullptr) next.py[n].load(y, place.tile(n), a.hidden);
        }
        x += a.x_stride;
        y += a.y_stride;
    }
    template <int kLater>
    __device__ __forceinline__ void wait()
    {
    }
    __device__ __forceinline__ Row row(uint32_t) const { return next; }
};

}  // namespace zccl
