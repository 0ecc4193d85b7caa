// zccl_fp8.h -- layouts and launch interface of the block-scaled e4m3 products
// (not part of the public ABI).
//
// An operand of a product is held block-major: its reduction axis is cut into
// blocks of 128, and block b of row r is the 128 bytes at (b * rows + r) * 128,
// its scale at b * rows + r (activations) or one per 128 rows (weights).  The
// last block is padded with zeros.  A tile of an operand is then one
// contiguous run of memory, whatever the sizes, and one swizzled TMA box.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "zccl_internal.h"

namespace zccl {

constexpr uint32_t kFp8Block = 128;
constexpr uint32_t kMaxGroupsFp8 = ZCCL_MAX_EXPERTS;

__host__ __device__ inline uint64_t blocks_of(uint64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

// The packed weight [groups][rows][red]: codes [groups][blocks(red)][rows][128],
// then scales [groups][blocks(rows)][blocks(red)].
__host__ __device__ inline uint64_t weight_code_bytes(uint64_t groups, uint64_t rows, uint64_t red)
{
    return groups * blocks_of(red) * rows * kFp8Block;
}
__host__ __device__ inline uint64_t weight_bytes(uint64_t groups, uint64_t rows, uint64_t red)
{
    return weight_code_bytes(groups, rows, red) + 4 * groups * blocks_of(rows) * blocks_of(red);
}

// out rows [offsets[g], offsets[g+1]) = rows of `a` times the transpose of group
// g's weight; rows outside every group get zeros.
struct MatmulArgs {
    const uint8_t* a;        // codes [KB][rows][128]
    const float* sa;         // [KB][rows]
    const uint8_t* b;        // packed weight codes [G][KB][n][128]
    const float* sb;         // [G][blocks(n)][KB]
    const int32_t* offsets;  // [G + 1], or nullptr: one group of all rows
    uint32_t rows, n, KB, G;
    void* out;               // [rows][n]
    int out_f32;
    uint32_t* ticket;        // zero before the launch
    uint32_t split;          // matmul_split()
    uint32_t* counters;      // kJoinCounters, zero before the launch
    float* parts;            // part_bytes()
    uint32_t* status;
};

// out[g] [m][n] = sum over the group's token blocks: `a` codes [blocks][m][128]
// with scales [blocks][m], `b` codes [blocks][n][128] with scales [blocks][n].
struct WgradArgs {
    const uint8_t* a;
    const float* sa;
    const uint8_t* b;
    const float* sb;
    const int32_t* offsets;
    uint32_t rows, m, n, G;
    uint32_t blocks;         // token blocks there is room for: rows / 128 + G
    void* out;               // [G][m][n]
    int out_f32;
    uint32_t* ticket;        // zero before the launch
    uint32_t split;          // wgrad_split()
    uint32_t* counters;      // kJoinCounters, zero before the launch
    float* parts;            // part_bytes()
    uint32_t* status;
};

struct QuantArgs {
    const void* x;
    uint64_t stride;
    uint32_t rows, cols;
    uint8_t* q;
    float* scale;
    const int32_t* offsets;  // along rows: the groups
    uint32_t G;
    uint8_t* q_rows;         // along rows: also the blocks of each row, or nullptr
    float* scale_rows;
    uint32_t* ticket;        // zeroed for the product that follows,
    uint32_t* counters;      // and so are these kJoinCounters, or nullptr
};

struct PackArgs {
    const void* w;           // BF16 or fp32 [G][n][k], or nullptr
    const uint8_t* codes;    // e4m3 [G][n][k]
    const float* scale;      // [G][blocks(n)][blocks(k)]
    uint32_t G, n, k;
    uint8_t* packed;         // may be nullptr
    uint8_t* packed_t;       // may be nullptr: the weight with its two axes exchanged
};

// Parts that the reduction of a product's tiles is cut into, and the room for
// their sums (0 without parts).
constexpr uint32_t kJoinParts = 160, kJoinCounters = 8 * kJoinParts;
uint32_t matmul_split(uint64_t rows, uint64_t n, uint64_t k, uint32_t groups);
uint32_t wgrad_split(uint64_t rows, uint64_t m, uint64_t n, uint32_t groups);
uint64_t part_bytes(uint32_t split);

cudaError_t launch_matmul(const MatmulArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_wgrad(const WgradArgs& a, int sms, cudaStream_t stream);
// Few rows a group: whether launch_small() is the faster of the two.
bool takes_small(uint64_t rows, uint64_t n, uint64_t k, uint32_t groups, int sms);
cudaError_t launch_small(const MatmulArgs& a, int sms, cudaStream_t stream);
cudaError_t launch_quantize_rows(const QuantArgs& a, int dtype, int sms, cudaStream_t stream);
cudaError_t launch_quantize_tokens(const QuantArgs& a, int dtype, int sms, cudaStream_t stream);
// Whether launch_quantize_tokens can make the blocks of each row, too.
bool quantizes_both(const QuantArgs& a, int dtype);
cudaError_t launch_pack(const PackArgs& a, int dtype, cudaStream_t stream);

}  // namespace zccl
