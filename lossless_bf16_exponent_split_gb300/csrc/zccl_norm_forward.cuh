// zccl_norm_forward.cuh -- the join of a block's output with the residual and the norm
// of the next block's input.
//
// Bound by HBM: x and y in, r and h out, once.  What comes between is issue: a row costs a
// warp about 95 instructions besides its tiles' 70 (the sums' exchange, the loop), post 40 a
// tile, dropout 70.  16384 x 2048 in BF16: 43.7 us with the join alone (6.1 TB/s, 91 % of
// measured), 48 with post and dropout; 4096 x 14336 (clusters of two) 85 us (5.5 TB/s);
// one row of 4096: 2.1 us.
#pragma once

#include "zccl_norm_feed.cuh"

namespace zccl {

namespace {

// A CTA a row, read once for each of its sums: any size.
template <typename Tx, typename Ty, bool kVec>
__global__ void __launch_bounds__(kTeamWarps * 32) norm_long_kernel(NormArgs a)
{
    __shared__ float red[2 * 32];
    uint32_t turn = 0;
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t warp = threadIdx.x >> 5, step = blockDim.x / 32 * kTile;
    for (uint32_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
        const Tx* x = static_cast<const Tx*>(a.x) + t * a.x_stride;
        const Ty* y = static_cast<const Ty*>(a.y) + t * a.y_stride;
        Tx* r = static_cast<Tx*>(a.r) + (uint64_t)t * a.hidden;
        float eta = 1.0f;
        float2 sum = twice(0.0f);
        if (a.y != nullptr && a.post) {
            for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
                const Eight v = load8<Ty, kVec>(y, tile, a.hidden);
                dot(sum, v, v);
            }
            float s[1] = {sum.x + sum.y};
            cta_sum<1>(s, red, turn);
            eta = rsqrtf(s[0] * a.inv_hidden + a.eps);
            sum = twice(0.0f);
        }
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            Eight v = load8<Tx, kVec>(x, tile, a.hidden);
            if (a.y != nullptr) {
                const Eight k = mul(join_factors<kVec>(a, t, tile), load_vector<kVec>(a.post_weight, 0, tile, a.hidden));
                const Eight b = mul(load8<Ty, kVec>(y, tile, a.hidden), eta);
                v = where_kept<kVec>(join_kept<kVec>(a, offset, t, tile), mul_then_add(k, b, v), v);
                v = store8<Tx, kVec>(r, v, tile, a.hidden);
            }
            dot(sum, v, v);
        }
        if (a.h == nullptr) continue;
        float s[1] = {sum.x + sum.y};
        cta_sum<1>(s, red, turn);
        const float rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            const Eight v = mul(load8<Tx, kVec>(a.y != nullptr ? r : x, tile, a.hidden), rho);
            store8<Ty, kVec>(static_cast<Ty*>(a.h) + (uint64_t)t * a.hidden, mul(v, load_vector<kVec>(a.weight, 0, tile, a.hidden)), tile,
                             a.hidden);
        }
    }
}

// A team a worker: a row is read once and stays in registers, with others on their way;
// weights and the gate stay there too.  kKind: which of post (1) and dropout (2) the
// call has.
// Two rows more on their way in shared memory; with two tiles a warp, of rows on 16 bytes,
// one in registers is as good (2048 columns in BF16 47.4 us, 48.3; in 32 bits with a BF16
// block 45.9, 34.6).
template <bool kVec, int kPieces>
constexpr int forward_stages = kPieces == 1 || !kVec ? 3 : 0;
template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces, int kKind>
__global__ void __launch_bounds__(kPieces == 1 ? 768 : kTeamWarps * 32) norm_kernel(NormArgs a)
{
    extern __shared__ uint4 smem[];
    __shared__ __align__(16) char red[in_warp<kTeam> ? 16 : kTeamBytes];
    using Rows = Feed<Tx, Ty, kVec, kPieces, forward_stages<kVec, kPieces>, false>;
    TeamSum<1, kTeam> team_sum(red, a.status);
    pdl_wait();
    const Place at = place<kTeam, kPieces>();
    const bool join = a.y != nullptr, normed = a.h != nullptr;
    constexpr bool post = (kKind & 1) != 0, drop = (kKind & 2) != 0;
    const uint64_t offset = drop ? drop_offset(a.drop) : 0;
    const uint32_t lo = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker) : 0;
    const uint32_t hi = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker + 1) : 0;
    const uint32_t end = last_step<kTeam>(lo, hi);
    Tx* r_at = static_cast<Tx*>(a.r) + (join ? (uint64_t)lo * a.hidden : 0);
    Ty* h_at = static_cast<Ty*>(a.h) + (normed ? (uint64_t)lo * a.hidden : 0);
    Rows rows(smem + (threadIdx.x >> 5) * (Rows::kWarpBytes / 16), a, at, lo);
    constexpr int kLater = forward_stages<kVec, kPieces> == 3 ? 1 : 0;  // rows behind the one that is waited for
#pragma unroll
    for (int i = 0; i <= kLater; ++i) rows.ask(a, at, lo + i < hi);
    Eight w[kPieces], k[kPieces];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) w[n] = load_vector<kVec>(a.weight, 0, at.tile(n), a.hidden);
    uint32_t gate_end = lo;  // where the gate changes
    for (uint32_t t = lo; t < end; ++t) {
        const bool live = team_lanes<kTeam> == 32 || t < hi;
        rows.template wait<kLater>();
        const auto row = rows.row(kLater);
        Eight x[kPieces], y[kPieces];
#pragma unroll
        for (int n = 0; n < kPieces; ++n) x[n] = row.x(n), y[n] = row.y(n);
        rows.ask(a, at, t + kLater + 1 < hi);
        if (join) {
            if (t == gate_end && live) {
                // the join's factor of each column, with the weight of the norm after the block
#pragma unroll
                for (int n = 0; n < kPieces; ++n)
                    k[n] = mul(join_factors<kVec>(a, t, at.tile(n)), load_vector<kVec>(a.post_weight, 0, at.tile(n), a.hidden));
                gate_end = a.gate.p != nullptr ? (t / a.gate_span + 1) * a.gate_span : a.rows;
            }
            if (t + 1 == gate_end && t + 1 < hi)
#pragma unroll
                for (int n = 0; n < kPieces; ++n) prefetch_gate<kVec>(a, t + 1, at.tile(n));
            if (post) {
                float2 sum = twice(0.0f);
#pragma unroll
                for (int n = 0; n < kPieces; ++n) dot(sum, y[n], y[n]);
                float s[1] = {sum.x + sum.y};
                team_sum(s);
                const float eta = rsqrtf(s[0] * a.inv_hidden + a.eps);
#pragma unroll
                for (int n = 0; n < kPieces; ++n) y[n] = mul(y[n], eta);
            }
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                // the product rounded by itself: without post r then has the bits of the formula's operations in their order
                const Eight r = mul_then_add(k[n], y[n], x[n]);
                x[n] = drop ? where_kept<kVec>(kept_piece<kVec>(a.drop, offset, t, at.tile(n)), r, x[n]) : r;
                if (live) x[n] = store8<Tx, kVec>(r_at, x[n], at.tile(n), a.hidden);
            }
            r_at += a.hidden;
        }
        if (!normed) continue;
        float2 sum = twice(0.0f);
#pragma unroll
        for (int n = 0; n < kPieces; ++n) dot(sum, x[n], x[n]);
        float s[1] = {sum.x + sum.y};
        team_sum(s);
        const float rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
#pragma unroll
        for (int n = 0; n < kPieces; ++n)
            if (live) store8<Ty, kVec>(h_at, mul(mul(x[n], rho), w[n]), at.tile(n), a.hidden);
        h_at += a.hidden;
    }
    team_sum.close();
}

template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces>
NormKernel norm_kind(bool post, bool drop, uint32_t* warp_bytes)
{
    *warp_bytes = Feed<Tx, Ty, kVec, kPieces, forward_stages<kVec, kPieces>, false>::kWarpBytes;
    return post ? (drop ? norm_kernel<Tx, Ty, kVec, kTeam, kPieces, 3> : norm_kernel<Tx, Ty, kVec, kTeam, kPieces, 1>)
                : (drop ? norm_kernel<Tx, Ty, kVec, kTeam, kPieces, 2> : norm_kernel<Tx, Ty, kVec, kTeam, kPieces, 0>);
}
template <typename Tx, typename Ty, bool kVec>
NormKernel norm_for(const Shape& s, bool post, bool drop, uint32_t* warp_bytes)
{
    constexpr int kMost = sizeof(Tx) == 2 && sizeof(Ty) == 2 ? 2 : 1;
    if (s.team == kWarpTeam) return norm_kind<Tx, Ty, kVec, kWarpTeam, 1>(post, drop, warp_bytes);
    if constexpr (kVec) {
        if (s.team == kHalfTeam) return norm_kind<Tx, Ty, kVec, kHalfTeam, 1>(post, drop, warp_bytes);
        if (s.team == kQuarterTeam) return norm_kind<Tx, Ty, kVec, kQuarterTeam, 1>(post, drop, warp_bytes);
    }
    if (s.team == kLong) return norm_long_kernel<Tx, Ty, kVec>;
    if (s.team == kCtaTeam)
        return s.pieces == 1 ? norm_kind<Tx, Ty, kVec, kCtaTeam, 1>(post, drop, warp_bytes) : norm_kind<Tx, Ty, kVec, kCtaTeam, kMost>(post, drop, warp_bytes);
    return s.pieces == 1 ? norm_kind<Tx, Ty, kVec, kClusterTeam, 1>(post, drop, warp_bytes)
                         : norm_kind<Tx, Ty, kVec, kClusterTeam, kMost>(post, drop, warp_bytes);
}

}  // namespace

template <typename Tx, typename Ty>
NormKernel norm_kernel_for(const Shape& s, bool vec, bool post, bool drop, uint32_t* warp_bytes)
{
    return vec ? norm_for<Tx, Ty, true>(s, post, drop, warp_bytes) : norm_for<Tx, Ty, false>(s, post, drop, warp_bytes);
}

}  // namespace zccl
