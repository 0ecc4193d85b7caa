// zccl_norm_backward.cuh -- gradients of the join of a block's output with the
// residual and of the norms around it.
//
// With a row's rho = rsqrt(mean r^2 + eps), eta = rsqrt(mean y^2 + eps), k = the
// join's factor (0 where dropped), w and p the two weights:
//   d    = dr + rho (dh w - r c),     c  = rho^2 mean(dh w r)      the gradient of x
//   dy   = eta (k d p - y c'),        c' = eta^2 mean(k d p y)     (k d without post)
//   dw  += dh r rho, dp += k d y eta, dgate += (k / gate) d N(y)
// c' needs d, but its sum is that of three others, mean(k d p y) = mean(k p y dr) +
// rho (mean(k p y dh w) - c mean(k p y r)): all six sums of a row are taken at once.
//
// Bound by HBM without post and dropout: 16384 x 2048 in BF16 55 us with the join of the
// workers' sums (r, dr, dh in, dx, dy out: 6.1 TB/s, 90 % of measured), 4096 x 14336 94 us
// (6.2); with post, dropout and a gate 72 us (y read too: 5.6 TB/s), where it issues in two
// of three slots: some 390 instructions a warp and tile of 256 columns.  Rows that do not
// begin on 16 bytes: 8203 x 1001, 32-bit residual, 41.5 us (3.6 TB/s), bound by loads of
// single values.
#pragma once

#include "zccl_norm_feed.cuh"

namespace zccl {

namespace {

constexpr int kSums = 6;  // r^2, dh w r, y^2, and k p y times dr, dh w and r

struct RowFactors {
    float rho, c, eta, cy;
};
__device__ __forceinline__ RowFactors row_factors(const NormArgs& a, bool post, const float (&s)[kSums])
{
    RowFactors f{0.0f, 0.0f, 1.0f, 0.0f};
    // without dh (which reads as zero, as r does then) nothing is multiplied by these
    f.rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
    f.c = s[1] * a.inv_hidden * f.rho * f.rho;
    if (post) {
        f.eta = rsqrtf(s[2] * a.inv_hidden + a.eps);
        f.cy = (s[3] + f.rho * (s[4] - f.c * s[5])) * a.inv_hidden * f.eta * f.eta;
    }
    return f;
}

// The pieces' part of a row's sums; kp: the join's factor times p, 0 where dropped.
__device__ __forceinline__ void add_sums(float2 (&s)[kSums], bool post, const Eight& r, const Eight& hw, const Eight& up,
                                         const Eight& y, const Eight& kp)
{
    dot(s[0], r, r);
    dot(s[1], hw, r);
    if (post) {
        const Eight q = mul(kp, y);
        dot(s[2], y, y);
        dot(s[3], q, up);
        dot(s[4], q, hw);
        dot(s[5], q, r);
    }
}

// The gradient that the join sees: d = dr + rho (dh w - r c).
__device__ __forceinline__ Eight joined(const RowFactors& f, const Eight& r, const Eight& hw, const Eight& up)
{
    return fma(hw, f.rho, fma(r, -f.rho * f.c, up));
}

// y's gradient.
__device__ __forceinline__ Eight branch(bool post, const RowFactors& f, const Eight& d, const Eight& y, const Eight& kp)
{
    const Eight u = mul(kp, d);
    return post ? fma(u, f.eta, mul(y, -f.eta * f.cy)) : u;
}

template <typename T, bool kVec>
__device__ __forceinline__ Eight load_or_zero(const void* p, uint64_t first, uint32_t tile, uint32_t hidden)
{
    return p != nullptr ? load8<T, kVec>(static_cast<const T*>(p) + first, tile, hidden) : all_eight(0.0f);
}

template <bool kVec>
__device__ __forceinline__ Eight add_to(float* p, const Eight& v, bool first, uint32_t tile, uint32_t hidden)
{
    return store8<float, kVec>(p, first ? v : fma(v, 1.0f, load8<float, kVec>(p, tile, hidden)), tile, hidden);
}

// Writes a gate row's gradient, of its own type.
template <bool kVec>
__device__ __forceinline__ void store_gate(const NormArgs& a, uint32_t gate_row, const Eight& v, uint32_t tile)
{
    if (a.gate.dtype == ZCCL_BF16)
        store8<__nv_bfloat16, kVec>(static_cast<__nv_bfloat16*>(a.grad_gate) + (uint64_t)gate_row * a.hidden, v, tile, a.hidden);
    else
        store8<float, kVec>(static_cast<float*>(a.grad_gate) + (uint64_t)gate_row * a.hidden, v, tile, a.hidden);
}

// A CTA a worker; its rows are read once for the sums and once for the gradients, and
// the sums over rows stay in the workspace: any size.
template <typename Tx, typename Ty, bool kVec>
__global__ void __launch_bounds__(kTeamWarps * 32) norm_backward_long_kernel(NormArgs a)
{
    __shared__ float red[2 * 32 * kSums];
    uint32_t turn = 0;
    pdl_wait();
    const uint64_t offset = drop_offset(a.drop);
    const uint32_t warp = threadIdx.x >> 5, step = blockDim.x / 32 * kTile, wk = blockIdx.x;
    const uint32_t lo = first_row(a.rows, a.workers, wk), hi = first_row(a.rows, a.workers, wk + 1);
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    float* sums = a.sums + wk * kWeightSlots * pitch;
    float* parts = a.parts + wk * kGateSlots * pitch;
    const bool join = a.grad_y != nullptr;
    for (uint32_t t = lo; t < hi; ++t) {
        const uint32_t gate_row = t / a.gate_span;
        float2 sum[kSums] = {};
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            const Eight r = load_or_zero<Tx, kVec>(a.x, t * a.x_stride, tile, a.hidden);
            const Eight hw = mul(load_or_zero<Ty, kVec>(a.grad_h, t * a.grad_h_stride, tile, a.hidden),
                                 load_vector<kVec>(a.weight, 0, tile, a.hidden));
            const Eight up = load_or_zero<Tx, kVec>(a.grad_r, t * a.grad_r_stride, tile, a.hidden);
            Eight y = all_eight(0.0f), kp = y;
            if (a.post) {
                y = load_or_zero<Ty, kVec>(a.y, t * a.y_stride, tile, a.hidden);
                kp = mul(join_factors<kVec>(a, t, tile), load_vector<kVec>(a.post_weight, 0, tile, a.hidden));
                kp = where_kept<kVec>(join_kept<kVec>(a, offset, t, tile), kp);
            }
            add_sums(sum, a.post, r, hw, up, y, kp);
        }
        float s[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) s[i] = sum[i].x + sum[i].y;
        cta_sum<kSums>(s, red, turn);
        const RowFactors f = row_factors(a, a.post, s);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            const Eight r = load_or_zero<Tx, kVec>(a.x, t * a.x_stride, tile, a.hidden);
            const Eight dh = load_or_zero<Ty, kVec>(a.grad_h, t * a.grad_h_stride, tile, a.hidden);
            const Eight up = load_or_zero<Tx, kVec>(a.grad_r, t * a.grad_r_stride, tile, a.hidden);
            Eight d = joined(f, r, mul(dh, load_vector<kVec>(a.weight, 0, tile, a.hidden)), up);
            if (a.grad_x != nullptr) store8<Tx, kVec>(static_cast<Tx*>(a.grad_x) + (uint64_t)t * a.hidden, d, tile, a.hidden);
            if (a.grad_weight != nullptr)
                add_to<kVec>(sums + kSlotWeight * pitch, mul(dh, mul(r, f.rho)), t == lo, tile, a.hidden);
            if (!join) continue;
            const Kept<kVec> kept = join_kept<kVec>(a, offset, t, tile);
            d = where_kept<kVec>(kept, d);
            Eight y = load_or_zero<Ty, kVec>(a.y, t * a.y_stride, tile, a.hidden);
            if (!a.post) y = where_kept<kVec>(kept, y);
            const Eight k = join_factors<kVec>(a, t, tile), p = load_vector<kVec>(a.post_weight, 0, tile, a.hidden);
            const Eight e = mul(d, mul(y, f.eta));
            if (a.grad_gate != nullptr) {
                const Eight v = mul(e, mul(p, a.factor));
                const uint32_t begin = gate_row * a.gate_span, end = begin + a.gate_span;
                Eight all = v;
                if (a.gate_span > 1)
                    all = add_to<kVec>(parts + (begin < lo ? kSlotBefore : kSlotBehind) * pitch, v, t == lo || t == begin, tile, a.hidden);
                if (begin >= lo && (t + 1 == end || t + 1 == a.rows)) store_gate<kVec>(a, gate_row, all, tile);
            }
            if (a.grad_post_weight != nullptr) add_to<kVec>(sums + kSlotPost * pitch, mul(e, k), t == lo, tile, a.hidden);
            store8<Ty, kVec>(static_cast<Ty*>(a.grad_y) + (uint64_t)t * a.hidden, branch(a.post, f, d, y, mul(k, p)), tile, a.hidden);
        }
    }
}

// A team a worker; the sums over rows stay in registers.  While a gate stays the same
// the sums of p's and of the gate's gradient are the same up to a factor of each column,
//   e = sum of (kept) d y eta:   dp += scale gate e,   dgate = scale p e
// so one sum serves both, and is taken out when the gate changes.  A cluster's exchange
// takes longer than a row's arithmetic, so a cluster sums the next row (kAhead) before it
// waits for this one's sums.  kKind: as in the forward kernel.
// Rows in shared memory, where both types have 16 bits: 128 columns without a join 36 us with
// four, 48 with two.  A wider residual's would take what L1 has (with the join 92, 87).
template <typename Tx, typename Ty, int kTeam, int kPieces>
constexpr int backward_stages = kTeam == kClusterTeam                ? 3
                                : sizeof(Tx) + sizeof(Ty) > 4 ? 2
                                : in_warp<kTeam>                     ? 4
                                : kPieces == 1                       ? 3
                                                                     : 2;
template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces, int kKind>
__global__ void __launch_bounds__(in_warp<kTeam> ? kWarpsPerCta * 32
                                  : kTeam == kCtaTeam && kPieces == 1 && sizeof(Tx) + sizeof(Ty) < 8 ? kMoreWarps * 32 : kTeamWarps * 32,
                                  in_warp<kTeam> ? 2 : 1)
    norm_backward_kernel(NormArgs a)
{
    extern __shared__ uint4 smem[];
    constexpr bool kAhead = kTeam == kClusterTeam;
    constexpr int kTeamSums = kKind & 1 ? kSums : 2;
    constexpr int kStages = backward_stages<Tx, Ty, kTeam, kPieces>;
    using Rows = Feed<Tx, Ty, kVec, kPieces, kStages, true>;
    // of each warp: its rows, and its sums of p's gradient (two 16-byte parts a piece); then the teams' sums
    constexpr uint32_t kWarpParts = Rows::kWarpBytes / 16 + 2 * kPieces * 32;
    uint4* const warp_smem = smem + (threadIdx.x >> 5) * kWarpParts;
    float4* const dp = reinterpret_cast<float4*>(warp_smem) + Rows::kWarpBytes / 16 + (threadIdx.x & 31);
    TeamSum<kTeamSums, kTeam> team_sum(smem + (blockDim.x >> 5) * kWarpParts, a.status);
    pdl_wait();
    const Place at = place<kTeam, kPieces>();
    const bool join = a.grad_y != nullptr, reads_y = a.y != nullptr;
    constexpr bool post = (kKind & 1) != 0, drop = (kKind & 2) != 0;
    const uint64_t offset = drop ? drop_offset(a.drop) : 0;
    const uint32_t lo = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker) : 0;
    const uint32_t hi = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker + 1) : 0;
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const auto put_dp = [&](int n, const Eight& v) {
        dp[64 * n] = make_float4(v[0], v[1], v[2], v[3]);
        dp[64 * n + 32] = make_float4(v[4], v[5], v[6], v[7]);
    };
    const auto get_dp = [&](int n, int warps) -> Eight {
        const float4 x = dp[64 * n + warps * kWarpParts], y = dp[64 * n + 32 + warps * kWarpParts];
        return {{make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)}};
    };
    Rows rows(warp_smem, a, at, lo);
    rows.ask(a, at, lo < hi);
    Eight w[kPieces], kp[kPieces], dw[kPieces], e[kPieces];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
        w[n] = load_vector<kVec>(a.weight, 0, at.tile(n), a.hidden);
        kp[n] = dw[n] = e[n] = all_eight(0.0f);
        put_dp(n, e[n]);
    }
    Tx* gx_at = static_cast<Tx*>(a.grad_x) + (a.grad_x != nullptr ? (uint64_t)lo * a.hidden : 0);
    Ty* gy_at = static_cast<Ty*>(a.grad_y) + (join ? (uint64_t)lo * a.hidden : 0);
    // the gate row that e belongs to, and where it ends
    uint32_t gate_row = lo / a.gate_span, gate_end = a.gate.p != nullptr ? (gate_row + 1) * a.gate_span : a.rows;
    const auto set_gate = [&](uint32_t t) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n)
            kp[n] = mul(join_factors<kVec>(a, t, at.tile(n)), load_vector<kVec>(a.post_weight, 0, at.tile(n), a.hidden));
    };
    const auto prefetch_gates = [&](uint32_t t) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) prefetch_gate<kVec>(a, t, at.tile(n));
    };
    const auto take_out = [&](uint32_t t) {
        const uint32_t begin = gate_row * a.gate_span;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const uint32_t tile = at.tile(n);
            if (a.grad_post_weight != nullptr) put_dp(n, fma(e[n], join_factors<kVec>(a, begin, tile), get_dp(n, 0)));
            if (a.grad_gate == nullptr) continue;
            const Eight v = mul(e[n], mul(load_vector<kVec>(a.post_weight, 0, tile, a.hidden), a.factor));
            if (begin >= lo && (t == begin + a.gate_span || t == a.rows))
                store_gate<kVec>(a, gate_row, v, tile);
            else
                store8<float, kVec>(a.parts + ((uint64_t)at.worker * kGateSlots + (begin < lo ? kSlotBefore : kSlotBehind)) * pitch, v,
                                    tile, a.hidden);
        }
    };
    // the factors of row t's gate, 0 where dropped
    const auto masked = [&](int n, const Kept<kVec>& kept) -> Eight { return drop ? where_kept<kVec>(kept, kp[n]) : kp[n]; };
    const auto kept_of = [&](uint32_t t, int n) -> Kept<kVec> {
        return drop ? kept_piece<kVec>(a.drop, offset, t, at.tile(n)) : kept_all<kVec>();
    };
    // a row's own sums
    const auto sums_of = [&](const typename Rows::Row& row, const Kept<kVec> (&kept)[kPieces]) -> float {
        float2 sum[kSums] = {};
#pragma unroll
        for (int n = 0; n < kPieces; ++n)
            add_sums(sum, post, row.x(n), mul(row.y(n), w[n]), row.x1(n), row.y1(n), post ? masked(n, kept[n]) : kp[n]);
        float s[kTeamSums];
#pragma unroll
        for (int i = 0; i < kTeamSums; ++i) s[i] = sum[i].x + sum[i].y;
        return warp_sums<kTeamSums, team_lanes<kTeam>>(s);
    };
    const auto factors = [&]() -> RowFactors {
        float s[kSums] = {}, got[kTeamSums];
        team_sum.take(got);
#pragma unroll
        for (int i = 0; i < kTeamSums; ++i) s[i] = got[i];
        return row_factors(a, post, s);
    };
    // a row's gradients and its part of the sums over rows
    const auto gradients = [&](const typename Rows::Row& row, uint32_t t, const RowFactors& f, const Kept<kVec> (&kept)[kPieces]) {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const uint32_t tile = at.tile(n);
            const Eight r = row.x(n), dh = row.y(n);
            Eight d = joined(f, r, mul(dh, w[n]), row.x1(n)), y = all_eight(0.0f);
            dw[n] = fma(dh, mul(r, f.rho), dw[n]);
            if (a.grad_x != nullptr) store8<Tx, kVec>(gx_at, d, tile, a.hidden);
            if (!join) continue;
            if (drop) d = where_kept<kVec>(kept[n], d);
            if (reads_y) {
                y = row.y1(n);
                // what is dropped may be infinite; with post it would have spoilt the whole row
                e[n] = fma(d, mul(drop && !post ? where_kept<kVec>(kept[n], y) : y, f.eta), e[n]);
            }
            store8<Ty, kVec>(gy_at, branch(post, f, d, y, kp[n]), tile, a.hidden);
        }
        gx_at += a.hidden;
        gy_at += a.hidden;
        if (t + 1 == gate_end && join && t + 1 < hi) {
            if (reads_y) take_out(t + 1);
            ++gate_row;
            gate_end += a.gate_span;
#pragma unroll
            for (int n = 0; n < kPieces; ++n) e[n] = all_eight(0.0f);
        }
    };
    if (kAhead) {
        // sums of a row use its gate's factors before the row before it is done with its own: those are had again then
        Kept<kVec> kept[kPieces], after[kPieces];
        rows.ask(a, at, lo + 1 < hi);
        if (lo < hi) {
            if (join) set_gate(lo);
            rows.template wait<1>();
#pragma unroll
            for (int n = 0; n < kPieces; ++n) kept[n] = kept_of(lo, n);
            team_sum.put(sums_of(rows.row(1), kept));
        }
#pragma unroll 1
        for (uint32_t t = lo; t < hi; ++t) {
            rows.ask(a, at, t + 2 < hi);  // into the stage of row t - 1
            if (join && t + 2 < hi && (a.gate_span == 1 || t + 2 == gate_end)) prefetch_gates(t + 2);
            const bool more = t + 1 < hi, turns = more && join && t + 1 == gate_end;
            float s = 0.0f;
            if (more) {
                rows.template wait<1>();
                if (turns) set_gate(t + 1);
#pragma unroll
                for (int n = 0; n < kPieces; ++n) after[n] = kept_of(t + 1, n);
                s = sums_of(rows.row(1), after);
                if (turns) set_gate(t);
            }
            team_sum.wait();
            const RowFactors f = factors();
            if (more) team_sum.put(s);
            gradients(rows.row(2), t, f, kept);
            if (turns) set_gate(t + 1);
#pragma unroll
            for (int n = 0; n < kPieces; ++n) kept[n] = after[n];
        }
    } else {
        constexpr int kLater = kStages - 2;  // rows behind the one that is waited for
#pragma unroll
        for (int i = 1; i <= kLater; ++i) rows.ask(a, at, lo + i < hi);
        if (join && lo < hi) set_gate(lo);
        const uint32_t end = last_step<kTeam>(lo, hi);
#pragma unroll 1
        for (uint32_t t = lo; t < end; ++t) {
            rows.template wait<kLater>();
            const bool turns = join && t + 1 == gate_end && t + 1 < hi;
            const auto row = rows.row(kLater);
            rows.ask(a, at, t + 1 + kLater < hi);
            if (turns) prefetch_gates(t + 1);
            Kept<kVec> kept[kPieces];
#pragma unroll
            for (int n = 0; n < kPieces; ++n) kept[n] = kept_of(t, n);
            team_sum.put(sums_of(row, kept));
            team_sum.wait();
            const RowFactors f = factors();
            if (team_lanes<kTeam> == 32 || t < hi) gradients(row, t, f, kept);
            if (turns) set_gate(t + 1);
        }
    }
    team_sum.close();
    if (reads_y && lo < hi) take_out(hi);
    if (a.joined) pdl_launch_dependents();
    // the weights' sums, of a CTA's warps where each is a team
    float* const sums = a.sums + (uint64_t)(in_warp<kTeam> ? blockIdx.x : at.worker) * kWeightSlots * pitch;
    const auto put_sums = [&](int slot) {
        if (in_warp<kTeam>) __syncthreads();
        if (in_warp<kTeam> && threadIdx.x >= 32) return;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            Eight v = get_dp(n, 0);
            if (in_warp<kTeam>)
#pragma unroll 1
                for (uint32_t i = 1; i < kWarpsPerCta; ++i) v = fma(get_dp(n, i), 1.0f, v);
#pragma unroll
            for (uint32_t o = 16; o >= team_lanes<kTeam>; o /= 2)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += __shfl_xor_sync(0xFFFFFFFFu, v[j], o);
            if (team_lanes<kTeam> == 32 || threadIdx.x < team_lanes<kTeam>) store8<float, kVec>(sums + slot * pitch, v, at.tile(n), a.hidden);
        }
    };
    if (a.grad_post_weight != nullptr) put_sums(kSlotPost);
    if (a.grad_weight != nullptr) {
        if (in_warp<kTeam>) __syncthreads();
#pragma unroll
        for (int n = 0; n < kPieces; ++n) put_dp(n, dw[n]);
        put_sums(kSlotWeight);
    }
}

template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces>
NormKernel backward_kind(bool post, bool drop, uint32_t* warp_bytes)
{
    *warp_bytes = Feed<Tx, Ty, kVec, kPieces, backward_stages<Tx, Ty, kTeam, kPieces>, true>::kWarpBytes + 1024 * kPieces;
    return post ? (drop ? norm_backward_kernel<Tx, Ty, kVec, kTeam, kPieces, 3> : norm_backward_kernel<Tx, Ty, kVec, kTeam, kPieces, 1>)
                : (drop ? norm_backward_kernel<Tx, Ty, kVec, kTeam, kPieces, 2> : norm_backward_kernel<Tx, Ty, kVec, kTeam, kPieces, 0>);
}
template <typename Tx, typename Ty, bool kVec>
NormKernel backward_for(const Shape& s, bool post, bool drop, uint32_t* warp_bytes)
{
    constexpr int kMost = sizeof(Tx) == 2 && sizeof(Ty) == 2 ? 2 : 1;
    if (s.team == kWarpTeam) return backward_kind<Tx, Ty, kVec, kWarpTeam, 1>(post, drop, warp_bytes);
    if constexpr (kVec) {
        if (s.team == kHalfTeam) return backward_kind<Tx, Ty, kVec, kHalfTeam, 1>(post, drop, warp_bytes);
        if (s.team == kQuarterTeam) return backward_kind<Tx, Ty, kVec, kQuarterTeam, 1>(post, drop, warp_bytes);
    }
    if (s.team == kLong) return norm_backward_long_kernel<Tx, Ty, kVec>;
    if (s.team == kCtaTeam)
        return s.pieces == 1 ? backward_kind<Tx, Ty, kVec, kCtaTeam, 1>(post, drop, warp_bytes)
                             : backward_kind<Tx, Ty, kVec, kCtaTeam, kMost>(post, drop, warp_bytes);
    return s.pieces == 1 ? backward_kind<Tx, Ty, kVec, kClusterTeam, 1>(post, drop, warp_bytes)
                         : backward_kind<Tx, Ty, kVec, kClusterTeam, kMost>(post, drop, warp_bytes);
}

}  // namespace

template <typename Tx, typename Ty>
NormKernel norm_backward_kernel_for(const Shape& s, bool vec, bool post, bool drop, uint32_t* warp_bytes)
{
    return vec ? backward_for<Tx, Ty, true>(s, post, drop, warp_bytes) : backward_for<Tx, Ty, false>(s, post, drop, warp_bytes);
}

}  // namespace zccl
