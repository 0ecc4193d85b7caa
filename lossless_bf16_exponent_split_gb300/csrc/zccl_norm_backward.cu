// zccl_norm_backward.cu -- gradients of the join of a block's output with the
// residual and of the norms around it.
//
// With a row's rho = rsqrt(mean r^2 + eps), eta = rsqrt(mean y^2 + eps), k = the
// join's factor (0 where dropped), w and p the two weights:
//   d    = dr + rho (dh w - r c),     c  = rho^2 mean(dh w r)      the gradient of x
//   dy   = eta (k d p - y c'),        c' = eta^2 mean(k d p y)     (k d without post)
//   dw  += dh r rho, dp += k d y eta, dgate += (k / gate) d N(y)
// c' needs d, but its sum is that of three others, mean(k d p y) = mean(k p y dr) +
// rho (mean(k p y dh w) - c mean(k p y r)): all six sums of a row are taken at once.
#include "zccl_norm.h"

namespace zccl {

namespace {

constexpr int kSums = 6;  // r^2, dh w r, y^2, and k p y times dr, dh w and r

struct RowFactors {
    float rho, c, eta, cy;
};
__device__ __forceinline__ RowFactors row_factors(const NormArgs& a, const float (&s)[kSums])
{
    RowFactors f{0.0f, 0.0f, 1.0f, 0.0f};
    if (a.grad_h != nullptr) {
        f.rho = rsqrtf(s[0] * a.inv_hidden + a.eps);
        f.c = s[1] * a.inv_hidden * f.rho * f.rho;
    }
    if (a.post) {
        f.eta = rsqrtf(s[2] * a.inv_hidden + a.eps);
        f.cy = (s[3] + f.rho * (s[4] - f.c * s[5])) * a.inv_hidden * f.eta * f.eta;
    }
    return f;
}

// The pieces' part of a row's sums; kp: the join's factor times p, 0 where dropped.
__device__ __forceinline__ void add_sums(float2 (&s)[kSums], const NormArgs& a, const Eight& r, const Eight& hw, const Eight& up,
                                         const Eight& y, const Eight& kp)
{
    if (a.grad_h != nullptr) {
        dot(s[0], r, r);
        dot(s[1], hw, r);
    }
    if (a.post) {
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
__device__ __forceinline__ Eight branch(const NormArgs& a, const RowFactors& f, const Eight& d, const Eight& y, const Eight& kp)
{
    const Eight u = mul(kp, d);
    return a.post ? fma(u, f.eta, mul(y, -f.eta * f.cy)) : u;
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
__device__ __forceinline__ void store_gate(const NormArgs& a, uint64_t gate_row, const Eight& v, uint32_t tile)
{
    if (a.gate.dtype == ZCCL_BF16)
        store8<__nv_bfloat16, kVec>(static_cast<__nv_bfloat16*>(a.grad_gate) + gate_row * a.hidden, v, tile, a.hidden);
    else
        store8<float, kVec>(static_cast<float*>(a.grad_gate) + gate_row * a.hidden, v, tile, a.hidden);
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
    const uint64_t lo = first_row(a.rows, a.workers, wk), hi = first_row(a.rows, a.workers, wk + 1);
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    float* sums = a.sums + wk * kWeightSlots * pitch;
    float* parts = a.parts + wk * kGateSlots * pitch;
    const bool join = a.grad_y != nullptr;
    for (uint64_t t = lo; t < hi; ++t) {
        const uint64_t gate_row = t / a.gate_span;
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
            add_sums(sum, a, r, hw, up, y, kp);
        }
        float s[kSums];
#pragma unroll
        for (int i = 0; i < kSums; ++i) s[i] = sum[i].x + sum[i].y;
        cta_sum<kSums>(s, red, turn);
        const RowFactors f = row_factors(a, s);
        for (uint32_t tile = warp * kTile; tile < a.hidden; tile += step) {
            const Eight r = load_or_zero<Tx, kVec>(a.x, t * a.x_stride, tile, a.hidden);
            const Eight dh = load_or_zero<Ty, kVec>(a.grad_h, t * a.grad_h_stride, tile, a.hidden);
            const Eight up = load_or_zero<Tx, kVec>(a.grad_r, t * a.grad_r_stride, tile, a.hidden);
            const Eight d = joined(f, r, mul(dh, load_vector<kVec>(a.weight, 0, tile, a.hidden)), up);
            if (a.grad_x != nullptr) store8<Tx, kVec>(static_cast<Tx*>(a.grad_x) + t * a.hidden, d, tile, a.hidden);
            if (a.grad_weight != nullptr)
                add_to<kVec>(sums + kSlotWeight * pitch, mul(dh, mul(r, f.rho)), t == lo, tile, a.hidden);
            if (!join) continue;
            const Eight y = load_or_zero<Ty, kVec>(a.y, t * a.y_stride, tile, a.hidden);
            const Eight k = join_factors<kVec>(a, t, tile), p = load_vector<kVec>(a.post_weight, 0, tile, a.hidden);
            const Kept<kVec> kept = join_kept<kVec>(a, offset, t, tile);
            const Eight e = where_kept<kVec>(kept, mul(d, mul(y, f.eta)));
            if (a.grad_gate != nullptr) {
                const Eight v = mul(e, mul(p, a.factor));
                const uint64_t begin = gate_row * a.gate_span, end = begin + a.gate_span;
                Eight all = v;
                if (a.gate_span > 1)
                    all = add_to<kVec>(parts + (begin < lo ? kSlotBefore : kSlotBehind) * pitch, v, t == lo || t == begin, tile, a.hidden);
                if (begin >= lo && (t + 1 == end || t + 1 == a.rows)) store_gate<kVec>(a, gate_row, all, tile);
            }
            if (a.grad_post_weight != nullptr) add_to<kVec>(sums + kSlotPost * pitch, mul(e, k), t == lo, tile, a.hidden);
            store8<Ty, kVec>(static_cast<Ty*>(a.grad_y) + t * a.hidden, branch(a, f, d, y, where_kept<kVec>(kept, mul(k, p))), tile,
                             a.hidden);
        }
    }
}

// A worker's rows on their way: r, dr, dh and y of the row at hand and of the next one.
// What the call does not have reads as zero.
template <typename Tx, typename Ty, bool kVec, int kPieces>
struct Feed;

// Rows on 16 bytes come by asynchronous copies into places of the thread's own, so that
// no thread waits for another's and no registers are held.
__device__ __forceinline__ void copy_16(uint4* to, const void* from, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(to)), "l"(from), "r"(there ? 16 : 0) : "memory");
}
template <typename Tx, typename Ty, int kPieces>
struct Feed<Tx, Ty, true, kPieces> {
    static constexpr int kX = sizeof(Tx) / 2, kY = sizeof(Ty) / 2, kAll = 2 * kX + 2 * kY;  // 16-byte parts of a piece
    static constexpr uint32_t kThreadBytes = 2 * kPieces * kAll * 16;
    uint4* mine;
    uint32_t turn = 0;
    __device__ __forceinline__ uint4* at(uint32_t turn, int n, int part) const
    {
        return mine + ((turn * kPieces + n) * kAll + part) * blockDim.x;
    }
    __device__ __forceinline__ Feed(uint4* smem, const NormArgs& a) : mine(smem + threadIdx.x)
    {
        for (int i = 0; i < 2 * kPieces * kAll; ++i) mine[i * blockDim.x] = make_uint4(0, 0, 0, 0);
    }
    template <typename T>
    __device__ __forceinline__ void copy(const void* p, uint64_t row, uint64_t stride, uint32_t turn, int n, int part, uint32_t tile,
                                         uint32_t hidden)
    {
        if (p == nullptr) return;
        const uint32_t c = column<true>(tile, 0);
        const T* from = static_cast<const T*>(p) + row * stride;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i)
            copy_16(at(turn, n, part + i), c < hidden ? from + c + 4 * i : from, c < hidden);
    }
    // Asks for row t, to be had after the next wait().
    __device__ __forceinline__ void ask(const NormArgs& a, const Place& place, uint64_t t)
    {
        turn ^= 1;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            copy<Tx>(a.x, t, a.x_stride, turn, n, 0, place.tile(n), a.hidden);
            copy<Tx>(a.grad_r, t, a.grad_r_stride, turn, n, kX, place.tile(n), a.hidden);
            copy<Ty>(a.grad_h, t, a.grad_h_stride, turn, n, 2 * kX, place.tile(n), a.hidden);
            copy<Ty>(a.y, t, a.y_stride, turn, n, 2 * kX + kY, place.tile(n), a.hidden);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // Until the row that was asked for is there; the caller asks for the next one then and
    // reads this one.
    __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
    template <typename T>
    __device__ __forceinline__ Eight read(uint32_t turn, int n, int part) const
    {
        if (sizeof(T) == 2) return widen(*at(turn, n, part));
        const float4 x = *reinterpret_cast<const float4*>(at(turn, n, part)), y = *reinterpret_cast<const float4*>(at(turn, n, part + 1));
        return {{make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)}};
    }
    struct Row {
        const Feed& f;
        uint32_t turn;
        __device__ __forceinline__ Eight r(int n) const { return f.template read<Tx>(turn, n, 0); }
        __device__ __forceinline__ Eight up(int n) const { return f.template read<Tx>(turn, n, kX); }
        __device__ __forceinline__ Eight dh(int n) const { return f.template read<Ty>(turn, n, 2 * kX); }
        __device__ __forceinline__ Eight y(int n) const { return f.template read<Ty>(turn, n, 2 * kX + kY); }
    };
    __device__ __forceinline__ Row row() const { return {*this, turn}; }
};

// Others by loads of single values into registers.
template <typename Tx, typename Ty, int kPieces>
struct Feed<Tx, Ty, false, kPieces> {
    static constexpr uint32_t kThreadBytes = 0;
    Piece<Tx, false> pr[kPieces], pu[kPieces];
    Piece<Ty, false> ph[kPieces], py[kPieces];
    __device__ __forceinline__ Feed(uint4*, const NormArgs&) : pr{}, pu{}, ph{}, py{} {}
    __device__ __forceinline__ void ask(const NormArgs& a, const Place& place, uint64_t t)
    {
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            if (a.x != nullptr) pr[n].load(static_cast<const Tx*>(a.x) + t * a.x_stride, place.tile(n), a.hidden);
            if (a.grad_r != nullptr) pu[n].load(static_cast<const Tx*>(a.grad_r) + t * a.grad_r_stride, place.tile(n), a.hidden);
            if (a.grad_h != nullptr) ph[n].load(static_cast<const Ty*>(a.grad_h) + t * a.grad_h_stride, place.tile(n), a.hidden);
            if (a.y != nullptr) py[n].load(static_cast<const Ty*>(a.y) + t * a.y_stride, place.tile(n), a.hidden);
        }
    }
    __device__ __forceinline__ void wait() {}
    struct Row {
        Piece<Tx, false> pr[kPieces], pu[kPieces];
        Piece<Ty, false> ph[kPieces], py[kPieces];
        __device__ __forceinline__ Eight r(int n) const { return pr[n].get(); }
        __device__ __forceinline__ Eight up(int n) const { return pu[n].get(); }
        __device__ __forceinline__ Eight dh(int n) const { return ph[n].get(); }
        __device__ __forceinline__ Eight y(int n) const { return py[n].get(); }
    };
    __device__ __forceinline__ Row row() const
    {
        Row o;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) o.pr[n] = pr[n], o.pu[n] = pu[n], o.ph[n] = ph[n], o.py[n] = py[n];
        return o;
    }
};

// A team a worker; the sums over rows stay in registers.  While a gate stays the same
// the sums of p's and of the gate's gradient are the same up to a factor of each column,
//   e = sum of (kept) d y eta:   dp += scale gate e,   dgate = scale p e
// so one sum serves both, and is taken out when the gate changes.
template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces>
__global__ void __launch_bounds__(kTeam == kWarpTeam ? kWarpsPerCta * 32 : kTeamWarps * 32, kTeam == kWarpTeam ? 2 : 1)
    norm_backward_kernel(NormArgs a)
{
    extern __shared__ uint4 smem[];
    using Rows = Feed<Tx, Ty, kVec, kPieces>;
    // a thread's sums of p's gradient (two 16-byte parts a piece), and the teams' sums
    float4* const post = reinterpret_cast<float4*>(smem) + Rows::kThreadBytes / 16 * blockDim.x + threadIdx.x;
    float* const red = reinterpret_cast<float*>(smem) + (Rows::kThreadBytes + 32 * kPieces) / 4 * blockDim.x;
    uint32_t turn = 0;
    pdl_wait();
    const Place at = place<kTeam>();
    const uint64_t offset = drop_offset(a.drop);
    const uint64_t lo = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker) : 0;
    const uint64_t hi = at.worker < a.workers ? first_row(a.rows, a.workers, at.worker + 1) : 0;
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const bool join = a.grad_y != nullptr;
    const auto put_post = [&](int n, const Eight& v) {
        post[(2 * n) * blockDim.x] = make_float4(v[0], v[1], v[2], v[3]);
        post[(2 * n + 1) * blockDim.x] = make_float4(v[4], v[5], v[6], v[7]);
    };
    const auto get_post = [&](int n, int warps) -> Eight {
        const float4 x = post[(2 * n) * blockDim.x + 32 * warps], y = post[(2 * n + 1) * blockDim.x + 32 * warps];
        return {{make_float2(x.x, x.y), make_float2(x.z, x.w), make_float2(y.x, y.y), make_float2(y.z, y.w)}};
    };
    Rows rows(smem, a);
    Eight w[kPieces], kp[kPieces], dw[kPieces], e[kPieces];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
        w[n] = load_vector<kVec>(a.weight, 0, at.tile(n), a.hidden);
        kp[n] = dw[n] = e[n] = all_eight(0.0f);
        put_post(n, e[n]);
    }
    if (lo < hi) rows.ask(a, at, lo);
    uint64_t gate_row = lo / a.gate_span, gate_end = lo;  // where the gate changes
    const auto take_out = [&](uint64_t t) {
        const uint64_t begin = gate_row * a.gate_span;
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const uint32_t tile = at.tile(n);
            if (a.grad_post_weight != nullptr) put_post(n, fma(e[n], join_factors<kVec>(a, begin, tile), get_post(n, 0)));
            if (a.grad_gate == nullptr) continue;
            const Eight v = mul(e[n], mul(load_vector<kVec>(a.post_weight, 0, tile, a.hidden), a.factor));
            if (begin >= lo && (t == begin + a.gate_span || t == a.rows))
                store_gate<kVec>(a, gate_row, v, tile);
            else
                store8<float, kVec>(a.parts + ((uint64_t)at.worker * kGateSlots + (begin < lo ? kSlotBefore : kSlotBehind)) * pitch, v,
                                    tile, a.hidden);
        }
    };
    for (uint64_t t = lo; t < hi; ++t) {
        rows.wait();
        const auto row = rows.row();
        if (t + 1 < hi) rows.ask(a, at, t + 1);
        if (join && t == gate_end) {
            if (t > lo) {
                take_out(t);
                ++gate_row;
            }
            gate_end = a.gate.p != nullptr ? (gate_row + 1) * a.gate_span : a.rows;
#pragma unroll
            for (int n = 0; n < kPieces; ++n) {
                kp[n] = mul(join_factors<kVec>(a, t, at.tile(n)), load_vector<kVec>(a.post_weight, 0, at.tile(n), a.hidden));
                e[n] = all_eight(0.0f);
            }
        }
        Kept<kVec> kept[kPieces];
#pragma unroll
        for (int n = 0; n < kPieces; ++n) kept[n] = join ? join_kept<kVec>(a, offset, t, at.tile(n)) : kept_all<kVec>();
        RowFactors f{0.0f, 0.0f, 1.0f, 0.0f};
        if (a.grad_h != nullptr || a.post) {
            float2 sum[kSums] = {};
#pragma unroll
            for (int n = 0; n < kPieces; ++n)
                add_sums(sum, a, row.r(n), mul(row.dh(n), w[n]), row.up(n), row.y(n), where_kept<kVec>(kept[n], kp[n]));
            float s[kSums];
#pragma unroll
            for (int i = 0; i < kSums; ++i) s[i] = sum[i].x + sum[i].y;
            if (a.post) {
                team_sum<kSums, kTeam>(s, red, turn);
            } else {
                float two[2] = {s[0], s[1]};
                team_sum<2, kTeam>(two, red, turn);
                s[0] = two[0], s[1] = two[1];
            }
            f = row_factors(a, s);
        }
#pragma unroll
        for (int n = 0; n < kPieces; ++n) {
            const uint32_t tile = at.tile(n);
            const Eight r = row.r(n), dh = row.dh(n), d = joined(f, r, mul(dh, w[n]), row.up(n));
            dw[n] = fma(dh, mul(r, f.rho), dw[n]);
            if (a.grad_x != nullptr) store8<Tx, kVec>(static_cast<Tx*>(a.grad_x) + t * a.hidden, d, tile, a.hidden);
            if (!join) continue;
            const Eight y = row.y(n);
            e[n] = fma(d, mul(where_kept<kVec>(kept[n], y), f.eta), e[n]);
            store8<Ty, kVec>(static_cast<Ty*>(a.grad_y) + t * a.hidden, branch(a, f, d, y, where_kept<kVec>(kept[n], kp[n])), tile,
                             a.hidden);
        }
    }
    if (join && lo < hi && a.y != nullptr) take_out(hi);
    pdl_launch_dependents();
    // the weights' sums, of a CTA's warps where each is a team
    uint64_t group = at.worker;
    if (kTeam == kWarpTeam) {
        group = blockIdx.x;
        __syncthreads();
        Eight all = all_eight(0.0f);
        if (threadIdx.x < 32)
            for (uint32_t i = 0; i < kWarpsPerCta; ++i) all = fma(get_post(0, i), 1.0f, all);
        __syncthreads();
        put_post(0, dw[0]);
        __syncthreads();
        if (threadIdx.x >= 32) return;
        dw[0] = all_eight(0.0f);
        for (uint32_t i = 0; i < kWarpsPerCta; ++i) dw[0] = fma(get_post(0, i), 1.0f, dw[0]);
        put_post(0, all);
    }
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
        float* sums = a.sums + group * kWeightSlots * pitch;
        if (a.grad_weight != nullptr) store8<float, kVec>(sums + kSlotWeight * pitch, dw[n], at.tile(n), a.hidden);
        if (a.grad_post_weight != nullptr) store8<float, kVec>(sums + kSlotPost * pitch, get_post(n, 0), at.tile(n), a.hidden);
    }
}

// Adds the partial sums up: blockIdx.y = 0, 1 a weight's, 2 + i those of a gate row that
// several workers have parts of: gate row i (kByRow), or the one that goes on behind
// worker i's rows.
constexpr uint32_t kJoinRows = 32;  // partial sums of a column that are added side by side

template <bool kByRow>
__global__ void __launch_bounds__(32 * kJoinRows) norm_join_kernel(NormArgs a, int weight_dtype)
{
    __shared__ float red[kJoinRows][33];
    pdl_wait();
    const uint64_t pitch = (a.hidden + 7) / 8 * 8;
    const uint32_t lane = threadIdx.x & 31, sub = threadIdx.x >> 5, col = blockIdx.x * 32 + lane, job = blockIdx.y;
    float sum = 0.0f;
    void* out;
    int dtype = weight_dtype;
    uint64_t at = col;
    if (job < 2) {
        out = job == 0 ? a.grad_weight : a.grad_post_weight;
        if (out == nullptr) return;
        const float* p = a.sums + job * pitch + col;
        if (col < a.hidden)
#pragma unroll 8
            for (uint32_t g = sub; g < a.groups; g += kJoinRows) sum += p[g * kWeightSlots * pitch];
    } else {
        uint64_t gate_row = job - 2;
        if (!kByRow) {
            const uint64_t next = first_row(a.rows, a.workers, job - 2 + 1);
            gate_row = (next - 1) / a.gate_span;
        }
        const uint64_t begin = gate_row * a.gate_span, end = begin + a.gate_span < a.rows ? begin + a.gate_span : a.rows;
        const uint32_t from = worker_of(a.rows, a.workers, begin), to = worker_of(a.rows, a.workers, end - 1);
        if (from == to || (!kByRow && from != job - 2)) return;  // the worker's own, or another's to add up
        if (col < a.hidden)
#pragma unroll 4
            for (uint32_t w = from + sub; w <= to; w += kJoinRows)
                sum += a.parts[((uint64_t)w * kGateSlots + (w == from ? kSlotBehind : kSlotBefore)) * pitch + col];
        out = a.grad_gate;
        dtype = a.gate.dtype;
        at += gate_row * a.hidden;
    }
    red[sub][lane] = sum;
    __syncthreads();
    if (sub != 0 || col >= a.hidden) return;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinRows; ++i) sum += red[i][lane];
    if (dtype == ZCCL_BF16)
        static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(sum);
    else
        static_cast<float*>(out)[at] = sum;
}

cudaError_t launch_join(const NormArgs& a, int weight_dtype, cudaStream_t stream)
{
    const bool gate = a.grad_gate != nullptr && a.gate_span > 1 && a.workers > 1;
    if (a.grad_weight == nullptr && a.grad_post_weight == nullptr && !gate) return cudaSuccess;
    const uint64_t gate_rows = (a.rows + a.gate_span - 1) / a.gate_span;
    const bool by_row = gate_rows < a.workers;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.hidden + 31) / 32, !gate ? 2 : by_row ? 2 + (uint32_t)gate_rows : 2 + a.workers - 1);
    cfg.blockDim = dim3(32 * kJoinRows);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, by_row ? norm_join_kernel<true> : norm_join_kernel<false>, a, weight_dtype);
}

using NormKernel = void (*)(NormArgs);
struct Launch {
    NormKernel kernel;
    uint32_t thread_bytes;  // of shared memory
};

template <typename Tx, typename Ty, bool kVec, int kTeam, int kPieces>
Launch team_launch()
{
    return {norm_backward_kernel<Tx, Ty, kVec, kTeam, kPieces>, Feed<Tx, Ty, kVec, kPieces>::kThreadBytes + 32 * kPieces};
}
template <typename Tx, typename Ty, bool kVec>
Launch backward_for(const Shape& s)
{
    constexpr int kMost = kVec && sizeof(Tx) == 2 && sizeof(Ty) == 2 ? 2 : 1;
    if (s.team == kWarpTeam) return team_launch<Tx, Ty, kVec, kWarpTeam, 1>();
    if (s.team == kLong) return {norm_backward_long_kernel<Tx, Ty, kVec>, 0};
    if (s.team == kCtaTeam)
        return s.pieces == 1 ? team_launch<Tx, Ty, kVec, kCtaTeam, 1>() : team_launch<Tx, Ty, kVec, kCtaTeam, kMost>();
    return s.pieces == 1 ? team_launch<Tx, Ty, kVec, kClusterTeam, 1>() : team_launch<Tx, Ty, kVec, kClusterTeam, kMost>();
}
template <typename Tx>
Launch backward_for(int dtype, bool vec, const Shape& s)
{
    if (dtype == ZCCL_BF16) return vec ? backward_for<Tx, __nv_bfloat16, true>(s) : backward_for<Tx, __nv_bfloat16, false>(s);
    return vec ? backward_for<Tx, float, true>(s) : backward_for<Tx, float, false>(s);
}

}  // namespace

zccl_status_t launch_norm_backward(NormArgs& a, int x_dtype, int dtype, int weight_dtype, bool vec, cudaStream_t stream)
{
    const Shape s = norm_shape(a.hidden, a.rows, vec && x_dtype == ZCCL_BF16 && dtype == ZCCL_BF16);
    a.workers = s.workers;
    a.groups = s.grid / s.ctas;
    a.parts = a.sums + (uint64_t)a.groups * kWeightSlots * ((a.hidden + 7) / 8 * 8);
    const Launch l = x_dtype == ZCCL_BF16 ? backward_for<__nv_bfloat16>(dtype, vec, s) : backward_for<float>(dtype, vec, s);
    const uint32_t threads = s.warps * 32;
    const size_t smem = s.team == kLong ? 0 : threads * l.thread_bytes + kTeamRed * sizeof(float);
    cudaError_t e = cudaSuccess;
    if (smem > 48 << 10) e = cudaFuncSetAttribute(l.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        e = s.team == kClusterTeam ? launch_clusters(l.kernel, s.grid, threads, smem, s.ctas, stream, a)
                                   : launch_dependent(l.kernel, s.grid, threads, smem, stream, a);
    if (e == cudaSuccess) e = launch_join(a, weight_dtype, stream);
    return launched(e);
}

}  // namespace zccl
