// zccl_route.cu -- the router: scores, choice and weights of each token's
// experts, and the gradient of the weights.
//
// L lanes of a warp hold one token's logits in registers, expert e in lane
// e % L, so a row is read once and nothing of it is written but the K chosen.
// With E logits a token the bytes are few (16384 x 64 BF16: 2 MB, 0.3 us of HBM
// time); what a call costs are the integer instructions of the choice, at half
// the issue rate: K rounds of a maximum over the lanes' values and the lanes.
// Fewer lanes a token and more tokens a warp share a round's instructions.
// The gradient waits for its loads: the choice, then the chosen logits, or all of
// them for a softmax that is not renormalised.  Top 8 of 64 for 16384 tokens (BF16,
// softmax): 7.1 us forward, 3.0 backward (4.0 not renormalised); top 8 of 256 in 8
// groups for 8192 (sigmoid): 13.6 and 5.5.
#include <cmath>

#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr int kRouteWarps = 4;
constexpr uint32_t kMaxGroups = 32;
constexpr float kInf = __builtin_huge_valf();

struct RouteArgs {
    const void* logits;
    uint64_t stride;
    const float* bias;
    uint64_t tokens;
    uint32_t E, K, G, top_groups;
    int sigmoid, renorm;
    float scale;
    uint32_t per, inv_per;  // experts of a group, and 2^20 / per rounded up
    int32_t* idx;
    float* weights;
    uint32_t* status;
    // backward
    const float* grad_weights;
    void* grad_logits;
    uint64_t grad_stride;
};

// The logistic function, exactly as the choice uses it.
__device__ __forceinline__ float logistic(float l) { return 1.0f / (1.0f + expf(-l)); }

// Over the L lanes of a token.
template <int L>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_max(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
    return x;
}

// Sum over a row by halves: entry i takes entry i + n/2 while n > 1.  Entries
// beyond the row are zero, so the result is that of the smallest power of two.
template <int L, int J>
__device__ __forceinline__ float halving_sum(const float (&x)[J])
{
    float t[J];
#pragma unroll
    for (int j = 0; j < J; ++j) t[j] = x[j];
#pragma unroll
    for (int h = J / 2; h > 0; h /= 2)
#pragma unroll
        for (int j = 0; j < h; ++j) t[j] += t[j + h];
    return lanes_sum<L>(t[0]);
}

// The factors u_k that the chosen logits' weights are proportional to: exp(l)
// or the logistic function, over a common factor that keeps the largest one
// away from underflow (so renormalised weights are exact however small the
// scores are).  Lane k holds chosen logit k; `on` marks lanes that hold one.
template <int L>
__device__ __forceinline__ float chosen_factor(float l, bool on, bool sigmoid)
{
    const float top = lanes_max<L>(on ? l : -kInf);
    if (!on) return 0.0f;
    if (!sigmoid) return expf(l - top);
    if (l >= 0.0f) return 1.0f / (1.0f + expf(-l));
    return expf(l - fminf(top, 0.0f)) / (1.0f + expf(l));
}

template <typename T, int L, int J>
__device__ __forceinline__ void load_logits(const RouteArgs& a, const T* row, bool there, uint32_t li, float (&l)[J])
{
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = li + L * j;
        l[j] = there && e < a.E ? to_float<T>(row[e]) : -kInf;
    }
}

// Largest logit of the row, 0 where there is none (an empty row's exponentials
// are then exp(-inf) = 0).
template <int L, int J>
__device__ __forceinline__ float row_max(const float (&l)[J])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
    m = lanes_max<L>(m);
    return m == -kInf ? 0.0f : m;
}

// Drops the experts outside the best groups.  The warp's values go through
// shared memory, group g's from row + g * (per + lanes_per): 32 / Gp lanes a
// group (Gp: groups rounded up to a power of two) keep its two largest.
template <int J>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, uint32_t lane, float* row, uint32_t lanes_per,
                                            const float (&v)[J], uint32_t (&key)[J])
{
    const uint32_t pitch = a.per + lanes_per;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        if (e < a.E) row[e + ((e * a.inv_per) >> 20) * lanes_per] = key[j] != 0 ? v[j] : -kInf;
    }
    __syncwarp();
    const uint32_t g = lane / lanes_per, sub = lane - g * lanes_per;
    float a1 = -kInf, a2 = -kInf;
    if (g < a.G)
        for (uint32_t i = sub; i < a.per; i += lanes_per) {
            const float x = row[g * pitch + i];
            a2 = fmaxf(a2, fminf(a1, x));
            a1 = fmaxf(a1, x);
        }
    __syncwarp();
    for (uint32_t o = lanes_per / 2; o > 0; o /= 2) {
        const float b1 = __shfl_xor_sync(0xFFFFFFFFu, a1, o), b2 = __shfl_xor_sync(0xFFFFFFFFu, a2, o);
        a2 = fmaxf(fmaxf(a2, b2), fminf(a1, b1));
        a1 = fmaxf(a1, b1);
    }
    // no expert: below every group that has one; one expert: its value alone
    uint32_t mine = a1 == -kInf ? 0u : order_key(a2 == -kInf ? a1 + 0.0f : a1 + a2);
    uint32_t rank = 0;
    for (uint32_t o = 0; o < a.G; ++o) {
        const uint32_t other = __shfl_sync(0xFFFFFFFFu, mine, o * lanes_per);
        rank += (other > mine || (other == mine && o < g)) ? 1u : 0u;
    }
    const uint32_t kept = __ballot_sync(0xFFFFFFFFu, g < a.G && rank < a.top_groups);
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        if (e < a.E && !((kept >> (((e * a.inv_per) >> 20) * lanes_per)) & 1u)) key[j] = 0;
    }
}

template <typename T, int L, int J>
__global__ void __launch_bounds__(kRouteWarps * 32, J <= 8 ? 8 : 6) route_kernel(RouteArgs a)
{
    extern __shared__ float scratch[];  // groups > 1: one row of values per warp
    pdl_wait();
    constexpr uint32_t kTokens = 32 / L;  // tokens of a warp
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % L;
    const uint64_t step = (uint64_t)gridDim.x * kRouteWarps * kTokens;
    for (uint64_t t0 = ((uint64_t)blockIdx.x * kRouteWarps + warp) * kTokens; t0 < a.tokens; t0 += step) {
        const uint64_t t = t0 + lane / L;
        const bool real = t < a.tokens;
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.stride;
        float l[J], v[J];
        load_logits<T, L, J>(a, row, real, li, l);
        float m = 0.0f, total = 1.0f;
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = logistic(l[j]);
        } else {
            m = row_max<L, J>(l);
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = expf(l[j] - m);
            total = halving_sum<L, J>(v);
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = v[j] / total;
        }
        uint32_t key[J];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t e = li + L * j;
            if (a.bias != nullptr && e < a.E) v[j] += a.bias[e];
            const bool there = e < a.E && l[j] != -kInf;
            bad = bad || (there && v[j] != v[j]);
            key[j] = there && v[j] != -kInf ? order_key(v[j] + 0.0f) : 0u;
        }
        const uint32_t all_bad = __ballot_sync(0xFFFFFFFFu, bad);
        if (all_bad != 0) {
            bad = ((all_bad >> (lane - li)) & (0xFFFFFFFFu >> (32 - L))) != 0;
            if (bad) {
                if (li == 0) report(a.status, ZCCL_ERR_INVALID_ARG);
#pragma unroll
                for (int j = 0; j < J; ++j) key[j] = 0;
            }
        }
        if (L == 32 && a.G > 1) {
            uint32_t gp = 1;
            while (gp < a.G) gp *= 2;
            const uint32_t lanes_per = 32 / gp;
            keep_groups<J>(a, lane, scratch + warp * (a.E + a.G * lanes_per), lanes_per, v, key);
        }
        // the K largest keys, one per round: the lane with the lowest expert among equals gives its own up
        int32_t mine = -1;
        for (uint32_t k = 0; k < a.K; ++k) {
            uint32_t best = key[0], e = 0;
#pragma unroll
            for (int j = 1; j < J; ++j)
                if (key[j] > best) best = key[j], e = j;
            e = li + L * e;
            if (L == 32) {
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
                e = __reduce_min_sync(0xFFFFFFFFu, best == top ? e : 0xFFFFFFFFu);
                best = top;
            } else {
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2) {
                    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, best, o), at = __shfl_xor_sync(0xFFFFFFFFu, e, o);
                    if (other > best || (other == best && at < e)) best = other, e = at;
                }
            }
            if (li == k && best != 0) mine = (int32_t)e;  // 0: none is left
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (li + L * j == e) key[j] = 0;
        }
        const bool on = mine >= 0;
        const float mine_l = on ? to_float<T>(row[mine]) : -kInf;
        float w = 0.0f;
        if (a.renorm) {
            const float u = chosen_factor<L>(mine_l, on, a.sigmoid != 0);
            const float sum = lanes_sum<L>(u);
            w = on ? u / sum * a.scale : 0.0f;
        } else if (on) {
            w = (a.sigmoid ? logistic(mine_l) : expf(mine_l - m) / total) * a.scale;
        }
        if (real && li < a.K) {
            a.idx[t * a.K + li] = mine;
            a.weights[t * a.K + li] = w;
        }
    }
}

template <typename T, int L, int J>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a)
{
    pdl_wait();
    constexpr uint32_t kTokens = 32 / L;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % L;
    const uint64_t step = (uint64_t)gridDim.x * kRouteWarps * kTokens;
    for (uint64_t t0 = ((uint64_t)blockIdx.x * kRouteWarps + warp) * kTokens; t0 < a.tokens; t0 += step) {
        const uint64_t t = t0 + lane / L;
        const bool real = t < a.tokens;
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.stride;
        // only a softmax that is not renormalised has a gradient at the logits that were not chosen
        const bool dense = !a.renorm && !a.sigmoid;
        float l[J], g[J];
        if (dense) load_logits<T, L, J>(a, row, real, li, l);
        int32_t e = -1;
        float up = 0.0f;
        if (real && li < a.K) {
            e = a.idx[t * a.K + li];
            if (e < 0 || (uint32_t)e >= a.E) e = -1;
            if (e >= 0) up = a.grad_weights[t * a.K + li] * a.scale;
        }
        const bool on = e >= 0;
#pragma unroll
        for (int j = 0; j < J; ++j) g[j] = 0.0f;
        // lane k's part of the gradient, for its own chosen logit
        float part = up;
        const float le = on ? to_float<T>(row[e]) : -kInf;
        if (a.renorm) {
            const float u = chosen_factor<L>(le, on, a.sigmoid != 0);
            const float total = lanes_sum<L>(u);
            const float p = on ? u / total : 0.0f;
            const float inner = lanes_sum<L>(p * up);
            part = p * (up - inner);
            if (a.sigmoid) part *= on ? 1.0f / (1.0f + expf(le)) : 0.0f;
        } else if (a.sigmoid) {
            part = on ? up * (logistic(le) * (1.0f / (1.0f + expf(le)))) : 0.0f;
        }
        for (uint32_t k = 0; k < a.K; ++k) {
            const int32_t ek = __shfl_sync(0xFFFFFFFFu, e, k, L);
            const float pk = __shfl_sync(0xFFFFFFFFu, part, k, L);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if ((int32_t)(li + L * j) == ek) g[j] += pk;
        }
        if (dense) {
            // every expert shares the denominator
            const float m = row_max<L, J>(l);
            float p[J];
#pragma unroll
            for (int j = 0; j < J; ++j) p[j] = expf(l[j] - m);
            const float total = halving_sum<L, J>(p);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[j] = p[j] / total;
                dot += p[j] * g[j];
            }
            dot = lanes_sum<L>(dot);
            // a row that chose nothing (its scores may be NaN) has none
            const bool any = (__ballot_sync(0xFFFFFFFFu, on) >> (lane - li) & (0xFFFFFFFFu >> (32 - L))) != 0;
#pragma unroll
            for (int j = 0; j < J; ++j) g[j] = any ? p[j] * (g[j] - dot) : 0.0f;
        }
        T* out = reinterpret_cast<T*>(a.grad_logits) + t * a.grad_stride;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t x = li + L * j;
            if (real && x < a.E) out[x] = from_float<T>(g[j]);
        }
    }
}

using RouteKernel = void (*)(RouteArgs);

// Registers for E logits over L lanes: the next power of two.
template <typename T, int L>
RouteKernel forward_kernel(uint32_t experts)
{
    const uint32_t columns = (experts + L - 1) / L;
    if (columns <= 2) return route_kernel<T, L, 2>;
    if (columns <= 4) return route_kernel<T, L, 4>;
    return L < 32 || columns <= 8 ? route_kernel<T, L, 8> : route_kernel<T, 32, 16>;
}
template <typename T, int L>
RouteKernel backward_kernel(uint32_t experts)
{
    const uint32_t columns = (experts + L - 1) / L;
    if (columns <= 2) return route_backward_kernel<T, L, 2>;
    if (columns <= 4) return route_backward_kernel<T, L, 4>;
    return L < 32 || columns <= 8 ? route_backward_kernel<T, L, 8> : route_backward_kernel<T, 32, 16>;
}

// Lanes of a token.  Forward: 8 where they hold its K chosen, and its logits in
// 8 registers, else a whole warp (16 lanes gain nothing: 12.8 us against 12.0
// for 16384 x 128), which compares groups too and which is the shorter way
// through while the tokens do not fill the machine.  Top 8 of 64, BF16, with 8
// lanes and with 32: 256 tokens 3.5 and 2.6 us, 4096: 3.9 and 3.8, 8192: 5.2 and
// 5.6, 65536: 21.6 and 29.5.
template <typename T>
RouteKernel forward_kernel_for(const RouteArgs& a, uint32_t* lanes)
{
    *lanes = a.G == 1 && a.tokens > 4096 && a.K <= 8 && a.E <= 64 ? 8 : 32;
    return *lanes == 8 ? forward_kernel<T, 8>(a.E) : forward_kernel<T, 32>(a.E);
}
// Backward, as few lanes as hold them: 65536 x 64 8.7 us with 8 lanes and 18.2
// with 32, 65536 x 128 17.8 with 16 and 23.8 with 32, 256 x 64 2.5 and 2.6.
template <typename T>
RouteKernel backward_kernel_for(const RouteArgs& a, uint32_t* lanes)
{
    *lanes = a.K <= 8 && a.E <= 64 ? 8 : a.K <= 16 && a.E <= 128 ? 16 : 32;
    return *lanes == 8    ? backward_kernel<T, 8>(a.E)
           : *lanes == 16 ? backward_kernel<T, 16>(a.E)
                          : backward_kernel<T, 32>(a.E);
}

template <typename T>
cudaError_t launch_route_as(const RouteArgs& a, bool backward, int sms, cudaStream_t stream)
{
    uint32_t gp = 1, lanes;
    while (gp < a.G) gp *= 2;
    const size_t smem = !backward && a.G > 1 ? kRouteWarps * (a.E + a.G * (32 / gp)) * sizeof(float) : 0;
    const RouteKernel k = backward ? backward_kernel_for<T>(a, &lanes) : forward_kernel_for<T>(a, &lanes);
    const uint64_t per_cta = kRouteWarps * 32 / lanes, ctas = (a.tokens + per_cta - 1) / per_cta, most = (uint64_t)sms * 64;
    return launch_dependent(k, (uint32_t)(ctas < most ? ctas : most), kRouteWarps * 32, smem, stream, a);
}

bool route_config(const zccl_route_t* c, RouteArgs* a)
{
    if (c == nullptr || c->experts == 0 || c->experts > ZCCL_MAX_EXPERTS || c->groups == 0 ||
        c->groups > kMaxGroups || c->experts % c->groups != 0 || c->top_groups == 0 || c->top_groups > c->groups ||
        c->top_k == 0 || c->top_k > ZCCL_MAX_TOP_K || c->top_k > c->top_groups * (c->experts / c->groups) ||
        (c->score != ZCCL_SCORE_SOFTMAX && c->score != ZCCL_SCORE_SIGMOID) || !std::isfinite(c->scale))
        return false;
    a->E = c->experts;
    a->K = c->top_k;
    a->G = c->groups;
    a->top_groups = c->top_groups;
    a->per = c->experts / c->groups;
    a->inv_per = ((1u << 20) + a->per - 1) / a->per;  // e * inv_per >> 20 = e / per: e * per < 2^20
    a->sigmoid = c->score == ZCCL_SCORE_SIGMOID;
    a->renorm = c->renormalize != 0;
    a->scale = c->scale;
    return true;
}

zccl_status_t launch_route(const RouteArgs& a, int dtype, bool backward, cudaStream_t stream)
{
    if (a.tokens == 0) return ZCCL_OK;
    const int sms = sm_count();
    if (sms == 0) return ZCCL_ERR_CUDA;
    return launched(dtype == ZCCL_BF16 ? launch_route_as<__nv_bfloat16>(a, backward, sms, stream)
                                       : launch_route_as<float>(a, backward, sms, stream));
}

}  // namespace

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_route(const zccl_route_t* cfg, const void* d_logits, int dtype, uint64_t stride,
                         const float* d_bias, uint64_t tokens, int32_t* d_idx, float* d_weights, uint32_t* d_status,
                         cudaStream_t stream)
{
    RouteArgs a{};
    if (!route_config(cfg, &a) || (dtype != ZCCL_BF16 && dtype != ZCCL_F32) || tokens >= (1ull << 31) / a.K ||
        stride >= kMaxElems || !is_aligned(d_bias, 4) || !is_aligned(d_status, 4))
        return ZCCL_ERR_INVALID_ARG;
    if (tokens > 0 && (!good_ptr(d_logits, dtype == ZCCL_BF16 ? 2 : 4) || !good_ptr(d_idx, 4) || !good_ptr(d_weights, 4)))
        return ZCCL_ERR_INVALID_ARG;
    a.logits = d_logits;
    a.stride = stride;
    a.bias = d_bias;
    a.tokens = tokens;
    a.idx = d_idx;
    a.weights = d_weights;
    a.status = d_status;
    return launch_route(a, dtype, false, stream);
}

zccl_status_t zccl_route_backward(const zccl_route_t* cfg, const void* d_logits, int dtype, uint64_t stride,
                                  const int32_t* d_idx, const float* d_grad_weights, uint64_t tokens,
                                  void* d_grad_logits, uint64_t grad_stride, cudaStream_t stream)
{
    RouteArgs a{};
    if (!route_config(cfg, &a) || (dtype != ZCCL_BF16 && dtype != ZCCL_F32) || tokens >= (1ull << 31) / a.K ||
        stride >= kMaxElems || grad_stride >= kMaxElems || (tokens > 1 && grad_stride < a.E))
        return ZCCL_ERR_INVALID_ARG;
    const uintptr_t al = dtype == ZCCL_BF16 ? 2 : 4;
    if (tokens > 0 && (!good_ptr(d_logits, al) || !good_ptr(d_idx, 4) || !good_ptr(d_grad_weights, 4) ||
                       !good_ptr(d_grad_logits, al)))
        return ZCCL_ERR_INVALID_ARG;
    a.logits = d_logits;
    a.stride = stride;
    a.idx = const_cast<int32_t*>(d_idx);
    a.grad_weights = d_grad_weights;
    a.tokens = tokens;
    a.grad_logits = d_grad_logits;
    a.grad_stride = grad_stride;
    return launch_route(a, dtype, true, stream);
}

}  // extern "C"
