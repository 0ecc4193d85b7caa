// zccl_route.cu -- the router: scores, choice and weights of each token's
// experts, and the gradient of the weights.
//
// One warp holds one token's logits in registers, expert e in lane e % 32, so
// a row is read once and nothing of it is written but the K chosen.  With E
// logits a token the bytes are few (16384 x 64 BF16: 2 MB, 0.3 us of HBM
// time); what a call costs is the chain of warp reductions, 2 K of them for
// the choice, hidden by the other warps of the SM.
#include <cmath>

#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr int kRouteWarps = 8;
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

// Sum over a row by halves: entry i takes entry i + n/2 while n > 1.  Entries
// beyond the row are zero, so the result is that of the smallest power of two.
template <int J>
__device__ __forceinline__ float halving_sum(const float (&x)[J])
{
    float t[J];
#pragma unroll
    for (int j = 0; j < J; ++j) t[j] = x[j];
#pragma unroll
    for (int h = J / 2; h > 0; h /= 2)
#pragma unroll
        for (int j = 0; j < h; ++j) t[j] += t[j + h];
    return warp_sum(t[0]);
}

// The factors u_k that the chosen logits' weights are proportional to: exp(l)
// or the logistic function, over a common factor that keeps the largest one
// away from underflow (so renormalised weights are exact however small the
// scores are).  Lane k holds chosen logit k; `on` marks lanes that hold one.
__device__ __forceinline__ float chosen_factor(float l, bool on, bool sigmoid)
{
    const float top = warp_max(on ? l : -kInf);
    if (!on) return 0.0f;
    if (!sigmoid) return expf(l - top);
    if (l >= 0.0f) return 1.0f / (1.0f + expf(-l));
    return expf(l - fminf(top, 0.0f)) / (1.0f + expf(l));
}

template <typename T, int J>
__device__ __forceinline__ void load_logits(const RouteArgs& a, uint64_t t, int lane, float (&l)[J])
{
    const T* row = reinterpret_cast<const T*>(a.logits) + t * a.stride;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        l[j] = e < a.E ? to_float<T>(row[e]) : -kInf;
    }
}

// Largest logit of the row, 0 where there is none (an empty row's exponentials
// are then exp(-inf) = 0).
template <int J>
__device__ __forceinline__ float row_max(const float (&l)[J])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    return m == -kInf ? 0.0f : m;
}

// Drops the experts outside the best groups.  The warp's values go through
// shared memory, group g's from row + g * (per + lanes_per): 32 / Gp lanes a
// group (Gp: groups rounded up to a power of two) keep its two largest.
template <int J>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, int lane, float* row, uint32_t per, uint32_t lanes_per,
                                            const uint32_t (&grp)[J], const float (&v)[J], uint32_t (&key)[J])
{
    const uint32_t pitch = per + lanes_per;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        if (e < a.E) row[grp[j] * pitch + (e - grp[j] * per)] = key[j] != 0 ? v[j] : -kInf;
    }
    __syncwarp();
    const uint32_t g = lane / lanes_per, sub = lane - g * lanes_per;
    float a1 = -kInf, a2 = -kInf;
    if (g < a.G)
        for (uint32_t i = sub; i < per; i += lanes_per) {
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
    for (int j = 0; j < J; ++j)
        if (!((kept >> (grp[j] * lanes_per)) & 1u)) key[j] = 0;
}

template <typename T, int J>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a)
{
    extern __shared__ float scratch[];  // groups > 1: one row of values per warp
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t per = a.E / a.G;
    uint32_t gp = 1;
    while (gp < a.G) gp *= 2;
    const uint32_t lanes_per = 32 / gp;
    uint32_t grp[J];
    float bias[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        grp[j] = e < a.E ? e / per : 0;
        bias[j] = a.bias != nullptr && e < a.E ? a.bias[e] : 0.0f;
    }
    float* row = scratch + warp * (a.E + a.G * lanes_per);
    for (uint64_t t = (uint64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (uint64_t)gridDim.x * kRouteWarps) {
        float l[J], v[J];
        load_logits<T, J>(a, t, lane, l);
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = logistic(l[j]);
        } else {
            const float m = row_max<J>(l);
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = expf(l[j] - m);
            const float total = halving_sum<J>(v);
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = v[j] / total;
        }
        uint32_t key[J];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (a.bias != nullptr) v[j] += bias[j];
            const bool there = lane + 32 * j < a.E && l[j] != -kInf;
            bad = bad || (there && v[j] != v[j]);
            key[j] = there && v[j] != -kInf ? order_key(v[j] + 0.0f) : 0u;
        }
        bad = __any_sync(0xFFFFFFFFu, bad);
        if (bad && lane == 0) report(a.status, ZCCL_ERR_INVALID_ARG);
        if (a.G > 1) keep_groups<J>(a, lane, row, per, lanes_per, grp, v, key);
        // the K largest keys, one per round: the lane with the lowest expert among equals gives its own up
        int32_t mine = -1;
        float mine_l = 0.0f;
        if (!bad) {
            for (uint32_t k = 0; k < a.K; ++k) {
                uint32_t best = key[0];
                int at = 0;
                float best_l = l[0];
#pragma unroll
                for (int j = 1; j < J; ++j)
                    if (key[j] > best) best = key[j], at = j, best_l = l[j];
                const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
                if (top == 0) break;
                const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, best == top ? (uint32_t)(lane + 32 * at) : 0xFFFFFFFFu);
                const float le = __shfl_sync(0xFFFFFFFFu, best_l, e & 31);
                if (lane == (int)k) mine = (int32_t)e, mine_l = le;
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (lane + 32 * j == e) key[j] = 0;
            }
        }
        const bool on = mine >= 0;
        float w = 0.0f;
        if (a.renorm) {
            const float u = chosen_factor(mine_l, on, a.sigmoid != 0);
            const float total = warp_sum(u);
            w = on ? u / total * a.scale : 0.0f;
        } else if (a.sigmoid) {
            w = on ? logistic(mine_l) * a.scale : 0.0f;
        } else {
            const float m = row_max<J>(l);
            float p[J];
#pragma unroll
            for (int j = 0; j < J; ++j) p[j] = expf(l[j] - m);
            const float total = halving_sum<J>(p);
            w = on ? expf(mine_l - m) / total * a.scale : 0.0f;
        }
        if (lane < (int)a.K) {
            a.idx[t * a.K + lane] = mine;
            a.weights[t * a.K + lane] = w;
        }
    }
}

template <typename T, int J>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (uint64_t t = (uint64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens; t += (uint64_t)gridDim.x * kRouteWarps) {
        int32_t e = -1;
        float up = 0.0f;
        if (lane < (int)a.K) {
            e = a.idx[t * a.K + lane];
            if (e < 0 || (uint32_t)e >= a.E) e = -1;
            if (e >= 0) up = a.grad_weights[t * a.K + lane] * a.scale;
        }
        const bool on = e >= 0;
        float l[J], g[J];
        load_logits<T, J>(a, t, lane, l);
#pragma unroll
        for (int j = 0; j < J; ++j) g[j] = 0.0f;
        // lane k's part of the gradient, for its own chosen logit
        float part = up;
        const float le = on ? to_float<T>(reinterpret_cast<const T*>(a.logits)[t * a.stride + e]) : -kInf;
        if (a.renorm) {
            const float u = chosen_factor(le, on, a.sigmoid != 0);
            const float total = warp_sum(u);
            const float p = on ? u / total : 0.0f;
            const float inner = warp_sum(p * up);
            part = p * (up - inner);
            if (a.sigmoid) part *= on ? 1.0f / (1.0f + expf(le)) : 0.0f;
        } else if (a.sigmoid) {
            part = on ? up * (logistic(le) * (1.0f / (1.0f + expf(le)))) : 0.0f;
        }
        for (uint32_t k = 0; k < a.K; ++k) {
            const int32_t ek = __shfl_sync(0xFFFFFFFFu, e, k);
            const float pk = __shfl_sync(0xFFFFFFFFu, part, k);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (lane + 32 * j == ek) g[j] += pk;
        }
        if (!a.renorm && !a.sigmoid && __any_sync(0xFFFFFFFFu, on)) {
            // softmax without renormalisation: every expert shares the denominator
            const float m = row_max<J>(l);
            float p[J];
#pragma unroll
            for (int j = 0; j < J; ++j) p[j] = expf(l[j] - m);
            const float total = halving_sum<J>(p);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[j] = p[j] / total;
                dot += p[j] * g[j];
            }
            dot = warp_sum(dot);
#pragma unroll
            for (int j = 0; j < J; ++j) g[j] = p[j] * (g[j] - dot);
        }
        T* out = reinterpret_cast<T*>(a.grad_logits) + t * a.grad_stride;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t x = lane + 32 * j;
            if (x < a.E) out[x] = from_float<T>(g[j]);
        }
    }
}

// Registers for E logits: the next power of two of 32-expert columns.
template <typename T>
cudaError_t launch_route_as(const RouteArgs& a, bool backward, uint32_t grid, cudaStream_t stream)
{
    uint32_t gp = 1;
    while (gp < a.G) gp *= 2;
    const size_t smem = !backward && a.G > 1 ? kRouteWarps * (a.E + a.G * (32 / gp)) * sizeof(float) : 0;
    const uint32_t columns = (a.E + 31) / 32;
    void (*k)(RouteArgs);
    if (columns <= 1)
        k = backward ? route_backward_kernel<T, 1> : route_kernel<T, 1>;
    else if (columns <= 2)
        k = backward ? route_backward_kernel<T, 2> : route_kernel<T, 2>;
    else if (columns <= 4)
        k = backward ? route_backward_kernel<T, 4> : route_kernel<T, 4>;
    else if (columns <= 8)
        k = backward ? route_backward_kernel<T, 8> : route_kernel<T, 8>;
    else
        k = backward ? route_backward_kernel<T, 16> : route_kernel<T, 16>;
    return launch_dependent(k, grid, kRouteWarps * 32, smem, stream, a);
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
    const uint64_t ctas = (a.tokens + kRouteWarps - 1) / kRouteWarps;
    const uint32_t grid = (uint32_t)(ctas < (uint64_t)sms * 8 ? ctas : (uint64_t)sms * 8);
    return launched(dtype == ZCCL_BF16 ? launch_route_as<__nv_bfloat16>(a, backward, grid, stream)
                                       : launch_route_as<float>(a, backward, grid, stream));
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
