// zccl_balance.cu -- how evenly a routing shares its slots out: the balance loss,
// each expert's slots, and the gradient of the logits.
//
// A warp holds a token's logits in registers, expert e in lane e % 32, and adds its
// scores to sums that it keeps over its tokens.  A sequence's tokens are cut into
// parts, a CTA each; the last part to arrive adds the parts' sums in their order, and
// the last sequence the sequences' losses, so results depend on the sizes alone.
#include <cmath>

#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr int kWarps = 8;
constexpr uint32_t kMaxParts = 304;  // CTAs of a call with one sequence
constexpr uint32_t kPartTokens = 32; // at least, for another part
constexpr uint32_t kCounters = ZCCL_MAX_SEQUENCES + 1;  // the same place for any call, as calls of other sizes may come between

struct BalanceArgs {
    const void* logits;
    uint64_t stride;
    const int32_t* idx;
    uint64_t tokens;
    const int32_t* seq;
    uint32_t sequences, parts;
    uint32_t E, K;
    int sigmoid;
    float coefficient;
    float* loss;
    int32_t* counts;
    int32_t* live;
    // workspace
    uint32_t* arrived;   // [kCounters], 0 between calls: a sequence's parts; last, the sequences
    float* losses;       // [sequences]
    float* part_scores;  // [sequences][parts][E]
    int32_t* part_counts;  // [sequences][parts][E + 1]: slots, and last the tokens
    // backward
    const float* grad_loss;
    void* grad;
    uint64_t grad_stride;
    int accumulate;
};

__device__ __forceinline__ float lanes_add(float x)
{
#pragma unroll
    for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// The tokens of a sequence (sequence `sequences`: those behind the last one), whatever
// the table holds.
__device__ __forceinline__ void sequence_tokens(const BalanceArgs& a, uint32_t s, uint64_t* lo, uint64_t* hi)
{
    if (a.seq == nullptr) {
        *lo = s == 0 ? 0 : a.tokens;
        *hi = a.tokens;
        return;
    }
    const int64_t n = (int64_t)a.tokens;
    int64_t b = ld_l2(a.seq + s), e = s < a.sequences ? ld_l2(a.seq + s + 1) : n;
    b = b < 0 ? 0 : b > n ? n : b;
    e = e < b ? b : e > n ? n : e;
    *lo = (uint64_t)b;
    *hi = (uint64_t)e;
}

// A row's shares q (softmax, or scores over their sum) and what their slopes multiply.
template <int J>
__device__ __forceinline__ void shares(const BalanceArgs& a, const float (&l)[J], float (&q)[J])
{
    float m = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
    m = warp_max(m);
    if (m == -__builtin_huge_valf()) m = 0.0f;
    float total = 0.0f;
    if (a.sigmoid) {
        // over a common factor, which keeps the largest from underflow
        const float low = fminf(m, 0.0f);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            q[j] = l[j] >= 0.0f ? 1.0f / (1.0f + expf(-l[j])) : expf(l[j] - low) / (1.0f + expf(l[j]));
            total += q[j];
        }
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            q[j] = expf(l[j] - m);
            total += q[j];
        }
    }
    total = lanes_add(total);
#pragma unroll
    for (int j = 0; j < J; ++j) q[j] = total == 0.0f ? 0.0f : q[j] / total;
}

template <typename T, int J>
__device__ __forceinline__ void load_row(const BalanceArgs& a, uint64_t t, uint32_t lane, float (&l)[J])
{
    const T* row = static_cast<const T*>(a.logits) + t * a.stride;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t e = lane + 32 * j;
        l[j] = e < a.E ? to_float<T>(row[e]) : -__builtin_huge_valf();
    }
}

// The lane's expert of a token, -1 for none.
__device__ __forceinline__ int32_t choice(const BalanceArgs& a, uint64_t t, uint32_t lane)
{
    const int32_t e = lane < a.K ? a.idx[t * a.K + lane] : -1;
    return e >= 0 && (uint32_t)e < a.E ? e : -1;
}

// Whether this CTA is the last of `n` to come by; what the others wrote before is visible to it then.
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t n)
{
    __shared__ uint32_t before;
    __syncthreads();
    if (threadIdx.x == 0) before = atom_inc_acq_rel(counter, n - 1);
    __syncthreads();
    return before == n - 1;
}

template <typename T, int J>
__global__ void __launch_bounds__(kWarps * 32) balance_kernel(BalanceArgs a)
{
    __shared__ float sums[kWarps][J * 32];
    __shared__ int32_t slots[J * 32];
    __shared__ int32_t live_tokens;
    __shared__ float red[kWarps];
    pdl_wait();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    for (uint32_t e = threadIdx.x; e < J * 32; e += kWarps * 32) slots[e] = 0;
    if (threadIdx.x == 0) live_tokens = 0;
    __syncthreads();
    uint64_t lo, hi;
    sequence_tokens(a, s, &lo, &hi);
    const uint64_t n = hi - lo;
    hi = lo + n * (part + 1) / a.parts;
    lo = lo + n * part / a.parts;
    float sum[J] = {};
    int32_t live = 0;
    for (uint64_t t = lo + warp; t < hi; t += kWarps) {
        float l[J], q[J];
        load_row<T, J>(a, t, lane, l);
        const int32_t e = choice(a, t, lane);
        if (__ballot_sync(0xFFFFFFFFu, e >= 0) == 0) continue;
        ++live;
        if (e >= 0) atomicAdd(&slots[e], 1);
        shares<J>(a, l, q);
#pragma unroll
        for (int j = 0; j < J; ++j) sum[j] += q[j];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) sums[warp][lane + 32 * j] = sum[j];
    if (lane == 0) atomicAdd(&live_tokens, live);
    __syncthreads();
    // the CTA's sums, then those of the sequence's parts
    float* const all = sums[0];
    for (uint32_t e = threadIdx.x; e < a.E; e += kWarps * 32) {
        float x = all[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x += sums[w][e];
        all[e] = x;
    }
    if (a.parts > 1) {
        const uint64_t at = (uint64_t)s * a.parts + part;
        for (uint32_t e = threadIdx.x; e < a.E; e += kWarps * 32) {
            a.part_scores[at * a.E + e] = all[e];
            a.part_counts[at * (a.E + 1) + e] = slots[e];
        }
        if (threadIdx.x == 0) a.part_counts[at * (a.E + 1) + a.E] = live_tokens;
        if (!last_of(a.arrived + s, a.parts)) return;
        const float* scores = a.part_scores + (uint64_t)s * a.parts * a.E;
        const int32_t* counts = a.part_counts + (uint64_t)s * a.parts * (a.E + 1);
        for (uint32_t e = threadIdx.x; e <= a.E; e += kWarps * 32) {
            float x = 0.0f;
            int32_t c = 0;
            for (uint32_t p = 0; p < a.parts; ++p) {
                if (e < a.E) x += scores[(uint64_t)p * a.E + e];
                c += counts[(uint64_t)p * (a.E + 1) + e];
            }
            if (e < a.E) all[e] = x, slots[e] = c;
            else live_tokens = c;
        }
        __syncthreads();
    }
    // the sequence's loss
    float dot = 0.0f;
    int32_t used = 0;
    for (uint32_t e = threadIdx.x; e < a.E; e += kWarps * 32) {
        dot += (float)slots[e] * all[e];
        used += slots[e];
        a.counts[(uint64_t)s * a.E + e] = slots[e];
    }
    dot = lanes_add(dot);
    used = __reduce_add_sync(0xFFFFFFFFu, used);
    __shared__ int32_t used_by[kWarps];
    if (lane == 0) red[warp] = dot, used_by[warp] = used;
    __syncthreads();
    if (threadIdx.x == 0) {
        float d = 0.0f;
        int32_t u = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) d += red[w], u += used_by[w];
        a.losses[s] = live_tokens > 0 ? d * ((float)a.E / ((float)u * (float)live_tokens)) : 0.0f;
        a.live[s] = live_tokens;
    }
    // the call's
    if (!last_of(a.arrived + kCounters - 1, a.sequences)) return;
    dot = 0.0f;
    int32_t alive = 0;
    for (uint32_t i = threadIdx.x; i < a.sequences; i += kWarps * 32) {
        dot += a.losses[i];
        alive += a.live[i] > 0 ? 1 : 0;
    }
    dot = lanes_add(dot);
    alive = __reduce_add_sync(0xFFFFFFFFu, alive);
    if (lane == 0) red[warp] = dot, used_by[warp] = alive;
    __syncthreads();
    if (threadIdx.x == 0) {
        float d = 0.0f;
        int32_t n = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) d += red[w], n += used_by[w];
        *a.loss = n > 0 ? a.coefficient * (d / (float)n) : 0.0f;
        a.live[a.sequences] = n;
    }
}

template <typename T, int J>
__global__ void __launch_bounds__(kWarps * 32) balance_backward_kernel(BalanceArgs a)
{
    pdl_wait();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    uint64_t lo, hi;
    sequence_tokens(a, s, &lo, &hi);
    const uint64_t n = hi - lo;
    hi = lo + n * (part + 1) / a.parts;
    lo = lo + n * part / a.parts;
    const bool counted = s < a.sequences;
    if (lo >= hi || (!counted && a.accumulate)) return;
    // what a unit of an expert's shares adds to the loss
    float f[J];
    if (counted) {
        int32_t c[J], used = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            c[j] = lane + 32 * j < a.E ? a.counts[(uint64_t)s * a.E + lane + 32 * j] : 0;
            used += c[j];
        }
        used = __reduce_add_sync(0xFFFFFFFFu, used);
        const float up = a.coefficient * (a.grad_loss != nullptr ? *a.grad_loss : 1.0f);
        const float each = (float)used * (float)a.live[s] * (float)a.live[a.sequences];
        const float unit = each > 0.0f ? up * ((float)a.E / each) : 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) f[j] = unit * (float)c[j];
    }
    for (uint64_t t = lo + warp; t < hi; t += kWarps) {
        float l[J], q[J];
        T* out = static_cast<T*>(a.grad) + t * a.grad_stride;
        const int32_t e = counted ? choice(a, t, lane) : -1;
        const bool live = __ballot_sync(0xFFFFFFFFu, e >= 0) != 0;
        if (!live && a.accumulate) continue;
        if (live) {
            load_row<T, J>(a, t, lane, l);
            shares<J>(a, l, q);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < J; ++j) dot = fmaf(f[j], q[j], dot);
            dot = lanes_add(dot);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                q[j] *= f[j] - dot;
                if (a.sigmoid) q[j] *= 1.0f / (1.0f + expf(l[j]));
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t x = lane + 32 * j;
            if (x < a.E) out[x] = from_float<T>((live ? q[j] : 0.0f) + (a.accumulate ? to_float<T>(out[x]) : 0.0f));
        }
    }
}

using BalanceKernel = void (*)(BalanceArgs);
template <typename T>
BalanceKernel balance_for(uint32_t experts, bool backward)
{
    if (experts <= 64) return backward ? balance_backward_kernel<T, 2> : balance_kernel<T, 2>;
    if (experts <= 128) return backward ? balance_backward_kernel<T, 4> : balance_kernel<T, 4>;
    if (experts <= 256) return backward ? balance_backward_kernel<T, 8> : balance_kernel<T, 8>;
    return backward ? balance_backward_kernel<T, 16> : balance_kernel<T, 16>;
}

uint32_t most_parts(uint32_t sequences) { return sequences >= kMaxParts ? 1 : kMaxParts / sequences; }

// Parts of a sequence of average length.
uint32_t parts_for(uint64_t tokens, uint32_t sequences)
{
    const uint64_t parts = tokens / sequences / kPartTokens, most = most_parts(sequences);
    return (uint32_t)(parts < 1 ? 1 : parts < most ? parts : most);
}

bool balance_config(const zccl_route_t* c, int dtype, uint64_t stride, uint64_t tokens, uint32_t sequences,
                    const int32_t* d_seq, float coefficient, BalanceArgs* a)
{
    if (c == nullptr || c->experts == 0 || c->experts > ZCCL_MAX_EXPERTS || c->top_k == 0 || c->top_k > ZCCL_MAX_TOP_K ||
        (c->score != ZCCL_SCORE_SOFTMAX && c->score != ZCCL_SCORE_SIGMOID) || (dtype != ZCCL_BF16 && dtype != ZCCL_F32) ||
        tokens >= (1ull << 31) / c->top_k || stride >= kMaxElems || sequences == 0 || sequences > ZCCL_MAX_SEQUENCES ||
        (sequences > 1 && d_seq == nullptr) || !is_aligned(d_seq, 4) || !std::isfinite(coefficient))
        return false;
    a->stride = stride;
    a->tokens = tokens;
    a->seq = d_seq;
    a->sequences = sequences;
    a->parts = parts_for(tokens, sequences);
    a->E = c->experts;
    a->K = c->top_k;
    a->sigmoid = c->score == ZCCL_SCORE_SIGMOID;
    a->coefficient = coefficient;
    return true;
}

}  // namespace

}  // namespace zccl

using namespace zccl;

extern "C" {

zccl_status_t zccl_balance_workspace_bytes(uint32_t sequences, uint32_t experts, uint64_t* bytes)
{
    if (bytes == nullptr || sequences == 0 || sequences > ZCCL_MAX_SEQUENCES || experts == 0 || experts > ZCCL_MAX_EXPERTS)
        return ZCCL_ERR_INVALID_ARG;
    const uint64_t most = most_parts(sequences), parts = most > 1 ? most * sequences : 0;
    *bytes = 4ull * (kCounters + sequences) + 4ull * parts * (2 * experts + 1);
    return ZCCL_OK;
}

zccl_status_t zccl_balance(const zccl_route_t* cfg, const void* d_logits, int dtype, uint64_t stride,
                           const int32_t* d_idx, uint64_t tokens, const int32_t* d_seq, uint32_t sequences,
                           float coefficient, float* d_loss, int32_t* d_counts, int32_t* d_tokens, void* d_ws,
                           uint64_t ws_bytes, cudaStream_t stream)
{
    BalanceArgs a{};
    uint64_t need = 0;
    if (!balance_config(cfg, dtype, stride, tokens, sequences, d_seq, coefficient, &a) || !good_ptr(d_loss, 4) ||
        !good_ptr(d_counts, 4) || !good_ptr(d_tokens, 4) || !good_ptr(d_ws, 4) ||
        (tokens > 0 && (!good_ptr(d_logits, dtype == ZCCL_BF16 ? 2 : 4) || !good_ptr(d_idx, 4))))
        return ZCCL_ERR_INVALID_ARG;
    zccl_balance_workspace_bytes(sequences, a.E, &need);
    if (ws_bytes < need) return ZCCL_ERR_BUFFER_TOO_SMALL;
    a.logits = d_logits;
    a.idx = d_idx;
    a.loss = d_loss;
    a.counts = d_counts;
    a.live = d_tokens;
    a.arrived = static_cast<uint32_t*>(d_ws);
    a.losses = reinterpret_cast<float*>(a.arrived + kCounters);
    a.part_scores = a.losses + sequences;
    a.part_counts = reinterpret_cast<int32_t*>(a.part_scores + (uint64_t)sequences * a.parts * a.E);
    return launched(launch_dependent(dtype == ZCCL_BF16 ? balance_for<__nv_bfloat16>(a.E, false) : balance_for<float>(a.E, false),
                                     sequences * a.parts, kWarps * 32, 0, stream, a));
}

zccl_status_t zccl_balance_backward(const zccl_route_t* cfg, const void* d_logits, int dtype, uint64_t stride,
                                    const int32_t* d_idx, uint64_t tokens, const int32_t* d_seq, uint32_t sequences,
                                    const int32_t* d_counts, const int32_t* d_tokens, float coefficient,
                                    const float* d_grad_loss, void* d_grad_logits, uint64_t grad_stride, int accumulate,
                                    cudaStream_t stream)
{
    BalanceArgs a{};
    const uintptr_t al = dtype == ZCCL_BF16 ? 2 : 4;
    if (!balance_config(cfg, dtype, stride, tokens, sequences, d_seq, coefficient, &a) || grad_stride >= kMaxElems ||
        (tokens > 1 && grad_stride < a.E) || !is_aligned(d_grad_loss, 4))
        return ZCCL_ERR_INVALID_ARG;
    if (tokens == 0) return ZCCL_OK;
    if (!good_ptr(d_logits, al) || !good_ptr(d_idx, 4) || !good_ptr(d_counts, 4) || !good_ptr(d_tokens, 4) ||
        !good_ptr(d_grad_logits, al))
        return ZCCL_ERR_INVALID_ARG;
    a.logits = d_logits;
    a.idx = d_idx;
    a.counts = const_cast<int32_t*>(d_counts);
    a.live = const_cast<int32_t*>(d_tokens);
    a.grad_loss = d_grad_loss;
    a.grad = d_grad_logits;
    a.grad_stride = grad_stride;
    a.accumulate = accumulate != 0;
    // one more "sequence": the tokens behind the last one
    return launched(launch_dependent(dtype == ZCCL_BF16 ? balance_for<__nv_bfloat16>(a.E, true) : balance_for<float>(a.E, true),
                                     (sequences + 1) * a.parts, kWarps * 32, 0, stream, a));
}

}  // extern "C"
