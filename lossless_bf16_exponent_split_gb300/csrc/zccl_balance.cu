// zccl_balance.cu -- how evenly a routing shares its slots out: the balance loss,
// each expert's slots, and the gradient of the logits.
//
// 8, 16 or 32 lanes hold a token's logits, 8 or 16 each, and keep the sums of their
// experts' shares over the tokens that come by.  A sequence's tokens are cut into parts
// of `chunk` tokens, a CTA each; the last part to arrive adds the parts' sums in their
// order, and the last sequence the sequences' losses, so results do not depend on who
// comes when.  Of more than kFewSequences sequences each is one part, however long.
//
// The bytes are few (16384 x 64 in BF16: 2 MB, 0.3 us of HBM time): a call is bound by its
// latencies (the table, the first logits, the hand-over to the last part), 10.7 us for the
// loss and the gradient; many experts by those and by a warp's one token at hand (65621 x 256
// in 32 bits with sigmoid scores: 152 and 194 instructions a warp and token, in 53 and 59 %
// of the issue slots; 46 us for both, 3.0 TB/s; logits three tokens ahead by asynchronous
// copies 49).  Exponentials and reciprocals are the fast ones: nothing here decides between
// close values.
#include <cmath>

#include "zccl_ops.cuh"

namespace zccl {

namespace {

constexpr int kWarps = 16;
constexpr uint32_t kFewSequences = 304;  // up to so many are cut into parts
constexpr uint32_t kCounters = ZCCL_MAX_SEQUENCES + 1;  // the same place for any call, as calls of other sizes may come between
constexpr int kThreads = kWarps * 32;
static_assert(kFewSequences < kThreads, "a thread each, and one for where the last ends");
constexpr float kInf = __builtin_huge_valf();

struct BalanceArgs {
    const void* logits;
    uint64_t stride;
    const int32_t* idx;
    uint64_t tokens;
    const int32_t* seq;
    uint32_t sequences;
    uint32_t chunk;      // tokens of a part; 0: a sequence is one part
    uint32_t E, K;
    int sigmoid;
    float coefficient;
    float* loss;
    int32_t* counts;
    int32_t* live;
    // workspace
    uint32_t* arrived;   // [kCounters], 0 between calls: a sequence's parts; last, the sequences
    float* losses;       // [sequences]
    float* part_scores;    // [parts][E]
    int32_t* part_counts;  // [parts][E + 1]: slots, and last the tokens
    // backward
    const float* grad_loss;
    void* grad;
    uint64_t grad_stride;
    int accumulate;
};

template <int L>
__device__ __forceinline__ float lanes_add(float x)
{
#pragma unroll
    for (int o = L / 2; o > 0; o /= 2) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// Two sums at once: half the lanes add up x, half y.
template <int L>
__device__ __forceinline__ void lanes_add(float& x, float& y)
{
    const bool upper = threadIdx.x & (L / 2);
    float mine = (upper ? y : x) + __shfl_xor_sync(0xFFFFFFFFu, upper ? x : y, L / 2);
    mine = lanes_add<L / 2>(mine);
    const float other = __shfl_xor_sync(0xFFFFFFFFu, mine, L / 2);
    x = upper ? other : mine;
    y = upper ? mine : other;
}

// A CTA's part: tokens lo..hi-1 of a sequence (`sequences`: the tokens before the first
// or behind the last one) that has `parts` of them, the first of them CTA `first`'s.
struct Part {
    uint32_t sequence, first, parts;
    uint64_t lo, hi;
};

// Over the CTA: the sum (or the largest) of x of all threads up to this one.
template <bool kMax>
__device__ __forceinline__ uint32_t cta_scan(uint32_t x, uint32_t* by_warp)
{
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if ((int)lane >= o) x = kMax ? max(x, y) : x + y;
    }
    if (lane == 31) by_warp[warp] = x;
    __syncthreads();
    uint32_t before = 0;
    for (uint32_t w = 0; w < warp; ++w) before = kMax ? max(before, by_warp[w]) : before + by_warp[w];
    __syncthreads();
    return kMax ? max(x, before) : x + before;
}

// This CTA's part; false: it has none.  Whatever the table holds, up to kFewSequences
// sequences are taken as runs of 0..tokens-1 one behind the other; of more, one that would
// end before it begins has no tokens and no parts.  kOthers: the tokens
// before the first sequence and those behind the last one are parts too, and a sequence
// without tokens is none (else it is one).
template <bool kOthers>
__device__ __forceinline__ bool part_of(const BalanceArgs& a, Part* p)
{
    __shared__ uint32_t begins[kThreads + 1], by_warp[kWarps];
    __shared__ Part found;
    const uint32_t id = blockIdx.x, i = threadIdx.x;
    const auto bound = [&](uint32_t at) -> uint32_t {
        const int32_t v = ld_l2(a.seq + at);
        return v < 0 ? 0 : (uint64_t)v > a.tokens ? (uint32_t)a.tokens : (uint32_t)v;
    };
    if (a.chunk == 0) {  // a CTA a sequence, and those behind share out the other tokens
        const uint32_t s = id < a.sequences ? id : a.sequences;
        const uint32_t b = bound(s), e = s < a.sequences ? bound(s + 1) : (uint32_t)a.tokens;
        *p = {s, id, e >= b ? 1u : 0u, b, e > b ? e : b};
        if (kOthers && id >= a.sequences) {
            const uint64_t before = bound(0), behind = p->hi - p->lo;
            uint64_t k = gridDim.x - a.sequences, j = id - a.sequences;  // two CTAs at least
            const uint64_t heads = before == 0 ? 0 : behind == 0 ? k : min(k - 1, 1 + k * before / (before + behind));
            if (j < heads)
                p->lo = 0, p->hi = before, k = heads;
            else
                j -= heads, k -= heads;
            const uint64_t n = p->hi - p->lo;
            p->hi = p->lo + n * (j + 1) / k;
            p->lo += n * j / k;
        }
        return true;
    }
    if (a.seq == nullptr) {
        const uint32_t all = (uint32_t)((a.tokens + a.chunk - 1) / a.chunk);
        *p = {0, 0, all > 0 ? all : 1, (uint64_t)id * a.chunk, min((uint64_t)(id + 1) * a.chunk, a.tokens)};
        return id < p->parts;
    }
    begins[i] = cta_scan<true>(i <= a.sequences ? bound(i) : (uint32_t)a.tokens, by_warp);
    if (i == 0) begins[kThreads] = (uint32_t)a.tokens, found.parts = 0;
    __syncthreads();
    const uint32_t n = begins[i + 1] - begins[i], most = kOthers ? a.sequences + 1 : a.sequences;
    uint32_t parts = i < most ? (n + a.chunk - 1) / a.chunk : 0;
    if (!kOthers && i < most && parts == 0) parts = 1;
    const uint32_t heads = kOthers ? (begins[0] + a.chunk - 1) / a.chunk : 0;  // of the tokens before the first: the first CTAs'
    const uint32_t behind = heads + cta_scan<false>(parts, by_warp);
    if (parts > 0 && id >= behind - parts && id < behind) {
        const uint64_t lo = begins[i] + (uint64_t)(id - (behind - parts)) * a.chunk;
        found = {i, behind - parts, parts, lo, min(lo + a.chunk, (uint64_t)begins[i + 1])};
    }
    if (kOthers && i == 0 && id < heads)
        found = {a.sequences, 0, heads, (uint64_t)id * a.chunk, min((uint64_t)(id + 1) * a.chunk, (uint64_t)begins[0])};
    __syncthreads();
    *p = found;
    return p->parts > 0;
}

// How a token's logits are read: 16 bytes at a time, the lanes' one behind the other
// (kNeighbours; kWhole: and the experts are as many as L lanes of J hold), or one by one.
enum Read { kOneByOne = 0, kNeighbours = 1, kWhole = 2 };

// A lane's logits of a token, as they are held in memory: 16 bytes of neighbours at a time, or
// L apart.
template <typename T, int kRead, int L, int J>
struct Logits {
    static constexpr bool kVec = kRead != kOneByOne;
    static constexpr int kWords = kVec ? J * sizeof(T) / 16 : 0, kPart = 16 / sizeof(T);
    uint4 q[kVec ? kWords : 1];
    float f[kVec ? 1 : J];
    static __device__ __forceinline__ uint32_t expert(uint32_t li, int j)
    {
        return kVec ? j / kPart * kPart * L + li * kPart + j % kPart : li + L * j;
    }
    __device__ __forceinline__ void load(const T* row, uint32_t li, uint32_t E)
    {
        if (kVec) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t e = expert(li, i * 16 / sizeof(T));
                q[i] = e < E ? *reinterpret_cast<const uint4*>(row + e) : make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j) f[j] = expert(li, j) < E ? to_float<T>(row[expert(li, j)]) : 0.0f;
        }
    }
    // -infinity where there is no expert
    __device__ __forceinline__ void get(float (&l)[J], uint32_t li, uint32_t E) const
    {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (!kVec) {
                l[j] = f[j];
            } else {
                const uint4 v = q[j * sizeof(T) / 16];
                const uint32_t w = (j * sizeof(T) / 4) % 4, x = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
                l[j] = sizeof(T) == 4 ? __uint_as_float(x) : j & 1 ? bf16_hi(x) : bf16_lo(x);
            }
            if (kRead != kWhole && expert(li, j) >= E) l[j] = -kInf;
        }
    }
};

template <typename T, int kRead, int L, int J>
__device__ __forceinline__ void store_row(T* row, const float (&g)[J], uint32_t li, uint32_t E)
{
    using Row = Logits<T, kRead, L, J>;
    if (Row::kVec) {
        constexpr int kEach = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < Row::kWords; ++i) {
            const uint32_t e = Row::expert(li, i * kEach);
            const float* v = g + i * kEach;
            const uint4 q = sizeof(T) == 2
                                ? make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]))
                                : make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
            if (e < E) *reinterpret_cast<uint4*>(row + e) = q;
        }
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (Row::expert(li, j) < E) row[Row::expert(li, j)] = from_float<T>(g[j]);
    }
}

// exp(x) to |x| 2^-23 and two units of the last place, zero below 2^-126, and 1 / x to one unit.
__device__ __forceinline__ float exp_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504f));
    return y;
}
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(-l); kFinite: 2^127 at most (a NaN stays one)
template <bool kFinite>
__device__ __forceinline__ float exp_of_minus(float l)
{
    float x = l * -1.44269504f, y;
    if (kFinite) asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(127.0f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's scores p and the factor that makes them its shares, 0 where it has none; with
// kSlope also the sigmoid's 1 - p, and the sum of the shares times f in `dot`.
template <bool kSlope, int L, int J>
__device__ __forceinline__ float scores(const BalanceArgs& a, const float (&l)[J], float (&p)[J], float (&slope)[J],
                                        const float (&f)[J], float* dot)
{
    const auto largest = [&]() {
        float m = l[0];
#pragma unroll
        for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        return m == -kInf ? 0.0f : m;
    };
    float total, weighted = 0.0f;
    const auto sum = [&]() {
        float2 s = make_float2(0.0f, 0.0f), u = s;
#pragma unroll
        for (int j = 0; j < J; j += 2) {
            s = __fadd2_rn(s, make_float2(p[j], p[j + 1]));
            if (kSlope) u = __ffma2_rn(make_float2(p[j], p[j + 1]), make_float2(f[j], f[j + 1]), u);
        }
        total = s.x + s.y;
        if (kSlope) {
            weighted = u.x + u.y;
            lanes_add<L>(total, weighted);
        } else {
            total = lanes_add<L>(total);
        }
    };
    if (a.sigmoid) {
#pragma unroll
        for (int j = 0; j < J; j += 2) {
            // t = exp(-l), p = 1 / (1 + t), 1 - p = t p: no difference of close values; from 2^126 on p is 0, and
            // the slope needs a finite t
            const float2 t = make_float2(exp_of_minus<kSlope>(l[j]), exp_of_minus<kSlope>(l[j + 1]));
            const float2 n = __fadd2_rn(t, make_float2(1.0f, 1.0f)), r = make_float2(reciprocal(n.x), reciprocal(n.y));
            p[j] = r.x, p[j + 1] = r.y;
            if (kSlope) {
                const float2 q = __fmul2_rn(t, r);
                slope[j] = q.x, slope[j + 1] = q.y;
            }
        }
        sum();
        // scores whose sum is below 2^-80: over a common factor, which keeps the largest from underflow (1 + exp(l) is 1)
        if (__any_sync(0xFFFFFFFFu, total < 0x1p-80f)) {
            const float m = largest();
            const bool small = total < 0x1p-80f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                p[j] = small ? exp_fast(l[j] - m) : p[j];
                if (kSlope) slope[j] = small ? 1.0f : slope[j];
            }
            sum();
        }
    } else {
        const float m = largest();
#pragma unroll
        for (int j = 0; j < J; ++j) p[j] = exp_fast(l[j] - m);
        sum();
    }
    const float share = total == 0.0f ? 0.0f : reciprocal(total);
    if (kSlope) *dot = weighted * share;
    return share;
}

// A lane's experts of a token (entries L apart).
template <int L>
struct Choices {
    static constexpr int kEach = ZCCL_MAX_TOP_K / L;
    int32_t e[kEach];
    // `at`: the lane's first entry of the token
    __device__ __forceinline__ void load(const int32_t* at, uint32_t K, bool there, uint32_t li)
    {
#pragma unroll
        for (int i = 0; i < kEach; ++i) e[i] = there && li + L * i < K ? at[L * i] : -1;
    }
    // Calls `use` with each of them; whether the token has any.
    template <typename Use>
    __device__ __forceinline__ bool each(uint32_t E, uint32_t li, Use use) const
    {
        bool any = false;
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            if ((uint32_t)e[i] < E) {
                any = true;
                use(e[i]);
            }
        __syncwarp();
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, any);
        return L == 32 ? who != 0 : (who >> ((threadIdx.x & 31) - li) & (0xFFFFFFFFu >> (32 - L))) != 0;
    }
};

// The tokens of a warp: kTokens at a time, the CTA's warps behind one another.
template <typename T, int kRead, int L, int J>
struct Walk {
    static constexpr uint32_t kTokens = 32 / L, kStep = kWarps * kTokens;
    uint32_t t, hi, li;           // this lane's token
    const T* logits;              // of the token to come
    const int32_t* idx;
    Logits<T, kRead, L, J> row;
    Choices<L> next;
    __device__ __forceinline__ void open(const BalanceArgs& a, uint64_t lo, uint64_t end, bool counted)
    {
        const uint32_t lane = threadIdx.x & 31;
        li = lane % L, hi = (uint32_t)end;
        t = (uint32_t)lo + (threadIdx.x >> 5) * kTokens + lane / L;
        logits = static_cast<const T*>(a.logits) + t * a.stride;
        idx = a.idx + (uint64_t)t * a.K + li;
        load(a, t, counted);
    }
    __device__ __forceinline__ void load(const BalanceArgs& a, uint32_t at, bool counted)
    {
        if (at < hi) row.load(logits, li, a.E);
        next.load(idx, a.K, at < hi && counted, li);
    }
    // Takes over what was loaded, and asks for the next.
    __device__ __forceinline__ Choices<L> take(const BalanceArgs& a, float (&l)[J], bool counted)
    {
        const Choices<L> chosen = next;
        row.get(l, li, a.E);
        logits += kStep * a.stride;
        idx += kStep * a.K;
        load(a, t + kStep, counted);
        return chosen;
    }
    // the warp's first token, and whether it has one
    __device__ __forceinline__ uint32_t at() const { return t - (threadIdx.x & 31) / L; }
    __device__ __forceinline__ bool more() const { return at() < hi; }
};

// Whether this CTA is the last of `n` to come by; what the others wrote before is visible to it then.
__device__ __forceinline__ bool last_of(uint32_t* counter, uint32_t n)
{
    __shared__ uint32_t before;
    __syncthreads();
    if (threadIdx.x == 0) before = atom_inc_acq_rel(counter, n - 1);
    __syncthreads();
    return before == n - 1;
}

// How many of its `steps` tokens a lane adds one after the other before their sum joins
// those of the runs before it: 256, of more than 65536 their square root at least, so that
// a sum has 512 roundings in a row, and of any number of tokens three times that root's (one
// after the other 65536 equal shares were off by 0.06 %).
__device__ __forceinline__ uint32_t run_of(uint32_t steps)
{
    uint32_t run = 256;
    while ((uint64_t)run * run < steps) run *= 2;
    return run;
}

template <typename T, int kRead, int L, int J>
__global__ void __launch_bounds__(kThreads) balance_kernel(BalanceArgs a)
{
    constexpr int kExperts = L * J;
    __shared__ float sums[kWarps][kExperts];
    __shared__ int32_t slots[kExperts];
    __shared__ int32_t live_tokens;
    __shared__ float red[kWarps];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (uint32_t e = threadIdx.x; e < kExperts; e += kThreads) slots[e] = 0;
    if (threadIdx.x == 0) live_tokens = 0;
    __syncthreads();
    pdl_wait();
    Part part;
    if (!part_of<false>(a, &part)) return;
    const uint32_t s = part.sequence;
    float sum[J] = {};
    int32_t live = 0;
    Walk<T, kRead, L, J> walk;
    walk.open(a, part.lo, part.hi, true);
    const uint32_t run = run_of((uint32_t)(part.hi - part.lo) / walk.kStep) * walk.kStep;
    bool first = true;
    do {
        const uint32_t till = min(walk.hi, walk.at() + run);
        for (; walk.at() < till; walk.t += walk.kStep) {
            float l[J], p[J], slope[J];
            const Choices<L> chosen = walk.take(a, l, true);
            const bool counts = chosen.each(a.E, walk.li, [&](int32_t e) { atomicAdd(&slots[e], 1); });
            live += counts && walk.li == 0 ? 1 : 0;
            if (!__all_sync(0xFFFFFFFFu, counts) && !counts)
#pragma unroll
                for (int j = 0; j < J; ++j) l[j] = -kInf;  // whatever it holds
            const float f = scores<false, L, J>(a, l, p, slope, l, nullptr);
#pragma unroll
            for (int j = 0; j < J; j += 2) {
                const float2 v = __ffma2_rn(make_float2(p[j], p[j + 1]), make_float2(f, f), make_float2(sum[j], sum[j + 1]));
                sum[j] = v.x, sum[j + 1] = v.y;
            }
        }
        // over the warp's tokens
#pragma unroll
        for (int o = 16; o >= L; o /= 2)
#pragma unroll
            for (int j = 0; j < J; ++j) sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], o);
        if (lane < L)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float& of_warp = sums[warp][walk.row.expert(walk.li, j)];
                of_warp = first ? sum[j] : of_warp + sum[j];
            }
#pragma unroll
        for (int j = 0; j < J; ++j) sum[j] = 0.0f;
        first = false;
    } while (walk.more());
    live = __reduce_add_sync(0xFFFFFFFFu, live);
    if (lane == 0) atomicAdd(&live_tokens, live);
    __syncthreads();
    // the CTA's sums, then those of the sequence's parts
    float* const all = sums[0];
    for (uint32_t e = threadIdx.x; e < a.E; e += kThreads) {
        float x = all[e];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x += sums[w][e];
        all[e] = x;
    }
    if (part.parts > 1) {
        const uint64_t at = blockIdx.x;
        for (uint32_t e = threadIdx.x; e < a.E; e += kThreads) {
            a.part_scores[at * a.E + e] = all[e];
            a.part_counts[at * (a.E + 1) + e] = slots[e];
        }
        if (threadIdx.x == 0) a.part_counts[at * (a.E + 1) + a.E] = live_tokens;
        if (!last_of(a.arrived + s, part.parts)) return;
        // the threads take a column each, as many times over as they go into the CTA, and every so many parts
        const float* scores = a.part_scores + (uint64_t)part.first * a.E;
        const int32_t* counts = a.part_counts + (uint64_t)part.first * (a.E + 1);
        constexpr int kSides = kThreads / kExperts > 0 ? kThreads / kExperts : 1;
        const uint32_t side = threadIdx.x / kExperts, e = threadIdx.x % kExperts;
        float x = 0.0f;
        int32_t c = 0;
        if (e < a.E)
#pragma unroll 8
            for (uint32_t p = side; p < part.parts; p += kSides) {
                x += scores[(uint64_t)p * a.E + e];
                c += counts[(uint64_t)p * (a.E + 1) + e];
            }
        int32_t m = 0;
        if (warp == 0)
            for (uint32_t p = lane; p < part.parts; p += 32) m += counts[(uint64_t)p * (a.E + 1) + a.E];
        // (the CTA's own sums have been written out; `sums` has room for kSides rows of them and of the counts)
        static_assert(2 * kSides <= kWarps, "room");
        sums[side][e] = x;
        sums[kSides + side][e] = __int_as_float(c);
        if (warp == 0) {
            m = __reduce_add_sync(0xFFFFFFFFu, m);
            if (lane == 0) live_tokens = m;
        }
        __syncthreads();
        if (threadIdx.x < kExperts) {
            x = sums[0][e];
            c = __float_as_int(sums[kSides][e]);
#pragma unroll
            for (int i = 1; i < kSides; ++i) x += sums[i][e], c += __float_as_int(sums[kSides + i][e]);
            all[e] = x;
            slots[e] = c;
        }
        __syncthreads();
    }
    // the sequence's loss
    float dot = 0.0f;
    int32_t used = 0;
    for (uint32_t e = threadIdx.x; e < a.E; e += kThreads) {
        dot += (float)slots[e] * all[e];
        used += slots[e];
        a.counts[(uint64_t)s * a.E + e] = slots[e];
    }
    dot = lanes_add<32>(dot);
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
        a.live[s] = part.parts > 0 ? live_tokens : -1;
    }
    // the call's
    if (a.sequences == 1)
        __syncthreads();
    else if (!last_of(a.arrived + kCounters - 1, a.sequences))
        return;
    dot = 0.0f;
    int32_t alive = 0;
    bool backwards = false;
    for (uint32_t i = threadIdx.x; i < a.sequences; i += kThreads) {
        const int32_t m = a.live[i];
        dot += a.losses[i];
        alive += m > 0 ? 1 : 0;
        backwards |= m < 0;
    }
    dot = lanes_add<32>(dot);
    alive = __reduce_add_sync(0xFFFFFFFFu, alive);
    if (__any_sync(0xFFFFFFFFu, backwards)) alive = -2 * (int32_t)ZCCL_MAX_SEQUENCES;  // below 0 whatever the others have
    if (lane == 0) red[warp] = dot, used_by[warp] = alive;
    __syncthreads();
    if (threadIdx.x == 0) {
        float d = 0.0f;
        int32_t n = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) d += red[w], n += used_by[w];
        // sequences of a table that runs backwards may share tokens: none of them has a loss, or a gradient
        *a.loss = n > 0 ? a.coefficient * (d / (float)n) : n < 0 ? __uint_as_float(0x7FC00000u) : 0.0f;
        n = max(n, 0);
        a.live[a.sequences] = n;
    }
}

template <typename T, int kRead, int L, int J>
__global__ void __launch_bounds__(kThreads) balance_backward_kernel(BalanceArgs a)
{
    pdl_wait();
    Part part;
    if (!part_of<true>(a, &part)) return;
    const uint32_t s = part.sequence;
    const bool counted = s < a.sequences;
    if (part.lo >= part.hi || (!counted && a.accumulate)) return;
    Walk<T, kRead, L, J> walk;
    walk.open(a, part.lo, part.hi, counted);
    T* out = static_cast<T*>(a.grad) + walk.t * a.grad_stride;
    // what a unit of an expert's shares adds to the loss
    float f[J] = {};
    uint32_t named = 0;  // experts below it count
    if (counted) {
        int32_t c[J], used = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const uint32_t e = walk.row.expert(walk.li, j);
            c[j] = e < a.E ? a.counts[(uint64_t)s * a.E + e] : 0;
            used += c[j];
        }
#pragma unroll
        for (int o = L / 2; o > 0; o /= 2) used += __shfl_xor_sync(0xFFFFFFFFu, used, o);
        const float up = a.coefficient * (a.grad_loss != nullptr ? *a.grad_loss : 1.0f);
        const float each = (float)used * (float)a.live[s] * (float)a.live[a.sequences];
        named = each > 0.0f ? a.E : 0;
        if (named == 0 && a.accumulate) return;
        const float unit = named > 0 ? up * ((float)a.E / each) : 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) f[j] = unit * (float)c[j];
    }
    for (; walk.more(); walk.t += walk.kStep, out += walk.kStep * a.grad_stride) {
        float l[J], g[J], slope[J], sum;
        const Choices<L> chosen = walk.take(a, l, counted);
        const bool there = walk.t < walk.hi, counts = chosen.each(named, walk.li, [](int32_t) {});
        if (!__all_sync(0xFFFFFFFFu, counts) && !counts)
#pragma unroll
            for (int j = 0; j < J; ++j) l[j] = -kInf;  // whatever it holds
        const float share = scores<true, L, J>(a, l, g, slope, f, &sum);
#pragma unroll
        for (int j = 0; j < J; j += 2) {
            float2 q = __fadd2_rn(make_float2(f[j], f[j + 1]), make_float2(-sum, -sum));
            q = __fmul2_rn(__fmul2_rn(make_float2(g[j], g[j + 1]), make_float2(share, share)), q);
            if (a.sigmoid) q = __fmul2_rn(q, make_float2(slope[j], slope[j + 1]));
            g[j] = q.x, g[j + 1] = q.y;
        }
        if (!counts) {  // none, whatever the loss's gradient is
            if (!there || a.accumulate) continue;
#pragma unroll
            for (int j = 0; j < J; ++j) g[j] = 0.0f;
            store_row<T, kRead, L, J>(out, g, walk.li, a.E);
            continue;
        }
        if (a.accumulate) {
            Logits<T, kRead, L, J> old;
            old.load(out, walk.li, a.E);
            old.get(l, walk.li, a.E);
#pragma unroll
            for (int j = 0; j < J; ++j) g[j] += l[j];
        }
        store_row<T, kRead, L, J>(out, g, walk.li, a.E);
    }
}

using BalanceKernel = void (*)(BalanceArgs);
template <typename T, int kRead>
BalanceKernel balance_for(uint32_t experts, bool backward)
{
    if (experts <= 64) return backward ? balance_backward_kernel<T, kRead, 8, 8> : balance_kernel<T, kRead, 8, 8>;
    if (experts <= 128) return backward ? balance_backward_kernel<T, kRead, 16, 8> : balance_kernel<T, kRead, 16, 8>;
    if (experts <= 256) return backward ? balance_backward_kernel<T, kRead, 32, 8> : balance_kernel<T, kRead, 32, 8>;
    return backward ? balance_backward_kernel<T, kRead, 32, 16> : balance_kernel<T, kRead, 32, 16>;
}
template <typename T>
BalanceKernel balance_for(const BalanceArgs& a, bool backward)
{
    const auto on_16 = [&](const void* p, uint64_t stride) {
        return is_aligned(p, 16) && (a.tokens <= 1 || stride * sizeof(T) % 16 == 0);
    };
    if (a.E % (16 / sizeof(T)) != 0 || !on_16(a.logits, a.stride) || (backward && !on_16(a.grad, a.grad_stride)))
        return balance_for<T, kOneByOne>(a.E, backward);
    const bool whole = a.E == 64 || a.E == 128 || a.E == 256 || a.E == ZCCL_MAX_EXPERTS;
    return whole ? balance_for<T, kWhole>(a.E, backward) : balance_for<T, kNeighbours>(a.E, backward);
}
BalanceKernel balance_for(const BalanceArgs& a, int dtype, bool backward)
{
    return dtype == ZCCL_BF16 ? balance_for<__nv_bfloat16>(a, backward) : balance_for<float>(a, backward);
}

// Tokens of a part, and the CTAs that there are parts for.  One sequence: as many parts
// as two a SM hold, or one where its registers (more than 256 experts) or the joining of
// its parts (more than 128) ask for fewer: 16384 x 512 (loss and gradient) 25 us
// with 152 parts, 36 with 304; x 256 19.3 and 21.5.  Several sequences have a part each that is not whole, which is counted in.
constexpr uint32_t kPartTokens = 64;
uint64_t most_parts(uint32_t sequences, uint32_t experts)
{
    const uint32_t most = experts > 256 || (sequences == 1 && experts > 128) ? 152 : 304;
    return sequences == 1 ? most : sequences < most / 2 ? most - sequences : most / 2;
}
uint32_t chunk_of(uint64_t tokens, uint32_t sequences, uint32_t experts)
{
    if (sequences > kFewSequences) return 0;
    const uint64_t most = most_parts(sequences, experts), chunk = (tokens + most - 1) / most;
    return (uint32_t)(chunk > kPartTokens ? chunk : kPartTokens);
}
uint32_t grid_of(uint64_t tokens, uint32_t sequences, uint32_t chunk, bool backward)
{
    if (chunk == 0) {
        const uint64_t others = (tokens + kPartTokens - 1) / kPartTokens + 1;
        return sequences + (backward ? (uint32_t)(others < 1216 ? others : 1216) : 0);
    }
    // each sequence (and the tokens before and behind them) has at most one part that is not whole
    return (uint32_t)(tokens / chunk) + sequences + (backward ? 2 : 1);
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
    const uint64_t parts = sequences > kFewSequences ? 0 : most_parts(sequences, experts) + sequences + 1;
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
    a.chunk = chunk_of(tokens, sequences, a.E);
    const uint32_t grid = grid_of(tokens, sequences, a.chunk, false);
    a.part_counts = reinterpret_cast<int32_t*>(a.part_scores + (uint64_t)grid * a.E);
    return launched(launch_dependent(balance_for(a, dtype, false), grid, kThreads, 0, stream, a));
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
    a.chunk = chunk_of(tokens, sequences, a.E);
    const uint32_t grid = grid_of(tokens, sequences, a.chunk, true);
    return launched(launch_dependent(balance_for(a, dtype, true), grid, kThreads, 0, stream, a));
}

}  // extern "C"
