// Log probabilities of given tokens, entropy, rank and the most likely tokens,
// from one pass over each row of logits.
//
//   m = max x,  l = sum 2^((x - m) c),  s = sum 2^((x - m) c) (x - m) c,  c = log2 e
//   log p(x) = (x - m) - ln l,   entropy = ln l - ln 2 s / l
// A thread's sums run against a reference R at most 8 below its m, so terms of s have both
// signs; (x - R) c is one fma, x c - M with M = R c rounded.  At the end they are moved to m,
// s by (m - R) c l, a few roundings of at most 12 l.  -infinity and NaN have probability
// 0: they are raised to a finite value whose exponential is 0.
//
// A thread keeps its own (m, l, s), in fp32, and rescales when a batch of 64 bytes
// brings a larger value, which is rare after the first ones.  Rank counts larger
// values, with a packed comparison for two 16-bit values, and only in batches whose
// maximum reaches the token's value.
//
// The k most likely.  The pass itself only leaves each group of 4 lanes with its
// largest value.  The k-th largest of those, tau, is no larger than the row's k-th
// value, so only threads that reach tau hold candidates, about k of 256: their values
// are read again (from L2) and those >= tau ordered by value, then by index.  Where
// many threads tie at tau (constant rows, rows masked with a type's lowest value) only
// larger values are gathered, and the ties are taken in the order of their indices
// until k are found.  What overflows the list of candidates even so is found one at a
// time; the result is exact in each case.
//
// Few rows: the CTAs of a cluster share a row, and the first joins their sums and
// lists, in order.  No atomics decide a result.  2049 rows of 151936 bf16 values: 135 us
// with 5 alternatives (4610 GB/s, 68% of a measured copy), 112 without; one row with 20
// alternatives 12 us.  Without alternatives it is near HBM's rate; with them a CTA reads
// nothing new while it searches, and the whole issues in 62% of the slots (9.4
// instructions a value).  Bulk prefetches to L2 ahead of the loads: 2049 rows 135 -> 129,
// but 300 rows 27 -> 34 us, 20 alternatives of fp16 161 -> 170.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "logits.cuh"
#include "qmv_common.cuh"

namespace bqd {
namespace {

using namespace qmvdev;

constexpr int kThreadsP = 256;
constexpr int kGroups = kThreadsP / 4;
constexpr int kMaxPartsP = 8;
constexpr int kMaxTop = BQD_MAX_TOP;
constexpr int kList = 2048;            // candidates
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

static_assert(kMaxTop <= kGroups, "the k-th largest of the groups' maxima is taken");

struct Params {
    const void *logits;
    int64_t stride;
    int V, parts, top;
    const int32_t *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t *rank, *top_ids;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint64_t two(float a, float b)
{
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float2 untwo(uint64_t x)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
    return f;
}

// two fp32 operations in one instruction, each rounded as by itself
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// Sums of a set of values, relative to its largest
struct Sums {
    float m, l, s;
};

__device__ __forceinline__ Sums join(const Sums &a, const Sums &b)
{
    Sums r = {fmaxf(a.m, b.m), 0.0f, 0.0f};
    const Sums both[2] = {a, b};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const Sums &x = both[i];
        if (x.l == 0.0f) continue;  // nothing: m may be -infinity
        const float d = x.m == r.m ? 0.0f : fmaxf((x.m - r.m) * kLog2e, -1e30f), f = ex2(d);
        r.l = fmaf(x.l, f, r.l);
        r.s = fmaf(fmaf(d, x.l, x.s), f, r.s);
    }
    return r;
}

// Larger keys come first: value, then the lower index.  0 stands for no entry.
__device__ __forceinline__ uint64_t key_of(float v, int i)
{
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 is 0
    return (uint64_t)(b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u)) << 32 | (0xFFFFFFFFu - (uint32_t)i);
}

__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b ^ ((b >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <typename T>
__global__ void __launch_bounds__(kThreadsP, 4)
token_logprobs_kernel(const Params p)
{
    using X = lg::Vec<T>;
    constexpr int E = X::E, B = 4;  // vectors of a batch
    __shared__ uint64_t list[kList];
    __shared__ uint64_t best[kMaxTop];      // this part's k first, in order
    __shared__ __align__(16) float group_max[kGroups];
    __shared__ int hit[kThreadsP];
    __shared__ Sums warp_sums[kThreadsP / 32], part_sums;
    __shared__ int warp_count[kThreadsP / 32], part_count, listed, threads_hit, threads_tied;
    __shared__ float tau;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = p.parts > 1 ? (int)cluster_ctarank() : 0;
    const int64_t r = blockIdx.x / p.parts;
    const T *row = static_cast<const T *>(p.logits) + r * p.stride;
    const lg::Part<T> at(row, p.V, part, p.parts);
    const int token = p.tokens ? p.tokens[r] : -1;
    const bool given = (unsigned)token < (unsigned)p.V;
    float xt = INFINITY;                    // no token: nothing comes before it
    if (given) {
        xt = X::one(row + token);
        if (!(xt == xt)) xt = -INFINITY;
    }
    const bool ranked = p.rank && given;

    // ---- the pass ----------------------------------------------------------------
    // The reference R starts at -kFar and follows m, the largest value so far, in steps of 8 or more;
    // t = x c - M with M = R c, one rounding each; what M is off from R c, less
    // than 1 up to there, is taken back at the end
    constexpr float kFar = X::kLow == -65504.0f ? 6e4f : 5e5f;  // (kLow is far below -kFar)
    float m = -INFINITY, R = -kFar, M = R * kLog2e;
    uint64_t l2 = two(0.0f, 0.0f), s2 = two(0.0f, 0.0f);
    int before = 0;                         // entries before the token
    const float xt_below = xt == -INFINITY ? xt : X::below(xt);
    auto rank_single = [&](float v, int i) {
        if (!(v == v)) v = -INFINITY;
        before += ranked && (v > xt || (v == xt && i < token));
    };
    auto rank_vector = [&](typename X::Count &n, const uint4 &u, int q) {
        const int i0 = at.first + q * E;
        if (i0 > token || (i0 + E <= token && xt > -INFINITY)) {
            n.add(u, i0 > token ? xt : xt_below);  // an equal value counts where it is before the token
        } else {
            float x[E];
            X::values(u, x);
#pragma unroll
            for (int e = 0; e < E; ++e) rank_single(x[e], i0 + e);
        }
    };
    auto raise = [&](float to) {            // the reference, once m is 8 above it
        const float N = to * kLog2e, d = fmaxf(M - N, -1e30f), f = ex2(d);
        const uint64_t dd = two(d, d), ff = two(f, f);
        s2 = mul2(fma2(dd, l2, s2), ff);
        l2 = mul2(l2, ff);
        R = to, M = N;
    };
    auto vector = [&](const uint4 &u) {
        float x[E];
        X::values(X::raised(u), x);
        const uint64_t mm = two(-M, -M), cc = two(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const uint64_t t2 = fma2(two(x[i], x[i + 1]), cc, mm);
            const float2 t = untwo(t2);
            const uint64_t e = two(ex2(t.x), ex2(t.y));
            l2 = add2(l2, e);
            s2 = fma2(e, t2, s2);
        }
    };
    auto single = [&](float v, int i) {
        rank_single(v, i);
        m = fmaxf(m, v);
        if (m > R + 8.0f) raise(m);
        const float t = fmaf(fmaxf(v, X::kLow), kLog2e, -M), e = ex2(t);
        l2 = add2(l2, two(e, 0.0f));
        s2 = fma2(two(e, 0.0f), two(t, 0.0f), s2);
    };
    if (tid < at.head) single(X::one(row + tid), tid);
    if (tid < at.tail) single(X::one(row + at.tail_at + tid), at.tail_at + tid);
    int q = at.q0 + tid;
    uint4 next[B];
    auto load = [&] {
        if (q + (B - 1) * kThreadsP < at.q1) {
#pragma unroll
            for (int j = 0; j < B; ++j) next[j] = __ldg(at.body + q + j * kThreadsP);
        }
    };
    load();
    while (q + (B - 1) * kThreadsP < at.q1) {
        uint4 u[B];
#pragma unroll
        for (int j = 0; j < B; ++j) u[j] = next[j];
        const int q_now = q;
        q += B * kThreadsP;
        load();                             // of the next batch, while this one is summed
        const float high = fmaxf(fmaxf(X::max(u[0]), X::max(u[1])), fmaxf(X::max(u[2]), X::max(u[3])));
        m = fmaxf(m, high);
        if (m > R + 8.0f) raise(m);
        if (ranked && !(high < xt)) {
            typename X::Count n;
#pragma unroll
            for (int j = 0; j < B; ++j) rank_vector(n, u[j], q_now + j * kThreadsP);
            before += n.value();
        }
#pragma unroll
        for (int j = 0; j < B; ++j) vector(u[j]);
    }
    for (; q < at.q1; q += kThreadsP) {
        const uint4 u = __ldg(at.body + q);
        const float high = X::max(u);
        m = fmaxf(m, high);
        if (m > R + 8.0f) raise(m);
        if (ranked && !(high < xt)) {
            typename X::Count n;
            rank_vector(n, u, q);
            before += n.value();
        }
        vector(u);
    }
    Sums mine = {m, 0.0f, 0.0f};
    if (m >= -kFar && m <= kFar) {
        const float2 l = untwo(l2), s = untwo(s2);
        const float off = fmaf(m, kLog2e, -M), f = ex2(-off);
        mine.l = (l.x + l.y) * f;
        mine.s = fmaf(-off, l.x + l.y, s.x + s.y) * f;
    } else if (m > -INFINITY) {
        // a thread whose largest value is far from 0: again, by differences from m (+infinity leaves l = 0)
        auto one = [&](float v) {
            const float t = fmaxf((v - m) * kLog2e, -1e30f), e = ex2(t);  // (-infinity and NaN: 0)
            mine.l += e;
            mine.s = fmaf(e, t, mine.s);
        };
        if (tid < at.head) one(X::one(row + tid));
        if (tid < at.tail) one(X::one(row + at.tail_at + tid));
        for (int k = at.q0 + tid; k < at.q1; k += kThreadsP) {
            float x[E];
            X::values(__ldg(at.body + k), x);
#pragma unroll
            for (int e = 0; e < E; ++e) one(x[e]);
        }
    }
    const float own_max = m;

    // ---- the part's sums -----------------------------------------------------------
    {
        Sums a = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Sums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o),
                            __shfl_xor_sync(0xffffffffu, a.s, o)};
            a = (lane & o) ? join(b, a) : join(a, b);  // the same sum in both lanes
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        if (lane == 0) warp_sums[warp] = a, warp_count[warp] = before;
    }
    if (p.top > 0) {
        float g = own_max;
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
        g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
        if ((tid & 3) == 0) group_max[tid >> 2] = g;
    }
    if (tid == 0) listed = threads_hit = threads_tied = 0;
    if (tid < kMaxTop) best[tid] = 0;
    __syncthreads();
    if (warp == kThreadsP / 32 - 1) {
        constexpr int kWarpsP = kThreadsP / 32;
        Sums a = warp_sums[lane % kWarpsP];
        int n = warp_count[lane % kWarpsP];
#pragma unroll
        for (int o = kWarpsP / 2; o > 0; o >>= 1) {
            const Sums b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.l, o),
                            __shfl_xor_sync(0xffffffffu, a.s, o)};
            a = (lane & o) ? join(b, a) : join(a, b);
            n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        if (lane == 0) part_sums = a, part_count = n;
    }

    // ---- the part's k first ----------------------------------------------------------
    if (p.top > 0) {
        if (tid < kGroups) {
            int n = 0;
            const float g = group_max[tid];
#pragma unroll 4
            for (int i = 0; i < kGroups; i += 4) {
                const float4 o = *reinterpret_cast<const float4 *>(&group_max[i]);
                n += (o.x > g || (o.x == g && i < tid)) + (o.y > g || (o.y == g && i + 1 < tid)) +
                     (o.z > g || (o.z == g && i + 2 < tid)) + (o.w > g || (o.w == g && i + 3 < tid));
            }
            if (n == p.top - 1) tau = g;
        }
        __syncthreads();
        const float t = tau;                // -infinity: every value above it is a candidate
        const bool tied = own_max == t && t > -INFINITY;
        if (own_max > t) hit[atomicAdd(&threads_hit, 1)] = tid;  // (their order is of no consequence)
        else if (tied) atomicAdd(&threads_tied, 1);
        __syncthreads();
        const bool few = threads_tied <= 16;  // ties are candidates like others
        if (few && tied) hit[atomicAdd(&threads_hit, 1)] = tid;
        __syncthreads();
        const int hits = threads_hit, each = at.q1 - at.q0 > 0 ? (at.q1 - at.q0 + kThreadsP - 1) / kThreadsP : 0;
        for (int ties = few; ; ties = 0) {
            auto offer = [&](float v, int i) {
                if (v > t || (ties && v == t && t > -INFINITY)) {
                    const int n = atomicAdd(&listed, 1);
                    if (n < kList) list[n] = key_of(v, i);
                }
            };
            if (tid < at.head) offer(X::one(row + tid), tid);
            if (tid < at.tail) offer(X::one(row + at.tail_at + tid), at.tail_at + tid);
            // all vectors of the threads that were hit, shared out over all threads, eight on their way
            const int all = hits * each;
            for (int i0 = tid; i0 < all; i0 += 8 * kThreadsP) {
                uint4 u[8];
                int qs[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int i = i0 + k * kThreadsP;
                    qs[k] = i < all ? at.q0 + hit[i / each] + i % each * kThreadsP : at.q1;
                    if (qs[k] < at.q1) u[k] = __ldg(at.body + qs[k]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (qs[k] >= at.q1) continue;
                    const float top = X::max(u[k]);
                    if (top > t || (ties && top == t)) {
                        float x[E];
                        X::values(u[k], x);
#pragma unroll
                        for (int e = 0; e < E; ++e) offer(x[e], at.first + qs[k] * E + e);
                    }
                }
            }
            __syncthreads();
            if (listed <= kList || !ties) {
                // ties in the order of their indices, until there are k
                if (!ties && listed <= kList && t > -INFINITY) {
                    const int lo = at.head ? 0 : at.first + at.q0 * E;
                    const int hi = at.tail ? p.V : at.first + at.q1 * E;
                    for (unsigned i0 = lo; i0 < (unsigned)hi; i0 += 16 * kThreadsP) {  // (passes 2^31 for the largest V)
                        const int have = listed;
                        if (have >= p.top) break;
                        const int a = (int)min((unsigned)hi, i0 + tid * 16), b = min(hi, a + 16);
                        int n = 0;
                        for (int i = a; i < b; ++i) n += X::one(row + i) == t;
                        int sum = n;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int x = __shfl_up_sync(0xffffffffu, sum, o);
                            if (lane >= o) sum += x;
                        }
                        if (lane == 31) warp_count[warp] = sum;
                        __syncthreads();
                        int to = have + sum - n, all = have;
                        for (int w = 0; w < kThreadsP / 32; ++w) {
                            if (w < warp) to += warp_count[w];
                            all += warp_count[w];
                        }
                        for (int i = a; i < b && to < p.top; ++i)
                            if (X::one(row + i) == t) list[to++] = key_of(t, i);
                        __syncthreads();
                        if (tid == 0) listed = min(all, p.top);
                        __syncthreads();
                    }
                }
                break;
            }
            __syncthreads();
            if (tid == 0) listed = 0;
            __syncthreads();
        }
        const int n = listed;
        if (n <= kList) {
            for (int i = tid; i < n; i += kThreadsP) {
                const uint64_t mine = list[i];
                int above = 0;
                for (int k = 0; k < n; ++k) above += list[k] > mine;
                if (above < p.top) best[above] = mine;
            }
        } else {
            // one at a time: the largest key below the last
            uint64_t last = ~0ull;
            for (int k = 0; k < p.top; ++k) {
                uint64_t top = 0;
                auto see = [&](float v, int i) {
                    if (!(v > -INFINITY)) return;
                    const uint64_t x = key_of(v, i);
                    if (x < last && x > top) top = x;
                };
                if (tid < at.head) see(X::one(row + tid), tid);
                if (tid < at.tail) see(X::one(row + at.tail_at + tid), at.tail_at + tid);
                for (int q = at.q0 + tid; q < at.q1; q += kThreadsP) {
                    float x[E];
                    X::values(__ldg(at.body + q), x);
#pragma unroll
                    for (int e = 0; e < E; ++e) see(x[e], at.first + q * E + e);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t x = __shfl_xor_sync(0xffffffffu, top, o);
                    if (x > top) top = x;
                }
                __syncthreads();
                if (lane == 0) list[warp] = top;
                __syncthreads();
                for (int w = 0; w < kThreadsP / 32; ++w)
                    if (list[w] > top) top = list[w];
                if (tid == 0) best[k] = top;
                last = top;
                if (top == 0) break;
            }
        }
    }
    __syncthreads();

    // ---- join the parts -------------------------------------------------------------
    Sums all = part_sums;
    int come_before = part_count;
    int n = p.top;
    const uint64_t *from = best;
    if (p.parts > 1) {
        cluster_sync();
        if (part == 0) {
            n = p.parts * p.top;
            for (int i = tid; i < n; i += kThreadsP) {
                uint32_t a;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(&best[i % p.top])), "r"(i / p.top));
                asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(list[i]) : "r"(a) : "memory");
            }
            from = list;
            for (int k = 1; k < p.parts; ++k) {
                uint32_t a, b;
                Sums x;
                int c;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(&part_sums)), "r"(k));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(b) : "r"(smem_addr(&part_count)), "r"(k));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.m) : "r"(a) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.l) : "r"(a + 4) : "memory");
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.s) : "r"(a + 8) : "memory");
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(b) : "memory");
                all = join(all, x);
                come_before += c;
            }
        }
        cluster_sync();  // no CTA leaves while another reads its shared memory
        if (part != 0) return;
        __syncthreads();
    }
    // a row without a value above -infinity has no distribution, nor has one with +infinity
    const bool none = all.m == -INFINITY;
    const float ln_l = all.m == INFINITY ? NAN : logf(all.l);
    auto log_p = [&](float x) { return none || x == -INFINITY ? (ln_l == ln_l || none ? -INFINITY : NAN) : x - all.m - ln_l; };
    if (tid == 0) {
        if (p.logprob) p.logprob[r] = given ? log_p(xt) : -INFINITY;
        if (p.entropy) p.entropy[r] = none ? 0.0f : ln_l - kLn2 * (all.s / all.l);
        if (p.rank) p.rank[r] = given ? come_before : -1;
    }
    for (int i = tid; i < n; i += kThreadsP) {
        const uint64_t mine = from[i];
        // the parts' lists are in order: larger keys of each, by bisection (keys are apart from each
        // other but for those of no entry, which keep their order)
        const int own = i / p.top;
        int above = i - own * p.top;
        for (int k = 0; k < p.parts; ++k) {
            if (k == own) continue;
            int lo = 0, hi = p.top;
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (from[k * p.top + mid] > mine || (mine == 0 && k < own)) lo = mid + 1;
                else hi = mid;
            }
            above += lo;
        }
        if (above >= p.top) continue;
        if (p.top_ids) p.top_ids[r * p.top + above] = mine ? (int32_t)(0xFFFFFFFFu - (uint32_t)mine) : -1;
        if (p.top_logprobs) p.top_logprobs[r * p.top + above] = mine ? log_p(value_of(mine)) : -INFINITY;
    }
}

template <typename T>
int launch(Params &p, int64_t rows, cudaStream_t s)
{
    // one CTA an SM is enough to share rows for: 150 rows of 151936, 21 us; two, 30 (each has its own list to find)
    p.parts = lg::parts_of(rows, p.V, sm_count(), kMaxPartsP);
    if (rows * p.parts > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.parts));
    cfg.blockDim = dim3(kThreadsP);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, static_cast<const Params &>(p)));
}

bool at(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace bqd

extern "C" int bqd_token_logprobs(const void *logits, int dtype, int64_t row_stride, int64_t rows, int64_t V,
                                  const int32_t *tokens, int top, float *logprob, float *entropy, int32_t *rank,
                                  int32_t *top_ids, float *top_logprobs, bqd_stream_t stream)
{
    using namespace bqd;
    if (dtype != BQD_DTYPE_F16 && dtype != BQD_DTYPE_F32 && dtype != BQD_DTYPE_BF16) return BQD_ERR_INVALID_ARG;
    if (rows < 0 || rows > ((int64_t)1 << 28) || V < 1 || V > ((int64_t)1 << 31) - 1024) return BQD_ERR_INVALID_ARG;
    if ((rows > 1 && row_stride < V) || row_stride > ((int64_t)1 << 40)) return BQD_ERR_INVALID_ARG;
    if (top < 0 || top > BQD_MAX_TOP || ((logprob || rank) && !tokens)) return BQD_ERR_INVALID_ARG;
    if (rows == 0) return BQD_OK;
    if (!logits) return BQD_ERR_INVALID_ARG;
    if (!at(logits, dtype == BQD_DTYPE_F32 ? 4 : 2) || !at(tokens, 4) || !at(logprob, 4) || !at(entropy, 4) ||
        !at(rank, 4) || !at(top_ids, 4) || !at(top_logprobs, 4))
        return BQD_ERR_ALIGNMENT;
    if (!top_ids && !top_logprobs) top = 0;
    if (top == 0 && !logprob && !entropy && !rank) return BQD_OK;
    Params p;
    p.logits = logits, p.stride = row_stride, p.V = (int)V, p.parts = 1, p.top = top;
    p.tokens = tokens;
    p.logprob = logprob, p.entropy = entropy, p.rank = rank, p.top_ids = top_ids, p.top_logprobs = top_logprobs;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == BQD_DTYPE_F16    ? launch<__half>(p, rows, s)
           : dtype == BQD_DTYPE_BF16 ? launch<__nv_bfloat16>(p, rows, s)
                                     : launch<float>(p, rows, s);
}
