// Attention over a paged 8-bit cache for many queries of a sequence (prefill
// chunks): both products on the 5th-generation tensor cores.
//
// The mathematics is that of the few-query kernel (kv_attend.cu): with f the
// score scale times log2(e) and s^k_b, s^v_b the scales of 16-token block b,
//   x_ij = f s^k_b (q_i . c^k_j) + log2 s^v_b,   p_ij = 2^(x_ij - m_i),
//   O_i = sum_j p_ij c^v_j,   l_i = sum_b (sum_{j in b} p_ij) / s^v_b,
//   out = O / l,   lse = ln 2 (m + log2 l),
// with m_i replaced only when x passes it by 15 (p < 2^15 fits fp16, and what is
// small keeps more bits, not fewer).
//
// Rows of a tile are (query, head of the group) pairs, so a tile of 128 rows
// reads each K and V code once for the whole group.  A CTA owns two tiles of
// 128 rows (one for head_dim 256, and where there are no more rows) and walks
// the keys in steps of KT.  Two forms share everything but what fills the K and
// V tiles:
//   staged   a first kernel converts a row's codes to fp16 tiles in scratch, once
//            for all of its query tiles, and one thread copies them by TMA.  For
//            calls of several query tiles.
//   direct   seven warps convert the codes in the kernel: for one query tile a
//            row, calls without scratch, and rows longer than planned.  Their
//            code and the softmax's share the instruction cache and the issue
//            slots: 2048 queries at 8192 keys take 311 us staged, 473 direct.
// K and V tiles have the same layout ([64-dim panel][key] rows of 128 bytes, 128-
// byte swizzle): K is a K-major operand of S = Q K^T, V an MN-major one of O = P V,
// so V needs no transpose.  Roles:
//   warps 0-3, 4-7   softmax of tile 0 / 1: one thread a row.  S goes from TMEM to
//                    registers, P back over it as fp16; O is rescaled in TMEM when
//                    m is replaced.  Staged: by halves of a step (head_dim 256: whole
//                    steps), so that P V of the first runs while the second is computed
//   staged: warp 8   TMA copies;  direct: warps 8-11 (K), 13-15 (V) convert, loads
//                    of the next step's codes in flight
//   last / 12th      TMEM, and one elected lane that issues every MMA
// With two tiles the tensor cores work on one while the other's softmax runs;
// with one tile S alternates between two TMEM buffers, so that S of the next
// step is computed during the softmax of this one.  Steps of 64 keys with two S
// buffers for each of two tiles would take the MMAs off a tile's own chain, but
// N = 64 score products take as long as N = 128 ones (476 us against 363).
// Bound by the chain of a tile's step: 275 cycles to read S, 2 x 540 of softmax,
// 150 to issue, 1130 of P V and the next S, 700 of waiting for tiles, against
// 2112 of MMAs for both tiles: the tensor pipe is active 58% of the time (1160
// TFLOP/s at 2048 queries, 8192 keys, 48 heads of 128).
// Where few tiles face many keys, several CTAs share a tile's steps (Split).
// Every wait is bounded; on expiry a role stops, what it issued is drained,
// TMEM is freed, and bqd_device_status reports it.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "kv_common.cuh"
#include "qmv_common.cuh"
#include "tc05.cuh"

namespace bqd {
namespace kv {
namespace {

using namespace qmvdev;
using namespace tc05;

constexpr int kSoftWarps = 8;
constexpr int kMmaWarpF = 12;
constexpr int kWarpsK = 4, kWarpsV = 3;           // warps 8-11 convert K, 13-15 V
constexpr int kThreadsF = 512;
constexpr int kThreadsStaged = (kSoftWarps + 2) * 32;  // warp 8 copies the staged tiles, warp 9 issues
constexpr int kStages = 2;
constexpr int kScaleRing = 4;  // steps whose scales are kept: a slot is written again only after
                               // both softmaxes of the step four before have finished
constexpr int64_t kMaxTiles = 65535;  // query tiles of a launch (its grid's slowest place)
constexpr int64_t kMaxScratch = (int64_t)2 << 30;  // bytes that a call may ask for
constexpr float kGrow = 15.0f;  // p stays below 2^15, inside fp16

__device__ unsigned int g_prefill_timeouts = 0;

template <int D>
struct Plan {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kRows = 128 * kTiles;
    static constexpr int KT = D == 256 ? 64 : 128;     // keys of a step
    static constexpr int kPanels = D / 64;
    static constexpr uint32_t kPanelQ = 128 * 128;     // bytes of 128 rows of a panel
    static constexpr uint32_t kPanelKV = KT * 128;
    static constexpr uint32_t kQ = kTiles * kPanels * kPanelQ;
    static constexpr uint32_t kKV = kPanels * kPanelKV;  // one K or V tile
    static constexpr uint32_t kOffK = kQ, kOffV = kOffK + kStages * kKV, kOffEnd = kOffV + kStages * kKV;
    static constexpr int kBlocks = KT / kBlock;
    // Parts of a step's softmax.  One tile's step of 64 keys is one part, its maximum found before the
    // exponentials: nothing hides a part's latency, and 32 columns are too few to do so by themselves
    // (2048 queries at 8192 keys: 361 us in halves, 340 in one part with the maximum beside the
    // exponentials, 326 so).
    static constexpr int kParts = kTiles == 1 ? 1 : 2;
    static constexpr size_t kSmem = 1024 + kOffEnd;
    // TMEM columns
    static constexpr uint32_t kS1 = KT, kO0 = 256, kO1 = 256 + D, kCols = 512;
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// The same value, unknown to the compiler: what is computed from it is computed
// where it is used, not kept in registers over a loop
__device__ __forceinline__ int opaque(int x)
{
    asm volatile("" : "+r"(x));
    return x;
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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Keys [lo, lo + steps * KT) of a row of length L that any of its queries sees; with a window, that any
// of the call's queries sees (without one the end stays the row's, so that nothing waits for `starts`).
struct RowSteps {
    int lo, steps;
    __device__ __forceinline__ RowSteps(int L, const Span &span, int window, int KT)
    {
        const int first = L - span.rest;  // position of query 0
        lo = window > 0 ? max(0, first + 1 - window) / KT * KT : 0;
        steps = span.n > 0 && L > lo ? (L - lo + KT - 1) / KT : 0;
        if (window > 0) steps = min(steps, max(0, first + span.n - lo + KT - 1) / KT);
    }
};

// Scratch of the staged form: the K and V tiles of every step as the MMAs read
// them, [row][head][step][K, V], then the scales of their blocks.
struct Staged {
    uint8_t *tiles;
    float2 *scales;
    int steps;      // of a row at most; 0: nothing is staged
};

// Where few query tiles face many keys, `count` CTAs share a tile's steps and
// leave O (not divided by l) with m and l; a second kernel joins them in order.
struct Split {
    float *o;       // [count][tokens * q_heads][D]
    float2 *ml;     // [count][tokens * q_heads]
    int count;      // 1: the CTA finishes its rows itself
    int first;      // row of the launch's first query tile: a launch has 65535 tiles at most
};

template <typename T, int D, int FMT, bool STAGED>
__global__ void __launch_bounds__(STAGED ? kThreadsStaged : kThreadsF, 1)
attend_prefill_kernel(const AttendArgs a, const Staged st, const Split sp, const __grid_constant__ CUtensorMap map,
                      unsigned long long wait_ns)
{
    using P = Plan<D>;
    using C = Code<FMT>;
    constexpr int kMmaWarp = STAGED ? kSoftWarps + 1 : kMmaWarpF;
    constexpr int kFillersK = STAGED ? 1 : kWarpsK, kFillersV = STAGED ? 1 : kWarpsV;
    using H = Half2Of<T>;
    constexpr int KT = P::KT;
    constexpr int kParts = STAGED ? P::kParts : 1;  // of a step's softmax
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[4 * kStages + 13 + kScaleRing];
    __shared__ __align__(16) float2 scales[kScaleRing][8];  // of a step's blocks: K's scale, log2 of V's
    __shared__ uint32_t tmem_at;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // query tiles in the slowest place of the grid, the last first: those see most keys, and
    // what starts last is short
    const int head = blockIdx.x, row = blockIdx.y;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int rows = span.n * a.group;
    const int share = blockIdx.z % sp.count;  // of the tile's steps
    const int r0 = (int)((gridDim.z - 1 - blockIdx.z) / sp.count) * P::kRows + sp.first;
    if (r0 >= rows) return;
    const int L = a.L.length(row);
    const RowSteps all_steps(L, span, a.window, KT);
    // rows that the scratch has no room for are the unstaged form's
    if (st.steps > 0 && (all_steps.steps <= st.steps) != STAGED) return;
    const int tiles = min(P::kTiles, (rows - r0 + 127) / 128);
    const int i_min = r0 / a.group, i_max = (min(r0 + P::kRows, rows) - 1) / a.group;
    const int p_first = L - span.rest;  // position of query 0
    const int hi = max(0, p_first + i_max + 1);
    const int lo = a.window > 0 ? max(0, p_first + i_min + 1 - a.window) : 0;
    const int k_first = lo / KT * KT, all = hi > k_first ? (hi - k_first + KT - 1) / KT : 0;
    const int from = (int)((int64_t)all * share / sp.count), steps = (int)((int64_t)all * (share + 1) / sp.count) - from;
    const int k_lo = k_first + from * KT;

    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    auto k_full = [&](int j) { return bar(j % kStages); };
    auto k_empty = [&](int j) { return bar(kStages + j % kStages); };
    auto v_full = [&](int j) { return bar(2 * kStages + j % kStages); };
    auto v_empty = [&](int j) { return bar(3 * kStages + j % kStages); };
    const uint32_t q_full = bar(4 * kStages);
    auto s_full = [&](int w) { return bar(4 * kStages + 1 + w); };
    auto p_full = [&](int w, int half) { return bar(half ? 4 * kStages + 9 + w : 4 * kStages + 3 + w); };
    auto pv_half = [&](int w) { return bar(4 * kStages + 11 + w); };
    auto o_full = [&](int w) { return bar(4 * kStages + 5 + w); };
    const uint32_t pv_done = bar(4 * kStages + 7), drained = bar(4 * kStages + 8);
    auto sc_full = [&](int j) { return bar(4 * kStages + 13 + j % kScaleRing); };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(k_full(i), kFillersK);
                mbar_init(k_empty(i), 1);
                mbar_init(v_full(i), kFillersV);
                mbar_init(v_empty(i), 1);
            }
            mbar_init(q_full, 128 * tiles);
            for (int w = 0; w < 2; ++w) {
                mbar_init(s_full(w), 1);
                mbar_init(p_full(w, 0), 128);
                mbar_init(p_full(w, 1), 128);
                mbar_init(pv_half(w), 1);
                mbar_init(o_full(w), 1);
            }
            mbar_init(pv_done, 1);
            mbar_init(drained, 1);
            for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full(i), 1);
        }
        __syncwarp();
        tmem_alloc(smem_addr(&tmem_at), P::kCols);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;
    const bool pair = tiles == 2;
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_for(b, parity & 1, wait_ns, &g_prefill_timeouts); };

    if (warp < kSoftWarps) {
        const int w = warp >> 2;  // tile
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // TMEM lane 32 (warp % 4), in bits 16..31
        const int trow = (warp & 3) * 32 + lane;
        const int r = r0 + w * 128 + trow;
        if (w < tiles) {
            const bool real = r < rows;
            const int pos = real ? p_first + r / a.group : -1;
            const uint32_t q_tile = base + w * (P::kPanels * P::kPanelQ);
            const int row0 = (warp & 3) * 32;  // the warp's rows of the tile
            // ---- q: scaled by 2^-e into fp16 (e of the row's largest magnitude) ----
            // fp16 keeps every bit of a bf16 value down to 2^-16 of that magnitude, and an absolute
            // 2^-25 of it below, of the order of what the fp32 sum of the scores rounds off
            // D / 8 lanes take a row, 16 bytes each, up to 16 passes in flight (one row a thread
            // took 8 us: each load touched 32 rows)
            constexpr int kRowLanes = D / 8, kRowsPass = 32 / kRowLanes, kPasses = kRowLanes;
            constexpr int kFlight = kPasses < 16 ? kPasses : 16;
            const unsigned group = a.group;
            float cs = 1.0f;  // of this thread's row: |f| 2^e
#pragma unroll 1
            for (int i0 = 0; i0 < kPasses; i0 += kFlight) {
                uint4 v[kFlight];
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const unsigned rr = r0 + w * 128 + row0 + (i0 + i) * kRowsPass + lane / kRowLanes;
                    v[i] = make_uint4(0, 0, 0, 0);
                    if (rr < (unsigned)rows) {
                        const unsigned i_q = rr / group;
                        const T *q = static_cast<const T *>(a.q) + (int64_t)(span.lo + i_q) * a.q_token +
                                     (int64_t)(head * group + rr - i_q * group) * a.q_head + lane % kRowLanes * 8;
                        if (a.q_vec) {
                            v[i] = __ldg(reinterpret_cast<const uint4 *>(q));
                        } else {
                            const unsigned short *u = reinterpret_cast<const unsigned short *>(q);
                            uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = (uint32_t)__ldg(u + 2 * k) | ((uint32_t)__ldg(u + 2 * k + 1) << 16);
                            v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kFlight; ++i) {
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t mx = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu),
                                           __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
                    uint32_t top = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                    for (int o = 1; o < kRowLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    int e = 0;
                    if (top != 0 && top < H::kInf)
                        e = max(-100, min(126, (int)((__float_as_uint(H::f1(top)) >> 23) & 0xFF) - 127));
                    // the sign of the scale goes with q, so that a larger product is a larger score
                    const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), a.scale);
                    const float up = fabsf(a.scale) * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int h = 0; h < kRowsPass; ++h) {
                        const float of_row = __shfl_sync(0xffffffffu, up, h * kRowLanes);
                        if (lane == (i0 + i) * kRowsPass + h) cs = of_row;
                    }
                    uint32_t h4[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = H::f2(x[k]);
                        h4[k] = Half2Of<__half>::pack(f.x * down, f.y * down);
                    }
                    const int tr = row0 + (i0 + i) * kRowsPass + lane / kRowLanes, u = lane % kRowLanes;
                    const uint32_t at = q_tile + (u >> 3) * P::kPanelQ + tr * 128 + (((u & 7) ^ (tr & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h4[0]), "r"(h4[1]), "r"(h4[2]),
                                 "r"(h4[3])
                                 : "memory");
                }
            }
            mbar_arrive(q_full);

            // ---- steps ------------------------------------------------------------
            const int p_low = p_first + (r0 + w * 128) / a.group;                               // positions of
            const int p_high = p_first + (min(r0 + w * 128 + 128, rows) - 1) / a.group;          // the tile's rows
            const uint32_t o_at = tmem + lanes + (w ? P::kO1 : P::kO0);
            // of a block's raw scores; above 0, so that -inf (masked) stays -inf
            auto factor = [&](float k) { return fmaxf(cs * k, 1.2e-38f); };
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int j = 0; j < steps; ++j) {
                const int slot = pair ? w : j & 1;
                const uint32_t s_at = tmem + lanes + (slot ? P::kS1 : 0);
                // the blocks' scales while S is on its way: shared memory answers slowly (300 to 400
                // cycles) while the MMAs read their operands from it
                ok = wait(sc_full(j), j / kScaleRing);
                float2 sr[P::kBlocks];
                if constexpr (STAGED) {
#pragma unroll
                    for (int b = 0; b < P::kBlocks; ++b) {
                        sr[b] = scales[j % kScaleRing][b];
                        sr[b].x = factor(sr[b].x);
                    }
                }
                ok = ok && wait(s_full(slot), pair ? j : j >> 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                fence_after();
                const int k0 = k_lo + j * KT;
                const bool whole = k0 + KT - 1 <= p_low && (a.window == 0 || k0 > p_high - a.window);
                const int last = pos - k0, first = a.window > 0 ? last - a.window : -1;  // seen: first < i <= last
                auto rescale = [&](float f) {  // O times f
                    fence_after();
#pragma unroll 1
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t o[16];
                        ld16(o_at + 16 * k, o);
                        ld_wait(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        st16(o_at + 16 * k, o);
                    }
                };
                if constexpr (STAGED) {
                    // Half of the step's columns at a time (but see kParts): the MMAs of the first half's P
                    // run while the second half is computed.  Exponentials are taken against the reference
                    // that is there, with the half's maximum found beside them; where a row passes its
                    // reference by too much (the first step, seldom after it) the warp replaces it and
                    // computes the half again.  P takes the place of scores that were read, two values a
                    // column.
                    constexpr int kHalf = KT / kParts, kHalfBlocks = kHalf / 16, kChunks = kHalf / 32;
                    uint32_t s[kParts][kChunks][32];
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) ld32(s_at + 32 * c, s[0][c]);
#pragma unroll
                    for (int half = 0; half < kParts; ++half) {
                        const float2 *v = sr + half * kHalfBlocks;
                        uint32_t (&sh)[kChunks][32] = s[half];
                        if (half == 1) {
#pragma unroll
                            for (int c = 0; c < kChunks; ++c) ld32(s_at + kHalf + 32 * c, sh[c]);
                        }
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) ld_wait(sh[c]);
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < kHalf; ++i)
                                if (half * kHalf + i > last || half * kHalf + i <= first) sh[i / 32][i % 32] = 0xFF800000u;  // -inf
                        }
                        if constexpr (kParts == 1) {
                            float mt = -INFINITY;
#pragma unroll
                            for (int b = 0; b < kHalfBlocks; ++b) {
                                const uint32_t *x = &sh[b / 2][16 * (b & 1)];
                                float top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
                                for (int i = 2; i < 16; i += 2)
                                    top = fmaxf(fmaxf(top, __uint_as_float(x[i])), __uint_as_float(x[i + 1]));
                                mt = fmaxf(mt, fmaf(top, v[b].x, v[b].y));
                            }
                            if (__any_sync(0xffffffffu, mt > m + kGrow)) {
                                const float mn = mt > m + kGrow ? mt : m;
                                const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                                m = mn;
                                l *= f;
                                if (j > 0) {
                                    ok = __all_sync(0xffffffffu, wait(pv_done, j - 1));  // it still adds to O
                                    if (!ok) break;
                                    rescale(f);
                                }
                            }
                        }
                        float sum;
                        while (true) {
                            const float ms = m == -INFINITY ? 0.0f : m;
                            float mt = -INFINITY;
                            sum = 0.0f;
#pragma unroll
                            for (int b = 0; b < kHalfBlocks; ++b) {
                                const uint32_t *x = &sh[b / 2][16 * (b & 1)];
                                const float add = v[b].y - ms;
                                const uint64_t ff = two(v[b].x, v[b].x), aa = two(add, add);
                                uint64_t part = two(0.0f, 0.0f);
                                float top = -INFINITY;
                                uint32_t p[8];
#pragma unroll
                                for (int i = 0; i < 16; i += 2) {
                                    const float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
                                    const float2 y = untwo(fma2(two(x0, x1), ff, aa));
                                    const float e0 = ex2(y.x), e1 = ex2(y.y);
                                    top = fmaxf(fmaxf(top, x0), x1);
                                    part = add2(part, two(e0, e1));
                                    p[i / 2] = Half2Of<__half>::pack(e0, e1);
                                }
                                if (kParts > 1) mt = fmaxf(mt, fmaf(top, v[b].x, v[b].y));
                                const float2 t = untwo(part);
                                sum = fmaf(t.x + t.y, ex2(-v[b].y), sum);
                                st8(s_at + half * (kHalf / 2) + 8 * b, p);
                            }
                            if (kParts == 1 || !__any_sync(0xffffffffu, mt > m + kGrow)) break;
                            const float mn = mt > m + kGrow ? mt : m;
                            const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                            m = mn;
                            l *= f;
                            if (j > 0 || half) {
                                // what still adds to O: the first half's product, or with one tile
                                // that of the step before (with two it is done before S comes)
                                if (!pair && j > 0) ok = wait(pv_done, j - 1);
                                if (ok && half) ok = wait(pv_half(w), j);
                                ok = __all_sync(0xffffffffu, ok);
                                if (!ok) break;
                                rescale(f);
                            }
                        }
                        if (!ok) break;
                        l += sum;
                        st_wait();
                        fence_before();
                        mbar_arrive(p_full(slot, half));
                    }
                } else {
                    // A small loop over 32 columns: unrolled over the step, this role and the converting
                    // ones outgrow the instruction cache and 128 registers (2048 queries at 8192 keys,
                    // head_dim 64 / 128 / 256: 337 / 473 / 713 us as a loop, 436 / 693 / 790 unrolled; 8 x 12
                    // of 128 at 8000 keys: 81 and 102).  Each load is waited for at once: nothing is in flight into
                    // registers over the loop's code.
                    const float2 *sc = scales[j % kScaleRing];
#pragma unroll 1
                    for (int c = 0; c < KT / 32; ++c) {
                        uint32_t s[32];
                        ld32(s_at + 32 * c, s);
                        ld_wait(s);
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (32 * c + i > last || 32 * c + i <= first) s[i] = 0xFF800000u;  // -inf
                        }
                        const float2 va = sc[2 * c], vb = sc[2 * c + 1];
                        const float fa = factor(va.x), fb = factor(vb.x);
                        float ta = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
                        float tb = fmaxf(__uint_as_float(s[16]), __uint_as_float(s[17]));
#pragma unroll
                        for (int i = 2; i < 16; i += 2) {
                            ta = fmaxf(fmaxf(ta, __uint_as_float(s[i])), __uint_as_float(s[i + 1]));
                            tb = fmaxf(fmaxf(tb, __uint_as_float(s[16 + i])), __uint_as_float(s[17 + i]));
                        }
                        const float mt = fmaxf(fmaf(ta, fa, va.y), fmaf(tb, fb, vb.y));
                        if (__any_sync(0xffffffffu, mt > m + kGrow)) {
                            // a new reference, a whole power of two away: l, this step's P so far and O follow
                            const float mn = mt > m + kGrow ? (m == -INFINITY ? mt : m + ceilf(mt - m)) : m;
                            const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                            m = mn;
                            l *= f;
                            st_wait();
#pragma unroll 1
                            for (int k = 0; k < c; ++k) {
                                uint32_t p[16];
                                ld16(s_at + 16 * k, p);
                                ld_wait(p);
#pragma unroll
                                for (int i = 0; i < 16; ++i) {
                                    const float2 v = Half2Of<__half>::f2(p[i]);  // f itself may be below fp16's range
                                    p[i] = Half2Of<__half>::pack(v.x * f, v.y * f);
                                }
                                st16(s_at + 16 * k, p);
                            }
                            if (j > 0) {
                                if (!pair) ok = __all_sync(0xffffffffu, wait(pv_done, j - 1));  // it still adds to O
                                if (!ok) break;
                                rescale(f);
                            }
                        }
                        const float ms = m == -INFINITY ? 0.0f : m;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t p[8];  // takes the place of S in TMEM, two values a column
                            const float f = h ? fb : fa, lv = h ? vb.y : va.y, add = lv - ms;
                            const uint64_t ff = two(f, f), aa = two(add, add);
                            uint64_t part = two(0.0f, 0.0f);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 x = untwo(fma2(two(__uint_as_float(s[16 * h + i]),
                                                                __uint_as_float(s[16 * h + i + 1])), ff, aa));
                                const float e0 = ex2(x.x), e1 = ex2(x.y);
                                part = add2(part, two(e0, e1));
                                p[i / 2] = Half2Of<__half>::pack(e0, e1);
                            }
                            const float2 t = untwo(part);
                            l = fmaf(t.x + t.y, ex2(-lv), l);
                            st8(s_at + 16 * c + 8 * h, p);
                        }
                    }
                    if (!ok) break;
                    st_wait();
                    fence_before();
                    mbar_arrive(p_full(slot, 0));
                }
                if (!ok) break;
            }
            // ---- out --------------------------------------------------------------
            if (ok && steps > 0) ok = __all_sync(0xffffffffu, wait(o_full(w), 0));
            if (ok) {
                fence_after();
                // O goes through this warp's part of the tile's Q (every MMA that reads it is done),
                // 32 columns at a time, so that rows are written in whole sectors
                const bool split = sp.count > 1;
                if (split) pdl_launch_dependents();
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const uint32_t buf = q_tile + (warp & 3) * 4096;
                // the rows of the output that this lane writes, in fp32 or rounded; -1: none
                int64_t to[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned rr = r0 + w * 128 + row0 + (split ? i * 4 + (lane >> 3) : (i & 3) * 8 + (lane >> 2));
                    const unsigned i_q = rr / group;
                    to[i] = rr < (unsigned)rows ? (int64_t)(span.lo + i_q) * a.q_heads + head * group + rr - i_q * group : -1;
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (steps > 0) {
                        ld32(o_at + 32 * c, o);
                        ld_wait(o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0;
                    }
                    if (!split) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = l == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[i]) * inv);
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 128 + ((u ^ (lane & 7)) << 4)),
                                     "r"(o[4 * u]), "r"(o[4 * u + 1]), "r"(o[4 * u + 2]), "r"(o[4 * u + 3])
                                     : "memory");
                    __syncwarp();
                    auto get = [&](int tr, int u) {
                        uint4 x;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                                     : "r"(buf + tr * 128 + ((u ^ (tr & 7)) << 4))
                                     : "memory");
                        return x;
                    };
                    if (split) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int tr = i * 4 + (lane >> 3), u = lane & 7;
                            const uint4 x = get(tr, u);
                            if (to[i] >= 0)
                                *reinterpret_cast<uint4 *>(sp.o + ((int64_t)share * a.tokens * a.q_heads + to[i]) * D +
                                                           32 * c + 4 * u) = x;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int tr = i * 8 + (lane >> 2), u = lane & 3;
                            const uint4 x = get(tr, 2 * u), y = get(tr, 2 * u + 1);
                            if (to[i] >= 0)
                                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + to[i] * D + 32 * c + 8 * u) =
                                    make_uint4(H::pack(__uint_as_float(x.x), __uint_as_float(x.y)),
                                               H::pack(__uint_as_float(x.z), __uint_as_float(x.w)),
                                               H::pack(__uint_as_float(y.x), __uint_as_float(y.y)),
                                               H::pack(__uint_as_float(y.z), __uint_as_float(y.w)));
                        }
                    }
                    __syncwarp();
                }
                const int64_t out_row = (int64_t)(span.lo + (real ? r / a.group : 0)) * a.q_heads + head * a.group +
                                        (real ? r % a.group : 0);
                if (real && split) sp.ml[(int64_t)share * a.tokens * a.q_heads + out_row] = make_float2(m, l);
                else if (real && a.lse)
                    a.lse[out_row] =
                        l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
            }
        }
    } else if (warp != kMmaWarp) {
        // ---- codes to fp16 tiles ---------------------------------------------------
        // An item is one panel (64 dims) of eight keys: four lanes take the 64 bytes of a
        // key, so that the 16-byte stores of a quarter warp (two keys) hit all banks once.
        // The warps take the items of a tile in turn.
        // Loads run one step ahead of the conversion and page ids one ahead of the loads, so
        // that no load's address waits for another load.  Lane b < KT / 16 keeps the place of
        // the step's block b; the others get it by shuffle.
        constexpr int kItems = P::kPanels * KT / 8;
        const int end = min(hi, k_lo + steps * KT);  // of this CTA's keys
        const int part = lane & 3, sub = lane >> 2;
        auto convert = [&](auto warps, int cw, const uint8_t *pool, uint32_t tile0, auto full, auto empty, bool is_k) {
            constexpr int kW = decltype(warps)::value, kEach = (kItems + kW - 1) / kW;
            const bool scaler = is_k && cw == 0;
            uint4 x[kEach];
            int page = 0;         // of the step after the next, as listed
            int64_t place = 0;    // of the next step: index of the block in the layer's pool
            float ksc = 1.0f, vsc = 1.0f;
            auto look_up = [&](int j) {
                const int t = k_lo + j * KT + lane * kBlock;
                page = lane < P::kBlocks && t < end ? a.L.listed(row, t) : 0;
            };
            auto load = [&](int j) {
                const int k0 = k_lo + j * KT;
                place = a.L.block_at((unsigned)page < (unsigned)a.L.pages ? page : 0, head, k0 + lane * kBlock);
                look_up(j + 1);
                const int c0 = opaque(cw);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int item = c0 + i * kW, eight = item % (KT / 8);
                    const int64_t b = __shfl_sync(0xffffffffu, place, eight >> 1);
                    // keys past the last that is seen: 0, never stale bytes
                    x[i] = ld_stream_v4_if(
                        pool + b * (kBlock * D) + ((eight & 1) * 8 + sub) * D + item / (KT / 8) * 64 + part * 16,
                        item < kItems && k0 + eight * 8 + sub < end);
                }
                ksc = vsc = 1.0f;
                if (scaler && lane < P::kBlocks && k0 + lane * kBlock < end) {
                    ksc = __ldg(a.L.ks + place);
                    vsc = __ldg(a.L.vs + place);
                }
            };
            look_up(0);
            load(0);
            for (int j = 0; j < steps; ++j) {
                bool ok = true;
                if (j >= kStages) ok = wait(empty(j), j / kStages - 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (scaler) {
                    const float v = fmaxf(vsc, 1e-37f);
                    if (lane < P::kBlocks)
                        scales[j % kScaleRing][lane] = make_float2(ksc, __log2f(v));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sc_full(j));
                }
                const uint32_t tile = tile0 + (j % kStages) * P::kKV;
                const int c0 = opaque(cw);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int item = c0 + i * kW, key = item % (KT / 8) * 8 + sub;
                    if (item >= kItems) break;
                    const uint32_t to = tile + item / (KT / 8) * P::kPanelKV + key * 128;
                    const uint32_t w[4] = {C::ready(x[i].x), C::ready(x[i].y), C::ready(x[i].z), C::ready(x[i].w)};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + (((2 * part + h) ^ sub) << 4)),
                                     "r"(C::template pair<0>(w[2 * h])), "r"(C::template pair<1>(w[2 * h])),
                                     "r"(C::template pair<0>(w[2 * h + 1])), "r"(C::template pair<1>(w[2 * h + 1]))
                                     : "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(full(j));
                load(j + 1);  // past the end: nothing is read
            }
        };
        if constexpr (STAGED) {
            // ---- copies of staged tiles -------------------------------------------------
            // a tile is one box of 128 or 256 rows of 128 bytes
            const int64_t first = ((int64_t)row * a.L.heads + head) * st.steps + (k_lo - all_steps.lo) / KT;
            auto copy = [&](uint32_t to, int64_t tile, uint32_t full) {
                if (lane == 0) {
                    mbar_arrive_expect_tx(full, P::kKV);
                    tma_load_2d(to, &map, 0, (int)(tile * (P::kPanels * KT)), full);
                }
            };
            int j = 0, v_issued = 0;
            for (; j < steps; ++j) {
                if (j >= kStages && !__all_sync(0xffffffffu, wait(k_empty(j), j / kStages - 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(sc_full(j), P::kBlocks * 8);
                    bulk_g2s(smem_addr(scales[j % kScaleRing]), st.scales + (first + j) * P::kBlocks, P::kBlocks * 8, sc_full(j));
                }
                copy(base + P::kOffK + (j % kStages) * P::kKV, 2 * (first + j), k_full(j));
                if (j >= kStages && !__all_sync(0xffffffffu, wait(v_empty(j), j / kStages - 1))) {
                    ++j;
                    break;
                }
                copy(base + P::kOffV + (j % kStages) * P::kKV, 2 * (first + j) + 1, v_full(j));
                v_issued = j + 1;
            }
            // nothing of this CTA's is in flight when it leaves
            for (int i = max(0, j - kStages); i < j; ++i) {
                mbar_wait_for(k_full(i), (i / kStages) & 1, kDrainWaitNs, &g_prefill_timeouts);
                if (i < v_issued) mbar_wait_for(v_full(i), (i / kStages) & 1, kDrainWaitNs, &g_prefill_timeouts);
                mbar_wait_for(sc_full(i), (i / kScaleRing) & 1, kDrainWaitNs, &g_prefill_timeouts);
            }
        } else if (steps > 0) {
            if (warp < kMmaWarp)
                convert(std::integral_constant<int, kWarpsK>(), warp - kSoftWarps, a.L.k, base + P::kOffK, k_full, k_empty, true);
            else
                convert(std::integral_constant<int, kWarpsV>(), warp - kMmaWarp - 1, a.L.v, base + P::kOffV, v_full, v_empty, false);
        }
    } else {
        // ---- MMA issue: the warp runs converged, one elected lane issues ---------------
        constexpr uint32_t i_qk = idesc_f16(128, KT, false), i_pv = idesc_f16(128, D, true), hi_word = desc128_hi(1024);
        const uint32_t q_lo = desc128_lo(base, 16), k_lo_word = desc128_lo(base + P::kOffK, 16);
        const uint32_t v_lo = desc128_lo(base + P::kOffV, P::kPanelKV);
        auto qk = [&](int j, int w, int slot) {
            const uint32_t q = q_lo + w * (P::kPanels * P::kPanelQ / 16), k = k_lo_word + (j % kStages) * (P::kKV / 16);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                mma_ss(tmem + (slot ? P::kS1 : 0), q + ((s / 4) * P::kPanelQ + (s % 4) * 32) / 16, hi_word,
                       k + ((s / 4) * P::kPanelKV + (s % 4) * 32) / 16, hi_word, i_qk, s > 0);
            commit(s_full(slot));
        };
        auto pv = [&](int j, int w, int slot, int half) {
            const uint32_t v = v_lo + (j % kStages) * (P::kKV / 16);
#pragma unroll
            for (int i = 0; i < KT / (16 * kParts); ++i) {
                const int s = half * (KT / (16 * kParts)) + i;
                mma_ts(tmem + (w ? P::kO1 : P::kO0), tmem + (slot ? P::kS1 : 0) + 8 * s, v + s * (16 * 128 / 16), hi_word,
                       i_pv, j > 0 || s > 0);
            }
            if (half + 1 < kParts) commit(pv_half(w));
        };
        // What ordinary stores wrote (Q, and the tiles of the direct form) is read by the MMAs: the
        // fence between the two stands here, after the wait, because the writers have loads in
        // flight that a fence of theirs would wait for.  Bulk copies need none.
        auto filled = [&] {
            fence_after();
            if (!STAGED) fence_proxy_async_smem();
        };
        auto all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        auto both = [&](int j, int w, int slot, int parity) {  // O += P V of a step, by parts
            for (int half = 0; half < kParts; ++half) {
                if (!all(p_full(slot, half), parity)) return false;
                fence_after();
                pv(j, w, slot, half);
            }
            return true;
        };
        bool ok = steps > 0 && all(q_full, 0) && all(k_full(0), 0);
        if (ok) {
            filled();
            fence_proxy_async_smem();
            qk(0, 0, 0);
            if (pair) qk(0, 1, 1);
            commit(k_empty(0));
        }
        for (int j = 0; j < steps && ok; ++j) {
            const bool next = j + 1 < steps;
            // the tiles of this step's second product and of the next step's first, and their
            // fence, before the wait for P that everything here follows
            if (pair) ok = all(v_full(j), j / kStages);
            if (ok && next) ok = all(k_full(j + 1), (j + 1) / kStages);
            if (!ok) break;
            filled();
            if (pair) {
                ok = both(j, 0, 0, j);
                if (!ok) break;
                if (next) qk(j + 1, 0, 0);
                else commit(o_full(0));
                ok = both(j, 1, 1, j);
                if (!ok) break;
                commit(v_empty(j));
                if (next) {
                    qk(j + 1, 1, 1);
                    commit(k_empty(j + 1));
                } else {
                    commit(o_full(1));
                }
            } else {
                if (next) {
                    qk(j + 1, 0, (j + 1) & 1);
                    commit(k_empty(j + 1));
                }
                ok = all(v_full(j), j / kStages);
                if (!ok) break;
                filled();
                ok = both(j, 0, j & 1, j >> 1);
                if (!ok) break;
                commit(v_empty(j));
                commit(pv_done);
                if (!next) commit(o_full(0));
            }
        }
        if (steps > 0) {
            // On every exit, since another role's wait may have run out although none of this one's
            // did: what was issued reads shared memory, writes TMEM and arrives on barriers of this
            // CTA.  Let it finish.
            commit(drained);
            mbar_wait_for(drained, 0, kDrainWaitNs, &g_prefill_timeouts);
        }
    }
    st_wait();  // a role that gave up may have stores to TMEM on their way
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, P::kCols);
}

// Joins the shares of every query and head of a row, in order
template <typename T, int D>
__global__ void __launch_bounds__(256)
join_kernel(const AttendArgs a, const Split sp)
{
    using H = Half2Of<T>;
    pdl_wait();
    const Span span(a.starts, blockIdx.y, a.tokens, a.max_new);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, at = i / (D / 4);
    const int d = (int)(i % (D / 4)) * 4;
    if (at >= (int64_t)span.n * a.q_heads) return;
    const int64_t row = (int64_t)span.lo * a.q_heads + at, all = (int64_t)a.tokens * a.q_heads;
    float m = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < sp.count; ++k) m = fmaxf(m, sp.ml[k * all + row].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.0f;
#pragma unroll 4
    for (int k = 0; k < sp.count; ++k) {
        const float2 ml = sp.ml[k * all + row];
        const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2(ml.x - m);  // (l is NaN where q is)
        const float4 x = *reinterpret_cast<const float4 *>(sp.o + (k * all + row) * D + d);
        o.x = fmaf(x.x, f, o.x), o.y = fmaf(x.y, f, o.y), o.z = fmaf(x.z, f, o.z), o.w = fmaf(x.w, f, o.w);
        l = fmaf(ml.y, f, l);
    }
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    T *to = static_cast<T *>(a.out) + row * D + d;
    *reinterpret_cast<uint2 *>(to) = make_uint2(H::pack(o.x * r, o.y * r), H::pack(o.z * r, o.w * r));
    if (a.lse && d == 0) a.lse[row] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
}

// Codes to fp16 tiles for the staged form: one CTA a tile (K or V of one step),
// as the MMAs will read it; the codes of a row are converted once for all of
// its query tiles.
template <int D, int FMT>
__global__ void __launch_bounds__(256)
stage_kernel(const AttendArgs a, const Staged st)
{
    using P = Plan<D>;
    using C = Code<FMT>;
    constexpr int KT = P::KT, kChunks = D / 16;  // 16-byte pieces of a token
    const int j = blockIdx.x >> 1, which = blockIdx.x & 1, head = blockIdx.y, row = blockIdx.z;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int L = a.L.length(row);
    const RowSteps all(L, span, a.window, KT);
    if (j >= all.steps || all.steps > st.steps) return;
    const int k0 = all.lo + j * KT;
    const int64_t step = ((int64_t)row * a.L.heads + head) * st.steps + j;
    uint8_t *tile = st.tiles + (2 * step + which) * P::kKV;
    const uint8_t *pool = which ? a.L.v : a.L.k;
    constexpr int kEach = KT * kChunks / 256;
    uint4 x[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x + i * 256, key = at / kChunks, t = k0 + key;
        x[i] = make_uint4(0, 0, 0, 0);  // keys past the row: 0, never stale bytes
        if (t < L)
            x[i] = __ldg(reinterpret_cast<const uint4 *>(pool + a.L.block_of(row, head, t) * (kBlock * D) + (t & 15) * D +
                                                         (at % kChunks) * 16));
    }
    if (which == 0 && threadIdx.x < P::kBlocks) {
        const int t = k0 + threadIdx.x * kBlock;
        float2 s = make_float2(1.0f, 0.0f);
        if (t < L) {
            const int64_t b = a.L.block_of(row, head, t);
            s = make_float2(__ldg(a.L.ks + b), __log2f(fmaxf(__ldg(a.L.vs + b), 1e-37f)));
        }
        st.scales[step * P::kBlocks + threadIdx.x] = s;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x + i * 256, key = at / kChunks, c = at % kChunks;
        uint8_t *to = tile + (c / 4) * P::kPanelKV + key * 128;
        const uint32_t w[4] = {C::ready(x[i].x), C::ready(x[i].y), C::ready(x[i].z), C::ready(x[i].w)};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4 *>(to + ((((c % 4) * 2 + h) ^ (key & 7)) << 4)) =
                make_uint4(C::template pair<0>(w[2 * h]), C::template pair<1>(w[2 * h]), C::template pair<0>(w[2 * h + 1]),
                           C::template pair<1>(w[2 * h + 1]));
    }
}

template <typename K>
bool configure(K kern, size_t smem, bool (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64 && done[dev]) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return true;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// Keys that a row of length `len` at most can need: a window and its queries hide the others
int64_t keys_of(const AttendArgs &a, int64_t len)
{
    return a.window > 0 ? std::min<int64_t>(len, (int64_t)a.window + a.max_new) : len;
}

// Steps of a row that the scratch is laid out for
template <int D>
int staged_steps(const AttendArgs &a)
{
    return (int)(keys_of(a, a.max_len) / Plan<D>::KT) + 2;  // a window's first step may start before its keys
}

// Steps that a row can need at most, whatever its length
template <int D>
int64_t most_steps(const AttendArgs &a)
{
    constexpr int KT = Plan<D>::KT;
    const int64_t capacity = (int64_t)a.L.row_pages << a.L.page_shift, all = (capacity + KT - 1) / KT;
    return std::min(all, keys_of(a, capacity) / KT + 2);
}

// CTAs that share a query tile's steps: the count with the least time, in steps
// of a full tile, over the waves of CTAs (one an SM).  A CTA costs about three
// steps to begin and end, and to leave and join its O three and a half more
// (2 x 128 KB at an SM's share of the bandwidth): 64 queries at 8192 keys, 48
// heads: 125 us with one, 45 us with nine.
template <int D>
int splits_of(const AttendArgs &a)
{
    using P = Plan<D>;
    const int64_t rows = (int64_t)a.max_new * a.group;
    const int64_t ctas = (rows + P::kRows - 1) / P::kRows * a.L.heads * a.L.rows;
    const double steps = (double)(keys_of(a, a.max_len) + P::KT - 1) / P::KT;
    const int sms = sm_count();
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 16 && (n == 1 || steps >= 4 * n); ++n) {
        const double cost = (double)((ctas * n + sms - 1) / sms) * (steps / n + (n == 1 ? 3.0 : 6.5));
        if (cost < least) least = cost, best = n;
    }
    return best;
}

// One query tile reads each code once: it converts them itself.  (Staging costs
// five bytes of traffic a code: 8 sequences of 8000 tokens, 11 queries: 137 us
// staged, 81 not; 2 x 256 queries of 8192 tokens, six tiles a head: 136 and 145.)
template <int D>
bool stages(const AttendArgs &a)
{
    return (int64_t)a.max_new * a.group > Plan<D>::kRows;
}

// The scratch: staged tiles and their scales, then the shares.  A plan for very long or very many rows
// goes without the tiles (the codes are converted in the kernel), and without shares only where those
// alone are too many.
template <int D>
struct Scratch {
    int steps = 0, splits = 1;  // staged steps of a row (0: none), CTAs that share a query tile's steps
    int64_t staged = 0, bytes = 0;
    explicit Scratch(const AttendArgs &a)
    {
        using P = Plan<D>;
        if (stages<D>(a)) {
            steps = staged_steps<D>(a);
            staged = (int64_t)a.L.rows * a.L.heads * steps * (2 * (int64_t)P::kKV + P::kBlocks * 8);
            if (staged > kMaxScratch) steps = 0, staged = 0;
        }
        bytes = staged;
        const int n = splits_of<D>(a);
        const int64_t q_tiles = ((int64_t)a.max_new * a.group + P::kRows - 1) / P::kRows;
        const int64_t shares = (int64_t)n * a.tokens * a.q_heads * (D * 4 + 8);
        if (n > 1 && q_tiles * n <= kMaxTiles && staged + shares <= kMaxScratch) splits = n, bytes += shares;
    }
};

template <typename T, int D, int FMT>
int launch_t(const AttendArgs &a, cudaStream_t s)
{
    using P = Plan<D>;
    auto direct = attend_prefill_kernel<T, D, FMT, false>;
    auto staged = attend_prefill_kernel<T, D, BQD_KV_INT8, true>;  // its tiles are fp16 in either format
    static bool done[2][64] = {};
    if (!configure(direct, P::kSmem, done[0]) || !configure(staged, P::kSmem, done[1])) return BQD_ERR_CUDA;
    const int64_t rows = (int64_t)a.max_new * a.group;
    const int64_t q_tiles = (rows + P::kRows - 1) / P::kRows;
    const Scratch<D> plan(a);
    Staged st = {nullptr, nullptr, a.work ? plan.steps : 0};
    Split sp = {nullptr, nullptr, a.work ? plan.splits : 1, 0};
    // (many rows of one launch: one call of the kernels in practice)
    auto each_launch = [&](auto launch) {
        for (int64_t at = 0; at < q_tiles; at += kMaxTiles) {
            sp.first = (int)(at * P::kRows);
            launch(dim3((unsigned)a.L.heads, (unsigned)a.L.rows, (unsigned)(std::min(q_tiles - at, kMaxTiles) * sp.count)));
        }
    };
    CUtensorMap map = {};
    uint8_t *end = static_cast<uint8_t *>(a.work) + plan.staged;
    sp.o = reinterpret_cast<float *>(end);
    sp.ml = reinterpret_cast<float2 *>(sp.o + (int64_t)sp.count * a.tokens * a.q_heads * D);
    if (st.steps > 0) {
        const int64_t tiles = (int64_t)a.L.rows * a.L.heads * st.steps;
        st.tiles = static_cast<uint8_t *>(a.work);
        st.scales = reinterpret_cast<float2 *>(st.tiles + tiles * 2 * P::kKV);
        // the scratch as rows of 64 fp16, already in the swizzled order of the operands
        auto enc = encode_fn();
        const cuuint64_t dims[2] = {64, (cuuint64_t)(tiles * 2 * P::kPanels * P::KT)}, strides[1] = {128};
        const cuuint32_t box[2] = {64, (cuuint32_t)(P::kPanels * P::KT)}, each[2] = {1, 1};
        if (!enc || enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, st.tiles, dims, strides, box, each,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return BQD_ERR_CUDA;
        stage_kernel<D, FMT><<<dim3(2 * st.steps, a.L.heads, a.L.rows), 256, 0, s>>>(a, st);
        each_launch([&](dim3 grid) { staged<<<grid, kThreadsStaged, P::kSmem, s>>>(a, st, sp, map, opt_wait_ns()); });
    }
    if (most_steps<D>(a) > st.steps)  // rows that need more steps than planned, or all of them
        each_launch([&](dim3 grid) { direct<<<grid, kThreadsF, P::kSmem, s>>>(a, st, sp, map, opt_wait_ns()); });
    if (sp.count == 1) return cuda_status(cudaGetLastError());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((int64_t)a.max_new * a.q_heads * (D / 4) + 255) / 256), (unsigned)a.L.rows);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t launched = cudaGetLastError();
    return cuda_status(launched != cudaSuccess ? launched : cudaLaunchKernelEx(&cfg, join_kernel<T, D>, a, sp));
}

template <typename T, int FMT>
int launch_d(const AttendArgs &a, cudaStream_t s)
{
    if (a.head_dim == 64) return launch_t<T, 64, FMT>(a, s);
    if (a.head_dim == 128) return launch_t<T, 128, FMT>(a, s);
    return launch_t<T, 256, FMT>(a, s);
}

}  // namespace

int64_t prefill_workspace(const AttendArgs &a)
{
    auto bytes = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return Scratch<D>(a).bytes;
    };
    return a.head_dim == 64    ? bytes(std::integral_constant<int, 64>())
           : a.head_dim == 128 ? bytes(std::integral_constant<int, 128>())
                               : bytes(std::integral_constant<int, 256>());
}

int launch_attend_prefill(const AttendArgs &a, cudaStream_t s)
{
    if (a.format == BQD_KV_INT8)
        return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_INT8>(a, s)
                                        : launch_d<__nv_bfloat16, BQD_KV_INT8>(a, s);
    return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_E4M3>(a, s)
                                    : launch_d<__nv_bfloat16, BQD_KV_E4M3>(a, s);
}

int take_prefill_timeouts(unsigned int *count)
{
    if (cudaMemcpyFromSymbol(count, g_prefill_timeouts, sizeof(*count)) != cudaSuccess) return BQD_ERR_CUDA;
    if (*count) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_prefill_timeouts, &zero, sizeof(zero)) != cudaSuccess) return BQD_ERR_CUDA;
    }
    return BQD_OK;
}

}  // namespace kv
}  // namespace bqd
