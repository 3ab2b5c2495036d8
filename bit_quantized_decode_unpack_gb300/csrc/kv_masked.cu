// Attention over a paged 8-bit cache under masks, for tens to hundreds of (query,
// head) rows that face the same keys: trees of drafted tokens.
//
// The mathematics is that of the few-query kernel (kv_attend.cu): with f the score
// scale times log2(e) and s^k_b, s^v_b the scales of 16-token block b,
//   x_ij = f s^k_b (q_i . c^k_j) + log2 s^v_b,   p_ij = 2^(x_ij - m_i),
//   O_i = sum_j p_ij c^v_j,   l_i = sum_b (sum_{j in b} p_ij) / s^v_b,
//   out = O / l,   lse = ln 2 (m + log2 l),
// with m_i replaced only when x passes it by 15 (p < 2^15 fits fp16).
//
// Both products run on the 5th-generation tensor cores, S = Q K^T with Q and K in
// shared memory, O += P V with P in TMEM where S was.  A CTA has up to two S and O
// (head_dim 256: two S, one O), each with four warps of softmax, one thread a row, and
// is used in one of three ways:
//   pair     256 rows: two tiles of 128, each sees every step of keys.  The tensor
//            cores work on one while the other's softmax runs
//   streams  128 rows: both have the same rows, one takes the even steps, the other the
//            odd ones; their sums are joined at the end through shared memory
//   single   head_dim 256, 128 rows: S alternates, so that the next one is computed
//            during this one's softmax
// The keys' codes reach shared memory by bulk copies that run ahead, and six warps turn
// them into fp16 tiles (128-byte swizzle): unlike a prompt's, a tree's few tiles of
// queries do not pay for tiles converted once in scratch (8 x 64 nodes at up to 16000
// tokens: 286 us that way).
//   warps 0-3, 4-7     softmax of S and O 0 / 1
//   warps 8-10, 11-13  K's, V's codes to fp16
//   warp 14            TMEM, and one elected lane that issues every MMA
//   warp 15            bulk copies of the codes, and the scales
//
// Work.  A unit is (row, KV head, tile of rows); a unit's key steps are cut into equal
// shares.  No host knows the rows' lengths: a first kernel, of one CTA, adds up the rows'
// steps, finds the share length with the least estimated time, and leaves each row's
// place among the CTAs, where every CTA looks its own work up.  Shares leave O, m and l in
// scratch, and a last kernel joins them in order; both followers are launched early.
// No atomics: the same bits every time.  Up to 16 rows every CTA makes the plan for
// itself, which saves that launch (8 ragged trees of up to 64 nodes 124 us, 131 with it;
// 24 rows, 4 of them live at 4000 tokens, 41 and 37).  With more it would take time by the
// square of the rows: 1024 of 8 KV heads, 8 of them live at 500 tokens, 4423 us and 127.
// Bound by neither HBM nor the tensor cores, but by the waits between the roles of a step:
// the tensor pipe is active 31% of the time, HBM read at 2.8 to 3.0 TB/s (4 x 65001
// tokens, 8 KV heads of 128, 30 to 126 rows: 187 to 189 us; 252 rows: 288 us).  Which
// wait decides is not isolated: a conversion takes 1600 to 1900 cycles of a step's 2200 to
// 3900, yet leaving out its loads or its stores (in a copy) left the period.  The same
// with the keys as the 128-row operand took 210 us with e4m3 codes (179 here) and 520 for
// 252 rows; codes loaded straight to registers, two steps ahead, 352.  Softmax warps
// without a query that skip their steps cost 1 to 2.5% (252 rows 293 us, 126 rows of 256
// at 4 KV heads 234 -> 240) and gain 1.3% only with heads of 64.
// Every wait is bounded; on expiry a role stops, what it issued is drained, TMEM is
// freed, and bqd_device_status reports it.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kv_common.cuh"
#include "qmv_common.cuh"
#include "tc05.cuh"

namespace bqd {
namespace kv {
namespace {

using namespace qmvdev;
using namespace tc05;

constexpr int kSoftWarps = 8, kWarpsKV = 3;
constexpr int kMmaWarp = kSoftWarps + 2 * kWarpsKV, kCopyWarp = kMmaWarp + 1;
constexpr int kThreadsM = (kCopyWarp + 1) * 32;
constexpr int kStages = 2;          // fp16 tiles of K and of V
constexpr int kMaxRows = kPlannedRows;
constexpr int kOwnRows = 16;        // rows up to which every CTA makes the plan
constexpr int kMaxShares = 64;      // shares of a unit
constexpr float kGrow = 15.0f;

__device__ unsigned int g_masked_timeouts = 0;

template <int D>
struct Plan {
    static constexpr int kTiles = D == 256 ? 1 : 2;      // O's, and tiles of a pair
    static constexpr int KT = D == 256 ? 64 : 128;       // keys of a step
    static constexpr int kBlocks = KT / kBlock;
    static constexpr int kPanels = D / 64;
    static constexpr int kParts = D == 256 ? 1 : 2;      // of a step's softmax: P V of the first runs during the second
    static constexpr uint32_t kPanelQ = 128 * 128, kTileQ = kPanels * kPanelQ, kQ = kTiles * kTileQ;
    static constexpr uint32_t kPanelKV = KT * 128, kKV = kPanels * kPanelKV;
    static constexpr uint32_t kUnit = KT * D;            // codes of a step's K or V
    // codes that are on their way: units of K and of V each.  With head_dim 128 the second one
    // lies in the second tile's place of Q, which only a pair needs
    static constexpr int kRing = D == 64 ? 4 : 1, kMaxRing = D == 64 ? 4 : D == 128 ? 2 : 1;
    static constexpr int kScaleRing = D == 64 ? 16 : 8;  // steps whose scales are kept: the copies run ahead of the
                                                         // softmax by the ring, two tiles and two S at most
    static constexpr uint32_t kOffK = kQ, kOffV = kOffK + kStages * kKV, kOffRaw = kOffV + kStages * kKV;
    static constexpr size_t kSmem = 1024 + kOffRaw + 2 * kRing * kUnit;
    static constexpr uint32_t kS1 = KT, kO0 = 256, kO1 = 256 + D, kCols = 512;  // TMEM columns
    static constexpr int kPiece = 128 * D + 256;         // floats of a share of a tile: O [128][D], m, l
};

// Shares of a tile of 128 rows: pieces first, first + step, ...; first < 0: the tile is done
struct Record {
    int first, count, step;
};

// CTAs and pieces of the rows before one; behind the last row: all CTAs, and the steps of a pair's share
struct Place {
    int cta, piece;
};

struct Scratch {
    float *pieces;
    Record *records;   // [rows * heads * tiles of max_new]
    Place *places;     // [rows + 1]
    int most;          // pieces; 0: nothing is shared, and there is no plan
    int tiles;         // 128-row tiles of max_new
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

// whether any of the threads that meet at this barrier says so
__device__ __forceinline__ bool any_of(int id, int threads, bool mine)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\tbarrier.cta.red.or.pred.aligned q, %1, %2, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((int)mine)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void meet(int id, int threads)
{
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Bits [0, n) of a word, n of any value
__device__ __forceinline__ uint32_t bits_below(int n)
{
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1;
}

// Which keys a query sees: those in (after, first) and, from `first` on (the first of its row's last
// tokens), those whose bit is set, below `end`.
struct Seen {
    const uint32_t *mask;  // 32-bit words of the query's mask
    int words;             // 0: a row of the tile that is no query
    int after, first, end;
    // of keys k .. k + 31
    __device__ __forceinline__ uint32_t at(int k) const
    {
        if (words == 0) return 0u;
        const int o = k - first;
        uint32_t v = 0;
        if (o > -32) {
            const int w = o >> 5;  // -1: the first word starts inside
            const uint32_t lo = (unsigned)w < (unsigned)words ? __ldg(mask + w) : 0u;
            const uint32_t hi = w + 1 < words ? __ldg(mask + w + 1) : 0u;
            v = __funnelshift_r(lo, hi, o & 31) & bits_below(end - k) & ~bits_below(-o);
        }
        return v | (bits_below(-o) & ~bits_below(after + 1 - k));
    }
};

// Keys of a row that any of its queries sees start at lo
template <int D>
__device__ __forceinline__ int first_key(const AttendArgs &a, int L, const Span &span)
{
    return a.window > 0 ? max(0, L - span.rest + 1 - a.window) / Plan<D>::KT * Plan<D>::KT : 0;
}

// What the CTA does
struct Job {
    int row, head, tile, share, count;
    int piece, step;  // of share 0 of its first tile, or -1; from a share's to the next one's
    bool pair;
};

// A row's tiles in pairs and alone, and the shares of each, of which `each` steps are a pair's and twice as
// many a single tile's
template <int D>
struct Cuts {
    int steps, pairs, ones, n2, n1;
    __device__ __forceinline__ Cuts(int steps_, int tiles, int each) : steps(steps_)
    {
        if constexpr (Plan<D>::kTiles == 2) {
            pairs = tiles / 2, ones = tiles & 1;
            n2 = (steps + each - 1) / each, n1 = (steps + 2 * each - 1) / (2 * each);
        } else {
            pairs = 0, ones = tiles;
            n2 = n1 = (steps + each - 1) / each;
        }
    }
    __device__ __forceinline__ int64_t ctas(int heads) const { return heads * ((int64_t)pairs * n2 + (int64_t)ones * n1); }
    __device__ __forceinline__ int64_t pieces(int heads) const
    {
        return heads * ((n2 > 1 ? 2ll * pairs * n2 : 0) + (n1 > 1 ? (int64_t)ones * n1 : 0));
    }
};

// Steps of a row's keys, and its tiles of queries
template <int D>
__device__ __forceinline__ int steps_of(const AttendArgs &a, int L, const Span &span)
{
    return max(1, (L - first_key<D>(a, L, span) + Plan<D>::KT - 1) / Plan<D>::KT);
}

__device__ __forceinline__ int tiles_of(const AttendArgs &a, const Span &span) { return (span.n * a.group + 127) / 128; }

// The share length, and the rows' places.  In units of a step of 128 rows a pair's step costs 2 and a share
// kFixed; S CTAs on `sms` SMs take the sum over sms and, beyond one wave, about half a share more for the
// tail.  The warps share the rows out, each lane with a candidate; sums are of whole numbers, so their order
// is of no consequence.
constexpr int kFixed = 8;

struct Planning {
    static constexpr int kWarps = kThreadsM / 32;
    int64_t of_warp[3][kWarps][32];  // work, CTAs and pieces of each candidate
    int steps[kMaxRows], tiles[kMaxRows], sums[2][kWarps], chosen;
};

template <int D>
__device__ void plan_rows(const AttendArgs &a, const Scratch &sc, int sms, Planning &in, Place *places)
{
    using P = Plan<D>;
    constexpr int kWarps = Planning::kWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = a.L.rows, heads = a.L.heads;
#pragma unroll 1
    for (int r = tid; r < rows; r += kThreadsM) {
        const Span span(a.starts, r, a.tokens, a.max_new);
        in.steps[r] = steps_of<D>(a, a.L.length(r), span);
        in.tiles[r] = tiles_of(a, span);
    }
    __syncthreads();
    int longest = 1;
#pragma unroll 1
    for (int r = lane; r < rows; r += 32)
        if (in.tiles[r]) longest = max(longest, in.steps[r]);
    longest = __reduce_max_sync(0xffffffffu, longest);
    // lane i tries shares of longest 2^(-i / 4) steps; lane 0 splits nothing
    int each = max(1, (int)ceilf(longest * exp2f(-0.25f * lane)));
    each = max(max(each, 2), (longest + kMaxShares - 1) / kMaxShares);
    if (lane == 0) each = longest;
    int64_t work = 0, ctas = 0, pieces = 0;
#pragma unroll 1
    for (int r = warp; r < rows; r += kWarps) {
        if (!in.tiles[r]) continue;
        const Cuts<D> c(in.steps[r], in.tiles[r], each);
        work += heads * ((int64_t)c.pairs * (2 * c.steps + c.n2 * kFixed) + (int64_t)c.ones * (c.steps + c.n1 * kFixed));
        ctas += c.ctas(heads), pieces += c.pieces(heads);
    }
    in.of_warp[0][warp][lane] = work, in.of_warp[1][warp][lane] = ctas, in.of_warp[2][warp][lane] = pieces;
    __syncthreads();
    if (warp == 0) {
#pragma unroll 1
        for (int w = 1; w < min(rows, kWarps); ++w)
            work += in.of_warp[0][w][lane], ctas += in.of_warp[1][w][lane], pieces += in.of_warp[2][w][lane];
        const float share = (P::kTiles == 2 ? 2 * each : each) + kFixed;
        float cost = (float)work / sms;
        if (ctas > sms) cost += 0.5f * share;
        cost = fmaxf(cost, share);
        if (pieces > sc.most) cost = 3.0e38f;
        // the least cost, of equals the longest shares
        int best = lane;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float c = __shfl_xor_sync(0xffffffffu, cost, o);
            const int b = __shfl_xor_sync(0xffffffffu, best, o);
            if (c < cost || (c == cost && b < best)) cost = c, best = b;
        }
        if (lane == best) in.chosen = each;
    }
    __syncthreads();
    each = in.chosen;
    // CTAs and pieces of the rows before each: a thread takes consecutive rows
    const int per = (rows + kThreadsM - 1) / kThreadsM, first = min(tid * per, rows), last = min(first + per, rows);
    int x = 0, y = 0;
#pragma unroll 1
    for (int r = first; r < last; ++r) {
        const Cuts<D> c(in.steps[r], in.tiles[r], each);
        x += (int)c.ctas(heads), y += (int)c.pieces(heads);
    }
    const int mine = x, cut = y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += p, y += q;
    }
    if (lane == 31) in.sums[0][warp] = x, in.sums[1][warp] = y;
    __syncthreads();
    Place at = {x - mine, y - cut};
    const int busy = min(warp, (rows + 32 * per - 1) / (32 * per));  // (warps before this one that have rows)
#pragma unroll 1
    for (int w = 0; w < busy; ++w) at.cta += in.sums[0][w], at.piece += in.sums[1][w];
#pragma unroll 1
    for (int r = first; r < last; ++r) {
        places[r] = at;
        const Cuts<D> c(in.steps[r], in.tiles[r], each);
        at.cta += (int)c.ctas(heads), at.piece += (int)c.pieces(heads);
    }
    if (tid == kThreadsM - 1) places[rows] = Place{at.cta, each};  // (its sums are those of all rows)
}

template <int D>
__global__ void __launch_bounds__(kThreadsM)
masked_plan_kernel(const AttendArgs a, const Scratch sc, int sms)
{
    __shared__ Planning in;
    pdl_launch_dependents();
    plan_rows<D>(a, sc, sms, in, sc.places);
}

// What the CTA does; its row is -1 where it has nothing to do
template <int D>
__device__ Job find_job(const AttendArgs &a, const Scratch &sc, int sms, Planning &in, Place *near, int *found)
{
    using P = Plan<D>;
    const int rows = a.L.rows, heads = a.L.heads, b = blockIdx.x;
    const bool pairs = P::kTiles == 2;
    if (sc.most == 0) {
        const int per = pairs ? (sc.tiles + 1) / 2 : sc.tiles, i = b % per;
        Job j = {b / per / heads, b / per % heads, pairs ? 2 * i : i, 0, 1, -1, 0, false};
        if (j.row >= rows) return Job{-1};
        const int tiles = tiles_of(a, Span(a.starts, j.row, a.tokens, a.max_new));
        j.pair = pairs && j.tile + 1 < tiles;
        if (j.tile >= tiles) j.row = -1;
        return j;
    }
    const Place *places = sc.places;
    if (rows <= kOwnRows) {
        plan_rows<D>(a, sc, sms, in, near);
        __syncthreads();
        places = near;
    } else {
        pdl_wait();
    }
    const Place all = places[rows];
    if (b >= all.cta) return Job{-1};
#pragma unroll 1
    for (int r = threadIdx.x; r < rows; r += kThreadsM) {
        const Place p = places[r];
        if (b >= p.cta && b < places[r + 1].cta) found[0] = r, found[1] = b - p.cta, found[2] = p.piece;
    }
    __syncthreads();  // (one thread of the CTA found it)
    Job j = {found[0], 0, 0, 0, 1, -1, 0, false};
    // a row's pairs first, then its single tiles; tiles fastest, then heads, then shares: CTAs that read the
    // same keys run together
    int i = found[1], first = found[2];
    const Span span(a.starts, j.row, a.tokens, a.max_new);
    const Cuts<D> c(steps_of<D>(a, a.L.length(j.row), span), tiles_of(a, span), all.piece);
    j.pair = i < c.pairs * heads * c.n2;
    if (!j.pair) {
        i -= c.pairs * heads * c.n2;
        if (c.n2 > 1) first += 2 * c.pairs * heads * c.n2;
    }
    const int t = j.pair ? c.pairs : c.ones, k = i % t;
    j.count = j.pair ? c.n2 : c.n1;
    j.head = i / t % heads;
    j.share = i / (t * heads);
    j.tile = j.pair ? 2 * k : 2 * c.pairs + k;
    j.step = j.pair ? 2 : 1;
    if (j.count > 1) j.piece = first + (j.head * t + k) * j.count * j.step;
    return j;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreadsM, 1)
attend_masked_kernel(const AttendArgs a, const Scratch sc, int sms, unsigned long long wait_ns)
{
    using P = Plan<D>;
    using C = Code<FMT>;
    constexpr int KT = P::KT, kScaleRing = P::kScaleRing;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[56];
    __shared__ __align__(16) float2 scales[kScaleRing][P::kBlocks];  // of a step's blocks: K's scale, log2 of V's
    __shared__ float cs_of[128];
    __shared__ Place near[kOwnRows + 1];
    __shared__ int found[3];
    __shared__ uint32_t tmem_at;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // a plan's working place is filled with other things later
    static_assert(sizeof(Planning) + 1024 <= P::kSmem, "");
    const Job job = find_job<D>(a, sc, sms, *reinterpret_cast<Planning *>(raw + (base - smem_addr(raw))), near, found);
    if (job.row < 0) return;
    const int row = job.row, head = job.head;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int rows = span.n * a.group, r0 = job.tile * 128;
    const bool pair = job.pair, streams = P::kTiles == 2 && !pair;
    const int L = a.L.length(row), before = L - span.rest;
    const int k_first = first_key<D>(a, L, span), all = max(0, (L - k_first + KT - 1) / KT);
    const int from = (int)((int64_t)all * job.share / job.count);
    const int steps = (int)((int64_t)all * (job.share + 1) / job.count) - from;
    const int k_lo = k_first + from * KT;
    if (sc.records && job.share == 0 && tid < (pair ? 2 : 1))
        sc.records[(row * a.L.heads + head) * sc.tiles + job.tile + tid] =
            Record{job.piece < 0 ? -1 : job.piece + tid, job.count, job.step};

    // units of codes on their way, and their places
    const int ring = D == 128 && pair ? 1 : P::kMaxRing;
    auto raw_at = [&](int which, int u) {
        const int slot = u % ring;
        return base + (slot < P::kRing ? P::kOffRaw + (which * P::kRing + slot) * P::kUnit : P::kTileQ + which * P::kUnit);
    };

    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    auto k_full = [&](int j) { return bar(j % kStages); };
    auto k_empty = [&](int j) { return bar(2 + j % kStages); };
    auto v_full = [&](int j) { return bar(4 + j % kStages); };
    auto v_empty = [&](int j) { return bar(6 + j % kStages); };
    auto s_full = [&](int w) { return bar(8 + w); };
    auto p_full = [&](int w, int half) { return bar(10 + 2 * w + half); };
    auto pv_half = [&](int w) { return bar(14 + w); };
    auto o_full = [&](int w) { return bar(16 + w); };
    const uint32_t q_full = bar(18), pv_done = bar(19), drained = bar(20);
    auto raw_full = [&](int which, int u) { return bar(21 + 4 * which + u % ring); };
    auto raw_empty = [&](int which, int u) { return bar(29 + 4 * which + u % ring); };
    auto sc_full = [&](int j) { return bar(37 + j % kScaleRing); };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(i), kWarpsKV);
                mbar_init(bar(2 + i), 1);
                mbar_init(bar(4 + i), kWarpsKV);
                mbar_init(bar(6 + i), 1);
                mbar_init(s_full(i), 1);
                mbar_init(p_full(i, 0), 128);
                mbar_init(p_full(i, 1), 128);
                mbar_init(pv_half(i), 1);
                mbar_init(o_full(i), 1);
            }
            mbar_init(q_full, pair ? 256 : 128);
            mbar_init(pv_done, 1);
            mbar_init(drained, 1);
            for (int i = 0; i < 8; ++i) mbar_init(bar(21 + i), 1), mbar_init(bar(29 + i), kWarpsKV);
            for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full(i), 1);
        }
        __syncwarp();
        tmem_alloc(smem_addr(&tmem_at), P::kCols);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_for(b, parity & 1, wait_ns, &g_masked_timeouts); };

    if (warp < kSoftWarps) {
        const int w = warp >> 2;                             // S and O
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // TMEM lane 32 (warp % 4), in bits 16..31
        const int tile_row = r0 + (pair ? w * 128 : 0);      // first row of the tile
        const int row0 = (warp & 3) * 32, trow = row0 + lane, r = tile_row + trow;
        const bool real = r < rows;
        const unsigned group = a.group;
        const uint32_t q_tile = base + (pair ? w * P::kTileQ : 0u);
        if (pair || w == 0 || streams) {
            Seen seen;
            {
                const int token = span.lo + (real ? r / a.group : 0);
                seen.mask = reinterpret_cast<const uint32_t *>(a.mask + (int64_t)token * a.words);
                seen.words = real ? 2 * a.words : 0;
                seen.first = before, seen.end = L, seen.after = -1;
                if (a.window > 0 && real) seen.after = before + max(0, min(__ldg(a.depth + token), span.rest - 1)) - a.window;
            }
            // ---- q: scaled by 2^-e into fp16 (e of the row's largest magnitude) ----------------
            // fp16 keeps every bit of a bf16 value down to 2^-16 of that magnitude, and an absolute
            // 2^-25 of it below, of the order of what the fp32 sum of the scores rounds off
            constexpr int kRowLanes = D / 8, kRowsPass = 32 / kRowLanes, kPasses = kRowLanes;
            constexpr int kFlight = kPasses < 8 ? kPasses : 8;
            const bool bf = a.dtype == BQD_DTYPE_BF16;
            const uint32_t inf = bf ? Half2Of<__nv_bfloat16>::kInf : Half2Of<__half>::kInf;
            float cs = 1.0f;  // of this thread's row: |f| 2^e
            if (pair || w == 0) {
#pragma unroll 1
                for (int i0 = 0; i0 < kPasses; i0 += kFlight) {
                    uint4 v[kFlight];
#pragma unroll
                    for (int i = 0; i < kFlight; ++i) {
                        const unsigned rr = tile_row + row0 + (i0 + i) * kRowsPass + lane / kRowLanes;
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (rr < (unsigned)rows) {
                            const unsigned i_q = rr / group;
                            const unsigned short *q = static_cast<const unsigned short *>(a.q) + (int64_t)(span.lo + i_q) * a.q_token +
                                                      (int64_t)(head * group + rr - i_q * group) * a.q_head + lane % kRowLanes * 8;
                            if (a.q_vec) {
                                v[i] = __ldg(reinterpret_cast<const uint4 *>(q));
                            } else {
                                uint32_t x[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) x[k] = (uint32_t)__ldg(q + 2 * k) | ((uint32_t)__ldg(q + 2 * k + 1) << 16);
                                v[i] = make_uint4(x[0], x[1], x[2], x[3]);
                            }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kFlight; ++i) {
                        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                        const uint32_t mx = __vmaxu2(__vmaxu2(x[0] & 0x7FFF7FFFu, x[1] & 0x7FFF7FFFu),
                                                     __vmaxu2(x[2] & 0x7FFF7FFFu, x[3] & 0x7FFF7FFFu));
                        uint32_t top = max(mx & 0xFFFFu, mx >> 16);
#pragma unroll
                        for (int o = 1; o < kRowLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        int e = 0;
                        if (top != 0 && top < inf) {
                            const float f = bf ? Half2Of<__nv_bfloat16>::f1(top) : Half2Of<__half>::f1(top);
                            e = max(-100, min(126, (int)((__float_as_uint(f) >> 23) & 0xFF) - 127));
                        }
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
                            const float2 f = bf ? Half2Of<__nv_bfloat16>::f2(x[k]) : Half2Of<__half>::f2(x[k]);
                            h4[k] = Half2Of<__half>::pack(f.x * down, f.y * down);
                        }
                        const int tr = row0 + (i0 + i) * kRowsPass + lane / kRowLanes, u = lane % kRowLanes;
                        const uint32_t at = q_tile + (u >> 3) * P::kPanelQ + tr * 128 + (((u & 7) ^ (tr & 7)) << 4);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h4[0]), "r"(h4[1]), "r"(h4[2]), "r"(h4[3])
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(q_full);
            }
            if (streams) {
                if (w == 0) cs_of[trow] = cs;
                meet(1, kSoftWarps * 32);
                cs = cs_of[trow];
            }

            // ---- steps -----------------------------------------------------------------------
            const uint32_t o_at = tmem + lanes + (w ? P::kO1 : P::kO0);
            auto factor = [&](float k) { return fmaxf(cs * k, 1.2e-38f); };  // above 0, so that -inf (masked) stays -inf
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            int n = 0;  // steps of this S (single: of both)
            for (int j = streams ? w : 0; j < steps; j += streams ? 2 : 1, ++n) {
                const int slot = P::kTiles == 1 ? j & 1 : w, phase = P::kTiles == 1 ? j >> 1 : n;
                const uint32_t s_at = tmem + lanes + (slot ? P::kS1 : 0);
                ok = wait(sc_full(j), j / kScaleRing) && wait(s_full(slot), phase);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                fence_after();
                const int k0 = k_lo + j * KT;
                const bool whole = k0 + KT <= before && (a.window == 0 || k0 > L - 1 - a.window);
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
                // A part of the step's columns at a time.  Exponentials are taken against the reference
                // that is there, with the part's maximum found beside them; where a row passes its reference
                // by too much (the first step, seldom after it) the warp replaces it and computes the part
                // again.  P takes the place of scores that were read, two values a column.
                constexpr int kPart = KT / P::kParts, kPartBlocks = kPart / 16, kChunks = kPart / 32;
                // (a small loop: its code and that of the other roles share the instruction cache)
#pragma unroll 1
                for (int part = 0; part < P::kParts; ++part) {
                    uint32_t s[kChunks][32];
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) ld32(s_at + part * kPart + 32 * c, s[c]);
                    float2 v[kPartBlocks];  // the blocks' scales, while S is on its way
#pragma unroll
                    for (int b = 0; b < kPartBlocks; ++b) {
                        v[b] = scales[j % kScaleRing][part * kPartBlocks + b];
                        v[b].x = factor(v[b].x);
                    }
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) ld_wait(s[c]);
                    if (!whole) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            const uint32_t bits = seen.at(k0 + part * kPart + 32 * c);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!(bits >> i & 1)) s[c][i] = 0xFF800000u;  // -inf
                        }
                    }
                    float sum;
                    while (true) {
                        const float ms = m == -INFINITY ? 0.0f : m;
                        float mt = -INFINITY;
                        sum = 0.0f;
#pragma unroll
                        for (int b = 0; b < kPartBlocks; ++b) {
                            const uint32_t *x = &s[b / 2][16 * (b & 1)];
                            const float add = v[b].y - ms;
                            const uint64_t ff = two(v[b].x, v[b].x), aa = two(add, add);
                            uint64_t acc = two(0.0f, 0.0f);
                            float top = -INFINITY;
                            uint32_t p[8];
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float x0 = __uint_as_float(x[i]), x1 = __uint_as_float(x[i + 1]);
                                const float2 y = untwo(fma2(two(x0, x1), ff, aa));
                                const float e0 = ex2(y.x), e1 = ex2(y.y);
                                top = fmaxf(fmaxf(top, x0), x1);
                                acc = add2(acc, two(e0, e1));
                                p[i / 2] = Half2Of<__half>::pack(e0, e1);
                            }
                            mt = fmaxf(mt, fmaf(top, v[b].x, v[b].y));
                            const float2 t = untwo(acc);
                            sum = fmaf(t.x + t.y, ex2(-v[b].y), sum);
                            st8(s_at + part * (kPart / 2) + 8 * b, p);
                        }
                        if (!__any_sync(0xffffffffu, mt > m + kGrow)) break;
                        const float mn = mt > m + kGrow ? mt : m;
                        const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                        m = mn;
                        l *= f;
                        if (n > 0 || part) {
                            // what still adds to O: the first part's product, or with a single tile that of
                            // the step before (else it is done before S comes)
                            if (P::kTiles == 1 && j > 0) ok = wait(pv_done, j - 1);
                            if (ok && part) ok = wait(pv_half(slot), phase);
                            ok = __all_sync(0xffffffffu, ok);
                            if (!ok) break;
                            rescale(f);
                        }
                    }
                    if (!ok) break;
                    l += sum;
                    st_wait();
                    fence_before();
                    mbar_arrive(p_full(slot, part));
                }
                if (!ok) break;
            }
            // ---- out -------------------------------------------------------------------------
            // (n: whether O was ever written; a share of one step leaves the second stream without)
            if (ok && n > 0) ok = __all_sync(0xffffffffu, wait(o_full(w), 0));
            float f_own = 1.0f;
            float *const smem = reinterpret_cast<float *>(raw + (base - smem_addr(raw)));
            if (streams) {
                // both streams' m and l meet; each hands the half of O that the other finishes over, times
                // its factor, through the place of the K tiles (every MMA that reads them is done)
                float2 *ml = reinterpret_cast<float2 *>(smem + P::kOffV / 4);
                float4 *part = reinterpret_cast<float4 *>(smem + P::kOffK / 4);  // [stream][D / 8 quads][128 rows]
                if (any_of(1, kSoftWarps * 32, !ok)) ok = false;
                if (ok) {
                    fence_after();
                    ml[w * 128 + trow] = make_float2(m, l);
                    meet(1, kSoftWarps * 32);
                    const float2 other = ml[(w ^ 1) * 128 + trow];
                    const float mm = fmaxf(m, other.x);
                    f_own = m == -INFINITY ? 0.0f : ex2(m - mm);
                    const float f_other = other.x == -INFINITY ? 0.0f : ex2(other.x - mm);
                    // (l is NaN where q is, and m may be -infinity then)
                    l = (m == -INFINITY ? l : l * f_own) + (other.x == -INFINITY ? other.y : other.y * f_other);
                    m = mm;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[16];
                        if (n > 0) {
                            ld16(o_at + (w ^ 1) * (D / 2) + 16 * c, o);
                            ld_wait(o);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (n > 0)
                                x = make_float4(__uint_as_float(o[4 * u]) * f_own, __uint_as_float(o[4 * u + 1]) * f_own,
                                                __uint_as_float(o[4 * u + 2]) * f_own, __uint_as_float(o[4 * u + 3]) * f_own);
                            part[((w ^ 1) * (D / 8) + 4 * c + u) * 128 + trow] = x;
                        }
                    }
                    meet(1, kSoftWarps * 32);
                }
            }
            if (ok) {
                fence_after();
                // 16 columns of O at a time through shared memory (this warp's part of Q: every MMA that
                // reads it is done), so that rows are written in whole sectors
                const bool split = job.piece >= 0;
                if (split) pdl_launch_dependents();
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                // (streams: each warp has a place of its own in the first tile's Q)
                const uint32_t buf = base + (streams ? warp * (P::kTileQ / 8) : (pair ? w * P::kTileQ : 0u) + (warp & 3) * (P::kTileQ / 4));
                float *piece = sc.pieces + (int64_t)(job.piece + job.share * job.step + (pair ? w : 0)) * P::kPiece;
                const float4 *part = reinterpret_cast<const float4 *>(smem + P::kOffK / 4);
                const int c_lo = streams ? w * (D / 2) : 0, c_hi = streams ? c_lo + D / 2 : D;
#pragma unroll 1
                for (int c = c_lo; c < c_hi; c += 16) {
                    uint32_t o[16];
                    if (n > 0) {
                        ld16(o_at + c, o);
                        ld_wait(o);
                    }
                    float x[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = n > 0 ? __uint_as_float(o[i]) : 0.0f;
                    if (streams) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float4 y = part[(w * (D / 8) + (c - c_lo) / 4 + u) * 128 + trow];
                            x[4 * u] = (n > 0 ? x[4 * u] * f_own : 0.0f) + y.x;
                            x[4 * u + 1] = (n > 0 ? x[4 * u + 1] * f_own : 0.0f) + y.y;
                            x[4 * u + 2] = (n > 0 ? x[4 * u + 2] * f_own : 0.0f) + y.z;
                            x[4 * u + 3] = (n > 0 ? x[4 * u + 3] * f_own : 0.0f) + y.w;
                        }
                    }
                    if (!split) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = l == 0.0f ? 0.0f : x[i] * inv;
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)),
                                     "f"(x[4 * u]), "f"(x[4 * u + 1]), "f"(x[4 * u + 2]), "f"(x[4 * u + 3])
                                     : "memory");
                    __syncwarp();
                    // four lanes write the 16 columns of a row
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tr = i * 8 + (lane >> 2), u = lane & 3;
                        float4 y;
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                                     : "r"(buf + tr * 64 + ((u ^ ((tr >> 1) & 3)) << 4))
                                     : "memory");
                        const unsigned rr = tile_row + row0 + tr;
                        if (rr < (unsigned)rows) {
                            if (split) {
                                *reinterpret_cast<float4 *>(piece + (row0 + tr) * D + c + 4 * u) = y;
                            } else {
                                const unsigned i_q = rr / group;
                                const int64_t to = ((int64_t)(span.lo + i_q) * a.q_heads + head * group + rr - i_q * group) * D + c + 4 * u;
                                uint2 h;
                                if (bf) h = make_uint2(Half2Of<__nv_bfloat16>::pack(y.x, y.y), Half2Of<__nv_bfloat16>::pack(y.z, y.w));
                                else h = make_uint2(Half2Of<__half>::pack(y.x, y.y), Half2Of<__half>::pack(y.z, y.w));
                                *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(a.out) + to) = h;
                            }
                        }
                    }
                    __syncwarp();
                }
                if (real && (!streams || w == 0)) {
                    if (split) {
                        piece[128 * D + trow] = m;
                        piece[128 * D + 128 + trow] = l;
                    } else if (a.lse) {
                        const unsigned i_q = r / group;
                        a.lse[(int64_t)(span.lo + i_q) * a.q_heads + head * group + r - i_q * group] =
                            l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
                    }
                }
            }
        }
    } else if (warp < kMmaWarp) {
        // ---- codes to fp16 tiles -----------------------------------------------------------
        // An item is 512 bytes of keys: D / 16 lanes take a key, 16 codes each, so that a
        // quarter warp reads 128 bytes in a row.  Its 16-byte stores hit all banks once too: a lane in
        // the upper half of a key's 128 bytes (another panel, same banks) stores its second eight first.
        constexpr int kRowLanes = D / 16, kItems = (int)P::kUnit / 512, kEach = (kItems + kWarpsKV - 1) / kWarpsKV;
        const bool is_v = warp >= kSoftWarps + kWarpsKV;
        const int cw = warp - kSoftWarps - (is_v ? kWarpsKV : 0);
        const uint32_t tile0 = base + (is_v ? P::kOffV : P::kOffK);
        const int end = min(L, k_lo + steps * KT);  // of this CTA's keys
        const int u = lane % kRowLanes, sub = lane / kRowLanes;
        const bool second = (u >> 2) & 1;
        for (int j = 0; j < steps; ++j) {
            bool ok = true;
            if (j >= kStages) ok = wait(is_v ? v_empty(j) : k_empty(j), j / kStages - 1);
            const uint32_t tile = tile0 + (j % kStages) * P::kKV;
            ok = wait(raw_full(is_v, j), j / ring) && ok;
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t at = raw_at(is_v, j) + lane * 16;
            const int k0 = k_lo + j * KT;
            const bool cut = k0 + KT > end;
            uint4 codes[kEach];  // all on their way: shared memory answers slowly while MMAs read it
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(codes[i].x), "=r"(codes[i].y), "=r"(codes[i].z), "=r"(codes[i].w)
                             : "r"(at + min(cw + i * kWarpsKV, kItems - 1) * 512)
                             : "memory");
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int item = cw + i * kWarpsKV;
                if (kItems % kWarpsKV != 0 && item >= kItems) break;
                uint4 x = codes[i];
                const int kk = item * (32 / kRowLanes) + sub;
                // keys past the last: 0, never stale bytes
                if (cut && k0 + kk >= end) x = make_uint4(0, 0, 0, 0);
                const uint32_t a0 = second ? x.z : x.x, a1 = second ? x.w : x.y, b0 = second ? x.x : x.z, b1 = second ? x.y : x.w;
                const int key = kk;
                const uint32_t to = tile + (u >> 2) * P::kPanelKV + key * 128;
                const uint32_t w[4] = {C::ready(a0), C::ready(a1), C::ready(b0), C::ready(b1)};
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + ((((u & 3) * 2 + (h ^ (int)second)) ^ (key & 7)) << 4)),
                                 "r"(C::template pair<0>(w[2 * h])), "r"(C::template pair<1>(w[2 * h])),
                                 "r"(C::template pair<0>(w[2 * h + 1])), "r"(C::template pair<1>(w[2 * h + 1]))
                                 : "memory");
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty(is_v, j));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(is_v ? v_full(j) : k_full(j));
        }
    } else if (warp == kCopyWarp) {
        // ---- copies of the codes -------------------------------------------------------------
        // Lane b < 8 has block b of a step.  Page ids are read one step ahead of the scales and the
        // copies that need them.
        constexpr uint32_t kBytes = kBlock * D;  // of a block
        const int end = min(L, k_lo + steps * KT);
        auto look_up = [&](int j) {
            const int t = k_lo + j * KT + lane * kBlock;
            return lane < P::kBlocks && t < end ? a.L.listed(row, t) : 0;
        };
        int page = look_up(0);
        int issued[2] = {0, 0};  // units whose copies are on their way
        bool ok = true;
        for (int j = 0; j < steps && ok; ++j) {
            const int t = k_lo + j * KT + lane * kBlock;
            const bool mine = lane < P::kBlocks && t < end;
            const int64_t place = a.L.block_at((unsigned)page < (unsigned)a.L.pages ? page : 0, head, t);
            page = look_up(j + 1);
            float2 sc_now = make_float2(1.0f, 1.0f);
            if (mine) sc_now = make_float2(__ldg(a.L.ks + place), __ldg(a.L.vs + place));
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * kBytes;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                if (j >= ring) ok = ok && __all_sync(0xffffffffu, wait(raw_empty(which, j), j / ring - 1));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(raw_full(which, j), bytes);
                __syncwarp();
                if (mine)
                    bulk_g2s(raw_at(which, j) + lane * kBytes, (which ? a.L.v : a.L.k) + place * kBytes, kBytes, raw_full(which, j));
                issued[which] = j + 1;
            }
            if (lane < P::kBlocks) scales[j % kScaleRing][lane] = make_float2(sc_now.x, __log2f(fmaxf(sc_now.y, 1e-37f)));
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_full(j));
        }
        // nothing of this CTA's is in flight when it leaves
#pragma unroll
        for (int which = 0; which < 2; ++which)
            for (int i = max(0, issued[which] - ring); i < issued[which]; ++i)
                mbar_wait_for(raw_full(which, i), (i / ring) & 1, kDrainWaitNs, &g_masked_timeouts);
    } else {
        // ---- MMA issue: the warp runs converged, one elected lane issues -------------------
        constexpr uint32_t i_qk = idesc_f16(128, KT, false), i_pv = idesc_f16(128, D, true), hi_word = desc128_hi(1024);
        const uint32_t q_lo = desc128_lo(base, 16), k_word = desc128_lo(base + P::kOffK, 16);
        const uint32_t v_word = desc128_lo(base + P::kOffV, P::kPanelKV);
        auto qk = [&](int j, int tile, int slot) {
            const uint32_t q = q_lo + tile * (P::kTileQ / 16), k = k_word + (j % kStages) * (P::kKV / 16);
#pragma unroll 1
            for (int s = 0; s < D / 16; ++s)
                mma_ss(tmem + (slot ? P::kS1 : 0), q + ((s / 4) * P::kPanelQ + (s % 4) * 32) / 16, hi_word,
                       k + ((s / 4) * P::kPanelKV + (s % 4) * 32) / 16, hi_word, i_qk, s > 0);
            commit(s_full(slot));
        };
        auto all_ok = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        // O += P V of a step, by parts; `first`: O starts here
        auto pv = [&](int j, int w, int slot, int phase, bool first) {
            const uint32_t v = v_word + (j % kStages) * (P::kKV / 16);
#pragma unroll
            for (int part = 0; part < P::kParts; ++part) {
                if (!all_ok(p_full(slot, part), phase)) return false;
                fence_after();
#pragma unroll
                for (int i = 0; i < KT / (16 * P::kParts); ++i) {
                    const int s = part * (KT / (16 * P::kParts)) + i;
                    mma_ts(tmem + (w ? P::kO1 : P::kO0), tmem + (slot ? P::kS1 : 0) + 8 * s, v + s * (16 * 128 / 16), hi_word, i_pv,
                           !first || s > 0);
                }
                if (part + 1 < P::kParts) commit(pv_half(slot));
            }
            return true;
        };
        auto tile_of = [&](uint32_t b, int j) {  // a converted tile
            const bool got = all_ok(b, j / kStages);
            fence_after();
            return got;
        };
        bool ok = steps > 0 && all_ok(q_full, 0) && tile_of(k_full(0), 0);
        if (ok) {
            qk(0, 0, 0);
            if (pair) qk(0, 1, 1);
            commit(k_empty(0));
        }
        if (pair) {
            for (int j = 0; j < steps && ok; ++j) {
                const bool next = j + 1 < steps;
                // the tiles of this step's second product and of the next step's first before the wait for
                // P that everything here follows
                ok = tile_of(v_full(j), j) && (!next || tile_of(k_full(j + 1), j + 1)) && pv(j, 0, 0, j, j == 0);
                if (!ok) break;
                if (next) qk(j + 1, 0, 0);
                else commit(o_full(0));
                ok = pv(j, 1, 1, j, j == 0);
                if (!ok) break;
                commit(v_empty(j));
                if (next) {
                    qk(j + 1, 1, 1);
                    commit(k_empty(j + 1));
                } else {
                    commit(o_full(1));
                }
            }
        } else if (streams) {
            if (ok && steps > 1) {
                ok = tile_of(k_full(1), 1);
                if (ok) {
                    qk(1, 0, 1);
                    commit(k_empty(1));
                }
            }
            for (int j = 0; j < steps && ok; ++j) {
                const int w = j & 1;
                const bool next = j + 2 < steps;
                ok = tile_of(v_full(j), j) && pv(j, w, w, j >> 1, j < 2);
                if (!ok) break;
                commit(v_empty(j));
                if (next) {
                    ok = tile_of(k_full(j + 2), j + 2);
                    if (!ok) break;
                    qk(j + 2, 0, w);
                    commit(k_empty(j + 2));
                } else {
                    commit(o_full(w));
                }
            }
        } else {
            for (int j = 0; j < steps && ok; ++j) {
                const bool next = j + 1 < steps;
                if (next) {
                    ok = tile_of(k_full(j + 1), j + 1);
                    if (!ok) break;
                    qk(j + 1, 0, (j + 1) & 1);
                    commit(k_empty(j + 1));
                }
                ok = tile_of(v_full(j), j) && pv(j, 0, j & 1, j >> 1, j == 0);
                if (!ok) break;
                commit(v_empty(j));
                commit(pv_done);
                if (!next) commit(o_full(0));
            }
        }
        if (steps > 0) {
            // On every exit: what was issued reads shared memory, writes TMEM and arrives on barriers
            // of this CTA.  Let it finish.
            commit(drained);
            mbar_wait_for(drained, 0, kDrainWaitNs, &g_masked_timeouts);
        }
    }
    st_wait();  // a role that gave up may have stores to TMEM on their way
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, P::kCols);
}

// Joins the shares of a tile, in order
template <int D>
__global__ void __launch_bounds__(256)
masked_join_kernel(const AttendArgs a, const Scratch sc)
{
    using P = Plan<D>;
    pdl_wait();
    const int tile = blockIdx.x % sc.tiles, head = blockIdx.x / sc.tiles % a.L.heads, row = blockIdx.x / sc.tiles / a.L.heads;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int rows = span.n * a.group, r0 = tile * 128, i = blockIdx.y * 256 + threadIdx.x;
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r0 + r >= rows) return;
    const Record rec = sc.records[blockIdx.x];
    if (rec.first < 0) return;
    const float *at = sc.pieces + (int64_t)rec.first * P::kPiece;
    const int64_t step = (int64_t)rec.step * P::kPiece;
    float m = -INFINITY, l = 0.0f;
#pragma unroll 4
    for (int k = 0; k < rec.count; ++k) m = fmaxf(m, at[k * step + 128 * D + r]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < rec.count; ++k) {
        const float *p = at + k * step;
        const float mk = p[128 * D + r], lk = p[128 * D + 128 + r];
        const float f = mk == -INFINITY ? (lk == 0.0f ? 0.0f : 1.0f) : ex2(mk - m);  // (l is NaN where q is)
        const float4 x = *reinterpret_cast<const float4 *>(p + r * D + d);
        o.x = fmaf(x.x, f, o.x), o.y = fmaf(x.y, f, o.y), o.z = fmaf(x.z, f, o.z), o.w = fmaf(x.w, f, o.w);
        l = fmaf(lk, f, l);
    }
    const int qi = (r0 + r) / a.group, h = (r0 + r) % a.group;
    const int64_t to = (int64_t)(span.lo + qi) * a.q_heads + head * a.group + h;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 v;
    if (a.dtype == BQD_DTYPE_BF16)
        v = make_uint2(Half2Of<__nv_bfloat16>::pack(o.x * inv, o.y * inv), Half2Of<__nv_bfloat16>::pack(o.z * inv, o.w * inv));
    else
        v = make_uint2(Half2Of<__half>::pack(o.x * inv, o.y * inv), Half2Of<__half>::pack(o.z * inv, o.w * inv));
    *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(a.out) + to * D + d) = v;
    if (a.lse && d == 0) a.lse[to] = l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
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

// Pieces that a call may leave: two waves of pairs' shares
int most_pieces(const AttendArgs &a) { return a.L.rows > kMaxRows ? 0 : 4 * sm_count(); }

int64_t planned_tiles(const AttendArgs &a) { return ((int64_t)a.max_new * a.group + 127) / 128; }

// bytes of the records of shares, at a multiple of a Place's alignment
int64_t record_bytes(const AttendArgs &a)
{
    return ((int64_t)a.L.rows * a.L.heads * planned_tiles(a) * (int64_t)sizeof(Record) + 7) / 8 * 8;
}

template <int D>
int64_t workspace_d(const AttendArgs &a)
{
    const int64_t most = most_pieces(a);
    return most == 0 ? 0 : most * Plan<D>::kPiece * (int64_t)sizeof(float) + record_bytes(a) +
                               ((int64_t)a.L.rows + 1) * (int64_t)sizeof(Place);
}

template <int D, int FMT>
int launch_t(const AttendArgs &a, cudaStream_t s)
{
    using P = Plan<D>;
    auto kern = attend_masked_kernel<D, FMT>;
    static bool done[64] = {};
    if (!configure(kern, P::kSmem, done)) return BQD_ERR_CUDA;
    const int64_t tiles = planned_tiles(a), all = (int64_t)a.L.rows * a.L.heads * tiles;
    if (all > 0x20000000) return BQD_ERR_INVALID_ARG;
    // every unit once, and what shares may add
    const int64_t units = (int64_t)a.L.rows * a.L.heads * (P::kTiles == 2 ? (tiles + 1) / 2 : tiles);
    Scratch sc = {nullptr, nullptr, nullptr, 0, (int)tiles};
    if (a.work) {
        sc.most = most_pieces(a);
        sc.pieces = static_cast<float *>(a.work);
        sc.records = reinterpret_cast<Record *>(sc.pieces + (int64_t)sc.most * P::kPiece);
        sc.places = reinterpret_cast<Place *>(reinterpret_cast<char *>(sc.records) + record_bytes(a));
    }
    const bool planned = sc.most > 0 && a.L.rows > kOwnRows;
    if (planned) {
        masked_plan_kernel<D><<<1, kThreadsM, 0, s>>>(a, sc, sm_count());
        const int st = cuda_status(cudaGetLastError());
        if (st != BQD_OK) return st;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units + sc.most));
    cfg.blockDim = dim3(kThreadsM);
    cfg.dynamicSmemBytes = P::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = planned ? 1 : 0;  // without a plan's kernel this one waits for whatever came before
    const int st = cuda_status(cudaLaunchKernelEx(&cfg, kern, a, sc, sm_count(), (unsigned long long)opt_wait_ns()));
    if (st != BQD_OK || sc.most == 0) return st;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)all, 128 * D / 4 / 256);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, masked_join_kernel<D>, a, sc));
}

template <int D>
int launch_f(const AttendArgs &a, cudaStream_t s)
{
    return a.format == BQD_KV_INT8 ? launch_t<D, BQD_KV_INT8>(a, s) : launch_t<D, BQD_KV_E4M3>(a, s);
}

}  // namespace

int64_t masked_workspace(const AttendArgs &a)
{
    return a.head_dim == 64 ? workspace_d<64>(a) : a.head_dim == 128 ? workspace_d<128>(a) : workspace_d<256>(a);
}

int launch_attend_masked(const AttendArgs &a, cudaStream_t s)
{
    return a.head_dim == 64 ? launch_f<64>(a, s) : a.head_dim == 128 ? launch_f<128>(a, s) : launch_f<256>(a, s);
}

int take_masked_timeouts(unsigned int *count)
{
    if (cudaMemcpyFromSymbol(count, g_masked_timeouts, sizeof(*count)) != cudaSuccess) return BQD_ERR_CUDA;
    if (*count) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_masked_timeouts, &zero, sizeof(zero)) != cudaSuccess) return BQD_ERR_CUDA;
    }
    return BQD_OK;
}

}  // namespace kv
}  // namespace bqd
