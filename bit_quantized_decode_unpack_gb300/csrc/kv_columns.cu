// Attention over a paged 8-bit cache under masks, for tens to hundreds of (query,
// head) columns that face the same keys: trees of drafted tokens.
//
// The mathematics is that of the few-query kernel (kv_attend.cu): with f the score
// scale times log2(e) and s^k_b, s^v_b the scales of 16-token block b,
//   x_jc = f s^k_b (c^k_j . q_c) + log2 s^v_b,   p_jc = 2^(x_jc - m_c),
//   O_c = sum_j p_jc c^v_j,   l_c = sum_b (sum_{j in b} p_jc) / s^v_b,
//   out = O / l,   lse = ln 2 (m + log2 l),
// with m_c replaced only when x passes it by 15 (p < 2^15 fits fp16).
//
// Both products run on the 5th-generation tensor cores with the cache as the 128-row
// operand: S^T = K Q^T (128 keys x columns) and O^T = V^T P^T (head_dim x columns).
// The columns are the N of an MMA, any multiple of 32 up to 128, so few columns
// cost what they are, not a tile of 128 queries, and a thread of the softmax has one
// key and half of the columns: its scales are its own, its exponentials and sums of l
// never leave it until the end, and only m_c (shared memory) and the vote whether one
// of them grows (a barrier of four warps for 32 columns) are common.
// O^T, S^T (two buffers) stay in TMEM; P^T goes to shared memory as the MN-major
// operand of the second product, V is the MN-major first one as it lies.
// Queries of a column tile are taken in fp16 with one power of two for all: elements
// below 2^-28 of the tile's largest lose bits, 2^-39 of that largest at most.
//   warps 0-7    softmax: warp % 4 gives the 32 keys (TMEM lanes), warps 0-3 take the
//                32-column pieces 0, 2 and warps 4-7 the pieces 1, 3
//   warps 8-10, 11-13  K's, V's codes from shared memory to fp16 tiles (128-byte swizzle)
//   warp 14      TMEM, and one elected lane that issues every MMA
//   warp 15      bulk copies of the codes, a ring ahead of the conversion, and the scales
//
// Work.  A unit is (row, KV head, column tile); a unit's key steps are cut into equal
// shares.  No host knows the rows' lengths: every CTA adds up the rows' steps and finds
// the same share length, the one with the least estimated time, and its own place.
// Shares leave O, m and l in scratch, and a second kernel, launched early, joins
// them in order.  No atomics: the same bits every time.
// Every wait is bounded; on expiry a role stops (the warps that meet at a barrier
// agree on it first), what it issued is drained, TMEM is freed, and bqd_device_status
// reports it.
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
constexpr int kMmaWarp = kSoftWarps + 2 * kWarpsKV;
constexpr int kCopyWarp = kMmaWarp + 1;
constexpr int kThreadsM = (kCopyWarp + 1) * 32;
constexpr int KT = 128;             // keys of a step
constexpr int kBlocks = KT / kBlock;
constexpr int kScaleRing = 8;       // steps whose scales are kept: the copies run ahead of the softmax by a
                                    // ring of codes, a tile and two S, five steps at most
constexpr int kMaxRows = 1024;      // rows that a CTA adds up
constexpr int kMaxShares = 64;      // shares of a unit
constexpr float kGrow = 15.0f;
constexpr float kNothing = -3.0e38f;  // m of a column that has seen nothing

__device__ unsigned int g_columns_timeouts = 0;

template <int D>
struct Plan {
    static constexpr int NT = D == 256 ? 64 : 128;       // columns of a tile
    static constexpr int kStages = D == 64 ? 2 : 1;      // fp16 tiles of K and of V
    // codes come in units of at most 16 KB, a ring of them for K and one for V
    static constexpr int kUnitKeys = D == 256 ? 64 : 128, kUnits = KT / kUnitKeys;  // units of a step
    static constexpr uint32_t kUnit = kUnitKeys * D;
    static constexpr int kRing = D == 64 ? 4 : D == 128 ? 2 : 1;
    static constexpr int kPanels = D / 64;
    static constexpr int kOut = D == 256 ? 2 : 1;        // 128-row parts of O^T
    static constexpr uint32_t kPanelKV = KT * 128, kKV = kPanels * kPanelKV;
    static constexpr uint32_t kPanelQ = NT * 128, kQ = kPanels * kPanelQ;
    static constexpr uint32_t kPanelP = KT * 128, kP = NT / 64 * kPanelP;
    static constexpr uint32_t kOffK = kQ, kOffV = kOffK + kStages * kKV, kOffP = kOffV + kStages * kKV;
    static constexpr uint32_t kOffRaw = kOffP + 2 * kP;
    static constexpr size_t kSmem = 1024 + kOffRaw + 2 * kRing * kUnit;
    static constexpr uint32_t kO = 2 * NT;               // TMEM: S, S, O
    static constexpr uint32_t kCols = NT == 64 ? 256 : 512;
    static constexpr int kPieces = NT / 64;              // 32-column pieces of a softmax warp
    static constexpr int kPiece = NT * D + 2 * NT;       // floats of a share: O [NT][D], m, l
};

struct Record {
    int first, count;  // pieces of a unit; count 1: the unit is done
};

struct Scratch {
    float *pieces;
    Record *records;   // [rows * heads * column tiles of max_new]
    int most;          // pieces
    int ctiles;        // column tiles of max_new
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

// whether any of the 128 threads that meet at this barrier says so
__device__ __forceinline__ bool any_of(int id, bool mine)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %2, 0;\n\tbarrier.cta.red.or.pred.aligned q, %1, 128, p;\n\t"
        "selp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"((int)mine)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void meet(int id, int threads)
{
    asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// floats as integers of the same order
__device__ __forceinline__ int ordered(float x)
{
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}

__device__ __forceinline__ float unordered(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF)); }

// Keys of a row that any of its queries sees start at lo
__device__ __forceinline__ int first_key(const AttendArgs &a, int L, const Span &span)
{
    return a.window > 0 ? max(0, L - span.rest + 1 - a.window) / KT * KT : 0;
}

// What the CTA does
struct Job {
    int row, head, ctile, share, count, piece;  // piece: of share 0, or -1
};

// Every CTA computes the same share length and finds its job in it.  A share costs its steps and
// kFixed more; S CTAs on `sms` SMs take S (steps + kFixed) / sms and, beyond one wave, about half
// a share more for the tail.
constexpr float kFixed = 6.0f;

template <int D>
__device__ Job find_job(const AttendArgs &a, const Scratch &sc, int sms, int *row_steps, int *row_units, int *row_at,
                        int *warp_sums, int *chosen)
{
    using P = Plan<D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rows = a.L.rows;
    if (rows > kMaxRows) {  // nothing is shared
        Job j = {(int)(blockIdx.x / (unsigned)(sc.ctiles * a.L.heads)), (int)(blockIdx.x / (unsigned)sc.ctiles % a.L.heads),
                 (int)(blockIdx.x % (unsigned)sc.ctiles), 0, 1, -1};
        const Span span(a.starts, j.row, a.tokens, a.max_new);
        if (j.ctile * P::NT >= span.n * a.group) j.row = -1;
        return j;
    }
    for (int r = tid; r < rows; r += kThreadsM) {
        const Span span(a.starts, r, a.tokens, a.max_new);
        const int L = a.L.length(r), lo = first_key(a, L, span);
        row_steps[r] = max(1, (L - lo + KT - 1) / KT);
        row_units[r] = (span.n * a.group + P::NT - 1) / P::NT * a.L.heads;
    }
    __syncthreads();
    if (warp == 0) {
        int longest = 1;
        for (int r = lane; r < rows; r += 32)
            if (row_units[r]) longest = max(longest, row_steps[r]);
        longest = __reduce_max_sync(0xffffffffu, longest);
        // lane i tries shares of longest 2^(-i / 4) steps; lane 0 splits nothing
        int each = max(1, (int)ceilf(longest * exp2f(-0.25f * lane)));
        each = max(max(each, 2), (longest + kMaxShares - 1) / kMaxShares);
        if (lane == 0 || sc.most == 0) each = longest;
        float work = 0.0f;
        int64_t ctas = 0, pieces = 0;
        for (int r = 0; r < rows; ++r) {
            const int u = row_units[r], n = (row_steps[r] + each - 1) / each;
            work += (float)u * (row_steps[r] + n * kFixed);
            ctas += (int64_t)u * n;
            if (n > 1) pieces += (int64_t)u * n;
        }
        float cost = work / sms;
        if (ctas > sms) cost += 0.5f * (each + kFixed);
        cost = fmaxf(cost, each + kFixed);
        if (pieces > sc.most) cost = 3.0e38f;
        // the least cost, of equals the longest shares
        int best = lane;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float c = __shfl_xor_sync(0xffffffffu, cost, o);
            const int b = __shfl_xor_sync(0xffffffffu, best, o);
            if (c < cost || (c == cost && b < best)) cost = c, best = b;
        }
        if (lane == best) *chosen = each;
    }
    __syncthreads();
    const int each = *chosen;
    // CTAs and pieces of the rows before each: a thread takes consecutive rows
    const int per = (rows + kThreadsM - 1) / kThreadsM;
    int mine = 0, cut = 0;
    for (int i = 0; i < per; ++i) {
        const int r = tid * per + i;
        if (r >= rows) break;
        const int n = (row_steps[r] + each - 1) / each;
        mine += row_units[r] * n;
        if (n > 1) cut += row_units[r] * n;
    }
    int x = mine, y = cut;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xffffffffu, x, o), q = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) x += p, y += q;
    }
    if (lane == 31) warp_sums[2 * warp] = x, warp_sums[2 * warp + 1] = y;
    __syncthreads();
    int at = x - mine, piece = y - cut;
    for (int w = 0; w < warp; ++w) at += warp_sums[2 * w], piece += warp_sums[2 * w + 1];
    const int b = blockIdx.x;
    if (tid == 0) row_at[0] = -1;
    __syncthreads();
    for (int i = 0; i < per; ++i) {
        const int r = tid * per + i;
        if (r >= rows) break;
        const int n = (row_steps[r] + each - 1) / each, ctas = row_units[r] * n;
        if (b >= at && b < at + ctas) {  // one thread of the CTA finds its row
            row_at[0] = r;
            row_at[1] = b - at;
            row_at[2] = n;
            row_at[3] = n > 1 ? piece : -1;
        }
        at += ctas;
        if (n > 1) piece += ctas;
    }
    __syncthreads();
    Job j = {row_at[0], 0, 0, 0, 1, -1};
    if (j.row < 0) return j;
    // column tiles fastest, then heads, then shares: CTAs that read the same keys run together
    const int i = row_at[1], units = row_units[j.row], ct = units / a.L.heads;
    j.count = row_at[2];
    j.ctile = i % ct;
    j.head = i / ct % a.L.heads;
    j.share = i / units;
    if (row_at[3] >= 0) j.piece = row_at[3] + (j.head * ct + j.ctile) * j.count;
    return j;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreadsM, 1)
attend_columns_kernel(const AttendArgs a, const Scratch sc, int sms, unsigned long long wait_ns)
{
    using P = Plan<D>;
    using C = Code<FMT>;
    constexpr int NT = P::NT, kStages = P::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[48];
    __shared__ __align__(16) float2 scales[kScaleRing][kBlocks];  // of a step's blocks: K's scale, log2 of V's
    __shared__ __align__(16) float m_of[NT];
    __shared__ int top_of[kSoftWarps], high_of[2][32];            // of the queries; of a piece's new scores
    __shared__ int found[4], chosen, sums[2 * (kCopyWarp + 1)];
    __shared__ uint32_t tmem_at;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // the rows' steps and units take the place of tiles that come later
    int *row_steps = reinterpret_cast<int *>(raw);
    const Job job = find_job<D>(a, sc, sms, row_steps, row_steps + kMaxRows, found, sums, &chosen);
    if (job.row < 0) return;
    const int row = job.row, head = job.head;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int cols = span.n * a.group, c0 = job.ctile * NT;
    const int nc = min(NT, cols - c0);            // columns of this tile
    const int N = (nc + 31) & ~31;                // of an MMA: whole pieces, the rest of them zeros
    const int L = a.L.length(row), before = L - span.rest;
    const int k_first = first_key(a, L, span), all = max(0, (L - k_first + KT - 1) / KT);
    const int from = (int)((int64_t)all * job.share / job.count);
    const int steps = (int)((int64_t)all * (job.share + 1) / job.count) - from;
    const int k_lo = k_first + from * KT;
    const int unit = (row * a.L.heads + head) * sc.ctiles + job.ctile;
    if (sc.records && job.share == 0 && tid == 0) sc.records[unit] = Record{job.piece, job.count};

    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    auto k_full = [&](int j) { return bar(j % kStages); };
    auto k_empty = [&](int j) { return bar(2 + j % kStages); };
    auto v_full = [&](int j) { return bar(4 + j % kStages); };
    auto v_empty = [&](int j) { return bar(6 + j % kStages); };
    auto s_full = [&](int j) { return bar(8 + (j & 1)); };
    auto p_full = [&](int j) { return bar(10 + (j & 1)); };
    auto pv_done = [&](int j) { return bar(12 + (j & 1)); };
    const uint32_t q_full = bar(14), o_full = bar(15), drained = bar(16);
    auto sc_full = [&](int j) { return bar(17 + j % kScaleRing); };
    auto raw_full = [&](int which, int u) { return bar(25 + 4 * which + u % P::kRing); };
    auto raw_empty = [&](int which, int u) { return bar(33 + 4 * which + u % P::kRing); };

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(bar(i), kWarpsKV);
                mbar_init(bar(2 + i), 1);
                mbar_init(bar(4 + i), kWarpsKV);
                mbar_init(bar(6 + i), 1);
                mbar_init(bar(8 + i), 1);
                mbar_init(bar(10 + i), kSoftWarps * 32);
                mbar_init(bar(12 + i), 1);
            }
            mbar_init(q_full, kSoftWarps * 32);
            mbar_init(o_full, 1);
            mbar_init(drained, 1);
            for (int i = 0; i < kScaleRing; ++i) mbar_init(sc_full(i), 1);
            for (int i = 0; i < 8; ++i) mbar_init(bar(25 + i), 1), mbar_init(bar(33 + i), kWarpsKV);
        }
        __syncwarp();
        tmem_alloc(smem_addr(&tmem_at), P::kCols);
    }
    if (tid < NT) m_of[tid] = kNothing;
    if (tid < 64) high_of[tid >> 5][lane] = ordered(-INFINITY);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_at;
    auto wait = [&](uint32_t b, uint32_t parity) { return mbar_wait_for(b, parity & 1, wait_ns, &g_columns_timeouts); };

    if (warp < kSoftWarps) {
        const int g = warp >> 2;                               // half of the pieces
        const int key = (warp & 3) * 32 + lane;                // of a step; also a row of O^T
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;     // TMEM lane 32 (warp % 4), in bits 16..31
        const int bar_id = 1 + g;
        const unsigned group = a.group;
        // ---- q: scaled by one power of two into fp16 -------------------------------------
        float cs;
        {
            constexpr int kRowLoads = D / 8, kEach = NT * kRowLoads / (kSoftWarps * 32);
            const bool bf = a.dtype == BQD_DTYPE_BF16;
            const uint32_t inf = bf ? Half2Of<__nv_bfloat16>::kInf : Half2Of<__half>::kInf;
            uint4 v[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = tid + i * kSoftWarps * 32;
                const unsigned c = c0 + at / kRowLoads, qi = c / group;
                v[i] = make_uint4(0, 0, 0, 0);
                if (c < (unsigned)cols) {
                    const unsigned short *q = static_cast<const unsigned short *>(a.q) + (int64_t)(span.lo + qi) * a.q_token +
                                              (int64_t)(head * group + c - qi * group) * a.q_head + at % kRowLoads * 8;
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
            uint32_t top = 0;  // the largest finite magnitude
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = x[k] & 0x7FFFu, hi = (x[k] >> 16) & 0x7FFFu;
                    if (lo < inf) top = max(top, lo);
                    if (hi < inf) top = max(top, hi);
                }
            }
            top = __reduce_max_sync(0xffffffffu, top);
            if (lane == 0) top_of[warp] = (int)top;
            meet(3, kSoftWarps * 32);
#pragma unroll
            for (int w = 0; w < kSoftWarps; ++w) top = max(top, (uint32_t)top_of[w]);
            // exponent of the largest: it goes to 2^13 .. 2^14
            int e = 13;
            if (top != 0) {
                const float f = bf ? Half2Of<__nv_bfloat16>::f1(top) : Half2Of<__half>::f1(top);
                e = max(-100, min(126, (int)((__float_as_uint(f) >> 23) & 0xFF) - 127));
            }
            // the sign of the scale goes with q
            const float down = copysignf(__uint_as_float((uint32_t)(127 + 13 - e) << 23), a.scale);
            cs = fabsf(a.scale) * __uint_as_float((uint32_t)(127 - 13 + e) << 23);
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int at = tid + i * kSoftWarps * 32, c = at / kRowLoads, u = at % kRowLoads;
                const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = bf ? Half2Of<__nv_bfloat16>::f2(x[k]) : Half2Of<__half>::f2(x[k]);
                    h[k] = Half2Of<__half>::pack(f.x * down, f.y * down);
                }
                const uint32_t to = base + (u >> 3) * P::kPanelQ + c * 128 + (((u & 7) ^ (c & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                             : "memory");
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
        }

        // ---- steps -----------------------------------------------------------------------
        uint64_t l2[P::kPieces][16];  // of the thread's key, two columns each
#pragma unroll
        for (int k = 0; k < P::kPieces; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) l2[k][i] = two(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < steps; ++j) {
            const int k0 = k_lo + j * KT;
            ok = wait(sc_full(j), j / kScaleRing);
            const float2 sr = scales[j % kScaleRing][key >> 4];
            const float f = cs * sr.x, lv = sr.y, rv = ex2(-lv);
            ok = wait(s_full(j), j >> 1) && ok;
            if (j >= 2) ok = wait(pv_done(j), (j >> 1) - 1) && ok;  // the place of P is free
            fence_after();
            const bool whole = k0 + KT <= before && (a.window == 0 || k0 > L - 1 - a.window);
            const uint32_t s_at = tmem + lanes + (j & 1) * NT;
            const uint32_t p_at = base + P::kOffP + (j & 1) * P::kP + key * 128;
#pragma unroll
            for (int k = 0; k < P::kPieces; ++k) {
                const int piece = 2 * k + g, cp = piece * 32;  // the piece's first column
                if (cp >= N) continue;                         // (the same for all that vote)
                uint32_t s[32];
                ld32(s_at + cp, s);
                ld_wait(s);
                uint32_t sees = 0xFFFFFFFFu;
                if (!whole) {
                    // bit i: column cp + i sees this thread's key
                    const int node = k0 + key - before;
                    unsigned c = c0 + cp, qi = c / group, h = c - qi * group;
                    sees = 0;
                    bool one = false;
#pragma unroll 1
                    for (int i = 0; i < 32; ++i, ++c) {
                        if (i == 0 || h == group) {
                            if (h == group) h = 0, ++qi;
                            const int token = span.lo + qi;
                            one = c < (unsigned)cols && k0 + key < L;
                            if (one && node >= 0)
                                one = node < 64 * a.words &&
                                      (__ldg(a.mask + (int64_t)token * a.words + (node >> 6)) >> (node & 63) & 1) != 0;
                            else if (one && a.window > 0)
                                one = node > max(0, min(__ldg(a.depth + token), span.rest - 1)) - a.window;
                        }
                        sees |= (uint32_t)one << i;
                        ++h;
                    }
                }
                float top = -INFINITY;
                const uint64_t ff = two(f, f), aa = two(lv, lv);
                uint64_t t2[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 mm = *reinterpret_cast<const float4 *>(&m_of[cp + 4 * i]);
                    t2[2 * i] = fma2(two(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), ff, add2(aa, two(-mm.x, -mm.y)));
                    t2[2 * i + 1] =
                        fma2(two(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), ff, add2(aa, two(-mm.z, -mm.w)));
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 t = untwo(t2[i]);
                        if (!(sees >> (2 * i) & 1)) t.x = -INFINITY;
                        if (!(sees >> (2 * i + 1) & 1)) t.y = -INFINITY;
                        t2[i] = two(t.x, t.y);
                    }
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 t = untwo(t2[i]);
                    top = fmaxf(top, fmaxf(t.x, t.y));
                }
                if (any_of(bar_id, !ok || top > kGrow)) {
                    // Seldom but in the first step: new references of the piece's columns.  Lane c
                    // of every warp follows column cp + c.
                    if (j > 0) ok = wait(pv_done(j - 1), (j - 1) >> 1) && ok;  // it still adds to O
                    float x[32];
                    int high = ordered(-INFINITY);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] = fmaf(__uint_as_float(s[i]), f, lv);
                        if (!(sees >> i & 1)) x[i] = -INFINITY;
                        const int w = __reduce_max_sync(0xffffffffu, ordered(x[i]));
                        if (lane == i) high = w;
                    }
                    atomicMax(&high_of[g][lane], high);
                    if (any_of(bar_id, !ok)) {
                        ok = false;
                        break;
                    }
                    const float old = m_of[cp + lane];
                    const float hx = unordered(high_of[g][lane]);
                    const float now = hx > old + kGrow ? hx : old;
                    const float factor = ex2(old - now);
                    meet(bar_id, 128);
                    if ((warp & 3) == 0) m_of[cp + lane] = now, high_of[g][lane] = ordered(-INFINITY);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float f0 = __shfl_sync(0xffffffffu, factor, 2 * i), f1 = __shfl_sync(0xffffffffu, factor, 2 * i + 1);
                        const float2 l = untwo(l2[k][i]);
                        l2[k][i] = two(l.x * f0, l.y * f1);
                        const float n0 = __shfl_sync(0xffffffffu, now, 2 * i), n1 = __shfl_sync(0xffffffffu, now, 2 * i + 1);
                        t2[i] = two(x[2 * i] - n0, x[2 * i + 1] - n1);
                    }
                    if (j > 0) {
                        fence_after();
#pragma unroll 1
                        for (int o = 0; o < 2 * P::kOut; ++o) {
                            uint32_t r[16];
                            const uint32_t at = tmem + lanes + P::kO + (o >> 1) * NT + cp + (o & 1) * 16;
                            ld16(at, r);
                            ld_wait(r);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xffffffffu, factor, (o & 1) * 16 + i));
                            st16(at, r);
                        }
                        st_wait();
                    }
                    meet(bar_id, 128);  // m is the new one for all
                }
                const uint64_t rr = two(rv, rv);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 t = untwo(t2[4 * u + i]);
                        const float e0 = ex2(t.x), e1 = ex2(t.y);
                        l2[k][4 * u + i] = fma2(two(e0, e1), rr, l2[k][4 * u + i]);
                        p[i] = Half2Of<__half>::pack(e0, e1);
                    }
                    const uint32_t to = p_at + (piece >> 1) * P::kPanelP + ((((piece & 1) * 4 + u) ^ (key & 7)) << 4);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3])
                                 : "memory");
                }
            }
            // (warps 4-7 vote on nothing where there are 32 columns: a wait that ran out ends them here)
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_proxy_async_smem();
            fence_before();
            mbar_arrive(p_full(j));
        }
        // ---- out ---------------------------------------------------------------------------
        if (ok && steps > 0) ok = wait(o_full, 0);
        ok = !any_of(bar_id, !ok);
        if (ok) {
            fence_after();
            if (job.piece >= 0) pdl_launch_dependents();
            // l: the sums over the warp's keys, lane c of column cp + c, then over the four warps
            float *l_part = reinterpret_cast<float *>(raw + (base - smem_addr(raw)) + P::kOffP);  // [4][NT], where P was
            float *l_of = l_part + 4 * NT;                                                        // [NT]: 1 / l
#pragma unroll
            for (int k = 0; k < P::kPieces; ++k) {
                const int cp = (2 * k + g) * 32;
                float l[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 v = untwo(l2[k][i]);
                    l[2 * i] = v.x, l[2 * i + 1] = v.y;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const bool up = lane & o;
                        const float send = up ? l[i] : l[i + o], keep = up ? l[i + o] : l[i];
                        l[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                l_part[(warp & 3) * NT + cp + lane] = l[0];
            }
            meet(bar_id, 128);
            const bool split = job.piece >= 0;
            float *piece = sc.pieces + (int64_t)(job.piece + job.share) * P::kPiece;
#pragma unroll
            for (int k = 0; k < P::kPieces; ++k) {
                const int c = (2 * k + g) * 32 + lane;
                if ((warp & 3) != 0 || c >= nc) continue;
                const float l = (l_part[c] + l_part[NT + c]) + (l_part[2 * NT + c] + l_part[3 * NT + c]), m = m_of[c];
                l_of[c] = l == 0.0f ? 0.0f : 1.0f / l;
                if (split) {
                    piece[NT * D + c] = m;
                    piece[NT * (D + 1) + c] = l;
                } else if (a.lse) {
                    const unsigned cc = c0 + c, qi = cc / group;
                    a.lse[(int64_t)(span.lo + qi) * a.q_heads + head * group + cc - qi * group] =
                        l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
                }
            }
            meet(bar_id, 128);
            const bool bf = a.dtype == BQD_DTYPE_BF16;
#pragma unroll 1
            for (int o = 0; o < 2 * P::kPieces * P::kOut; ++o) {
                const int part = o % P::kOut, cp = (2 * (o / (2 * P::kOut)) + g) * 32 + (o / P::kOut & 1) * 16;
                const int d = part * 128 + key;
                if (cp >= nc) continue;  // (the same for the warp)
                uint32_t r[16];
                if (steps > 0) {
                    ld16(tmem + lanes + P::kO + part * NT + cp, r);
                    ld_wait(r);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = 0;
                }
                if (d >= D) continue;    // head_dim 64: the upper rows are a copy
                unsigned cc = c0 + cp, qi = cc / group, h = cc - qi * group;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (cp + i < nc) {
                        const float x = __uint_as_float(r[i]);
                        if (split) {
                            piece[(cp + i) * D + d] = x;
                        } else {
                            const float y = l_of[cp + i] == 0.0f ? 0.0f : x * l_of[cp + i];
                            const int64_t to = ((int64_t)(span.lo + qi) * a.q_heads + head * group + h) * D + d;
                            if (bf) static_cast<__nv_bfloat16 *>(a.out)[to] = __float2bfloat16_rn(y);
                            else static_cast<__half *>(a.out)[to] = __float2half_rn(y);
                        }
                    }
                    if (++h == group) h = 0, ++qi;
                }
            }
        }
    } else if (warp < kMmaWarp) {
        // ---- codes to fp16 tiles -----------------------------------------------------------
        // An item is 512 bytes of a unit's keys: D / 16 lanes take a key, 16 codes each, so that a
        // quarter warp reads 128 bytes in a row.  Its 16-byte stores hit all banks once too: a lane in
        // the upper half of a key's 128 bytes (another panel, same banks) stores its second eight first.
        constexpr int kRowLanes = D / 16, kItems = (int)P::kUnit / 512, kEach = (kItems + kWarpsKV - 1) / kWarpsKV;
        const bool is_v = warp >= kSoftWarps + kWarpsKV;
        const int cw = warp - kSoftWarps - (is_v ? kWarpsKV : 0);
        const uint32_t tile0 = base + (is_v ? P::kOffV : P::kOffK);
        const uint32_t raw0 = base + P::kOffRaw + (is_v ? P::kRing * P::kUnit : 0u);
        const int end = min(L, k_lo + steps * KT);  // of this CTA's keys
        const int u = lane % kRowLanes, sub = lane / kRowLanes;
        const bool second = (u >> 2) & 1;
        for (int j = 0; j < steps; ++j) {
            bool ok = true;
            if (j >= kStages) ok = wait(is_v ? v_empty(j) : k_empty(j), j / kStages - 1);
            const uint32_t tile = tile0 + (j % kStages) * P::kKV;
            for (int n = 0; n < P::kUnits; ++n) {
                const int at = j * P::kUnits + n;
                ok = wait(raw_full(is_v, at), at / P::kRing) && ok;
                if (!__all_sync(0xffffffffu, ok)) break;
                const uint32_t raw_at = raw0 + (at % P::kRing) * P::kUnit + lane * 16;
                const int k0 = k_lo + j * KT + n * P::kUnitKeys;
                const bool cut = k0 + P::kUnitKeys > end;
                uint4 codes[kEach];  // all on their way: shared memory answers slowly while MMAs read it
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(codes[i].x), "=r"(codes[i].y), "=r"(codes[i].z), "=r"(codes[i].w)
                                 : "r"(raw_at + min(cw + i * kWarpsKV, kItems - 1) * 512)
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
                    const int key = n * P::kUnitKeys + kk;
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
                if (lane == 0) mbar_arrive(raw_empty(is_v, at));
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(is_v ? v_full(j) : k_full(j));
        }
    } else if (warp == kCopyWarp) {
        // ---- copies of the codes -------------------------------------------------------------
        // Lane b < 8 has block b of a step.  Page ids are read one step ahead of the scales and the
        // copies that need them.
        constexpr int kUnitBlocks = P::kUnitKeys / kBlock;
        constexpr uint32_t kBytes = kBlock * D;  // of a block
        const int end = min(L, k_lo + steps * KT);
        auto look_up = [&](int j) {
            const int t = k_lo + j * KT + lane * kBlock;
            return lane < kBlocks && t < end ? a.L.listed(row, t) : 0;
        };
        int page = look_up(0);
        int j = 0, issued[2] = {0, 0};  // units whose copies are on their way
        bool ok = true;
        for (; j < steps && ok; ++j) {
            const int t = k_lo + j * KT + lane * kBlock;
            const bool real = lane < kBlocks && t < end;
            const int64_t place = a.L.block_at((unsigned)page < (unsigned)a.L.pages ? page : 0, head, t);
            page = look_up(j + 1);
            float2 sc_now = make_float2(1.0f, 1.0f);
            if (real) sc_now = make_float2(__ldg(a.L.ks + place), __ldg(a.L.vs + place));
            for (int n = 0; n < P::kUnits && ok; ++n) {
                const int at = j * P::kUnits + n;
                const bool mine = real && lane / kUnitBlocks == n;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, mine)) * kBytes;
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    if (at >= P::kRing) ok = __all_sync(0xffffffffu, wait(raw_empty(which, at), at / P::kRing - 1));
                    if (!ok) break;
                    if (lane == 0) {
                        if (bytes) mbar_arrive_expect_tx(raw_full(which, at), bytes);
                        else mbar_arrive(raw_full(which, at));
                    }
                    __syncwarp();
                    if (mine)
                        bulk_g2s(base + P::kOffRaw + (which * P::kRing + at % P::kRing) * P::kUnit + lane % kUnitBlocks * kBytes,
                                 (which ? a.L.v : a.L.k) + place * kBytes, kBytes, raw_full(which, at));
                    issued[which] = at + 1;
                }
            }
            if (lane < kBlocks) scales[j % kScaleRing][lane] = make_float2(sc_now.x, __log2f(fmaxf(sc_now.y, 1e-37f)));
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_full(j));
        }
        // nothing of this CTA's is in flight when it leaves
#pragma unroll
        for (int which = 0; which < 2; ++which)
            for (int i = max(0, issued[which] - P::kRing); i < issued[which]; ++i)
                mbar_wait_for(raw_full(which, i), (i / P::kRing) & 1, kDrainWaitNs, &g_columns_timeouts);
    } else {
        // ---- MMA issue: the warp runs converged, one elected lane issues -------------------
        // fp32 accumulator, 128 rows; the second product has both operands MN-major
        const uint32_t i_qk = idesc_f16(128, N, false), i_pv = idesc_f16(128, N, true) | 1u << 15;
        constexpr uint32_t hi_word = desc128_hi(1024);
        const uint32_t q_lo = desc128_lo(base, 16), k_word = desc128_lo(base + P::kOffK, 16);
        const uint32_t v_word = desc128_lo(base + P::kOffV, P::kPanelKV), p_word = desc128_lo(base + P::kOffP, P::kPanelP);
        auto qk = [&](int j) {
            const uint32_t k = k_word + (j % kStages) * (P::kKV / 16);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                mma_ss(tmem + (j & 1) * NT, k + ((s / 4) * P::kPanelKV + (s % 4) * 32) / 16, hi_word,
                       q_lo + ((s / 4) * P::kPanelQ + (s % 4) * 32) / 16, hi_word, i_qk, s > 0);
            commit(s_full(j));
        };
        auto pv = [&](int j) {
            const uint32_t v = v_word + (j % kStages) * (P::kKV / 16), p = p_word + (j & 1) * (P::kP / 16);
#pragma unroll
            for (int o = 0; o < P::kOut; ++o)
#pragma unroll
                for (int s = 0; s < KT / 16; ++s)
                    mma_ss(tmem + P::kO + o * NT, v + (o * 2 * P::kPanelKV + s * (16 * 128)) / 16, hi_word,
                           p + s * (16 * 128) / 16, hi_word, i_pv, j > 0 || s > 0);
        };
        auto all_ok = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)) != 0; };
        bool ok = steps > 0 && all_ok(q_full, 0) && all_ok(k_full(0), 0);
        if (ok) {
            fence_after();
            qk(0);
            commit(k_empty(0));
        }
        for (int j = 0; j < steps && ok; ++j) {
            if (j + 1 < steps) {
                ok = all_ok(k_full(j + 1), (j + 1) / kStages);
                if (!ok) break;
                fence_after();
                qk(j + 1);
                commit(k_empty(j + 1));
            }
            ok = all_ok(v_full(j), j / kStages);
            if (!ok) break;
            fence_after();
            ok = all_ok(p_full(j), j >> 1);
            if (!ok) break;
            fence_after();
            pv(j);
            commit(v_empty(j));
            commit(pv_done(j));
            if (j + 1 == steps) commit(o_full);
        }
        if (steps > 0) {
            // On every exit: what was issued reads shared memory, writes TMEM and arrives on barriers
            // of this CTA.  Let it finish.
            commit(drained);
            mbar_wait_for(drained, 0, kDrainWaitNs, &g_columns_timeouts);
        }
    }
    st_wait();  // a role that gave up may have stores to TMEM on their way
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, P::kCols);
}

// Joins the shares of a unit, in order
template <int D>
__global__ void __launch_bounds__(256)
columns_join_kernel(const AttendArgs a, const Scratch sc)
{
    using P = Plan<D>;
    pdl_wait();
    const int ctile = blockIdx.x % sc.ctiles, head = blockIdx.x / sc.ctiles % a.L.heads, row = blockIdx.x / sc.ctiles / a.L.heads;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int cols = span.n * a.group, c0 = ctile * P::NT, i = blockIdx.y * 256 + threadIdx.x;
    const int c = i / (D / 4), d = i % (D / 4) * 4;
    if (c >= P::NT || c0 + c >= cols) return;
    const Record rec = sc.records[blockIdx.x];
    if (rec.first < 0) return;
    const float *at = sc.pieces + (int64_t)rec.first * P::kPiece;
    float m = kNothing, l = 0.0f;
    for (int k = 0; k < rec.count; ++k) m = fmaxf(m, at[(int64_t)k * P::kPiece + P::NT * D + c]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < rec.count; ++k) {
        const float *p = at + (int64_t)k * P::kPiece;
        const float f = ex2(p[P::NT * D + c] - m);
        const float4 x = *reinterpret_cast<const float4 *>(p + c * D + d);
        o.x = fmaf(x.x, f, o.x), o.y = fmaf(x.y, f, o.y), o.z = fmaf(x.z, f, o.z), o.w = fmaf(x.w, f, o.w);
        l = fmaf(p[P::NT * (D + 1) + c], f, l);
    }
    const int qi = (c0 + c) / a.group, h = (c0 + c) % a.group;
    const int64_t to = (int64_t)(span.lo + qi) * a.q_heads + head * a.group + h;
    const float r = l == 0.0f ? 0.0f : 1.0f / l;
    uint2 v;
    if (a.dtype == BQD_DTYPE_BF16)
        v = make_uint2(Half2Of<__nv_bfloat16>::pack(o.x * r, o.y * r), Half2Of<__nv_bfloat16>::pack(o.z * r, o.w * r));
    else
        v = make_uint2(Half2Of<__half>::pack(o.x * r, o.y * r), Half2Of<__half>::pack(o.z * r, o.w * r));
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

// Pieces that a call may leave: three waves of shares
int most_pieces(const AttendArgs &a) { return a.L.rows > kMaxRows ? 0 : 3 * sm_count(); }

template <int D>
int64_t ctiles_of(const AttendArgs &a)
{
    return ((int64_t)a.max_new * a.group + Plan<D>::NT - 1) / Plan<D>::NT;
}

template <int D>
int64_t workspace_d(const AttendArgs &a)
{
    const int64_t most = most_pieces(a);
    return most == 0 ? 0 : most * Plan<D>::kPiece * (int64_t)sizeof(float) +
                               (int64_t)a.L.rows * a.L.heads * ctiles_of<D>(a) * (int64_t)sizeof(Record);
}

template <int D, int FMT>
int launch_t(const AttendArgs &a, cudaStream_t s)
{
    using P = Plan<D>;
    auto kern = attend_columns_kernel<D, FMT>;
    static bool done[64] = {};
    if (!configure(kern, P::kSmem, done)) return BQD_ERR_CUDA;
    const int64_t ctiles = ctiles_of<D>(a), units = (int64_t)a.L.rows * a.L.heads * ctiles;
    if (units > 0x40000000) return BQD_ERR_INVALID_ARG;
    Scratch sc = {nullptr, nullptr, 0, (int)ctiles};
    if (a.work) {
        sc.most = most_pieces(a);
        sc.pieces = static_cast<float *>(a.work);
        sc.records = reinterpret_cast<Record *>(sc.pieces + (int64_t)sc.most * P::kPiece);
    }
    kern<<<(unsigned)(units + sc.most), kThreadsM, P::kSmem, s>>>(a, sc, sm_count(), opt_wait_ns());
    const cudaError_t launched = cudaGetLastError();
    if (launched != cudaSuccess || sc.most == 0) return cuda_status(launched);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units, (P::NT * D / 4 + 255) / 256);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, columns_join_kernel<D>, a, sc));
}

template <int D>
int launch_f(const AttendArgs &a, cudaStream_t s)
{
    return a.format == BQD_KV_INT8 ? launch_t<D, BQD_KV_INT8>(a, s) : launch_t<D, BQD_KV_E4M3>(a, s);
}

}  // namespace

int64_t columns_workspace(const AttendArgs &a)
{
    return a.head_dim == 64 ? workspace_d<64>(a) : a.head_dim == 128 ? workspace_d<128>(a) : workspace_d<256>(a);
}

int launch_attend_columns(const AttendArgs &a, cudaStream_t s)
{
    return a.head_dim == 64 ? launch_f<64>(a, s) : a.head_dim == 128 ? launch_f<128>(a, s) : launch_f<256>(a, s);
}

int take_columns_timeouts(unsigned int *count)
{
    if (cudaMemcpyFromSymbol(count, g_columns_timeouts, sizeof(*count)) != cudaSuccess) return BQD_ERR_CUDA;
    if (*count) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(g_columns_timeouts, &zero, sizeof(zero)) != cudaSuccess) return BQD_ERR_CUDA;
    }
    return BQD_OK;
}

}  // namespace kv
}  // namespace bqd
