// Attention over a paged 8-bit cache for few queries of a sequence (a decode
// step, the verification of draft tokens).
//
// With c^k, c^v the codes, s^k_b, s^v_b the scales of block b (16 tokens) and
// f = scale log2(e), all in powers of two:
//   x_j = f s^k_b (q . c^k_j) + log2 s^v_b          (j in block b; masked: -inf)
//   p_j = 2^(x_j - m),  m >= max x - 8 per query, grown when a tile passes it
//   O = sum_j p_j c^v_j,   l = sum_b (sum_{j in b} p_j) / s^v_b
//   out = O / l,   lse = ln 2 (m + log2 l)
// Both scales cost nothing per value: K's is folded into the fma that forms
// x, V's into its addend, and l takes one product a block.  p includes V's
// scale, so the fp16 rounding of p is relative to the largest contribution to
// O whatever the spread of the scales; l adds the fp32 values before it.
//
// Layout.  A warp takes 16-token tiles: S = K q^T and O^T = V^T p run as
// mma.sync m16n8k16 with the cache as the 16-row operand, because a group of
// q_heads / kv_heads queries fills 8 columns far better than 16 rows.  The
// contraction index may be permuted freely, so a lane's A fragment of K is 16
// contiguous bytes a chunk of its token row, and of V 16 contiguous bytes of
// each of its four tokens: both operands go from global memory to registers by
// fully used 16-byte loads, and a byte permute that converts to fp16 also
// interleaves two tokens' bytes for V.  K's registers are refilled for the
// next tile as soon as the scores are done, V's after the second product, so
// a tile (32 D bytes) is always in flight for each warp.
// Codes are exact in fp16.  q is scaled by a power of two into its range: every
// bit of a bf16 value stays down to 2^-16 of its row's largest magnitude, and what
// is smaller is off by 2^-25 of it at most, of the order of what the fp32 sum of the
// scores rounds off.  Exponentials, and the logarithm of a scale (it drops out of
// p / l), are the approximate instructions: their relative error of about 2^-22 is
// far below the 2^-11 of the fp16 weights.
//
// Work.  A unit is (row, KV head, column tile of 8 NT queries); its key tiles are
// interleaved over the warps of a CTA, whose partial (m, l, O) are joined through
// shared memory.  Units are spread over the GPU in one of two ways:
//   shares   the tiles of all units, laid end to end, are cut into equal shares,
//            one for each CTA that can be resident (no launch knows the rows'
//            lengths: each CTA adds them up).  What a share cuts off a unit goes
//            to scratch, and a second kernel, launched early, joins the pieces
//            in order.  Lengths of any mix load the GPU evenly: 32 sequences of 0
//            to 8191 tokens 58 us with clusters, 43 us with shares.
//   cluster  the CTAs of a cluster split a unit's keys and join through
//            distributed shared memory: one launch, no scratch.  For calls whose
//            few keys would not fill the shares (latency counts), for batches of
//            more rows than a CTA adds up, and where there is no scratch.
// Both are free of atomics, and give the same bits every time.
//
// Bound by HBM for one column tile: 4 x 130001 tokens, 8 heads of 128, 165 us for
// 1.067 GB (6487 GB/s, 97% of a measured copy; reads 1.000 of the codes).  With
// more columns the conversions of each pass count: two passes of 16 columns (8 x 5
// queries) take 53 us for 116 MB, at 1.6 instructions a cycle of an SM and 12
// warps of 168 registers, of which the head_dim 128 form spills 146 bytes; 32
// columns a pass take 73.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "qmv_common.cuh"

namespace bqd {
namespace kv {
namespace {

using namespace qmvdev;

constexpr int kMaxSplit = 8;      // CTAs of a cluster (16 are placed badly: 130001 tokens, 227 us against 165)
constexpr int kMaxPlanRows = 1024; // rows that a CTA adds up
constexpr int kMinShare = 32;     // tiles of a share at least
constexpr int kUnitCost = 24;     // what a unit costs beside its tiles (q, the first loads, the join), in tiles:
                                  // 32 mixed sequences 81 us with 0, 58 with 8, 45 with 24, 47 with 48
constexpr float kGrow = 8.0f;   // a reference m is replaced when x passes it by this much
// m of a column that has seen nothing: below every score, and finite, so that
// neither x - m (x = -inf where masked) nor a difference of two m is NaN
constexpr float kNothing = -3.0e38f;

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t local_addr, uint32_t rank)
{
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t local_addr, uint32_t rank)
{
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local_addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

// Warps and resident CTAs follow the registers: K and V words, O and q take
// D / 4 + 8 NT (D / 16) + ...: 128 a thread for 8 columns of D <= 128.
template <int D, int NT>
struct Tile {
    static constexpr int kWarps = NT > 1 ? 4 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kResident = D == 256 ? 1 : NT > 1 ? 3 : 2;  // CTAs of an SM
    static constexpr int kCols = 8 * NT;
    static constexpr int kPitch = D + 4;  // floats of a column in shared memory
    // floats: per-warp partials, then the CTA's joined partial and its m, l
    static constexpr int kWarpFloats = kCols * kPitch;
    static constexpr size_t kFloats = (size_t)kWarps * kWarpFloats + 2 * kWarps * kCols + (size_t)kWarpFloats + 2 * kCols;
    static constexpr size_t kSmem = sizeof(float) * kFloats;
    // scratch of a piece: O [cols][D], m [cols], l [cols]
    static constexpr int kPiece = kCols * D + 2 * kCols;
};

// The first piece of a unit that goes on in later shares
struct Cut {
    int lo, cols, c0, head;  // first query of its row, columns of the row and before the unit's
    int last;                // the share with its last piece; -1: no unit is cut
};

struct Shares {
    float *pieces;  // [shares][2][kPiece]: what began earlier, what goes on
    Cut *cuts;      // [shares]
    int count;      // 0: clusters
};

// What the queries of a column tile see
struct View {
    Span span;
    int L, cols, c0, p_min, p_max, lo, hi;
    __device__ __forceinline__ View(const AttendArgs &a, int row, int ctile, int kCols)
        : span(a.starts, row, a.tokens, a.max_new)
    {
        L = a.L.length(row);
        cols = span.n * a.group;  // columns: query-major, then head of the group
        c0 = ctile * kCols;
        const int i_min = c0 / a.group, i_max = (min(c0 + kCols, cols) - 1) / a.group;
        p_min = L - span.rest + i_min;
        p_max = L - span.rest + i_max;
        hi = max(0, p_max + 1);
        lo = a.window > 0 ? max(0, p_min + 1 - a.window) : 0;
    }
};

// Tiles of a row that any of its queries sees: [lo, lo + n) (n >= 1: a row that
// sees nothing has one, so that its zeros are written)
struct RowTiles {
    int lo, n, ctiles;
    __device__ __forceinline__ RowTiles(const AttendArgs &a, int row, int kCols)
    {
        const Span span(a.starts, row, a.tokens, a.max_new);
        const int L = a.L.length(row);
        lo = a.window > 0 ? max(0, L - span.rest + 1 - a.window) >> 4 : 0;
        n = max(1, ((L + 15) >> 4) - lo);
        ctiles = (span.n * a.group + kCols - 1) / kCols;
    }
};

template <typename T, int D>
__device__ __forceinline__ void finish(const AttendArgs &a, int lo, int cols, int c0, int head, int col, int d, float4 o,
                                       float mm, float ll)
{
    using H = Half2Of<T>;
    const int c = c0 + col;
    if (c >= cols) return;
    const int token = lo + c / a.group, hq = head * a.group + c % a.group;
    const float r = ll == 0.0f ? 0.0f : 1.0f / ll;
    T *at = static_cast<T *>(a.out) + ((int64_t)token * a.q_heads + hq) * D + d;
    *reinterpret_cast<uint2 *>(at) = make_uint2(H::pack(o.x * r, o.y * r), H::pack(o.z * r, o.w * r));
    if (a.lse && d == 0)
        a.lse[(int64_t)token * a.q_heads + hq] = ll == 0.0f ? -INFINITY : 0.69314718055994531f * (mm + log2f(ll));
}

// Columns of a unit against its tiles [j0, j1): each warp takes every kWarps-th.
// The joined (o, m, l) of each quad of dims goes to emit(col, d, o, m, l).
template <typename T, int D, int FMT, int NT, typename Emit>
__device__ __forceinline__ void unit_tiles(const AttendArgs &a, const View &vw_, int row, int head, int j0, int j1,
                                           float *smem, Emit emit)
{
    using C = Code<FMT>;
    using H = Half2Of<T>;
    using TL = Tile<D, NT>;
    constexpr int kWarpsD = TL::kWarps;
    constexpr int KW = D / 16;   // 32-bit words of a lane's part of one K row
    constexpr int VW = D / 32;   // words of a lane's part of one V token
    constexpr int KS = D / 16;   // k16 steps of S, m16 tiles of O^T
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const Span &span = vw_.span;
    const int cols = vw_.cols, c0 = vw_.c0, L = vw_.L, p_min = vw_.p_min, p_max = vw_.p_max;

    // the first tile is on its way while q is prepared
    uint32_t kw[2][KW], vw[4][VW];
    float ksc = 0.0f, vsc = 1.0f;
    auto load_k = [&](int64_t blk) {
        const uint8_t *at = a.L.k + blk * (kBlock * D) + 16 * t;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint4 v = ld_stream_v4(at + (g + 8 * r) * D + 64 * j);
                kw[r][4 * j] = v.x, kw[r][4 * j + 1] = v.y, kw[r][4 * j + 2] = v.z, kw[r][4 * j + 3] = v.w;
            }
        ksc = __ldg(a.L.ks + blk);
    };
    auto load_v = [&](int64_t blk) {
        const uint8_t *at = a.L.v + blk * (kBlock * D);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint8_t *tok = at + (2 * t + (r & 1) + 8 * (r >> 1)) * D;
            if constexpr (D == 64) {
                const uint2 v = ld_stream_v2(tok + 8 * g);
                vw[r][0] = v.x, vw[r][1] = v.y;
            } else {
#pragma unroll
                for (int j = 0; j < D / 128; ++j) {
                    const uint4 v = ld_stream_v4(tok + 16 * (g + 8 * j));
                    vw[r][4 * j] = v.x, vw[r][4 * j + 1] = v.y, vw[r][4 * j + 2] = v.z, vw[r][4 * j + 3] = v.w;
                }
            }
        }
        vsc = __ldg(a.L.vs + blk);
    };

    int j = j0 + warp;
    int64_t blk = 0;
    int next_page = 0;  // as listed, of the tile after the next
    if (j < j1) {
        blk = a.L.block_of(row, head, j << 4);
        load_k(blk);
        load_v(blk);
        if (j + kWarpsD < j1) next_page = a.L.listed(row, (j + kWarpsD) << 4);
    }
    // q: column n*8 + g, the dims of this lane's K chunks, scaled by 2^-e
    uint32_t qf[NT][KS][2];
    float cs[NT][2];             // f 2^e of columns n*8 + 2t, + 2t + 1
    int pos[NT][2];              // their positions (-1: nothing)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int c = c0 + n * 8 + g;
        uint32_t w[2 * KW];
        if (c < cols) {
            const T *q = static_cast<const T *>(a.q) + (int64_t)(span.lo + c / a.group) * a.q_token +
                         (int64_t)(head * a.group + c % a.group) * a.q_head;
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const T *at = q + 16 * (t + 4 * j);
                if (a.q_vec) {
                    const uint4 v0 = __ldg(reinterpret_cast<const uint4 *>(at));
                    const uint4 v1 = __ldg(reinterpret_cast<const uint4 *>(at) + 1);
                    w[8 * j] = v0.x, w[8 * j + 1] = v0.y, w[8 * j + 2] = v0.z, w[8 * j + 3] = v0.w;
                    w[8 * j + 4] = v1.x, w[8 * j + 5] = v1.y, w[8 * j + 6] = v1.z, w[8 * j + 7] = v1.w;
                } else {
                    const unsigned short *u = reinterpret_cast<const unsigned short *>(at);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[8 * j + e] = (uint32_t)__ldg(u + 2 * e) | ((uint32_t)__ldg(u + 2 * e + 1) << 16);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 2 * KW; ++e) w[e] = 0;
        }
        uint32_t mx = 0;
#pragma unroll
        for (int e = 0; e < 2 * KW; ++e) mx = __vmaxu2(mx, w[e] & 0x7FFF7FFFu);
        uint32_t top = max(mx & 0xFFFFu, mx >> 16);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent of the largest |q|; 0 for an all-zero row and for infinities and NaN
        int e = 0;
        if (top != 0 && top < H::kInf) e = max(-100, min(126, (int)((__float_as_uint(H::f1(top)) >> 23) & 0xFF) - 127));
        const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float2 f = H::f2(w[2 * k + h]);
                qf[n][k][h] = Half2Of<__half>::pack(f.x * down, f.y * down);
            }
        const float mine = a.scale * up;
        cs[n][0] = __shfl_sync(0xffffffffu, mine, 8 * t);
        cs[n][1] = __shfl_sync(0xffffffffu, mine, 8 * t + 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int cc = c0 + n * 8 + 2 * t + h;
            pos[n][h] = cc < cols ? L - span.rest + cc / a.group : -1;
        }
    }

    float acc[NT][KS][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = kNothing;
        l[n][0] = l[n][1] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) acc[n][k][0] = acc[n][k][1] = acc[n][k][2] = acc[n][k][3] = 0.0f;
    }

    for (; j < j1; j += kWarpsD) {
        const int t0 = j << 4;
        const bool more = j + kWarpsD < j1;
        int64_t next = 0;
        if (more) {
            next = a.L.block_at((unsigned)next_page < (unsigned)a.L.pages ? next_page : 0, head, (j + kWarpsD) << 4);
            if (j + 2 * kWarpsD < j1) next_page = a.L.listed(row, (j + 2 * kWarpsD) << 4);
        }
        // scores of 16 tokens
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const uint32_t u0 = C::ready(kw[0][k]), u1 = C::ready(kw[1][k]);
            const uint32_t a0 = C::template pair<0>(u0), a1 = C::template pair<0>(u1);
            const uint32_t a2 = C::template pair<1>(u0), a3 = C::template pair<1>(u1);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(s[n], a0, a1, a2, a3, qf[n][k][0], qf[n][k][1]);
        }
        const float kscale = ksc, vscale = vsc;
        if (more) load_k(next);

        // rv from lv: what lg2 is off by drops out of p / l
        const float lv = lg2(fmaxf(vscale, 1e-37f)), rv = ex2(-lv);
        const bool whole = t0 + 15 <= p_min && (a.window == 0 || t0 > p_max - a.window);
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float f0 = cs[n][0] * kscale, f1 = cs[n][1] * kscale;
            s[n][0] = fmaf(s[n][0], f0, lv), s[n][1] = fmaf(s[n][1], f1, lv);
            s[n][2] = fmaf(s[n][2], f0, lv), s[n][3] = fmaf(s[n][3], f1, lv);
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int tok = t0 + g + 8 * (e >> 1), pp = pos[n][e & 1];
                    if (tok > pp || (a.window > 0 && tok <= pp - a.window)) s[n][e] = -INFINITY;
                }
            }
            grow |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kGrow || fmaxf(s[n][1], s[n][3]) > m[n][1] + kGrow;
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float n0 = fmaxf(s[n][0], s[n][2]), n1 = fmaxf(s[n][1], s[n][3]);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, o));
                    n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, o));
                }
                n0 = fmaxf(n0, m[n][0]), n1 = fmaxf(n1, m[n][1]);
                const float r0 = ex2(m[n][0] - n0), r1 = ex2(m[n][1] - n1);
                m[n][0] = n0, m[n][1] = n1;
                l[n][0] *= r0, l[n][1] *= r1;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    acc[n][k][0] *= r0, acc[n][k][2] *= r0;
                    acc[n][k][1] *= r1, acc[n][k][3] *= r1;
                }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float e0 = ex2(s[n][0] - m[n][0]), e1 = ex2(s[n][1] - m[n][1]);
            const float e2 = ex2(s[n][2] - m[n][0]), e3 = ex2(s[n][3] - m[n][1]);
            l[n][0] = fmaf(e0 + e2, rv, l[n][0]);
            l[n][1] = fmaf(e1 + e3, rv, l[n][1]);
            pb[n][0] = transpose8x8(Half2Of<__half>::pack(e0, e1));
            pb[n][1] = transpose8x8(Half2Of<__half>::pack(e2, e3));
        }
        if (FMT == BQD_KV_E4M3 && t0 + 15 >= L) {
            // bytes past the row's end may be anything, NaN among them, and 0 * NaN is NaN
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (t0 + 2 * t + (r & 1) + 8 * (r >> 1) >= L) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) vw[r][w] = 0;
                }
        }
        // O^T += V^T p: word w of the lane's tokens gives m tiles 2w, 2w + 1
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            const uint32_t v0 = C::ready(vw[0][w]), v1 = C::ready(vw[1][w]);
            const uint32_t v2 = C::ready(vw[2][w]), v3 = C::ready(vw[3][w]);
            const uint32_t a01 = __byte_perm(v0, v1, 0x5140), b01 = __byte_perm(v0, v1, 0x7362);
            const uint32_t a23 = __byte_perm(v2, v3, 0x5140), b23 = __byte_perm(v2, v3, 0x7362);
            const uint32_t x0 = C::template pair<0>(a01), x1 = C::template pair<1>(a01);
            const uint32_t x2 = C::template pair<0>(a23), x3 = C::template pair<1>(a23);
            const uint32_t y0 = C::template pair<0>(b01), y1 = C::template pair<1>(b01);
            const uint32_t y2 = C::template pair<0>(b23), y3 = C::template pair<1>(b23);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816(acc[n][2 * w], x0, x1, x2, x3, pb[n][0], pb[n][1]);
                mma16816(acc[n][2 * w + 1], y0, y1, y2, y3, pb[n][0], pb[n][1]);
            }
        }
        if (more) load_v(next);
    }

    // ---- join the warps --------------------------------------------------------
    float *part = smem;                                  // [warp][col][kPitch]
    float *wm = part + kWarpsD * TL::kWarpFloats;        // [warp][col]
    float *wl = wm + kWarpsD * TL::kCols;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float sum = l[n][h];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            const int col = n * 8 + 2 * t + h;
            if (g == 0) {
                wm[warp * TL::kCols + col] = m[n][h];
                wl[warp * TL::kCols + col] = sum;
            }
            // m tile i holds dims base + 2i, + 1 (rows g and g + 8)
            float *at = part + warp * TL::kWarpFloats + col * TL::kPitch;
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                const int d = D == 64 ? 8 * g + 2 * k : 16 * (g + 8 * (k / 8)) + 2 * (k % 8);
                *reinterpret_cast<float4 *>(at + d) =
                    make_float4(acc[n][k][h], acc[n][k][2 + h], acc[n][k + 1][h], acc[n][k + 1][2 + h]);
            }
        }
    }
    __syncthreads();
    constexpr int kQuads = TL::kCols * D / 4;
    for (int i = threadIdx.x; i < kQuads; i += kWarpsD * 32) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float mm = kNothing;
#pragma unroll
        for (int w = 0; w < kWarpsD; ++w) mm = fmaxf(mm, wm[w * TL::kCols + col]);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarpsD; ++w) {
            const float r = ex2(wm[w * TL::kCols + col] - mm);
            const float4 v = *reinterpret_cast<const float4 *>(part + w * TL::kWarpFloats + col * TL::kPitch + d);
            o.x = fmaf(v.x, r, o.x), o.y = fmaf(v.y, r, o.y), o.z = fmaf(v.z, r, o.z), o.w = fmaf(v.w, r, o.w);
            ll = fmaf(wl[w * TL::kCols + col], r, ll);
        }
        emit(col, d, o, mm, ll);
    }
    __syncthreads();  // the partials' place may be written again
}

template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(Tile<D, NT>::kThreads, Tile<D, NT>::kResident)
attend_cluster_kernel(const AttendArgs a, int S)
{
    using TL = Tile<D, NT>;
    extern __shared__ __align__(16) float smem[];
    const int rank = S > 1 ? (int)cluster_ctarank() : 0;
    const int ctile = blockIdx.x / S, head = blockIdx.y, row = blockIdx.z;
    const View v(a, row, ctile, TL::kCols);
    if (v.c0 >= v.cols) return;              // the whole cluster leaves
    // this CTA's tiles of 16 tokens
    const int tile_lo = v.lo >> 4, tiles = max(0, ((v.hi + 15) >> 4) - tile_lo);
    const int j0 = tile_lo + (int)((int64_t)tiles * rank / S), j1 = tile_lo + (int)((int64_t)tiles * (rank + 1) / S);
    float *joined = smem + TL::kWarps * (TL::kWarpFloats + 2 * TL::kCols);  // [col][kPitch]
    float *jm = joined + TL::kWarpFloats, *jl = jm + TL::kCols;
    unit_tiles<T, D, FMT, NT>(a, v, row, head, j0, j1, smem, [&](int col, int d, float4 o, float mm, float ll) {
        if (S == 1) {
            finish<T, D>(a, v.span.lo, v.cols, v.c0, head, col, d, o, mm, ll);
        } else {
            *reinterpret_cast<float4 *>(joined + col * TL::kPitch + d) = o;
            if (d == 0) jm[col] = mm, jl[col] = ll;
        }
    });
    if (S == 1) return;
    // rank r finishes the quads r, r + S, ...
    cluster_sync();
    constexpr int kQuads = TL::kCols * D / 4;
    for (int i = threadIdx.x * S + rank; i < kQuads; i += TL::kThreads * S) {
        const int col = i / (D / 4), d = (i % (D / 4)) * 4;
        float mm = kNothing;
        for (int r = 0; r < S; ++r) mm = fmaxf(mm, ld_cluster_f32(smem_addr(jm + col), r));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float ll = 0.0f;
        for (int r = 0; r < S; ++r) {
            const float f = ex2(ld_cluster_f32(smem_addr(jm + col), r) - mm);
            const float4 x = ld_cluster_f32x4(smem_addr(joined + col * TL::kPitch + d), r);
            o.x = fmaf(x.x, f, o.x), o.y = fmaf(x.y, f, o.y), o.z = fmaf(x.z, f, o.z), o.w = fmaf(x.w, f, o.w);
            ll = fmaf(ld_cluster_f32(smem_addr(jl + col), r), f, ll);
        }
        finish<T, D>(a, v.span.lo, v.cols, v.c0, head, col, d, o, mm, ll);
    }
    cluster_sync();  // no CTA leaves while another reads its shared memory
}

template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(Tile<D, NT>::kThreads, Tile<D, NT>::kResident)
attend_shares_kernel(const AttendArgs a, const Shares sh)
{
    using TL = Tile<D, NT>;
    extern __shared__ __align__(16) float smem[];
    __shared__ int64_t before[kMaxPlanRows + 1];  // tiles of all units of the rows before
    __shared__ int64_t warp_sums[TL::kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, share = blockIdx.x;
    // the rows' tiles and their sums: a thread takes consecutive rows
    const int rows = a.L.rows, each = (rows + TL::kThreads - 1) / TL::kThreads;
    int64_t mine = 0;
    for (int i = 0; i < each; ++i) {
        const int r = tid * each + i;
        if (r >= rows) break;
        const RowTiles rt(a, r, TL::kCols);
        const int64_t w = (int64_t)(rt.n + kUnitCost) * rt.ctiles * a.L.heads;
        before[r] = w;
        mine += w;
    }
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int64_t total = 0, base = 0;
    for (int w = 0; w < TL::kWarps; ++w) {
        if (w == warp) base = total;
        total += warp_sums[w];
    }
    int64_t at = base + x - mine;
    for (int i = 0; i < each; ++i) {
        const int r = tid * each + i;
        if (r >= rows) break;
        const int64_t w = before[r];
        before[r] = at;
        at += w;
    }
    if (tid == 0) before[rows] = total;
    __syncthreads();
    const int64_t per = max((int64_t)kMinShare, (total + sh.count - 1) / sh.count);
    int64_t pos = min(total, share * per);
    const int64_t end = min(total, pos + per);
    bool cut = false;
    int row = 0;
    while (pos < end) {
        {
            int lo = row, hi = rows - 1;  // the last row with before <= pos
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (before[mid] <= pos) lo = mid;
                else hi = mid - 1;
            }
            row = lo;
        }
        const RowTiles rt(a, row, TL::kCols);
        const int64_t off = pos - before[row];
        const int cost = rt.n + kUnitCost;  // the first kUnitCost of a unit stand for no tile
        const int unit = (int)(off / cost), j = (int)(off - (int64_t)unit * cost);
        const int head = unit % a.L.heads, ctile = unit / a.L.heads;
        const int stop = (int)min((int64_t)cost, j + (end - pos));
        const View v(a, row, ctile, TL::kCols);
        const bool starts = j == 0, ends = stop == cost;
        float *piece = sh.pieces + ((int64_t)share * 2 + (starts ? 1 : 0)) * TL::kPiece;
        // tiles that this column tile sees of them
        const int j0 = max(rt.lo + max(0, j - kUnitCost), v.lo >> 4);
        const int j1 = min(rt.lo + max(0, stop - kUnitCost), (v.hi + 15) >> 4);
        unit_tiles<T, D, FMT, NT>(a, v, row, head, j0, j1, smem, [&](int col, int d, float4 o, float mm, float ll) {
            if (starts && ends) {
                finish<T, D>(a, v.span.lo, v.cols, v.c0, head, col, d, o, mm, ll);
            } else {
                *reinterpret_cast<float4 *>(piece + col * D + d) = o;
                if (d == 0) {
                    piece[TL::kCols * D + col] = mm;
                    piece[TL::kCols * (D + 1) + col] = ll;
                }
            }
        });
        if (starts && !ends) {
            cut = true;
            if (tid == 0) sh.cuts[share] = Cut{v.span.lo, v.cols, v.c0, head, (int)((pos - j + cost - 1) / per)};
        }
        pos += stop - j;
    }
    if (!cut && tid == 0) sh.cuts[share] = Cut{0, 0, 0, 0, -1};
    pdl_launch_dependents();
}

// Joins the pieces of the unit that goes on from share blockIdx.x, in order.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(256)
attend_join_kernel(const AttendArgs a, const Shares sh)
{
    using TL = Tile<D, NT>;
    pdl_wait();
    const int share = blockIdx.x;
    const Cut cut = sh.cuts[share];
    const int i = blockIdx.y * 256 + threadIdx.x, col = i / (D / 4), d = (i % (D / 4)) * 4;
    if (cut.last < 0 || col >= TL::kCols || cut.c0 + col >= cut.cols) return;
    // piece 0 is what goes on, the others began earlier; eight at a time are on their way
    const int n = cut.last - share + 1;
    float mm = kNothing, ll = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kFlight = 8;
    for (int k0 = 0; k0 < n; k0 += kFlight) {
        float mk[kFlight], lk[kFlight];
        float4 x[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const int s = k0 + k;
            mk[k] = kNothing, lk[k] = 0.0f, x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s < n) {
                const float *p = sh.pieces + ((int64_t)(share + s) * 2 + (s ? 0 : 1)) * TL::kPiece;
                mk[k] = p[TL::kCols * D + col];
                lk[k] = p[TL::kCols * (D + 1) + col];
                x[k] = *reinterpret_cast<const float4 *>(p + col * D + d);
            }
        }
        float top = mm;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) top = fmaxf(top, mk[k]);
        const float r = ex2(mm - top);
        mm = top;
        o.x *= r, o.y *= r, o.z *= r, o.w *= r, ll *= r;
#pragma unroll
        for (int k = 0; k < kFlight; ++k) {
            const float f = ex2(mk[k] - mm);
            o.x = fmaf(x[k].x, f, o.x), o.y = fmaf(x[k].y, f, o.y), o.z = fmaf(x[k].z, f, o.z), o.w = fmaf(x[k].w, f, o.w);
            ll = fmaf(lk[k], f, ll);
        }
    }
    finish<T, D>(a, cut.lo, cut.cols, cut.c0, cut.head, col, d, o, mm, ll);
}

// Makes a kernel ready on the current device, once per device.
template <typename K>
bool configure(K kern, size_t smem, bool (&done)[64])
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < 64 && done[dev]) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return true;
}

// Shares of a call, or 0 where it takes clusters: with what the planned lengths
// can come to, each share keeps kMinShare tiles for each resident CTA.
template <int D, int NT>
int shares_of(const AttendArgs &a)
{
    using TL = Tile<D, NT>;
    if (a.L.rows > kMaxPlanRows) return 0;
    const int64_t ctiles = ((int64_t)a.max_new * a.group + TL::kCols - 1) / TL::kCols;
    const int64_t span = a.window > 0 ? std::min<int64_t>(a.max_len, (int64_t)a.window + a.max_new) : a.max_len;
    const int64_t most = ctiles * a.L.heads * a.L.rows * ((span + 15) / 16);
    const int slots = sm_count() * TL::kResident;
    return most >= (int64_t)slots * kMinShare ? slots : 0;
}

template <int D, int NT>
int64_t shares_bytes(int shares)
{
    return (int64_t)shares * (2 * Tile<D, NT>::kPiece * (int64_t)sizeof(float) + (int64_t)sizeof(Cut));
}

template <typename T, int D, int FMT, int NT>
int launch_t(const AttendArgs &a, cudaStream_t s)
{
    using TL = Tile<D, NT>;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(TL::kThreads);
    cfg.dynamicSmemBytes = TL::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    cfg.attrs = attr;
    const int shares = a.work ? shares_of<D, NT>(a) : 0;
    if (shares > 0) {
        auto kern = attend_shares_kernel<T, D, FMT, NT>;
        static bool done[64] = {};
        if (!configure(kern, TL::kSmem, done)) return BQD_ERR_CUDA;
        Shares sh;
        sh.pieces = static_cast<float *>(a.work);
        sh.cuts = reinterpret_cast<Cut *>(sh.pieces + (int64_t)shares * 2 * TL::kPiece);
        sh.count = shares;
        cfg.gridDim = dim3((unsigned)shares);
        if (cudaLaunchKernelEx(&cfg, kern, a, sh) != cudaSuccess) return BQD_ERR_CUDA;
        cfg.gridDim = dim3((unsigned)shares, (TL::kCols * D / 4 + 255) / 256);
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 1;
        return cuda_status(cudaLaunchKernelEx(&cfg, attend_join_kernel<T, D, NT>, a, sh));
    }
    auto kern = attend_cluster_kernel<T, D, FMT, NT>;
    static bool done[64] = {};
    if (!configure(kern, TL::kSmem, done)) return BQD_ERR_CUDA;
    const int64_t ctiles = ((int64_t)a.max_new * a.group + TL::kCols - 1) / TL::kCols;
    const int64_t units = ctiles * a.L.heads * a.L.rows;
    // split the keys until there are two CTAs an SM, as long as each warp
    // keeps a tile
    int S = 1;
    while (S < kMaxSplit && units * S < 2 * sm_count() && a.max_len >= kBlock * TL::kWarps * 2 * S) S *= 2;
    if (ctiles * S > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    cfg.gridDim = dim3((unsigned)(ctiles * S), (unsigned)a.L.heads, (unsigned)a.L.rows);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, a, S));
}

// Column tiles of 16 where there are more than 8 columns (D = 256 has no registers for them)
bool wide(const AttendArgs &a) { return (int64_t)a.max_new * a.group > 8; }

template <typename T, int FMT>
int launch_d(const AttendArgs &a, cudaStream_t s)
{
    if (a.head_dim == 256) return launch_t<T, 256, FMT, 1>(a, s);
    if (a.head_dim == 64) return wide(a) ? launch_t<T, 64, FMT, 2>(a, s) : launch_t<T, 64, FMT, 1>(a, s);
    return wide(a) ? launch_t<T, 128, FMT, 2>(a, s) : launch_t<T, 128, FMT, 1>(a, s);
}

}  // namespace

int64_t decode_workspace(const AttendArgs &a)
{
    if (a.head_dim == 256) return shares_bytes<256, 1>(shares_of<256, 1>(a));
    if (a.head_dim == 64)
        return wide(a) ? shares_bytes<64, 2>(shares_of<64, 2>(a)) : shares_bytes<64, 1>(shares_of<64, 1>(a));
    return wide(a) ? shares_bytes<128, 2>(shares_of<128, 2>(a)) : shares_bytes<128, 1>(shares_of<128, 1>(a));
}

int launch_attend_decode(const AttendArgs &a, cudaStream_t s)
{
    if (a.format == BQD_KV_INT8)
        return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_INT8>(a, s)
                                        : launch_d<__nv_bfloat16, BQD_KV_INT8>(a, s);
    return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_E4M3>(a, s)
                                    : launch_d<__nv_bfloat16, BQD_KV_E4M3>(a, s);
}

}  // namespace kv
}  // namespace bqd
