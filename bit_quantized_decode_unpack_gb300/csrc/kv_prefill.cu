// Attention over a paged 8-bit cache for many queries of a sequence (prefill
// chunks): both products on the 5th-generation tensor cores.
//
// The mathematics is that of the few-query kernel (kv_attend.cu): with f the
// score scale times log2(e) and s^k_b, s^v_b the scales of 16-token block b,
//   x_ij = f s^k_b (q_i . c^k_j) + log2 s^v_b,   p_ij = 2^(x_ij - m_i),
//   O_i = sum_j p_ij c^v_j,   l_i = sum_b (sum_{j in b} p_ij) / s^v_b,
//   out = O / l,   lse = ln 2 (m + log2 l),
// with m_i replaced only when a tile's maximum passes it by 8.
//
// Rows of a tile are (query, head of the group) pairs, so a tile of 128 rows
// reads each K and V code once for the whole group.  A CTA owns two tiles of
// 128 rows (one for head_dim 256, and where there are no more rows) and walks
// the keys in steps of KT.  Roles:
//   warps 0-3, 4-7   softmax of tile 0 / 1: one thread a row.  S is read from
//                    TMEM twice (maximum, then exponentials), P written over it
//                    as fp16 in TMEM, O rescaled in TMEM when m is replaced
//   warps 8-11       cache codes to fp16: 16-byte loads of codes for the next
//                    step are in flight while this step's are converted into
//                    128-byte-swizzled tiles.  K and V tiles have the same
//                    layout ([64-dim panel][key] rows of 128 bytes): K is a
//                    K-major operand of S = Q K^T, V an MN-major one of O = P V,
//                    so V needs no transpose
//   warp 12          TMEM, and one thread that issues every MMA
// With two tiles the tensor cores work on one while the other's softmax runs;
// with one tile S alternates between two TMEM buffers, so that S of the next
// step is computed during the softmax of this one.
// Every wait is bounded; on expiry a role stops, what it issued is drained,
// TMEM is freed, and bqd_device_status reports it.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "qmv_common.cuh"
#include "tc05.cuh"

namespace bqd {
namespace kv {
namespace {

using namespace qmvdev;
using namespace tc05;

constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kConvThreads = kConvWarps * 32;
constexpr int kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kThreadsF = (kMmaWarp + 1) * 32;
constexpr int kStages = 2;
constexpr int kScaleRing = 4;  // steps whose scales are kept: a slot is written again only after
                               // both softmaxes of the step four before have finished
constexpr float kGrow = 8.0f;

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
    static constexpr size_t kSmem = 1024 + kOffEnd;
    // TMEM columns
    static constexpr uint32_t kS1 = KT, kO0 = 256, kO1 = 256 + D, kCols = 512;
};

struct Scales {
    float k[8], lv[8], rv[8];
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kThreadsF, 1)
attend_prefill_kernel(const AttendArgs a, unsigned long long wait_ns)
{
    using P = Plan<D>;
    using C = Code<FMT>;
    using H = Half2Of<T>;
    constexpr int KT = P::KT;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[4 * kStages + 9];
    __shared__ Scales scales[kScaleRing];
    __shared__ uint32_t tmem_at;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int head = blockIdx.y, row = blockIdx.z;
    const Span span(a.starts, row, a.tokens, a.max_new);
    const int rows = span.n * a.group;
    const int r0 = (int)(gridDim.x - 1 - blockIdx.x) * P::kRows;  // the last queries see most keys: first
    if (r0 >= rows) return;
    const int L = a.L.length(row);
    const int tiles = min(P::kTiles, (rows - r0 + 127) / 128);
    const int i_min = r0 / a.group, i_max = (min(r0 + P::kRows, rows) - 1) / a.group;
    const int p_first = L - span.n;  // position of query 0
    const int hi = max(0, p_first + i_max + 1);
    const int lo = a.window > 0 ? max(0, p_first + i_min + 1 - a.window) : 0;
    const int k_lo = lo / KT * KT;
    const int steps = hi > k_lo ? (hi - k_lo + KT - 1) / KT : 0;

    auto bar = [&](int i) { return smem_addr(&bars[i]); };
    auto k_full = [&](int j) { return bar(j % kStages); };
    auto k_empty = [&](int j) { return bar(kStages + j % kStages); };
    auto v_full = [&](int j) { return bar(2 * kStages + j % kStages); };
    auto v_empty = [&](int j) { return bar(3 * kStages + j % kStages); };
    const uint32_t q_full = bar(4 * kStages);
    auto s_full = [&](int w) { return bar(4 * kStages + 1 + w); };
    auto p_full = [&](int w) { return bar(4 * kStages + 3 + w); };
    auto o_full = [&](int w) { return bar(4 * kStages + 5 + w); };
    const uint32_t pv_done = bar(4 * kStages + 7), drained = bar(4 * kStages + 8);

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(k_full(i), kConvThreads);
                mbar_init(k_empty(i), 1);
                mbar_init(v_full(i), kConvThreads);
                mbar_init(v_empty(i), 1);
            }
            mbar_init(q_full, 128 * tiles);
            for (int w = 0; w < 2; ++w) {
                mbar_init(s_full(w), 1);
                mbar_init(p_full(w), 128);
                mbar_init(o_full(w), 1);
            }
            mbar_init(pv_done, 1);
            mbar_init(drained, 1);
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
            // ---- q: scaled by 2^-e into fp16 (e of the row's largest magnitude) ----
            const bool real = r < rows;
            const int token = span.lo + (real ? r / a.group : 0);
            const int hq = head * a.group + (real ? r % a.group : 0);
            const int pos = real ? p_first + r / a.group : -1;
            const T *q = static_cast<const T *>(a.q) + (int64_t)token * a.q_token + (int64_t)hq * a.q_head;
            const uint32_t q_at = base + w * (P::kPanels * P::kPanelQ) + trow * 128;
            uint32_t top = 0;
            auto load = [&](int u) {  // dims 8u .. 8u + 7
                uint4 v = make_uint4(0, 0, 0, 0);
                if (real) {
                    if (a.q_vec) {
                        v = __ldg(reinterpret_cast<const uint4 *>(q) + u);
                    } else {
                        const unsigned short *s = reinterpret_cast<const unsigned short *>(q) + 8 * u;
                        uint32_t x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = (uint32_t)__ldg(s + 2 * i) | ((uint32_t)__ldg(s + 2 * i + 1) << 16);
                        v = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
                return v;
            };
            uint32_t mx = 0;
#pragma unroll 8
            for (int u = 0; u < D / 8; ++u) {
                const uint4 v = load(u);
                mx = __vmaxu2(__vmaxu2(mx, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
                mx = __vmaxu2(__vmaxu2(mx, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
            }
            top = max(mx & 0xFFFFu, mx >> 16);
            int e = 0;
            if (top != 0 && top < H::kInf)
                e = max(-100, min(126, (int)((__float_as_uint(H::f1(top)) >> 23) & 0xFF) - 127));
            // the sign of the scale goes with q, so that a larger product is a larger score
            const float down = copysignf(__uint_as_float((uint32_t)(127 - e) << 23), a.scale);
            const float cs = fabsf(a.scale) * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 8
            for (int u = 0; u < D / 8; ++u) {
                const uint4 v = load(u);
                uint32_t h[4];
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = H::f2(x[i]);
                    h[i] = Half2Of<__half>::pack(f.x * down, f.y * down);
                }
                const uint32_t at = q_at + (u >> 3) * P::kPanelQ + (((u & 7) ^ (trow & 7)) << 4);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                             "r"(h[3])
                             : "memory");
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);

            // ---- steps ------------------------------------------------------------
            const int p_low = p_first + (r0 + w * 128) / a.group;                               // positions of
            const int p_high = p_first + (min(r0 + w * 128 + 128, rows) - 1) / a.group;          // the tile's rows
            const uint32_t o_at = tmem + lanes + (w ? P::kO1 : P::kO0);
            float m = -INFINITY, l = 0.0f;
            bool ok = true;
            for (int j = 0; j < steps; ++j) {
                const int slot = pair ? w : j & 1;
                const uint32_t s_at = tmem + lanes + (slot ? P::kS1 : 0);
                ok = wait(s_full(slot), pair ? j : j >> 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                fence_after();
                const int k0 = k_lo + j * KT;
                const Scales &sc = scales[j % kScaleRing];
                const bool whole = k0 + KT - 1 <= p_low && (a.window == 0 || k0 > p_high - a.window);
                const int last = pos - k0;                                          // columns <= last and
                const int first = a.window > 0 ? pos - a.window - k0 : -1;          // > first are seen
                // maximum
                float mt = -INFINITY;
#pragma unroll
                for (int c = 0; c < KT / 32; ++c) {
                    uint32_t s[32];
                    ld32(s_at + 32 * c, s);
                    ld_wait(s);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float x = -INFINITY;
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) x = fmaxf(x, __uint_as_float(s[16 * b + i]));
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int col = 32 * c + 16 * b + i;
                                if (col <= last && col > first) x = fmaxf(x, __uint_as_float(s[16 * b + i]));
                            }
                        }
                        mt = fmaxf(mt, fmaf(x, cs * sc.k[2 * c + b], sc.lv[2 * c + b]));
                    }
                }
                if (__any_sync(0xffffffffu, mt > m + kGrow)) {
                    const float mn = mt > m + kGrow ? mt : m;
                    const float f = mn == -INFINITY ? 1.0f : ex2(m - mn);
                    m = mn;
                    l *= f;
                    if (j > 0) {
                        if (!pair) {
                            ok = wait(pv_done, j - 1);  // the product of the step before still adds to O
                            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                            fence_after();
                        }
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            ld32(o_at + 32 * c, o);
                            ld_wait(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            st32(o_at + 32 * c, o);
                        }
                        st_wait();
                    }
                }
                const float ms = m == -INFINITY ? 0.0f : m;
                // exponentials: P of columns 32c .. goes to TMEM columns 16c .., whose S is read
#pragma unroll
                for (int c = 0; c < KT / 32; ++c) {
                    uint32_t s[32], p[16];
                    ld32(s_at + 32 * c, s);
                    ld_wait(s);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float f = cs * sc.k[2 * c + b], add = sc.lv[2 * c + b] - ms;
                        float sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float x0 = fmaf(__uint_as_float(s[16 * b + i]), f, add);
                            float x1 = fmaf(__uint_as_float(s[16 * b + i + 1]), f, add);
                            if (!whole) {
                                const int col = 32 * c + 16 * b + i;
                                if (col > last || col <= first) x0 = -INFINITY;
                                if (col + 1 > last || col + 1 <= first) x1 = -INFINITY;
                            }
                            const float e0 = ex2(x0), e1 = ex2(x1);
                            sum += e0 + e1;
                            p[8 * b + i / 2] = Half2Of<__half>::pack(e0, e1);
                        }
                        l = fmaf(sum, sc.rv[2 * c + b], l);
                    }
                    st16(s_at + 16 * c, p);
                }
                st_wait();
                fence_before();
                mbar_arrive(p_full(slot));
            }
            // ---- out --------------------------------------------------------------
            if (ok && steps > 0) ok = __all_sync(0xffffffffu, wait(o_full(w), 0));
            if (ok) {
                fence_after();
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                T *out = static_cast<T *>(a.out) + ((int64_t)token * a.q_heads + hq) * D;
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
                    if (real) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = H::pack(l == 0.0f ? 0.0f : __uint_as_float(o[i + 2 * k]) * inv,
                                               l == 0.0f ? 0.0f : __uint_as_float(o[i + 2 * k + 1]) * inv);
                            *reinterpret_cast<uint4 *>(out + 32 * c + i) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                }
                if (real && a.lse)
                    a.lse[(int64_t)token * a.q_heads + hq] =
                        l == 0.0f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
            }
        }
    } else if (warp < kMmaWarp) {
        // ---- codes to fp16 tiles ---------------------------------------------------
        // four lanes take the 64 bytes of a key's panel, eight keys a warp: the 16-byte
        // stores of a quarter warp (two keys) hit all banks once
        constexpr int kGroups = KT / 32;  // keys of a thread in each panel: gi * 32 + key
        const int ct = tid - kSoftWarps * 32, key = ct >> 2, part = ct & 3;
        uint4 kx[kGroups * P::kPanels], vx[kGroups * P::kPanels];
        int64_t blk[kGroups];
        auto find = [&](int j) {
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi) {
                const int t = k_lo + j * KT + gi * 32 + key;
                blk[gi] = t < hi ? a.L.block_of(row, head, t) : -1;
            }
        };
        auto load = [&](const uint8_t *pool, uint4 (&x)[kGroups * P::kPanels]) {
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi)
#pragma unroll
                for (int p = 0; p < P::kPanels; ++p) {
                    uint4 v = make_uint4(0, 0, 0, 0);  // keys past the last that is seen: 0, never stale bytes
                    if (blk[gi] >= 0)
                        v = __ldg(reinterpret_cast<const uint4 *>(pool + blk[gi] * (kBlock * D) + (key & 15) * D +
                                                                  p * 64 + part * 16));
                    x[gi * P::kPanels + p] = v;
                }
        };
        auto store = [&](uint32_t tile, const uint4 (&x)[kGroups * P::kPanels]) {
#pragma unroll
            for (int gi = 0; gi < kGroups; ++gi)
#pragma unroll
                for (int p = 0; p < P::kPanels; ++p) {
                    const int kk = gi * 32 + key;
                    const uint32_t at = tile + p * P::kPanelKV + kk * 128;
                    const uint4 v = x[gi * P::kPanels + p];
                    const uint32_t w[4] = {C::ready(v.x), C::ready(v.y), C::ready(v.z), C::ready(v.w)};
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         at + (((2 * part + h) ^ (kk & 7)) << 4)),
                                     "r"(C::template pair<0>(w[2 * h])), "r"(C::template pair<1>(w[2 * h])),
                                     "r"(C::template pair<0>(w[2 * h + 1])), "r"(C::template pair<1>(w[2 * h + 1]))
                                     : "memory");
                }
        };
        bool ok = true;
        if (steps > 0) {
            find(0);
            load(a.L.k, kx);
        }
        for (int j = 0; j < steps && ok; ++j) {
            load(a.L.v, vx);
            float ksc = 0.0f, vsc = 1.0f;
            if (ct < P::kBlocks) {
                const int t = k_lo + j * KT + ct * kBlock;
                if (t < hi) {
                    const int64_t b = a.L.block_of(row, head, t);
                    ksc = __ldg(a.L.ks + b);
                    vsc = fmaxf(__ldg(a.L.vs + b), 1e-37f);
                }
            }
            if (j >= kStages) ok = wait(k_empty(j), j / kStages - 1);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            if (ct < P::kBlocks) {
                Scales &sc = scales[j % kScaleRing];
                sc.k[ct] = ksc;
                sc.lv[ct] = __log2f(vsc);
                sc.rv[ct] = __frcp_rn(vsc);
            }
            store(base + P::kOffK + (j % kStages) * P::kKV, kx);
            fence_proxy_async_smem();
            mbar_arrive(k_full(j));
            if (j + 1 < steps) {
                find(j + 1);
                load(a.L.k, kx);
            }
            if (j >= kStages) ok = wait(v_empty(j), j / kStages - 1);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            store(base + P::kOffV + (j % kStages) * P::kKV, vx);
            fence_proxy_async_smem();
            mbar_arrive(v_full(j));
        }
    } else if (lane == 0) {
        // ---- MMA issue --------------------------------------------------------------
        constexpr uint32_t i_qk = idesc_f16(128, KT, false), i_pv = idesc_f16(128, D, true);
        auto qk = [&](int j, int w, int slot) {
            const uint32_t q = base + w * (P::kPanels * P::kPanelQ), k = base + P::kOffK + (j % kStages) * P::kKV;
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
                mma_ss(tmem + (slot ? P::kS1 : 0), desc128(q + (s / 4) * P::kPanelQ + (s % 4) * 32, 16, 1024),
                       desc128(k + (s / 4) * P::kPanelKV + (s % 4) * 32, 16, 1024), i_qk, s > 0);
            commit(s_full(slot));
        };
        auto pv = [&](int j, int w, int slot) {
            const uint32_t v = base + P::kOffV + (j % kStages) * P::kKV;
#pragma unroll
            for (int s = 0; s < KT / 16; ++s)
                mma_ts(tmem + (w ? P::kO1 : P::kO0), tmem + (slot ? P::kS1 : 0) + 8 * s,
                       desc128(v + s * 16 * 128, P::kPanelKV, 1024), i_pv, j > 0 || s > 0);
        };
        bool ok = steps > 0 && wait(q_full, 0) && wait(k_full(0), 0);
        if (ok) {
            fence_after();
            qk(0, 0, 0);
            if (pair) qk(0, 1, 1);
            commit(k_empty(0));
        }
        for (int j = 0; j < steps && ok; ++j) {
            const bool next = j + 1 < steps;
            if (pair) {
                ok = wait(v_full(j), j / kStages) && wait(p_full(0), j);
                if (!ok) break;
                fence_after();
                pv(j, 0, 0);
                if (next) {
                    ok = wait(k_full(j + 1), (j + 1) / kStages);
                    if (!ok) break;
                    fence_after();
                    qk(j + 1, 0, 0);
                } else {
                    commit(o_full(0));
                }
                ok = wait(p_full(1), j);
                if (!ok) break;
                fence_after();
                pv(j, 1, 1);
                commit(v_empty(j));
                if (next) {
                    qk(j + 1, 1, 1);
                    commit(k_empty(j + 1));
                } else {
                    commit(o_full(1));
                }
            } else {
                if (next) {
                    ok = wait(k_full(j + 1), (j + 1) / kStages);
                    if (!ok) break;
                    fence_after();
                    qk(j + 1, 0, (j + 1) & 1);
                    commit(k_empty(j + 1));
                }
                ok = wait(v_full(j), j / kStages) && wait(p_full(j & 1), j >> 1);
                if (!ok) break;
                fence_after();
                pv(j, 0, j & 1);
                commit(v_empty(j));
                commit(pv_done);
                if (!next) commit(o_full(0));
            }
        }
        if (!ok && steps > 0) {
            // what was issued reads and writes this CTA's memory: let it finish
            commit(drained);
            mbar_wait_for(drained, 0, kDrainWaitNs, &g_prefill_timeouts);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, P::kCols);
}

template <typename T, int D, int FMT>
int launch_t(const AttendArgs &a, cudaStream_t s)
{
    using P = Plan<D>;
    auto kern = attend_prefill_kernel<T, D, FMT>;
    static bool done[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return BQD_ERR_CUDA;
    if (dev < 0 || dev >= 64 || !done[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)P::kSmem) != cudaSuccess)
            return BQD_ERR_CUDA;
        if (dev >= 0 && dev < 64) done[dev] = true;
    }
    const int64_t rows = (int64_t)a.max_new * a.group;
    const dim3 grid((unsigned)((rows + P::kRows - 1) / P::kRows), (unsigned)a.L.heads, (unsigned)a.L.rows);
    kern<<<grid, kThreadsF, P::kSmem, s>>>(a, opt_wait_ns());
    return cuda_status(cudaGetLastError());
}

template <typename T, int FMT>
int launch_d(const AttendArgs &a, cudaStream_t s)
{
    if (a.head_dim == 64) return launch_t<T, 64, FMT>(a, s);
    if (a.head_dim == 128) return launch_t<T, 128, FMT>(a, s);
    return launch_t<T, 256, FMT>(a, s);
}

}  // namespace

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
