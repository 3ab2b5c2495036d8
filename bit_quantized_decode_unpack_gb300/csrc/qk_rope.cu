// Norm of each query and key head, and the rotation by position, in one pass.
//
//   y = x w / sqrt(mean(x^2) + eps)            (over the head's D values)
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = position * inv_freq[j]
// for the pairs j of the head's first `rotary` values: (j, j + rotary / 2), or
// (2 j, 2 j + 1) where interleaved.  What lies past `rotary` is only normalised.
// Everything is fp32 and rounded once.
//
// Angles.  A frequency is held in turns, as a 64-bit fraction F = inv_freq / 2 pi *
// 2^64, so that position * F in wrapping integers is the angle modulo a turn with
// an error below 2^-64 position turns: no position is too far.  The upper 32 bits
// go to sincospi, whose argument is then off by at most 2^-25 turns.
//
// Layout.  A lane has 16 values of a head, the members a and b of 8 pairs (what is not
// rotated counts as pairs too), so the only exchange is the sum of squares over D / 16
// lanes.  A warp takes 512 / D heads at a time and several such groups of one token, the
// next two groups' loads in flight while one is computed.  Its lanes share the token's
// angles out among them and exchange them once, weights are folded into the sines and
// cosines, and two values go through each fp32 instruction:
//   y_a = r (a (w_a cos) - b (w_b sin)),  y_b = r (a (w_a sin) + b (w_b cos)),
// r the reciprocal root.  Bound by memory, 2 bytes read and 2 written a value: 16384
// tokens of 28 heads of 256 in 82 us for 470 MB (5710 GB/s, 84% of a measured copy); 2049
// tokens of 56 heads of 128, 12.1 us; 16 tokens 2.8 us, the launch.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"

namespace bqd {
namespace {

using kv::Half2Of;

constexpr int kWarpsR = 4;
constexpr int kAhead = 2;  // head groups in flight of a warp: with 24 warps an SM, 82 us for 470 MB; 4 and 16 warps: 101

struct RopeParams {
    const void *x[2];            // q, k
    void *y[2];
    int64_t xt[2], xh[2], yt[2], yh[2];  // strides of token and head
    const void *w[2];            // weights or nullptr
    const int32_t *positions;
    const uint64_t *freqs;
    int heads[2];
    int64_t units;               // warps with work
    int parts, q_parts, each;    // warps of a token, those with heads of q, head groups of a warp
    int pair_lanes;              // rotary / 16: lanes of a head whose values are rotated
    int rotary;
    bool norm, w_f32;
    float eps, amplitude;
};

template <bool VEC>
__device__ __forceinline__ uint4 load8(const unsigned short *p)
{
    // not through the read-only path: the output may be the input
    if constexpr (VEC) {
        return __ldcs(reinterpret_cast<const uint4 *>(p));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldcs(p + 2 * i) | ((uint32_t)__ldcs(p + 2 * i + 1) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool VEC>
__device__ __forceinline__ void store8(unsigned short *p, const uint4 &v)
{
    if constexpr (VEC) {
        *reinterpret_cast<uint4 *>(p) = v;
    } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[2 * i] = (unsigned short)(w[i] & 0xFFFFu);
            p[2 * i + 1] = (unsigned short)(w[i] >> 16);
        }
    }
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

template <typename T, int D, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kWarpsR * 32, 6)
qk_rope_kernel(const RopeParams p)
{
    using H = Half2Of<T>;
    constexpr int kLanes = D / 16;        // lanes of a head
    constexpr int kHeads = 32 / kLanes;   // heads of a warp's pass
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarpsR + (threadIdx.x >> 5);
    if (unit >= p.units) return;
    const int64_t token = unit / p.parts;
    const int part = (int)(unit - token * p.parts);
    const int c = lane % kLanes, sub = lane / kLanes;
    // The lane's two runs of 8 values, each next to its neighbours' (whole sectors in each access), and
    // whether they are rotated.  Interleaved: four pairs a run.  Else the members of eight pairs, first
    // those of the rotated values, then of the others.
    const bool in = c < p.pair_lanes;
    const int e0 = INTERLEAVED || in ? 8 * c : p.rotary + 8 * (c - p.pair_lanes);
    const int e1 = INTERLEAVED ? D / 2 + 8 * c : e0 + (in ? p.rotary / 2 : (D - p.rotary) / 2);
    const bool turned0 = INTERLEAVED ? e0 < p.rotary : in, turned1 = INTERLEAVED ? e1 < p.rotary : in;

    // a warp has heads of q or of k
    const int which = part >= p.q_parts, g0 = (which ? part - p.q_parts : part) * p.each;
    const int heads = p.heads[which], groups = min(p.each, (heads + kHeads - 1) / kHeads - g0);
    const int head = g0 * kHeads + sub;  // of the lane's first group
    const int64_t x_step = kHeads * p.xh[which], y_step = kHeads * p.yh[which];
    const unsigned short *x_at = static_cast<const unsigned short *>(p.x[which]) + token * p.xt[which] + head * p.xh[which];
    unsigned short *y_at = static_cast<unsigned short *>(p.y[which]) + token * p.yt[which] + head * p.yh[which];
    const int mine = head < heads ? min(groups, (heads - head + kHeads - 1) / kHeads) : 0;  // groups with a head of the lane's
    uint4 ring[kAhead][2];               // values of the next groups, on their way
    auto load = [&](int i, uint4 (&n)[2]) {
        n[0] = n[1] = make_uint4(0, 0, 0, 0);
        if (i < mine) n[0] = load8<VEC>(x_at + e0), n[1] = load8<VEC>(x_at + e1);
        x_at += x_step;
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, ring[i]);

    // lane (sub, c) computes 8 / kHeads of the angles of lanes (., c), and gets the others from there
    uint64_t cs[4], sn[4];  // two pairs each
    {
        constexpr int kMine = 8 / kHeads;
        float co[kMine], si[kMine];
        const int64_t pos = p.pair_lanes ? p.positions[token] : 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            co[i] = 1.0f, si[i] = 0.0f;
            const int pair = sub * kMine + i;  // of the lane's 8
            if (pair < 4 ? turned0 : turned1) {
                const int j = !INTERLEAVED ? 8 * c + pair : 4 * c + (pair < 4 ? pair : D / 4 + pair - 4);
                const uint64_t t = (uint64_t)pos * __ldg(p.freqs + j);
                sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &si[i], &co[i]);  // 2^-31: half turns
                co[i] *= p.amplitude, si[i] *= p.amplitude;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s0 = c + kLanes * ((2 * i) / kMine), s1 = c + kLanes * ((2 * i + 1) / kMine);
            cs[i] = two(__shfl_sync(0xffffffffu, co[(2 * i) % kMine], s0), __shfl_sync(0xffffffffu, co[(2 * i + 1) % kMine], s1));
            sn[i] = two(__shfl_sync(0xffffffffu, si[(2 * i) % kMine], s0), __shfl_sync(0xffffffffu, si[(2 * i + 1) % kMine], s1));
        }
    }
    uint64_t ac[4], as[4], bc[4], bs[4];  // w_a cos, w_a sin, w_b cos, - w_b sin
    {
        const void *w = p.w[which];
        auto weight = [&](int e) {
            return !w ? 1.0f
                   : p.w_f32 ? __ldg(static_cast<const float *>(w) + e)
                             : H::f1(__ldg(static_cast<const unsigned short *>(w) + e));
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (members of pairs 2i, 2i + 1)
            const int at = INTERLEAVED ? (i < 2 ? e0 + 4 * i : e1 + 4 * i - 8) : e0 + 2 * i;
            const uint64_t wa = INTERLEAVED ? two(weight(at), weight(at + 2)) : two(weight(at), weight(at + 1));
            const uint64_t wb = INTERLEAVED ? two(weight(at + 1), weight(at + 3)) : two(weight(e1 + 2 * i), weight(e1 + 2 * i + 1));
            ac[i] = mul2(wa, cs[i]), as[i] = mul2(wa, sn[i]), bc[i] = mul2(wb, cs[i]);
            bs[i] = mul2(mul2(wb, sn[i]), two(-1.0f, -1.0f));
        }
    }
    const bool all = p.rotary == D;  // nothing is left as it is
    for (int ib = 0; ib < groups; ib += kAhead)
#pragma unroll
    for (int slot = 0; slot < kAhead; ++slot) {
        if (ib + slot >= groups) break;
        const uint32_t u[8] = {ring[slot][0].x, ring[slot][0].y, ring[slot][0].z, ring[slot][0].w,
                               ring[slot][1].x, ring[slot][1].y, ring[slot][1].z, ring[slot][1].w};
        load(ib + slot + kAhead, ring[slot]);
        uint64_t a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (INTERLEAVED) {
                const float2 f = H::f2(u[2 * i]), h = H::f2(u[2 * i + 1]);
                a[i] = two(f.x, h.x), b[i] = two(f.y, h.y);
            } else {
                const float2 f = H::f2(u[i]), h = H::f2(u[4 + i]);
                a[i] = two(f.x, f.y), b[i] = two(h.x, h.y);
            }
        }
        float r = 1.0f;
        if (p.norm) {
            uint64_t s2 = two(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = fma2(b[i], b[i], fma2(a[i], a[i], s2));
            const float2 f = untwo(s2);
            float ss = f.x + f.y;
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
        }
        const uint64_t rr = two(r, r);
        float ya[8], yb[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint64_t x = mul2(a[i], ac[i]), y = mul2(b[i], bc[i]);
            // (what is not rotated stays apart: an infinity would meet a sine of 0)
            if (all || (i < 2 ? turned0 : turned1)) x = fma2(b[i], bs[i], x), y = fma2(a[i], as[i], y);
            const float2 fx = untwo(mul2(x, rr)), fy = untwo(mul2(y, rr));
            ya[2 * i] = fx.x, ya[2 * i + 1] = fx.y, yb[2 * i] = fy.x, yb[2 * i + 1] = fy.y;
        }
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = INTERLEAVED ? H::pack(ya[i], yb[i]) : i < 4 ? H::pack(ya[2 * i], ya[2 * i + 1]) : H::pack(yb[2 * i - 8], yb[2 * i - 7]);
        if (ib + slot < mine) {
            store8<VEC>(y_at + e0, make_uint4(v[0], v[1], v[2], v[3]));
            store8<VEC>(y_at + e1, make_uint4(v[4], v[5], v[6], v[7]));
        }
        y_at += y_step;
    }
}

template <typename T, int D>
int launch_t(RopeParams &p, int64_t tokens, bool interleaved, bool vec, cudaStream_t s)
{
    constexpr int kHeads = 512 / D;
    const int groups[2] = {(p.heads[0] + kHeads - 1) / kHeads, (p.heads[1] + kHeads - 1) / kHeads};
    // a warp takes more of a token's head groups once there are 32 warps an SM (two waves) with fewer
    const int64_t warps = (int64_t)sm_count() * 32, most = std::max(groups[0], groups[1]);
    p.each = (int)std::max<int64_t>(1, std::min<int64_t>(most, tokens * (groups[0] + groups[1]) / warps));
    const int64_t shares = (most + p.each - 1) / p.each;
    p.each = (int)((most + shares - 1) / shares);
    p.q_parts = (groups[0] + p.each - 1) / p.each;
    p.parts = p.q_parts + (groups[1] + p.each - 1) / p.each;
    p.units = tokens * p.parts;
    const int64_t grid = (p.units + kWarpsR - 1) / kWarpsR;
    if (grid > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    const dim3 b(kWarpsR * 32), n((unsigned)grid);
    if (interleaved) {
        if (vec) qk_rope_kernel<T, D, true, true><<<n, b, 0, s>>>(p);
        else qk_rope_kernel<T, D, true, false><<<n, b, 0, s>>>(p);
    } else {
        if (vec) qk_rope_kernel<T, D, false, true><<<n, b, 0, s>>>(p);
        else qk_rope_kernel<T, D, false, false><<<n, b, 0, s>>>(p);
    }
    return cuda_status(cudaGetLastError());
}

template <typename T>
int launch_d(RopeParams &p, int64_t tokens, int head_dim, bool interleaved, bool vec, cudaStream_t s)
{
    if (head_dim == 64) return launch_t<T, 64>(p, tokens, interleaved, vec, s);
    if (head_dim == 128) return launch_t<T, 128>(p, tokens, interleaved, vec, s);
    return launch_t<T, 256>(p, tokens, interleaved, vec, s);
}

bool at(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// strides of token and head that stay within 2^57 elements
bool strides_ok(int64_t tokens, int64_t ts, int64_t heads, int64_t hs)
{
    const int64_t most = (int64_t)1 << 40;
    return ts >= 0 && hs >= 0 && ts < most && hs < most && (double)tokens * (double)ts < 1e17 &&
           (double)heads * (double)hs < 1e17;
}

bool vec_ok(const void *p, int64_t ts, int64_t hs) { return at(p, 16) && ts % 8 == 0 && hs % 8 == 0; }

}  // namespace
}  // namespace bqd

extern "C" int bqd_qk_norm_rope(const bqd_qk_rope *plan, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                int q_heads, const void *k, int64_t k_token_stride, int64_t k_head_stride, int k_heads,
                                int dtype, const int32_t *positions, int64_t tokens, void *q_out,
                                int64_t q_out_token_stride, int64_t q_out_head_stride, void *k_out,
                                int64_t k_out_token_stride, int64_t k_out_head_stride, bqd_stream_t stream)
{
    using namespace bqd;
    if (!plan) return BQD_ERR_INVALID_ARG;
    const int d = plan->head_dim, rot = plan->rotary_dim;
    if (d != 64 && d != 128 && d != 256) return BQD_ERR_INVALID_ARG;
    if (rot < 0 || rot > d || rot % 16 != 0 || (rot > 0 && !plan->freqs)) return BQD_ERR_INVALID_ARG;
    if ((dtype != BQD_DTYPE_F16 && dtype != BQD_DTYPE_BF16) ||
        (plan->weight_dtype != dtype && plan->weight_dtype != BQD_DTYPE_F32 && (plan->q_weight || plan->k_weight)))
        return BQD_ERR_INVALID_ARG;
    if (!std::isfinite(plan->amplitude) || (plan->norm && !(plan->eps > 0.0f && std::isfinite(plan->eps))))
        return BQD_ERR_INVALID_ARG;
    if (tokens < 0 || tokens > ((int64_t)1 << 30) || q_heads < 0 || k_heads < 0 || q_heads > 65535 || k_heads > 65535)
        return BQD_ERR_INVALID_ARG;
    RopeParams p;
    const void *x[2] = {q, k};
    void *y[2] = {q_out, k_out};
    const int64_t xt[2] = {q_token_stride, k_token_stride}, xh[2] = {q_head_stride, k_head_stride};
    const int64_t yt[2] = {q_out_token_stride, k_out_token_stride}, yh[2] = {q_out_head_stride, k_out_head_stride};
    const void *w[2] = {plan->q_weight, plan->k_weight};
    p.heads[0] = q_heads, p.heads[1] = k_heads;
    bool vec = true;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = x[i], p.y[i] = y[i], p.xt[i] = xt[i], p.xh[i] = xh[i], p.yt[i] = yt[i], p.yh[i] = yh[i], p.w[i] = w[i];
        if (p.heads[i] == 0 || tokens == 0) continue;
        if (!x[i] || !y[i]) return BQD_ERR_INVALID_ARG;
        if (!strides_ok(tokens, xt[i], p.heads[i], xh[i]) || !strides_ok(tokens, yt[i], p.heads[i], yh[i]))
            return BQD_ERR_INVALID_ARG;
        if (!at(x[i], 2) || !at(y[i], 2) || !at(w[i], plan->weight_dtype == BQD_DTYPE_F32 ? 4 : 2)) return BQD_ERR_ALIGNMENT;
        // no two heads of an output share memory
        const int64_t h1 = p.heads[i] - 1, t1 = tokens - 1;
        if ((h1 > 0 && yh[i] < d) || (t1 > 0 && yt[i] < d) || (h1 > 0 && t1 > 0 && yt[i] < h1 * yh[i] + d && yh[i] < t1 * yt[i] + d))
            return BQD_ERR_INVALID_ARG;
        vec = vec && vec_ok(x[i], xt[i], xh[i]) && vec_ok(y[i], yt[i], yh[i]);
    }
    if (tokens == 0 || q_heads + k_heads == 0) return BQD_OK;
    if (rot > 0 && !positions) return BQD_ERR_INVALID_ARG;
    if (!at(positions, 4) || !at(plan->freqs, 8)) return BQD_ERR_ALIGNMENT;
    p.positions = positions, p.freqs = plan->freqs;
    p.pair_lanes = rot / 16, p.rotary = rot;
    p.norm = plan->norm != 0, p.w_f32 = plan->weight_dtype == BQD_DTYPE_F32;
    p.eps = plan->eps, p.amplitude = plan->amplitude;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == BQD_DTYPE_F16 ? launch_d<__half>(p, tokens, d, plan->interleaved != 0, vec, s)
                                  : launch_d<__nv_bfloat16>(p, tokens, d, plan->interleaved != 0, vec, s);
}
