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
// Layout.  A lane has 16 values of a head: 8 from each half of the pairs, so both
// members of its 8 pairs are its own and the only exchange is the sum of squares
// over D / 16 lanes.  A warp takes 512 / D heads at a time and keeps the sines and
// cosines of one token for all of its heads.  Few tokens: a token's heads are
// spread over warps, each computes the angles again (latency counts).  Many: one
// warp takes a token, with the next heads' loads in flight while these are computed.
// Bound by memory, 2 bytes read and 2 written a value.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"

namespace bqd {
namespace {

using kv::Half2Of;

constexpr int kWarpsR = 4;

struct RopeParams {
    const void *x[2];            // q, k
    void *y[2];
    int64_t xt[2], xh[2], yt[2], yh[2];  // strides of token and head
    const void *w[2];            // weights or nullptr
    const int32_t *positions;
    const uint64_t *freqs;
    int heads[2];
    int64_t units;               // warps with work
    int parts, each;             // warps of a token, head groups of a warp
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

template <typename T, int D, bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kWarpsR * 32)
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
    const bool turned = c < p.pair_lanes;
    // the lane's two runs of 8 values
    const int e0 = INTERLEAVED ? 16 * c : turned ? 8 * c : p.rotary + 16 * (c - p.pair_lanes);
    const int e1 = !INTERLEAVED && turned ? e0 + p.rotary / 2 : e0 + 8;

    const int q_groups = (p.heads[0] + kHeads - 1) / kHeads, k_groups = (p.heads[1] + kHeads - 1) / kHeads;
    const int g0 = part * p.each, g1 = min(g0 + p.each, q_groups + k_groups);
    uint4 n0, n1;  // the next group's values
    auto load = [&](int g) {
        n0 = n1 = make_uint4(0, 0, 0, 0);
        if (g >= g1) return;
        const int which = g >= q_groups, head = (which ? g - q_groups : g) * kHeads + sub;
        if (head >= p.heads[which]) return;
        const unsigned short *x = static_cast<const unsigned short *>(p.x[which]) + token * p.xt[which] + head * p.xh[which];
        n0 = load8<VEC>(x + e0);
        n1 = load8<VEC>(x + e1);
    };
    load(g0);

    float cs[8], sn[8];
    if (turned) {
        const int64_t pos = p.positions[token];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t t = (uint64_t)pos * __ldg(p.freqs + 8 * c + i);
            sincospif((float)(int32_t)(t >> 32) * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: half turns
            cs[i] *= p.amplitude, sn[i] *= p.amplitude;
        }
    }
    float w[16];
    int loaded = -1;  // whose weights are in w
    for (int g = g0; g < g1; ++g) {
        const int which = g >= q_groups, head = (which ? g - q_groups : g) * kHeads + sub;
        const uint32_t u[8] = {n0.x, n0.y, n0.z, n0.w, n1.x, n1.y, n1.z, n1.w};
        load(g + 1);
        if (loaded != which) {
            loaded = which;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = i < 8 ? e0 + i : e1 + i - 8;
                w[i] = !p.w[which] ? 1.0f
                       : p.w_f32   ? __ldg(static_cast<const float *>(p.w[which]) + e)
                                   : H::f1(__ldg(static_cast<const unsigned short *>(p.w[which]) + e));
            }
        }
        float x[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = H::f2(u[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
        if (p.norm) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(fmaf(ss, 1.0f / D, p.eps));
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * r * w[i];
        }
        if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float &a = INTERLEAVED ? x[2 * i] : x[i], &b = INTERLEAVED ? x[2 * i + 1] : x[8 + i];
                const float ya = fmaf(a, cs[i], -b * sn[i]), yb = fmaf(a, sn[i], b * cs[i]);
                a = ya, b = yb;
            }
        }
        if (head >= p.heads[which]) continue;
        unsigned short *y = static_cast<unsigned short *>(p.y[which]) + token * p.yt[which] + head * p.yh[which];
        store8<VEC>(y + e0, make_uint4(H::pack(x[0], x[1]), H::pack(x[2], x[3]), H::pack(x[4], x[5]), H::pack(x[6], x[7])));
        store8<VEC>(y + e1, make_uint4(H::pack(x[8], x[9]), H::pack(x[10], x[11]), H::pack(x[12], x[13]), H::pack(x[14], x[15])));
    }
}

template <typename T, int D>
int launch_t(RopeParams &p, int64_t tokens, bool interleaved, bool vec, cudaStream_t s)
{
    constexpr int kHeads = 512 / D;
    const int groups = (p.heads[0] + kHeads - 1) / kHeads + (p.heads[1] + kHeads - 1) / kHeads;
    // a warp takes all of a token's heads once there are 16 warps an SM without splitting them
    const int64_t warps = (int64_t)sm_count() * 16;
    p.each = (int)std::max<int64_t>(1, std::min<int64_t>(groups, tokens * groups / warps));
    p.parts = (groups + p.each - 1) / p.each;
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
