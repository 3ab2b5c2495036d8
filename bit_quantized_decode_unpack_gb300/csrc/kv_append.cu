// Quantise new keys and values into a paged 8-bit cache.
//
// For a block of 16 tokens and one head, with x its new values and c, s the
// codes and scale it may already hold:
//   s' = max(s, fp32(max(amax |x|, 2^-80) * fp32(1/top))),  r = fp32(1 / s')
//   new code = rnd(fp32(x r)),   kept code' = rnd(fp32(fp32(c s) r)) if s' > s
// The scale of a block only grows, so a block's tokens can arrive one at a
// time; each growth costs the earlier codes one more rounding.
//
// One warp owns one (block, head) of K or of V: it holds the block's new
// values in registers (16 D / 32 values a lane, all loads in flight at once),
// takes the maximum with one warp reduction, and writes the codes.  Nothing is
// read twice and no other warp touches the block, so there are no atomics and
// the result does not depend on any order.  Bound by memory, 2 bytes read and 1
// written a value: 65536 tokens of 8 heads of 128, 403 MB in 63.6 us (6340 GB/s,
// 95% of a measured copy); 16 single tokens 2.7 us, the launch.
// Consecutive warps take consecutive heads of a block, then K and V, so that
// the inputs of one token are read together.
#include <algorithm>

#include "kv_common.cuh"

namespace bqd {
namespace kv {
namespace {

constexpr int kWarpsA = 8;
constexpr float kFloor = 8.271806125530277e-25f;  // 2^-80

struct AppendParams {
    Layer L;
    const void *x[2];            // k, v
    int64_t token_stride[2], head_stride[2];
    const int32_t *base, *starts;
    int tokens, max_new, blocks; // blocks: of a row that max_new tokens can touch
};

template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (FMT == BQD_KV_INT8) {
        // 1.5 * 2^23 + t has the integer nearest to t (ties to even) in its low bits
        const float m = 12582912.0f;
        const uint32_t ua = __float_as_uint(__fadd_rn(a, m)), ub = __float_as_uint(__fadd_rn(b, m));
        const uint32_t uc = __float_as_uint(__fadd_rn(c, m)), ud = __float_as_uint(__fadd_rn(d, m));
        return __byte_perm(__byte_perm(ua, ub, 0x0040), __byte_perm(uc, ud, 0x0040), 0x5410);
    } else {
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
        return (uint32_t)lo | ((uint32_t)hi << 16);
    }
}

// x r of a value that may be infinite or NaN
template <int FMT>
__device__ __forceinline__ float tame(float t)
{
    return t != t ? 0.0f : fminf(fmaxf(t, -Code<FMT>::kTop), Code<FMT>::kTop);
}

template <typename T, bool VEC>
__device__ __forceinline__ uint4 load8(const T *p)
{
    if constexpr (VEC) {
        uint4 v;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
        return v;
    } else {
        const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(u + 2 * i) | ((uint32_t)__ldg(u + 2 * i + 1) << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T, int D, int FMT, bool VEC>
__global__ void __launch_bounds__(kWarpsA * 32)
append_kernel(const AppendParams p)
{
    constexpr int kRowLanes = D / 8;            // lanes of one token (8 values each)
    constexpr int kRowsPass = 32 / kRowLanes;   // tokens of one pass of the warp
    constexpr int kPasses = kBlock / kRowsPass;
    using H = Half2Of<T>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // unit: head fastest, then K / V, then block, then row
    const int64_t unit = (int64_t)blockIdx.x * kWarpsA + warp;
    const int head = (int)(unit % p.L.heads);
    int64_t u = unit / p.L.heads;
    const int which = (int)(u & 1);
    u >>= 1;
    const int bi = (int)(u % p.blocks);
    const int64_t row64 = u / p.blocks;
    if (row64 >= p.L.rows) return;
    const int row = (int)row64;
    const int base = p.base[row];
    if (base < 0 || base >= p.L.capacity()) return;
    const Span span(p.starts, row, p.tokens, p.max_new);
    const int end = min(base + span.n, p.L.capacity());
    const int t0 = (base / kBlock + bi) * kBlock;  // the block's first token
    if (t0 >= end) return;
    const int page = p.L.listed(row, t0);
    if ((unsigned)page >= (unsigned)p.L.pages) return;
    const int64_t blk = p.L.block_at(page, head, t0);
    uint8_t *codes = (which ? p.L.v : p.L.k) + blk * (kBlock * D);
    float *scale = (which ? p.L.vs : p.L.ks) + blk;

    const int r0 = lane / kRowLanes, col = (lane % kRowLanes) * 8;
    const int first = max(0, base - t0), last = min(kBlock, end - t0);  // new tokens of the block
    const T *src = static_cast<const T *>(p.x[which]) + (int64_t)(span.lo + t0 - base) * p.token_stride[which] +
                   head * p.head_stride[which] + col;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRowsPass + r0;
        x[i] = make_uint4(0, 0, 0, 0);
        if (r >= first && r < last) x[i] = load8<T, VEC>(src + (int64_t)r * p.token_stride[which]);
    }
    const float s0 = first > 0 ? *scale : 0.0f;

    // largest magnitude: the bits of |x| order like |x|
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        mx = __vmaxu2(mx, x[i].x & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[i].y & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[i].z & 0x7FFF7FFFu);
        mx = __vmaxu2(mx, x[i].w & 0x7FFF7FFFu);
    }
    uint32_t top = max(mx & 0xFFFFu, mx >> 16);
    const bool odd = __any_sync(0xffffffffu, top >= H::kInf);  // an infinity or a NaN somewhere
    if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = w[j] & 0x7FFFu, b = (w[j] >> 16) & 0x7FFFu;
                if (a < H::kInf) top = max(top, a);
                if (b < H::kInf) top = max(top, b);
            }
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const float s1 = fmaxf(s0, __fmul_rn(fmaxf(H::f1(top), kFloor), (float)(1.0 / Code<FMT>::kTop)));
    const float inv = __frcp_rn(s1);

#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int r = i * kRowsPass + r0;
        if (r < first || r >= last) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float2 a = H::f2(w[2 * j]), b = H::f2(w[2 * j + 1]);
            a.x = __fmul_rn(a.x, inv), a.y = __fmul_rn(a.y, inv);
            b.x = __fmul_rn(b.x, inv), b.y = __fmul_rn(b.y, inv);
            if (odd) a.x = tame<FMT>(a.x), a.y = tame<FMT>(a.y), b.x = tame<FMT>(b.x), b.y = tame<FMT>(b.y);
            c[j] = encode4<FMT>(a.x, a.y, b.x, b.y);
        }
        *reinterpret_cast<uint2 *>(codes + r * D + col) = make_uint2(c[0], c[1]);
    }
    if (s1 > s0) {
        // the scale grew: the tokens that were there (r < first) take it too
#pragma unroll 1
        for (int r = r0; r < first; r += kRowsPass) {
            uint2 *at = reinterpret_cast<uint2 *>(codes + r * D + col);
            const uint2 old = *at;
            const uint32_t w[2] = {old.x, old.y};
            uint32_t c[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    f[e] = tame<FMT>(__fmul_rn(__fmul_rn(Code<FMT>::value((w[j] >> (8 * e)) & 0xFF), s0), inv));
                c[j] = encode4<FMT>(f[0], f[1], f[2], f[3]);
            }
            *at = make_uint2(c[0], c[1]);
        }
        if (lane == 0) *scale = s1;
    }
}

template <typename T, int D, int FMT>
int launch_t(const AppendParams &p, bool vec, cudaStream_t s)
{
    const int64_t units = (int64_t)p.L.rows * p.blocks * 2 * p.L.heads;
    const int64_t grid = (units + kWarpsA - 1) / kWarpsA;
    if (grid > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    if (vec) append_kernel<T, D, FMT, true><<<(unsigned)grid, kWarpsA * 32, 0, s>>>(p);
    else append_kernel<T, D, FMT, false><<<(unsigned)grid, kWarpsA * 32, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}

template <typename T, int FMT>
int launch_d(const AppendParams &p, int head_dim, bool vec, cudaStream_t s)
{
    if (head_dim == 64) return launch_t<T, 64, FMT>(p, vec, s);
    if (head_dim == 128) return launch_t<T, 128, FMT>(p, vec, s);
    return launch_t<T, 256, FMT>(p, vec, s);
}

}  // namespace

int launch_append(const AppendArgs &a, cudaStream_t s)
{
    AppendParams p;
    p.L = a.L;
    for (int i = 0; i < 2; ++i) {
        p.x[i] = a.x[i];
        p.token_stride[i] = a.token_stride[i];
        p.head_stride[i] = a.head_stride[i];
    }
    p.base = a.base;
    p.starts = a.starts;
    p.tokens = a.tokens;
    p.max_new = a.max_new;
    // the most blocks that max_new consecutive tokens can touch, and no more
    // than the table can list
    p.blocks = (int)std::min<int64_t>(((int64_t)a.max_new + 2 * kBlock - 2) / kBlock,
                                      ((int64_t)a.L.row_pages << a.L.page_shift) / kBlock);
    if (a.format == BQD_KV_INT8)
        return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_INT8>(p, a.head_dim, a.vec, s)
                                        : launch_d<__nv_bfloat16, BQD_KV_INT8>(p, a.head_dim, a.vec, s);
    return a.dtype == BQD_DTYPE_F16 ? launch_d<__half, BQD_KV_E4M3>(p, a.head_dim, a.vec, s)
                                    : launch_d<__nv_bfloat16, BQD_KV_E4M3>(p, a.head_dim, a.vec, s);
}

}  // namespace kv
}  // namespace bqd
