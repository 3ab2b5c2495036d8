// Shared parts of the kernels that read rows of logits: 16-byte vectors of
// fp16, bf16 or fp32 values, and a row's parts.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cmath>

namespace bqd {
namespace lg {

// One 16-byte vector of T.  max() and the counts ignore NaN.
template <typename T>
struct Vec;

template <>
struct Vec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void values(const uint4 &u, float (&x)[E])
    {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ float max(const uint4 &u)
    {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    // values raised to at least kLow; NaN too
    static constexpr float kLow = -1e38f;
    static __device__ __forceinline__ uint4 raised(const uint4 &u)
    {
        auto f = [](uint32_t w) { return __float_as_uint(fmaxf(__uint_as_float(w), kLow)); };
        return make_uint4(f(u.x), f(u.y), f(u.z), f(u.w));
    }
    // how many values of a few vectors are larger than a bound
    struct Count {
        int n = 0;
        __device__ __forceinline__ void add(const uint4 &u, float bound)
        {
            n += __uint_as_float(u.x) > bound, n += __uint_as_float(u.y) > bound;
            n += __uint_as_float(u.z) > bound, n += __uint_as_float(u.w) > bound;
        }
        __device__ __forceinline__ int value() const { return n; }
    };
    // the next value below one above -infinity
    static __device__ __forceinline__ float below(float x)
    {
        const uint32_t b = __float_as_uint(x + 0.0f);
        return b == 0u ? -1.4e-45f : __uint_as_float((b >> 31) ? b + 1 : b - 1);
    }
};

template <>
struct Vec<__half> {
    static constexpr int E = 8;
    static __device__ __forceinline__ __half2 h(uint32_t u) { return *reinterpret_cast<const __half2 *>(&u); }
    static __device__ __forceinline__ void values(const uint4 &u, float (&x)[E])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h(w[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float max(const uint4 &u)
    {
        const float2 f = __half22float2(__hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w))));
        return fmaxf(f.x, f.y);
    }
    static __device__ __forceinline__ float one(const __half *p) { return __half2float(*p); }
    // values raised to at least kLow, the lowest finite one; NaN too
    static constexpr float kLow = -65504.0f;
    static __device__ __forceinline__ uint4 raised(const uint4 &u)
    {
        auto f = [](uint32_t w) {
            const __half2 m = __hmax2(h(w), h(0xFBFFFBFFu));
            return *reinterpret_cast<const uint32_t *>(&m);
        };
        return make_uint4(f(u.x), f(u.y), f(u.z), f(u.w));
    }
    // how many values of a few vectors (up to 32) are larger than a bound: 1 or 0 in each half, an exact sum
    struct Count {
        uint32_t n = 0;
        __device__ __forceinline__ void add(const uint4 &u, float b)
        {
            const __half2 y = __float2half2_rn(b);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __half2 m = __hadd2(h(n), __hgt2(h(w[i]), y));
                n = *reinterpret_cast<const uint32_t *>(&m);
            }
        }
        __device__ __forceinline__ int value() const { return (int)(__low2float(h(n)) + __high2float(h(n))); }
    };
    // the next value below one above -infinity
    static __device__ __forceinline__ float below(float x)
    {
        const uint32_t b = __half_as_ushort(__float2half_rn(x + 0.0f));
        const uint32_t y = b == 0u ? 0x8001u : (b >> 15) ? b + 1 : b - 1;
        return __half2float(__ushort_as_half((unsigned short)y));
    }
};

template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ __nv_bfloat162 h(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); }
    static __device__ __forceinline__ void values(const uint4 &u, float (&x)[E])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    static __device__ __forceinline__ float max(const uint4 &u)
    {
        const __nv_bfloat162 m = __hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w)));
        const uint32_t w = *reinterpret_cast<const uint32_t *>(&m);
        return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float one(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    // values raised to at least kLow (0xFE96); NaN too
    static constexpr float kLow = -0x1.2cp126f;
    static __device__ __forceinline__ uint4 raised(const uint4 &u)
    {
        auto f = [](uint32_t w) {
            const __nv_bfloat162 m = __hmax2(h(w), h(0xFE96FE96u));
            return *reinterpret_cast<const uint32_t *>(&m);
        };
        return make_uint4(f(u.x), f(u.y), f(u.z), f(u.w));
    }
    // how many values of a few vectors (up to 32) are larger than a bound: 1 or 0 in each half, an exact sum
    struct Count {
        uint32_t n = 0;
        __device__ __forceinline__ void add(const uint4 &u, float b)
        {
            const __nv_bfloat162 y = __float2bfloat162_rn(b);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 m = __hadd2(h(n), __hgt2(h(w[i]), y));
                n = *reinterpret_cast<const uint32_t *>(&m);
            }
        }
        __device__ __forceinline__ int value() const { return (int)(__low2float(h(n)) + __high2float(h(n))); }
    };
    // the next value below one above -infinity
    static __device__ __forceinline__ float below(float x)
    {
        const uint32_t b = __bfloat16_as_ushort(__float2bfloat16_rn(x + 0.0f));
        const uint32_t y = b == 0u ? 0x8001u : (b >> 15) ? b + 1 : b - 1;
        return __uint_as_float((uint32_t)y << 16);
    }
};

// Part `part` of `parts` of a row of n values: 16-byte vectors [q0, q1) behind the first
// 16-byte boundary, and in the first and the last part the few values around them.
template <typename T>
struct Part {
    static constexpr int E = Vec<T>::E;
    const uint4 *body;
    int head, tail, tail_at;  // values before the vectors and after them (0 where another part has them)
    int first;                // index of the vectors' first value
    int q0, q1;
    __device__ __forceinline__ Part(const T *row, int n, int part, int parts)
    {
        first = min(n, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
        const int nvec = (n - first) / E;
        body = reinterpret_cast<const uint4 *>(row + first);
        q0 = (int)((int64_t)nvec * part / parts), q1 = (int)((int64_t)nvec * (part + 1) / parts);
        head = part == 0 ? first : 0;
        tail_at = first + nvec * E;
        tail = part == parts - 1 ? n - tail_at : 0;
    }
};

// CTAs that share a row of n values: until there are `ctas` of them, with 4096 values for each at least
inline int parts_of(int64_t rows, int64_t n, int64_t ctas, int most)
{
    int parts = 1;
    while (parts < most && rows * parts < ctas && n >= (int64_t)4096 * 2 * parts) parts *= 2;
    return parts;
}

}  // namespace lg
}  // namespace bqd
