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

// CTAs that share a row of n values: until each SM has two, with 4096 values for each at least
inline int parts_of(int64_t rows, int64_t n, int sms, int most)
{
    int parts = 1;
    while (parts < most && rows * parts < 2 * sms && n >= (int64_t)4096 * 2 * parts) parts *= 2;
    return parts;
}

}  // namespace lg
}  // namespace bqd
