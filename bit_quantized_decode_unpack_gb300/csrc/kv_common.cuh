// Shared parts of the paged 8-bit KV cache's kernels: one layer's view, page
// lookup, and the code conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "bqd_internal.cuh"

namespace bqd {
namespace kv {

constexpr int kBlock = BQD_KV_BLOCK;  // tokens that share a scale

// One layer of a cache (pointers already at the layer).
struct Layer {
    uint8_t *k, *v;       // [pages, heads, page_tokens, D]
    float *ks, *vs;       // [pages, heads, page_tokens / 16]
    const int32_t *table; // [rows, row_pages]
    const int32_t *lens;  // [rows]
    int pages, heads, rows, row_pages;
    int page_shift;       // log2(page_tokens)

    __device__ __forceinline__ int capacity() const { return row_pages << page_shift; }
    // tokens of a row, cut to what the table can list
    __device__ __forceinline__ int length(int row) const { return max(0, min(lens[row], capacity())); }
    // page id as listed, of the block that starts at token t
    __device__ __forceinline__ int listed(int row, int t) const
    {
        return table[(int64_t)row * row_pages + (t >> page_shift)];
    }
    // index of (page, head, block of token t) among all blocks of the layer
    __device__ __forceinline__ int64_t block_at(int page, int head, int t) const
    {
        const int per = 1 << (page_shift - 4);
        return ((int64_t)page * heads + head) * per + ((t >> 4) & (per - 1));
    }
    // same, for reading: an id outside the pool reads page 0
    __device__ __forceinline__ int64_t block_of(int row, int head, int t) const
    {
        const int p = listed(row, t);
        return block_at((unsigned)p < (unsigned)pages ? p : 0, head, t);
    }
};

// Tokens [lo, lo + n) of row r among T that the call takes: starts[r] .. starts[r + 1],
// or token r, cut to T and to max_new of them.  `rest` counts the tokens from lo to
// the row's end as starts gives it: token lo + i is the (rest - i)-th from the end,
// whatever the cuts left out.
struct Span {
    int lo, n, rest;
    __device__ __forceinline__ Span(const int32_t *starts, int row, int tokens, int max_new)
    {
        if (starts) {
            lo = max(0, min(starts[row], tokens));
            const int end = starts[row + 1];
            n = min(max(0, min(end, tokens) - lo), max_new);
            rest = min(max(end, lo) - lo, 1 << 30);  // (a row has no more tokens than a call may)
        } else {
            lo = row;
            n = rest = 1;
        }
    }
};

template <typename T>
struct Half2Of;  // conversions of a packed pair
template <>
struct Half2Of<__half> {
    static constexpr uint32_t kInf = 0x7C00;
    static __device__ __forceinline__ float2 f2(uint32_t u)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ float f1(uint32_t bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ __half one(float a) { return __float2half_rn(a); }
};
template <>
struct Half2Of<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7F80;
    static __device__ __forceinline__ float2 f2(uint32_t u)
    {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    }
    static __device__ __forceinline__ float f1(uint32_t bits) { return __uint_as_float(bits << 16); }
    static __device__ __forceinline__ uint32_t pack(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ __nv_bfloat16 one(float a) { return __float2bfloat16_rn(a); }
};

// ---- codes to fp16 -----------------------------------------------------------
// Exact in both formats.  int8: flip the sign bit (c + 128 as an unsigned
// byte), place it in the mantissa of 1024 (0x6400), subtract 1152.

template <int FMT>
struct Code;

template <>
struct Code<BQD_KV_INT8> {
    static constexpr float kTop = 127.0f;
    // bytes of a word, ready for pair() (applied once per word)
    static __device__ __forceinline__ uint32_t ready(uint32_t w) { return w ^ 0x80808080u; }
    // bytes 0, 1 (HI = 0) or 2, 3 (HI = 1) of a ready word, as fp16x2
    template <int HI>
    static __device__ __forceinline__ uint32_t pair(uint32_t w)
    {
        const uint32_t u = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
        uint32_t d;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(u), "r"(0x64806480u));
        return d;
    }
    static __device__ __forceinline__ float value(uint32_t byte) { return (float)(int8_t)byte; }
};

template <>
struct Code<BQD_KV_E4M3> {
    static constexpr float kTop = 448.0f;
    static __device__ __forceinline__ uint32_t ready(uint32_t w) { return w; }
    template <int HI>
    static __device__ __forceinline__ uint32_t pair(uint32_t w)
    {
        uint32_t d;
        const uint16_t h = (uint16_t)(HI ? w >> 16 : w);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(h));
        return d;
    }
    static __device__ __forceinline__ float value(uint32_t byte)
    {
        uint32_t d;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)(byte & 0xFF)));
        return __half2float(__ushort_as_half((unsigned short)(d & 0xFFFF)));
    }
};

// Request of bqd_kv_attend after host validation.
struct AttendArgs {
    Layer L;
    const void *q;
    int64_t q_token, q_head;  // strides in elements
    const int32_t *starts;
    void *out;
    float *lse;
    float scale;              // of q . K, times log2(e)
    int dtype, format, head_dim, q_heads, group;
    int tokens, max_new, max_len, window;
    bool q_vec;               // 16-byte loads of q are possible
    void *work;               // scratch of decode_workspace / prefill_workspace bytes, or nullptr
};

// Request of bqd_kv_append after host validation.
struct AppendArgs {
    Layer L;
    const void *x[2];  // k, v
    int64_t token_stride[2], head_stride[2];
    const int32_t *base, *starts;
    int dtype, format, head_dim, tokens, max_new;
    bool vec;          // 16-byte loads of both are possible
};

int launch_append(const AppendArgs &a, cudaStream_t s);
int launch_attend_decode(const AttendArgs &a, cudaStream_t s);
int launch_attend_prefill(const AttendArgs &a, cudaStream_t s);
int64_t decode_workspace(const AttendArgs &a);   // bytes of their scratch
int64_t prefill_workspace(const AttendArgs &a);
int launch_reserve(const bqd_kv_cache &c, const int32_t *counts, int32_t *base, int32_t *copies, int32_t *status,
                   cudaStream_t s);
int launch_fork(const bqd_kv_cache &from, const bqd_kv_cache &to, const int32_t *parents, const int32_t *keep,
                cudaStream_t s);
int launch_compact(const bqd_kv_cache &from, const bqd_kv_cache &to, int32_t *work, int32_t *moved, cudaStream_t s);
int launch_copy_pages(const bqd_kv_cache &c, const int32_t *src, const int32_t *dst, int64_t n, cudaStream_t s);

}  // namespace kv
}  // namespace bqd
