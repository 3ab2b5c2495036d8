// Drafts as a tree: ancestor masks, and greedy verification.
//
// Row r's nodes are tokens starts[r] .. starts[r + 1] - 1; parents[i] is the row's
// own index of node i's parent, below i; any other value makes node i a root.
//
// bqd_tree_mask: one thread a node walks up and sets the bits of what it passes, from
// the highest word down, since a parent's index is below its child's.  A row's nodes
// go in groups of 128, in order: a walk that leaves its group takes the rest from what
// the ancestor there already has, so that it is 128 steps at most, whatever the depth.
//
// bqd_spec_tree_verify: t[i] = argmax of node i's logits (ties: the smallest index;
// NaN is never chosen; -1 for a row of NaNs) in a first kernel, which is bound by
// HBM: a vector of 16 bytes costs three packed maxima and one comparison, and only
// the vector with the largest value is looked at again.  The CTAs of a cluster
// share a row of logits where there are few.  A second kernel, launched early,
// walks each tree with one warp: from node 0 to the lowest child whose token is t.
// 16 trees of 64 nodes, 151936 bf16 logits each: 55 us with the masks (5610 GB/s, 83% of a
// measured copy); one tree of 26 nodes 9.6 us in three launches.
#include <algorithm>
#include <climits>

#include "kv_common.cuh"
#include "logits.cuh"
#include "qmv_common.cuh"

namespace bqd {
namespace {

using namespace qmvdev;
using kv::Span;

constexpr int kThreadsT = 256;
constexpr int kMaxParts = 8;

__global__ void __launch_bounds__(128)
tree_mask_kernel(const int32_t *parents, const int32_t *starts, int tokens, int words, const int32_t *base, uint64_t *mask,
                 int32_t *depth, int32_t *positions)
{
    const int row = blockIdx.x;
    const Span span(starts, row, tokens, INT_MAX);
    for (int i0 = 0; i0 < span.n; i0 += 128) {
        if (i0 > 0) __syncthreads();  // the groups before are written
        const int i = i0 + threadIdx.x;
        if (i >= span.n) continue;    // (of the last group)
        uint64_t *to = mask ? mask + (int64_t)(span.lo + i) * words : nullptr;
        int word = words - 1, above = -1, at = i;
        uint64_t bits = 0;
        while (at >= i0) {
            ++above;
            if (to && (at >> 6) < words) {
                while (word > at >> 6) {
                    to[word--] = bits;
                    bits = 0;
                }
                bits |= (uint64_t)1 << (at & 63);
            }
            const int p = __ldg(parents + span.lo + at);
            at = p < at ? max(p, -1) : -1;
        }
        // an ancestor of an earlier group: its bits lie in words below this group's
        const int64_t up = at < 0 ? -1 : (int64_t)span.lo + at;
        if (to)
            while (word >= 0) {
                to[word] = up >= 0 && word < i0 >> 6 ? mask[up * words + word] : bits;
                bits = 0;
                --word;
            }
        if (up >= 0 && depth) above += 1 + depth[up];
        else if (up >= 0 && positions) above += 1 + positions[up] - base[row];
        if (depth) depth[span.lo + i] = above;
        if (positions) positions[span.lo + i] = base[row] + above;
    }
}

struct Best {
    float v;
    int i;  // INT_MAX: none
};

// larger value first, then the smaller index; NaN never wins
__device__ __forceinline__ bool better(const Best &a, const Best &b) { return a.v > b.v || (a.v == b.v && a.i < b.i); }

__device__ __forceinline__ Best best_of_block(Best b, Best *red)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Best x = {__shfl_down_sync(0xffffffffu, b.v, o), __shfl_down_sync(0xffffffffu, b.i, o)};
        if (better(x, b)) b = x;
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = b;
    __syncthreads();
    b = red[0];
#pragma unroll
    for (int w = 1; w < kThreadsT / 32; ++w)
        if (better(red[w], b)) b = red[w];
    __syncthreads();
    return b;
}

template <typename T>
__global__ void __launch_bounds__(kThreadsT)
argmax_kernel(const T *logits, int64_t stride, int V, int parts, int32_t *out)
{
    using X = lg::Vec<T>;
    __shared__ Best red[kThreadsT / 32];
    __shared__ Best mine;
    const int part = parts > 1 ? (int)cluster_ctarank() : 0, tid = threadIdx.x;
    const int64_t r = blockIdx.x / parts;
    const T *row = logits + r * stride;
    pdl_launch_dependents();
    const lg::Part<T> p(row, V, part, parts);
    // values around the vectors by their index; a vector by its first value's
    Best one = {-INFINITY, INT_MAX}, vec = {-INFINITY, INT_MAX};
    if (tid < p.head) one = Best{X::one(row + tid), tid};
    if (tid < p.tail) {
        const Best x = {X::one(row + p.tail_at + tid), p.tail_at + tid};
        if (!(one.v == one.v) || better(x, one)) one = x;
    }
    int q = p.q0 + tid;
    constexpr int U = 8;
    for (; q + (U - 1) * kThreadsT < p.q1; q += U * kThreadsT) {
        uint4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) u[j] = __ldcs(p.body + q + j * kThreadsT);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const float m = X::max(u[j]);
            if (m > vec.v) vec.v = m, vec.i = q + j * kThreadsT;
        }
    }
    for (; q < p.q1; q += kThreadsT) {
        const float m = X::max(__ldcs(p.body + q));
        if (m > vec.v) vec.v = m, vec.i = q;
    }
    vec = best_of_block(vec, red);
    one = best_of_block(one.v > -INFINITY ? one : Best{-INFINITY, INT_MAX}, red);
    if (tid == 0) {
        Best b = {vec.v, INT_MAX};
        if (vec.i != INT_MAX) {
            float x[X::E];
            X::values(p.body[vec.i], x);
#pragma unroll
            for (int e = X::E - 1; e >= 0; --e)
                if (x[e] == vec.v) b.i = p.first + vec.i * X::E + e;
        }
        if (better(one, b)) b = one;
        mine = b;
    }
    Best b;
    if (parts > 1) {
        cluster_sync();
        b = mine;
        if (part == 0) {
            for (int k = 1; k < parts; ++k) {
                uint32_t at;
                Best x;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&mine)), "r"(k));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x.v) : "r"(at) : "memory");
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x.i) : "r"(at + 4) : "memory");
                if (better(x, b)) b = x;
            }
        }
        cluster_sync();  // no CTA leaves while another reads its shared memory
        if (part != 0) return;
    } else {
        __syncthreads();
        b = mine;
    }
    if (b.i == INT_MAX) {
        // nothing above -infinity: the first -infinity
        Best x = {-INFINITY, INT_MAX};
        for (int i = tid; i < V && x.i == INT_MAX; i += kThreadsT)
            if (X::one(row + i) == -INFINITY) x.i = i;
        b = best_of_block(x, red);
    }
    if (tid == 0) out[r] = b.i == INT_MAX ? -1 : b.i;
}

__global__ void __launch_bounds__(32)
tree_walk_kernel(const int32_t *best, const int32_t *drafted, const int32_t *parents, const int32_t *starts, int tokens,
                 int max_path, int32_t *accepted, int32_t *next_token, int32_t *path)
{
    pdl_wait();
    const int row = blockIdx.x, lane = threadIdx.x;
    const Span span(starts, row, tokens, INT_MAX);
    int32_t *to = path + (int64_t)row * max_path;
    int length = 0, t = -1;
    for (int at = 0; at < span.n && length < max_path;) {
        if (lane == 0) to[length] = at;
        ++length;
        t = __ldcg(best + span.lo + at);
        int next = span.n;
        for (int i0 = at + 1; i0 < span.n && t >= 0; i0 += 32) {
            const int i = i0 + lane;
            const bool hit = i < span.n && __ldg(parents + span.lo + i) == at && __ldg(drafted + span.lo + i) == t;
            const unsigned hits = __ballot_sync(0xffffffffu, hit);
            if (hits) {
                next = i0 + __ffs(hits) - 1;
                break;
            }
        }
        at = next;
    }
    for (int k = length + lane; k < max_path; k += 32) to[k] = -1;
    if (lane == 0) {
        accepted[row] = max(0, length - 1);
        next_token[row] = t;
    }
}

template <typename T>
int launch_argmax(const void *logits, int64_t stride, int64_t tokens, int64_t V, int32_t *out, cudaStream_t s)
{
    // two CTAs an SM: 104 rows of 151936, 14.6 us; one, 16.5; four, 14.4, but 580 rows 36.9 and 38.5
    const int parts = lg::parts_of(tokens, V, 2 * (int64_t)sm_count(), kMaxParts);
    if (tokens * parts > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tokens * parts));
    cfg.blockDim = dim3(kThreadsT);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, argmax_kernel<T>, static_cast<const T *>(logits), stride, (int)V, parts, out));
}

bool at(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace
}  // namespace bqd

extern "C" int bqd_tree_mask(const int32_t *parents, const int32_t *starts, int64_t rows, int64_t tokens, int words,
                             const int32_t *base, uint64_t *mask, int32_t *depth, int32_t *positions, bqd_stream_t stream)
{
    using namespace bqd;
    if (rows < 0 || rows > 0x7FFFFFFF || tokens < 0 || tokens > ((int64_t)1 << 30)) return BQD_ERR_INVALID_ARG;
    if (words < 1 || words > BQD_TREE_MAX_WORDS || (positions && !base)) return BQD_ERR_INVALID_ARG;
    if (rows == 0 || tokens == 0 || (!mask && !depth && !positions)) return BQD_OK;
    if (!parents || !starts) return BQD_ERR_INVALID_ARG;
    if (!at(parents, 4) || !at(starts, 4) || !at(base, 4) || !at(mask, 8) || !at(depth, 4) || !at(positions, 4))
        return BQD_ERR_ALIGNMENT;
    tree_mask_kernel<<<(unsigned)rows, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        parents, starts, (int)tokens, words, base, mask, depth, positions);
    return cuda_status(cudaGetLastError());
}

extern "C" int bqd_spec_tree_verify(const void *logits, int dtype, int64_t row_stride, int64_t V, const int32_t *drafted,
                                    const int32_t *parents, const int32_t *starts, int64_t rows, int64_t tokens,
                                    int max_path, int32_t *accepted, int32_t *next_token, int32_t *path,
                                    int32_t *argmax_out, bqd_stream_t stream)
{
    using namespace bqd;
    if (dtype != BQD_DTYPE_F16 && dtype != BQD_DTYPE_F32 && dtype != BQD_DTYPE_BF16) return BQD_ERR_INVALID_ARG;
    if (rows < 0 || rows > 0x7FFFFFFF || tokens < 0 || tokens > ((int64_t)1 << 28) || V < 1 || V > ((int64_t)1 << 31) - 1024)
        return BQD_ERR_INVALID_ARG;
    if (max_path < 1 || (tokens > 1 && row_stride < V) || row_stride > ((int64_t)1 << 40)) return BQD_ERR_INVALID_ARG;
    if (rows == 0) return BQD_OK;
    if (!starts || !accepted || !next_token || !path) return BQD_ERR_INVALID_ARG;
    if (tokens > 0 && (!logits || !drafted || !parents || !argmax_out)) return BQD_ERR_INVALID_ARG;
    if (!at(logits, dtype == BQD_DTYPE_F32 ? 4 : 2) || !at(drafted, 4) || !at(parents, 4) || !at(starts, 4) ||
        !at(accepted, 4) || !at(next_token, 4) || !at(path, 4) || !at(argmax_out, 4))
        return BQD_ERR_ALIGNMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (tokens > 0) {
        const int st = dtype == BQD_DTYPE_F16    ? launch_argmax<__half>(logits, row_stride, tokens, V, argmax_out, s)
                       : dtype == BQD_DTYPE_BF16 ? launch_argmax<__nv_bfloat16>(logits, row_stride, tokens, V, argmax_out, s)
                                                 : launch_argmax<float>(logits, row_stride, tokens, V, argmax_out, s);
        if (st != BQD_OK) return st;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = tokens > 0 ? 1 : 0;  // without the first kernel this one waits for whatever came before
    return cuda_status(cudaLaunchKernelEx(&cfg, tree_walk_kernel, static_cast<const int32_t *>(argmax_out), drafted, parents, starts,
                                          (int)tokens, max_path, accepted, next_token, path));
}
