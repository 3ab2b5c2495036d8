// Page operations of the KV cache: reserve (allocate, copy on write), fork
// (share, reorder, cut back, free), compact, copy.
//
// The whole state is table, lens and refs; a page is free when refs is 0.
// Allocation takes the lowest free indices in the order of the rows, found by
// an ordered scan of refs in one CTA, so the result is a function of the
// state alone and the pool stays dense without a free list.  The only atomics
// are integer counts, whose order does not matter.  Planning touches 4 bytes a
// page and a table entry and is bound by latency; moving pages is a copy bound
// by memory (16-byte accesses, 64 bytes a thread in flight): 525 MB of moves with
// their plan 97 us (5431 GB/s, 81% of a measured copy; about 8 us are the plan).
// 64 beams of 16 parents with their copies: 19 us on the GPU in three launches,
// 32 to 47 us a call of fork and reserve from Python, by the host.
#include <algorithm>

#include "kv_common.cuh"
#include "qmv_common.cuh"

namespace bqd {
namespace kv {
namespace {

constexpr int kThreadsP = 1024;
constexpr int kWarpsP = kThreadsP / 32;
constexpr int kScan = 4;           // pages a thread looks at between barriers
constexpr int kCopyThreads = 256;
constexpr int kUnit = 16384;       // bytes that a CTA copies at a time
// entries and pages up to which one CTA forks by itself: one launch instead of
// a copy and a launch
constexpr int64_t kSmallFork = 16384;

// Exclusive prefix of v over the CTA's threads; `sum` gets the total.
__device__ int block_prefix(int v, int *warp_sums, int &sum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    sum = warp_sums[kWarpsP - 1];
    const int before = warp ? warp_sums[warp - 1] : 0;
    __syncthreads();
    return before + x - v;
}

// Calls take(k, page) for the pages of [lo, hi) for which want(page) holds, in
// ascending order, k = first, first + 1, ...; stops once `most` have been
// seen.  Returns first + how many were found (before `most` it is exact).
template <typename Want, typename Take>
__device__ int ordered_scan(int lo, int hi, int first, int most, int *warp_sums, Want want, Take take)
{
    int seen = first;
    for (int64_t p0 = lo; p0 < hi && seen < most; p0 += kScan * kThreadsP) {
        // a thread looks at kScan consecutive pages
        int mask = 0;
        const int64_t mine = p0 + (int64_t)threadIdx.x * kScan;
#pragma unroll
        for (int i = 0; i < kScan; ++i)
            if (mine + i < hi && want((int)(mine + i))) mask |= 1 << i;
        int sum;
        int k = seen + block_prefix(__popc(mask), warp_sums, sum);
#pragma unroll
        for (int i = 0; i < kScan; ++i)
            if (mask >> i & 1) {
                if (k < most) take(k, (int)(mine + i));
                ++k;
            }
        seen += sum;
    }
    return seen;
}

struct ReserveParams {
    int32_t *table, *lens, *refs;
    const int32_t *counts;
    int32_t *base, *copies, *status;
    int pages, rows, row_pages, page_shift;
};

__global__ void __launch_bounds__(kThreadsP)
reserve_kernel(const ReserveParams p)
{
    qmvdev::pdl_launch_dependents();  // the copies' CTAs take their places and wait
    extern __shared__ int32_t dyn[];
    int32_t *last = dyn;               // [rows]: partly filled last page, or -1
    int32_t *before = dyn + p.rows;    // [rows]: pages given to the rows before
    __shared__ int warp_sums[kWarpsP];
    __shared__ int overflow;
    const int pt = 1 << p.page_shift, cap = p.row_pages << p.page_shift;
    auto length = [&](int r) { return max(0, min(p.lens[r], cap)); };
    auto count = [&](int r) { return p.counts ? max(0, min(p.counts[r], cap + 1)) : (p.lens[r] > 0 ? 1 : 0); };
    if (threadIdx.x == 0) overflow = 0;
    __syncthreads();
    for (int r = threadIdx.x; r < p.rows; r += kThreadsP) {
        const int len = length(r), n = count(r);
        int at = -1;
        if (n > 0 && (len & (pt - 1))) {
            at = p.table[(int64_t)r * p.row_pages + (len >> p.page_shift)];
            if ((unsigned)at >= (unsigned)p.pages) at = -1;
        }
        last[r] = at;
        if (n > cap - len) atomicAdd(&overflow, 1);
    }
    __syncthreads();
    // rows in blocks of consecutive ones a thread: the prefix follows the rows
    const int per = (p.rows + kThreadsP - 1) / kThreadsP;
    const int r0 = min(p.rows, (int)threadIdx.x * per), r1 = min(p.rows, r0 + per);
    int mine = 0;
    for (int r = r0; r < r1; ++r) {
        const int len = length(r), n = count(r);
        int need = 0;
        if (n > 0 && n <= cap - len) {
            need = ((len + n + pt - 1) >> p.page_shift) - ((len + pt - 1) >> p.page_shift);
            const int at = last[r];
            if (at >= 0 && p.refs[at] > 1) {
                // kept by the first of the rows that end in it if they are all its references
                int same = 0;
                bool is_first = true;
                for (int o = 0; o < p.rows; ++o) {
                    if (last[o] != at) continue;
                    ++same;
                    if (o < r) is_first = false;
                }
                if (!(is_first && same == p.refs[at])) ++need;
            }
        }
        before[r] = need;
        mine += need;
    }
    int total;
    int at = block_prefix(mine, warp_sums, total);
    for (int r = r0; r < r1; ++r) {
        const int need = before[r];
        before[r] = at;
        at += need;
    }
    __syncthreads();
    auto need_of = [&](int r) { return (r + 1 < p.rows ? before[r + 1] : total) - before[r]; };
    auto is_free = [&](int q) { return p.refs[q] == 0; };
    const int found = ordered_scan(0, p.pages, 0, total, warp_sums, is_free, [](int, int) {});
    const bool ok = found >= total && overflow == 0;
    if (threadIdx.x == 0) {
        p.status[0] = max(0, total - found);
        p.status[1] = overflow;
    }
    if (!ok) {
        for (int r = threadIdx.x; r < p.rows; r += kThreadsP) {
            p.base[r] = -1;
            p.copies[2 * r] = p.copies[2 * r + 1] = -1;
        }
        return;
    }
    // slots of a row that get new pages: the replaced last page first, if any
    ordered_scan(0, p.pages, 0, total, warp_sums, is_free, [&](int k, int page) {
        int lo = 0, hi = p.rows - 1;  // the last row with before <= k (rows without need share their value)
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= k) lo = mid;
            else hi = mid - 1;
        }
        const int len = length(lo), n = count(lo);
        const int end = (len + n + pt - 1) >> p.page_shift;
        p.table[(int64_t)lo * p.row_pages + end - need_of(lo) + (k - before[lo])] = page;
        p.refs[page] = 1;
        if (k == before[lo] && need_of(lo) > end - ((len + pt - 1) >> p.page_shift)) {
            p.copies[2 * lo] = last[lo];
            p.copies[2 * lo + 1] = page;
        }
    });
    __syncthreads();
    for (int r = threadIdx.x; r < p.rows; r += kThreadsP) {
        const int len = length(r), n = count(r);
        const bool copied = need_of(r) > ((len + n + pt - 1) >> p.page_shift) - ((len + pt - 1) >> p.page_shift);
        if (copied) atomicSub(&p.refs[last[r]], 1);
        else p.copies[2 * r] = p.copies[2 * r + 1] = -1;
        p.base[r] = len;
        p.lens[r] = len + n;
    }
}

struct Pools {
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t page_bytes, page_scales;    // of one page of one layer
    int64_t layer_bytes, layer_scales;  // of one layer
    int layers, pages;
};

// Units of copying one page: each layer's K and V in pieces of kUnit bytes
// (the first piece brings the scales).
__host__ __device__ inline int64_t units_of(const Pools &p)
{
    return (int64_t)p.layers * 2 * ((p.page_bytes + kUnit - 1) / kUnit);
}

__device__ void copy_unit(const Pools &p, int src, int dst, int64_t unit)
{
    const int64_t pieces = (p.page_bytes + kUnit - 1) / kUnit;
    const int64_t piece = unit % pieces;
    const int which = (int)(unit / pieces) & 1;
    const int64_t layer = unit / pieces / 2;
    uint8_t *pool = (which ? p.v : p.k) + layer * p.layer_bytes;
    const uint8_t *from = pool + src * p.page_bytes + piece * kUnit;
    uint8_t *to = pool + dst * p.page_bytes + piece * kUnit;
    const int n = (int)min((int64_t)kUnit, p.page_bytes - piece * kUnit) / 16;
    constexpr int kEach = kUnit / 16 / kCopyThreads;
    uint4 x[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x + i * kCopyThreads;
        if (at < n) x[i] = *reinterpret_cast<const uint4 *>(from + 16 * at);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x + i * kCopyThreads;
        if (at < n) *reinterpret_cast<uint4 *>(to + 16 * at) = x[i];
    }
    if (piece == 0) {
        float *s = (which ? p.vs : p.ks) + layer * p.layer_scales;
        for (int i = threadIdx.x; i < p.page_scales; i += kCopyThreads)
            s[dst * p.page_scales + i] = s[src * p.page_scales + i];
    }
}

// Pairs (src[i * stride], dst[i * stride]), i < n (or *count).
__global__ void __launch_bounds__(kCopyThreads)
copy_pages_kernel(const Pools p, const int32_t *src, const int32_t *dst, int stride, int64_t n)
{
    qmvdev::pdl_wait();
    const int64_t per = units_of(p);
    for (int64_t u = blockIdx.x; u < n * per; u += gridDim.x) {
        const int64_t i = u / per;
        const int s = src[i * stride], d = dst[i * stride];
        if ((unsigned)s >= (unsigned)p.pages || (unsigned)d >= (unsigned)p.pages) continue;
        copy_unit(p, s, d, u % per);
    }
}

struct ForkParams {
    const int32_t *table, *lens;   // old rows
    int32_t *new_table, *new_lens, *refs;
    const int32_t *parents, *keep;
    int rows, new_rows, row_pages, page_shift, pages;
};

// What entry e of the old rows' tables, then of the new rows', does to the counts
__device__ __forceinline__ void fork_entry(const ForkParams &p, int64_t e)
{
    const int64_t old_n = (int64_t)p.rows * p.row_pages;
    const int pt = 1 << p.page_shift, cap = p.row_pages << p.page_shift;
    if (e < old_n) {
        const int r = (int)(e / p.row_pages), j = (int)(e % p.row_pages);
        const int len = max(0, min(p.lens[r], cap));
        if (j >= (len + pt - 1) >> p.page_shift) return;
        const int page = p.table[e];
        if ((unsigned)page < (unsigned)p.pages) atomicSub(&p.refs[page], 1);
    } else {
        const int64_t f = e - old_n;
        const int i = (int)(f / p.row_pages), j = (int)(f % p.row_pages);
        const int par = p.parents[i];
        int len = 0;
        if ((unsigned)par < (unsigned)p.rows) {
            len = max(0, min(p.lens[par], cap));
            if (p.keep) len = max(0, min(len, p.keep[i]));
        }
        int page = -1;
        if (j < (len + pt - 1) >> p.page_shift) page = p.table[(int64_t)par * p.row_pages + j];
        p.new_table[f] = page;
        if (j == 0) p.new_lens[i] = len;
        if ((unsigned)page < (unsigned)p.pages) atomicAdd(&p.refs[page], 1);
    }
}

// refs already holds the old counts: take away what the old rows name, add
// what the new rows name
__global__ void fork_kernel(const ForkParams p)
{
    const int64_t n = ((int64_t)p.rows + p.new_rows) * p.row_pages;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x)
        fork_entry(p, e);
}

// The same with the copy of the old counts, in one CTA
__global__ void __launch_bounds__(kThreadsP) fork_small_kernel(const ForkParams p, const int32_t *old_refs)
{
    for (int i = threadIdx.x; i < p.pages; i += kThreadsP) p.refs[i] = old_refs[i];
    __syncthreads();
    const int n = (p.rows + p.new_rows) * p.row_pages;
    for (int e = threadIdx.x; e < n; e += kThreadsP) fork_entry(p, e);
}

struct CompactParams {
    const int32_t *table, *lens, *refs;
    int32_t *new_table, *new_lens, *new_refs;
    int32_t *work;   // [pages]: pairs (from, to); [pages]: new index of each live page
    int32_t *moved;
    int pages, rows, row_pages, page_shift;
};

__global__ void __launch_bounds__(kThreadsP)
compact_plan_kernel(const CompactParams p)
{
    __shared__ int warp_sums[kWarpsP];
    int mine = 0, live;
    for (int q = threadIdx.x; q < p.pages; q += kThreadsP) mine += p.refs[q] > 0;
    block_prefix(mine, warp_sums, live);
    int32_t *to_of = p.work + p.pages;
    for (int q = threadIdx.x; q < p.pages; q += kThreadsP) {
        to_of[q] = q;
        p.new_refs[q] = q < live ? p.refs[q] : 0;
    }
    auto is_live = [&](int q) { return p.refs[q] > 0; };
    const int holes = ordered_scan(0, live, 0, p.pages, warp_sums, [&](int q) { return !is_live(q); },
                                   [&](int k, int q) { p.work[2 * k + 1] = q; });
    __syncthreads();
    ordered_scan(live, p.pages, 0, holes, warp_sums, is_live, [&](int k, int q) {
        const int to = p.work[2 * k + 1];
        p.work[2 * k] = q;
        to_of[q] = to;
        p.new_refs[to] = p.refs[q];
    });
    if (threadIdx.x == 0) *p.moved = holes;
}

__global__ void __launch_bounds__(kCopyThreads)
compact_apply_kernel(const CompactParams p, const Pools pools)
{
    const int pt = 1 << p.page_shift, cap = p.row_pages << p.page_shift;
    const int64_t entries = (int64_t)p.rows * p.row_pages;
    for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kCopyThreads) {
        const int r = (int)(e / p.row_pages), j = (int)(e % p.row_pages);
        const int len = max(0, min(p.lens[r], cap));
        int page = -1;
        if (j < (len + pt - 1) >> p.page_shift) {
            page = p.table[e];
            if ((unsigned)page < (unsigned)p.pages) page = p.work[p.pages + page];
        }
        p.new_table[e] = page;
        if (j == 0) p.new_lens[r] = p.lens[r];
    }
    const int64_t per = units_of(pools), n = *p.moved;
    for (int64_t u = blockIdx.x; u < n * per; u += gridDim.x) {
        const int64_t i = u / per;
        copy_unit(pools, p.work[2 * i], p.work[2 * i + 1], u % per);
    }
}

Pools pools_of(const bqd_kv_cache &c)
{
    Pools p;
    p.k = static_cast<uint8_t *>(c.k_codes);
    p.v = static_cast<uint8_t *>(c.v_codes);
    p.ks = c.k_scales;
    p.vs = c.v_scales;
    p.page_scales = (int64_t)c.kv_heads * (c.page_tokens / kBlock);
    p.page_bytes = p.page_scales * kBlock * c.head_dim;
    p.layer_bytes = p.page_bytes * c.pages;
    p.layer_scales = p.page_scales * c.pages;
    p.layers = c.layers;
    p.pages = (int)c.pages;
    return p;
}

int shift_of(int page_tokens)
{
    int s = 0;
    while ((1 << s) < page_tokens) ++s;
    return s;
}

// early: the kernel before it is the one that writes src and dst, and lets this
// one be launched while it runs
int launch_copy(const Pools &p, const int32_t *src, const int32_t *dst, int stride, int64_t n, cudaStream_t s,
                bool early = false)
{
    const int64_t units = n * units_of(p);
    if (units == 0) return BQD_OK;
    const unsigned grid = (unsigned)std::min<int64_t>(units, (int64_t)sm_count() * 64);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, copy_pages_kernel, p, src, dst, stride, n));
}

}  // namespace

int launch_reserve(const bqd_kv_cache &c, const int32_t *counts, int32_t *base, int32_t *copies, int32_t *status,
                   cudaStream_t s)
{
    ReserveParams p{c.table, c.lens, c.refs, counts, base, copies, status,
                    (int)c.pages, c.rows, c.row_pages, shift_of(c.page_tokens)};
    reserve_kernel<<<1, kThreadsP, 2 * sizeof(int32_t) * (size_t)c.rows, s>>>(p);
    const int st = cuda_status(cudaGetLastError());
    return st != BQD_OK ? st : launch_copy(pools_of(c), copies, copies + 1, 2, c.rows, s, true);
}

int launch_fork(const bqd_kv_cache &from, const bqd_kv_cache &to, const int32_t *parents, const int32_t *keep,
                cudaStream_t s)
{
    ForkParams p{from.table, from.lens, to.table, to.lens, to.refs, parents, keep,
                 from.rows, to.rows, from.row_pages, shift_of(from.page_tokens), (int)from.pages};
    const int64_t entries = ((int64_t)from.rows + to.rows) * from.row_pages;
    if (entries + from.pages <= kSmallFork) {
        fork_small_kernel<<<1, kThreadsP, 0, s>>>(p, from.refs);
        return cuda_status(cudaGetLastError());
    }
    if (cudaMemcpyAsync(to.refs, from.refs, sizeof(int32_t) * (size_t)from.pages, cudaMemcpyDeviceToDevice, s) !=
        cudaSuccess)
        return BQD_ERR_CUDA;
    if (entries == 0) return BQD_OK;
    const unsigned grid = (unsigned)std::min<int64_t>((entries + 255) / 256, (int64_t)sm_count() * 32);
    fork_kernel<<<grid, 256, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}

int launch_compact(const bqd_kv_cache &from, const bqd_kv_cache &to, int32_t *work, int32_t *moved, cudaStream_t s)
{
    CompactParams p{from.table, from.lens, from.refs, to.table, to.lens, to.refs, work, moved,
                    (int)from.pages, from.rows, from.row_pages, shift_of(from.page_tokens)};
    compact_plan_kernel<<<1, kThreadsP, 0, s>>>(p);
    int st = cuda_status(cudaGetLastError());
    if (st != BQD_OK) return st;
    // the number of pages to move is device data: a grid that fills the GPU, and loops
    compact_apply_kernel<<<(unsigned)sm_count() * 8, kCopyThreads, 0, s>>>(p, pools_of(from));
    return cuda_status(cudaGetLastError());
}

int launch_copy_pages(const bqd_kv_cache &c, const int32_t *src, const int32_t *dst, int64_t n, cudaStream_t s)
{
    return launch_copy(pools_of(c), src, dst, 1, n, s);
}

}  // namespace kv
}  // namespace bqd
