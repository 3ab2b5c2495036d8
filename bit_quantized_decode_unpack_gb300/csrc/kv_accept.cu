// Acceptance of a drafted tree's path: the cache keeps the tokens that the path
// names, moved to the front of the row's nodes, in every layer.
//
// Path entries rise, so a token moves to its own place or a lower one, and the
// sources of a block lie in that block or later ones: blocks are handled in
// rising order, each with all of its tokens in registers before any is written.
//   s' = max of the scales of the tokens that the block then holds,
//   code' = code where its scale is s', else rnd(fp32(fp32(code s) fp32(1 / s')))
// A row with fewer tokens than nodes has a node for each token, from its first one.
// One warp owns (row, layer, head, K or V): nothing is shared, no atomics.  Blocks
// before the first entry that moves keep what they have.  A path is a few tokens:
// the time is the chain of path, table, codes, and the launches: one row in 4 layers 5 us with
// the new table, 32 rows in 8 layers 9.5 us.
#include <algorithm>

#include "kv_common.cuh"

namespace bqd {
namespace kv {
namespace {

constexpr int kWarpsC = 8;

struct AcceptParams {
    Layer L;                      // the first layer
    int64_t layer_codes, layer_scales;
    int layers;
    const int32_t *path, *starts;
    int width;
    int32_t *keep;                // [rows]: the rows' new lengths
};

template <int D, int FMT>
__global__ void __launch_bounds__(kWarpsC * 32)
accept_kernel(const AcceptParams p)
{
    constexpr int kRowLanes = D / 16;          // lanes of one token (16 codes each)
    constexpr int kRowsPass = 32 / kRowLanes;  // tokens of one pass of the warp
    constexpr int kPasses = kBlock / kRowsPass;
    using C = Code<FMT>;
    const int lane = threadIdx.x & 31;
    // unit: head fastest, then K / V, then layer, then row
    const int64_t unit = (int64_t)blockIdx.x * kWarpsC + (threadIdx.x >> 5);
    const int head = (int)(unit % p.L.heads);
    int64_t u = unit / p.L.heads;
    const int which = (int)(u & 1);
    u >>= 1;
    const int layer = (int)(u % p.layers);
    const int64_t row64 = u / p.layers;
    if (row64 >= p.L.rows) return;
    const int row = (int)row64;
    const int length = p.L.length(row);
    const int n = p.starts ? (int)max((int64_t)0, min((int64_t)p.starts[row + 1] - p.starts[row], (int64_t)length))
                           : min(1, length);
    const bool tells = layer == 0 && which == 0 && head == 0 && lane == 0;
    if (n == 0) {
        if (tells) p.keep[row] = length;
        return;
    }
    const int base = length - n;
    const int32_t *path = p.path + (int64_t)row * p.width;
    // entries that rise within [0, n), and the first that is not its own place
    int kept = 0, first = -1;
    for (int k0 = 0, last = -1; k0 < p.width; k0 += 32) {
        const int k = k0 + lane;
        const int at = k < p.width ? path[k] : -1;
        int before = __shfl_up_sync(0xffffffffu, at, 1);
        if (lane == 0) before = last;
        const unsigned bad = __ballot_sync(0xffffffffu, at <= before || at >= n);
        const int good = bad ? __ffs(bad) - 1 : 32;
        const unsigned moves = __ballot_sync(0xffffffffu, at != k) & (good < 32 ? (1u << good) - 1 : 0xffffffffu);
        if (first < 0 && moves) first = k0 + __ffs(moves) - 1;
        kept += good;
        if (good < 32) break;
        last = __shfl_sync(0xffffffffu, at, 31);
    }
    if (tells) p.keep[row] = base + kept;
    if (first < 0) return;

    uint8_t *codes = (which ? p.L.v : p.L.k) + layer * p.layer_codes;
    float *scales = (which ? p.L.vs : p.L.ks) + layer * p.layer_scales;
    const int r0 = lane / kRowLanes, col = (lane % kRowLanes) * 16;
    const int end = base + kept;
    for (int t0 = (base + first) / kBlock * kBlock; t0 < end; t0 += kBlock) {
        uint4 x[kPasses];
        float s[kPasses];
        bool moved[kPasses];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int t = t0 + i * kRowsPass + r0;
            x[i] = make_uint4(0, 0, 0, 0), s[i] = 0.0f, moved[i] = false;
            if (t < end) {
                const int from = t < base ? t : base + path[t - base];
                const int64_t blk = p.L.block_of(row, head, from);
                x[i] = *reinterpret_cast<const uint4 *>(codes + (blk * kBlock + (from & (kBlock - 1))) * D + col);
                s[i] = scales[blk];
                moved[i] = from != t;
            }
            top = fmaxf(top, s[i]);
        }
#pragma unroll
        for (int o = kRowLanes; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        __syncwarp();  // everything is read before anything is written
        const int page = p.L.listed(row, t0);
        if ((unsigned)page < (unsigned)p.L.pages) {
            const int64_t blk = p.L.block_at(page, head, t0);
            const float inv = __frcp_rn(top);
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int t = t0 + i * kRowsPass + r0;
                if (t >= end || (!moved[i] && s[i] == top)) continue;
                if (s[i] != top) {
                    uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float f[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[e] = tame<FMT>(__fmul_rn(__fmul_rn(C::value((w[j] >> (8 * e)) & 0xFF), s[i]), inv));
                        w[j] = encode4<FMT>(f[0], f[1], f[2], f[3]);
                    }
                    x[i] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                *reinterpret_cast<uint4 *>(codes + (blk * kBlock + (t & (kBlock - 1))) * D + col) = x[i];
            }
            if (lane == 0) scales[blk] = top;
        }
        __syncwarp();
    }
}

template <int FMT>
int launch_f(const AcceptParams &p, int head_dim, cudaStream_t s)
{
    const int64_t units = (int64_t)p.L.rows * p.layers * 2 * p.L.heads, grid = (units + kWarpsC - 1) / kWarpsC;
    if (grid > 0x7FFFFFFF) return BQD_ERR_INVALID_ARG;
    if (head_dim == 64) accept_kernel<64, FMT><<<(unsigned)grid, kWarpsC * 32, 0, s>>>(p);
    else if (head_dim == 128) accept_kernel<128, FMT><<<(unsigned)grid, kWarpsC * 32, 0, s>>>(p);
    else accept_kernel<256, FMT><<<(unsigned)grid, kWarpsC * 32, 0, s>>>(p);
    return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_accept(const bqd_kv_cache &from, const bqd_kv_cache &to, const Layer &first, const int32_t *path, int width,
                  const int32_t *starts, cudaStream_t s)
{
    if (from.rows > 0) {
        AcceptParams p;
        p.L = first;
        p.layer_scales = from.pages * from.kv_heads * (from.page_tokens / kBlock);
        p.layer_codes = p.layer_scales * kBlock * from.head_dim;
        p.layers = from.layers;
        p.path = path, p.starts = starts, p.width = width;
        p.keep = to.lens;
        const int st = from.format == BQD_KV_INT8 ? launch_f<BQD_KV_INT8>(p, from.head_dim, s)
                                                  : launch_f<BQD_KV_E4M3>(p, from.head_dim, s);
        if (st != BQD_OK) return st;
    }
    // the new lengths stand in to.lens already, and are written there again as they are
    return launch_fork(from, to, nullptr, to.lens, s);
}

}  // namespace kv
}  // namespace bqd
