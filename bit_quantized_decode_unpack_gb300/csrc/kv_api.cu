// Host side of the KV cache's C ABI: argument validation, then the launchers.
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"

using namespace bqd;
using namespace bqd::kv;

namespace {

bool at(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Status of a cache's sizes and pointers.  A cache of no rows needs no table.
int check_cache(const bqd_kv_cache *c)
{
    if (!c) return BQD_ERR_INVALID_ARG;
    if (c->format != BQD_KV_INT8 && c->format != BQD_KV_E4M3) return BQD_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BQD_ERR_INVALID_ARG;
    const int pt = c->page_tokens;
    if (pt != 16 && pt != 32 && pt != 64 && pt != 128 && pt != 256) return BQD_ERR_INVALID_ARG;
    if (c->layers < 1 || c->kv_heads < 1 || c->kv_heads > 65535) return BQD_ERR_INVALID_ARG;
    if (c->pages < 1 || c->pages >= ((int64_t)1 << 30)) return BQD_ERR_INVALID_ARG;
    if (c->rows < 0 || c->rows > 65535 || c->row_pages < 1) return BQD_ERR_INVALID_ARG;
    if ((int64_t)c->row_pages * pt >= ((int64_t)1 << 30)) return BQD_ERR_INVALID_ARG;
    // bytes of a pool stay far below 2^63
    if ((double)c->layers * (double)c->pages * c->kv_heads * pt * c->head_dim > 1e15) return BQD_ERR_INVALID_ARG;
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->refs) return BQD_ERR_INVALID_ARG;
    if (c->rows > 0 && (!c->table || !c->lens)) return BQD_ERR_INVALID_ARG;
    if (!at(c->k_codes, 16) || !at(c->v_codes, 16) || !at(c->k_scales, 4) || !at(c->v_scales, 4) ||
        !at(c->table, 4) || !at(c->lens, 4) || !at(c->refs, 4))
        return BQD_ERR_ALIGNMENT;
    return BQD_OK;
}

Layer layer_of(const bqd_kv_cache &c, int layer)
{
    const int64_t blocks = (int64_t)c.pages * c.kv_heads * (c.page_tokens / kBlock);
    Layer L;
    L.k = static_cast<uint8_t *>(c.k_codes) + layer * blocks * kBlock * c.head_dim;
    L.v = static_cast<uint8_t *>(c.v_codes) + layer * blocks * kBlock * c.head_dim;
    L.ks = c.k_scales + layer * blocks;
    L.vs = c.v_scales + layer * blocks;
    L.table = c.table;
    L.lens = c.lens;
    L.pages = (int)c.pages;
    L.heads = c.kv_heads;
    L.rows = c.rows;
    L.row_pages = c.row_pages;
    L.page_shift = 0;
    while ((1 << L.page_shift) < c.page_tokens) ++L.page_shift;
    return L;
}

bool half_type(int dtype) { return dtype == BQD_DTYPE_F16 || dtype == BQD_DTYPE_BF16; }

// sizes of a ragged batch: tokens and the bound of a row's new ones
bool check_tokens(const bqd_kv_cache &c, const int32_t *starts, int64_t tokens, int64_t max_new)
{
    const int64_t most = (int64_t)1 << 30;
    if (tokens < 0 || tokens > most || max_new < 0 || max_new > most) return false;
    return starts ? true : (tokens == c.rows && max_new >= 1);
}

bool strides_ok(int64_t tokens, int64_t ts, int64_t heads, int64_t hs)
{
    const int64_t most = (int64_t)1 << 40;
    return ts >= 0 && hs >= 0 && ts < most && hs < most && (double)tokens * (double)ts < 1e17 &&
           (double)heads * (double)hs < 1e17;
}

// 16-byte accesses of a strided tensor of 2-byte elements
bool vec_ok(const void *p, int64_t ts, int64_t hs) { return at(p, 16) && ts % 8 == 0 && hs % 8 == 0; }

// two states of one cache: same pools and sizes, separate tables
bool same_pools(const bqd_kv_cache &a, const bqd_kv_cache &b)
{
    return a.k_codes == b.k_codes && a.v_codes == b.v_codes && a.k_scales == b.k_scales && a.v_scales == b.v_scales &&
           a.pages == b.pages && a.layers == b.layers && a.kv_heads == b.kv_heads && a.head_dim == b.head_dim &&
           a.page_tokens == b.page_tokens && a.row_pages == b.row_pages && a.format == b.format && a.refs != b.refs &&
           (!a.table || a.table != b.table) && (!a.lens || a.lens != b.lens);
}

int planned_length(const bqd_kv_cache &c, int64_t max_len)
{
    const int64_t capacity = (int64_t)c.row_pages * c.page_tokens;
    return (int)(max_len > 0 && max_len < capacity ? max_len : capacity);
}

// Queries enough for 128-row tiles on tcgen05.  The other kernel reads the keys
// once for each 16 (query, head) columns (8 with head_dim 256).  Measured with 8
// sequences of 8000 tokens, head_dim 64 / 128, it takes 53 / 86 us at 48 columns and
// 65 / 118 at 54; the tiles 56 / 81 at any.  With head_dim 256 it takes 73 us at 24
// columns, 93 at 30 and 113 at 36, the tiles 83; with one sequence 17, 19 and 20
// against 29 to 31.
bool many_queries(const AttendArgs &a) { return (int64_t)a.max_new * a.group > (a.head_dim == 256 ? 32 : 48); }

// Masked calls: the few-query kernel reads the keys once for each 16 (query, head) columns (8 with
// head_dim 256), the kernel of 128-row tiles once for each pair of tiles, and starts later.  Times in us
// with u the million (row, head, key) triples that the call is planned for, measured at 4 to 60 columns,
// one to 2000 rows of 200 to 65001 tokens (few / tiles at 48 columns, head_dim 128: 11 / 23 at one row of 700,
// 88 / 70 at 8 x 8000, 306 / 188 at 4 x 65001).  Work beyond a wave costs what starting it costs, which
// decides for many short rows (256 of 200 tokens: 181 / 322; of 4000: 1383 / 868).  The tokens given tell how
// many rows are live, about.  The tile kernel has a CTA for what the others could have been, the few-query
// kernel's shares pass them over (1024 rows, 8 of them live at 4000 tokens: 57 / 150) as long as it plans any.
// Over 660 shapes of three head sizes the choice takes 0.6% more than the better kernel, 61% at most.
bool many_rows(const AttendArgs &a)
{
    struct Cost {
        double few0, few, few_unit, few_idle, tile0, tile, pair, tile_unit, tile_idle;
    };
    Cost c = a.head_dim == 64    ? Cost{8, 32, 0.01, 0.0014, 17, 71, 114, 0.08, 0.009}
             : a.head_dim == 128 ? Cost{10, 48, 0.0175, 0.0014, 20, 80, 127, 0.13, 0.013}
                                 : Cost{9, 84, 0.0175, 0.0027, 24, 200, 400, 0.13, 0.013};
    if (a.L.rows <= kPlannedRows) c.few_idle = 0;
    else c.tile_idle = 0.005;  // (no plan to look up)
    const int64_t columns = (int64_t)a.max_new * a.group, each = a.head_dim == 256 ? 8 : 16, tiles = (columns + 127) / 128;
    const int64_t keys = a.window > 0 ? std::min<int64_t>(a.max_len, (int64_t)a.window + a.max_new) : a.max_len;
    const int64_t rows = std::min<int64_t>(a.L.rows, ((int64_t)a.tokens + a.max_new - 1) / a.max_new);
    const double units = (double)rows * a.L.heads, idle = (double)(a.L.rows - rows) * a.L.heads;
    const double u = 1e-6 * units * (double)keys, sms = sm_count();
    const double few_tiles = (double)((columns + each - 1) / each);
    const double ctas = (double)(a.head_dim == 256 ? tiles : (tiles + 1) / 2);
    const double few = c.few0 + c.few * u * few_tiles + c.few_unit * std::max(0.0, units * few_tiles - 2 * sms) +
                       c.few_idle * idle * few_tiles;
    const double tile = c.tile0 + u * (c.pair * (double)(tiles / 2) + c.tile * (double)(tiles % 2)) +
                        c.tile_unit * std::max(0.0, units * ctas - sms) + c.tile_idle * idle * ctas;
    return few > tile;
}

// bytes of scratch that a call is better with, or 0
int64_t scratch_need(const AttendArgs &a, bool masked)
{
    if (masked) return many_rows(a) ? masked_workspace(a) : decode_workspace(a);
    return many_queries(a) ? prefill_workspace(a) : decode_workspace(a);
}

cudaStream_t to_stream(bqd_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" int bqd_kv_append(const bqd_kv_cache *cache, int layer, const void *k, int64_t k_token_stride,
                             int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                             int dtype, const int32_t *base, const int32_t *starts, int64_t tokens, int64_t max_new,
                             bqd_stream_t stream)
{
    const int st = check_cache(cache);
    if (st != BQD_OK) return st;
    const bqd_kv_cache &c = *cache;
    if (layer < 0 || layer >= c.layers || !half_type(dtype)) return BQD_ERR_INVALID_ARG;
    if (!check_tokens(c, starts, tokens, max_new)) return BQD_ERR_INVALID_ARG;
    if (!strides_ok(tokens, k_token_stride, c.kv_heads, k_head_stride) ||
        !strides_ok(tokens, v_token_stride, c.kv_heads, v_head_stride))
        return BQD_ERR_INVALID_ARG;
    if (c.rows == 0 || tokens == 0 || max_new == 0) return BQD_OK;
    if (!k || !v || !base) return BQD_ERR_INVALID_ARG;
    if (!at(k, 2) || !at(v, 2) || !at(base, 4) || !at(starts, 4)) return BQD_ERR_ALIGNMENT;
    AppendArgs a;
    a.L = layer_of(c, layer);
    a.x[0] = k, a.x[1] = v;
    a.token_stride[0] = k_token_stride, a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride, a.head_stride[1] = v_head_stride;
    a.base = base, a.starts = starts;
    a.dtype = dtype, a.format = c.format, a.head_dim = c.head_dim;
    a.tokens = (int)tokens, a.max_new = starts ? (int)(max_new < tokens ? max_new : tokens) : 1;
    a.vec = vec_ok(k, k_token_stride, k_head_stride) && vec_ok(v, v_token_stride, v_head_stride);
    return launch_append(a, to_stream(stream));
}

namespace {

int64_t workspace_common(const bqd_kv_cache *cache, int q_heads, int64_t tokens, int64_t max_new, int64_t max_len,
                         int64_t window, bool masked)
{
    if (check_cache(cache) != BQD_OK) return 0;
    const bqd_kv_cache &c = *cache;
    const int64_t most = (int64_t)1 << 30;
    if (q_heads < c.kv_heads || q_heads % c.kv_heads != 0 || max_len < 0 || window < 0 || c.rows == 0) return 0;
    if (tokens < 1 || tokens > most || max_new < 1 || max_new > most) return 0;
    if (max_new > tokens) max_new = tokens;
    if (max_new * (q_heads / c.kv_heads) >= most) return 0;
    AttendArgs a;
    a.L = layer_of(c, 0);
    a.head_dim = c.head_dim;
    a.q_heads = q_heads;
    a.group = q_heads / c.kv_heads;
    a.tokens = (int)tokens;
    a.max_new = (int)max_new;
    a.max_len = planned_length(c, max_len);
    a.window = (int)(window < most ? window : 0);
    a.mask = nullptr, a.depth = nullptr, a.words = 0;
    return scratch_need(a, masked);
}

}  // namespace

extern "C" int64_t bqd_kv_attend_workspace(const bqd_kv_cache *cache, int q_heads, int64_t tokens, int64_t max_new,
                                           int64_t max_len, int64_t window)
{
    return workspace_common(cache, q_heads, tokens, max_new, max_len, window, false);
}

extern "C" int64_t bqd_kv_attend_masked_workspace(const bqd_kv_cache *cache, int q_heads, int64_t tokens, int64_t max_new,
                                                  int64_t max_len, int64_t window)
{
    return workspace_common(cache, q_heads, tokens, max_new, max_len, window, true);
}

namespace {

int attend_common(const bqd_kv_cache *cache, int layer, const void *q, int64_t q_token_stride, int64_t q_head_stride,
                  int dtype, int q_heads, const int32_t *starts, int64_t tokens, int64_t max_new, int64_t max_len,
                  float scale, int64_t window, const uint64_t *mask, int words, const int32_t *depth, void *out,
                  float *lse, void *work, int64_t work_bytes, bqd_stream_t stream)
{
    const int st = check_cache(cache);
    if (st != BQD_OK) return st;
    const bqd_kv_cache &c = *cache;
    if (layer < 0 || layer >= c.layers || !half_type(dtype)) return BQD_ERR_INVALID_ARG;
    if (q_heads < c.kv_heads || q_heads % c.kv_heads != 0) return BQD_ERR_INVALID_ARG;
    if (!check_tokens(c, starts, tokens, max_new) || !strides_ok(tokens, q_token_stride, q_heads, q_head_stride))
        return BQD_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || window < 0 || max_len < 0 || work_bytes < 0 || (!work && work_bytes > 0))
        return BQD_ERR_INVALID_ARG;
    if (c.rows == 0 || tokens == 0 || max_new == 0) return BQD_OK;
    const int64_t group = q_heads / c.kv_heads, most = (int64_t)1 << 30;
    if (!starts) max_new = 1;
    if (max_new > tokens) max_new = tokens;
    if (max_new * group >= most) return BQD_ERR_INVALID_ARG;
    if (!q || !out) return BQD_ERR_INVALID_ARG;
    if (!at(q, 2) || !at(out, 16) || !at(lse, 4) || !at(starts, 4) || !at(work, 16) || !at(mask, 8) || !at(depth, 4))
        return BQD_ERR_ALIGNMENT;
    AttendArgs a;
    a.L = layer_of(c, layer);
    a.q = q, a.q_token = q_token_stride, a.q_head = q_head_stride;
    a.starts = starts;
    a.out = out, a.lse = lse;
    a.scale = scale * 1.4426950408889634f;
    a.dtype = dtype, a.format = c.format, a.head_dim = c.head_dim;
    a.q_heads = q_heads, a.group = (int)group;
    a.tokens = (int)tokens, a.max_new = (int)max_new;
    a.max_len = planned_length(c, max_len);
    a.window = (int)(window < most ? window : 0);  // one past any position hides nothing
    a.q_vec = vec_ok(q, q_token_stride, q_head_stride);
    a.mask = mask, a.words = words, a.depth = depth;
    a.work = nullptr;
    const int64_t need = scratch_need(a, mask != nullptr);
    if (need > 0 && work_bytes >= need) a.work = work;
    if (mask) return many_rows(a) ? launch_attend_masked(a, to_stream(stream)) : launch_attend_decode(a, to_stream(stream));
    return many_queries(a) ? launch_attend_prefill(a, to_stream(stream)) : launch_attend_decode(a, to_stream(stream));
}

}  // namespace

extern "C" int bqd_kv_attend(const bqd_kv_cache *cache, int layer, const void *q, int64_t q_token_stride,
                             int64_t q_head_stride, int dtype, int q_heads, const int32_t *starts, int64_t tokens,
                             int64_t max_new, int64_t max_len, float scale, int64_t window, void *out, float *lse,
                             void *work, int64_t work_bytes, bqd_stream_t stream)
{
    return attend_common(cache, layer, q, q_token_stride, q_head_stride, dtype, q_heads, starts, tokens, max_new, max_len,
                         scale, window, nullptr, 0, nullptr, out, lse, work, work_bytes, stream);
}

extern "C" int bqd_kv_attend_masked(const bqd_kv_cache *cache, int layer, const void *q, int64_t q_token_stride,
                                    int64_t q_head_stride, int dtype, int q_heads, const int32_t *starts, int64_t tokens,
                                    int64_t max_new, int64_t max_len, float scale, int64_t window, const uint64_t *mask,
                                    int words, const int32_t *depth, void *out, float *lse, void *work,
                                    int64_t work_bytes, bqd_stream_t stream)
{
    if (words < 1 || words > BQD_TREE_MAX_WORDS || (window > 0 && !depth)) return BQD_ERR_INVALID_ARG;
    if (!mask && tokens > 0) return BQD_ERR_INVALID_ARG;
    return attend_common(cache, layer, q, q_token_stride, q_head_stride, dtype, q_heads, starts, tokens, max_new, max_len,
                         scale, window, mask, words, depth, out, lse, work, work_bytes, stream);
}

extern "C" int bqd_kv_reserve(const bqd_kv_cache *cache, const int32_t *counts, int32_t *base, int32_t *copies,
                              int32_t *status, bqd_stream_t stream)
{
    const int st = check_cache(cache);
    if (st != BQD_OK) return st;
    if (cache->rows > 4096 || !status) return BQD_ERR_INVALID_ARG;
    if (cache->rows > 0 && (!base || !copies)) return BQD_ERR_INVALID_ARG;
    if (!at(counts, 4) || !at(base, 4) || !at(copies, 4) || !at(status, 4)) return BQD_ERR_ALIGNMENT;
    if (cache->rows == 0) return cuda_status(cudaMemsetAsync(status, 0, 2 * sizeof(int32_t), to_stream(stream)));
    return launch_reserve(*cache, counts, base, copies, status, to_stream(stream));
}

extern "C" int bqd_kv_fork(const bqd_kv_cache *from, const bqd_kv_cache *to, const int32_t *parents,
                           const int32_t *keep, bqd_stream_t stream)
{
    int st = check_cache(from);
    if (st == BQD_OK) st = check_cache(to);
    if (st != BQD_OK) return st;
    if (!same_pools(*from, *to) || (to->rows > 0 && !parents)) return BQD_ERR_INVALID_ARG;
    if (!at(parents, 4) || !at(keep, 4)) return BQD_ERR_ALIGNMENT;
    return launch_fork(*from, *to, parents, keep, to_stream(stream));
}

extern "C" int bqd_kv_accept(const bqd_kv_cache *from, const bqd_kv_cache *to, const int32_t *path, int width,
                             const int32_t *starts, bqd_stream_t stream)
{
    int st = check_cache(from);
    if (st == BQD_OK) st = check_cache(to);
    if (st != BQD_OK) return st;
    if (!same_pools(*from, *to) || from->rows != to->rows || width < 1) return BQD_ERR_INVALID_ARG;
    if (from->rows > 0 && !path) return BQD_ERR_INVALID_ARG;
    if (!at(path, 4) || !at(starts, 4)) return BQD_ERR_ALIGNMENT;
    return launch_accept(*from, *to, layer_of(*from, 0), path, width, starts, to_stream(stream));
}

extern "C" int bqd_kv_compact(const bqd_kv_cache *from, const bqd_kv_cache *to, int32_t *work, int32_t *moved,
                              bqd_stream_t stream)
{
    int st = check_cache(from);
    if (st == BQD_OK) st = check_cache(to);
    if (st != BQD_OK) return st;
    if (!same_pools(*from, *to) || from->rows != to->rows || !work || !moved) return BQD_ERR_INVALID_ARG;
    if (!at(work, 4) || !at(moved, 4)) return BQD_ERR_ALIGNMENT;
    return launch_compact(*from, *to, work, moved, to_stream(stream));
}

extern "C" int bqd_kv_copy_pages(const bqd_kv_cache *cache, const int32_t *src, const int32_t *dst, int64_t n,
                                 bqd_stream_t stream)
{
    const int st = check_cache(cache);
    if (st != BQD_OK) return st;
    if (n < 0 || n > cache->pages) return BQD_ERR_INVALID_ARG;
    if (n == 0) return BQD_OK;
    if (!src || !dst) return BQD_ERR_INVALID_ARG;
    if (!at(src, 4) || !at(dst, 4)) return BQD_ERR_ALIGNMENT;
    return launch_copy_pages(*cache, src, dst, n, to_stream(stream));
}
