// C ABI of the attention layers over a paged cache: pool handles and argument
// checks.  The kernels are in attn_prologue.cu, attn_tc.cu, attn_f32.cu and kv_pages.cu.
#include <cmath>
#include <new>

#include "gdn_device.cuh"
#include "gdn_internal.h"

using gdn::api_cuda_fail;
using gdn::api_error_word;
using gdn::api_fail;
using gdn::api_ok;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t dtype_size(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

constexpr long long kMaxTokens = 1ll << 30; // a row's; positions and their tiles' ends stay within an int

bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128; }

int check_pool_geometry(int num_pages, int page_size, int layers, int hkv, int d, int dtype)
{
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return api_fail(GDN_EINVAL, "bad dtype %d", dtype);
    if (num_pages < 1 || layers < 1 || hkv < 1)
        return api_fail(GDN_EINVAL, "num_pages=%d layers=%d hkv=%d", num_pages, layers, hkv);
    if (!page_size_ok(page_size))
        return api_fail(GDN_EUNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", page_size);
    if (d != 64 && d != 128 && d != 256)
        return api_fail(GDN_EUNSUPPORTED, "d=%d (64, 128 or 256)", d);
    if ((double)num_pages * hkv * layers > 2147483647.0)
        return api_fail(GDN_EUNSUPPORTED, "layers * num_pages * hkv is over 2^31 - 1");
    return GDN_OK;
}

size_t layer_bytes(const kv_page_pool *p)
{
    return (size_t)p->num_pages * p->hkv * p->page_size * p->d * dtype_size(p->dtype);
}

gdn::PageView view(const kv_page_pool *p, int layer)
{
    gdn::PageView v;
    v.k = static_cast<char *>(p->k) + layer_bytes(p) * layer;
    v.v = static_cast<char *>(p->v) + layer_bytes(p) * layer;
    v.num_pages = p->num_pages;
    v.page_size = p->page_size;
    v.page_shift = 0;
    while ((1 << v.page_shift) < p->page_size)
        ++v.page_shift;
    v.hkv = p->hkv;
    v.d = p->d;
    v.layer = layer;
    return v;
}

// what attn_prologue and paged_attention check alike
int check_rows(const kv_page_pool *pool, int layer, const int32_t *table, int max_pages, const int32_t *seq_len,
               const int32_t *cu_seqlens, int hq, int rows, int total_tokens, int dtype)
{
    if (!pool)
        return api_fail(GDN_EINVAL, "pool is NULL");
    if (dtype != pool->dtype)
        return api_fail(GDN_EINVAL, "dtype %d, but the pool's is %d", dtype, pool->dtype);
    if (layer < 0 || layer >= pool->layers)
        return api_fail(GDN_EINVAL, "layer %d outside [0, %d)", layer, pool->layers);
    if (hq < 1 || hq % pool->hkv != 0)
        return api_fail(GDN_EINVAL, "hq=%d is not a multiple of hkv=%d", hq, pool->hkv);
    if (rows < 0 || total_tokens < 0 || (rows == 0 && total_tokens > 0))
        return api_fail(GDN_EINVAL, "rows=%d total_tokens=%d", rows, total_tokens);
    if (max_pages < 1)
        return api_fail(GDN_EINVAL, "max_pages=%d < 1", max_pages);
    if ((long long)max_pages * pool->page_size > kMaxTokens)
        return api_fail(GDN_EUNSUPPORTED, "max_pages=%d pages hold over 2^30 tokens", max_pages);
    if (total_tokens > 0 && (!table || !seq_len || !cu_seqlens))
        return api_fail(GDN_EINVAL, "table, seq_len and cu_seqlens must be non-NULL");
    return GDN_OK;
}

int check_stride(const char *what, const void *p, int64_t stride, int heads, int d, int dtype)
{
    if (!p)
        return api_fail(GDN_EINVAL, "%s is NULL", what);
    if (stride < (int64_t)heads * d)
        return api_fail(GDN_EINVAL, "%s: token stride %lld below %d heads of %d", what, (long long)stride, heads, d);
    if (!aligned16(p) || (stride * dtype_size(dtype)) % 16 != 0)
        return api_fail(GDN_EINVAL, "%s: address and token stride must be multiples of 16 bytes", what);
    return GDN_OK;
}

int check_tables(const int32_t *table, int table_rows, int max_pages, const int32_t *refs, int num_pages)
{
    if (!table || !refs)
        return api_fail(GDN_EINVAL, "table and refs must be non-NULL");
    if (table_rows < 1 || max_pages < 1 || num_pages < 1)
        return api_fail(GDN_EINVAL, "table_rows=%d max_pages=%d num_pages=%d", table_rows, max_pages, num_pages);
    return GDN_OK;
}

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? api_ok() : api_cuda_fail(e, what); }

size_t workspace_bytes_of(const kv_page_pool *pool, int hq, int rows, int total_tokens, bool shared)
{
    if (!pool || hq < 1 || hq % pool->hkv != 0 || rows < 1 || total_tokens < 1)
        return 0;
    return pool->dtype == GDN_BF16 ? gdn::attention_tc_workspace_bytes(pool->d, hq, pool->hkv, total_tokens, shared)
                                   : gdn::attention_f32_workspace_bytes(pool->d, hq, pool->hkv, total_tokens, shared);
}

// paged_attention (f NULL) and paged_attention_shared
int attention(const void *q, int64_t q_stride, kv_page_pool *pool, int layer, const int32_t *table, int max_pages,
              const int32_t *seq_len, const int32_t *cu_seqlens, const gdn::SharedPrefix *f, float scale, void *out, int hq,
              int rows, int total_tokens, void *workspace, size_t workspace_bytes, int dtype, void *stream, const char *what)
{
    int rc = check_rows(pool, layer, table, max_pages, seq_len, cu_seqlens, hq, rows, total_tokens, dtype);
    if (rc)
        return rc;
    if (!(scale > 0.f) || !std::isfinite(scale))
        return api_fail(GDN_EINVAL, "scale must be positive and finite");
    if (total_tokens == 0)
        return api_ok();
    if ((rc = check_stride("q", q, q_stride, hq, pool->d, dtype)))
        return rc;
    if (!out || !aligned16(out))
        return api_fail(GDN_EINVAL, "out must be non-NULL and 16-byte aligned");
    const size_t need = workspace_bytes_of(pool, hq, rows, total_tokens, f != nullptr);
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need))
        return api_fail(GDN_EINVAL, "workspace must be 16-byte aligned and hold %zu bytes (given %zu)", need,
                        workspace ? workspace_bytes : (size_t)0);
    gdn::AttentionArgs a = {};
    if ((rc = api_error_word(&a.err)))
        return rc;
    a.q = q, a.q_stride = q_stride;
    a.pages = view(pool, layer);
    a.c = {table, seq_len, cu_seqlens, max_pages, rows, total_tokens};
    a.scale = scale, a.out = out, a.hq = hq, a.work = workspace;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return launched(dtype == GDN_BF16 ? gdn::launch_paged_attention_tc(a, f, *pool, s) : gdn::launch_paged_attention_f32(a, f, s),
                    what);
}

} // namespace

extern "C" {

// ---- page pools -----------------------------------------------------------------

int kv_page_pool_wrap(void *k, void *v, int num_pages, int page_size, int layers, int hkv, int d, int dtype,
                      kv_page_pool **out)
{
    if (!out)
        return api_fail(GDN_EINVAL, "out is NULL");
    *out = nullptr;
    if (!k || !v)
        return api_fail(GDN_EINVAL, "k and v must be non-NULL");
    if (!aligned16(k) || !aligned16(v))
        return api_fail(GDN_EINVAL, "page pool memory must be 16-byte aligned");
    int rc = check_pool_geometry(num_pages, page_size, layers, hkv, d, dtype);
    if (rc)
        return rc;
    *out = new (std::nothrow) kv_page_pool(k, v, num_pages, page_size, layers, hkv, d, dtype, false);
    return *out ? api_ok() : api_fail(GDN_ENOMEM, "no host memory for a page pool handle");
}

int kv_page_pool_create(int num_pages, int page_size, int layers, int hkv, int d, int dtype, void *stream,
                        kv_page_pool **out)
{
    if (!out)
        return api_fail(GDN_EINVAL, "out is NULL");
    *out = nullptr;
    int rc = check_pool_geometry(num_pages, page_size, layers, hkv, d, dtype);
    if (rc)
        return rc;
    kv_page_pool *p = new (std::nothrow) kv_page_pool(nullptr, nullptr, num_pages, page_size, layers, hkv, d, dtype, true);
    if (!p)
        return api_fail(GDN_ENOMEM, "no host memory for a page pool handle");
    const size_t bytes = layer_bytes(p) * layers;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMalloc(&p->k, bytes);
    if (e == cudaSuccess)
        e = cudaMalloc(&p->v, bytes);
    if (e == cudaSuccess)
        e = cudaMemsetAsync(p->k, 0, bytes, s);
    if (e == cudaSuccess)
        e = cudaMemsetAsync(p->v, 0, bytes, s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) {
        cudaFree(p->k);
        cudaFree(p->v);
        delete p;
        if (e == cudaErrorMemoryAllocation) {
            cudaGetLastError();
            return api_fail(GDN_ENOMEM, "cudaMalloc(2 x %zu bytes) for the page pool failed", bytes);
        }
        return api_cuda_fail(e, "making the page pool");
    }
    *out = p;
    return api_ok();
}

int kv_page_pool_destroy(kv_page_pool *pool)
{
    if (!pool)
        return api_ok();
    cudaError_t e = cudaSuccess;
    if (pool->owned) {
        e = cudaFree(pool->k);
        const cudaError_t e2 = cudaFree(pool->v);
        if (e == cudaSuccess)
            e = e2;
    }
    delete pool;
    return launched(e, "cudaFree(page pool)");
}

void *kv_page_pool_k(const kv_page_pool *pool) { return pool ? pool->k : nullptr; }
void *kv_page_pool_v(const kv_page_pool *pool) { return pool ? pool->v : nullptr; }
int kv_page_pool_num_pages(const kv_page_pool *pool) { return pool ? pool->num_pages : 0; }

// ---- prologue ---------------------------------------------------------------------

int rope_table(const double *inv_freq, int rot, int positions, double mscale, float *table, void *stream)
{
    if (rot < 16 || rot % 16 != 0)
        return api_fail(GDN_EINVAL, "rot=%d is not a positive multiple of 16", rot);
    if (positions < 0)
        return api_fail(GDN_EINVAL, "positions=%d < 0", positions);
    if (!std::isfinite(mscale))
        return api_fail(GDN_EINVAL, "mscale is not finite");
    if (positions == 0)
        return api_ok();
    if (!inv_freq || !table)
        return api_fail(GDN_EINVAL, "inv_freq and table must be non-NULL");
    return launched(gdn::launch_rope_table(inv_freq, rot, positions, mscale, table, static_cast<cudaStream_t>(stream)),
                    "rope_table launch");
}

int attn_prologue(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                  kv_page_pool *pool, int layer, const float *rope, int rope_positions, int rot, int interleaved,
                  const float *q_norm, const float *k_norm, float eps, const int32_t *table, int max_pages,
                  const int32_t *seq_len, const int32_t *cu_seqlens, void *q_out, int hq, int rows,
                  int total_tokens, int dtype, void *stream)
{
    int rc = check_rows(pool, layer, table, max_pages, seq_len, cu_seqlens, hq, rows, total_tokens, dtype);
    if (rc)
        return rc;
    if (rot < 0 || rot % 16 != 0 || rot > pool->d)
        return api_fail(GDN_EINVAL, "rot=%d is not a multiple of 16 up to d=%d", rot, pool->d);
    if (rot > 0 && (!rope || !aligned16(rope) || rope_positions < 1))
        return api_fail(GDN_EINVAL, "rope must be a 16-byte aligned table of at least one position");
    if ((q_norm || k_norm) && !(eps >= 0.f && std::isfinite(eps)))
        return api_fail(GDN_EINVAL, "eps must be finite and not negative");
    if (!aligned16(q_norm) || !aligned16(k_norm))
        return api_fail(GDN_EINVAL, "q_norm and k_norm must be 16-byte aligned");
    if (total_tokens == 0)
        return api_ok();
    if ((rc = check_stride("q", q, q_stride, hq, pool->d, dtype)) ||
        (rc = check_stride("k", k, k_stride, pool->hkv, pool->d, dtype)) ||
        (rc = check_stride("v", v, v_stride, pool->hkv, pool->d, dtype)))
        return rc;
    if (!q_out || !aligned16(q_out))
        return api_fail(GDN_EINVAL, "q_out must be non-NULL and 16-byte aligned");
    gdn::PrologueArgs a = {};
    if ((rc = api_error_word(&a.err)))
        return rc;
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.pages = view(pool, layer);
    a.c = {table, seq_len, cu_seqlens, max_pages, rows, total_tokens};
    a.rope = rope, a.rope_positions = rope_positions, a.rot = rot, a.interleaved = interleaved != 0;
    a.q_norm = q_norm, a.k_norm = k_norm, a.eps = eps;
    a.q_out = q_out, a.hq = hq;
    return launched(gdn::launch_attn_prologue(a, dtype, static_cast<cudaStream_t>(stream)), "attn_prologue launch");
}

// ---- attention ----------------------------------------------------------------------

size_t paged_attention_workspace_bytes(const kv_page_pool *pool, int hq, int rows, int total_tokens)
{
    return workspace_bytes_of(pool, hq, rows, total_tokens, false);
}

int paged_attention(const void *q, int64_t q_stride, kv_page_pool *pool, int layer, const int32_t *table,
                    int max_pages, const int32_t *seq_len, const int32_t *cu_seqlens, float scale, void *out, int hq,
                    int rows, int total_tokens, void *workspace, size_t workspace_bytes, int dtype, void *stream)
{
    return attention(q, q_stride, pool, layer, table, max_pages, seq_len, cu_seqlens, nullptr, scale, out, hq, rows,
                     total_tokens, workspace, workspace_bytes, dtype, stream, "paged_attention launch");
}

size_t paged_attention_shared_workspace_bytes(const kv_page_pool *pool, int hq, int rows, int total_tokens)
{
    return workspace_bytes_of(pool, hq, rows, total_tokens, true);
}

int paged_attention_shared(const void *q, int64_t q_stride, kv_page_pool *pool, int layer, const int32_t *table,
                           int max_pages, const int32_t *seq_len, const int32_t *cu_seqlens, const int32_t *bounds,
                           int groups, const int32_t *prefix, float scale, void *out, int hq, int rows,
                           int total_tokens, void *workspace, size_t workspace_bytes, int dtype, void *stream)
{
    if (groups < (rows > 0) || groups > rows)
        return api_fail(GDN_EINVAL, "groups=%d for rows=%d: every row is in a group", groups, rows);
    if (total_tokens > 0 && (!bounds || !prefix))
        return api_fail(GDN_EINVAL, "bounds and prefix must be non-NULL");
    if (reinterpret_cast<uintptr_t>(prefix) & 7u)
        return api_fail(GDN_EINVAL, "prefix must be 8-byte aligned");
    const gdn::SharedPrefix f = {bounds, prefix, groups};
    return attention(q, q_stride, pool, layer, table, max_pages, seq_len, cu_seqlens, &f, scale, out, hq, rows,
                     total_tokens, workspace, workspace_bytes, dtype, stream, "paged_attention_shared launch");
}

int kv_pages_shared(const int32_t *table, int rows, int max_pages, const int32_t *seq_len, const int32_t *cu_seqlens,
                    const int32_t *bounds, int groups, int page_size, int32_t *prefix, void *stream)
{
    if (rows < 0 || max_pages < 1)
        return api_fail(GDN_EINVAL, "rows=%d max_pages=%d", rows, max_pages);
    if (!page_size_ok(page_size))
        return api_fail(GDN_EUNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", page_size);
    if ((long long)max_pages * page_size > kMaxTokens)
        return api_fail(GDN_EUNSUPPORTED, "max_pages=%d pages hold over 2^30 tokens", max_pages);
    if (groups < 0 || groups > rows)
        return api_fail(GDN_EINVAL, "groups=%d outside [0, rows=%d]", groups, rows);
    if (rows == 0)
        return api_ok();
    if (groups == 0)
        return api_fail(GDN_EINVAL, "groups=0 with rows=%d", rows);
    if (!table || !seq_len || !cu_seqlens || !bounds || !prefix)
        return api_fail(GDN_EINVAL, "table, seq_len, cu_seqlens, bounds and prefix must be non-NULL");
    if (reinterpret_cast<uintptr_t>(prefix) & 7u)
        return api_fail(GDN_EINVAL, "prefix must be 8-byte aligned");
    int *err = nullptr;
    int rc = api_error_word(&err);
    if (rc)
        return rc;
    const gdn::CacheRows c = {table, seq_len, cu_seqlens, max_pages, rows, 0};
    return launched(gdn::launch_pages_shared(c, bounds, groups, page_size, prefix, err, static_cast<cudaStream_t>(stream)),
                    "kv_pages_shared launch");
}

// ---- pages ----------------------------------------------------------------------------

int kv_pages_reserve(int32_t *table, int table_rows, int max_pages, int32_t *refs, int num_pages, int page_size,
                     const int32_t *list_rows, const int32_t *tokens, int n, int32_t *status, void *stream)
{
    int rc = check_tables(table, table_rows, max_pages, refs, num_pages);
    if (rc)
        return rc;
    if (!page_size_ok(page_size))
        return api_fail(GDN_EUNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", page_size);
    if ((long long)max_pages * page_size > kMaxTokens)
        return api_fail(GDN_EUNSUPPORTED, "max_pages=%d pages hold over 2^30 tokens", max_pages);
    if (n < 0 || n > GDN_MAX_PAGE_ROWS)
        return api_fail(GDN_EINVAL, "n=%d outside [0, %d]", n, GDN_MAX_PAGE_ROWS);
    if (n == 0)
        return api_ok();
    if (!list_rows || !tokens || !status)
        return api_fail(GDN_EINVAL, "list_rows, tokens and status must be non-NULL");
    gdn::PageTables t = {table, table_rows, max_pages, nullptr, refs, num_pages, page_size, nullptr};
    if ((rc = api_error_word(&t.err)))
        return rc;
    return launched(gdn::launch_pages_reserve(t, list_rows, tokens, n, status, static_cast<cudaStream_t>(stream)),
                    "kv_pages_reserve launch");
}

int kv_pages_fork(int32_t *table, int table_rows, int max_pages, int32_t *seq_len, int32_t *refs, int num_pages,
                  int page_size, const int32_t *src_rows, const int32_t *dst_rows, int n, int32_t *move_src,
                  int32_t *move_dst, int32_t *move_count, int32_t *status, void *stream)
{
    int rc = check_tables(table, table_rows, max_pages, refs, num_pages);
    if (rc)
        return rc;
    if (!page_size_ok(page_size))
        return api_fail(GDN_EUNSUPPORTED, "page_size=%d (16, 32, 64 or 128)", page_size);
    if ((long long)max_pages * page_size > kMaxTokens)
        return api_fail(GDN_EUNSUPPORTED, "max_pages=%d pages hold over 2^30 tokens", max_pages);
    if (n < 0 || n > GDN_MAX_PAGE_ROWS)
        return api_fail(GDN_EINVAL, "n=%d outside [0, %d]", n, GDN_MAX_PAGE_ROWS);
    if (!move_count)
        return api_fail(GDN_EINVAL, "move_count must be non-NULL");
    if (n > 0 && (!seq_len || !src_rows || !dst_rows || !move_src || !move_dst || !status))
        return api_fail(GDN_EINVAL, "seq_len, src_rows, dst_rows, the move lists and status must be non-NULL");
    gdn::PageTables t = {table, table_rows, max_pages, seq_len, refs, num_pages, page_size, nullptr};
    if ((rc = api_error_word(&t.err)))
        return rc;
    return launched(gdn::launch_pages_fork(t, src_rows, dst_rows, n, move_src, move_dst, move_count, status,
                                           static_cast<cudaStream_t>(stream)),
                    "kv_pages_fork launch");
}

int kv_pages_free(int32_t *table, int table_rows, int max_pages, int32_t *seq_len, int32_t *refs, int num_pages,
                  const int32_t *list_rows, int n, void *stream)
{
    int rc = check_tables(table, table_rows, max_pages, refs, num_pages);
    if (rc)
        return rc;
    if (n < 0)
        return api_fail(GDN_EINVAL, "n=%d < 0", n);
    if (n == 0)
        return api_ok();
    if (!seq_len || !list_rows)
        return api_fail(GDN_EINVAL, "seq_len and list_rows must be non-NULL");
    gdn::PageTables t = {table, table_rows, max_pages, seq_len, refs, num_pages, 0, nullptr};
    if ((rc = api_error_word(&t.err)))
        return rc;
    return launched(gdn::launch_pages_free(t, list_rows, n, static_cast<cudaStream_t>(stream)),
                    "kv_pages_free launch");
}

int kv_pages_compact(const int32_t *table, int table_rows, int max_pages, const int32_t *refs, int num_pages,
                     int32_t *table_out, int32_t *refs_out, int32_t *remap, int32_t *move_src, int32_t *move_dst,
                     int32_t *move_count, int32_t *scratch, void *stream)
{
    int rc = check_tables(table, table_rows, max_pages, refs, num_pages);
    if (rc)
        return rc;
    if (!table_out || !refs_out || !remap || !move_src || !move_dst || !move_count || !scratch)
        return api_fail(GDN_EINVAL, "the outputs, the move lists and scratch must be non-NULL");
    gdn::PageTables t = {const_cast<int32_t *>(table), table_rows, max_pages, nullptr, const_cast<int32_t *>(refs),
                         num_pages, 0, nullptr};
    if ((rc = api_error_word(&t.err)))
        return rc;
    return launched(gdn::launch_pages_compact(t, table_out, refs_out, remap, move_src, move_dst, move_count, scratch,
                                              static_cast<cudaStream_t>(stream)),
                    "kv_pages_compact launch");
}

int kv_pages_copy(kv_page_pool *pool, const int32_t *src, const int32_t *dst, int n, const int32_t *count,
                  void *stream)
{
    if (!pool)
        return api_fail(GDN_EINVAL, "pool is NULL");
    if (n < 0)
        return api_fail(GDN_EINVAL, "n=%d < 0", n);
    if (n == 0)
        return api_ok();
    if (!src || !dst)
        return api_fail(GDN_EINVAL, "src and dst must be non-NULL");
    int *err = nullptr;
    int rc = api_error_word(&err);
    if (rc)
        return rc;
    return launched(gdn::launch_pages_copy(*pool, src, dst, n, count, err, static_cast<cudaStream_t>(stream)),
                    "kv_pages_copy launch");
}

} // extern "C"
