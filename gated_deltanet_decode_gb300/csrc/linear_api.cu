// C ABI of linear attention with a decay for each head: argument checks.  The
// kernels are in linear_attn.cu, linear_attn_tc.cu and linear_attn_f32.cu.
#include <cmath>

#include "gdn_device.cuh"
#include "gdn_internal.h"

using gdn::api_cuda_fail;
using gdn::api_error_word;
using gdn::api_fail;
using gdn::api_ok;

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_stride(const char *what, const void *p, int64_t stride, int heads, int d, int dtype)
{
    if (!p)
        return api_fail(GDN_EINVAL, "%s is NULL", what);
    if (stride < (int64_t)heads * d)
        return api_fail(GDN_EINVAL, "%s: token stride %lld below %d heads of %d", what, (long long)stride, heads, d);
    if (!aligned16(p) || (stride * (dtype == GDN_BF16 ? 2 : 4)) % 16 != 0)
        return api_fail(GDN_EINVAL, "%s: address and token stride must be multiples of 16 bytes", what);
    return GDN_OK;
}

// What both forms check alike, and the kernels' arguments.
int check(gdn::LinearArgs &a, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
          int64_t v_stride, const float *log_decay, int decay_per_token, gdn_pool *pool, const int32_t *read_slot,
          const int32_t *write_slot, float scale, void *out, int rows, int tokens, int keep_in_place, int dtype)
{
    if (!pool)
        return api_fail(GDN_EINVAL, "state pool is NULL");
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return api_fail(GDN_EINVAL, "bad dtype %d", dtype);
    if (!std::isfinite(scale))
        return api_fail(GDN_EINVAL, "scale is not finite");
    if (rows > 0 && !read_slot)
        return api_fail(GDN_EINVAL, "read_slot must be non-NULL");
    if (rows > 0 && !keep_in_place && !write_slot)
        return api_fail(GDN_EINVAL, "write_slot is NULL in twin mode");
    const gdn_dims d = pool->dims;
    int rc;
    if (tokens > 0) {
        if (!log_decay || !out)
            return api_fail(GDN_EINVAL, "log_decay and out must be non-NULL");
        if ((rc = check_stride("q", q, q_stride, d.hk, d.dk, dtype)) ||
            (rc = check_stride("k", k, k_stride, d.hk, d.dk, dtype)) ||
            (rc = check_stride("v", v, v_stride, d.hv, d.dv, dtype)))
            return rc;
        if (!aligned16(out))
            return api_fail(GDN_EINVAL, "out must be 16-byte aligned");
    }
    a.q = q, a.k = k, a.v = v;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
    a.log_decay = log_decay, a.decay_stride = decay_per_token ? d.hv : 0;
    a.pool = pool->data, a.num_slots = pool->num_slots;
    a.read_slot = read_slot, a.write_slot = keep_in_place ? nullptr : write_slot;
    a.scale = scale, a.out = out;
    a.rows = rows, a.total_tokens = tokens;
    a.hk = d.hk, a.hv = d.hv, a.dk = d.dk, a.dv = d.dv;
    return GDN_OK;
}

} // namespace

extern "C" {

int linear_attention_decode(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                            int64_t v_stride, const float *log_decay, int decay_per_token, gdn_pool *pool,
                            const int32_t *read_slot, const int32_t *write_slot, float scale, void *out, int rows,
                            int keep_in_place, int dtype, void *stream)
{
    if (rows < 0)
        return api_fail(GDN_EINVAL, "rows=%d < 0", rows);
    gdn::LinearArgs a = {};
    int rc = check(a, q, q_stride, k, k_stride, v, v_stride, log_decay, decay_per_token, pool, read_slot, write_slot, scale,
                   out, rows, rows, keep_in_place, dtype);
    if (rc)
        return rc;
    if (rows == 0)
        return api_ok();
    if ((rc = api_error_word(&a.err)))
        return rc;
    const cudaError_t e = gdn::launch_linear_decode(a, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "linear_attention_decode launch");
}

size_t linear_attention_prefill_workspace_bytes(const gdn_pool *pool, int nseq, int total_tokens, int dtype)
{
    if (!pool || nseq < 1 || total_tokens < 1 || (dtype != GDN_F32 && dtype != GDN_BF16))
        return 0;
    gdn::LinearArgs a = {};
    a.rows = nseq, a.total_tokens = total_tokens;
    a.hk = pool->dims.hk, a.hv = pool->dims.hv, a.dk = pool->dims.dk, a.dv = pool->dims.dv;
    gdn::linear_divide(a, dtype);
    return gdn::linear_prefill_workspace_bytes(a);
}

int linear_attention_prefill(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const float *log_decay, int decay_per_token, gdn_pool *pool,
                             const int32_t *cu_seqlens, const int32_t *read_slot, const int32_t *write_slot, float scale,
                             void *out, int nseq, int total_tokens, int keep_in_place, void *workspace,
                             size_t workspace_bytes, int dtype, void *stream)
{
    if (nseq < 0 || total_tokens < 0)
        return api_fail(GDN_EINVAL, "nseq=%d and total_tokens=%d must be >= 0", nseq, total_tokens);
    gdn::LinearArgs a = {};
    int rc = check(a, q, q_stride, k, k_stride, v, v_stride, log_decay, decay_per_token, pool, read_slot, write_slot, scale,
                   out, nseq, total_tokens, keep_in_place, dtype);
    if (rc)
        return rc;
    if (nseq == 0)
        return api_ok();
    if (!cu_seqlens)
        return api_fail(GDN_EINVAL, "cu_seqlens must be non-NULL");
    if (total_tokens > 0)
        gdn::linear_divide(a, dtype);
    const size_t need = total_tokens > 0 ? gdn::linear_prefill_workspace_bytes(a) : 0;
    if (need && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 127u)))
        return api_fail(GDN_EINVAL, "workspace must be 128-byte aligned and hold %zu bytes (given %zu)", need,
                        workspace ? workspace_bytes : (size_t)0);
    if ((rc = api_error_word(&a.err)))
        return rc;
    a.cu_seqlens = cu_seqlens, a.work = workspace;
    const cudaError_t e = gdn::launch_linear_prefill(a, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? api_ok() : api_cuda_fail(e, "linear_attention_prefill launch");
}

} // extern "C"
