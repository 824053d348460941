// Attention of new tokens over a paged cache (sm_103a): one warp per (token,
// query head), keys one after the other with a running maximum and sum.
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 4; // keys in flight

template <typename T, int D> __global__ void __launch_bounds__(32 * kWarps) simple_kernel(const AttentionArgs a)
{
    constexpr int E = D / 32; // elements a lane
    const int lane = threadIdx.x & 31;
    const long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    wait_prior_grid();
    if (u >= (long long)a.c.total_tokens * a.hq)
        return;
    const int t = (int)(u / a.hq), h = (int)(u - (long long)t * a.hq);
    // the last row that starts at or before t
    int lo = 0, hi = a.c.rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.c.cu_seqlens[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int b = a.c.cu_seqlens[lo], e = a.c.cu_seqlens[lo + 1], len = a.c.seq_len[lo];
    const int ps = a.pages.page_size, hkv = a.pages.hkv, kvh = h / (a.hq / hkv);
    T *const out = static_cast<T *>(a.out) + (size_t)u * D + lane * E;
    bool bad = t < b || t >= e || len < 0 || (len > 0 && (len < e - b || (len - 1) / ps >= a.c.max_pages));
    const int see = bad || len == 0 ? 0 : len - (e - b) + (t - b) + 1;
    float q[E], o[E], top = -INFINITY, sum = 0.f;
    const T *qp = static_cast<const T *>(a.q) + (size_t)t * a.q_stride + h * D + lane * E;
#pragma unroll
    for (int i = 0; i < E; ++i)
        q[i] = to_f(qp[i]) * a.scale, o[i] = 0.f;
    const int32_t *const table = a.c.table + (size_t)lo * a.c.max_pages;
    for (int j0 = 0; j0 < see && !bad; j0 += kKeys) {
        const int page = table[j0 >> a.pages.page_shift]; // kKeys divides the page size
        if (page <= 0 || page >= a.pages.num_pages) {
            bad = true;
            break;
        }
        const size_t at = (((size_t)page * hkv + kvh) * ps + (j0 & (ps - 1))) * D + lane * E;
        const T *kp = static_cast<const T *>(a.pages.k) + at, *vp = static_cast<const T *>(a.pages.v) + at;
        float s[kKeys];
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i)
                s[j] = fmaf(q[i], to_f(kp[j * D + i]), s[j]);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
#pragma unroll
            for (int j = 0; j < kKeys; ++j)
                s[j] += __shfl_xor_sync(0xffffffffu, s[j], off);
        float m = top;
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
            if (j0 + j < see)
                m = fmaxf(m, s[j]);
        const float f = m == -INFINITY ? 1.f : expf(top - m);
        sum *= f;
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] *= f;
        top = m;
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
            if (j0 + j < see) {
                const float p = expf(s[j] - (m == -INFINITY ? 0.f : m));
                sum += p;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    o[i] = fmaf(p, to_f(vp[j * D + i]), o[i]);
            }
    }
    if (bad && lane == 0)
        report(a.err, GDN_DEVERR_BAD_PAGE);
#pragma unroll
    for (int i = 0; i < E; ++i)
        out[i] = from_f<T>(bad || see == 0 ? 0.f : o[i] / sum);
}

template <typename T, int D> cudaError_t go(const AttentionArgs &a, cudaStream_t s)
{
    const long long blocks = ((long long)a.c.total_tokens * a.hq + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffffll)
        return cudaErrorInvalidValue;
    return launch_pdl(simple_kernel<T, D>, dim3((unsigned)blocks), dim3(32 * kWarps), 0, s, a);
}

template <typename T> cudaError_t by_d(const AttentionArgs &a, cudaStream_t s)
{
    switch (a.pages.d) {
    case 64:
        return go<T, 64>(a, s);
    case 128:
        return go<T, 128>(a, s);
    default:
        return go<T, 256>(a, s);
    }
}

} // namespace

size_t attention_workspace_bytes(int d, int dtype, int hq, int hkv, int, int total_tokens)
{
    return dtype == GDN_BF16 && attention_tc_supported(hq, hkv) ? attention_tc_workspace_bytes(d, hq, hkv, total_tokens) : 0;
}

cudaError_t launch_paged_attention(const AttentionArgs &a, kv_page_pool &pool, int dtype, cudaStream_t s)
{
    if (dtype == GDN_BF16 && attention_tc_supported(a.hq, a.pages.hkv))
        return launch_paged_attention_tc(a, pool, s);
    return dtype == GDN_BF16 ? by_d<__nv_bfloat16>(a, s) : by_d<float>(a, s);
}

} // namespace gdn
