// The prologue of an attention layer (sm_103a): RMS norm of q and k, rotary
// positions, and the append of k and v to the pages of each token's row, in
// one pass; and the rotation table.
//
// Bound: HBM.  A token's q, k and v are read once, q_out and the cache slots
// written once; the rotation row is shared by all heads of a token.
#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

typedef __nv_bfloat16 bf16;
constexpr int kMaxThreads = 512;
constexpr int kMaxTokens = 8; // tokens a CTA

// Eight consecutive elements as fp32.
struct V8 {
    float x[8];
};
__device__ __forceinline__ V8 load8(const float *p)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ V8 load8(const bf16 *p)
{
    const uint4 r = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v.x[2 * i] = __uint_as_float(w[i] << 16);
        v.x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return v;
}
__device__ __forceinline__ void store8(float *p, const V8 &v)
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(v.x[0], v.x[1], v.x[2], v.x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v.x[4], v.x[5], v.x[6], v.x[7]);
}
__device__ __forceinline__ void store8(bf16 *p, const V8 &v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x[2 * i], v.x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The last row r with cu[r] <= t, by a warp: 32 probes a round.
__device__ __forceinline__ int find_row(const int32_t *cu, int rows, int t, int lane)
{
    int lo = 0, n = rows; // the row is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lo + lane * step;
        const unsigned ok = __ballot_sync(0xffffffffu, at < lo + n && cu[at] <= t);
        const int last = ok ? 31 - __clz(ok) : 0;
        const int end = lo + n;
        lo += last * step;
        n = min(step, end - lo);
    }
    return lo;
}

// TPH threads a head of 8 TPH elements; a thread keeps one place of the head
// (its norm weights and, for a token, its rotation) and walks over heads.
template <typename T, int TPH>
__global__ void __launch_bounds__(kMaxThreads) prologue_kernel(const PrologueArgs a, int tokens_per_cta, int groups)
{
    __shared__ int s_pos[kMaxTokens], s_page[kMaxTokens];
    constexpr int D = 8 * TPH;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, a.c.total_tokens - t0);
    wait_prior_grid();
    for (int i = warp; i < nt; i += warps) {
        const int t = t0 + i;
        const int r = find_row(a.c.cu_seqlens, a.c.rows, t, lane);
        const int b = a.c.cu_seqlens[r], e = a.c.cu_seqlens[r + 1], len = a.c.seq_len[r];
        int pos = -1, page = 0;
        if (t < b || t >= e || len < 0) {
            if (lane == 0)
                report(a.err, GDN_DEVERR_BAD_PAGE);
        } else if (len > 0) {
            const long long p = (long long)len - (e - b) + (t - b); // len below n: the whole row is bad
            const int at = (int)(p >> a.pages.page_shift);
            if (len >= e - b && (a.rot == 0 || p < a.rope_positions) && at < a.c.max_pages)
                page = a.c.table[(size_t)r * a.c.max_pages + at];
            if (page > 0 && page < a.pages.num_pages)
                pos = (int)p;
            else if (lane == 0)
                report(a.err, GDN_DEVERR_BAD_PAGE);
        }
        if (lane == 0)
            s_pos[i] = pos, s_page[i] = page;
    }
    __syncthreads();

    const int th = tid % TPH, grp = tid / TPH;
    const int hkv = a.pages.hkv, units = a.hq + 2 * hkv, ps = a.pages.page_size;
    const bool idle = grp >= groups; // threads that round the block up to whole warps
    V8 qw, kw;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        qw.x[j] = 1.f, kw.x[j] = 1.f;
    if (a.q_norm)
        qw = load8(a.q_norm + 8 * th);
    if (a.k_norm)
        kw = load8(a.k_norm + 8 * th);
    const int half = a.rot >> 1, e0 = 8 * th;
    const bool turns = e0 < a.rot, low = e0 < half;
    // the lane that holds the other elements of this one's pairs
    const int mate = (lane & ~(TPH - 1)) | (turns ? (low ? th + (half >> 3) : th - (half >> 3)) : th);

    for (int i = 0; i < nt; ++i) {
        const int t = t0 + i, pos = s_pos[i];
        V8 cs, sn;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            cs.x[j] = 1.f, sn.x[j] = 0.f;
        if (turns && pos >= 0) {
            const float *row = a.rope + (size_t)pos * a.rot;
            if (a.interleaved) {
                const float4 c = *reinterpret_cast<const float4 *>(row + (e0 >> 1));
                const float4 s = *reinterpret_cast<const float4 *>(row + half + (e0 >> 1));
                cs = {{c.x, c.x, c.y, c.y, c.z, c.z, c.w, c.w}};
                sn = {{-s.x, s.x, -s.y, s.y, -s.z, s.z, -s.w, s.w}};
            } else {
                cs = load8(row + (low ? e0 : e0 - half));
                sn = load8(row + half + (low ? e0 : e0 - half));
                if (low) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sn.x[j] = -sn.x[j];
                }
            }
        }
        // the slot of the token in its page, for head 0
        const size_t slot = pos < 0 ? 0 : ((size_t)s_page[i] * hkv * ps + (pos & (ps - 1))) * D + e0;
        for (int h0 = 0; h0 < units; h0 += groups) {
            const int h = h0 + grp;
            const bool live = !idle && h < units && pos >= 0;
            const int kind = h < a.hq ? 0 : h < a.hq + hkv ? 1 : 2; // q, k, v
            V8 x;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x.x[j] = 0.f;
            if (live) {
                const T *from = kind == 0   ? static_cast<const T *>(a.q) + (size_t)t * a.q_stride + h * D
                                : kind == 1 ? static_cast<const T *>(a.k) + (size_t)t * a.k_stride + (h - a.hq) * D
                                            : static_cast<const T *>(a.v) + (size_t)t * a.v_stride + (h - a.hq - hkv) * D;
                x = load8(from + e0);
            }
            V8 y = x;
            if (a.q_norm || a.k_norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    ss = fmaf(x.x[j], x.x[j], ss);
#pragma unroll
                for (int o = TPH / 2; o > 0; o >>= 1)
                    ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float rms = rsqrtf(ss * (1.f / D) + a.eps);
                if (kind == 0 && a.q_norm) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y.x[j] = x.x[j] * rms * qw.x[j];
                } else if (kind == 1 && a.k_norm) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y.x[j] = x.x[j] * rms * kw.x[j];
                }
            }
            if (a.rot > 0) {
                V8 z;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float across = __shfl_sync(0xffffffffu, y.x[j], mate);
                    z.x[j] = a.interleaved ? y.x[j ^ 1] : across;
                }
                if (turns && kind < 2) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        y.x[j] = fmaf(z.x[j], sn.x[j], y.x[j] * cs.x[j]);
                }
            }
            if (!idle && h < units) {
                if (kind == 0)
                    store8(static_cast<T *>(a.q_out) + ((size_t)t * a.hq + h) * D + e0, y);
                else if (live)
                    store8(static_cast<T *>(kind == 1 ? a.pages.k : a.pages.v) +
                               (size_t)(h - (kind == 1 ? a.hq : a.hq + hkv)) * ps * D + slot, y);
            }
        }
    }
}

// cos and sin in 64 bits: positions reach 10^5 and more, where an fp32 angle
// is off by 10^-2.
__global__ void rope_table_kernel(const double *inv_freq, int half, size_t total, double mscale, float *table)
{
    wait_prior_grid();
    for (size_t i = (size_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (size_t)gridDim.x * blockDim.x) {
        const size_t p = i / half;
        const int j = (int)(i - p * half);
        double s, c;
        sincos((double)p * inv_freq[j], &s, &c);
        table[p * 2 * half + j] = (float)(c * mscale);
        table[p * 2 * half + half + j] = (float)(s * mscale);
    }
}

template <typename T, int TPH> cudaError_t go(const PrologueArgs &a, cudaStream_t s)
{
    const int units = a.hq + 2 * a.pages.hkv;
    // as few passes over the heads as the block size allows, evenly filled
    const int passes = (units * TPH + kMaxThreads - 1) / kMaxThreads;
    const int groups = (units + passes - 1) / passes;
    const int threads = (groups * TPH + 31) / 32 * 32;
    int per = a.c.total_tokens / (152 * 4);
    per = per < 1 ? 1 : per > kMaxTokens ? kMaxTokens : per;
    return launch_pdl(prologue_kernel<T, TPH>, dim3((unsigned)((a.c.total_tokens + per - 1) / per)), dim3(threads), 0, s,
                      a, per, groups);
}

template <typename T> cudaError_t by_d(const PrologueArgs &a, cudaStream_t s)
{
    switch (a.pages.d) {
    case 64:
        return go<T, 8>(a, s);
    case 128:
        return go<T, 16>(a, s);
    default:
        return go<T, 32>(a, s);
    }
}

} // namespace

cudaError_t launch_attn_prologue(const PrologueArgs &a, int dtype, cudaStream_t s)
{
    return dtype == GDN_BF16 ? by_d<bf16>(a, s) : by_d<float>(a, s);
}

cudaError_t launch_rope_table(const double *inv_freq, int rot, int positions, double mscale, float *table,
                              cudaStream_t s)
{
    const size_t total = (size_t)positions * (rot / 2);
    const size_t blocks = (total + 255) / 256;
    return launch_pdl(rope_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s, inv_freq,
                      rot / 2, total, mscale, table);
}

} // namespace gdn
