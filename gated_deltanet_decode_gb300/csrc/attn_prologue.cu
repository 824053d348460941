// The prologue of an attention layer (sm_103a): RMS norm of q and k, rotary
// positions, and the append of k and v to the pages of each token's row, in
// one pass; and the rotation table.
//
// Bound: HBM.  A token's q, k and v are read once, q_out and the cache slots
// written once; the rotation row is shared by all heads of a token.
#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

typedef __nv_bfloat16 bf16;
constexpr int kMaxThreads = 256, kResident = 3;
constexpr int kBatch = 128;  // tokens whose places are looked up together
template <typename T> constexpr int kStages = sizeof(T) == 2 ? 4 : 3; // tokens in flight a CTA, of four CTAs an SM

// Eight consecutive elements as they lie, and as four pairs of fp32: pairs,
// since one instruction multiplies or adds two.
template <typename T> struct Raw;
template <> struct Raw<float> { float4 a, b; };
template <> struct Raw<bf16> { uint4 a; };
__device__ __forceinline__ Raw<float> load8(const float *p)
{
    return {reinterpret_cast<const float4 *>(p)[0], reinterpret_cast<const float4 *>(p)[1]};
}
__device__ __forceinline__ Raw<bf16> load8(const bf16 *p) { return {*reinterpret_cast<const uint4 *>(p)}; }
__device__ __forceinline__ void copy8(float *p, const Raw<float> &r)
{
    reinterpret_cast<float4 *>(p)[0] = r.a, reinterpret_cast<float4 *>(p)[1] = r.b;
}
__device__ __forceinline__ void copy8(bf16 *p, const Raw<bf16> &r) { *reinterpret_cast<uint4 *>(p) = r.a; }
__device__ __forceinline__ void widen(const Raw<float> &r, float2 *x)
{
    x[0] = make_float2(r.a.x, r.a.y), x[1] = make_float2(r.a.z, r.a.w);
    x[2] = make_float2(r.b.x, r.b.y), x[3] = make_float2(r.b.z, r.b.w);
}
__device__ __forceinline__ float2 widen2(uint32_t w)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void widen(const Raw<bf16> &r, float2 *x)
{
    x[0] = widen2(r.a.x), x[1] = widen2(r.a.y), x[2] = widen2(r.a.z), x[3] = widen2(r.a.w);
}
__device__ __forceinline__ Raw<float> narrow(const float2 *x, float)
{
    return {make_float4(x[0].x, x[0].y, x[1].x, x[1].y), make_float4(x[2].x, x[2].y, x[3].x, x[3].y)};
}
__device__ __forceinline__ uint32_t narrow2(float2 x)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ Raw<bf16> narrow(const float2 *x, bf16)
{
    return {make_uint4(narrow2(x[0]), narrow2(x[1]), narrow2(x[2]), narrow2(x[3]))};
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

// TPH threads a head of 16 TPH elements, sixteen each: two runs of eight, which
// are the two sides of eight rotation pairs (half layout), eight adjacent pairs
// (interleaved), or elements past the rotation.  So no value crosses threads
// but the norm's sum, and both layouts read cosines and sines 8 th .. 8 th + 7.
//
// A CTA takes consecutive tokens and `heads` of the q | k | v heads (blockIdx.y
// says which); a thread keeps its place and its head.  The tokens' heads and
// rotation rows come by bulk copies into a ring of kStages, issued by one
// thread: loads to registers leave too few bytes under way (48 us and more for
// 16.8 k tokens of 16 + 4 heads of 128 in bf16, against 43: 5.0 TB/s, 75 % of
// a plain copy's rate, with issue slots half busy).  A decode step of 64 tokens
// takes 3.3 us, latency: launch, lengths, page, copy.
template <typename T, int TPH>
__global__ void __launch_bounds__(kMaxThreads, kResident)
    prologue_kernel(const PrologueArgs a, int tokens_per_cta, int heads, int stage_bytes, int rope_at)
{
    extern __shared__ __align__(128) unsigned char ring[];
    constexpr int S = kStages<T>, D = 16 * TPH;
    __shared__ int s_pos[kBatch];
    __shared__ long long s_slot[kBatch]; // elements of the cache before the token's slot, head 0
    __shared__ __align__(8) unsigned long long s_full[S], s_empty[S];
    const int tid = threadIdx.x, lane = tid & 31;
    const int th = tid % TPH, grp = tid / TPH;
    const int hq = a.hq, hkv = a.pages.hkv, ps = a.pages.page_size, half = a.rot >> 1;
    const int lo = blockIdx.y * heads, hi = min(lo + heads, hq + 2 * hkv), h = lo + grp;
    const bool mine = h < hi; // the last warp may have threads to spare
    const int kind = h < hq ? 0 : h < hq + hkv ? 1 : 2; // q, k, v
    const int hh = kind == 0 ? h : kind == 1 ? h - hq : h - hq - hkv;
    const bool turns = 16 * th < a.rot, across = turns && !a.interleaved;
    const int p0 = across ? 8 * th : 16 * th, p1 = across ? half + 8 * th : 16 * th + 8;
    const int begin = blockIdx.x * tokens_per_cta, end = min(begin + tokens_per_cta, a.c.total_tokens);
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(sm_addr(&s_full[i]), 2); // the heads' bytes, the rotation's
            mbar_init(sm_addr(&s_empty[i]), blockDim.x >> 5);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    wait_prior_grid();

    // by thread 0: token t's heads lo .. hi into stage st, then its rotation
    auto issue_heads = [&](int t, int st) {
        const uint32_t bar = sm_addr(&s_full[st]), to = sm_addr(ring) + st * stage_bytes;
        mbar_arrive_tx(bar, (uint32_t)((hi - lo) * D * sizeof(T)));
        auto part = [&](const void *x, long long stride, int first, int n) {
            const int u = max(lo, first), v = min(hi, first + n);
            if (u < v)
                bulk_load(to + (u - lo) * D * sizeof(T), static_cast<const T *>(x) + t * stride + (u - first) * D,
                          (uint32_t)((v - u) * D * sizeof(T)), bar);
        };
        part(a.q, a.q_stride, 0, hq);
        part(a.k, a.k_stride, hq, hkv);
        part(a.v, a.v_stride, hq + hkv, hkv);
    };
    auto issue_turn = [&](int pos, int st) {
        const uint32_t bar = sm_addr(&s_full[st]);
        if (a.rot > 0 && pos >= 0) {
            mbar_arrive_tx(bar, (uint32_t)a.rot * 4);
            bulk_load(sm_addr(ring) + st * stage_bytes + rope_at, a.rope + (size_t)pos * a.rot, (uint32_t)a.rot * 4, bar);
        } else {
            mbar_arrive(bar);
        }
    };

    const float *const norm = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    const bool norms = a.q_norm || a.k_norm, rotates = turns && kind < 2;
    float2 w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        w[e] = mine && norm ? *reinterpret_cast<const float2 *>(norm + (e < 4 ? p0 + 2 * e : p1 + 2 * e - 8)) : make_float2(1.f, 1.f);
    T *const cache = static_cast<T *>(kind == 1 ? a.pages.k : a.pages.v) + (size_t)hh * ps * D;
    const size_t q_step = (size_t)hq * D;
    T *q_out = static_cast<T *>(a.q_out) + begin * q_step + hh * D;
    const bool all_v = __all_sync(0xffffffffu, kind == 2);
    unsigned done = 0; // tokens of this CTA before the batch
    bool alive = true;
    for (int t0 = begin; t0 < end && alive; done += min(kBatch, end - t0), t0 += kBatch) {
        const int nt = min(kBatch, end - t0);
        __syncthreads(); // the last batch is through: its places and stages are free
        if (tid == 0)
            for (int i = 0; i < min(S, nt); ++i)
                issue_heads(t0 + i, (done + i) % S);
        // the tokens' places, while the first copies are under way
        const int r0 = find_row(a.c.cu_seqlens, a.c.rows, t0, lane);
        for (int i = tid; i < nt; i += blockDim.x) {
            const int t = t0 + i;
            int r = r0, last = i == 0 ? r0 : a.c.rows - 1; // the last row that starts at or before t
            while (r < last) {
                const int mid = (r + last + 1) >> 1;
                if (a.c.cu_seqlens[mid] <= t)
                    r = mid;
                else
                    last = mid - 1;
            }
            const int b = a.c.cu_seqlens[r], e = a.c.cu_seqlens[r + 1], len = a.c.seq_len[r];
            int pos = -1, page = 0;
            if (t < b || t >= e || len < 0) {
                report(a.err, GDN_DEVERR_BAD_PAGE);
            } else if (len > 0) {
                const long long p = (long long)len - (e - b) + (t - b); // len below n: the whole row is bad
                const int at = (int)(p >> a.pages.page_shift);
                if (len >= e - b && (a.rot == 0 || p < a.rope_positions) && at < a.c.max_pages)
                    page = a.c.table[(size_t)r * a.c.max_pages + at];
                if (page > 0 && page < a.pages.num_pages)
                    pos = (int)p;
                else
                    report(a.err, GDN_DEVERR_BAD_PAGE);
            }
            s_pos[i] = pos;
            s_slot[i] = pos < 0 ? 0 : ((long long)page * hkv * ps + (pos & (ps - 1))) * D;
        }
        __syncthreads();
        if (tid == 0)
            for (int i = 0; i < min(S, nt); ++i)
                issue_turn(s_pos[i], (done + i) % S);
        for (int i = 0; i < nt; ++i, q_out += q_step) {
            const unsigned n = done + i;
            const int st = n % S;
            if (!__all_sync(0xffffffffu, mbar_wait(sm_addr(&s_full[st]), (n / S) & 1))) {
                report(a.err, GDN_DEVERR_TIMEOUT);
                alive = false;
                break;
            }
            const unsigned char *const stage = ring + st * stage_bytes;
            const T *const head = reinterpret_cast<const T *>(stage) + grp * D;
            const bool live = s_pos[i] >= 0;
            Raw<T> raw0 = {}, raw1 = {};
            if (mine && live)
                raw0 = load8(head + p0), raw1 = load8(head + p1);
            if (!all_v) { // v goes as it is
                float2 x[8];
                widen(raw0, x), widen(raw1, x + 4);
                if (norms) {
                    float2 s2 = mul2(x[0], x[0]);
#pragma unroll
                    for (int e = 1; e < 8; ++e)
                        s2 = fma2(x[e], x[e], s2);
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int o = TPH / 2; o > 0; o >>= 1)
                        ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    if (norm) {
                        const float rms = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x[e] = mul2(mul2(x[e], make_float2(rms, rms)), w[e]);
                    }
                }
                if (rotates && live) {
                    const float *const row = reinterpret_cast<const float *>(stage + rope_at) + 8 * th;
                    const float4 *const cp = reinterpret_cast<const float4 *>(row), *const sp = reinterpret_cast<const float4 *>(row + half);
#pragma unroll
                    for (int f = 0; f < 2; ++f) { // four cosines and sines at a time
                        const float4 c = cp[f], s = sp[f];
                        if (a.interleaved) {
                            const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float2 &y = x[4 * f + e];
                                y = fma2(make_float2(y.y, y.x), make_float2(-sc[e], sc[e]), mul2(y, make_float2(cc[e], cc[e])));
                            }
                        } else {
                            const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
                            const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float2 u = x[2 * f + e], v = x[4 + 2 * f + e];
                                x[2 * f + e] = fma2(make_float2(-s2[e].x, -s2[e].y), v, mul2(u, c2[e]));
                                x[4 + 2 * f + e] = fma2(s2[e], u, mul2(v, c2[e]));
                            }
                        }
                    }
                }
                if (kind < 2) {
                    raw0 = narrow(x, T()), raw1 = narrow(x + 4, T());
                    if (!live) // and not what the norm or the rotation made of zeros
                        raw0 = {}, raw1 = {};
                }
            }
            if (mine && (kind == 0 || live)) {
                T *const at = kind == 0 ? q_out : cache + s_slot[i];
                copy8(at + p0, raw0);
                copy8(at + p1, raw1);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(sm_addr(&s_empty[st]));
            // the stage of the token before this one takes a later token
            if (tid == 0 && i > 0 && i - 1 + S < nt) {
                const int old = (n - 1) % S;
                if (mbar_wait(sm_addr(&s_empty[old]), ((n - 1) / S) & 1)) {
                    issue_heads(t0 + i - 1 + S, old);
                    issue_turn(s_pos[i - 1 + S], old);
                }
            }
            __syncwarp();
        }
    }
    // after a wait that ran out: the copies still in flight land first
    if (!alive && tid == 0)
        for (int i = 0; i < S; ++i)
            for (int parity = 0; parity < 2; ++parity)
                mbar_wait(sm_addr(&s_full[i]), parity, kWaitNs / 16);
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
    // as few shares of the heads as the block size allows, evenly filled
    const int least = (units * TPH + kMaxThreads - 1) / kMaxThreads;
    const int heads = (units + least - 1) / least, shares = (units + heads - 1) / heads;
    const int threads = (heads * TPH + 31) / 32 * 32;
    const int rope_at = heads * 16 * TPH * (int)sizeof(T), stage = rope_at + (a.rot * 4 + 127) / 128 * 128;
    const int smem = kStages<T> * stage;
    static std::atomic<unsigned long long> configured{0}; // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        const int most = kStages<T> * (kMaxThreads * 16 * (int)sizeof(T) + 1024);
        e = cudaFuncSetAttribute(prologue_kernel<T, TPH>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        // the resident CTAs' rings take more shared memory than the default split leaves
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(prologue_kernel<T, TPH>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     (int)cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    // as many CTAs as are resident together, each with an even share of the tokens: one while they last
    const int resident = std::max(1, std::min(kResident * kMaxThreads / threads, 227 * 1024 / (smem + 3 * 1024)));
    const int ctas = std::max(1, 152 * resident / shares);
    const int per = (a.c.total_tokens + ctas - 1) / ctas;
    return launch_pdl(prologue_kernel<T, TPH>, dim3((unsigned)((a.c.total_tokens + per - 1) / per), shares), dim3(threads),
                      (size_t)smem, s, a, per, heads, stage, rope_at);
}

template <typename T> cudaError_t by_d(const PrologueArgs &a, cudaStream_t s)
{
    switch (a.pages.d) {
    case 64:
        return go<T, 4>(a, s);
    case 128:
        return go<T, 8>(a, s);
    default:
        return go<T, 16>(a, s);
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
