// Linear attention with a decay for each head over packed sequences in chunks
// of C = 64 tokens to fp32's precision (sm_103a): fp32 activations, and bf16 ones whose head
// sizes the tensor core kernel (linear_attn_tc.cu, with the formula) is not made
// for.  Work is divided as linear_plan.cuh says; a CTA takes a block of VB value
// rows of a head through a segment, with its state in shared memory.
//
// All four products are sums over the last dimension of two tiles in shared
// memory, rows DK + 4 or C + 4 floats apart, so that a fragment's loads fall in
// 32 banks:
//   P = Q K^T,   O = e^G Q S^T + (P e^{G_i - G_j}) V,   S += (e^{G_C - G} V)^T K
// with V kept transposed, and K transposed into Q's place for the last.  They run
// on the tensor cores in tf32 with split operands (tf32_ops.cuh), eight warps as
// 2 x 4 blocks of a result of 64 x 64.  In packed FMAs of 4 x 4 results a thread,
// whose operands' loads took all of shared memory's bandwidth, five sequences of 200
// to 900 tokens (8 heads of 64 x 64, fp32) took 71 us instead of 41, of which
// the sums took 10, the scan 5 and the outputs 18; with the kernels beside each other 30.3
// in a graph, 31.2 called back to back.
//
// Every operand lies in shared memory at half its value: a head is rounded, and rounding would take finite values from 3.402e38
// on out of the range (their products with the mask's zeros are NaN).  Halves, and the factors of four that make up for them,
// are exact, but for the last bit of denormal numbers; they cost 1 % (a bound on each operand at its splitting 3 to 9).
//
// Bound: latency.  A segment is mostly a single chunk; its loads, five barriers
// and the products' chains follow each other, with one to two CTAs an SM.
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"
#include "linear_plan.cuh"
#include "tf32_ops.cuh"

namespace gdn {
namespace {

constexpr int kC = 64;       // tokens a chunk
constexpr int kThreads = 256;
constexpr int kLd = kC + 4;  // floats a row of tokens

template <int DK> struct FGeo {
    static constexpr int VB = DK == 256 ? 32 : 64; // value rows a CTA: shared memory
    static constexpr int LD = DK + 4;
    // floats: K; Q, later K transposed; the state; V transposed; the weights
    static constexpr int K = 0, Q = K + kC * LD, KT = (DK > 32 ? DK : 32) * kLd, QN = kC * LD > KT ? kC * LD : KT;
    static constexpr int S = Q + QN, V = S + VB * LD, P = V + VB * kLd, END = P + kC * kLd;
};

struct FCtrl {
    LItem item;
    int more;
    float hi[kC], lo[kC], w[kC], all; // G_j in two floats, e^{G_C - G_j}, e^{G_C} (in units of log2)
    int badfrom[64], dirty;           // first token with a value that is not finite, by value row
};

// A warp's 32 x 8 N of a result: sums over k < k1 (a multiple of 16) of rows of a and of b.  Result fragments: rows
// 16 m + g and + 8, columns 8 n + 2 c and + 1, with g = lane / 4, c = lane % 4.
template <int N> __device__ __forceinline__ void products(const float *a, int lda, const float *b, int ldb, int k1, float (&sum)[2][N][4])
{
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[m][n][e] = 0.f;
    a += g * lda + c, b += g * ldb + c;
#pragma unroll 2
    for (int k0 = 0; k0 < k1; k0 += 16) { // the tensor cores sum two steps of eight
        float t[2][N][4] = {};
#pragma unroll
        for (int k = k0; k < k0 + 16; k += 8) {
            uint32_t ah[2][4], al[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                split2(a[16 * m * lda + k], a[(16 * m + 8) * lda + k], ah[m][0], al[m][0], ah[m][1], al[m][1]);
                split2(a[16 * m * lda + k + 4], a[(16 * m + 8) * lda + k + 4], ah[m][2], al[m][2], ah[m][3], al[m][3]);
            }
#pragma unroll
            for (int n = 0; n < N; ++n) {
                uint32_t h0, l0, h1, l1;
                split2(b[8 * n * ldb + k], b[8 * n * ldb + k + 4], h0, l0, h1, l1);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    mma8(t[m][n], al[m], h0, h1);
                    mma8(t[m][n], ah[m], l0, l1);
                    mma8(t[m][n], ah[m], h0, h1);
                }
            }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sum[m][n][e] += t[m][n][e];
    }
}

__device__ __forceinline__ float4 times(float f, float4 x) { return make_float4(f * x.x, f * x.y, f * x.z, f * x.w); }

// four elements in fp32
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
}

__device__ __forceinline__ void store2(float *p, float x, float y) { *reinterpret_cast<float2 *>(p) = make_float2(x, y); }
__device__ __forceinline__ void store2(__nv_bfloat16 *p, float x, float y)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
}

// The decays of a chunk, by one warp, two tokens a lane.
__device__ __forceinline__ void chunk_decays(const LinearArgs &a, int tok, int n, int head, FCtrl &t)
{
    const int lane = threadIdx.x & 31;
    Two g[2], upto = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int j = 2 * lane + e;
        float x = j < n ? a.log_decay[(long long)(tok + j) * a.decay_stride + head] : 0.f;
        x = x > 0.f ? 0.f : x < -110.f ? -110.f : x; // (a NaN stays)
        upto = upto + log2_units(x);
        g[e] = upto;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two x = shuffle(upto, lane < o ? lane : lane - o);
        if (lane >= o)
            upto = upto + x;
    }
    const Two all = shuffle(upto, 31);
    Two before = shuffle(upto, lane == 0 ? 0 : lane - 1);
    if (lane == 0)
        before = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const Two G = before + g[e];
        t.hi[2 * lane + e] = G.h;
        t.lo[2 * lane + e] = G.l;
        t.w[2 * lane + e] = exp2f(minus(all, G));
    }
    if (lane == 0)
        t.all = exp2f(all.h + all.l);
}

// SUM: the segments' own sums; else the outputs, and the states at the sequences' ends.
template <typename T, int DK, bool SUM> __global__ void __launch_bounds__(kThreads) linear_f32_kernel(const ChunkArgs p)
{
    typedef FGeo<DK> G;
    constexpr int VB = G::VB, LD = G::LD, N = VB / 32, VQ = VB * kC / 4 / kThreads;
    extern __shared__ __align__(16) float sm[];
    __shared__ FCtrl ctl;
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // this warp's rows r0 .. + 32 of a result, and columns c0 .. + 8 N of VB, k0 .. + 16 of 64; this thread's place in them
    const int r0 = 32 * (warp >> 2), c0 = VB / 4 * (warp & 3), k0 = 16 * (warp & 3), g = lane >> 2, c = lane & 3;
    const int blocks = (a.dv + VB - 1) / VB;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    begin_chunks();
    if (SUM ? p.rare && !any_with(p, 2) : p.none && !any_with(p, 1)) {
        wait_prior_grid();
        return;
    }
    ItemWalk<SUM> walk(p); // warp 0's is followed
    for (;;) {
        __syncthreads();
        if (warp == 0) {
            LItem x;
            const bool more = walk.next(x);
            if (lane == 0)
                ctl.item = x, ctl.more = more;
        }
        __syncthreads();
        if (!ctl.more)
            break;
        const LItem it = ctl.item;
        const int head = it.head / blocks, v0 = (it.head - head * blocks) * VB, rows = min(VB, a.dv - v0), hk = head / (a.hv / a.hk);
        const size_t slot = (size_t)a.hv * a.dv * DK, mine = ((size_t)head * a.dv + v0) * DK;
        // the state
        {
            const float *const from = SUM ? nullptr : it.from < 0 ? a.pool + slot * it.rs + mine : p.state + slot * it.from + mine;
            if (!SUM && it.from >= 0)
                wait_prior_grid(); // the scan
            for (int x = tid; x < VB * (DK / 4); x += kThreads) {
                const int v = x / (DK / 4), k = 4 * (x - v * (DK / 4));
                *reinterpret_cast<float4 *>(sm + G::S + v * LD + k) =
                    !SUM && v < rows ? times(0.5f, load4(from + (size_t)v * DK + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float total = 1.f;
        for (int t = 0; t < it.n; t += kC) {
            const int n = min(kC, it.n - t);
            const long long tok = it.tok + t;
            // V, on its way: eight tokens x 16 values a warp
            float4 ahead[VQ];
#pragma unroll
            for (int i = 0; i < VQ; ++i) {
                const int x = tid + i * kThreads, j = (x & 7) + 8 * (x / (2 * VB)), v = 4 * ((x >> 3) % (VB / 4));
                ahead[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < n && v < rows)
                    ahead[i] = load4(static_cast<const T *>(a.v) + (tok + j) * a.v_stride + head * a.dv + v0 + v);
            }
            __syncthreads(); // the chunk before is done with the tiles
            if (tid < VB)
                ctl.badfrom[tid] = kC;
            if (tid == 0)
                ctl.dirty = 0;
            // K and Q in their order, V transposed; zeros past the end
#pragma unroll 4
            for (int x = tid; x < kC * (DK / 4); x += kThreads) {
                const int j = x / (DK / 4), k = 4 * (x - j * (DK / 4));
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
                if (j < n) {
                    y = load4(static_cast<const T *>(a.k) + (tok + j) * a.k_stride + hk * DK + k);
                    if (!SUM)
                        z = load4(static_cast<const T *>(a.q) + (tok + j) * a.q_stride + hk * DK + k);
                }
                *reinterpret_cast<float4 *>(sm + G::K + j * LD + k) = times(0.5f, y);
                if (!SUM)
                    *reinterpret_cast<float4 *>(sm + G::Q + j * LD + k) = times(0.5f, z);
            }
            if (warp == 0)
                chunk_decays(a, (int)tok, n, head, ctl);
            __syncthreads(); // (the marks are clear)
#pragma unroll
            for (int i = 0; i < VQ; ++i) {
                const int x = tid + i * kThreads, j = (x & 7) + 8 * (x / (2 * VB)), v = 4 * ((x >> 3) % (VB / 4));
                float z[4] = {ahead[i].x, ahead[i].y, ahead[i].z, ahead[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a weight of zero does not hide a value that is not finite: it is left out, and its row marked
                    if (!(fabsf(z[e]) <= 3.402823466e38f)) {
                        z[e] = 0.f;
                        atomicMin(&ctl.badfrom[v + e], j);
                        ctl.dirty = 1;
                    }
                    sm[G::V + (v + e) * kLd + j] = 0.5f * z[e];
                }
            }
            __syncthreads();
            if constexpr (!SUM) {
                { // the weights: tokens r0 .., keys k0 ..
                    float p2[2][2][4] = {};
                    if (k0 < r0 + 32) // (else all keys are behind all tokens)
                        products<2>(sm + G::Q + r0 * LD, LD, sm + G::K + k0 * LD, LD, DK, p2);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n2 = 0; n2 < 2; ++n2)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int r = r0 + 16 * m + g + 8 * (e >> 1), k = k0 + 8 * n2 + 2 * c + (e & 1);
                                sm[G::P + r * kLd + k] =
                                    k <= r ? 2.f * p2[m][n2][e] * exp2f((ctl.hi[r] - ctl.hi[k]) + (ctl.lo[r] - ctl.lo[k])) : 0.f;
                            }
                }
                float o[2][N][4], own[2][N][4];
                products<N>(sm + G::Q + r0 * LD, LD, sm + G::S + c0 * LD, LD, DK, o);
                __syncthreads(); // the weights are there
                products<N>(sm + G::P + r0 * kLd, kLd, sm + G::V + c0 * kLd, kLd, r0 + 32, own);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int r = r0 + 16 * m + g + 8 * h;
                        const float f = exp2f(ctl.hi[r] + ctl.lo[r]);
#pragma unroll
                        for (int n2 = 0; n2 < N; ++n2) {
                            const int v = c0 + 8 * n2 + 2 * c;
                            float x[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                x[e] = 4.f * fmaf(o[m][n2][2 * h + e], f, own[m][n2][2 * h + e]) * a.scale;
                                if (ctl.dirty && ctl.badfrom[v + e] <= r)
                                    x[e] = __int_as_float(0x7fc00000);
                            }
                            if (r < n && v < rows)
                                store2(static_cast<T *>(a.out) + ((tok + r) * a.hv + head) * a.dv + v0 + v, x[0], x[1]);
                        }
                    }
                if (t + kC >= it.n && !it.last)
                    continue; // the next segment's state comes from the scan
                __syncthreads(); // Q and V are read
            }
            // V times its weights, K transposed
            for (int x = tid; x < VB * kC; x += kThreads) {
                const int v = x / kC, j = x % kC;
                sm[G::V + v * kLd + j] *= ctl.w[j];
            }
            for (int x = tid; x < kC * (DK / 4); x += kThreads) {
                const int j = (x & 7) + 8 * (x / (2 * DK)), k = 4 * ((x >> 3) % (DK / 4));
                const float4 y = *reinterpret_cast<const float4 *>(sm + G::K + j * LD + k);
                float *const to = sm + G::Q + k * kLd + j;
                to[0] = y.x, to[kLd] = y.y, to[2 * kLd] = y.z, to[3 * kLd] = y.w;
            }
            __syncthreads();
            const float all = ctl.all;
            total *= all;
            for (int x0 = r0; x0 < DK; x0 += 64) { // rows x0 .. + 32 of the state's dk
                float y[2][N][4];
                products<N>(sm + G::Q + x0 * kLd, kLd, sm + G::V + c0 * kLd, kLd, kC, y);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n2 = 0; n2 < N; ++n2)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = x0 + 16 * m + g + 8 * (e >> 1), v = c0 + 8 * n2 + 2 * c + (e & 1);
                            if (DK >= 32 || k < DK) {
                                float *const s = sm + G::S + v * LD + k;
                                *s = fmaf(*s, all, 2.f * y[m][n2][e]) + (ctl.dirty && ctl.badfrom[v] < kC ? __int_as_float(0x7fc00000) : 0.f);
                            }
                        }
            }
        }
        if (SUM || it.last) {
            __syncthreads();
            float *const to = SUM ? p.state + slot * it.at + mine : a.pool + slot * it.ws + mine;
            for (int x = tid; x < rows * (DK / 4); x += kThreads) {
                const int v = x / (DK / 4), k = 4 * (x - v * (DK / 4));
                *reinterpret_cast<float4 *>(to + (size_t)v * DK + k) = times(2.f, load4(sm + G::S + v * LD + k));
            }
            if (SUM && v0 == 0 && tid == 0)
                p.decay[(size_t)it.at * a.hv + head] = total;
        }
    }
    wait_prior_grid();
}

// Chunks a segment, as in linear_attn_tc.cu: the fewest rounds of CTAs, in chunks, where a segment costs half a chunk's time to
// begin and a chunk a quarter of its time in the sums.  Against a chunk a segment (several only where that gave 8 x 152 CTAs): a
// sequence of 16,000 (8 heads of 64) takes 160 us instead of 177, of 4,000 47 instead of 57, 64 of 200 125 instead of 146, 8 of
// 2,000 with 32 heads of 128 2.2 ms instead of 2.6; 32 of 100 to 900 154 instead of 143.
int segment_chunks(const LinearArgs &a, bool &cut)
{
    const int vb = a.dk == 256 ? FGeo<256>::VB : FGeo<128>::VB, at_once = kSms * (a.dk > 64 ? 1 : 2);
    const long long m = ((long long)a.total_tokens + (long long)a.rows * kC - 1) / ((long long)a.rows * kC); // chunks a sequence
    const long long blocks = (long long)a.rows * a.hv * ((a.dv + vb - 1) / vb);
    auto rounds = [&](long long n) { return (double)((n * blocks + at_once - 1) / at_once); };
    const long long best = cheapest_length(m, 2 * at_once, [&](long long segs, long long len) {
        return rounds(segs) * (len + 0.5) + (segs > 1 ? rounds(segs - 1) * (0.25 * len + 0.5) + 1 : 0);
    });
    cut = best < m;
    return (int)(best < kMostChunks ? best : kMostChunks);
}

template <typename T, int DK> cudaError_t go(const LinearArgs &a, cudaStream_t s)
{
    typedef FGeo<DK> G;
    constexpr int BYTES = G::END * 4;
    static_assert(BYTES + sizeof(FCtrl) <= 232448, "shared memory");
    static std::atomic<unsigned long long> configured{0}; // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(linear_f32_kernel<T, DK, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(linear_f32_kernel<T, DK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    ChunkArgs p;
    p.a = a;
    p.rare = !a.cut;
    p.none = a.total_tokens <= (long long)kSerial * a.rows;
    p.least = kSerial;
    p.heads = a.hv * ((a.dv + G::VB - 1) / G::VB);
    chunk_layout(p);
    const long long most = places(a.rows, a.total_tokens, a.span) * p.heads; // items
    const dim3 grid((unsigned)(most < 8 * kSms ? most : 8 * kSms));
    if (a.total_tokens > a.span) { // a sequence can have several segments
        e = launch_pdl(linear_f32_kernel<T, DK, true>, grid, dim3(kThreads), (size_t)BYTES, s, p);
        if (e == cudaSuccess)
            e = launch_scan(p, s);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(linear_f32_kernel<T, DK, false>, grid, dim3(kThreads), (size_t)BYTES, s, p);
}
template <typename T> cudaError_t by_dk(const LinearArgs &a, cudaStream_t s)
{
    switch (a.dk) {
    case 16:
        return go<T, 16>(a, s);
    case 32:
        return go<T, 32>(a, s);
    case 64:
        return go<T, 64>(a, s);
    case 128:
        return go<T, 128>(a, s);
    default:
        return go<T, 256>(a, s);
    }
}

bool on_tensor_cores(const LinearArgs &a, int dtype)
{
    return dtype == GDN_BF16 && (a.dk == 64 || a.dk == 128) && (a.dv == 64 || a.dv == 128);
}

} // namespace

void linear_divide(LinearArgs &a, int dtype)
{
    a.span = on_tensor_cores(a, dtype) ? linear_chunked_segment(a, a.cut) : kC * segment_chunks(a, a.cut);
}

size_t linear_prefill_workspace_bytes(const LinearArgs &a)
{
    return a.total_tokens > kSerial && a.total_tokens > a.span ? chunk_bytes(a) : 0;
}

cudaError_t launch_linear_prefill(LinearArgs a, int dtype, cudaStream_t s)
{
    a.most = kSerial; // the short sequences, the padding and the bad ones
    const cudaError_t e = launch_linear_serial(a, dtype, s);
    if (e != cudaSuccess || a.total_tokens <= kSerial)
        return e;
    if (on_tensor_cores(a, dtype))
        return launch_linear_chunked(a, s);
    return dtype == GDN_BF16 ? by_dk<__nv_bfloat16>(a, s) : by_dk<float>(a, s);
}

} // namespace gdn
