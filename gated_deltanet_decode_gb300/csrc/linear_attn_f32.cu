// Linear attention with a decay for each head over packed sequences in chunks
// of C = 64 tokens in fp32 (sm_103a): fp32 activations, and bf16 ones whose head
// sizes the tensor core kernel (linear_attn_tc.cu, with the formula) is not made
// for.  Work is divided as linear_plan.cuh says; a CTA takes a block of VB value
// rows of a head through a segment, with its state in shared memory.
//
// All four products are sums over the last dimension of two tiles in shared
// memory, rows DK + 4 or C + 4 floats apart:
//   P = Q K^T,   O = e^G Q S^T + (P e^{G_i - G_j}) V,   S += (e^{G_C - G} V)^T K
// with V kept transposed, and K transposed into Q's place for the last.  A thread
// has 4 x 4 of a result, rows 4 and 8 apart, so that a warp's loads of 16 bytes
// are of rows in different banks.  Multiplications are packed fp32 FMAs of pairs
// along the sum: three tf32 products of split operands (attn_f32.cu) would be as
// fast, and cut their sums short.
//
// Bound: the FMAs, two wide, a chunk's 3/4 + 5/8 + 1 + 1 products of 64 x 64 x
// DK each.
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"
#include "linear_plan.cuh"

namespace gdn {
namespace {

constexpr int kC = 64;       // tokens a chunk
constexpr int kThreads = 256;
constexpr int kLd = kC + 4;  // floats a row of tokens

template <int DK> struct FGeo {
    static constexpr int VB = DK == 256 ? 32 : 64; // value rows a CTA: shared memory
    static constexpr int LD = DK + 4;
    // floats: K; Q, later K transposed; the state; V transposed; the weights
    static constexpr int K = 0, Q = K + kC * LD, QN = kC * LD > DK * kLd ? kC * LD : DK * kLd;
    static constexpr int S = Q + QN, V = S + VB * LD, P = V + VB * kLd, END = P + kC * kLd;
};

struct FCtrl {
    LItem item;
    int more;
    float hi[kC], lo[kC], w[kC], all; // G_j in two floats, e^{G_C - G_j}, e^{G_C} (in units of log2)
    int badfrom[64], dirty;           // first token with a value that is not finite, by value row
};

// acc += sum over k0 <= k < k1 of rows of a (r0 + 4 i) and of b (c0 + 8 j), pairs of k
template <int N> __device__ __forceinline__ void dots(const float *a, int lda, const float *b, int ldb, int k0, int k1, float2 (&acc)[4][N])
{
#pragma unroll 2
    for (int k = k0; k < k1; k += 4) {
        float4 x[4], y[N];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const float4 *>(a + 4 * i * lda + k);
#pragma unroll
        for (int j = 0; j < N; ++j)
            y[j] = *reinterpret_cast<const float4 *>(b + 8 * j * ldb + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                acc[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), acc[i][j]);
                acc[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), acc[i][j]);
            }
    }
}
template <int N> __device__ __forceinline__ void clear(float2 (&acc)[4][N])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j)
            acc[i][j] = make_float2(0.f, 0.f);
}

// four elements in fp32
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u));
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
template <typename T, int DK, bool SUM> __global__ void __launch_bounds__(kThreads) linear_ffma_kernel(const ChunkArgs p)
{
    typedef FGeo<DK> G;
    constexpr int VB = G::VB, LD = G::LD, N = VB / 16;
    extern __shared__ __align__(16) float sm[];
    __shared__ FCtrl ctl;
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // this thread's rows r0 + 4 i of a result, and columns c0 + 8 j of VB, k0 + 8 j of 64
    const int r0 = 16 * (warp >> 1) + (lane >> 3), c0 = VB / 2 * (warp & 1) + (lane & 7), k0 = 32 * (warp & 1) + (lane & 7);
    const int blocks = (a.dv + VB - 1) / VB;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
            for (int x = tid; x < VB * (DK / 4); x += kThreads) {
                const int v = x / (DK / 4), k = 4 * (x - v * (DK / 4));
                *reinterpret_cast<float4 *>(sm + G::S + v * LD + k) =
                    !SUM && v < rows ? load4(from + (size_t)v * DK + k) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float total = 1.f;
        for (int t = 0; t < it.n; t += kC) {
            const int n = min(kC, it.n - t);
            const long long tok = it.tok + t;
            __syncthreads(); // the chunk before is done with the tiles
            if (tid < VB)
                ctl.badfrom[tid] = kC;
            if (tid == 0)
                ctl.dirty = 0;
            if (warp == 0)
                chunk_decays(a, (int)tok, n, head, ctl);
            // K and Q as they are, V transposed; zeros past the end
            for (int x = tid; x < kC * (DK / 4); x += kThreads) {
                const int j = x / (DK / 4), k = 4 * (x - j * (DK / 4));
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
                if (j < n) {
                    y = load4(static_cast<const T *>(a.k) + (tok + j) * a.k_stride + hk * DK + k);
                    if (!SUM)
                        z = load4(static_cast<const T *>(a.q) + (tok + j) * a.q_stride + hk * DK + k);
                }
                *reinterpret_cast<float4 *>(sm + G::K + j * LD + k) = y;
                if (!SUM)
                    *reinterpret_cast<float4 *>(sm + G::Q + j * LD + k) = z;
            }
            __syncthreads(); // (the marks are clear)
            for (int x = tid; x < kC * (VB / 4); x += kThreads) { // eight tokens x 16 values a warp
                const int j = (x & 7) + 8 * (x / (2 * VB)), v = 4 * ((x >> 3) % (VB / 4));
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
                if (j < n && v < rows)
                    y = load4(static_cast<const T *>(a.v) + (tok + j) * a.v_stride + head * a.dv + v0 + v);
                float z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a weight of zero does not hide a value that is not finite: it is left out, and its row marked
                    if (!(fabsf(z[e]) <= 3.402823466e38f)) {
                        z[e] = 0.f;
                        atomicMin(&ctl.badfrom[v + e], j);
                        ctl.dirty = 1;
                    }
                    sm[G::V + (v + e) * kLd + j] = z[e];
                }
            }
            __syncthreads();
            if constexpr (!SUM) {
                // the weights: the rows' tokens r0 + 4 i, keys k0 + 8 j
                {
                    float2 acc[4][4];
                    clear(acc);
                    const bool hidden = (warp & 1) && warp < 4; // all keys behind all tokens
                    if (!hidden)
                        dots<4>(sm + G::Q + r0 * LD, LD, sm + G::K + k0 * LD, LD, 0, DK, acc);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = r0 + 4 * i, c = k0 + 8 * j;
                            sm[G::P + r * kLd + c] =
                                c <= r ? (acc[i][j].x + acc[i][j].y) * exp2f((ctl.hi[r] - ctl.hi[c]) + (ctl.lo[r] - ctl.lo[c])) : 0.f;
                        }
                }
                float2 acc[4][N];
                clear(acc);
                dots<N>(sm + G::Q + r0 * LD, LD, sm + G::S + c0 * LD, LD, 0, DK, acc);
                float o[4][N];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = exp2f(ctl.hi[r0 + 4 * i] + ctl.lo[r0 + 4 * i]);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        o[i][j] = (acc[i][j].x + acc[i][j].y) * f;
                }
                __syncthreads(); // the weights are there
                clear(acc);
                dots<N>(sm + G::P + r0 * kLd, kLd, sm + G::V + c0 * kLd, kLd, 0, 16 * (warp >> 1) + 16, acc);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int r = r0 + 4 * i, c = c0 + 8 * j;
                        float x = (o[i][j] + (acc[i][j].x + acc[i][j].y)) * a.scale;
                        if (ctl.dirty && ctl.badfrom[c] <= r)
                            x = __int_as_float(0x7fc00000);
                        if (r < n && c < rows)
                            static_cast<T *>(a.out)[((tok + r) * a.hv + head) * a.dv + v0 + c] = from_f<T>(x);
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
            for (int m = 0; m < DK; m += 64) { // rows m .. of the state's dk
                if (m + 16 * (warp >> 1) >= DK)
                    continue;
                float2 acc[4][N];
                clear(acc);
                dots<N>(sm + G::Q + (m + r0) * kLd, kLd, sm + G::V + c0 * kLd, kLd, 0, kC, acc);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const int c = c0 + 8 * j;
                        float *const s = sm + G::S + c * LD + m + r0 + 4 * i;
                        *s = fmaf(*s, all, acc[i][j].x + acc[i][j].y) + (ctl.dirty && ctl.badfrom[c] < kC ? __int_as_float(0x7fc00000) : 0.f);
                    }
            }
        }
        if (SUM || it.last) {
            __syncthreads();
            float *const to = SUM ? p.state + slot * it.at + mine : a.pool + slot * it.ws + mine;
            for (int x = tid; x < rows * (DK / 4); x += kThreads) {
                const int v = x / (DK / 4), k = 4 * (x - v * (DK / 4));
                *reinterpret_cast<float4 *>(to + (size_t)v * DK + k) = load4(sm + G::S + v * LD + k);
            }
            if (SUM && v0 == 0 && tid == 0)
                p.decay[(size_t)it.at * a.hv + head] = total;
        }
    }
}

// Chunks a segment: one, unless that gives more CTAs than would stand on the GPU eight times over, and their states more
// room than they save time.
int segment_chunks(const LinearArgs &a, int vb)
{
    const long long chunks = ((long long)a.total_tokens / kC + a.rows) * a.hv * ((a.dv + vb - 1) / vb);
    return (int)((chunks + 8 * kSms - 1) / (8 * kSms));
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
        e = cudaFuncSetAttribute(linear_ffma_kernel<T, DK, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(linear_ffma_kernel<T, DK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    ChunkArgs p;
    p.a = a;
    p.span = kC * segment_chunks(a, G::VB);
    p.least = kSerial;
    p.heads = a.hv * ((a.dv + G::VB - 1) / G::VB);
    chunk_layout(p);
    const long long most = places(a.rows, a.total_tokens, p.span) * p.heads; // items
    const dim3 grid((unsigned)(most < 8 * kSms ? most : 8 * kSms));
    if (a.total_tokens > p.span) { // a sequence can have several segments
        e = launch_pdl(linear_ffma_kernel<T, DK, true>, grid, dim3(kThreads), (size_t)BYTES, s, p);
        if (e == cudaSuccess)
            e = launch_scan(p, s);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(linear_ffma_kernel<T, DK, false>, grid, dim3(kThreads), (size_t)BYTES, s, p);
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

size_t linear_prefill_workspace_bytes(const LinearArgs &a, int dtype)
{
    if (a.total_tokens <= kSerial)
        return 0;
    if (on_tensor_cores(a, dtype))
        return linear_chunked_workspace_bytes(a);
    const long long span = (long long)kC * segment_chunks(a, a.dk == 256 ? FGeo<256>::VB : FGeo<128>::VB);
    return a.total_tokens > span ? chunk_bytes(a, span) : 0;
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
