// Linear attention with a decay for each head (sm_103a): the recurrent form,
//   S' = a S + v k^T,   o = scale S' q,   a = exp(log_decay),
// for one token a row (decode) and token after token over packed sequences.
//
// The state is a slot of a GDN pool, [hv][dv][dk] fp32, and its value rows are
// independent of each other: a row needs k, q, one element of v and a.  A row
// of dk floats lies in dk / 16 lanes, 16 floats a lane in four 16-byte pieces,
// piece j of lane l at 4 (l + j dk / 16), so that every load of a warp covers
// whole 128-byte lines (dk >= 32).  A CTA takes a block of rows of one head.
//
// Decode is bound by the state's bytes, once in and once out; see
// linear_decode_kernel.  Over a sequence the state stays in registers and the
// tokens stream through shared memory; that is bound by the latency of a token
// (its products with k and q and the sum over a row's lanes), so sequences of
// more than a few tokens are for the chunked forms (linear_attn_tc.cu,
// linear_attn_f32.cu; the bound is in linear_plan.cuh).
//
// Measured: decode of 64 rows (16 heads of 128 x 128, bf16; 118 MB) 20.2 us, 5.9
// TB/s, 86 % of a plain copy's rate, of 203 (2 and 32 heads, 128 x 64, fp32; 429
// MB) 66.3 us, 95 %; one row 4.2, a launch's latency.  37 sequences of 1 to 9
// tokens (8 and 16 heads of 128 x 128, bf16; 80 MB) 20.5 us in a graph and 21.7
// called back to back: the states' loads and stores, 12 at a copy's rate, have
// the tokens' arithmetic between them (issue slots 58 % busy).
#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;

template <int DK, int R> struct LGeo {
    static constexpr int LPR = DK / 16;             // lanes a row
    static constexpr int RPW = 32 / LPR;            // rows a warp and pass
    static constexpr int PASS = RPW * kThreads / 32; // rows a CTA and pass
    static constexpr int ROWS = PASS * R;
};

// 16 elements of a lane, to fp32
__device__ __forceinline__ void load4(const float *p, float (&x)[4])
{
    *reinterpret_cast<float4 *>(x) = *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4])
{
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
}

// S' of 16 elements, and this lane's share of S' q
__device__ __forceinline__ float update(float (&s)[4][4], float a, float v, const float (&k)[4][4], const float (&q)[4][4])
{
    const float2 a2 = make_float2(a, a), v2 = make_float2(v, v);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float2 x = mul2(make_float2(s[j][e], s[j][e + 1]), a2);
            x = fma2(v2, make_float2(k[j][e], k[j][e + 1]), x);
            sum = fma2(x, make_float2(q[j][e], q[j][e + 1]), sum);
            s[j][e] = x.x, s[j][e + 1] = x.y;
        }
    return sum.x + sum.y;
}
__device__ __forceinline__ float decay_of(float g) { return expf(g > 0.f ? 0.f : g); }
template <int LPR> __device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ---- one token a row ----
template <typename T, int DK, int R> __global__ void __launch_bounds__(kThreads) linear_decode_kernel(const LinearArgs p)
{
    typedef LGeo<DK, R> G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % G::LPR;
    const int blocks = (p.dv + G::ROWS - 1) / G::ROWS;
    const int block = blockIdx.x % blocks, x = blockIdx.x / blocks, h = x % p.hv, r = x / p.hv;
    const int row0 = block * G::ROWS + warp * G::RPW + lane / G::LPR; // this lane's first row
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_prior_grid();
    const int rs = p.read_slot[r], ws = p.write_slot ? p.write_slot[r] : rs;
    const int cls = classify_row(rs, ws, p.num_slots, p.write_slot == nullptr);
    T *const out = static_cast<T *>(p.out) + ((size_t)r * p.hv + h) * p.dv;
    if (cls != 1) {
        if (cls < 0 && threadIdx.x == 0)
            report(p.err, GDN_DEVERR_BAD_SLOT);
        for (int i = threadIdx.x; i < G::ROWS; i += kThreads)
            if (block * G::ROWS + i < p.dv)
                out[block * G::ROWS + i] = from_f<T>(0.f);
        return;
    }
    const size_t head = (size_t)h * p.dv * DK, slot = (size_t)p.hv * p.dv * DK;
    const float *const from = p.pool + slot * rs + head + 4 * l;
    float *const to = p.pool + slot * ws + head + 4 * l;
    float s[R][4][4] = {}, k[4][4], q[4][4], v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = row0 + i * G::PASS;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (row < p.dv)
                *reinterpret_cast<float4 *>(s[i][j]) = ld_state(from + (size_t)row * DK + 4 * G::LPR * j);
    }
    const int hk = h / (p.hv / p.hk);
    const T *const kp = static_cast<const T *>(p.k) + r * p.k_stride + hk * DK + 4 * l;
    const T *const qp = static_cast<const T *>(p.q) + r * p.q_stride + hk * DK + 4 * l;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        load4(kp + 4 * G::LPR * j, k[j]), load4(qp + 4 * G::LPR * j, q[j]);
#pragma unroll
    for (int i = 0; i < R; ++i)
        v[i] = row0 + i * G::PASS < p.dv ? to_f(static_cast<const T *>(p.v)[r * p.v_stride + h * p.dv + row0 + i * G::PASS]) : 0.f;
    const float a = decay_of(p.log_decay[r * p.decay_stride + h]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = row0 + i * G::PASS;
        const float o = row_sum<G::LPR>(update(s[i], a, v[i], k, q));
        if (row < p.dv) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                st_state(to + (size_t)row * DK + 4 * G::LPR * j, *reinterpret_cast<float4 *>(s[i][j]));
            if (l == 0)
                out[row] = from_f<T>(o * p.scale);
        }
    }
}

// ---- token after token ----
constexpr int kStages = 3;

template <typename T, int DK, int R> struct SGeo : LGeo<DK, R> {
    static constexpr int ROWS = LGeo<DK, R>::ROWS;
    static constexpr int TOKENS = DK * sizeof(T) > 512 ? 4 : 8; // a stage of the ring: three are 5 to 28 KB
    static constexpr int STAGE = TOKENS * (2 * DK + ROWS);      // elements: q, k, v of the tokens
    static constexpr int BYTES = kStages * STAGE * (int)sizeof(T);
};

__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm_addr(dst)), "l"(src) : "memory");
}

template <typename T, int DK, int R> __global__ void __launch_bounds__(kThreads) linear_serial_kernel(const LinearArgs p)
{
    typedef SGeo<T, DK, R> G;
    extern __shared__ __align__(16) unsigned char sm[];
    __shared__ float decay[kStages][G::TOKENS];
    constexpr int kTokens = G::TOKENS;
    T *const ring = reinterpret_cast<T *>(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane % G::LPR;
    const int blocks = (p.dv + G::ROWS - 1) / G::ROWS;
    const int row_in = warp * G::RPW + lane / G::LPR;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); // (the chunks' kernel goes on beside this one)
    const long long items = (long long)p.rows * p.hv * blocks;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int block = (int)(it % blocks), h = (int)(it / blocks % p.hv), r = (int)(it / blocks / p.hv);
        const int b = p.cu_seqlens[r], e = p.cu_seqlens[r + 1], rs = p.read_slot[r], ws = p.write_slot ? p.write_slot[r] : rs;
        const int cls = classify_seq(rs, ws, p.write_slot == nullptr, nullptr, b, e, p.total_tokens, p.num_slots);
        const int first = block * G::ROWS, rows = min(G::ROWS, p.dv - first);
        if (cls != 1) {
            if (cls < 0 && tid == 0)
                report(p.err, GDN_DEVERR_BAD_SLOT);
            const int vecs = rows * (int)sizeof(T) / 16; // of a token
            if (b >= 0 && e <= p.total_tokens) // (its own tokens, when there are such)
                for (int t = b + tid / vecs; tid < kThreads / vecs * vecs && t < e; t += kThreads / vecs)
                    reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + ((size_t)t * p.hv + h) * p.dv + first)[tid % vecs] =
                        make_uint4(0, 0, 0, 0);
            continue;
        }
        const int n = e - b;
        if (n > p.most || (n == 0 && !p.write_slot))
            continue;
        const size_t head = (size_t)h * p.dv * DK, slot = (size_t)p.hv * p.dv * DK;
        const float *const from = p.pool + slot * rs + head + (size_t)first * DK + 4 * l;
        float *const to = p.pool + slot * ws + head + (size_t)first * DK + 4 * l;
        float s[R][4][4] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = row_in + i * G::PASS;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (row < rows)
                    *reinterpret_cast<float4 *>(s[i][j]) = ld_state(from + (size_t)row * DK + 4 * G::LPR * j);
        }
        const int hk = h / (p.hv / p.hk);
        constexpr int VE = 16 / (int)sizeof(T), QV = DK / VE, VV = G::ROWS / VE; // elements a copy, copies of q and of v a token
        auto load = [&](int stage) { // a group of copies, empty past the end
            const int t0 = stage * kTokens, here = min(kTokens, n - t0);
            T *const to_s = ring + (stage % kStages) * G::STAGE;
            for (int i = tid; i < here * (2 * QV + VV); i += kThreads) {
                const int t = i / (2 * QV + VV), x = i - t * (2 * QV + VV);
                const long long tok = b + t0 + t;
                if (x < QV)
                    copy16(to_s + t * DK + x * VE, static_cast<const T *>(p.q) + tok * p.q_stride + hk * DK + x * VE);
                else if (x < 2 * QV)
                    copy16(to_s + (kTokens + t) * DK + (x - QV) * VE, static_cast<const T *>(p.k) + tok * p.k_stride + hk * DK + (x - QV) * VE);
                else if ((x - 2 * QV) * VE < rows)
                    copy16(to_s + 2 * kTokens * DK + t * G::ROWS + (x - 2 * QV) * VE,
                           static_cast<const T *>(p.v) + tok * p.v_stride + h * p.dv + first + (x - 2 * QV) * VE);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (tid < here)
                decay[stage % kStages][tid] = decay_of(p.log_decay[(b + t0 + tid) * p.decay_stride + h]);
        };
        __syncthreads(); // the item before is done with the ring
        const int stages = (n + kTokens - 1) / kTokens;
        load(0), load(1);
        for (int st = 0; st < stages; ++st) {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncthreads(); // the stage is there for all, and the one before it is done with
            load(st + 2);
            const T *const q = ring + (st % kStages) * G::STAGE + 4 * l, *const k = q + kTokens * DK;
            const T *const v = ring + (st % kStages) * G::STAGE + 2 * kTokens * DK + row_in;
            const int here = min(kTokens, n - st * kTokens);
            for (int t = 0; t < here; ++t) {
                float kf[4][4], qf[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load4(k + t * DK + 4 * G::LPR * j, kf[j]), load4(q + t * DK + 4 * G::LPR * j, qf[j]);
                const float a = decay[st % kStages][t];
                T *const out = static_cast<T *>(p.out) + ((size_t)(b + st * kTokens + t) * p.hv + h) * p.dv + first + row_in;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const bool there = row_in + i * G::PASS < rows;
                    const float o = row_sum<G::LPR>(update(s[i], a, there ? to_f(v[t * G::ROWS + i * G::PASS]) : 0.f, kf, qf));
                    if (there && l == 0)
                        out[i * G::PASS] = from_f<T>(o * p.scale);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int row = row_in + i * G::PASS;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (row < rows)
                    st_state(to + (size_t)row * DK + 4 * G::LPR * j, *reinterpret_cast<float4 *>(s[i][j]));
        }
    }
}

template <typename T, int DK> cudaError_t decode(const LinearArgs &a, cudaStream_t s)
{
    constexpr int R = 2; // rows a lane: with one the 64 rows above take 22.6 us and the 203 81, with four 20.5 and 65.4
    const long long blocks = (long long)a.rows * a.hv * ((a.dv + LGeo<DK, R>::ROWS - 1) / LGeo<DK, R>::ROWS);
    if (blocks > 0x7fffffffll)
        return cudaErrorInvalidConfiguration;
    return launch_pdl(linear_decode_kernel<T, DK, R>, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
}
template <typename T, int DK> cudaError_t serial(const LinearArgs &a, cudaStream_t s)
{
    constexpr int R = 2;
    typedef SGeo<T, DK, R> G;
    static_assert(G::BYTES <= 48 * 1024, "shared memory");
    const long long items = (long long)a.rows * a.hv * ((a.dv + G::ROWS - 1) / G::ROWS);
    const unsigned grid = (unsigned)(items < 152 * 64 ? items : 152 * 64);
    return launch_pdl(linear_serial_kernel<T, DK, R>, dim3(grid), dim3(kThreads), (size_t)G::BYTES, s, a);
}
template <typename T> cudaError_t by_dk(const LinearArgs &a, bool prefill, cudaStream_t s)
{
    switch (a.dk) {
    case 16:
        return prefill ? serial<T, 16>(a, s) : decode<T, 16>(a, s);
    case 32:
        return prefill ? serial<T, 32>(a, s) : decode<T, 32>(a, s);
    case 64:
        return prefill ? serial<T, 64>(a, s) : decode<T, 64>(a, s);
    case 128:
        return prefill ? serial<T, 128>(a, s) : decode<T, 128>(a, s);
    default:
        return prefill ? serial<T, 256>(a, s) : decode<T, 256>(a, s);
    }
}

} // namespace

cudaError_t launch_linear_decode(const LinearArgs &a, int dtype, cudaStream_t s)
{
    return dtype == GDN_BF16 ? by_dk<__nv_bfloat16>(a, false, s) : by_dk<float>(a, false, s);
}
cudaError_t launch_linear_serial(const LinearArgs &a, int dtype, cudaStream_t s)
{
    return dtype == GDN_BF16 ? by_dk<__nv_bfloat16>(a, true, s) : by_dk<float>(a, true, s);
}

} // namespace gdn
