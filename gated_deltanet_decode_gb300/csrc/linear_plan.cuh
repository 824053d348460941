// How the chunked kernels of linear attention divide packed sequences (sm_103a).
//
// A sequence is cut into segments of `span` tokens, whole chunks, so that few
// sequences still fill the GPU: as a decay is a number, S' = a S + sum, the sums
// of different segments do not depend on each other.  One kernel forms every
// segment's own sum (all but a sequence's last), linear_scan_kernel turns them
// into the states after each segment, and another kernel goes through the
// segments, each from its state.  Sequences of one segment need only the last.
// Included by one translation unit a kernel; everything here has internal
// linkage.
#pragma once

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kSms = 152;
constexpr int kMostChunks = 1 << 20; // of a segment: its tokens stay within an int
// Tokens up to which a sequence is the serial kernel's: a chunk takes the time of some tens of its steps.  37 sequences of 12
// (bf16, 16 heads of 128) take 31.8 us there and 44.3 in chunks, of 20 49.6 and 60.3, of 32 83.7 and 60.0; 4 sequences of 12
// 7.7 and 13.6, of 24 17.4 and 13.6; in fp32 (8 heads of 64) 37 of 12 15.6 and 23.7, of 24 22.5 and 24.4, of 32 26.6 and 24.7.
constexpr int kSerial = 20;

struct ChunkArgs {
    LinearArgs a;
    int least;    // sequences of more tokens than this are divided into segments; the others are the serial kernel's
    // Whether the host expects no sequence of several segments.  The sums' kernel and the scan, there for a long sequence among
    // short ones, then look for one first: 8 sequences of 1,500 to 2,600 tokens take 92.6 us, without the look 94.5, and 87.4
    // without the two kernels; 8 of 300 27.7, 30.6 and 23.7.  (Here and below in a graph; called back to back 1 more.)
    int rare;
    // Whether it expects no sequence for the chunks at all, by the mean: their kernel then looks before it sets up.  37
    // sequences of 1 to 9 tokens take 20.5 us, without the look 22.2, 4 of 12 7.7 and 10.1; with chunks to do it costs 0.5.
    int none;
    int heads;    // value heads, or blocks of their rows where a CTA takes less than a head
    float *state; // [segments][hv][dv][dk]: a segment's sum, then the state after it (a sequence's last: the state before all)
    float *decay; // [segments][hv]: the segment's decay
};

// The kernels of a call run beside each other as far as they can: each lets the next one start at once, but for the serial one,
// which does so when its own wait for the grid before is over.  What came before the call is complete then, and of the call's
// own kernels only the scan reads what another one wrote (the sums), and then the segments that begin with the scan's states:
// those wait, a sequence of a single segment does not.  Every kernel waits at its end at the latest, so that who comes next
// has all of them behind it.  One after the other, a sequence of 16,000 tokens (bf16, 16 heads of 128) takes 99.6 us instead of
// 95.0, five of 200 to 900 in fp32 (8 heads of 64) 39.1 instead of 30.0, 37 of 1 to 9 in bf16 1.0 less.
__device__ __forceinline__ void begin_chunks()
{
    __threadfence(); // this SM's L1 may hold lines of a grid before the call
}

// A segment of a sequence and head.
struct LItem {
    int tok, n, head; // first token, tokens (0: no more items), value head (or block)
    int rs, ws;       // the sequence's slots
    int at, from;     // places in the workspace: the segment's, and of the state before it (-1: read slot)
    int last;         // of its sequence
};

// A sequence's segments: none where it is the serial kernel's, padding or bad.
__device__ __forceinline__ int segments(const ChunkArgs &p, int r, int &b, int &n, int &rs, int &ws)
{
    b = p.a.cu_seqlens[r];
    const int e = p.a.cu_seqlens[r + 1];
    rs = p.a.read_slot[r], ws = p.a.write_slot ? p.a.write_slot[r] : rs;
    n = 0;
    if (classify_seq(rs, ws, p.a.write_slot == nullptr, nullptr, b, e, p.a.total_tokens, p.a.num_slots) != 1)
        return 0;
    n = e - b;
    return n > p.least ? n / p.a.span + (n % p.a.span != 0) : 0;
}
// The workspace's places of a sequence's segments begin at its first token's
// place over a segment's length and one a sequence before it, so no two meet.
__device__ __forceinline__ int first_place(const ChunkArgs &p, int b, int r) { return b / p.a.span + r; }
// Whether a sequence has `most` segments or more.  By all threads of a CTA.
__device__ __forceinline__ bool any_with(const ChunkArgs &p, int most)
{
    int any = 0;
    for (int r = threadIdx.x; r < p.a.rows; r += blockDim.x) {
        int b, n, rs, ws;
        any |= segments(p, r, b, n, rs, ws) >= most;
    }
    return __syncthreads_or(any);
}
inline long long places(int nseq, int tokens, long long span) { return tokens / span + nseq + 1; }

// The items of a CTA: number blockIdx.x and every gridDim.x-th on, heads of a
// segment next to each other.  By one warp; SUM leaves out the last segments.
template <bool SUM> struct ItemWalk {
    const ChunkArgs &p;
    const int lane;
    long long i;     // the next item
    long long done;  // items of the sequences before `row`
    int row;         // the window's first sequence
    int b, n, rs, ws, segs;
    __device__ explicit ItemWalk(const ChunkArgs &p_) : p(p_), lane(threadIdx.x & 31), i(blockIdx.x), done(0), row(0) { look(); }
    __device__ void look()
    {
        segs = 0;
        if (row + lane < p.a.rows)
            segs = segments(p, row + lane, b, n, rs, ws);
        if (SUM && segs > 0)
            --segs;
    }
    __device__ bool next(LItem &it)
    {
        for (; row < p.a.rows; row += 32, look()) {
            int upto = segs;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o)
                    upto += x;
            }
            const long long all = (long long)__shfl_sync(0xffffffffu, upto, 31) * p.heads;
            if (i >= done + all) {
                done += all;
                continue;
            }
            const int s = (int)((i - done) / p.heads), h = (int)((i - done) - (long long)s * p.heads);
            const int who = __ffs(__ballot_sync(0xffffffffu, upto > s)) - 1;
            const int seg = s - __shfl_sync(0xffffffffu, upto - segs, who), span = p.a.span;
            const int wb = __shfl_sync(0xffffffffu, b, who), wn = __shfl_sync(0xffffffffu, n, who);
            const int count = __shfl_sync(0xffffffffu, segs, who) + (SUM ? 1 : 0);
            it.tok = wb + seg * span, it.n = min(span, wn - seg * span), it.head = h;
            it.rs = __shfl_sync(0xffffffffu, rs, who), it.ws = __shfl_sync(0xffffffffu, ws, who);
            it.at = first_place(p, wb, row + who) + seg;
            it.from = seg > 0 ? it.at - 1 : count > 1 ? it.at + count - 1 : -1;
            it.last = seg == count - 1;
            i += gridDim.x;
            return true;
        }
        return false;
    }
};

// A number in two floats, and the sum of two such (Knuth's two-sum; in fp64 128
// sums took 11,000 clocks, more than all else of a chunk).
struct Two {
    float h, l;
};
__device__ __forceinline__ Two operator+(Two a, Two b)
{
    const float s = a.h + b.h, x = s - a.h, e = ((a.h - (s - x)) + (b.h - x)) + (a.l + b.l);
    const float h = s + e;
    return {h, e - (h - s)};
}
__device__ __forceinline__ Two shuffle(Two a, int from) { return {__shfl_sync(0xffffffffu, a.h, from), __shfl_sync(0xffffffffu, a.l, from)}; }
__device__ __forceinline__ Two log2_units(float x) // x log2 e
{
    constexpr float L = 1.44269504f, M = 1.92596303e-8f; // log2 e in two floats
    const float h = x * L;
    return {h, fmaf(x, L, -h) + x * M};
}
__device__ __forceinline__ float minus(Two a, Two b) { return (a.h - b.h) + (a.l - b.l); }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The state after each segment but a sequence's last, from the segments' sums,
// in their places: a thread four floats of a (sequence, head).
__global__ void __launch_bounds__(256) linear_scan_kernel(const ChunkArgs p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_prior_grid();
    if (p.rare && !any_with(p, 2))
        return;
    const int floats = p.a.dv * p.a.dk, parts = (floats + 1023) / 1024;
    for (long long at = blockIdx.x; at < (long long)p.a.rows * p.a.hv * parts; at += gridDim.x) {
        const int part = (int)(at % parts), x = (int)(at / parts), h = x % p.a.hv, r = x / p.a.hv;
        int b, n, rs, ws;
        const int segs = segments(p, r, b, n, rs, ws);
        if (segs < 2 || part * 1024 + 4 * (int)threadIdx.x >= floats)
            continue;
        const size_t slot = (size_t)p.a.hv * floats, mine = (size_t)h * floats + part * 1024 + 4 * threadIdx.x;
        const size_t place = first_place(p, b, r);
        float4 s = *reinterpret_cast<const float4 *>(p.a.pool + slot * rs + mine);
        // (the first segment takes its state from the last one's place: in place, the slot is written by the last segment)
        *reinterpret_cast<float4 *>(p.state + slot * (place + segs - 1) + mine) = s;
        constexpr int U = 4; // segments under way
        for (int i0 = 0; i0 < segs - 1; i0 += U) {
            float4 y[U];
            float f[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < segs - 1) {
                    y[u] = *reinterpret_cast<const float4 *>(p.state + slot * (place + i0 + u) + mine);
                    f[u] = p.decay[(place + i0 + u) * p.a.hv + h];
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u < segs - 1) {
                    s.x = fmaf(s.x, f[u], y[u].x), s.y = fmaf(s.y, f[u], y[u].y);
                    s.z = fmaf(s.z, f[u], y[u].z), s.w = fmaf(s.w, f[u], y[u].w);
                    *reinterpret_cast<float4 *>(p.state + slot * (place + i0 + u) + mine) = s;
                }
        }
    }
}

inline cudaError_t launch_scan(const ChunkArgs &p, cudaStream_t s)
{
    const long long blocks = (long long)p.a.rows * p.a.hv * ((p.a.dv * p.a.dk + 1023) / 1024);
    const long long most = (p.rare ? 1 : 4) * kSms;
    return launch_pdl(linear_scan_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s, p);
}

// The cheapest of the lengths that m chunks have when cut evenly in up to `most` pieces, each looked at once (about 2 sqrt(m);
// looking at every number of pieces took 9 us of host time for 40,000 tokens).  cost(segments, length)
template <typename Cost> long long cheapest_length(long long m, long long most, const Cost &cost)
{
    long long best = m;
    double least = 1e30;
    for (long long cuts = 1; cuts <= m && cuts <= most;) {
        const long long len = (m + cuts - 1) / cuts;
        const double c = cost((m + len - 1) / len, len);
        if (c < least)
            least = c, best = len;
        if (len == 1)
            break;
        cuts = (m + len - 2) / (len - 1); // the fewest that give a shorter one
    }
    return best;
}

// The workspace: states, then decays.
inline size_t chunk_bytes(const LinearArgs &a)
{
    return sizeof(float) * (size_t)places(a.rows, a.total_tokens, a.span) * a.hv * ((size_t)a.dv * a.dk + 1);
}
inline void chunk_layout(ChunkArgs &p)
{
    p.state = static_cast<float *>(p.a.work);
    p.decay = p.state + (size_t)places(p.a.rows, p.a.total_tokens, p.a.span) * p.a.hv * p.a.dv * p.a.dk;
}

} // namespace
} // namespace gdn
