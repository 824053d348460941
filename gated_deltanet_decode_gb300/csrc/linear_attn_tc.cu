// Linear attention with a decay for each head over packed sequences in chunks
// of C = 128 tokens on the tensor cores (sm_103a), bf16 activations, dk and dv
// 64 or 128.  With G_i the sum of the log decays up to token i of a chunk and S
// the state before it,
//   o_i = scale (e^{G_i} S q_i + sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j)
//   S'  = e^{G_C} S + sum_j e^{G_C - G_j} v_j k_j^T,
// which regroups the recurrence token after token (linear_attn.cu); as a decay
// is a number, the sums over j of different chunks do not depend on each other.
//
// Work.  A sequence's chunks are cut into segments of L, so that few sequences
// still fill the GPU.  linear_sum_kernel forms every segment's own sum (all but
// a sequence's last), linear_scan_kernel turns them into the states after each
// segment, and linear_chunk_kernel goes through the segments, each from its
// state.  Sequences of one segment need only the last.  Sequences of up to
// kSerial tokens are the serial kernel's: a chunk's products take the time of
// some tens of its steps.
//
// linear_chunk_kernel: persistent, one CTA an SM.  Warp 0 brings Q, K and V by
// tensor copies into four tiles that change roles (a chunk's V takes the tile
// that was free, K the last Q's, Q the last V's), so that each copy runs a chunk
// ahead as soon as its tile is read; warp 1 issues the products, warp 2 forms
// the decays, warp 3 walks the items.  Eight warps compute, a thread a row and
// half of its columns: Q K^T to weights (bf16, over the scores in tensor
// memory), V times its weights, the outputs, and the state, which stays in their
// registers.
//
// Precision.  The state is to be right to fp32, and its products' operands are
// bf16: e^{G_C - G_j} v_j is cut into three bf16 values that make it up exactly
// (8 bits each of 24), so a chunk's sum takes three products; K is bf16 as it
// comes.  A chunk's sum is added to the state in fp32 outside the tensor cores,
// whose own additions cut results short.  The weights and the state, as
// operands of the outputs alone, are rounded to bf16 once: outputs are off by
// 0.0023 of their norm instead of the 0.0017 of their own rounding, and three
// products of each would take as long again as all of them.
#include <atomic>
#include <cstring>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "tc_ops.cuh"

namespace gdn {
namespace {

constexpr int kC = 128;        // tokens a chunk
constexpr int kThreads = 384;  // 4 warps of their own and 8 that compute
constexpr int kQueue = 4;      // items in flight between the walking warp and the others
constexpr int kReaders = 11;   // warps 0, 1, 2 and the computing ones
constexpr int kSerial = 32;    // tokens up to which a sequence is the serial kernel's
constexpr int kSms = 152;

struct ChunkArgs {
    LinearArgs a;
    int seg;      // chunks a segment
    float *state; // [segments][hv][dv][dk]: a segment's sum, then the state after it (a sequence's last: the state before all)
    float *decay; // [segments][hv]: the segment's decay
};

// A segment of a sequence and head.
struct LItem {
    int tok, n, head; // first token, tokens (0: no more items), value head
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
    const int span = kC * p.seg;
    return n > kSerial ? n / span + (n % span != 0) : 0;
}
// The workspace's places of a sequence's segments begin at its first token's
// place over a segment's length and one a sequence before it, so no two meet.
__device__ __forceinline__ int first_place(const ChunkArgs &p, int b, int r) { return b / (kC * p.seg) + r; }
inline long long places(int nseq, int tokens, int seg) { return (long long)tokens / ((long long)kC * seg) + nseq + 1; }

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
            const long long all = (long long)__shfl_sync(0xffffffffu, upto, 31) * p.a.hv;
            if (i >= done + all) {
                done += all;
                continue;
            }
            const int s = (int)((i - done) / p.a.hv), h = (int)((i - done) - (long long)s * p.a.hv);
            const int who = __ffs(__ballot_sync(0xffffffffu, upto > s)) - 1;
            const int seg = s - __shfl_sync(0xffffffffu, upto - segs, who), span = kC * p.seg;
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

// Decays of a chunk, by warp 2.  In units of log2: -G is up to 2^15 for decays
// that forget everything (a token's is cut off at e^-110, below half of the
// smallest number), and differences of it are wanted to 2^-24, so it comes in
// two floats.
struct alignas(16) Decays {
    float hi[kC], lo[kC];     // G_j
    float w[kC];              // e^{G_C - G_j}
    float c[kC];              // e^{R - G_j}, R = G at the end of token j's block of 32
    float rhi[4], rlo[4];     // R
    float all;                // e^{G_C}
};
// FULL: all of it, else w and `all`
template <bool FULL, typename Tab>
__device__ __forceinline__ void form_decays(const LinearArgs &a, int tok, int n, int head, Tab &t)
{
    const int lane = threadIdx.x & 31;
    double g[4];
    double sum = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = 4 * lane + e;
        float x = j < n ? a.log_decay[(long long)(tok + j) * a.decay_stride + head] : 0.f;
        x = x > 0.f ? 0.f : x < -110.f ? -110.f : x; // (a NaN stays)
        sum += (double)x * 1.4426950408889634;
        g[e] = sum;
    }
    double upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o)
            upto += x;
    }
    const double before = upto - sum, all = __shfl_sync(0xffffffffu, upto, 31);
    const double block = __shfl_sync(0xffffffffu, upto, lane | 7);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = 4 * lane + e;
        const double G = before + g[e];
        t.w[j] = exp2f((float)(all - G));
        if constexpr (FULL) {
            t.hi[j] = (float)G;
            t.lo[j] = (float)(G - (double)(float)G);
            t.c[j] = exp2f((float)(block - G));
        }
    }
    if constexpr (FULL)
        if ((lane & 7) == 7) {
            t.rhi[lane >> 3] = (float)block;
            t.rlo[lane >> 3] = (float)(block - (double)(float)block);
        }
    if (lane == 0)
        t.all = exp2f((float)all);
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Whether one of eight bf16 is not finite
__device__ __forceinline__ bool odd8(uint4 z)
{
    const uint32_t m = 0x7f807f80u, c = 0x00800080u;
    return ((((z.x & m) + c) | ((z.y & m) + c) | ((z.z & m) + c) | ((z.w & m) + c)) & 0x80008000u) != 0;
}
// Two floats, each cut into three bf16 values that make it up: heads, middles, tails as pairs.
__device__ __forceinline__ void cut3(float x, float y, uint32_t &h, uint32_t &m, uint32_t &l)
{
    const uint32_t xh = __float_as_uint(x), yh = __float_as_uint(y);
    h = __byte_perm(xh, yh, 0x7632);
    const float x1 = x - __uint_as_float(xh & 0xffff0000u), y1 = y - __uint_as_float(yh & 0xffff0000u);
    const uint32_t xm = __float_as_uint(x1), ym = __float_as_uint(y1);
    m = __byte_perm(xm, ym, 0x7632);
    const float x2 = x1 - __uint_as_float(xm & 0xffff0000u), y2 = y1 - __uint_as_float(ym & 0xffff0000u);
    l = __byte_perm(__float_as_uint(x2), __float_as_uint(y2), 0x7632);
}
// 16 bytes of V times a weight, cut in three
__device__ __forceinline__ void weigh(uint4 z, float w, unsigned char *to, int term)
{
    uint4 h, m, l;
    const uint32_t in[4] = {z.x, z.y, z.z, z.w};
    uint32_t o[3][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = mul2(make_float2(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xffff0000u)), make_float2(w, w));
        cut3(x.x, x.y, o[0][e], o[1][e], o[2][e]);
    }
    h = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
    m = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
    l = make_uint4(o[2][0], o[2][1], o[2][2], o[2][3]);
    *reinterpret_cast<uint4 *>(to) = h;
    *reinterpret_cast<uint4 *>(to + term) = m;
    *reinterpret_cast<uint4 *>(to + 2 * term) = l;
}

template <int DK, int DV> struct CGeo {
    static constexpr int D = DK > DV ? DK : DV;
    static constexpr int TILE = kC * D * 2;           // a Q, K or V tile, as 64-column blocks of kC rows
    static constexpr int BLOCK = kC * 128;            // one such block
    static constexpr int KBYTES = kC * DK * 2, VBYTES = kC * DV * 2;
    static constexpr int TERM = 64 * DV * 2;          // a third of weighted V for half of a chunk
    static constexpr int WBYTES = (DV == 64 ? 4 : 3) * TERM; // (products take 128 rows of it: with dv = 64 the next term's, unused)
    static constexpr int SBYTES = DV * DK * 2;        // the state in bf16
};

// What both kernels wait for each other with.
struct Bars {
    unsigned long long ifull[kQueue], iempty[kQueue];
    unsigned long long gfull[2], gempty[2]; // decays
    unsigned long long full[4], empty[4];   // tiles
    unsigned long long wready[2], wdone[2]; // halves of weighted V: written; read by their products
    unsigned long long drain;
};

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int blocks, int head, int tok, uint32_t bar, int bytes)
{
    mbar_arrive_tx(bar, bytes);
    for (int c = 0; c < blocks; ++c)
        tma3(dst + c * kC * 128, map, 64 * c, head, tok, bar);
}

// ---- the outputs, and the states at the sequences' ends ----
template <int DK, int DV> struct ChunkCtrl {
    Bars b;
    unsigned long long qk, pready, odone, dsdone, sready;
    LItem item[kQueue];
    Decays tab[2];
    int badfrom[3][kC]; // by chunk: first token with a value that is not finite, by column
    int dirty[3];       // whether there is one
    uint32_t tmem;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const ChunkArgs p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap)
{
    typedef CGeo<DK, DV> G;
    typedef ChunkCtrl<DK, DV> Ctrl;
    constexpr int SAT = 4 * G::TILE, WAT = SAT + G::SBYTES, CAT = WAT + G::WBYTES;
    static_assert(CAT % 1024 == 0 && CAT + sizeof(Ctrl) <= 232448, "shared memory");
    constexpr uint32_t CS = 0, CO1 = 128, CO2 = 256, CD = 384; // tensor memory: scores and weights, the chunk's own part, the
                                                               // state's part, the chunk's sum
    constexpr int HK = DK / 2, HV = DV / 2;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctrl &ctl = *reinterpret_cast<Ctrl *>(smem + CAT);
    const uint32_t sbase = sm_addr(smem);
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](unsigned long long &b) { return sm_addr(&b); };
    if (sbase & 1023) { // the swizzled tiles need it; the whole CTA leaves
        if (tid == 0)
            report(a.err, GDN_DEVERR_TIMEOUT);
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&ctl.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 64) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < kQueue; ++i)
            mbar_init(bar(ctl.b.ifull[i]), 1), mbar_init(bar(ctl.b.iempty[i]), kReaders);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctl.b.gfull[i]), 1), mbar_init(bar(ctl.b.gempty[i]), 8);
            mbar_init(bar(ctl.b.wready[i]), 8), mbar_init(bar(ctl.b.wdone[i]), 1);
        }
        for (int i = 0; i < 4; ++i)
            mbar_init(bar(ctl.b.full[i]), 1), mbar_init(bar(ctl.b.empty[i]), 1);
        mbar_init(bar(ctl.qk), 1), mbar_init(bar(ctl.pready), 8), mbar_init(bar(ctl.odone), 1);
        mbar_init(bar(ctl.dsdone), 1), mbar_init(bar(ctl.sready), 8), mbar_init(bar(ctl.b.drain), 1);
        ctl.dirty[0] = ctl.dirty[1] = ctl.dirty[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 3 * kC; i += kThreads)
        (&ctl.badfrom[0][0])[i] = kC;
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = ctl.tmem;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true; // false once a bounded wait ran out
    auto wait_at = [&](uint32_t b, uint32_t parity) { // by a whole warp, which goes on or leaves as one
        if (!__all_sync(0xffffffffu, mbar_try(b, parity)) && alive && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
            alive = false;
            report(a.err, GDN_DEVERR_TIMEOUT);
        }
        return alive;
    };
    auto wait = [&](unsigned long long &b, uint32_t parity) { return wait_at(bar(b), parity); };
    auto arrive = [&](unsigned long long &b) { // a warp
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(b));
        __syncwarp();
    };
    // the item of the queue's turn q
    auto take = [&](int q, LItem &it) {
        const int slot = q % kQueue;
        if (!wait(ctl.b.ifull[slot], (q / kQueue) & 1))
            return false;
        it = ctl.item[slot];
        arrive(ctl.b.iempty[slot]);
        return it.n > 0;
    };
    // the tiles' roles in the current chunk, and the phases of their barriers, a bit a tile
    int tq = 0, tk = 1, tv = 2, tf = 3;
    auto turn = [&] {
        const int q = tv, k = tq, v = tf, f = tk;
        tq = q, tk = k, tv = v, tf = f;
    };
    uint32_t phase = 0;
    auto wait_tile = [&](int t) {
        const uint32_t parity = (phase >> t) & 1;
        phase ^= 1u << t;
        return wait(ctl.b.full[t], parity);
    };
    auto tile = [&](int t) { return sbase + t * G::TILE; };
    unsigned ch = 0; // chunks done
    LItem it;

    if (warp == 3) {
        ItemWalk<false> walk(p);
        for (int q = 0; alive; ++q) {
            LItem x;
            const bool more = walk.next(x);
            const int slot = q % kQueue;
            if (!wait(ctl.b.iempty[slot], (q / kQueue + 1) & 1))
                break;
            if (!more)
                x.n = 0;
            if (lane == 0) {
                ctl.item[slot] = x;
                mbar_arrive(bar(ctl.b.ifull[slot]));
            }
            __syncwarp();
            if (!more)
                break;
        }
    } else if (warp == 0) {
        // ---- Q, K and V
        uint32_t loaded = 0; // tiles that were asked for at least once
        auto load = [&](int t, const CUtensorMap *map, int blocks, int head, int tok, int bytes) {
            if (!wait(ctl.b.empty[t], ((phase >> t) & 1) ^ 1))
                return false;
            phase ^= 1u << t;
            loaded |= 1u << t;
            if (lane == 0)
                load_tile(tile(t), map, blocks, head, tok, bar(ctl.b.full[t]), bytes);
            __syncwarp();
            return true;
        };
        for (int q = 0; take(q, it); ++q) {
            const int hk = it.head / (a.hv / a.hk);
            for (int t = 0; t < it.n && alive; t += kC, turn()) {
                if (!load(tv, &vmap, DV / 64, it.head, it.tok + t, G::VBYTES) || !load(tk, &kmap, DK / 64, hk, it.tok + t, G::KBYTES) ||
                    !load(tq, &qmap, DK / 64, hk, it.tok + t, G::KBYTES))
                    break;
            }
            if (!alive)
                break;
        }
        // the last copies land before the CTA leaves, whoever still waits for them
        for (int t = 0; t < 4; ++t)
            if (loaded >> t & 1)
                mbar_wait(bar(ctl.b.full[t]), ((phase >> t) & 1) ^ 1);
    } else if (warp == 1) {
        // ---- the products, issued by one elected lane of the whole warp's walk
        const bool leader = elect();
        auto scores = [&] { // Q K^T of the current tiles
            if (!wait_tile(tq) || !wait_tile(tk))
                return false;
            after_sync();
            if (leader) {
                const uint64_t qd = desc_k(tile(tq)), kd = desc_k(tile(tk));
#pragma unroll
                for (int k = 0; k < DK / 16; ++k) {
                    const uint64_t at = ((k >> 2) * G::BLOCK + (k & 3) * 32) >> 4;
                    mma_ss(tmem + CS, qd + at, kd + at, idesc(kC, false), k > 0);
                }
                commit(bar(ctl.qk));
            }
            return true;
        };
        auto sum = [&](int half) { // of the chunk's weighted V and K, tokens 64 half ..
            if (leader) {
                const uint64_t kd = desc_mn(tile(tk) + half * 64 * 128, G::BLOCK);
                const uint64_t wd = desc_mn(sbase + WAT, 64 * 128);
#pragma unroll
                for (int x = 2; x >= 0; --x) // the small terms first
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ss(tmem + CD, wd + ((x * G::TERM + k * 2048) >> 4), kd + (k * 2048 >> 4), idesc(DK, true, true),
                               half > 0 || x < 2 || k > 0);
            }
        };
        auto own = [&](int half) { // the weights times V
            if (leader) {
                const uint64_t vd = desc_mn(tile(tv) + half * 64 * 128, G::BLOCK);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_ts(tmem + CO1, tmem + CS + 64 * half + 8 * k, vd + (k * 2048 >> 4), idesc(DV, true), half > 0 || k > 0);
            }
        };
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                const uint32_t par = ch & 1;
                if (t == 0 && !scores())
                    break;
                if (!wait(ctl.sready, par))
                    break;
                after_sync();
                if (leader) { // the state times q
                    const uint64_t qd = desc_k(tile(tq)), sd = desc_k(sbase + SAT);
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_ss(tmem + CO2, qd + (((k >> 2) * G::BLOCK + (k & 3) * 32) >> 4),
                               sd + (((k >> 2) * DV * 128 + (k & 3) * 32) >> 4), idesc(DV, false), k > 0);
                    commit(bar(ctl.b.empty[tq]));
                }
                if (!wait(ctl.b.wready[0], par) || !wait_tile(tv))
                    break;
                after_sync();
                sum(0);
                if (leader)
                    commit(bar(ctl.b.wdone[0]));
                if (!wait(ctl.pready, par))
                    break;
                after_sync();
                own(0);
                if (!wait(ctl.b.wready[1], par))
                    break;
                after_sync();
                own(1);
                if (leader) {
                    commit(bar(ctl.odone));
                    commit(bar(ctl.b.empty[tv]));
                }
                sum(1);
                if (leader) {
                    commit(bar(ctl.dsdone));
                    commit(bar(ctl.b.empty[tk]));
                }
                turn();
                if (t + kC < it.n && !scores())
                    break;
            }
            if (!alive)
                break;
        }
        // everything issued is done before tensor memory and the barriers go
        __syncwarp();
        if (leader)
            commit(bar(ctl.b.drain));
        __syncwarp();
        mbar_wait(bar(ctl.b.drain), 0);
    } else if (warp == 2) {
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                if (!wait(ctl.b.gempty[ch & 1], ((ch >> 1) & 1) ^ 1))
                    break;
                form_decays<true>(a, it.tok + t, min(kC, it.n - t), it.head, ctl.tab[ch & 1]);
                arrive(ctl.b.gfull[ch & 1]);
            }
            if (!alive)
                break;
        }
    } else {
        const int w4 = warp & 3, hb = (warp - 4) >> 2, row = 32 * w4 + lane, ct = tid - 128; // 0 .. 255
        const uint32_t lanes = (uint32_t)w4 << 21;
        const bool has = row < DV; // whether this thread keeps a part of the state: row `row`, columns hb HK ..
        float s[HK];
        auto write_state = [&] { // in bf16, for the products
            if (has) {
#pragma unroll
                for (int k = 0; k < HK; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(s[k + 2 * e], s[k + 2 * e + 1]);
                        w[e] = *reinterpret_cast<const uint32_t *>(&h2);
                    }
                    const int col = hb * HK + k;
                    *reinterpret_cast<uint4 *>(smem + SAT + (col >> 6) * DV * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            smem_to_async();
            before_sync();
            arrive(ctl.sready);
        };
        for (int q = 0; take(q, it); ++q) {
            const size_t head = (size_t)it.head * DV * DK, slot = (size_t)a.hv * DV * DK, mine = (size_t)row * DK + hb * HK;
            {
                const float *const from = it.from < 0 ? a.pool + slot * it.rs + head + mine : p.state + slot * it.from + head + mine;
#pragma unroll
                for (int k = 0; k < HK; k += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (has)
                        x = *reinterpret_cast<const float4 *>(from + k);
                    s[k] = x.x, s[k + 1] = x.y, s[k + 2] = x.z, s[k + 3] = x.w;
                }
            }
            write_state();
            for (int t = 0; t < it.n && alive; t += kC, ++ch, turn()) {
                const uint32_t par = ch & 1;
                const int n = min(kC, it.n - t), buf = ch % 3;
                const Decays &tab = ctl.tab[ch & 1];
                if (!wait(ctl.b.gfull[ch & 1], (ch >> 1) & 1) || !wait_tile(tv))
                    break;
                // (the phase of K's barrier is followed, and waited for where its rows past the end are cleared)
                const uint32_t kpar = (phase >> tk) & 1;
                phase ^= 1u << tk;
                phase ^= 1u << tq;
                if (n < kC && !wait(ctl.b.full[tk], kpar))
                    break;
                // V times its weights, cut in three.  Rows past the end become zeros, in K and V too, and so do the elements of
                // V that are not finite, which the weights of zero of earlier tokens would not hide: the outputs from such an
                // element on are set at the end, and the sum takes it as it is.
                auto weights = [&](int half) {
#pragma unroll
                    for (int i = 0; i < DV / 32; ++i) {
                        const int x = i * 256 + ct, r = x / (DV / 8), c = x % (DV / 8), tok = half * 64 + r;
                        const uint32_t swz = ((c & 7) ^ (r & 7)) << 4;
                        uint4 *const at = reinterpret_cast<uint4 *>(smem + tv * G::TILE + (c >> 3) * G::BLOCK + tok * 128 + swz);
                        uint4 z = *at;
                        if (tok >= n) {
                            z = make_uint4(0, 0, 0, 0);
                            *at = z;
                        } else if (odd8(z)) {
                            uint4 y = z;
                            y.x = drop2(z.x), y.y = drop2(z.y), y.z = drop2(z.z), y.w = drop2(z.w);
                            *at = y;
                            const uint32_t in[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if ((in[e >> 1] >> (16 * (e & 1)) & 0x7f80u) == 0x7f80u)
                                    atomicMin(&ctl.badfrom[buf][8 * c + e], tok);
                            *reinterpret_cast<volatile int *>(&ctl.dirty[buf]) = 1;
                        }
                        weigh(z, tab.w[tok], smem + WAT + (c >> 3) * 64 * 128 + r * 128 + swz, G::TERM);
                    }
                    if (n < half * 64 + 64)
                        for (int x = ct; x < 64 * (DK / 8); x += 256) {
                            const int tok = half * 64 + x / (DK / 8), c = x % (DK / 8);
                            if (tok >= n)
                                *reinterpret_cast<uint4 *>(smem + tk * G::TILE + (c >> 3) * G::BLOCK + tok * 128 + ((c & 7) << 4)) =
                                    make_uint4(0, 0, 0, 0);
                        }
                    smem_to_async();
                    arrive(ctl.b.wready[half]);
                };
                weights(0);
                // the weights of the chunk's tokens
                if (!wait(ctl.qk, par))
                    break;
                after_sync();
                const float gh = tab.hi[row], gl = tab.lo[row];
                {
                    uint32_t w[32];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int jb = 2 * hb + y; // a block of 32 tokens
                        if (jb > w4) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[16 * y + e] = 0;
                            continue;
                        }
                        uint32_t r[32];
                        tld(tmem + lanes + CS + 32 * jb, r);
                        if (jb < w4) { // e^{G_i - G_j} = e^{G_i - R} e^{R - G_j}, neither above one
                            const float f = ex2((gh - tab.rhi[jb]) + (gl - tab.rlo[jb]));
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                const float4 c = *reinterpret_cast<const float4 *>(&tab.c[32 * jb + e]);
                                const float2 f2 = make_float2(f, f);
                                const float2 x = mul2(mul2(make_float2(c.x, c.y), f2), make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
                                const float2 z = mul2(mul2(make_float2(c.z, c.w), f2), make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])));
                                const __nv_bfloat162 a2 = __floats2bfloat162_rn(x.x, x.y), b2 = __floats2bfloat162_rn(z.x, z.y);
                                w[16 * y + e / 2] = *reinterpret_cast<const uint32_t *>(&a2);
                                w[16 * y + e / 2 + 1] = *reinterpret_cast<const uint32_t *>(&b2);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 2) {
                                const int j = 32 * jb + e;
                                const float2 h2 = *reinterpret_cast<const float2 *>(&tab.hi[j]), l2 = *reinterpret_cast<const float2 *>(&tab.lo[j]);
                                const float x = e <= lane ? __uint_as_float(r[e]) * ex2((gh - h2.x) + (gl - l2.x)) : 0.f;
                                const float z = e + 1 <= lane ? __uint_as_float(r[e + 1]) * ex2((gh - h2.y) + (gl - l2.y)) : 0.f;
                                const __nv_bfloat162 a2 = __floats2bfloat162_rn(x, z);
                                w[16 * y + e / 2] = *reinterpret_cast<const uint32_t *>(&a2);
                            }
                        }
                    }
                    tst(tmem + lanes + CS + 64 * hb, w);
                    tst_wait();
                    before_sync();
                    arrive(ctl.pready);
                }
                if (!wait(ctl.b.wdone[0], par))
                    break;
                weights(1);
                // every warp has been over V: what was found of it is there for all, and nobody looks at the chunk's before
                if (!wait(ctl.b.wready[1], par))
                    break;
                if (ct < kC) {
                    const int old = (ch + 2) % 3;
                    ctl.badfrom[old][ct] = kC;
                    if (ct == 0)
                        ctl.dirty[old] = 0;
                }
                // ---- outputs
                if (!wait(ctl.odone, par))
                    break;
                after_sync();
                const bool dirty = *reinterpret_cast<volatile int *>(&ctl.dirty[buf]) != 0;
                {
                    const float f = ex2(gh + gl) * a.scale;
                    bf16 *const out = static_cast<bf16 *>(a.out) + ((size_t)(it.tok + t + row) * a.hv + it.head) * DV + hb * HV;
#pragma unroll
                    for (int k = 0; k < HV; k += 32) {
                        uint32_t x[32], y[32];
                        tld(tmem + lanes + CO1 + hb * HV + k, x);
                        tld(tmem + lanes + CO2 + hb * HV + k, y);
                        if (dirty) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (ctl.badfrom[buf][hb * HV + k + e] <= row)
                                    x[e] = 0x7fffffffu;
                        }
                        if (row < n) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint32_t w[4];
#pragma unroll
                                for (int z = 0; z < 4; ++z) {
                                    const float o0 = fmaf(__uint_as_float(y[e + 2 * z]), f, __uint_as_float(x[e + 2 * z]) * a.scale);
                                    const float o1 = fmaf(__uint_as_float(y[e + 2 * z + 1]), f, __uint_as_float(x[e + 2 * z + 1]) * a.scale);
                                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(o0, o1);
                                    w[z] = *reinterpret_cast<const uint32_t *>(&h2);
                                }
                                *reinterpret_cast<uint4 *>(out + k + e) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        }
                        __syncwarp();
                    }
                }
                // ---- the state
                const float all = tab.all;
                if (!wait(ctl.dsdone, par))
                    break;
                after_sync();
#pragma unroll
                for (int k = 0; k < HK; k += 32) {
                    uint32_t r[32];
                    tld(tmem + lanes + CD + hb * HK + k, r);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        s[k + e] = fmaf(s[k + e], all, __uint_as_float(r[e]));
                }
                arrive(ctl.b.gempty[ch & 1]);
                if (t + kC < it.n) {
                    write_state();
                } else if (it.last && has) {
                    float *const to = a.pool + slot * it.ws + head + mine;
#pragma unroll
                    for (int k = 0; k < HK; k += 4)
                        *reinterpret_cast<float4 *>(to + k) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
                }
                before_sync();
            }
            if (!alive)
                break;
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// ---- the segments' own sums ----
// As above without Q: two tiles of V and two of K in turn, the halves of the
// weighted V each in a place of its own, two chunks' sums in tensor memory, so
// that a chunk's products run beside the next one's weights.
template <int DK, int DV> struct SumCtrl {
    Bars b;
    LItem item[kQueue];
    struct {
        float w[kC];
        float all;
    } tab[2];
    uint32_t tmem;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_sum_kernel(const ChunkArgs p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    typedef CGeo<DK, DV> G;
    typedef SumCtrl<DK, DV> Ctrl;
    constexpr int WAT = 4 * G::TILE, CAT = WAT + 2 * G::WBYTES;
    static_assert(CAT % 1024 == 0 && CAT + sizeof(Ctrl) <= 232448, "shared memory");
    constexpr int HK = DK / 2;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctrl &ctl = *reinterpret_cast<Ctrl *>(smem + CAT);
    const uint32_t sbase = sm_addr(smem);
    const LinearArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto bar = [&](unsigned long long &b) { return sm_addr(&b); };
    if (sbase & 1023) { // the swizzled tiles need it; the whole CTA leaves
        if (tid == 0)
            report(a.err, GDN_DEVERR_TIMEOUT);
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&ctl.tmem)), "r"(256) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < kQueue; ++i)
            mbar_init(bar(ctl.b.ifull[i]), 1), mbar_init(bar(ctl.b.iempty[i]), kReaders);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctl.b.gfull[i]), 1), mbar_init(bar(ctl.b.gempty[i]), 8);
            mbar_init(bar(ctl.b.wready[i]), 8), mbar_init(bar(ctl.b.wdone[i]), 1);
        }
        for (int i = 0; i < 4; ++i) // V's tiles are read by the computing warps, K's by the products
            mbar_init(bar(ctl.b.full[i]), 1), mbar_init(bar(ctl.b.empty[i]), i < 2 ? 8 : 1);
        mbar_init(bar(ctl.b.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = ctl.tmem;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true; // false once a bounded wait ran out
    auto wait = [&](unsigned long long &b, uint32_t parity) { // by a whole warp, which goes on or leaves as one
        if (!__all_sync(0xffffffffu, mbar_try(bar(b), parity)) && alive && !__all_sync(0xffffffffu, mbar_wait(bar(b), parity))) {
            alive = false;
            report(a.err, GDN_DEVERR_TIMEOUT);
        }
        return alive;
    };
    auto arrive = [&](unsigned long long &b) { // a warp
        __syncwarp();
        if (lane == 0)
            mbar_arrive(bar(b));
        __syncwarp();
    };
    auto take = [&](int q, LItem &it) {
        const int slot = q % kQueue;
        if (!wait(ctl.b.ifull[slot], (q / kQueue) & 1))
            return false;
        it = ctl.item[slot];
        arrive(ctl.b.iempty[slot]);
        return it.n > 0;
    };
    auto tile = [&](int t) { return sbase + t * G::TILE; };
    unsigned ch = 0; // chunks done
    LItem it;

    if (warp == 3) {
        ItemWalk<true> walk(p);
        for (int q = 0; alive; ++q) {
            LItem x;
            const bool more = walk.next(x);
            const int slot = q % kQueue;
            if (!wait(ctl.b.iempty[slot], (q / kQueue + 1) & 1))
                break;
            if (!more)
                x.n = 0;
            if (lane == 0) {
                ctl.item[slot] = x;
                mbar_arrive(bar(ctl.b.ifull[slot]));
            }
            __syncwarp();
            if (!more)
                break;
        }
    } else if (warp == 0) {
        unsigned asked = 0; // chunks whose copies were asked for
        for (int q = 0; take(q, it); ++q) {
            const int hk = it.head / (a.hv / a.hk);
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                const uint32_t free = ((ch >> 1) & 1) ^ 1;
                if (!wait(ctl.b.empty[ch & 1], free) || !wait(ctl.b.empty[2 + (ch & 1)], free))
                    break;
                if (lane == 0) {
                    load_tile(tile(ch & 1), &vmap, DV / 64, it.head, it.tok + t, bar(ctl.b.full[ch & 1]), G::VBYTES);
                    load_tile(tile(2 + (ch & 1)), &kmap, DK / 64, hk, it.tok + t, bar(ctl.b.full[2 + (ch & 1)]), G::KBYTES);
                }
                __syncwarp();
                ++asked;
            }
            if (!alive)
                break;
        }
        // the last copies land before the CTA leaves, whoever still waits for them
        for (unsigned i = asked > 2 ? asked - 2 : 0; i < asked; ++i) {
            mbar_wait(bar(ctl.b.full[i & 1]), (i >> 1) & 1);
            mbar_wait(bar(ctl.b.full[2 + (i & 1)]), (i >> 1) & 1);
        }
    } else if (warp == 1) {
        const bool leader = elect();
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                const int kt = 2 + (ch & 1);
                if (!wait(ctl.b.full[kt], (ch >> 1) & 1))
                    break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait(ctl.b.wready[half], ch & 1))
                        break;
                    after_sync();
                    if (leader) {
                        const uint64_t kd = desc_mn(tile(kt) + half * 64 * 128, G::BLOCK);
                        const uint64_t wd = desc_mn(sbase + WAT + half * G::WBYTES, 64 * 128);
#pragma unroll
                        for (int x = 2; x >= 0; --x) // the small terms first
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ss(tmem + 128 * (ch & 1), wd + ((x * G::TERM + k * 2048) >> 4), kd + (k * 2048 >> 4),
                                       idesc(DK, true, true), half > 0 || x < 2 || k > 0);
                        commit(bar(ctl.b.wdone[half]));
                        if (half)
                            commit(bar(ctl.b.empty[kt]));
                    }
                }
            }
            if (!alive)
                break;
        }
        // everything issued is done before tensor memory and the barriers go
        __syncwarp();
        if (leader)
            commit(bar(ctl.b.drain));
        __syncwarp();
        mbar_wait(bar(ctl.b.drain), 0);
    } else if (warp == 2) {
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                if (!wait(ctl.b.gempty[ch & 1], ((ch >> 1) & 1) ^ 1))
                    break;
                form_decays<false>(a, it.tok + t, min(kC, it.n - t), it.head, ctl.tab[ch & 1]);
                arrive(ctl.b.gfull[ch & 1]);
            }
            if (!alive)
                break;
        }
    } else {
        const int w4 = warp & 3, hb = (warp - 4) >> 2, row = 32 * w4 + lane, ct = tid - 128; // 0 .. 255
        const uint32_t lanes = (uint32_t)w4 << 21;
        float s[HK];
        auto add = [&](unsigned c, float all) { // the sum of chunk c, which is done
            after_sync();
#pragma unroll
            for (int k = 0; k < HK; k += 32) {
                uint32_t r[32];
                tld(tmem + lanes + 128 * (c & 1) + hb * HK + k, r);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    s[k + e] = fmaf(s[k + e], all, __uint_as_float(r[e]));
            }
            before_sync();
        };
        for (int q = 0; take(q, it); ++q) {
            float total = 1.f, last = 0.f;
#pragma unroll
            for (int k = 0; k < HK; ++k)
                s[k] = 0.f;
            for (int t = 0; t < it.n && alive; t += kC, ++ch) { // (whole chunks: a segment with another behind it)
                if (!wait(ctl.b.gfull[ch & 1], (ch >> 1) & 1) || !wait(ctl.b.full[ch & 1], (ch >> 1) & 1))
                    break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!wait(ctl.b.wdone[half], (ch & 1) ^ 1)) // the chunk before is done with the place
                        break;
#pragma unroll
                    for (int i = 0; i < DV / 32; ++i) {
                        const int x = i * 256 + ct, r = x / (DV / 8), c = x % (DV / 8), tok = half * 64 + r;
                        const uint32_t swz = ((c & 7) ^ (r & 7)) << 4;
                        const uint4 z = *reinterpret_cast<const uint4 *>(smem + (ch & 1) * G::TILE + (c >> 3) * G::BLOCK + tok * 128 + swz);
                        weigh(z, ctl.tab[ch & 1].w[tok], smem + WAT + half * G::WBYTES + (c >> 3) * 64 * 128 + r * 128 + swz, G::TERM);
                    }
                    smem_to_async();
                    arrive(ctl.b.wready[half]);
                }
                if (!alive)
                    break;
                const float all = ctl.tab[ch & 1].all;
                arrive(ctl.b.empty[ch & 1]);
                arrive(ctl.b.gempty[ch & 1]);
                if (t > 0)
                    add(ch - 1, last);
                last = all;
                total *= all;
            }
            if (!alive || !wait(ctl.b.wdone[1], (ch - 1) & 1))
                break;
            add(ch - 1, last);
            if (row < DV) {
                float *const to = p.state + ((size_t)it.at * a.hv + it.head) * DV * DK + (size_t)row * DK + hb * HK;
#pragma unroll
                for (int k = 0; k < HK; k += 4)
                    *reinterpret_cast<float4 *>(to + k) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
            }
            if (ct == 0)
                p.decay[(size_t)it.at * a.hv + it.head] = total;
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(256) : "memory");
}

// The state after each segment but a sequence's last, from the segments' sums,
// in their places: a thread four floats of a (sequence, head).
__global__ void __launch_bounds__(256) linear_scan_kernel(const ChunkArgs p)
{
    wait_prior_grid();
    const int floats = p.a.dv * p.a.dk, parts = floats / 1024;
    const int part = blockIdx.x % parts, x = blockIdx.x / parts, h = x % p.a.hv, r = x / p.a.hv;
    int b, n, rs, ws;
    const int segs = segments(p, r, b, n, rs, ws);
    if (segs < 2)
        return;
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

// ---- host ----
// Chunks a segment, from what the host knows (the lengths are on the device; sequences are taken as equal): the fewest
// rounds of CTAs, in chunks, where a segment costs one more to begin, and forming the sums half a chunk's time.
int segment_chunks(int nseq, int tokens, int hv)
{
    const int m = (int)(((long long)tokens + (long long)nseq * kC - 1) / ((long long)nseq * kC)); // chunks a sequence
    int best = m;
    double least = 1e30;
    for (int cuts = 1; cuts <= m && cuts <= kSms; ++cuts) {
        const int len = (m + cuts - 1) / cuts, segs = (m + len - 1) / len;
        auto rounds = [&](long long n) { return (double)((n * nseq * hv + kSms - 1) / kSms); };
        const double cost = rounds(segs) * (len + 1) + (segs > 1 ? rounds(segs - 1) * (0.5 * len + 1) + 3 : 0);
        if (cost < least)
            least = cost, best = len;
    }
    return best;
}
// Whether a sequence can have several segments
bool divided(int tokens, int seg) { return tokens > (long long)seg * kC; }

// [tokens][heads][d] bf16, boxes of 64 d of one head x kC tokens
bool encode_tokens(CUtensorMap *m, const void *base, int d, int heads, int tokens, long long stride)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kC}, step[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV> cudaError_t go(const LinearArgs &a, cudaStream_t s)
{
    typedef CGeo<DK, DV> G;
    constexpr int CHUNK = 4 * G::TILE + G::SBYTES + G::WBYTES + (int)sizeof(ChunkCtrl<DK, DV>);
    constexpr int SUM = 4 * G::TILE + 2 * G::WBYTES + (int)sizeof(SumCtrl<DK, DV>);
    static std::atomic<unsigned long long> configured{0}; // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(linear_chunk_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, CHUNK);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(linear_sum_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, SUM);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    CUtensorMap qmap, kmap, vmap;
    if (!encode_tokens(&qmap, a.q, DK, a.hk, a.total_tokens, a.q_stride) || !encode_tokens(&kmap, a.k, DK, a.hk, a.total_tokens, a.k_stride) ||
        !encode_tokens(&vmap, a.v, DV, a.hv, a.total_tokens, a.v_stride))
        return cudaErrorInvalidValue;
    ChunkArgs p;
    p.a = a;
    p.seg = segment_chunks(a.rows, a.total_tokens, a.hv);
    const long long most = places(a.rows, a.total_tokens, p.seg) * a.hv; // items
    p.state = static_cast<float *>(a.work);
    p.decay = p.state + (size_t)most * DV * DK;
    const dim3 grid((unsigned)(most < kSms ? most : kSms));
    if (divided(a.total_tokens, p.seg)) {
        e = launch_pdl(linear_sum_kernel<DK, DV>, grid, dim3(kThreads), (size_t)SUM, s, p, kmap, vmap);
        if (e != cudaSuccess)
            return e;
        e = launch_pdl(linear_scan_kernel, dim3((unsigned)a.rows * a.hv * (DV * DK / 1024)), dim3(256), 0, s, p);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(linear_chunk_kernel<DK, DV>, grid, dim3(kThreads), (size_t)CHUNK, s, p, qmap, kmap, vmap);
}

} // namespace

bool linear_chunked_supported(int dk, int dv, int dtype)
{
    return dtype == GDN_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}

size_t linear_chunked_workspace_bytes(int nseq, int tokens, int hv, int dk, int dv)
{
    const int seg = segment_chunks(nseq, tokens, hv);
    return divided(tokens, seg) ? sizeof(float) * (size_t)places(nseq, tokens, seg) * hv * ((size_t)dv * dk + 1) : 0;
}

cudaError_t launch_linear_chunked(LinearArgs a, cudaStream_t s)
{
    // the short sequences, the padding and the bad ones
    a.most = kSerial;
    const cudaError_t e = launch_linear_serial(a, GDN_BF16, s);
    if (e != cudaSuccess || a.total_tokens <= kSerial)
        return e;
    if (a.dk == 128)
        return a.dv == 128 ? go<128, 128>(a, s) : go<128, 64>(a, s);
    return a.dv == 128 ? go<64, 128>(a, s) : go<64, 64>(a, s);
}

} // namespace gdn
