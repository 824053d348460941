// Linear attention with a decay for each head over packed sequences in chunks
// of C = 128 tokens on the tensor cores (sm_103a), bf16 activations, dk and dv
// 64 or 128.  With G_i the sum of the log decays up to token i of a chunk and S
// the state before it,
//   o_i = scale (e^{G_i} S q_i + sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j)
//   S'  = e^{G_C} S + sum_j e^{G_C - G_j} v_j k_j^T,
// which regroups the recurrence token after token (linear_attn.cu); as a decay
// is a number, the sums over j of different chunks do not depend on each other.
//
// Work: as linear_plan.cuh divides it, by linear_sum_kernel, linear_scan_kernel
// and linear_chunk_kernel.
//
// linear_chunk_kernel: persistent, one CTA an SM.  Warp 0 brings Q, K and V by
// tensor copies (two tiles of K and of V, one of Q, which is done with early),
// warp 1 issues the products, warp 2 forms the decays and sends the outputs
// off, warp 3 walks the items.  Of sixteen computing warps eight weigh V, 32
// tokens at a time into two places in turn, and eight turn Q K^T into weights
// (bf16, in the scores' place in tensor memory) and write the outputs, through
// V's tile; the state is in the registers of all, a thread a row and a quarter
// of its columns.
//
// Shared memory's 128 bytes a clock bound the chunk kernel's first forms: a 128 x
// 128 x 16 product with both operands there takes all of them.  So weighted V
// goes to tensor memory, transposed as it is read (a thread a column of V), and
// only K comes from shared memory; the outputs' two parts are summed in one
// place, the state's part being multiplied by its tokens' decays there.
//
// Precision.  The state is to be right to fp32, and its products' operands are
// bf16: e^{G_C - G_j} v_j is cut into three bf16 values that make it up exactly
// (8 bits each of 24), so a chunk's sum takes three products; K is bf16 as it
// comes.  A chunk's sum is added to the state in fp32 outside the tensor cores,
// whose own additions cut results short.  The weights and the state, as
// operands of the outputs alone, are rounded to bf16 once: outputs are off by
// 0.0023 of their norm instead of the 0.0017 of their own rounding, and three
// products of each would take as long again as all of them.
//
// Measured (16 heads of 128 x 128, in a graph): 8 sequences of 1,500 to 2,600 tokens 92.6 us,
// half of the rate of their bytes; 128 chains of up to 21 chunks on 152 SMs, a
// chunk 6,700 clocks.  One of 16,000 tokens 95 us: sums 34, scan 5, the segments
// 62, less what lies beside each other.  Bound: the chain of a chunk, scores,
// weights, outputs and state, each waiting for products or for the other warps;
// the tensor pipe is busy 37 %, issue slots 47 %, and instructions come late
// where loops are unrolled or inlined further (102 to 113 us then).
#include <atomic>
#include <cstring>

#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "linear_plan.cuh"
#include "tc_ops.cuh"

namespace gdn {
namespace {

constexpr int kC = 128;        // tokens a chunk
constexpr int kComp = 16;      // warps that compute: a thread a row and a quarter of its columns
constexpr int kThreads = 32 * (4 + kComp);
constexpr int kRun = 32;       // tokens whose weighted V is written and taken at a time
constexpr int kQueue = 4;      // items in flight between the walking warp and the others
constexpr int kReaders = 3 + kComp; // warps 0, 1, 2 and the computing ones

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
// Four tokens' log decays a lane, zero past the end
__device__ __forceinline__ void load_decays(const LinearArgs &a, int tok, int n, int head, float (&x)[4])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = 4 * (threadIdx.x & 31) + e;
        x[e] = j < n ? a.log_decay[(long long)(tok + j) * a.decay_stride + head] : 0.f;
    }
}
// FULL: all of it, else w and `all`
template <bool FULL, typename Tab> __device__ __forceinline__ void form_decays(const float (&in)[4], Tab &t)
{
    const int lane = threadIdx.x & 31;
    Two g[4], upto = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float x = in[e] > 0.f ? 0.f : in[e] < -110.f ? -110.f : in[e]; // (a NaN stays)
        upto = upto + log2_units(x);
        g[e] = upto;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two x = shuffle(upto, lane < o ? lane : lane - o);
        if (lane >= o)
            upto = upto + x;
    }
    const Two all = shuffle(upto, 31), block = shuffle(upto, lane | 7);
    Two before = shuffle(upto, lane == 0 ? 0 : lane - 1);
    if (lane == 0)
        before = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int j = 4 * lane + e;
        const Two G = before + g[e];
        t.w[j] = exp2f(minus(all, G));
        if constexpr (FULL) {
            t.hi[j] = G.h;
            t.lo[j] = G.l;
            t.c[j] = exp2f(minus(block, G));
        }
    }
    if constexpr (FULL)
        if ((lane & 7) == 7) {
            t.rhi[lane >> 3] = block.h;
            t.rlo[lane >> 3] = block.l;
        }
    if (lane == 0)
        t.all = exp2f(all.h + all.l);
}

__device__ __forceinline__ uint32_t bf16_pair(float x, float y)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two floats, each cut into three bf16 values that make it up: heads, middles, tails as pairs.
__device__ __forceinline__ void cut3(float2 x, uint32_t &h, uint32_t &m, uint32_t &l)
{
    auto rest = [](float2 v, uint32_t &pair) { // takes off the upper halves
        const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
        pair = __byte_perm(a, b, 0x7632);
        return fma2(make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)), make_float2(-1.f, -1.f), v);
    };
    const float2 y = rest(x, h), z = rest(y, m);
    l = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
}
// Sixteen tokens of a column of V (a tile's byte `at`: its column, its first token) times their weights, cut in three, to
// tensor memory, eight columns at `to` and every `term` on; a token's weight in `w`.  x gets V's values, for a look at them.
__device__ __forceinline__ void read_column(const unsigned char *smem, uint32_t at, float (&x)[16])
{
#pragma unroll
    for (int e = 0; e < 16; ++e) // (16-byte pieces of a row lie at their number ^ the row's)
        x[e] = __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short *>(smem + (at ^ ((e & 7) << 4)) + e * 128) << 16);
}
__device__ __forceinline__ void weigh_column(const float (&x)[16], const float *w, uint32_t to, int term)
{
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(w + e);
        cut3(mul2(make_float2(x[e], x[e + 1]), make_float2(f.x, f.y)), h[e / 2], m[e / 2], l[e / 2]);
        cut3(mul2(make_float2(x[e + 2], x[e + 3]), make_float2(f.z, f.w)), h[e / 2 + 1], m[e / 2 + 1], l[e / 2 + 1]);
    }
    tst(to, h);
    tst(to + term, m);
    tst(to + 2 * term, l);
}
// What of a column is not finite becomes zero in V's tile (and the values stay as they are); the first such token.
__device__ __noinline__ int clear_column(unsigned char *smem, uint32_t at, int tok)
{
    int first = kC;
    for (int e = 15; e >= 0; --e) {
        unsigned short *const v = reinterpret_cast<unsigned short *>(smem + (at ^ ((e & 7) << 4)) + e * 128);
        if ((*v & 0x7f80) == 0x7f80)
            *v = 0, first = tok + e;
    }
    return first;
}

template <int DK, int DV> struct CGeo {
    static constexpr int D = DK > DV ? DK : DV;
    static constexpr int TILE = kC * D * 2;           // a Q, K or V tile, as 64-column blocks of kC rows
    static constexpr int BLOCK = kC * 128;            // one such block
    static constexpr int KBYTES = kC * DK * 2, VBYTES = kC * DV * 2;
    static constexpr int SBYTES = DV * DK * 2;        // the state in bf16
    static constexpr int WK = DK / 4;                 // a thread's columns of the state
};

// The waits go on in one place: where they did in line, the computing warps' loops left the instruction cache.
__device__ __noinline__ bool wait_on(uint32_t b, uint32_t parity) { return mbar_wait(b, parity); }

// What both kernels wait for each other with.
struct Bars {
    unsigned long long ifull[kQueue], iempty[kQueue];
    unsigned long long gfull[2], gempty[2]; // decays
    unsigned long long full[6], empty[6];   // tiles
    unsigned long long wready[2], wdone[2]; // places of weighted V: written; read by their products
    unsigned long long drain;
};

__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int blocks, int head, int tok, uint32_t bar, int bytes)
{
    mbar_arrive_tx(bar, bytes);
    for (int c = 0; c < blocks; ++c)
        tma3(dst + c * kC * 128, map, 64 * c, head, tok, bar);
}

// What both kernels do with a wait of theirs, `wait(barrier, parity)`, by a whole warp that goes on or leaves as one.
__device__ __forceinline__ void arrive_warp(unsigned long long &b)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(sm_addr(&b));
    __syncwarp();
}
// The queue's items: one warp walks them, and the readers take turn q's.
template <bool SUM, typename Ctrl, typename Wait> __device__ __forceinline__ void walk_items(const ChunkArgs &p, Ctrl &ctl, const Wait &wait)
{
    ItemWalk<SUM> walk(p);
    bool more = true;
    for (int q = 0; more; ++q) {
        LItem x;
        more = walk.next(x);
        const int slot = q % kQueue;
        if (!wait(ctl.b.iempty[slot], (q / kQueue + 1) & 1))
            break;
        if (!more)
            x.n = 0;
        if (walk.lane == 0) {
            ctl.item[slot] = x;
            mbar_arrive(sm_addr(&ctl.b.ifull[slot]));
        }
        __syncwarp();
    }
}
template <typename Ctrl, typename Wait> __device__ __forceinline__ bool take_item(Ctrl &ctl, const Wait &wait, int q, LItem &it) // false: no more
{
    const int slot = q % kQueue;
    if (!wait(ctl.b.ifull[slot], (q / kQueue) & 1))
        return false;
    it = ctl.item[slot];
    arrive_warp(ctl.b.iempty[slot]);
    return it.n > 0;
}
// Tensor memory, all of it, by one warp.
__device__ __forceinline__ void take_tmem(uint32_t &at)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&at)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

// ---- the outputs, and the states at the sequences' ends ----
template <int DK, int DV> struct ChunkCtrl {
    Bars b;
    unsigned long long qk, qs, pready, odone, ofree, dsdone, sready, vseen;
    LItem item[kQueue];
    Decays tab[2];
    int badfrom[4][kC]; // by chunk: first token with a value that is not finite, by column
    int dirty[4];       // whether there is one
    uint32_t tmem;
};

template <int DK, int DV>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const ChunkArgs p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap)
{
    typedef CGeo<DK, DV> G;
    typedef ChunkCtrl<DK, DV> Ctrl;
    constexpr int SAT = 5 * G::TILE, CAT = SAT + G::SBYTES;
    static_assert(CAT % 1024 == 0 && CAT + sizeof(Ctrl) <= 232448, "shared memory");
    // tensor memory: scores and weights, outputs, the chunk's sum, two places of weighted V (three terms of 16 columns)
    constexpr uint32_t CS = 0, CO = 128, CD = 256, CW = 384, PLACE = 48;
    constexpr int WK = G::WK, HV = DV / 2;
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
    begin_chunks();
    if (p.none && !any_with(p, 1)) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        wait_prior_grid();
        return;
    }
    if (warp == 0)
        take_tmem(ctl.tmem);
    if (tid == 64) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&qmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&omap) : "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < kQueue; ++i)
            mbar_init(bar(ctl.b.ifull[i]), 1), mbar_init(bar(ctl.b.iempty[i]), kReaders);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctl.b.gfull[i]), 1), mbar_init(bar(ctl.b.gempty[i]), kComp);
            mbar_init(bar(ctl.b.wready[i]), kComp / 2), mbar_init(bar(ctl.b.wdone[i]), 1);
        }
        for (int i = 0; i < 5; ++i)
            mbar_init(bar(ctl.b.full[i]), 1), mbar_init(bar(ctl.b.empty[i]), 1);
        mbar_init(bar(ctl.qk), 1), mbar_init(bar(ctl.qs), 1), mbar_init(bar(ctl.pready), kComp / 2);
        mbar_init(bar(ctl.odone), 1), mbar_init(bar(ctl.ofree), kComp / 2), mbar_init(bar(ctl.vseen), kComp / 2);
        mbar_init(bar(ctl.dsdone), 1), mbar_init(bar(ctl.sready), kComp), mbar_init(bar(ctl.b.drain), 1);
        ctl.dirty[0] = ctl.dirty[1] = ctl.dirty[2] = ctl.dirty[3] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < 4 * kC; i += kThreads)
        (&ctl.badfrom[0][0])[i] = kC;
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = ctl.tmem;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true; // false once a bounded wait ran out
    auto wait_at = [&](uint32_t b, uint32_t parity) { // by a whole warp, which goes on or leaves as one
        if (!__all_sync(0xffffffffu, mbar_try(b, parity)) && alive && !__all_sync(0xffffffffu, wait_on(b, parity))) {
            alive = false;
            report(a.err, GDN_DEVERR_TIMEOUT);
        }
        return alive;
    };
    auto wait = [&](unsigned long long &b, uint32_t parity) { return wait_at(bar(b), parity); };
    auto arrive = [](unsigned long long &b) { arrive_warp(b); };
    auto take = [&](int q, LItem &it) { return take_item(ctl, wait, q, it); };
    // tiles: V of even and odd chunks, K of even and odd chunks, Q
    constexpr int TQ = 4;
    auto tile = [&](int t) { return sbase + t * G::TILE; };
    unsigned ch = 0; // chunks done
    LItem it;

    if (warp == 3) {
        walk_items<false>(p, ctl, wait);
    } else if (warp == 0) {
        // ---- Q, K and V
        auto load = [&](int t, uint32_t use, const CUtensorMap *map, int blocks, int head, int tok, int bytes) {
            if (!wait(ctl.b.empty[t], (use & 1) ^ 1))
                return false;
            if (lane == 0)
                load_tile(tile(t), map, blocks, head, tok, bar(ctl.b.full[t]), bytes);
            __syncwarp();
            return true;
        };
        unsigned asked[3] = {0, 0, 0}; // copies of V, K and Q
        for (int q = 0; take(q, it); ++q) {
            const int hk = it.head / (a.hv / a.hk);
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                if (!load(2 + (ch & 1), ch >> 1, &kmap, DK / 64, hk, it.tok + t, G::KBYTES))
                    break;
                ++asked[1];
                if (!load(ch & 1, ch >> 1, &vmap, DV / 64, it.head, it.tok + t, G::VBYTES))
                    break;
                ++asked[0];
                if (!load(TQ, ch, &qmap, DK / 64, hk, it.tok + t, G::KBYTES))
                    break;
                ++asked[2];
            }
            if (!alive)
                break;
        }
        // the last copies land before the CTA leaves, whoever still waits for them
        for (int x = 0; x < 2; ++x)
            for (unsigned c = asked[x] > 2 ? asked[x] - 2 : 0; c < asked[x]; ++c)
                mbar_wait(bar(ctl.b.full[2 * x + (c & 1)]), (c >> 1) & 1);
        if (asked[2])
            mbar_wait(bar(ctl.b.full[TQ]), (asked[2] - 1) & 1);
    } else if (warp == 1) {
        // ---- the products, issued by one elected lane of the whole warp's walk
        const bool leader = elect();
        auto sum = [&](int run) { // of a run's weighted V and K
            if (!wait(ctl.b.wready[run & 1], run >> 1))
                return false;
            after_sync();
            if (leader) {
                const uint64_t kd = desc_mn(tile(2 + (ch & 1)) + run * kRun * 128, G::BLOCK);
#pragma unroll
                for (int x = 2; x >= 0; --x) // the small terms first
#pragma unroll
                    for (int k = 0; k < kRun / 16; ++k)
                        mma_ts(tmem + CD, tmem + CW + PLACE * (run & 1) + 16 * x + 8 * k, kd + (k * 2048 >> 4), idesc(DK, true),
                               run > 0 || x < 2 || k > 0);
                commit(bar(ctl.b.wdone[run & 1]));
            }
            return true;
        };
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                const uint32_t par = ch & 1, par2 = (ch >> 1) & 1;
                const int tv = ch & 1, tk = 2 + (ch & 1);
                const uint64_t qd = desc_k(tile(TQ));
                if (!wait(ctl.b.full[TQ], par) || !wait(ctl.b.full[tk], par2))
                    break;
                after_sync();
                if (leader) { // Q K^T
                    const uint64_t kd = desc_k(tile(tk));
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k) {
                        const uint64_t at = ((k >> 2) * G::BLOCK + (k & 3) * 32) >> 4;
                        mma_ss(tmem + CS, qd + at, kd + at, idesc(kC, false), k > 0);
                    }
                    commit(bar(ctl.qk));
                }
                if (!wait(ctl.sready, par)) // the state is written, the sum before is read
                    break;
                if (!sum(0) || !sum(1) || !wait(ctl.ofree, par ^ 1)) // the outputs before are read
                    break;
                after_sync();
                if (leader) { // the state times q
                    const uint64_t sd = desc_k(sbase + SAT);
#pragma unroll
                    for (int k = 0; k < DK / 16; ++k)
                        mma_ss(tmem + CO, qd + (((k >> 2) * G::BLOCK + (k & 3) * 32) >> 4),
                               sd + (((k >> 2) * DV * 128 + (k & 3) * 32) >> 4), idesc(DV, false), k > 0);
                    commit(bar(ctl.qs));
                    commit(bar(ctl.b.empty[TQ]));
                }
                if (!sum(2) || !sum(3))
                    break;
                if (leader) {
                    commit(bar(ctl.dsdone));
                    commit(bar(ctl.b.empty[tk]));
                }
                if (!wait(ctl.pready, par) || !wait(ctl.b.full[tv], par2))
                    break;
                after_sync();
                if (leader) { // and the weights times V
                    const uint64_t vd = desc_mn(tile(tv), G::BLOCK);
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_ts(tmem + CO, tmem + CS + 64 * (k >> 2) + 8 * (k & 3), vd + (k * 2048 >> 4), idesc(DV, true), true);
                    commit(bar(ctl.odone));
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
        // ---- the decays, and whole chunks of outputs from V's tile; the tile is then free
        int to[2] = {0, 0}, head[2] = {0, 0}; // of the last two chunks: first token (-1: no store), head
        auto send = [&](unsigned c) {
            const int t = c & 1, tok = t ? to[1] : to[0], h = t ? head[1] : head[0];
            if (lane == 0) {
                if (tok >= 0) {
                    for (int x = 0; x < DV / 64; ++x)
                        tma3_store(&omap, tile(t) + x * G::BLOCK, 64 * x, h, tok);
                    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
                }
                mbar_arrive(bar(ctl.b.empty[t]));
            }
            __syncwarp();
        };
        for (int q = 0; take(q, it); ++q) {
            float x[4], next[4];
            load_decays(a, it.tok, it.n, it.head, next);
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = next[e];
                load_decays(a, it.tok + t + kC, it.n - t - kC, it.head, next); // the next chunk's, under way meanwhile
                if (!wait(ctl.b.gempty[ch & 1], ((ch >> 1) & 1) ^ 1))
                    break;
                if (ch >= 2)
                    send(ch);
                const int tok = it.n - t >= kC ? it.tok + t : -1;
                if (ch & 1)
                    to[1] = tok, head[1] = it.head;
                else
                    to[0] = tok, head[0] = it.head;
                form_decays<true>(x, ctl.tab[ch & 1]);
                arrive(ctl.b.gfull[ch & 1]);
            }
            if (!alive)
                break;
        }
        for (unsigned c = ch > 2 ? ch : 2; c < ch + 2 && alive; ++c) // the last two
            if (wait(ctl.b.gempty[c & 1], ((c >> 1) & 1) ^ 1))
                send(c);
        if (lane == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
        const int w4 = warp & 3, quarter = (warp - 4) >> 2, row = 32 * w4 + lane;
        const uint32_t lanes = (uint32_t)w4 << 21;
        const bool has = row < DV; // whether this thread keeps a part of the state: row `row`, columns quarter WK ..
        const bool whole = (reinterpret_cast<uintptr_t>(a.pool) & 31) == 0; // (a pool's memory is aligned to 16 bytes)
        alignas(16) float s[WK];
        auto write_state = [&] { // in bf16, for the products
            if (has) {
#pragma unroll
                for (int k = 0; k < WK; k += 8) {
                    const int col = quarter * WK + k;
                    *reinterpret_cast<uint4 *>(smem + SAT + (col >> 6) * DV * 128 + row * 128 + ((((col & 63) >> 3) ^ (row & 7)) << 4)) =
                        make_uint4(bf16_pair(s[k], s[k + 1]), bf16_pair(s[k + 2], s[k + 3]), bf16_pair(s[k + 4], s[k + 5]),
                                   bf16_pair(s[k + 6], s[k + 7]));
                }
            }
            smem_to_async();
            before_sync();
            arrive(ctl.sready);
        };
        auto begin = [&] { // an item: its state
            const size_t slot = (size_t)a.hv * DV * DK, mine = (size_t)it.head * DV * DK + (size_t)row * DK + quarter * WK;
            const float *const from = it.from < 0 ? a.pool + slot * it.rs + mine : p.state + slot * it.from + mine;
            if (it.from >= 0)
                wait_prior_grid(); // the scan
#pragma unroll
            for (int k = 0; k < WK; k += 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    s[k + e] = 0.f;
                if (has && (whole || it.from >= 0)) {
                    load8(from + k, &s[k]);
                } else if (has) {
                    *reinterpret_cast<float4 *>(&s[k]) = *reinterpret_cast<const float4 *>(from + k);
                    *reinterpret_cast<float4 *>(&s[k + 4]) = *reinterpret_cast<const float4 *>(from + k + 4);
                }
            }
            write_state();
        };
        auto update = [&](unsigned c, float all, bool more) { // the state, with the sum of chunk c, and whether the item has more
            if (!wait(ctl.dsdone, c & 1))
                return false;
            after_sync();
            {
                uint32_t r[WK];
                tld(tmem + lanes + CD + quarter * WK, r);
#pragma unroll
                for (int e = 0; e < WK; ++e)
                    s[e] = fmaf(s[e], all, __uint_as_float(r[e]));
            }
            if (more) {
                write_state();
            } else {
                if (it.last && has) {
                    float *const to = a.pool + (size_t)a.hv * DV * DK * it.ws + (size_t)it.head * DV * DK + (size_t)row * DK + quarter * WK;
#pragma unroll
                    for (int k = 0; k < WK; k += 8)
                        if (whole) {
                            store8(to + k, &s[k]);
                        } else {
                            *reinterpret_cast<float4 *>(to + k) = make_float4(s[k], s[k + 1], s[k + 2], s[k + 3]);
                            *reinterpret_cast<float4 *>(to + k + 4) = make_float4(s[k + 4], s[k + 5], s[k + 6], s[k + 7]);
                        }
                }
                before_sync();
            }
            return true;
        };
        if (warp < 4 + kComp / 2) {
            // ---- V times its weights, a thread a column of V and half of a run's tokens.  What lies past the end becomes zero,
            // in K and V too, and so do the elements of V that are not finite, which the weights of zero of earlier tokens
            // would not hide: the outputs from such an element on are set when they are written, and the sum takes it as it is.
            const int half = (warp - 4) >> 2, ct = tid - 128;
            for (int q = 0; take(q, it); ++q) {
                begin();
                float all = 0.f;
                for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                    const int n = min(kC, it.n - t), buf = ch & 3;
                    const Decays &tab = ctl.tab[ch & 1];
                    if (!wait(ctl.b.gfull[ch & 1], (ch >> 1) & 1) || !wait(ctl.b.full[ch & 1], (ch >> 1) & 1))
                        break;
                    if (n < kC && !wait(ctl.b.full[2 + (ch & 1)], (ch >> 1) & 1))
                        break;
#pragma unroll 1
                    for (int run = 0; run < kC / kRun; ++run) {
                        const int tok = run * kRun + 16 * half;
                        const uint32_t at = (ch & 1) * G::TILE + (row >> 6) * G::BLOCK + tok * 128 + ((row & 63) >> 3 << 4) + (row & 7) * 2;
                        float x[16];
                        bool wrote = false;
                        if (has) {
                            read_column(smem, at, x);
                            if (tok + 16 > n) {
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (tok + e >= n) {
                                        x[e] = 0.f;
                                        *reinterpret_cast<unsigned short *>(smem + (at ^ ((e & 7) << 4)) + e * 128) = 0;
                                    }
                                wrote = true;
                            }
                            float z = 0.f; // stays zero unless a value is not finite
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                z = fmaf(x[e], 0.f, z);
                            if (z != 0.f) {
                                atomicMin(&ctl.badfrom[buf][row], clear_column(smem, at, tok));
                                *reinterpret_cast<volatile int *>(&ctl.dirty[buf]) = 1;
                                wrote = true;
                            }
                        }
                        if (n < run * kRun + kRun) {
                            for (int i = ct; i < kRun * (DK / 8); i += 16 * kComp) {
                                const int r = run * kRun + i / (DK / 8), c = i % (DK / 8);
                                if (r >= n)
                                    *reinterpret_cast<uint4 *>(smem + (2 + (ch & 1)) * G::TILE + (c >> 3) * G::BLOCK + r * 128 + ((c & 7) << 4)) =
                                        make_uint4(0, 0, 0, 0);
                            }
                            wrote = true;
                        }
                        if (wrote)
                            smem_to_async();
                        __syncwarp(); // what follows is for whole warps
                        if (!wait(ctl.b.wdone[run & 1], (run >> 1) ^ 1)) // the products before are done with the place
                            break;
                        after_sync();
                        if (w4 < DV / 32)
                            weigh_column(x, &tab.w[tok], tmem + lanes + CW + PLACE * (run & 1) + 8 * half, 16);
                        tst_wait();
                        before_sync();
                        arrive(ctl.b.wready[run & 1]);
                        if (run == 1 && t > 0 && !update(ch - 1, all, true)) // the chunk before's sum, when it is there
                            break;
                    }
                    arrive(ctl.vseen);
                    if (!alive)
                        break;
                    // nobody looks at the marks of two chunks before any more: the products of the last waited for its outputs
                    const int old = (ch + 2) & 3;
                    if (half == 0)
                        ctl.badfrom[old][ct] = kC;
                    if (ct == 0)
                        ctl.dirty[old] = 0;
                    all = tab.all;
                    arrive(ctl.b.gempty[ch & 1]);
                }
                if (!alive || !update(ch - 1, all, false))
                    break;
            }
        } else {
            // ---- the weights of the chunk's tokens, a thread a row and half of its columns, and the outputs
            const int hb = (warp - 4 - kComp / 2) >> 2;
            for (int q = 0; take(q, it); ++q) {
                begin();
                for (int t = 0; t < it.n && alive; t += kC, ++ch) {
                    const uint32_t par = ch & 1;
                    const int n = min(kC, it.n - t), buf = ch & 3;
                    const Decays &tab = ctl.tab[ch & 1];
                    if (!wait(ctl.b.gfull[ch & 1], (ch >> 1) & 1) || !wait(ctl.qk, par))
                        break;
                    after_sync();
                    const float gh = tab.hi[row], gl = tab.lo[row];
#pragma unroll 1
                    for (int y = 0; y < 2; ++y) { // blocks of 32 x 32, each into half of its scores' place
                        const int jb = 2 * hb + y;
                        uint32_t w[16];
                        if (jb > w4) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                w[e] = 0;
                        } else {
                            uint32_t r[32];
                            tld(tmem + lanes + CS + 32 * jb, r);
                            if (jb < w4) { // e^{G_i - G_j} = e^{G_i - R} e^{R - G_j}, neither above one
                                const float f = ex2((gh - tab.rhi[jb]) + (gl - tab.rlo[jb]));
                                const float2 f2 = make_float2(f, f);
#pragma unroll
                                for (int e = 0; e < 32; e += 4) {
                                    const float4 c = *reinterpret_cast<const float4 *>(&tab.c[32 * jb + e]);
                                    const float2 x = mul2(mul2(make_float2(c.x, c.y), f2), make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
                                    const float2 z = mul2(mul2(make_float2(c.z, c.w), f2), make_float2(__uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])));
                                    w[e / 2] = bf16_pair(x.x, x.y);
                                    w[e / 2 + 1] = bf16_pair(z.x, z.y);
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const int j = 32 * jb + e;
                                    const float2 h2 = *reinterpret_cast<const float2 *>(&tab.hi[j]), l2 = *reinterpret_cast<const float2 *>(&tab.lo[j]);
                                    const float x = e <= lane ? __uint_as_float(r[e]) * ex2((gh - h2.x) + (gl - l2.x)) : 0.f;
                                    const float z = e + 1 <= lane ? __uint_as_float(r[e + 1]) * ex2((gh - h2.y) + (gl - l2.y)) : 0.f;
                                    w[e / 2] = bf16_pair(x, z);
                                }
                            }
                        }
                        tst(tmem + lanes + CS + 64 * hb + 16 * y, w); // (columns that this warp alone reads, and has read)
                    }
                    // the state's part of the outputs times the decays, in its place
                    const float f = ex2(gh + gl);
                    if (!wait(ctl.qs, par))
                        break;
                    after_sync();
#pragma unroll 1
                    for (int k = 0; k < HV; k += 32) {
                        uint32_t x[32];
                        tld(tmem + lanes + CO + hb * HV + k, x);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
                        tst(tmem + lanes + CO + hb * HV + k, x);
                    }
                    tst_wait();
                    before_sync();
                    arrive(ctl.pready);
                    // all of V was looked at (waited for before the update, without which nobody goes on to the next chunk's)
                    if (!wait(ctl.vseen, par) || !update(ch, tab.all, t + kC < it.n) || !wait(ctl.odone, par))
                        break;
                    after_sync();
                    const bool dirty = *reinterpret_cast<volatile int *>(&ctl.dirty[buf]) != 0;
                    unsigned char *const mine = smem + (ch & 1) * G::TILE + ((hb * HV) >> 6) * G::BLOCK; // over V, laid out alike
                    auto piece = [&](int r, int i) {
                        return reinterpret_cast<uint4 *>(mine + r * 128 + (((((hb * HV) & 63) / 8 + i) ^ (r & 7)) << 4));
                    };
#pragma unroll 1
                    for (int k = 0; k < HV; k += 32) {
                        uint32_t x[32];
                        tld(tmem + lanes + CO + hb * HV + k, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t w[4];
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                w[z] = bf16_pair(__uint_as_float(x[8 * i + 2 * z]) * a.scale, __uint_as_float(x[8 * i + 2 * z + 1]) * a.scale);
                            *piece(row, k / 8 + i) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    if (dirty) {
#pragma unroll 1
                        for (int v = 0; v < HV; ++v)
                            if (ctl.badfrom[buf][hb * HV + v] <= row)
                                reinterpret_cast<unsigned short *>(piece(row, v >> 3))[v & 7] = 0x7fff;
                    }
                    before_sync();
                    arrive(ctl.ofree);
                    if (n < kC) { // the last tokens of a sequence: the rows that there are, by this warp itself
                        constexpr int P = HV / 8; // pieces of a row
                        bf16 *const out = static_cast<bf16 *>(a.out) + ((size_t)(it.tok + t) * a.hv + it.head) * DV + hb * HV;
                        for (int i = lane; i < 32 * P; i += 32) {
                            const int r = 32 * w4 + i / P;
                            if (r < n)
                                *reinterpret_cast<uint4 *>(out + (size_t)r * a.hv * DV + 8 * (i % P)) = *piece(r, i % P);
                        }
                    }
                    smem_to_async();
                    arrive(ctl.b.gempty[ch & 1]);
                }
                if (!alive)
                    break;
            }
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    wait_prior_grid();
}

// ---- the segments' own sums ----
// As above without Q, all sixteen warps weighing V: three tiles of V and three
// of K in turn, a place for each half of the weighted V, two chunks' sums in
// tensor memory, so that a chunk's products run beside the next one's weights.
template <int DK, int DV> struct SumCtrl {
    Bars b;
    unsigned long long added[2]; // a chunk's sum is done, by chunk parity
    LItem item[kQueue];
    struct alignas(16) {
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
    constexpr int STAGES = 3, CAT = 2 * STAGES * G::TILE;
    static_assert(CAT % 1024 == 0 && CAT + sizeof(Ctrl) <= 232448, "shared memory");
    constexpr uint32_t CW = 256, PLACE = 96; // tensor memory: two sums of 128 columns, two places of three terms of 32
    constexpr int WK = G::WK;
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
    begin_chunks();
    if (p.rare && !any_with(p, 2)) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        wait_prior_grid();
        return;
    }
    if (warp == 0)
        take_tmem(ctl.tmem);
    if (tid == 32) {
        for (int i = 0; i < kQueue; ++i)
            mbar_init(bar(ctl.b.ifull[i]), 1), mbar_init(bar(ctl.b.iempty[i]), kReaders);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctl.b.gfull[i]), 1), mbar_init(bar(ctl.b.gempty[i]), kComp);
            mbar_init(bar(ctl.b.wready[i]), kComp / 2), mbar_init(bar(ctl.b.wdone[i]), 1);
            mbar_init(bar(ctl.added[i]), 1);
        }
        for (int i = 0; i < 2 * STAGES; ++i) // V's tiles are read by the computing warps, K's by the products
            mbar_init(bar(ctl.b.full[i]), 1), mbar_init(bar(ctl.b.empty[i]), i < STAGES ? kComp : 1);
        mbar_init(bar(ctl.b.drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = ctl.tmem;
    // (now, with tensor memory taken: a CTA of the last kernel may hold an SM's while it waits for the scan, and so for this grid)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    bool alive = true; // false once a bounded wait ran out
    auto wait = [&](unsigned long long &b, uint32_t parity) { // by a whole warp, which goes on or leaves as one
        if (!__all_sync(0xffffffffu, mbar_try(bar(b), parity)) && alive && !__all_sync(0xffffffffu, wait_on(bar(b), parity))) {
            alive = false;
            report(a.err, GDN_DEVERR_TIMEOUT);
        }
        return alive;
    };
    auto arrive = [](unsigned long long &b) { arrive_warp(b); };
    auto take = [&](int q, LItem &it) { return take_item(ctl, wait, q, it); };
    auto tile = [&](int t) { return sbase + t * G::TILE; };
    unsigned ch = 0; // chunks done
    int st = 0;      // the chunk's tiles: V in st, K in STAGES + st, with the phase `turn` of their barriers
    uint32_t turn = 0;
    auto advance = [&] {
        ++ch;
        if (++st == STAGES)
            st = 0, turn ^= 1;
    };
    LItem it;

    if (warp == 3) {
        walk_items<true>(p, ctl, wait);
    } else if (warp == 0) {
        unsigned asked = 0; // chunks whose copies were asked for
        for (int q = 0; take(q, it); ++q) {
            const int hk = it.head / (a.hv / a.hk);
            for (int t = 0; t < it.n && alive; t += kC, advance()) {
                if (!wait(ctl.b.empty[st], turn ^ 1) || !wait(ctl.b.empty[STAGES + st], turn ^ 1))
                    break;
                if (lane == 0) {
                    load_tile(tile(st), &vmap, DV / 64, it.head, it.tok + t, bar(ctl.b.full[st]), G::VBYTES);
                    load_tile(tile(STAGES + st), &kmap, DK / 64, hk, it.tok + t, bar(ctl.b.full[STAGES + st]), G::KBYTES);
                }
                __syncwarp();
                ++asked;
            }
            if (!alive)
                break;
        }
        // the last copies land before the CTA leaves, whoever still waits for them
        for (unsigned i = asked > STAGES ? asked - STAGES : 0; i < asked; ++i) {
            mbar_wait(bar(ctl.b.full[i % STAGES]), (i / STAGES) & 1);
            mbar_wait(bar(ctl.b.full[STAGES + i % STAGES]), (i / STAGES) & 1);
        }
    } else if (warp == 1) {
        const bool leader = elect();
        for (int q = 0; take(q, it); ++q) {
            for (int t = 0; t < it.n && alive; t += kC, advance()) {
                // (both halves: every warp has then read the sum that was in this chunk's place)
                if (!wait(ctl.b.full[STAGES + st], turn) || !wait(ctl.b.wready[0], ch & 1) || !wait(ctl.b.wready[1], ch & 1))
                    break;
                after_sync();
                if (leader) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint64_t kd = desc_mn(tile(STAGES + st) + half * 64 * 128, G::BLOCK);
#pragma unroll
                        for (int x = 2; x >= 0; --x) // the small terms first
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_ts(tmem + 128 * (ch & 1), tmem + CW + PLACE * half + 32 * x + 8 * k, kd + (k * 2048 >> 4),
                                       idesc(DK, true), half > 0 || x < 2 || k > 0);
                        commit(bar(ctl.b.wdone[half]));
                    }
                    commit(bar(ctl.added[ch & 1]));
                    commit(bar(ctl.b.empty[STAGES + st]));
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
            float x[4], next[4];
            load_decays(a, it.tok, it.n, it.head, next);
            for (int t = 0; t < it.n && alive; t += kC, ++ch) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = next[e];
                load_decays(a, it.tok + t + kC, it.n - t - kC, it.head, next); // the next chunk's, under way meanwhile
                if (!wait(ctl.b.gempty[ch & 1], ((ch >> 1) & 1) ^ 1))
                    break;
                form_decays<false>(x, ctl.tab[ch & 1]);
                arrive(ctl.b.gfull[ch & 1]);
            }
            if (!alive)
                break;
        }
    } else {
        const int w4 = warp & 3, quarter = (warp - 4) >> 2, row = 32 * w4 + lane;
        const bool has = row < DV;
        const int tok = 32 * quarter, half = quarter >> 1; // this warp's tokens of a chunk, and their place
        const uint32_t lanes = (uint32_t)w4 << 21;
        float s[WK];
        auto add = [&](unsigned c, float all) { // the sum of chunk c, which is done
            after_sync();
            uint32_t r[WK];
            tld(tmem + lanes + 128 * (c & 1) + quarter * WK, r);
#pragma unroll
            for (int e = 0; e < WK; ++e)
                s[e] = fmaf(s[e], all, __uint_as_float(r[e]));
            before_sync();
        };
        for (int q = 0; take(q, it); ++q) {
            float total = 1.f, last = 0.f;
#pragma unroll
            for (int k = 0; k < WK; ++k)
                s[k] = 0.f;
            for (int t = 0; t < it.n && alive; t += kC, advance()) { // (whole chunks: a segment with another behind it)
                if (!wait(ctl.b.gfull[ch & 1], (ch >> 1) & 1) || !wait(ctl.b.full[st], turn))
                    break;
                const uint32_t at = st * G::TILE + (row >> 6) * G::BLOCK + ((row & 63) >> 3 << 4) + (row & 7) * 2;
                float x[16];
                if (has)
                    read_column(smem, at + tok * 128, x);
                if (!wait(ctl.b.wdone[half], (ch & 1) ^ 1)) // the chunk before is done with the place
                    break;
                after_sync();
                const uint32_t to = tmem + lanes + CW + PLACE * half + (tok & 63) / 2;
                if (w4 < DV / 32)
                    weigh_column(x, &ctl.tab[ch & 1].w[tok], to, 32);
                if (has)
                    read_column(smem, at + (tok + 16) * 128, x);
                if (w4 < DV / 32)
                    weigh_column(x, &ctl.tab[ch & 1].w[tok + 16], to + 8, 32);
                tst_wait();
                before_sync();
                arrive(ctl.b.wready[half]);
                const float all = ctl.tab[ch & 1].all;
                arrive(ctl.b.empty[st]);
                arrive(ctl.b.gempty[ch & 1]);
                if (t > 0) {
                    if (!wait(ctl.added[(ch - 1) & 1], ((ch - 1) >> 1) & 1))
                        break;
                    add(ch - 1, last);
                }
                last = all;
                total *= all;
            }
            if (!alive || !wait(ctl.added[(ch - 1) & 1], ((ch - 1) >> 1) & 1))
                break;
            add(ch - 1, last);
            if (has) {
                float *const to = p.state + ((size_t)it.at * a.hv + it.head) * DV * DK + (size_t)row * DK + quarter * WK;
#pragma unroll
                for (int k = 0; k < WK; k += 8)
                    store8(to + k, &s[k]);
            }
            if (tid == 128)
                p.decay[(size_t)it.at * a.hv + it.head] = total;
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    wait_prior_grid();
}

// ---- host ----
// Chunks a segment, from what the host knows (the lengths are on the device; sequences are taken as equal): the fewest
// rounds of CTAs, in chunks, where a segment costs one more to begin, and forming the sums half a chunk's time.  Uncut,
// sequences of up to twice their mean length and of four chunks stay whole: a short piece too many is a round too many.
// One of 16,000 tokens (16 heads of 128) takes 95 us, whole 410; 2 of 4,000 64 and 115; one of 1,000 27 and 35; 8 of 1,500 to
// 2,600, whole, 93, and 174 where those over the mean are cut.
int segment_chunks(int nseq, int tokens, int hv, bool &cut)
{
    const int m = (int)(((long long)tokens + (long long)nseq * kC - 1) / ((long long)nseq * kC)); // chunks a sequence
    auto rounds = [&](long long n) { return (double)((n * nseq * hv + kSms - 1) / kSms); };
    const int len = (int)cheapest_length(m, kSms, [&](long long segs, long long chunks) {
        return rounds(segs) * (chunks + 1) + (segs > 1 ? rounds(segs - 1) * (0.5 * chunks + 1) + 3 : 0);
    });
    cut = len < m;
    const int best = cut ? len : 2 * m > 4 ? 2 * m : 4;
    return best < kMostChunks ? best : kMostChunks;
}
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
    constexpr int CHUNK = 5 * G::TILE + G::SBYTES + (int)sizeof(ChunkCtrl<DK, DV>);
    constexpr int SUM = 6 * G::TILE + (int)sizeof(SumCtrl<DK, DV>);
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
    CUtensorMap qmap, kmap, vmap, omap;
    if (!encode_tokens(&qmap, a.q, DK, a.hk, a.total_tokens, a.q_stride) || !encode_tokens(&kmap, a.k, DK, a.hk, a.total_tokens, a.k_stride) ||
        !encode_tokens(&vmap, a.v, DV, a.hv, a.total_tokens, a.v_stride) ||
        !encode_tokens(&omap, a.out, DV, a.hv, a.total_tokens, (long long)a.hv * DV))
        return cudaErrorInvalidValue;
    ChunkArgs p;
    p.a = a;
    p.rare = !a.cut;
    p.none = a.total_tokens <= (long long)kSerial * a.rows;
    p.least = kSerial;
    p.heads = a.hv;
    chunk_layout(p);
    const long long most = places(a.rows, a.total_tokens, a.span) * a.hv; // items
    const dim3 grid((unsigned)(most < kSms ? most : kSms));
    if (a.total_tokens > a.span) { // a sequence can have several segments
        e = launch_pdl(linear_sum_kernel<DK, DV>, grid, dim3(kThreads), (size_t)SUM, s, p, kmap, vmap);
        if (e == cudaSuccess)
            e = launch_scan(p, s);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(linear_chunk_kernel<DK, DV>, grid, dim3(kThreads), (size_t)CHUNK, s, p, qmap, kmap, vmap, omap);
}

} // namespace

int linear_chunked_segment(const LinearArgs &a, bool &cut) { return kC * segment_chunks(a.rows, a.total_tokens, a.hv, cut); }

cudaError_t launch_linear_chunked(const LinearArgs &a, cudaStream_t s)
{
    if (a.dk == 128)
        return a.dv == 128 ? go<128, 128>(a, s) : go<128, 64>(a, s);
    return a.dv == 128 ? go<64, 128>(a, s) : go<64, 64>(a, s);
}

} // namespace gdn
