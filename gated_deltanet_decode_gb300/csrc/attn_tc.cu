// Attention of new tokens over a paged cache on the tensor cores (sm_103a),
// bf16: softmax(scale Q K^T) V with a running maximum and sum per row.
//
// Rows.  The g = hq / hkv query heads that share a key head are packed as rows
// (token, head) of M = 128 products, floor(128 / g) tokens a tile, so a decode
// step with one token uses g rows of a tile and reads each key once.
//
// Work.  An item is one key head and one tile of tokens (a pair of tiles when
// the row has more tokens than one holds); its keys come in tiles of KT.  All
// items' key tiles, in order, are cut into equal runs, one a CTA, whatever the
// lengths: the plan is made on the device from the lengths there.  An item cut
// by a run's end leaves partial sums (m, l, O in fp32) in the workspace, which
// attn_combine_kernel joins in the order of the keys.
//
// A CTA: warp 0 brings K and V pages by tensor copies into a ring, warp 1
// issues the products, warp 2 brings Q, warp 3 walks the work, and two groups
// of four warps take the softmax, a thread a row.  S = Q K^T lands in tensor
// memory, the weights go back over it as bf16, and P V sums up in tensor
// memory.  The two groups work on alternate steps: on the two tiles of a pair,
// or on alternate key tiles of a single tile, each with its own O, m and l,
// merged at the item's end.  At d = 256 tensor memory holds one O, so one
// group takes all steps.
//
// The products go out in the steps' order, P V of step i and then S of step i +
// 2, so that one group's softmax runs beside the other's products; with a
// product warp for each group the two fell into step and took turns with the
// tensor cores instead (297 us against 286 for a 2,048-token chunk over 16 k).
// The queue of products is a few deep, so the issuing warp is held up until
// they are nearly done; the weights are handed over by halves, so that the
// first half's product runs while the second half's are computed.
//
// Bound.  Decode streams the cache: 64 rows of 0.5 to 8 k (477 MB) take 95 us,
// two of 180 to 210 k (763 MB) 124 us, 92 % of a plain copy's rate once
// started; a start costs 5 us, the end with the joining 5.  A 2,048-token chunk
// over 16 k (16 heads of 128) takes 230 us, 1,240 TFLOP/s: the products are at
// work for 60 % of it.  A group's first weights come about 1,150 clocks after
// its scores, the other group's products cover 1,024, and the next scores wait
// for the weights' product, as tensor memory is full.  (Key tiles of 64 leave
// room for a second score tile, but N = 64 products take as long as N = 128
// ones: 301 us.)
//
// The weights are rounded to bf16 for their product with V (the row's sum takes
// them as they are): A and B of a product have one type, and a head and a tail
// of every weight would take a second product with V a step.  Results are off
// by 0.0022 of their norm instead of the 0.0017 of their own rounding.
//
// O is rescaled only when a row's maximum has grown by over 2^8 since the
// value in use (kLazy): weights then stay below 2^8 and sums in fp32 lose
// nothing.
#include <atomic>
#include <mutex>
#include <type_traits>

#include "attn_plan.cuh"
#include "gdn_device.cuh"
#include "gdn_internal.h"
#include "gdn_ptx.cuh"
#include "tc_ops.cuh"

namespace gdn {
namespace {

constexpr int kQueue = 4;   // items in flight between the walking warp and the others
constexpr int kMeta = 16;   // key tiles whose valid-row count is kept; over a ring's tiles
constexpr float kLazy = 8.f;
constexpr int kPairTokens = 1024; // and rows of new tokens of a key head from which items are pairs of tiles
constexpr int kTmemCols = 512;

// Rows' own keys behind shared prefixes make items of a few tiles, of which each takes about as long as three tiles to begin
// and to end (its copies' latency, and sums that are not ready before their products): 64 samples of 16,000 tokens took 43.2 us,
// with two tiles 45.2, with five 51.0.
struct SharedCost : EvenCost {
    static constexpr int item = 3;
};

template <int D> struct Geo {
    static constexpr int KT = D == 256 ? 64 : 128;       // keys a tile
    static constexpr int NO = D == 256 ? 1 : 2;          // O accumulators, softmax groups, tiles of an item at most
    static constexpr int CH = D / 64;                    // 128-byte columns of a row
    static constexpr int QBYTES = 128 * D * 2;           // one Q tile
    static constexpr int SBYTES = KT * D * 2;            // one ring stage: a K or V tile
    static constexpr int STAGES = D == 64 ? 10 : 5;
    static constexpr int NQ = NO;                        // Q tiles in shared memory
    static constexpr int THREADS = 128 + 128 * NO;
    static constexpr int QUEUE_READERS = 3 + 4 * NO;     // warps 0, 1, 2 and the softmax warps
    static constexpr int HALVES = KT / 64;               // parts in which a step's weights are handed over
    // tensor memory columns
    static constexpr int S0 = 0;                         // S (and P) of step parity b: S0 + b KT
    static constexpr int O0 = 2 * KT;                    // O of accumulator o: O0 + o D
    static constexpr int RING = QBYTES * NQ;
    static constexpr int CTRL = RING + SBYTES * STAGES;
    static constexpr int TOTAL = CTRL + 3 * 1024;            // and the control block
};

// The control block in shared memory, after Q and the ring.
template <typename V> struct CtrlOf {
    unsigned long long full[12], empty[12];    // ring
    unsigned long long qfull[2], qempty[2];
    unsigned long long sready[2], pready[2][2], odone[2];
    unsigned long long ifull[kQueue], iempty[kQueue];
    unsigned long long drain; // the last products
    unsigned long long merge; // the two softmax groups, at the end of a single tile's item
    typename V::ItemT item[kQueue];
    int valid[kMeta];       // good rows of a key tile, by the tile's count
    long long scan[13];
    FoundOf<V> found;       // this run's first row, by the plan
    uint32_t tmem;
    float ml[2][128][2];    // (m, l) of the two groups' rows, for the merge
    int bad[2];             // first key that could not be read, by group
    // 1 + the last item of a queue parity with a non-finite V element that only some of its tokens see.  Two words, as the
    // groups of a pair do not meet at its end: a warp may be in item q + 1 before another has looked at item q's word.  None
    // is in item q + 2 then, whose scores come after weights that every warp hands over in item q + 1, or after a meeting.
    int dirty[2];
};
static_assert(sizeof(CtrlOf<Plain>) <= 3 * 1024 && sizeof(CtrlOf<Shared>) <= 3 * 1024, "control block");

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// x[at] += y without indexing the registers
__device__ __forceinline__ void poison(float (&x)[32], int at, float y)
{
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e == at)
            x[e] += y;
}

// ---------------------------------------------------------------------------
template <int D, bool SH>
__global__ void __launch_bounds__(Geo<D>::THREADS, 1)
    attn_tc_kernel(const __grid_constant__ typename Kind<SH>::Args p, const __grid_constant__ CUtensorMap kmap,
                   const __grid_constant__ CUtensorMap vmap)
{
    typedef Geo<D> G;
    typedef typename std::conditional<SH, Shared, Plain>::type View;
    typedef CtrlOf<View> Ctrl;
    typedef typename Kind<SH>::ItemT ItemT;
    typedef typename std::conditional<SH, SharedCost, EvenCost>::type Cost;
    constexpr int KT = G::KT;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctrl &ctl = *reinterpret_cast<Ctrl *>(smem + G::CTRL);
    const uint32_t sbase = sm_addr(smem);
    const AttentionArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mt = item_tokens(p, G::NO), hkv = a.pages.hkv, ps = a.pages.page_size;
    auto bar = [&](unsigned long long &b) { return sm_addr(&b); };

    if (sbase & 1023) { // the swizzled tiles need it; the whole CTA leaves
        if (tid == 0)
            report(a.err, GDN_DEVERR_TIMEOUT);
        return;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sm_addr(&ctl.tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 64) { // the copies' descriptors, while the lengths are looked up
        asm volatile("prefetch.tensormap [%0];" ::"l"(&kmap) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&vmap) : "memory");
    }
    if (tid == 32) {
        for (int i = 0; i < G::STAGES; ++i)
            mbar_init(bar(ctl.full[i]), 1), mbar_init(bar(ctl.empty[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(ctl.qfull[i]), 1), mbar_init(bar(ctl.qempty[i]), 1);
            mbar_init(bar(ctl.sready[i]), 1), mbar_init(bar(ctl.odone[i]), 1);
            mbar_init(bar(ctl.pready[i][0]), 4), mbar_init(bar(ctl.pready[i][1]), 4);
        }
        for (int i = 0; i < kQueue; ++i)
            mbar_init(bar(ctl.ifull[i]), 1), mbar_init(bar(ctl.iempty[i]), G::QUEUE_READERS);
        mbar_init(bar(ctl.drain), 1);
        mbar_init(bar(ctl.merge), 8);
        ctl.dirty[0] = ctl.dirty[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    before_sync();
    __syncthreads();
    after_sync();
    const uint32_t tmem = ctl.tmem;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const RunOf<View> run = plan_run<G::THREADS, KT, Cost, View>(p, mt, ctl.scan, ctl.found);
    bool alive = true; // false once a bounded wait ran out
    auto wait_at = [&](uint32_t b, uint32_t parity) { // by a whole warp, which goes on or leaves as one
        if (!__all_sync(0xffffffffu, mbar_try(b, parity)) && alive && !__all_sync(0xffffffffu, mbar_wait(b, parity))) {
            alive = false;
            report(a.err, GDN_DEVERR_TIMEOUT);
        }
        return alive;
    };
    auto wait = [&](unsigned long long &b, uint32_t parity) { return wait_at(bar(b), parity); };
    auto stage_addr = [&](int s) { return sbase + G::RING + s * G::SBYTES; };
    // place of the item's V tiles in the ring's order: one tile at a time K0 K1 V0 K2 V1 ... (a single tile's steps look
    // one key tile ahead), in pairs K0 V0 K1 V1 ...
    auto v_place = [](bool pair, int j, int n) { return pair ? 2 * j + 1 : j == n - 1 ? 2 * n - 1 : 2 * j + 2; };

    if (warp < 4) {
        if constexpr (G::NO == 2)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 3) {
            // ---- the walk: this run's items, in order
            Walk<Cost, View, typename Kind<SH>::Args> walk(p, run, mt, KT);
            ItemT it;
            for (int q = 0; alive; ++q) {
                const bool more = walk.next(it);
                const int slot = q % kQueue;
                if (!wait(ctl.iempty[slot], (q / kQueue + 1) & 1))
                    break;
                if (!more)
                    it.ntok = 0;
                if (lane == 0) {
                    ctl.item[slot] = it;
                    mbar_arrive(bar(ctl.ifull[slot]));
                }
                __syncwarp();
                if (!more)
                    break;
            }
        } else if (warp == 0) {
            // ---- K and V pages into the ring
            const int ppt = max(1, KT / ps);              // pages of a key tile (a page may hold several tiles)
            const int box = min(KT, ps);                  // keys a copy
            unsigned issued = 0, tiles = 0;
            for (int q = 0;; ++q) {
                const int slot = q % kQueue;
                if (!wait(ctl.ifull[slot], (q / kQueue) & 1))
                    break;
                const ItemT it = ctl.item[slot];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(ctl.iempty[slot]));
                if (it.ntok == 0)
                    break;
                const int32_t *const table = item_table(a.c, it);
                const int kvh = it.head / p.groups;
                const int end = it.see + (it.ntok - 1) * see_step(it); // keys the item's last token sees
                const int pages = (end + ps - 1) >> a.pages.page_shift;
                const bool pair = G::NO == 2 && it.ntok > p.tq;
                const int n = it.jb - it.ja;
                // pages win .. win + 63 are in the lanes, two each; V is below win + 32, and K at most a tile ahead
                int win = (it.ja * KT) >> a.pages.page_shift;
                auto fetch = [&](int i) { return i < pages ? table[i] : 0; };
                int near = fetch(win + lane), far = fetch(win + 32 + lane);
                int broken = 0x7fffffff;                  // first key on a page that cannot be read
                auto copy = [&](bool is_v, int j) {       // key tile ja + j
                    const int key = (it.ja + j) * KT, pg = key >> a.pages.page_shift;
                    const int i = min(lane, ppt - 1);
                    const int w = pg + i - win;
                    const int pn = __shfl_sync(0xffffffffu, near, w & 31), pf = __shfl_sync(0xffffffffu, far, w & 31);
                    int page = w < 32 ? pn : pf;
                    const bool inside = lane < ppt && key + i * box < end;
                    const bool fine = page > 0 && page < a.pages.num_pages;
                    const unsigned wrong = __ballot_sync(0xffffffffu, inside && !fine);
                    if (wrong) {
                        if (lane == 0)
                            report(a.err, GDN_DEVERR_BAD_PAGE);
                        broken = min(broken, key + (__ffs(wrong) - 1) * box);
                    }
                    const bool take = inside && key + i * box < broken;
                    const int st = issued % G::STAGES;
                    if (!wait(ctl.empty[st], (issued / G::STAGES + 1) & 1))
                        return;
                    if (!is_v && lane == 0)
                        ctl.valid[(tiles + j) % kMeta] = max(0, min(KT, min(end, broken) - key));
                    const int count = __popc(__ballot_sync(0xffffffffu, take));
                    const uint32_t b = bar(ctl.full[st]);
                    if (lane == 0) {
                        if (count)
                            mbar_arrive_tx(b, (uint32_t)(count * box * D * 2));
                        else
                            mbar_arrive(b);
                    }
                    __syncwarp();
                    if (take) {
                        const uint32_t dst = stage_addr(st) + i * box * 128;
#pragma unroll
                        for (int c = 0; c < G::CH; ++c)
                            tma3(dst + c * KT * 128, is_v ? &vmap : &kmap, 64 * c, key & (ps - 1),
                                 (a.pages.layer * a.pages.num_pages + page) * hkv + kvh, b);
                    }
                    __syncwarp();
                    ++issued;
                };
                auto slide = [&](int j) { // the window starts at or before V's tile
                    const int pg = ((it.ja + j) * KT) >> a.pages.page_shift;
                    if (pg >= win + 32) {
                        win += 32;
                        near = far;
                        far = fetch(win + 32 + lane);
                    }
                };
                if (pair) {
                    for (int j = 0; j < n && alive; ++j)
                        slide(j), copy(false, j), copy(true, j);
                } else {
                    copy(false, 0);
                    for (int j = 0; j < n && alive; ++j) {
                        slide(j);
                        if (j + 1 < n)
                            copy(false, j + 1);
                        copy(true, j);
                    }
                }
                tiles += n;
            }
            // the last copies land before the CTA leaves, whoever still waits for them
            for (unsigned i = issued > (unsigned)G::STAGES ? issued - G::STAGES : 0; i < issued; ++i)
                mbar_wait(bar(ctl.full[i % G::STAGES]), (i / G::STAGES) & 1);
        } else if (warp == 1) {
            // ---- the products.  The whole warp walks, on values that the broadcasts make uniform to the compiler, and
            // one elected lane issues: an issue loop in a divergent branch took 1,970 cycles a step, twice the products'.
            const bool leader = elect();
            int st = 0, kst = 0, vst = 0; // the ring's next place; the places of the K and V tiles in use
            uint32_t parity = 0, pparity[2] = {0, 0};
            unsigned qc = 0;
            const uint32_t full0 = bar(ctl.full[0]), empty0 = bar(ctl.empty[0]);
            // The places of the ring are waited for in order, every one: a parity wait tells a phase only from the one
            // before it, and copies may land out of order.
            auto advance = [&](int &at) {
                at = st;
                if (++st == G::STAGES)
                    st = 0, parity ^= 1;
            };
            for (int q = 0;; ++q) {
                const int slot = q % kQueue;
                if (!wait(ctl.ifull[slot], (q / kQueue) & 1))
                    break;
                const int ntok = __shfl_sync(0xffffffffu, ctl.item[slot].ntok, 0);
                const int n = __shfl_sync(0xffffffffu, ctl.item[slot].jb - ctl.item[slot].ja, 0);
                // keys from the run's first tile to the last that a token sees (see `used` below)
                const int left = !SH ? 0 : __shfl_sync(0xffffffffu, ctl.item[slot].see + (ntok - 1) * see_step(ctl.item[slot]) - ctl.item[slot].ja * KT, 0);
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(ctl.iempty[slot]));
                if (ntok == 0)
                    break;
                const bool pair = G::NO == 2 && ntok > p.tq;
                const int steps = pair ? 2 * n : n, qn = pair ? 2 : 1;
                for (int i = 0; i < qn; ++i)
                    wait(ctl.qfull[(qc + i) % G::NQ], ((qc + i) / G::NQ) & 1);
                const uint32_t q0 = sbase + (qc % G::NQ) * G::QBYTES, q1 = pair ? sbase + ((qc + 1) % G::NQ) * G::QBYTES : q0;
                // S of a step of parity b
                auto s_step = [&](int i, const int b) {
                    if (!pair || b == 0) {
                        if (!wait_at(full0 + 8 * st, parity))
                            return;
                        advance(kst);
                    }
                    after_sync();
                    const uint64_t qd = desc_k(b ? q1 : q0), kd = desc_k(stage_addr(kst));
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            mma_ss(tmem + G::S0 + b * KT, qd + (((k >> 2) * 128 * 128 + (k & 3) * 32) >> 4),
                                   kd + (((k >> 2) * KT * 128 + (k & 3) * 32) >> 4), idesc(KT, false), k > 0);
                        commit(bar(ctl.sready[b]));
                        if (!pair || b)
                            commit(empty0 + 8 * kst);
                        if (i == steps - 1)
                            for (int k = 0; k < qn; ++k)
                                commit(bar(ctl.qempty[(qc + k) % G::NQ]));
                    }
                };
                // P V of step i, of parity b, then S of step i + 2
                auto step = [&](int i, const int b) {
                    const int o = G::NO == 2 ? b : 0;
                    if (!pair || b == 0) {
                        if (!wait_at(full0 + 8 * st, parity))
                            return;
                        advance(vst);
                    }
                    const uint64_t vd = desc_mn(stage_addr(vst), KT * 128);
                    const bool more = i >= G::NO;
                    const int last = left - (pair ? i >> 1 : i) * KT; // keys of the tile that are seen, where they are few
#pragma unroll
                    for (int half = 0; half < G::HALVES; ++half) {
                        if (!wait(ctl.pready[b][half], pparity[b]))
                            return;
                        after_sync();
                        if (leader) {
                            auto product = [&](int k) {
                                mma_ts(tmem + G::O0 + o * D, tmem + G::S0 + b * KT + 8 * k, vd + k * (2048 >> 4), idesc(D, true), k > 0 || more);
                            };
                            if (!SH || last > KT - 16) {
#pragma unroll
                                for (int k = 4 * half; k < 4 * half + 4; ++k)
                                    product(k);
                            } else { // 16 keys a product: those past the last key are left out, and V's rows there not looked at
#pragma unroll 1
                                for (int k = 4 * half; k < 4 * half + 4 && 16 * k < last; ++k)
                                    product(k);
                            }
                            if (half == G::HALVES - 1) {
                                // O is waited for at an item's end and, with one group, before it is rescaled
                                if (G::NO == 1 || i + 2 >= steps)
                                    commit(bar(ctl.odone[b]));
                                if (!pair || b)
                                    commit(empty0 + 8 * vst);
                            }
                        }
                    }
                    pparity[b] ^= 1;
                    if (i + 2 < steps)
                        s_step(i + 2, b);
                };
                if (!alive)
                    break;
                s_step(0, 0);
                if (steps > 1)
                    s_step(1, 1);
                for (int i = 0; i < steps && alive; i += 2) {
                    step(i, 0);
                    if (i + 1 < steps)
                        step(i + 1, 1);
                }
                qc += qn;
                if (!alive)
                    break;
            }
            // everything issued is done, and has said so, before tensor memory and the barriers go
            __syncwarp();
            if (leader)
                commit(bar(ctl.drain));
            __syncwarp();
            mbar_wait(bar(ctl.drain), 0);
        } else {
            // ---- Q tiles.  By 16-byte asynchronous copies; with shared prefixes by a tensor copy, as one warp's copies take 4 us
            // for 128 rows, and a group's item, cut into many parts, has its Q in each of them (8 chunks of 64 tokens behind
            // 4,000 shared ones: 57.1 us by copies, 40.8; 64 samples of 16,000: 44.5 and 43.7; 16 of 512: 16.4 and 15.6)
            unsigned qc = 0;
            for (int q = 0;; ++q) {
                const int slot = q % kQueue;
                if (!wait(ctl.ifull[slot], (q / kQueue) & 1))
                    break;
                const ItemT it = ctl.item[slot];
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(bar(ctl.iempty[slot]));
                if (it.ntok == 0)
                    break;
                const bool pair = G::NO == 2 && it.ntok > p.tq;
                for (int i = 0; i < (pair ? 2 : 1); ++i, ++qc) {
                    const int s = qc % G::NQ;
                    if (!wait(ctl.qempty[s], (qc / G::NQ + 1) & 1))
                        break;
                    if constexpr (SH) { // a tile at once, with the rows of other tokens behind the item's
                        if (lane == 0) {
                            mbar_arrive_tx(bar(ctl.qfull[s]), (uint32_t)(p.tq * p.g * D * 2));
                            for (int c = 0; c < G::CH; ++c)
                                tma3(sbase + s * G::QBYTES + c * 128 * 128, &p.qmap, 64 * c, it.head * p.g, it.tok + i * p.tq,
                                     bar(ctl.qfull[s]));
                        }
                        __syncwarp();
                    } else {
                        const int rows = (min(it.ntok - i * p.tq, p.tq)) * p.g;
                        constexpr int VR = D / 8; // 16-byte vectors a row
                        const bf16 *const src = static_cast<const bf16 *>(a.q) + (size_t)(it.tok + i * p.tq) * a.q_stride +
                                                (size_t)it.head * p.g * D;
                        const uint32_t dst = sbase + s * G::QBYTES;
                        constexpr int RP = 32 / VR;                                // rows a pass
                        const int vec = lane % VR;
                        int row = lane / VR, tok = row / p.g, head = row - tok * p.g;
                        const uint32_t at = dst + (vec >> 3) * 128 * 128;
#pragma unroll 4
                        for (; row < rows; row += RP) {
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                             at + row * 128 + (((vec & 7) ^ (row & 7)) << 4)),
                                         "l"(src + (size_t)tok * a.q_stride + head * D + vec * 8)
                                         : "memory");
                            for (head += RP; head >= p.g; head -= p.g)
                                ++tok;
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        smem_to_async();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(ctl.qfull[s]));
                    }
                }
                if (!alive)
                    break;
            }
            if constexpr (SH) // the last copies land before the CTA leaves, whoever still waits for them
                for (unsigned i = qc > (unsigned)G::NQ ? qc - G::NQ : 0; i < qc; ++i)
                    mbar_wait(bar(ctl.qfull[i % G::NQ]), (i / G::NQ) & 1);
        }
    } else {
        if constexpr (G::NO == 2)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        // ---- softmax: a thread a row; first, zeros where no live row writes
        zero_dead<bf16, D, 128 * G::NO, View>(p, tid - 128);
        const int grp = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21; // 32 tensor-memory lanes a warp
        const float c = a.scale * 1.44269504088896341f;    // weights are 2^(c (s - m))
        const int tok = row / p.g;
        unsigned cnt[2] = {0, 0};  // steps done, by step parity
        unsigned ends[2] = {0, 0}; // items done that have steps of the parity
        unsigned tiles = 0, place0 = 0, meets = 0;
        auto meet = [&] { // of the two groups
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(ctl.merge));
            return wait(ctl.merge, meets++ & 1);
        };
        for (int q = 0;; ++q) {
            const int slot = q % kQueue;
            if (!wait(ctl.ifull[slot], (q / kQueue) & 1))
                break;
            const ItemT it = ctl.item[slot];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar(ctl.iempty[slot]));
            if (it.ntok == 0)
                break;
            const bool pair = G::NO == 2 && it.ntok > p.tq;
            const int n = it.jb - it.ja, steps = pair ? 2 * n : n;
            const int tt = tok + (pair ? grp * p.tq : 0);            // this row's token in the item
            const bool mine = tok < p.tq && tt < it.ntok;
            const int see = mine ? it.see + tt * see_step(it) : 0;   // keys this row sees
            const int end = it.see + (it.ntok - 1) * see_step(it);
            const bool idle = __all_sync(0xffffffffu, !mine);
            float m = -INFINITY, l = 0.f;
            int broken = 0x7fffffff;
            for (int i = G::NO == 2 ? grp : 0; i < steps; i += G::NO) {
                const int j = pair ? i >> 1 : i, b = i & 1, o = G::NO == 2 ? b : 0;
                if (!wait(ctl.sready[b], cnt[b] & 1))
                    break;
                ++cnt[b];
                after_sync();
                const int key = (it.ja + j) * KT;
                const int valid = *reinterpret_cast<volatile int *>(&ctl.valid[(tiles + j) % kMeta]);
                if (valid < min(KT, end - key))
                    broken = min(broken, key + valid);
                const int later = max(0, it.see - key); // keys of the tile from here on are hidden from some tokens
                // and those that the product with V takes (with shared prefixes, whose rows' own keys are few: else the choice
                // takes 2 % of a prompt's chunk)
                const int used = SH ? min(KT, (end - key + 15) & ~15) : KT;
                // A weight of zero does not hide a NaN or an infinity.  Rows of V past the good ones may hold anything:
                // they become zeros.  Elements that only some tokens see become zeros too where they are not finite,
                // and the item's end adds them to the rows that do see them.
                auto clean = [&] {
                    if (later >= used)
                        return true;
                    const unsigned pl = place0 + v_place(pair, j, n);
                    const int st = pl % G::STAGES;
                    if (!wait(ctl.full[st], (pl / G::STAGES) & 1))
                        return false;
                    unsigned char *const v = smem + G::RING + st * G::SBYTES;
                    constexpr int VR = 8 * G::CH; // 16-byte vectors a key; a thread keeps its place in it (a division a vector took
                                                  // 3 us of a tile)
                    for (int r = later + row / VR; r < used; r += 128 / VR) {
                        uint4 *const at = reinterpret_cast<uint4 *>(v + (row % VR >> 3) * KT * 128 + r * 128 + (row & 7) * 16);
                        if (r >= valid) {
                            *at = make_uint4(0, 0, 0, 0);
                        } else {
                            uint4 z = *at;
                            if (!(finite2(z.x) && finite2(z.y) && finite2(z.z) && finite2(z.w))) {
                                *reinterpret_cast<volatile int *>(&ctl.dirty[q & 1]) = q + 1;
                                __threadfence_block(); // before the zeros: the other group may scan this tile too
                                z.x = drop2(z.x), z.y = drop2(z.y), z.z = drop2(z.z), z.w = drop2(z.w);
                                *at = z;
                            }
                        }
                    }
                    smem_to_async();
                    __syncwarp(); // what follows is for whole warps
                    return true;
                };
                if (!idle) {
                    const uint32_t sa = tmem + lanes + G::S0 + b * KT;
                    float s[KT];
                    tld(sa, *reinterpret_cast<uint32_t(*)[KT]>(&s[0]));
                    // rows that are no token's are left to compute what they hold: masking them cost decode steps, where
                    // most rows of the warp are such, as much as the weights
                    const int nv = mine ? min(valid, see - key) : KT;
                    if (__any_sync(0xffffffffu, nv < KT)) {
#pragma unroll
                        for (int k = 0; k < KT; ++k)
                            s[k] = k < nv ? s[k] : -INFINITY;
                    }
                    float t[4] = {m, s[0], s[1], s[2]};
#pragma unroll
                    for (int k = 3; k + 1 < KT; k += 2)
                        t[(k >> 1) & 3] = max3(t[(k >> 1) & 3], s[k], s[k + 1]);
                    const float top = fmaxf(max3(t[0], t[1], t[2]), fmaxf(t[3], s[KT - 1]));
                    const bool grow = mine && (top - m) * c > kLazy; // -inf to -inf is no growth
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2((m - top) * c) : 1.f;
                        if (grow)
                            m = top;
                        l *= f;
                        const bool has_o = G::NO == 2 ? i >= 2 : i >= 1;
                        if (has_o) {
                            // The products into O are done: with two groups all, as this step's S was issued after them;
                            // with one group the last step's may be under way, and the one before it is done, so the
                            // parity tells the two apart.
                            if (G::NO == 1) {
                                if (!wait(ctl.odone[b ^ 1], (cnt[b ^ 1] - 1) & 1))
                                    break;
                                after_sync();
                            }
#pragma unroll
                            for (int k = 0; k < D; k += 32) {
                                uint32_t r[32];
                                tld(tmem + lanes + G::O0 + o * D + k, r);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                                tst(tmem + lanes + G::O0 + o * D + k, r);
                            }
                        }
                    }
                    const float shift = m == -INFINITY ? 0.f : -m * c;
                    const float2 c2 = make_float2(c, c), sh2 = make_float2(shift, shift);
                    if (!clean())
                        break;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int half = 0; half < G::HALVES; ++half) {
                        uint32_t w[32];
#pragma unroll
                        for (int k = 0; k < 64; k += 2) {
                            float2 x = fma2(make_float2(s[64 * half + k], s[64 * half + k + 1]), c2, sh2);
                            x.x = ex2(x.x), x.y = ex2(x.y);
                            sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], x);
                            const __nv_bfloat162 hx = __floats2bfloat162_rn(x.x, x.y);
                            w[k / 2] = *reinterpret_cast<const uint32_t *>(&hx);
                        }
                        tst(sa + 32 * half, w);
                        tst_wait();
                        before_sync();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive(bar(ctl.pready[b][half]));
                        __syncwarp();
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                } else {
                    if (!clean())
                        break;
                    before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(ctl.pready[b][0]));
                        if (G::HALVES == 2)
                            mbar_arrive(bar(ctl.pready[b][1]));
                    }
                    __syncwarp();
                }
            }
            // steps of the other group, which its counters follow
            if (G::NO == 2)
                cnt[grp ^ 1] += grp == 0 ? steps / 2 : (steps + 1) / 2;
            if (!alive)
                break;
            tiles += n;
            place0 += 2 * n;

            // ---- the item's end
            const float NaN = __int_as_float(0x7fc00000);
            bf16 *const out = static_cast<bf16 *>(a.out) + ((size_t)(it.tok + tt) * a.hq + it.head * p.g + (row - tok * p.g)) * D;
            const bool both = G::NO == 2 && !pair && steps > 1; // two accumulators hold parts of the same rows
            float f0 = 1.f, f1 = 0.f;
            if (G::NO == 2 && !pair) {
                ctl.ml[grp][row][0] = m, ctl.ml[grp][row][1] = l;
                if (row == 0)
                    ctl.bad[grp] = broken;
                if (!meet())
                    break;
                const float m0 = ctl.ml[0][row][0], m1 = ctl.ml[1][row][0];
                broken = min(ctl.bad[0], ctl.bad[1]);
                m = fmaxf(m0, m1);
                f0 = m0 == -INFINITY ? 0.f : ex2((m0 - m) * c);
                f1 = m1 == -INFINITY ? 0.f : ex2((m1 - m) * c);
                l = ctl.ml[0][row][1] * f0 + ctl.ml[1][row][1] * f1;
            }
            // every product into the accumulators that this group reads is done
            {
                const int last = (steps - 1) & 1; // with one group: the last step's product is after all others
                const bool own0 = G::NO == 1 ? last == 0 : !pair || grp == 0;
                const bool own1 = G::NO == 1 ? last == 1 : both || (pair && grp == 1);
                // completions so far: one a step with one group, else one an item
                const unsigned c0 = G::NO == 1 ? cnt[0] : ends[0] + 1, c1 = G::NO == 1 ? cnt[1] : ends[1] + 1;
                if ((own0 && !wait(ctl.odone[0], (c0 - 1) & 1)) || (own1 && !wait(ctl.odone[1], (c1 - 1) & 1)))
                    break;
                ++ends[0];
                ends[1] += steps > 1;
                after_sync();
            }
            const bool bad = see > broken;
            const bool dirty = *reinterpret_cast<volatile int *>(&ctl.dirty[q & 1]) == q + 1;
            if (!idle) {
                const int o = pair ? grp : 0;
                const int k0 = G::NO == 2 && !pair ? grp * (D / 2) : 0, k1 = G::NO == 2 && !pair ? k0 + D / 2 : D;
                const bool partial = it.part != -1;
                const float inv = partial ? 1.f : 1.f / l;
                const size_t prow = part_row(p, it, it.tok + tt, it.head * p.g + (row - tok * p.g), row + (pair ? grp * 128 : 0));
                float *const po = p.part_o + prow * D;
                if (partial && mine && k0 == 0)
                    p.part_ml[prow] = make_float2(bad ? NaN : m, l);
#pragma unroll 1
                for (int k = k0; k < k1; k += 32) {
                    uint32_t r[32];
                    float x[32];
                    tld(tmem + lanes + G::O0 + o * D + k, r);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        x[e] = __uint_as_float(r[e]) * (f0 * inv);
                    if (both) {
                        tld(tmem + lanes + G::O0 + D + k, r);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = fmaf(__uint_as_float(r[e]), f1 * inv, x[e]);
                    }
                    if (dirty && !bad) {
                        // the elements that the tiles lost, from the cache itself
                        for (int key = max(it.see, it.ja * KT); key < min(see, it.jb * KT); ++key) {
                            const int page = item_table(a.c, it)[key >> a.pages.page_shift];
                            const bf16 *const v = static_cast<const bf16 *>(a.pages.v) +
                                                  (((size_t)page * hkv + it.head / p.groups) * ps + (key & (ps - 1))) * D + k;
#pragma unroll 1
                            for (int e = 0; e < 32; ++e) {
                                const float y = __bfloat162float(v[e]);
                                if (!isfinite(y))
                                    poison(x, e, y);
                            }
                        }
                    }
                    if (mine && partial) {
#pragma unroll
                        for (int e = 0; e < 32; e += SH ? 8 : 4) {
                            if constexpr (SH)
                                store8(po + k + e, &x[e]);
                            else
                                *reinterpret_cast<float4 *>(po + k + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                        }
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[e + 2 * y], x[e + 2 * y + 1]);
                                w[y] = bad ? 0u : *reinterpret_cast<const uint32_t *>(&h2);
                            }
                            *reinterpret_cast<uint4 *>(out + k + e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    __syncwarp();
                }
            }
            before_sync();
            // both groups have read both accumulators before either starts the next item
            if (G::NO == 2 && !pair && !meet())
                break;
        }
    }
    before_sync();
    __syncthreads();
    after_sync();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// ---- host ----
// a pool's K or V as [layers x pages x heads][page_size][d], boxes of 64 d x `box` keys
bool encode_pages(CUtensorMap *m, void *base, const kv_page_pool &v, int box)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)v.d, (cuuint64_t)v.page_size, (cuuint64_t)v.layers * v.num_pages * v.hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)v.d * 2, (cuuint64_t)v.page_size * v.d * 2};
    const cuuint32_t boxes[3] = {64u, (cuuint32_t)box, 1u};
    const cuuint32_t step[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, boxes, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [tokens][heads][d], boxes of 64 d x the heads of a group x the tokens of a tile: its rows, in order
bool encode_q(CUtensorMap *m, const AttentionArgs &a, int g, int tq)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_tiled();
    if (!fn)
        return false;
    const cuuint64_t dims[3] = {(cuuint64_t)a.pages.d, (cuuint64_t)a.hq, (cuuint64_t)a.c.total_tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)a.pages.d * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t boxes[3] = {64u, (cuuint32_t)g, (cuuint32_t)tq}, step[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, boxes, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// With shared prefixes an item is a single tile where pairs would be few: a group's item over long shared keys is cut into
// many parts, and each costs its rows' partial sums.  Of 64 samples of a prompt of 16,000 (288 rows a key head) pairs take
// 44.8 us and single tiles 44.4; of 8 chunks of 64 tokens (2,048 rows) 41.0 and 45.5, of 512 tokens 205 and 279.
bool single_tiles(int d, int g, int total_tokens, bool shared) { return d == 256 || (shared && total_tokens < kPairTokens / g); }

int slot_rows(int d, int g, int total_tokens, bool shared)
{
    const int tq = 128 / g, one = tq * g;
    if (single_tiles(d, g, total_tokens, shared) || total_tokens <= tq)
        return total_tokens < tq ? total_tokens * g : one;
    return 128 + one; // a pair of tiles, the second's rows from 128 on
}

// The kernel's shared memory, once a device.
template <int D, bool SH> cudaError_t configure()
{
    static_assert(Geo<D>::TOTAL <= 232448, "shared memory");
    static std::atomic<unsigned long long> configured{0}; // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(attn_tc_kernel<D, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<D>::TOTAL);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int D> cudaError_t go(const AttentionArgs &a, const SharedPrefix *f, kv_page_pool &pool, cudaStream_t s)
{
    typedef Geo<D> G;
    cudaError_t e = f ? configure<D, true>() : configure<D, false>();
    if (e != cudaSuccess)
        return e;
    SharedArgs p;
    p.a = a;
    p.g = group_heads(a.hq, a.pages.hkv, 128);
    p.groups = a.hq / a.pages.hkv / p.g;
    p.tq = 128 / p.g;
    p.runs = kSms; // one CTA an SM: its tensor memory is taken whole
    p.rows_max = slot_rows(D, p.g, a.c.total_tokens, f != nullptr);
    p.second = single_tiles(D, p.g, a.c.total_tokens, f != nullptr) ? 0 : 128;
    {
        const std::lock_guard<std::mutex> lk(pool.map_mutex);
        const int box = pool.page_size < G::KT ? pool.page_size : G::KT;
        if (!pool.mapped) {
            if (!encode_pages(&pool.kmap, pool.k, pool, box) || !encode_pages(&pool.vmap, pool.v, pool, box))
                return cudaErrorInvalidValue;
            pool.mapped = true;
        }
    }
    const dim3 grid(p.runs), block(G::THREADS);
    if (f) {
        shared_layout(p, *f);
        if (!encode_q(&p.qmap, a, p.g, p.tq))
            return cudaErrorInvalidValue;
        e = launch_pdl(attn_tc_kernel<D, true>, grid, block, (size_t)G::TOTAL, s, p, pool.kmap, pool.vmap);
        return e == cudaSuccess ? launch_join<bf16, D>(p, s) : e;
    }
    work_layout(p);
    e = launch_pdl(attn_tc_kernel<D, false>, grid, block, (size_t)G::TOTAL, s, static_cast<const WorkArgs &>(p), pool.kmap, pool.vmap);
    return e == cudaSuccess ? launch_combine<bf16, D>(p, s) : e;
}

} // namespace

size_t attention_tc_workspace_bytes(int d, int hq, int hkv, int total_tokens, bool shared)
{
    const int g = group_heads(hq, hkv, 128), rows = slot_rows(d, g, total_tokens, shared);
    return shared ? shared_bytes(d, hq, hq / g, total_tokens, kSms, rows) : work_bytes(d, kSms, rows);
}

cudaError_t launch_paged_attention_tc(const AttentionArgs &a, const SharedPrefix *f, kv_page_pool &pool, cudaStream_t s)
{
    switch (a.pages.d) {
    case 64:
        return go<64>(a, f, pool, s);
    case 128:
        return go<128>(a, f, pool, s);
    default:
        return go<256>(a, f, pool, s);
    }
}

} // namespace gdn
