// Attention of new tokens over a paged cache in fp32 (sm_103a).
//
// Products run on the tensor cores in tf32 (mma.sync m16n8k8) with both
// operands split in a head and a tail, x = hi + lo, and three products hi hi +
// hi lo + lo hi: what is dropped is about 2^-22 of a term, as much as an fp32
// product's own rounding.  One tf32 product (2^-11) would not do, and tcgen05
// takes its operands from shared memory, where every head and tail would have
// to be written first.  Sums, weights and statistics are fp32.
//
// Rows (token, head) are packed as in the bf16 kernel, 16 WR a tile; 8 warps
// stand as WR row blocks of 16 x WK shares of a tile's keys.  Few rows (decode,
// verification) take WR small and split the keys instead.  Each warp keeps its
// own O, m and l; shares are joined through shared memory at the item's end.  K
// and V tiles come by 16-byte asynchronous copies, three or four tiles ahead.
//
// Bound: issue slots and the products together.  Of 13 rows of 1 to 250 tokens
// over up to 2.1 k (12 heads over 4 of 64), 145 us, the products' own time is
// 64 at 301 TFLOP/s (packed fp32 FMAs would take 81), and splitting operands
// takes as many slots.  Decode of 48 rows of 3,000 keys takes 84, 163 and 260 us
// at d = 64, 128 and 256: 3.5, 3.6 and 2.3 TB/s.
//
// A weight of zero does not hide a NaN or an infinity, infinity has no tail,
// and rounding to a head takes the largest finite values out of the range.  So
// an item whose sums come out finite is done; otherwise a second pass takes the
// elements of V that are not finite as zero, and the item's end adds them to
// the rows that see them; it also splits with care for the range, so that an
// infinite score is one.  (Looking at every tile as it lands cost decode up to
// 11 %.)
#include "attn_plan.cuh"

#include <atomic>
#include <type_traits>

#include "gdn_ptx.cuh"
#include "tf32_ops.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <int D> struct Geo32 {
    static constexpr int KT = D == 256 ? 16 : 32;  // keys a tile
    static constexpr int LD = D + 4;               // row stride: fragment reads hit 32 banks
    static constexpr int WRB = D == 256 ? 4 : 8;   // row blocks with many rows: 8 / WRB shares of a tile,
    static constexpr int WRS = D == 256 ? 2 : 1;   // and with up to 16 WRS rows: 8 / WRS shares of two tiles
    static constexpr int M = 16 * WRB;
    // Row blocks with more than few rows: up to 32 rows two, with four shares of the keys (a CTA's tile takes 2.0 us
    // instead of 3.0 at d = 64 and of 3.6 at d = 128); up to 64 four at d = 128 (3.0 us; at d = 64, where two CTAs share an
    // SM, it makes no difference).
    static __device__ __forceinline__ int blocks(int rows)
    {
        return D == 256 ? WRB : rows <= 32 ? 2 : D == 128 && rows <= 64 ? 4 : WRB;
    }
    static constexpr int TILE = KT * LD;           // floats of a K or V tile
    static constexpr int ROOM = D == 64 ? 28600 : 57600; // floats: half or all of an SM's shared memory
    static constexpr int STAGES = 4;               // tiles of K and V in shared memory: about 100 KB an SM under way
    static constexpr int FEW = 16 * WRS;           // rows that count as few: less room for Q, more for tiles
    static constexpr int STAGES_FEW = D == 256 ? 5 : 6;
    static constexpr int FLOATS0 = M * LD + 2 * STAGES * TILE, FLOATS1 = FEW * LD + 2 * STAGES_FEW * TILE;
    static constexpr int FLOATS = FLOATS0 > FLOATS1 ? FLOATS0 : FLOATS1;
    static_assert(FLOATS <= ROOM, "shared memory");
    static constexpr int PER_SM = D == 64 ? 2 : 1; // CTAs an SM, by shared memory
};

// Units of a tile, by its time.  (Measured, us of a CTA: up to 16, 32, 64 and 128 rows 1.13, 2.0, 3.1 and 5.3 at d = 64
// and 1.19, 2.0, 3.0 and 5.3 at d = 128; up to 32 and 64 rows 2.0 and 3.7 at d = 256.)
template <int D> struct Cost32 {
    static constexpr int least = 4, most = D == 256 ? 7 : 18, item = 0;
    static __device__ __forceinline__ int of(int rows)
    {
        return rows <= 16 * Geo32<D>::WRS ? least : D == 256 ? most : rows <= 32 ? 7 : rows <= 64 ? 11 : most;
    }
};

// With shared prefixes items are many and short: their begins and ends count (2 to 3 us).  32 rows x 4 tokens behind 300 to
// 2,000 shared ones take 30.1 us, with 14 units 32.9 (and 64 rows behind 8,000 75.4 and 72.5).
template <int D> struct SharedCost32 : Cost32<D> {
    static constexpr int item = 10;
};

template <typename V> struct Ctrl32 {
    long long scan[kThreads / 32];
    FoundOf<V> found;
    typename V::ItemT item;
    int more, broken, dirty;
    float2 ml[8 * 16]; // (m, l) by (share, row): 128 pairs in every form
};

template <int N> struct Width {
    static constexpr int value = N;
};
__device__ __forceinline__ bool odd(uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; } // not finite
// The second pass's: a head that rounding up would take out of the range (from 3.402e38 on) is cut short instead, and a
// value that is not finite has no tail; `fine` is the head, or zero in place of such a value.
__device__ __forceinline__ void split_any(float x, uint32_t &hi, uint32_t &lo, uint32_t &fine)
{
    split(x, hi, lo);
    if (odd(hi)) {
        hi = __float_as_uint(x) & 0xffffe000u;
        lo = __float_as_uint(x - __uint_as_float(hi));
    }
    fine = hi;
    if (odd(__float_as_uint(x)))
        hi = isnan(x) ? 0x7fffffffu : __float_as_uint(x), lo = fine = 0;
}
__device__ __forceinline__ void copy16(float *dst, const float *src, bool there) // zeros where it is not there
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

// One warp's keys kb .. kb + 8 NT of a tile, rows g and g + 8 of its block
// (g = lane / 4, c = lane % 4).  Fragments: A (row g, k c), (g + 8, c), (g, c +
// 4), (g + 8, c + 4); B (k c, n g), (c + 4, g); D (g, 2c), (g, 2c + 1), (g + 8,
// 2c), (g + 8, 2c + 1).  P V names key 2c as its k = c and key 2c + 1 as k = c +
// 4, so the weights are an A fragment as they stand.  ANY: the operands may be
// at the top of the range, and Q and K beyond it; then the products with tails
// take the other side's finite heads, as infinity times a tail of zero or of
// the other sign would be NaN.
template <int D, int NT, bool ANY>
__device__ __forceinline__ void tile_step(const float *q, const float *k, const float *v, int see0, int see8, float c2,
                                          float (&o)[D / 8][4], float &m0, float &m8, float &l0, float &l8)
{
    constexpr int LD = Geo32<D>::LD;
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    // The tensor cores cut their sums short instead of rounding them, which showed (5e-6 of a result's norm) in the sums
    // over a head's dimensions and over all keys.  So they only sum four steps of eight dimensions, or a tile's keys, and
    // the rest is fp32 additions.  A single column tile takes the four steps apart, for latency.
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[n][e] = 0.f;
#pragma unroll 2
    for (int k0 = 0; k0 < D / 8; k0 += 4) {
        constexpr int APART = NT == 1 ? 4 : 1;
        float t[NT][APART][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < APART; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    t[n][h][e] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            const float *qp = q + g * LD + 8 * (k0 + ks) + c;
            uint32_t ah[4], al[4], af[4];
            const float qv[4] = {qp[0], qp[8 * LD], qp[4], qp[8 * LD + 4]};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if constexpr (ANY)
                    split_any(qv[e], ah[e], al[e], af[e]);
                else
                    split(qv[e], ah[e], al[e]), af[e] = ah[e];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float *kp = k + (8 * n + g) * LD + 8 * (k0 + ks) + c;
                uint32_t h0, h1, t0, t1, fine0, fine1;
                if constexpr (ANY)
                    split_any(kp[0], h0, t0, fine0), split_any(kp[4], h1, t1, fine1);
                else
                    split2(kp[0], kp[4], h0, t0, h1, t1), fine0 = h0, fine1 = h1;
                float(&d)[4] = t[n][ks % APART];
                mma8(d, al, fine0, fine1);
                mma8(d, af, t0, t1);
                mma8(d, ah, h0, h1);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[n][e] += APART == 4 ? (t[n][0][e] + t[n][1 % APART][e]) + (t[n][2 % APART][e] + t[n][3 % APART][e]) : t[n][0][e];
    }
    // weights 2^(c2 (s - m))
    float top0 = m0, top8 = m8;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int at = 8 * n + 2 * c + e;
            s[n][e] = at < see0 ? s[n][e] : -INFINITY;
            s[n][e + 2] = at < see8 ? s[n][e + 2] : -INFINITY;
            top0 = fmaxf(top0, s[n][e]);
            top8 = fmaxf(top8, s[n][e + 2]);
        }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, x));
        top8 = fmaxf(top8, __shfl_xor_sync(0xffffffffu, top8, x));
    }
    const float z0 = top0 == -INFINITY ? 0.f : -top0 * c2, z8 = top8 == -INFINITY ? 0.f : -top8 * c2;
    // (exactly one where the maximum stays: a factor of 1 + 10^-7 a tile adds up)
    const float f0 = m0 == -INFINITY ? 0.f : ex2((m0 - top0) * c2), f8 = m8 == -INFINITY ? 0.f : ex2((m8 - top8) * c2);
    m0 = top0, m8 = top8;
    l0 *= f0, l8 *= f8;
    uint32_t ah[NT][4], al[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const float p0 = ex2(fmaf(s[n][0], c2, z0)), p1 = ex2(fmaf(s[n][1], c2, z0));
        const float p2 = ex2(fmaf(s[n][2], c2, z8)), p3 = ex2(fmaf(s[n][3], c2, z8));
        l0 += p0 + p1, l8 += p2 + p3;
        split(p0, ah[n][0], al[n][0]);
        split(p2, ah[n][1], al[n][1]);
        split(p1, ah[n][2], al[n][2]);
        split(p3, ah[n][3], al[n][3]);
    }
    const float *vp = v + 2 * c * LD + g;
#pragma unroll
    for (int e = 0; e < D / 8; ++e) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t h0, h1, t0, t1, fine0, fine1;
            const float v0 = vp[8 * n * LD + 8 * e], v1 = vp[8 * n * LD + 8 * e + LD];
            if constexpr (ANY) // V's values are finite here
                split_any(v0, h0, t0, fine0), split_any(v1, h1, t1, fine1);
            else
                split2(v0, v1, h0, t0, h1, t1);
            mma8(d, al[n], h0, h1);
            mma8(d, ah[n], t0, t1);
            mma8(d, ah[n], h0, h1);
        }
        o[e][0] = fmaf(o[e][0], f0, d[0]), o[e][1] = fmaf(o[e][1], f0, d[1]);
        o[e][2] = fmaf(o[e][2], f8, d[2]), o[e][3] = fmaf(o[e][3], f8, d[3]);
    }
}

template <int D, bool SH>
__global__ void __launch_bounds__(kThreads, Geo32<D>::PER_SM) attn_f32_kernel(const typename Kind<SH>::Args p)
{
    typedef Geo32<D> G;
    typedef typename std::conditional<SH, Shared, Plain>::type View;
    typedef typename Kind<SH>::ItemT ItemT;
    typedef typename std::conditional<SH, SharedCost32<D>, Cost32<D>>::type Cost;
    typedef Walk<Cost, View, typename Kind<SH>::Args> WalkT;
    constexpr int KT = G::KT, LD = G::LD;
    extern __shared__ __align__(16) float sm[];
    __shared__ Ctrl32<View> ctl;
    float *const Q = sm;
    const AttentionArgs &a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int ps = a.pages.page_size, hkv = a.pages.hkv;
    const float c2 = a.scale * 1.44269504088896341f;
    wait_prior_grid();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const RunOf<View> run = plan_run<kThreads, KT, Cost, View>(p, p.tq, ctl.scan, ctl.found);
    zero_dead<float, D, kThreads, View>(p, tid);
    WalkT walk(p, run, p.tq, KT); // warp 0's is followed (another warp's writes the same zero)
    for (;;) {
        __syncthreads();
        if (warp == 0) {
            ItemT next;
            const bool more = walk.next(next);
            if (lane == 0) {
                ctl.item = next;
                ctl.more = more, ctl.broken = 0x7fffffff, ctl.dirty = 0;
            }
        }
        __syncthreads();
        if (!ctl.more)
            break;
        const ItemT it = ctl.item;
        const int32_t *const table = item_table(a.c, it);
        const int step = see_step(it);
        const int kvh = it.head / p.groups, rows = it.ntok * p.g, end = it.see + (it.ntok - 1) * step;
        const bool few = rows <= G::FEW;
        float *const ring = sm + (few ? G::FEW : G::M) * LD;
        const int wr_n = few ? G::WRS : G::blocks(rows), wk_n = 8 / wr_n, wr = warp % wr_n, wk = warp / wr_n; // row block, share
        // Q: token rows of this head group
        {
            const float *const src = static_cast<const float *>(a.q) + (size_t)it.tok * a.q_stride + (size_t)it.head * p.g * D;
            for (int x = tid; x < 16 * wr_n * (D / 4); x += kThreads) {
                const int row = x / (D / 4), vec = x - row * (D / 4), t = row / p.g;
                const bool there = row < rows;
                copy16(Q + row * LD + 4 * vec, there ? src + (size_t)t * a.q_stride + (row - t * p.g) * D + 4 * vec : src, there);
            }
        }
        const int n = it.jb - it.ja;
        // A group of copies a tile, empty past the last; a thread keeps its column.  Pages are looked up a step
        // before their copies, so that no copy waits for the table.
        constexpr int VR = D / 4 < kThreads ? D / 4 : kThreads, RP = kThreads / VR, NR = KT / RP; // vectors a row, rows a pass
        const int vrow = tid / VR, col = 4 * (tid % VR);
        typedef int Pages[NR];
        auto look = [&](Pages &pages, int j) {
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int key = (it.ja + j) * KT + i * RP + vrow;
                pages[i] = j < n && key < end ? table[key >> a.pages.page_shift] : -1;
            }
        };
        auto load = [&](const Pages &pages, int j, int stage) {
            if (j < n) {
                float *const K = ring + stage * 2 * G::TILE, *const V = K + G::TILE;
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    const int row = i * RP + vrow, key = (it.ja + j) * KT + row;
                    int page = pages[i];
                    if (key < end && (page <= 0 || page >= a.pages.num_pages)) {
                        page = 0;
                        atomicMin(&ctl.broken, key);
                        report(a.err, GDN_DEVERR_BAD_PAGE);
                    }
                    const size_t at = (((size_t)max(page, 0) * hkv + kvh) * ps + (key & (ps - 1))) * D + col;
                    copy16(K + row * LD + col, static_cast<const float *>(a.pages.k) + at, page > 0);
                    copy16(V + row * LD + col, static_cast<const float *>(a.pages.v) + at, page > 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // the elements of V that this thread copied: what is not finite becomes zero
        auto scan = [&](int stage) {
            float *const V = ring + (stage * 2 + 1) * G::TILE;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                uint4 *const at = reinterpret_cast<uint4 *>(V + (i * RP + vrow) * LD + col);
                uint4 v = *at;
                if (odd(v.x) || odd(v.y) || odd(v.z) || odd(v.w)) {
                    v = make_uint4(odd(v.x) ? 0u : v.x, odd(v.y) ? 0u : v.y, odd(v.z) ? 0u : v.z, odd(v.w) ? 0u : v.w);
                    *at = v;
                    ctl.dirty = 1;
                }
            }
        };
        const int r0 = 16 * wr + g, r8 = r0 + 8;
        const int s0 = r0 < rows ? it.see + r0 / p.g * step : 0, s8 = r8 < rows ? it.see + r8 / p.g * step : 0; // keys the rows see
        float o[D / 8][4], m0, m8, l0, l8;
        // this warp's step on tile j, on keys kb .. of it
        auto work = [&](int j, int stage, int kb, auto nt, auto again) {
            const int key = (it.ja + j) * KT + kb;
            const float *const K = ring + stage * 2 * G::TILE + kb * LD;
            tile_step<D, decltype(nt)::value, decltype(again)::value != 0>(Q + 16 * wr * LD, K, K + G::TILE, s0 - key, s8 - key, c2, o, m0, m8, l0, l8);
        };
        auto pass = [&](auto second) { // true where every sum is finite
            constexpr bool again = decltype(second)::value;
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
                o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
            m0 = m8 = -INFINITY, l0 = l8 = 0.f;
            if (few) { // two tiles at a time, 8 keys a warp; SF - 2 tiles ahead
                constexpr int NS = KT / 8, SF = G::STAGES_FEW, A = SF - 2; // shares of a tile
                Pages pages[A];
#pragma unroll
                for (int i = 0; i < A; ++i)
                    look(pages[i], i);
#pragma unroll
                for (int i = 0; i < A; ++i)
                    load(pages[i], i, i);
                look(pages[0], A), look(pages[1], A + 1);
                for (int j = 0; j < n; j += 2) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(A - 2) : "memory");
                    if (again) {
                        scan(j % SF);
                        if (j + 1 < n)
                            scan((j + 1) % SF);
                    }
                    __syncthreads(); // the tiles are there for all, and those before them are done with
                    load(pages[0], j + A, (j + A) % SF);
                    load(pages[1], j + A + 1, (j + A + 1) % SF);
                    look(pages[0], j + A + 2), look(pages[1], j + A + 3);
                    const int mine = j + wk / NS;
                    if (16 * wr < rows && mine < n)
                        work(mine, mine % SF, wk % NS * 8, Width<1>(), second);
                }
            } else {
                constexpr int S = G::STAGES, A = S - 1;
                Pages pages[A];
#pragma unroll
                for (int i = 0; i < A; ++i)
                    look(pages[i], i);
#pragma unroll
                for (int i = 0; i < A; ++i)
                    load(pages[i], i, i);
                look(pages[0], A);
                for (int j = 0; j < n; ++j) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(A - 1) : "memory");
                    if (again)
                        scan(j % S);
                    __syncthreads(); // the tile is there for all, and the one before it is done with
                    load(pages[0], j + A, (j + A) % S);
                    look(pages[0], j + A + 1);
                    const int kb = wk * (KT / wk_n);
                    if (16 * wr >= rows)
                        continue;
                    if (D == 256 || wr_n == 2)
                        work(j, j % S, kb, Width<1>(), second);
                    else if (D == 128 && wr_n == 4)
                        work(j, j % S, kb, Width<2>(), second);
                    else
                        work(j, j % S, kb, Width<KT / 8>(), second);
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            float z = 0.f; // stays zero unless a sum is not finite
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
                z = fmaf(o[e][0], 0.f, fmaf(o[e][1], 0.f, fmaf(o[e][2], 0.f, fmaf(o[e][3], 0.f, z))));
            return __syncthreads_and(again || z == 0.f) != 0;
        };
        if (!pass(Width<0>()))
            pass(Width<1>());
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l8 += __shfl_xor_sync(0xffffffffu, l8, x);
        }
        const float NaN = __int_as_float(0x7fc00000);
        const bool partial = ctl.item.part != -1; // (not from `it`: no register across the tiles)
        if (wk_n == 1 && !ctl.dirty) { // a warp has all of its rows' sums: out of its registers
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = x ? r8 : r0, t = row / p.g;
                const bool bad = (x ? s8 : s0) > ctl.broken;
                const float m = x ? m8 : m0, l = x ? l8 : l0, i = partial ? 1.f : 1.f / l;
                float *const to = partial ? p.part_o + part_row(p, it, it.tok + t, it.head * p.g + (row - t * p.g), row) * D
                                          : static_cast<float *>(a.out) + ((size_t)(it.tok + t) * a.hq + it.head * p.g + (row - t * p.g)) * D;
                if (row < rows) {
                    if (partial && c == 0)
                        p.part_ml[part_row(p, it, it.tok + t, it.head * p.g + (row - t * p.g), row)] = make_float2(bad ? NaN : m, l);
#pragma unroll
                    for (int e = 0; e < D / 8; ++e)
                        *reinterpret_cast<float2 *>(to + 8 * e + 2 * c) = !partial && bad ? make_float2(0.f, 0.f)
                                                                                             : make_float2(o[e][2 * x] * i, o[e][2 * x + 1] * i);
                }
            }
            continue;
        }
        // the shares' sums to shared memory, in place of the tiles
        float *const mine = ring + (size_t)(wk * 16 * wr_n + r0) * LD;
        if (16 * wr < rows) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e) {
                *reinterpret_cast<float2 *>(mine + 8 * e + 2 * c) = make_float2(o[e][0], o[e][1]);
                *reinterpret_cast<float2 *>(mine + 8 * LD + 8 * e + 2 * c) = make_float2(o[e][2], o[e][3]);
            }
            if (c == 0)
                ctl.ml[wk * 16 * wr_n + r0] = make_float2(m0, l0), ctl.ml[wk * 16 * wr_n + r8] = make_float2(m8, l8);
        }
        __syncthreads();
        for (int x = tid; x < rows * (D / 4); x += kThreads) {
            const int row = x / (D / 4), col = 4 * (x - row * (D / 4)), t = row / p.g, see = it.see + t * step;
            const bool bad = see > ctl.broken;
            float m = -INFINITY, l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
            for (int w = 0; w < wk_n; ++w)
                m = fmaxf(m, ctl.ml[w * 16 * wr_n + row].x);
            for (int w = 0; w < wk_n; ++w) {
                const float2 s = ctl.ml[w * 16 * wr_n + row];
                const float f = s.x == -INFINITY ? 0.f : ex2((s.x - m) * c2);
                const float4 z = *reinterpret_cast<const float4 *>(ring + (size_t)(w * 16 * wr_n + row) * LD + col);
                l = fmaf(s.y, f, l);
                y[0] = fmaf(z.x, f, y[0]), y[1] = fmaf(z.y, f, y[1]), y[2] = fmaf(z.z, f, y[2]), y[3] = fmaf(z.w, f, y[3]);
            }
            if (ctl.dirty && !bad) {
                for (int key = it.ja * KT; key < min(see, it.jb * KT); ++key) {
                    const float *const v = static_cast<const float *>(a.pages.v) +
                                           (((size_t)table[key >> a.pages.page_shift] * hkv + kvh) * ps + (key & (ps - 1))) * D + col;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (!isfinite(v[e]))
                            y[e] += v[e];
                }
            }
            if (partial) {
                const size_t prow = part_row(p, it, it.tok + t, it.head * p.g + (row - t * p.g), row);
                *reinterpret_cast<float4 *>(p.part_o + prow * D + col) = make_float4(y[0], y[1], y[2], y[3]);
                if (col == 0)
                    p.part_ml[prow] = make_float2(bad ? NaN : m, l);
            } else {
                const float i = 1.f / l;
                float *const out = static_cast<float *>(a.out) + ((size_t)(it.tok + t) * a.hq + it.head * p.g + (row - t * p.g)) * D + col;
                *reinterpret_cast<float4 *>(out) =
                    bad ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(y[0] * i, y[1] * i, y[2] * i, y[3] * i);
            }
        }
    }
}

int slot_rows32(int m, int g, int total_tokens)
{
    const int tq = m / g;
    return (total_tokens < tq ? total_tokens : tq) * g;
}

// The kernel's shared memory, once a device.
template <int D, bool SH> cudaError_t configure()
{
    static_assert(Geo32<D>::FLOATS * 4 + sizeof(Ctrl32<Shared>) <= 232448, "shared memory");
    static std::atomic<unsigned long long> configured{0}; // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(configured.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(attn_f32_kernel<D, SH>, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo32<D>::FLOATS * 4);
        if (e != cudaSuccess)
            return e;
        configured.fetch_or(bit, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int D> cudaError_t go(const AttentionArgs &a, const SharedPrefix *f, cudaStream_t s)
{
    typedef Geo32<D> G;
    cudaError_t e = f ? configure<D, true>() : configure<D, false>();
    if (e != cudaSuccess)
        return e;
    SharedArgs p;
    p.a = a;
    p.g = group_heads(a.hq, a.pages.hkv, G::M);
    p.groups = a.hq / a.pages.hkv / p.g;
    p.tq = G::M / p.g;
    p.runs = kSms * G::PER_SM;
    p.rows_max = slot_rows32(G::M, p.g, a.c.total_tokens);
    p.second = 0;
    const dim3 grid(p.runs), block(kThreads);
    if (f) {
        shared_layout(p, *f);
        e = launch_pdl(attn_f32_kernel<D, true>, grid, block, (size_t)G::FLOATS * 4, s, p);
        return e == cudaSuccess ? launch_join<float, D>(p, s) : e;
    }
    work_layout(p);
    e = launch_pdl(attn_f32_kernel<D, false>, grid, block, (size_t)G::FLOATS * 4, s, static_cast<const WorkArgs &>(p));
    return e == cudaSuccess ? launch_combine<float, D>(p, s) : e;
}

} // namespace

size_t attention_f32_workspace_bytes(int d, int hq, int hkv, int total_tokens, bool shared)
{
    const int m = d == 256 ? Geo32<256>::M : Geo32<128>::M; // 64 as 128
    const int g = group_heads(hq, hkv, m), rows = slot_rows32(m, g, total_tokens), runs = kSms * (d == 64 ? Geo32<64>::PER_SM : 1);
    return shared ? shared_bytes(d, hq, hq / g, total_tokens, runs, rows) : work_bytes(d, runs, rows);
}

cudaError_t launch_paged_attention_f32(const AttentionArgs &a, const SharedPrefix *f, cudaStream_t s)
{
    switch (a.pages.d) {
    case 64:
        return go<64>(a, f, s);
    case 128:
        return go<128>(a, f, s);
    default:
        return go<256>(a, f, s);
    }
}

} // namespace gdn
