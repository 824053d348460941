// How the attention kernels over a paged cache divide their work (sm_103a),
// and how the parts of a divided item are joined.
//
// An item is one key head (or a share of its query heads, where it has more
// than a tile holds) and up to `mt` consecutive new tokens of a cache row; its
// keys come in tiles of KT.  All items' key tiles, in order, are cut into runs
// of equal cost, one a CTA: every CTA finds its run from the lengths on the
// device.  Costs are in units, a tile's given by its item's rows.
// Included by one translation unit a kernel; everything here has internal
// linkage.
#pragma once

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kSms = 152;

struct Item {
    int tok, ntok, head, row; // first token, tokens, head group, cache row
    int see;                  // keys the first token sees; one more each token on
    int ja, jb;               // key tiles of this run
    int part;                 // workspace slot of a cut item, or -1
};

// Attention over shared prefixes (see Shared below) has two kinds of items:
// the shared keys of a group of rows, for all their tokens, and a row's own
// keys behind them.
struct SharedItem : Item {
    int skip; // pages of the row's table before the item's keys
    int step; // 1, or 0 where every token sees all keys (shared ones)
    int kind; // 1: shared keys
};
constexpr int kDense = -2; // SharedItem::part: the item's first part, at its tokens' place

// One cut item, for the combining kernel: written by the run that holds the
// item's second part.
struct Cut {
    int parts, tok, ntok, head;
};

// Units of a key tile of an item with `rows` rows: kernels whose tiles cost the
// same whatever the rows, and others.  `item` units more are for an item to
// begin and end, where items of few tiles are many; its first tile counts them.
struct EvenCost {
    static constexpr int least = 1, most = 1, item = 0;
    static __device__ __forceinline__ int of(int) { return 1; }
};

// A call's arguments with its division.  Query heads are taken g at a time
// (head groups of one key head); a tile holds tq tokens of a group.
struct WorkArgs {
    AttentionArgs a;
    int g, groups, tq; // heads a group, groups a key head, tokens a tile
    int runs;          // CTAs
    int rows_max;      // rows of a workspace slot
    int second;        // rows before an item's second tile (0: items have one tile)
    float *part_o;     // [2 runs][rows_max][D]
    float2 *part_ml;
    Cut *cuts;         // [runs]
};

// The same with groups of rows that share their first pages.
//   part_o, part_ml: [2 kinds][tokens][hq], every item's first part (the one
//                    with its first key) at its tokens' and heads' place, then
//                    [runs][rows_max], the part of an item that began before
//                    the run
struct SharedArgs : WorkArgs {
    const int32_t *bounds; // [ngroups + 1] rows of the groups
    const int2 *prefix;    // [rows] (row whose pages they are, pages), alike within a group
    int ngroups;
    size_t dense;          // rows of part_o before the runs' slots
    int4 *rec;             // [2 kinds][tokens][head groups]: first token of the item, its first run, further runs (-1: a dead
                           // token), whether shared keys go with them
    CUtensorMap qmap;      // bf16: Q
};
template <bool SH> struct Kind {
    typedef Item ItemT;
    typedef WorkArgs Args;
};
template <> struct Kind<true> {
    typedef SharedItem ItemT;
    typedef SharedArgs Args;
};

// Tokens an item at most, of kernels whose items have up to `tiles` tiles.
__device__ __forceinline__ int item_tokens(const WorkArgs &p, int tiles) { return p.tq * tiles; }
__device__ __forceinline__ int item_tokens(const SharedArgs &p, int) { return p.second ? 2 * p.tq : p.tq; }

// The workspace: cuts, then (m, l) and O of the cut items' parts.
inline size_t work_bytes(int d, int runs, int rows_max)
{
    return sizeof(Cut) * runs + 2 * (size_t)runs * rows_max * (sizeof(float2) + sizeof(float) * d);
}
inline void work_layout(WorkArgs &p)
{
    p.cuts = static_cast<Cut *>(p.a.work);
    p.part_ml = reinterpret_cast<float2 *>(p.cuts + p.runs);
    p.part_o = reinterpret_cast<float *>(p.part_ml + 2 * (size_t)p.runs * p.rows_max);
}
// Heads a group: the largest divisor of hq / hkv that a tile of `rows` rows holds.
inline int group_heads(int hq, int hkv, int rows)
{
    const int all = hq / hkv;
    int g = all < rows ? all : rows;
    while (all % g)
        --g;
    return g;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A cache row's work: its tokens [b, b + n) and length, live when it is a real
// row whose table can hold it.
struct Row {
    int b, n, len;
    bool live, bad;
};
__device__ __forceinline__ Row row_of(const CacheRows &c, int page_size, int r)
{
    Row x;
    x.b = c.cu_seqlens[r];
    const int e = c.cu_seqlens[r + 1];
    x.len = c.seq_len[r];
    x.n = 0;
    x.live = x.bad = false;
    if (x.b < 0 || e < x.b || e > c.total_tokens) {
        x.bad = true;
    } else {
        x.n = e - x.b;
        x.bad = x.n > 0 && (x.len < 0 || (x.len > 0 && (x.len < x.n || x.len > c.max_pages * page_size)));
        x.live = x.n > 0 && x.len > 0 && !x.bad;
    }
    return x;
}

// The rows that the plan divides: a call's rows, or with shared prefixes first
// the groups (their tokens over the shared keys, which all of them see), then
// the rows (over their own keys).
struct SharedRow : Row {
    int row, skip, step, kind; // as in SharedItem
};
struct Plain {
    typedef Row RowT;
    typedef Item ItemT;
    static __device__ __forceinline__ int count(const WorkArgs &p) { return p.a.c.rows; }
    static __device__ __forceinline__ Row get(const WorkArgs &p, int r) { return row_of(p.a.c, p.a.pages.page_size, r); }
    static __device__ __forceinline__ int step(const Row &) { return 1; }
};
struct Shared {
    typedef SharedRow RowT;
    typedef SharedItem ItemT;
    static __device__ __forceinline__ int count(const SharedArgs &p) { return p.ngroups + p.a.c.rows; }
    static __device__ __forceinline__ int step(const SharedRow &x) { return x.step; }
    static __device__ SharedRow get(const SharedArgs &p, int i)
    {
        const CacheRows &c = p.a.c;
        const int ps = p.a.pages.page_size;
        SharedRow x = {};
        if (i < p.ngroups) {
            const int r0 = p.bounds[i], r1 = p.bounds[i + 1];
            x.bad = (i == 0 && r0 != 0) || (i == p.ngroups - 1 && r1 != c.rows); // (rows of no group, which does not concern this one)
            if (r0 < 0 || r1 < r0 || r1 > c.rows)
                x.bad = true;
            else if (r0 < r1) {
                const int2 f = p.prefix[r0];
                const int b = c.cu_seqlens[r0], e = c.cu_seqlens[r1];
                if (f.y != 0) {
                    const bool wrong = f.x < 0 || f.x >= c.rows || f.y < 0 || f.y > c.max_pages || b < 0 || e < b || e > c.total_tokens;
                    x.bad |= wrong;
                    x.live = !wrong && e > b;
                    if (x.live)
                        x.b = b, x.n = e - b, x.len = f.y * ps, x.row = f.x, x.kind = 1;
                }
            }
            return x;
        }
        const int r = i - p.ngroups, pages = p.prefix[r].y;
        static_cast<Row &>(x) = row_of(c, ps, r);
        x.row = r, x.step = 1;
        if (x.live) { // its own keys begin behind the shared pages, which lie before its new tokens
            x.bad = pages < 0 || pages > c.max_pages || (long long)pages * ps > x.len - x.n;
            x.live = !x.bad;
            if (x.live)
                x.skip = pages, x.len -= pages * ps;
        }
        return x;
    }
};

// Key tiles of the row's item t (mt tokens an item).
template <typename V> __device__ __forceinline__ int item_tiles(const typename V::RowT &x, int t, int mt, int kt)
{
    const int last = min(x.n, (t + 1) * mt);
    return (x.len - (x.n - last) * V::step(x) + kt - 1) / kt;
}
__device__ __forceinline__ int items_of(const Row &x, int mt) { return (x.n + mt - 1) / mt; }
template <typename Cost, typename V>
__device__ long long head_units(const typename V::RowT &x, int mt, int kt, int g) // of one key head
{
    long long s = 0;
    const int n = items_of(x, mt);
    for (int t = 0; t < n; ++t)
        s += item_tiles<V>(x, t, mt, kt) * (long long)Cost::of(min(mt, x.n - t * mt) * g);
    return s;
}

// Exclusive sum over the CTA's threads; `part` is one long long a warp, and one.
__device__ __forceinline__ long long scan64(long long v, long long *part, int warps, long long &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += x;
    }
    if (lane == 31)
        part[warp] = s;
    __syncthreads();
    long long before = s - v;
    total = 0;
    for (int w = 0; w < warps; ++w) {
        const long long x = part[w];
        if (w < warp)
            before += x;
        total += x;
    }
    __syncthreads();
    return before;
}

// This CTA's run of the units 0 .. total, the tiles that begin in [u0, u1): u0
// lies in `row`, whose units begin at `base`.  A run is no shorter than a tile,
// so that every run between an item's first and last has a part of it.  Called
// by the whole CTA; `part` is a long long a warp, and `found` the place where
// one thread leaves the row.
template <typename V> struct RunOf {
    long long share, u0, u1, base;
    long long per;           // units a head of the row it begins in
    int row;
    int item;                // units of an item besides its tiles'
    typename V::RowT first;  // that row
};
template <typename V> struct FoundOf { // shared memory
    long long base, per;
    int row;
    typename V::RowT first;
};
template <int THREADS, int KT, typename Cost, typename V, typename Args>
__device__ RunOf<V> plan_run(const Args &p, int mt, long long *part, FoundOf<V> &found)
{
    const int count = V::count(p), heads = p.a.pages.hkv * p.groups, tid = threadIdx.x;
    typename V::RowT x = {};
    long long per = 0, items = 0; // units of the tiles of a key head of this thread's row, and its items
    long long cost = 0;
    auto look = [&](int r) {
        per = items = cost = 0;
        if (r >= count)
            return;
        x = V::get(p, r);
        if (x.live) {
            per = head_units<Cost, V>(x, mt, KT, p.g);
            cost = per * heads;
            if (Cost::item)
                items = items_of(x, mt);
        }
    };
    int dearest = 1; // tile of this thread's rows
    RunOf<V> run;
    long long total = 0, begun = 0, before = 0, sum, n0 = 0, n;
    for (int b = 0; b < count; b += THREADS) {
        look(b + tid);
        if (cost > 0)
            dearest = max(dearest, Cost::of(min(x.n, mt) * p.g));
        if (x.bad && blockIdx.x == 0)
            report(p.a.err, GDN_DEVERR_BAD_PAGE);
        before = scan64(cost, part, THREADS / 32, sum);
        total += sum;
        if (Cost::item) {
            n0 = scan64(items * heads, part, THREADS / 32, n);
            begun += n;
        }
    }
    // (Cost's values are few, and one barrier tells whether a thread has seen more than the least)
    const int least = Cost::least, tile = Cost::most == least ? least : __syncthreads_or(dearest > least) ? Cost::most : least;
    // A run is no shorter than an item's first tile, with what the item takes besides.  Where there is less work than that
    // for every run, it is better spread than weighed.
    run.item = Cost::item && total + Cost::item * begun >= (long long)(tile + Cost::item) * gridDim.x ? Cost::item : 0;
    total += run.item * begun;
    run.share = (total + gridDim.x - 1) / gridDim.x;
    if (run.share < tile + run.item)
        run.share = tile + run.item;
    run.u0 = run.share * blockIdx.x;
    run.u1 = min(total, run.u0 + run.share);
    auto weigh = [&] {
        if constexpr (Cost::item != 0) {
            per += run.item * items;
            cost = per * heads;
        }
    };
    if (count <= THREADS) { // the one pass has it
        weigh();
        before += run.item * n0;
        if (cost > 0 && before <= run.u0 && run.u0 < before + cost)
            found = {before, per, tid, x};
    } else {
        long long seen = 0;
        for (int b = 0; b < count && seen <= run.u0 && run.u0 < total; b += THREADS) {
            look(b + tid);
            weigh();
            before = seen + scan64(cost, part, THREADS / 32, sum);
            if (cost > 0 && before <= run.u0 && run.u0 < before + cost)
                found = {before, per, b + tid, x};
            seen += sum;
        }
    }
    __syncthreads();
    run.row = found.row;
    run.base = found.base;
    run.per = found.per;
    run.first = found.first;
    return run;
}

// Zeros for the outputs of tokens that no live row has, by THREADS threads (tid)
// of all CTAs together.
template <typename T, int D, int THREADS, typename V, typename Args> __device__ void zero_dead(const Args &p, int tid)
{
    constexpr bool SH = sizeof(Args) != sizeof(WorkArgs);
    const CacheRows &c = p.a.c;
    const size_t vecs = (size_t)p.a.hq * D * sizeof(T) / 16; // a token's
    uint4 *const out = static_cast<uint4 *>(p.a.out);
    auto zero = [&](int t0, int t1) {
        for (size_t i = (size_t)t0 * vecs + tid; i < (size_t)t1 * vecs; i += THREADS)
            out[i] = make_uint4(0, 0, 0, 0);
        if constexpr (SH) { // nothing to be joined
            const size_t heads = (size_t)p.a.pages.hkv * p.groups;
            for (size_t i = t0 * heads + tid; i < t1 * heads; i += THREADS)
                p.rec[i] = make_int4(0, 0, -1, 0);
        }
    };
    for (int r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const auto x = V::get(p, V::count(p) - c.rows + r);
        if (!x.live && x.n > 0)
            zero(x.b, x.b + x.n);
    }
    if (blockIdx.x == 0) {
        const int first = c.cu_seqlens[0], last = c.cu_seqlens[c.rows];
        if (first > 0)
            zero(0, min(first, c.total_tokens));
        if (last >= 0 && last < c.total_tokens)
            zero(last, c.total_tokens);
        if (tid == 0 && (first != 0 || last != c.total_tokens))
            report(p.a.err, GDN_DEVERR_BAD_PAGE);
    }
}

// The items of a run, in order, by one warp.
template <typename Cost, typename V, typename Args> struct Walk {
    typedef typename V::RowT RowT;
    typedef typename V::ItemT ItemT;
    const Args &p;
    const RunOf<V> &run;
    int mt, kt, heads, lane;
    long long u;     // where the next tile begins
    int r, win;      // row; rows win .. win + 31 are in the lanes
    RowT mine, x;    // a lane's row; the current one
    int items, h, t, ja;
    bool in_row;

    __device__ Walk(const Args &p_, const RunOf<V> &run_, int mt_, int kt_)
        : p(p_), run(run_), mt(mt_), kt(kt_), heads(p_.a.pages.hkv * p_.groups), lane(threadIdx.x & 31), u(run_.u0),
          r(run_.row), win(run_.row), in_row(false)
    {
        if constexpr (!SH) {
            if (lane == 0)
                p.cuts[blockIdx.x].parts = 0;
            __syncwarp();
        }
        fetch(); // the next rows' lengths, while the first row's items are handed out
        if (u < run.u1) {
            enter(run.first);
            long long rem = u - run.base; // the run begins inside this row
            for (; rem >= run.per; ++h)
                rem -= run.per;
            for (;; ++t) {
                const long long units = extra() + item_tiles<V>(x, t, mt, kt) * (long long)unit();
                if (rem < units)
                    break;
                rem -= units;
            }
            // a tile that began before u0 is the run's before
            if constexpr (Cost::item == 0) {
                ja = (int)((rem + unit() - 1) / unit());
                u += (long long)ja * unit() - rem;
            } else {
                ja = tile_from(rem, unit());
                u += tile_begin(ja, unit()) - rem;
            }
            if (ja == item_tiles<V>(x, t, mt, kt))
                done();
        }
    }
    static constexpr bool SH = sizeof(Args) != sizeof(WorkArgs);
    __device__ int extra() const { return Cost::item ? run.item : 0; }
    // Where tile j of an item begins, in units from the item's begin, and the first tile to begin at `at` or later.
    __device__ long long tile_begin(int j, int w) const { return j == 0 ? 0 : extra() + (long long)j * w; }
    __device__ int tile_from(long long at, int w) const
    {
        const int j = (int)((at - extra() + w - 1) / w);
        return at <= 0 ? 0 : max(1, j);
    }
    __device__ int unit() const { return Cost::of(min(mt, x.n - t * mt) * p.g); }
    __device__ void done() // with item t
    {
        ja = 0;
        if (++t == items) {
            t = 0;
            if (++h == heads)
                in_row = false, ++r;
        }
    }
    __device__ void enter(const RowT &row)
    {
        x = row;
        in_row = true;
        items = items_of(x, mt);
        h = t = ja = 0;
    }
    __device__ void fetch()
    {
        win = r;
        mine = RowT{};
        if (u < run.u1 && win + lane < V::count(p))
            mine = V::get(p, win + lane);
    }
    // The next item; false at the run's end.  Lane 0 lists a cut.
    __device__ bool next(ItemT &it)
    {
        if (u >= run.u1)
            return false;
        while (!in_row) {
            if (r >= win + 32)
                fetch();
            x.b = __shfl_sync(0xffffffffu, mine.b, r - win);
            x.n = __shfl_sync(0xffffffffu, mine.n, r - win);
            x.len = __shfl_sync(0xffffffffu, mine.len, r - win);
            x.live = true, x.bad = false;
            if constexpr (SH) {
                x.row = __shfl_sync(0xffffffffu, mine.row, r - win);
                x.skip = __shfl_sync(0xffffffffu, mine.skip, r - win);
                x.step = __shfl_sync(0xffffffffu, mine.step, r - win);
                x.kind = __shfl_sync(0xffffffffu, mine.kind, r - win);
            }
            if (!__shfl_sync(0xffffffffu, (int)mine.live, r - win)) {
                if (++r >= V::count(p))
                    return false;
                continue;
            }
            enter(x);
        }
        const int J = item_tiles<V>(x, t, mt, kt);
        const int w = unit();
        const long long start = u - tile_begin(ja, w);
        const int jb = Cost::item == 0 ? (int)min((long long)J, ja + (run.u1 - u + w - 1) / w) : min(J, tile_from(run.u1 - start, w));
        const int t0 = t * mt, ntok = min(mt, x.n - t0);
        const bool cut = ja > 0 || jb < J;
        if constexpr (SH) {
            static_cast<Item &>(it) = {x.b + t0, ntok, h, x.row, x.len - (x.n - t0 - 1) * x.step, ja, jb,
                                       ja > 0 ? (int)blockIdx.x : cut || x.kind || x.skip > 0 ? kDense : -1};
            it.skip = x.skip, it.step = x.step, it.kind = x.kind;
            if (ja == 0) { // the item's first part says where the others are
                const int more = (int)((start + tile_begin(J - 1, w)) / run.share) - (int)blockIdx.x;
                for (int i = lane; i < ntok; i += 32)
                    p.rec[((size_t)x.kind * p.a.c.total_tokens + x.b + t0 + i) * heads + h] =
                        make_int4(x.b + t0, (int)blockIdx.x, more, x.skip > 0);
            }
        } else {
            it = {x.b + t0, ntok, h, r, x.len - x.n + t0 + 1, ja, jb, cut ? 2 * (int)blockIdx.x + (ja > 0 ? 0 : 1) : -1};
            // the run that holds an item's second part lists it for the combining kernel
            if (lane == 0 && ja > 0 && start >= run.u0 - run.share)
                p.cuts[blockIdx.x] = {2 + (int)((start + (J - 1ll) * w) / run.share) - (int)blockIdx.x, x.b + t0, ntok, h};
        }
        if constexpr (Cost::item == 0)
            u += (long long)(jb - ja) * w;
        else
            u = start + tile_begin(jb, w);
        done();
        return true;
    }
};

// Row of part_o and part_ml that a row (token `tok` of all, head `head` of all;
// `row` of the item's tiles) of a partial item writes.
__device__ __forceinline__ size_t part_row(const WorkArgs &p, const Item &it, int, int, int row)
{
    return (size_t)it.part * p.rows_max + row;
}
__device__ __forceinline__ size_t part_row(const SharedArgs &p, const SharedItem &it, int tok, int head, int row)
{
    return it.part == kDense ? ((size_t)it.kind * p.a.c.total_tokens + tok) * p.a.hq + head
                             : p.dense + (size_t)max(it.part, 0) * p.rows_max + row;
}
__device__ __forceinline__ int see_step(const Item &) { return 1; }
__device__ __forceinline__ int see_step(const SharedItem &it) { return it.step; }
__device__ __forceinline__ const int32_t *item_table(const CacheRows &c, const Item &it)
{
    return c.table + (size_t)it.row * c.max_pages;
}
__device__ __forceinline__ const int32_t *item_table(const CacheRows &c, const SharedItem &it)
{
    return c.table + (size_t)it.row * c.max_pages + it.skip;
}

// Joins the parts of R rows of the cut that run w listed, by one warp.
template <typename T, int D, int R> __device__ __forceinline__ void combine_rows(const WorkArgs &p, const Cut &c, int w, int row0, int rows)
{
    const int lane = threadIdx.x & 31;
    constexpr int V = D / 32 < 4 ? D / 32 : 4, N = D / (32 * V); // a lane's columns: N runs of V
    const float k2 = p.a.scale * 1.44269504088896341f;
    // the first part lies in run w - 1 (its last item), the others are the first items of runs w ..
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * (w - 1) + 1 : 2 * (w + i - 1)) * p.rows_max; };
    float m[R], l[R], x[R][N][V];
    bool bad[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY, l[r] = 0.f, bad[r] = false;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[r][n][e] = 0.f;
    }
    for (int i0 = 0; i0 < c.parts; i0 += 32) {
        const bool there = i0 + lane < c.parts;
        float2 ml[R];
        float f[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            ml[r] = there && row0 + r < rows ? p.part_ml[slot(i0 + lane) + row0 + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            bad[r] |= __any_sync(0xffffffffu, ml[r].x != ml[r].x);
            float top = fmaxf(m[r], ml[r].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float old = m[r] == -INFINITY ? 0.f : ex2((m[r] - top) * k2); // of what the parts before gave
            f[r] = ml[r].x == -INFINITY ? 0.f : ex2((ml[r].x - top) * k2);
            m[r] = top;
            float sum = ml[r].y * f[r];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[r] = fmaf(l[r], old, sum);
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[r][n][e] *= old;
        }
        const int here = min(32, c.parts - i0);
        constexpr int U = R == 1 ? (N == 1 ? 8 : 4) : 2;
#pragma unroll U
        for (int i = 0; i < here; ++i) {
            float y[R][N][V];
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (row0 + r < rows) {
                    const float *const o = p.part_o + (slot(i0 + i) + row0 + r) * D + V * lane;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        if constexpr (V == 4)
                            *reinterpret_cast<float4 *>(y[r][n]) = *reinterpret_cast<const float4 *>(o + 32 * V * n);
                        else
                            *reinterpret_cast<float2 *>(y[r][n]) = *reinterpret_cast<const float2 *>(o + 32 * V * n);
                    }
                }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float fi = __shfl_sync(0xffffffffu, f[r], i);
                if (row0 + r < rows) {
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int e = 0; e < V; ++e) // a part without keys for this row has weight zero, and zeros
                            x[r][n][e] = fmaf(y[r][n][e], fi, x[r][n][e]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r;
        const int tile = p.second && row >= p.second, in = row - tile * p.second, t = in / p.g, tok = t + tile * p.tq;
        if (row >= rows || t >= p.tq || tok >= c.ntok)
            continue;
        T *const out = static_cast<T *>(p.a.out) + ((size_t)(c.tok + tok) * p.a.hq + c.head * p.g + (in - t * p.g)) * D + V * lane;
        const float inv = 1.f / l[r];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < V; ++e)
                out[32 * V * n + e] = from_f<T>(bad[r] ? 0.f : x[r][n][e] * inv);
    }
}

// Joins the parts of cut items: block x holds the cut listed by run x.  Bound:
// the latency of three loads in a row (the cut, a part's (m, l) a lane, the
// parts' O), so much is in flight together: a row a warp and eight parts' loads
// where the blocks have a warp for every row, else four rows a warp.
template <typename T, int D> __global__ void __launch_bounds__(128) attn_combine_kernel(const WorkArgs p)
{
    wait_prior_grid();
    const Cut c = p.cuts[blockIdx.x];
    if (c.parts == 0)
        return;
    const int rows = c.ntok > p.tq ? p.second + (c.ntok - p.tq) * p.g : c.ntok * p.g;
    const int w = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (rows <= 4 * (int)gridDim.y) {
        if (w < rows)
            combine_rows<T, D, 1>(p, c, blockIdx.x, w, rows);
    } else if (4 * w < rows) {
        combine_rows<T, D, 4>(p, c, blockIdx.x, 4 * w, rows);
    }
}

template <typename T, int D> cudaError_t launch_combine(const WorkArgs &p, cudaStream_t s)
{
    const int blocks = p.rows_max <= 64 ? (p.rows_max + 3) / 4 : (p.rows_max + 15) / 16;
    return launch_pdl(attn_combine_kernel<T, D>, dim3(p.runs, blocks), dim3(128), 0, s, p);
}

// Joins what a token's head has of its own and of the shared keys: a warp a
// (token, head), parts in the order own, shared, each in the order of its keys.
// Bound, as above, by latency: the items' records, then a part's (m, l) a lane
// and U parts' O.  Where there is a place for every warp at once, 64 registers
// of O are under way: 64 samples of 16,000 tokens with the join take 41.6 us
// instead of 43.5 with eight parts in a loop behind the (m, l), 32 rows x 4
// tokens in fp32 30.1 instead of 36.3.  Where there is not, registers cost
// more: 8 chunks of 512 tokens 224 us, with four 200.
template <typename T, int D, int U> __global__ void __launch_bounds__(128) attn_join_kernel(const SharedArgs p)
{
    wait_prior_grid();
    const int lane = threadIdx.x & 31, hq = p.a.hq, heads = p.a.pages.hkv * p.groups;
    const long long i = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (i >= (long long)p.a.c.total_tokens * hq)
        return;
    const int tok = (int)(i / hq), head = (int)(i - (long long)tok * hq), h = head / p.g;
    int4 own = p.rec[(size_t)tok * heads + h], all = p.rec[((size_t)p.a.c.total_tokens + tok) * heads + h];
    if (own.z < 0 || (own.z == 0 && !own.w))
        return; // a dead token, or the item has written the output
    // (a token that no row has, by tables that are wrong, has no record: whatever is read as one stays within the workspace)
    auto within = [&](int4 &x) {
        x.y = min(max(x.y, 0), p.runs - 1);
        x.z = min(max(x.z, 0), p.runs - 1 - x.y);
        const int in = min(max(tok - x.x, 0), p.second ? 2 * p.tq - 1 : p.tq - 1), tile = p.second && in >= p.tq;
        x.x = min(tile * p.second + (in - tile * p.tq) * p.g + (head - h * p.g), p.rows_max - 1); // row of the item's tiles
    };
    within(own), within(all);
    const int no = 1 + own.z, parts = no + (own.w ? 1 + all.z : 0);
    auto slot = [&](int j) -> size_t {
        const int4 &x = j < no ? own : all;
        const int k = j < no ? j : j - no;
        return k == 0 ? (size_t)((j < no ? 0 : (long long)p.a.c.total_tokens * hq) + i) : p.dense + (size_t)(x.y + k) * p.rows_max + x.x;
    };
    constexpr int V = D / 32 < 4 ? D / 32 : 4, N = D / (32 * V); // a lane's columns: N runs of V
    const float k2 = p.a.scale * 1.44269504088896341f;
    float m = -INFINITY, l = 0.f, x[N][V] = {};
    bool bad = false;
    float y[U][N][V];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= parts)
                break;
            const float *const o = p.part_o + slot(j0 + u) * D + V * lane;
#pragma unroll
            for (int n = 0; n < N; ++n)
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(y[u][n]) = *reinterpret_cast<const float4 *>(o + 32 * V * n);
                else
                    *reinterpret_cast<float2 *>(y[u][n]) = *reinterpret_cast<const float2 *>(o + 32 * V * n);
        }
    };
    for (int i0 = 0; i0 < parts; i0 += 32) {
        const float2 ml = i0 + lane < parts ? p.part_ml[slot(i0 + lane)] : make_float2(-INFINITY, 0.f);
        fetch(i0);
        bad |= __any_sync(0xffffffffu, ml.x != ml.x);
        float top = fmaxf(m, ml.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float old = m == -INFINITY ? 0.f : ex2((m - top) * k2), f = ml.x == -INFINITY ? 0.f : ex2((ml.x - top) * k2);
        m = top;
        float sum = ml.y * f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = fmaf(l, old, sum);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < V; ++e)
                x[n][e] *= old;
        for (int j0 = 0; j0 < min(32, parts - i0); j0 += U) {
            if (j0 > 0)
                fetch(i0 + j0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + j0 + u >= parts)
                    break;
                const float fj = __shfl_sync(0xffffffffu, f, j0 + u);
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int e = 0; e < V; ++e) // (what a value that is not finite gave stays; a part without weight is finite)
                        x[n][e] = fmaf(y[u][n][e], fj, x[n][e]);
            }
        }
    }
    T *const out = static_cast<T *>(p.a.out) + i * D + V * lane;
    const float inv = 1.f / l;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < V; ++e)
            out[32 * V * n + e] = from_f<T>(bad ? 0.f : x[n][e] * inv);
}

// The workspace with shared prefixes: the records, then (m, l) and O.
inline size_t shared_bytes(int d, int hq, int heads, int tokens, int runs, int rows_max)
{
    const size_t rows = 2 * (size_t)tokens * hq + (size_t)runs * rows_max;
    return ((2 * sizeof(int4) * (size_t)tokens * heads + rows * sizeof(float2) + 31) & ~(size_t)31) + 16 + rows * sizeof(float) * d;
}
inline void shared_layout(SharedArgs &p, const SharedPrefix &f)
{
    const size_t tokens = p.a.c.total_tokens;
    p.bounds = f.bounds, p.prefix = reinterpret_cast<const int2 *>(f.prefix), p.ngroups = f.groups;
    p.cuts = nullptr;
    p.dense = 2 * tokens * p.a.hq;
    const size_t rows = p.dense + (size_t)p.runs * p.rows_max;
    p.rec = static_cast<int4 *>(p.a.work);
    p.part_ml = reinterpret_cast<float2 *>(p.rec + 2 * tokens * p.a.pages.hkv * p.groups);
    p.part_o = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(p.part_ml + rows) + 31) & ~(uintptr_t)31); // (32-byte stores)
}
template <typename T, int D> cudaError_t launch_join(const SharedArgs &p, cudaStream_t s)
{
    const long long warps = (long long)p.a.c.total_tokens * p.a.hq;
    const dim3 grid((unsigned)((warps + 3) / 4));
    return warps <= 32 * kSms ? launch_pdl(attn_join_kernel<T, D, 2048 / D>, grid, dim3(128), 0, s, p)
                              : launch_pdl(attn_join_kernel<T, D, 4>, grid, dim3(128), 0, s, p);
}

} // namespace
} // namespace gdn
