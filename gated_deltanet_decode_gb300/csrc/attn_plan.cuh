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

// One cut item, for the combining kernel: written by the run that holds the
// item's second part.
struct Cut {
    int parts, tok, ntok, head;
};

// Units of a key tile of an item with `rows` rows: kernels whose tiles cost the
// same whatever the rows, and others.
struct EvenCost {
    static constexpr int least = 1, most = 1;
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
// Key tiles of the row's item t (mt tokens an item).
__device__ __forceinline__ int item_tiles(const Row &x, int t, int mt, int kt)
{
    const int last = min(x.n, (t + 1) * mt);
    return (x.len - x.n + last + kt - 1) / kt;
}
__device__ __forceinline__ int items_of(const Row &x, int mt) { return (x.n + mt - 1) / mt; }
template <typename Cost> __device__ long long head_units(const Row &x, int mt, int kt, int g) // of one key head
{
    long long s = 0;
    const int n = items_of(x, mt);
    for (int t = 0; t < n; ++t)
        s += item_tiles(x, t, mt, kt) * (long long)Cost::of(min(mt, x.n - t * mt) * g);
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
struct Run {
    long long share, u0, u1, base;
    long long per; // units a head of the row it begins in
    int row;
    Row first;     // that row
};
struct Found { // shared memory
    long long base, per;
    int row;
    Row first;
};
template <int THREADS, int KT, typename Cost> __device__ Run plan_run(const WorkArgs &p, int mt, long long *part, Found &found)
{
    const CacheRows &c = p.a.c;
    const int ps = p.a.pages.page_size, heads = p.a.pages.hkv * p.groups, tid = threadIdx.x;
    Row x{0, 0, 0, false, false};
    long long per = 0;
    auto cost_of = [&](int r) -> long long {
        if (r >= c.rows)
            return 0;
        x = row_of(c, ps, r);
        per = x.live ? head_units<Cost>(x, mt, KT, p.g) : 0;
        return per * heads;
    };
    int dearest = 1; // tile of this thread's rows
    Run run;
    long long total = 0, cost = 0, before = 0, sum;
    for (int b = 0; b < c.rows; b += THREADS) {
        cost = cost_of(b + tid);
        if (cost > 0)
            dearest = max(dearest, Cost::of(min(x.n, mt) * p.g));
        if (x.bad && blockIdx.x == 0)
            report(p.a.err, GDN_DEVERR_BAD_PAGE);
        before = scan64(cost, part, THREADS / 32, sum);
        total += sum;
    }
    run.share = (total + gridDim.x - 1) / gridDim.x;
    // (Cost's values are few, and one barrier tells whether a thread has seen more than the least)
    const int least = Cost::least, tile = Cost::most == least ? least : __syncthreads_or(dearest > least) ? Cost::most : least;
    if (run.share < tile)
        run.share = tile;
    run.u0 = run.share * blockIdx.x;
    run.u1 = min(total, run.u0 + run.share);
    if (c.rows <= THREADS) { // the one pass has it
        if (cost > 0 && before <= run.u0 && run.u0 < before + cost)
            found = {before, per, tid, x};
    } else {
        long long seen = 0;
        for (int b = 0; b < c.rows && seen <= run.u0 && run.u0 < total; b += THREADS) {
            cost = cost_of(b + tid);
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
template <typename T, int D, int THREADS> __device__ void zero_dead(const WorkArgs &p, int tid)
{
    const CacheRows &c = p.a.c;
    const size_t vecs = (size_t)p.a.hq * D * sizeof(T) / 16; // a token's
    uint4 *const out = static_cast<uint4 *>(p.a.out);
    auto zero = [&](int t0, int t1) {
        for (size_t i = (size_t)t0 * vecs + tid; i < (size_t)t1 * vecs; i += THREADS)
            out[i] = make_uint4(0, 0, 0, 0);
    };
    for (int r = blockIdx.x; r < c.rows; r += gridDim.x) {
        const Row x = row_of(c, p.a.pages.page_size, r);
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
template <typename Cost> struct Walk {
    const WorkArgs &p;
    const Run &run;
    int mt, kt, heads, lane;
    long long u;     // where the next tile begins
    int r, win;      // row; rows win .. win + 31 are in the lanes
    Row mine, x;     // a lane's row; the current one
    int items, h, t, ja;
    bool in_row;

    __device__ Walk(const WorkArgs &p_, const Run &run_, int mt_, int kt_)
        : p(p_), run(run_), mt(mt_), kt(kt_), heads(p_.a.pages.hkv * p_.groups), lane(threadIdx.x & 31), u(run_.u0),
          r(run_.row), win(run_.row), in_row(false)
    {
        if (lane == 0)
            p.cuts[blockIdx.x].parts = 0;
        __syncwarp();
        fetch(); // the next rows' lengths, while the first row's items are handed out
        if (u < run.u1) {
            enter(run.first);
            long long rem = u - run.base; // the run begins inside this row
            for (; rem >= run.per; ++h)
                rem -= run.per;
            for (;; ++t) {
                const long long units = item_tiles(x, t, mt, kt) * (long long)unit();
                if (rem < units)
                    break;
                rem -= units;
            }
            ja = (int)((rem + unit() - 1) / unit());
            u += (long long)ja * unit() - rem; // a tile that began before u0 is the run's before
            if (ja == item_tiles(x, t, mt, kt))
                done();
        }
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
    __device__ void enter(const Row &row)
    {
        x = row;
        in_row = true;
        items = items_of(x, mt);
        h = t = ja = 0;
    }
    __device__ void fetch()
    {
        win = r;
        mine = Row{0, 0, 0, false, false};
        if (u < run.u1 && win + lane < p.a.c.rows)
            mine = row_of(p.a.c, p.a.pages.page_size, win + lane);
    }
    // The next item; false at the run's end.  Lane 0 lists a cut.
    __device__ bool next(Item &it)
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
            if (!__shfl_sync(0xffffffffu, (int)mine.live, r - win)) {
                if (++r >= p.a.c.rows)
                    return false;
                continue;
            }
            enter(x);
        }
        const int J = item_tiles(x, t, mt, kt);
        const int w = unit(), jb = (int)min((long long)J, ja + (run.u1 - u + w - 1) / w);
        const int t0 = t * mt, ntok = min(mt, x.n - t0);
        it = {x.b + t0, ntok, h, r, x.len - x.n + t0 + 1, ja, jb,
              ja > 0 || jb < J ? 2 * (int)blockIdx.x + (ja > 0 ? 0 : 1) : -1};
        // the run that holds an item's second part lists it for the combining kernel
        const long long start = u - (long long)ja * w;
        if (lane == 0 && ja > 0 && start >= run.u0 - run.share)
            p.cuts[blockIdx.x] = {2 + (int)((start + (J - 1ll) * w) / run.share) - (int)blockIdx.x, x.b + t0, ntok, h};
        u += (long long)(jb - ja) * w;
        done();
        return true;
    }
};

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

} // namespace
} // namespace gdn
