// Pages of cache rows (sm_103a): reserving, forking and freeing them,
// compacting a pool, copying page contents, and finding what rows share.
//
// The reference counts are the only record of what is free, so every
// allocation ranks the free pages (refs == 0, page 0 apart) in ascending order
// and hands rank r to the r-th page asked for: the result depends on the
// tables alone, never on timing.
#include <cooperative_groups.h>

#include "gdn_device.cuh"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kPlanThreads = 1024; // one CTA plans a reservation or a fork
constexpr int kRowThreads = 256;
constexpr int kChunk = 1024;       // pages a CTA ranks in a compaction
constexpr int kPer = kChunk / kRowThreads;
constexpr int kLook = 8;           // entries a lane loads together when a fork's source is looked over

// Exclusive sum of v over the CTA's threads (a multiple of 32, at most 1024);
// `total` gets the whole sum.  `part` is 33 ints of shared memory.
__device__ __forceinline__ int block_scan(int v, int *part, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o)
            s += x;
    }
    if (lane == 31)
        part[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const int x0 = lane < warps ? part[lane] : 0;
        int x = x0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o)
                x += y;
        }
        part[lane] = x - x0;
        if (lane == 31)
            part[32] = x;
    }
    __syncthreads();
    const int before = part[warp] + s - v;
    total = part[32];
    __syncthreads();
    return before;
}

// Exclusive sums of start[0 .. n) in place; returns the total.
__device__ int scan_array(int *start, int n, int *part)
{
    int sum = 0;
    for (int base = 0; base < n; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int total;
        const int before = block_scan(i < n ? start[i] : 0, part, total);
        if (i < n)
            start[i] = sum + before;
        sum += total;
    }
    __syncthreads();
    return sum;
}

// Calls take(page, rank) for the free pages of rank below `want`; returns how
// many there were (at most want).
template <typename F> __device__ int rank_free(const int32_t *refs, int num_pages, int want, int *part, F take)
{
    int found = 0;
    for (int base = 0; base < num_pages && found < want; base += 4 * kPlanThreads) {
        const int p0 = base + 4 * threadIdx.x;
        bool free[4];
        int mine = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            free[j] = p0 + j > 0 && p0 + j < num_pages && refs[p0 + j] == 0;
            mine += free[j];
        }
        int total;
        int rank = found + block_scan(mine, part, total);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (free[j]) {
                if (rank < want)
                    take(p0 + j, rank);
                ++rank;
            }
        found += total;
    }
    __syncthreads();
    return found < want ? found : want;
}

__global__ void __launch_bounds__(kPlanThreads) reserve_kernel(const PageTables t, const int32_t *rows,
                                                               const int32_t *tokens, int n, int32_t *status)
{
    __shared__ int start[GDN_MAX_PAGE_ROWS]; // pages asked for by the entries before this one
    __shared__ int part[33];
    wait_prior_grid();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int r = rows[i];
        const long long tok = tokens[i];
        const bool good = r >= 0 && r < t.table_rows && tok >= 0 && tok <= (long long)t.max_pages * t.page_size;
        int ask = 0;
        if (good) {
            const int32_t *row = t.table + (size_t)r * t.max_pages;
            int lo = 0, hi = t.max_pages; // pages held: the entries before the first zero
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (row[mid] != 0)
                    lo = mid + 1;
                else
                    hi = mid;
            }
            ask = max(0, (int)((tok + t.page_size - 1) / t.page_size) - lo);
        } else {
            report(t.err, GDN_DEVERR_BAD_PAGE);
        }
        status[i] = good ? 0 : GDN_DEVERR_BAD_PAGE;
        start[i] = ask;
    }
    __syncthreads();
    const int want = scan_array(start, n, part);
    auto asked = [&](int i) { return (i + 1 < n ? start[i + 1] : want) - start[i]; };
    // entry i's pages end at ceil(tokens / page_size)
    auto place = [&](int i, int j) {
        return t.table + (size_t)rows[i] * t.max_pages +
               ((tokens[i] + (long long)t.page_size - 1) / t.page_size - asked(i) + j);
    };
    const int found = rank_free(t.refs, t.num_pages, want, part, [&](int page, int rank) {
        int lo = 0, hi = n - 1; // the last entry that starts at or before rank
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start[mid] <= rank)
                lo = mid;
            else
                hi = mid - 1;
        }
        *place(lo, rank - start[lo]) = page;
        t.refs[page] = 1;
    });
    if (found == want)
        return;
    // too few: entries that did not get all of theirs give back what they got
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int ask = asked(i);
        if (ask == 0 || start[i] + ask <= found)
            continue;
        for (int j = 0; j < ask && start[i] + j < found; ++j) {
            int32_t *e = place(i, j);
            t.refs[*e] = 0;
            *e = 0;
        }
        status[i] = GDN_DEVERR_NO_PAGES;
        report(t.err, GDN_DEVERR_NO_PAGES);
    }
}

// Entry e of the row that fork i makes: full pages shared, entries past the
// row's pages zeroed.  (The plan has looked at the source's pages; they are
// looked at again only so that a source which the call itself makes, against
// the contract, counts no page out of range.)
__device__ __forceinline__ void fork_entry(const PageTables &t, const int32_t *src_rows, const int32_t *dst_rows, int i, int e)
{
    const int s = src_rows[i], len = t.seq_len[s], full = len / t.page_size;
    int32_t *const to = t.table + (size_t)dst_rows[i] * t.max_pages + e;
    if (e < full) {
        int page = t.table[(size_t)s * t.max_pages + e];
        if (page > 0 && page < t.num_pages) {
            atomicAdd(t.refs + page, 1);
        } else {
            report(t.err, GDN_DEVERR_BAD_PAGE);
            page = 0;
        }
        *to = page;
    } else if (e > full || len % t.page_size == 0) {
        *to = 0;
    }
}

// The pages that forks need for partial last pages, their lengths and move
// list.  Where `rows` is set the rows of the entries with status 0 are filled
// here too, else by fork_rows_kernel.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PageTables t, const int32_t *src_rows,
                                                                 const int32_t *dst_rows, int n, int32_t *move_src,
                                                                 int32_t *move_dst, int32_t *move_count,
                                                                 int32_t *status, int rows)
{
    __shared__ int start[GDN_MAX_PAGE_ROWS]; // partial pages of the entries before this one
    __shared__ int owner[GDN_MAX_PAGE_ROWS]; // the entry that gets the free page of a rank
    __shared__ int part[33];
    wait_prior_grid();
    // A fork is done whole or not at all, so all pages of its source are looked at before any is given out.  A warp takes up
    // to 32 forks together, the rows and length of one a lane, then a source's entries at a time; a source that repeats is
    // looked at once (a prompt sampled several times).  This takes 0.2 us for a row of 63 pages and 2.4 us for 192 forks of
    // 48 rows of up to 375.
    const int lane = threadIdx.x & 31, warps = kPlanThreads / 32, per = min(32, (n + warps - 1) / warps);
    for (int i0 = (threadIdx.x >> 5) * per; i0 < n; i0 += warps * per) {
        const int i = i0 + lane;
        const bool mine = lane < per && i < n;
        int s = -1, len = 0;
        bool good = false;
        if (mine) {
            s = src_rows[i];
            const int d = dst_rows[i];
            if (s >= 0 && s < t.table_rows && d >= 0 && d < t.table_rows && s != d) {
                len = t.seq_len[s];
                good = len >= 0 && len <= (long long)t.max_pages * t.page_size && t.table[(size_t)d * t.max_pages] == 0;
            }
        }
        const int held = good ? (len + t.page_size - 1) / t.page_size : 0;
        int row = -1;
        bool whole = true; // row's pages are pages
        for (int k = 0; k < per; ++k) {
            const int h = __shfl_sync(0xffffffffu, held, k), from = __shfl_sync(0xffffffffu, s, k);
            if (h == 0)
                continue;
            if (from != row) {
                row = from;
                const int32_t *const entries = t.table + (size_t)row * t.max_pages;
                bool bad = false;
                for (int j0 = lane; j0 < h; j0 += 32 * kLook) {
                    int page[kLook]; // past the last entry: the last again
#pragma unroll
                    for (int j = 0; j < kLook; ++j)
                        page[j] = entries[min(j0 + 32 * j, h - 1)];
#pragma unroll
                    for (int j = 0; j < kLook; ++j)
                        bad |= page[j] <= 0 || page[j] >= t.num_pages;
                }
                whole = !__any_sync(0xffffffffu, bad);
            }
            if (lane == k)
                good = whole;
        }
        if (mine) {
            if (!good)
                report(t.err, GDN_DEVERR_BAD_PAGE);
            status[i] = good ? 0 : GDN_DEVERR_BAD_PAGE;
            start[i] = good && len % t.page_size != 0;
        }
    }
    __syncthreads();
    const int want = scan_array(start, n, part);
    auto asks = [&](int i) { return (i + 1 < n ? start[i + 1] : want) > start[i]; };
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        if (asks(i))
            owner[start[i]] = i;
    __syncthreads();
    const int found = rank_free(t.refs, t.num_pages, want, part, [&](int page, int rank) {
        const int i = owner[rank];
        const int s = src_rows[i], e = t.seq_len[s] / t.page_size;
        t.table[(size_t)dst_rows[i] * t.max_pages + e] = page;
        t.refs[page] = 1;
        move_src[rank] = t.table[(size_t)s * t.max_pages + e];
        move_dst[rank] = page;
    });
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        if (i >= found)
            move_src[i] = 0, move_dst[i] = 0;
        if (status[i] != 0)
            continue;
        if (asks(i) && start[i] >= found) {
            status[i] = GDN_DEVERR_NO_PAGES;
            report(t.err, GDN_DEVERR_NO_PAGES);
        } else {
            t.seq_len[dst_rows[i]] = t.seq_len[src_rows[i]];
        }
    }
    if (threadIdx.x == 0)
        *move_count = found;
    if (!rows)
        return;
    __syncthreads(); // the statuses are written
    for (long long x = threadIdx.x; x < (long long)n * t.max_pages; x += kPlanThreads) {
        const int i = (int)(x / t.max_pages), e = (int)(x - (long long)i * t.max_pages);
        if (status[i] == 0)
            fork_entry(t, src_rows, dst_rows, i, e);
    }
}

// One table entry a thread.
__global__ void __launch_bounds__(kRowThreads) fork_rows_kernel(const PageTables t, const int32_t *src_rows,
                                                                const int32_t *dst_rows, const int32_t *status,
                                                                int chunks)
{
    wait_prior_grid();
    const int i = blockIdx.x / chunks;
    const int e = (blockIdx.x - i * chunks) * kRowThreads + threadIdx.x;
    if (e >= t.max_pages || status[i] != 0)
        return;
    fork_entry(t, src_rows, dst_rows, i, e);
}

// One table entry a thread.  The exchange makes a row that is listed twice
// give up its pages once.
__global__ void __launch_bounds__(kRowThreads) free_kernel(const PageTables t, const int32_t *rows, int chunks)
{
    wait_prior_grid();
    const int i = blockIdx.x / chunks;
    const int e = (blockIdx.x - i * chunks) * kRowThreads + threadIdx.x;
    const int r = rows[i];
    if (r < 0 || r >= t.table_rows) {
        if (e == 0)
            report(t.err, GDN_DEVERR_BAD_PAGE);
        return;
    }
    if (e == 0)
        t.seq_len[r] = 0;
    if (e >= t.max_pages)
        return;
    int32_t *const at = t.table + (size_t)r * t.max_pages + e;
    if (*at == 0)
        return;
    const int page = atomicExch(at, 0);
    if (page == 0)
        return;
    if (page < 0 || page >= t.num_pages) {
        report(t.err, GDN_DEVERR_BAD_PAGE);
    } else if (atomicSub(t.refs + page, 1) <= 0) {
        atomicAdd(t.refs + page, 1);
        report(t.err, GDN_DEVERR_BAD_PAGE);
    }
}

// ---- compaction ------------------------------------------------------------------
// Page p < L (L pages in use) that is free is a hole: its rank among the holes
// is p minus the live pages before it.  A live page p >= L has rank (live
// pages before p) - (live pages before L); there are as many of these as
// holes, and equal ranks are matched.  Bound: the latency of four small
// launches; a CTA ranks kChunk pages, and takes the sums of the chunks before
// its own from the first launch.  59 k pages take about 25 us with the tables.

__device__ __forceinline__ bool live_page(const int32_t *refs, int p) { return p == 0 || refs[p] > 0; }

__global__ void __launch_bounds__(kRowThreads) compact_count_kernel(const int32_t *refs, int num_pages, int32_t *counts)
{
    __shared__ int part[33];
    wait_prior_grid();
    int mine = 0;
    for (int j = 0; j < kPer; ++j) {
        const int p = blockIdx.x * kChunk + j * kRowThreads + threadIdx.x;
        mine += p < num_pages && live_page(refs, p);
    }
    int total;
    block_scan(mine, part, total);
    if (threadIdx.x == 0)
        counts[blockIdx.x] = total;
}

// Sum of counts[0 .. n), by the whole CTA.
__device__ int sum_counts(const int32_t *counts, int n, int *part)
{
    int mine = 0, total;
    for (int c = threadIdx.x; c < n; c += blockDim.x)
        mine += counts[c];
    block_scan(mine, part, total);
    return total;
}

__global__ void __launch_bounds__(kRowThreads) compact_plan_kernel(const int32_t *refs, int num_pages,
                                                                   const int32_t *counts, int32_t *remap,
                                                                   int32_t *move_src, int32_t *move_dst,
                                                                   int32_t *move_count)
{
    __shared__ int part[33];
    wait_prior_grid();
    const int live = sum_counts(counts, gridDim.x, part);
    const int before = sum_counts(counts, blockIdx.x, part);
    // live pages below L: whole chunks, then the chunk that holds L
    const int lc = live / kChunk;
    int below = sum_counts(counts, lc, part);
    {
        int mine = 0, total;
        for (int p = lc * kChunk + threadIdx.x; p < live; p += kRowThreads)
            mine += live_page(refs, p);
        block_scan(mine, part, total);
        below += total;
    }
    const int moves = live - below;
    bool is_live[kPer];
    int mine = 0, total;
    const int p0 = blockIdx.x * kChunk + threadIdx.x * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        is_live[j] = p0 + j < num_pages && live_page(refs, p0 + j);
        mine += is_live[j];
    }
    int rank = before + block_scan(mine, part, total); // live pages before p0 + j
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int p = p0 + j;
        if (p >= num_pages)
            break;
        if (p >= moves)
            move_src[p] = 0, move_dst[p] = 0;
        if (p < live) {
            if (!is_live[j])
                move_dst[p - rank] = p;
            remap[p] = is_live[j] ? p : 0;
        } else if (is_live[j]) {
            move_src[rank - below] = p;
        } else {
            remap[p] = 0;
        }
        rank += is_live[j];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        *move_count = moves;
}

// remap of the moved pages, and the reference counts in their new places.  A
// thread writes only what no other thread reads, so refs_out may be refs.
__global__ void __launch_bounds__(kRowThreads) compact_refs_kernel(const int32_t *refs, int32_t *refs_out,
                                                                   int num_pages, const int32_t *counts, int chunks,
                                                                   const int32_t *move_src, const int32_t *move_dst,
                                                                   const int32_t *move_count, int32_t *remap)
{
    __shared__ int part[33];
    wait_prior_grid();
    const int live = sum_counts(counts, chunks, part);
    const int p = blockIdx.x * kRowThreads + threadIdx.x;
    if (p >= num_pages)
        return;
    if (p < *move_count) {
        const int from = move_src[p], to = move_dst[p];
        const int n = refs[from];
        refs_out[to] = n;
        refs_out[from] = 0;
        remap[from] = to;
    }
    const bool here = live_page(refs, p);
    if (p < live ? here : !here)
        refs_out[p] = refs[p];
}

__global__ void __launch_bounds__(kRowThreads) compact_table_kernel(const int32_t *table, int32_t *table_out,
                                                                    size_t entries, const int32_t *remap,
                                                                    int num_pages, int *err)
{
    wait_prior_grid();
    for (size_t i = (size_t)blockIdx.x * kRowThreads + threadIdx.x; i < entries; i += (size_t)gridDim.x * kRowThreads) {
        const int p = table[i];
        const bool good = p >= 0 && p < num_pages;
        if (!good)
            report(err, GDN_DEVERR_BAD_PAGE);
        table_out[i] = good && p > 0 ? remap[p] : 0;
    }
}

// ---- page contents ---------------------------------------------------------------
// A CTA moves 16 KB pieces (four 16-byte vectors a thread, all loaded before
// the first store), over (pair, layer, K or V, piece).  Bound: HBM; eight CTAs
// an SM keep 128 KB under way there.  1.9 GB (a compaction of four layers) take
// 291 us, 6.4 TB/s, 96 % of a plain copy's rate.
constexpr int kCopyVecs = 4;
constexpr int kPieceVecs = kRowThreads * kCopyVecs;

__global__ void __launch_bounds__(kRowThreads) copy_kernel(uint4 *k, uint4 *v, int num_pages, int layers, int page_vecs,
                                                           int pieces, const int32_t *src, const int32_t *dst, int n,
                                                           const int32_t *count, int *err)
{
    wait_prior_grid();
    const int pairs = count ? min(n, max(0, *count)) : n;
    const size_t total = (size_t)pairs * layers * 2 * pieces;
    for (size_t u = blockIdx.x; u < total; u += gridDim.x) {
        const int piece = (int)(u % pieces);
        const size_t w = u / pieces;
        const int layer = (int)((w >> 1) % layers);
        const int pair = (int)((w >> 1) / layers);
        const int s = src[pair], d = dst[pair];
        if (s <= 0 || s >= num_pages || d <= 0 || d >= num_pages) {
            if ((s != 0 || d != 0) && threadIdx.x == 0)
                report(err, GDN_DEVERR_BAD_PAGE);
            continue;
        }
        uint4 *const base = (w & 1 ? v : k) + (size_t)layer * num_pages * page_vecs;
        const uint4 *const from = base + (size_t)s * page_vecs;
        uint4 *const to = base + (size_t)d * page_vecs;
        uint4 x[kCopyVecs];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j) {
            const int i = piece * kPieceVecs + j * kRowThreads + threadIdx.x;
            if (i < page_vecs)
                x[j] = from[i];
        }
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j) {
            const int i = piece * kPieceVecs + j * kRowThreads + threadIdx.x;
            if (i < page_vecs)
                to[i] = x[j];
        }
    }
}

int sm_count()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 1;
    return n;
}

// The pages that the rows of a group share: a cluster of CTAs a group.  Every
// CTA looks over the group's lengths (the first live row leads, and no row's
// new tokens may lie in a shared page); then the warps of the cluster compare
// the live rows' entries with the leader's, kSpan of them at a time, and leave
// out what lies behind the first difference found so far.  Bound: latency, of
// four or five loads in a row; the entries themselves are few.
constexpr int kSpan = 256;

__global__ void __launch_bounds__(kRowThreads) shared_kernel(const CacheRows c, const int32_t *bounds, int groups, int page_shift,
                                                             int2 *prefix, int *err)
{
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ int lead, live, limit; // this CTA's, then the cluster's in its first CTA
    const int tid = threadIdx.x, lane = tid & 31, warps = kRowThreads / 32, size = cluster.num_blocks(), rank = cluster.block_rank();
    const int g = blockIdx.x / size;
    wait_prior_grid();
    const int b0 = bounds[g], b1 = bounds[g + 1];
    const int r0 = min(max(b0, 0), c.rows), r1 = min(max(b1, r0), c.rows);
    if (tid == 0) {
        lead = r1, live = 0, limit = c.max_pages;
        if (rank == 0 && (r0 != b0 || r1 != b1 || (g == 0 && b0 != 0) || (g == groups - 1 && b1 != c.rows)))
            report(err, GDN_DEVERR_BAD_PAGE);
    }
    __syncthreads();
    auto before = [&](int r) { // tokens before the new ones, or -1
        const int n = c.seq_len[r], fresh = c.cu_seqlens[r + 1] - c.cu_seqlens[r];
        return n > 0 && fresh > 0 && n >= fresh ? n - fresh : -1;
    };
    for (int r = r0 + tid; r < r1; r += kRowThreads) {
        const int n = before(r);
        if (n >= 0) {
            atomicMin(&lead, r);
            atomicAdd(&live, 1);
            atomicMin(&limit, n >> page_shift);
        }
    }
    __syncthreads();
    const int first = lead < r1 ? lead : r0;
    const int most = live > 1 ? limit : 0; // (the same in every CTA)
    __syncthreads();
    if (tid == 0)
        limit = most;
    cluster.sync();
    int *const found = cluster.map_shared_rank(&limit, 0);
    const int32_t *const model = c.table + (size_t)first * c.max_pages;
    const int spans = (most + kSpan - 1) / kSpan;
    const long long units = (long long)spans * (r1 - r0);
    for (long long u = (long long)rank * warps + tid / 32; u < units; u += (long long)size * warps) {
        const int span = (int)(u / (r1 - r0)), r = r0 + (int)(u - (long long)span * (r1 - r0)), at = span * kSpan + lane;
        if (r == first || span * kSpan >= *reinterpret_cast<volatile int *>(&limit) || before(r) < 0)
            continue;
        const int32_t *const row = c.table + (size_t)r * c.max_pages;
        int differs = most;
#pragma unroll
        for (int k = kSpan / 32 - 1; k >= 0; --k) {
            const int i = at + 32 * k;
            if (i < most && row[i] != model[i])
                differs = i;
        }
        differs = __reduce_min_sync(0xffffffffu, differs);
        if (lane == 0 && differs < most) {
            atomicMin(&limit, differs);
            if (rank != 0)
                atomicMin(found, differs);
        }
    }
    cluster.sync();
    const int2 answer = make_int2(first, *reinterpret_cast<volatile int *>(found));
    for (int r = r0 + rank * kRowThreads + tid; r < r1; r += size * kRowThreads)
        prefix[r] = answer;
    if (g == 0 && rank == 0) // rows of no group, by bounds that are wrong
        for (int r = tid; r < r0; r += kRowThreads)
            prefix[r] = make_int2(r, 0);
    if (g == groups - 1 && rank == 0)
        for (int r = r1 + tid; r < c.rows; r += kRowThreads)
            prefix[r] = make_int2(r, 0);
    cluster.sync(); // the first CTA's memory is read by the others
}

} // namespace

cudaError_t launch_pages_shared(const CacheRows &c, const int32_t *bounds, int groups, int page_size, int32_t *prefix, int *err,
                                cudaStream_t s)
{
    // CTAs a group: 32 groups of 32 rows over 1,000 to 16,000 tokens (pages of 16) take 15.2 us with one, 10.0 with two, 6.8
    // with four, 5.1 with eight; one group of 16 rows over 512 3.9 with one, 3.3 with eight.
    constexpr unsigned kCluster = 8;
    if (groups > (int)(0x7fffffff / kCluster))
        return cudaErrorInvalidConfiguration;
    int shift = 0;
    while ((1 << shift) < page_size)
        ++shift;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)groups * kCluster);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster, attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, shared_kernel, c, bounds, groups, shift, reinterpret_cast<int2 *>(prefix), err);
}

cudaError_t launch_pages_reserve(const PageTables &t, const int32_t *list_rows, const int32_t *tokens, int n,
                                 int32_t *status, cudaStream_t s)
{
    return launch_pdl(reserve_kernel, dim3(1), dim3(kPlanThreads), 0, s, t, list_rows, tokens, n, status);
}

cudaError_t launch_pages_fork(const PageTables &t, const int32_t *src_rows, const int32_t *dst_rows, int n,
                              int32_t *move_src, int32_t *move_dst, int32_t *move_count, int32_t *status,
                              cudaStream_t s)
{
    // a second launch costs about 2 us, as does filling eight entries a thread in the first
    const int rows = (long long)n * t.max_pages <= 8 * kPlanThreads;
    cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, t, src_rows, dst_rows, n, move_src,
                               move_dst, move_count, status, rows);
    if (e != cudaSuccess || rows)
        return e;
    const int chunks = (t.max_pages + kRowThreads - 1) / kRowThreads;
    if ((long long)chunks * n > 0x7fffffffll)
        return cudaErrorInvalidValue;
    return launch_pdl(fork_rows_kernel, dim3((unsigned)(chunks * n)), dim3(kRowThreads), 0, s, t, src_rows, dst_rows,
                      static_cast<const int32_t *>(status), chunks);
}

cudaError_t launch_pages_free(const PageTables &t, const int32_t *list_rows, int n, cudaStream_t s)
{
    const int chunks = (t.max_pages + kRowThreads - 1) / kRowThreads;
    if ((long long)chunks * n > 0x7fffffffll)
        return cudaErrorInvalidValue;
    return launch_pdl(free_kernel, dim3((unsigned)(chunks * n)), dim3(kRowThreads), 0, s, t, list_rows, chunks);
}

cudaError_t launch_pages_compact(const PageTables &t, int32_t *table_out, int32_t *refs_out, int32_t *remap,
                                 int32_t *move_src, int32_t *move_dst, int32_t *move_count, int32_t *scratch,
                                 cudaStream_t s)
{
    const int chunks = (int)(((long long)t.num_pages + kChunk - 1) / kChunk);
    const int32_t *refs = t.refs, *table = t.table;
    cudaError_t e = launch_pdl(compact_count_kernel, dim3(chunks), dim3(kRowThreads), 0, s, refs, t.num_pages, scratch);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(compact_plan_kernel, dim3(chunks), dim3(kRowThreads), 0, s, refs, t.num_pages,
                   static_cast<const int32_t *>(scratch), remap, move_src, move_dst, move_count);
    if (e != cudaSuccess)
        return e;
    e = launch_pdl(compact_refs_kernel, dim3((unsigned)(((long long)t.num_pages + kRowThreads - 1) / kRowThreads)),
                   dim3(kRowThreads), 0, s, refs, refs_out, t.num_pages, static_cast<const int32_t *>(scratch), chunks,
                   static_cast<const int32_t *>(move_src), static_cast<const int32_t *>(move_dst),
                   static_cast<const int32_t *>(move_count), remap);
    if (e != cudaSuccess)
        return e;
    const size_t entries = (size_t)t.table_rows * t.max_pages;
    const size_t blocks = (entries + kRowThreads - 1) / kRowThreads;
    return launch_pdl(compact_table_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kRowThreads), 0, s,
                      table, table_out, entries, static_cast<const int32_t *>(remap), t.num_pages, t.err);
}

cudaError_t launch_pages_copy(const kv_page_pool &pool, const int32_t *src, const int32_t *dst, int n,
                              const int32_t *count, int *err, cudaStream_t s)
{
    const int page_vecs = (int)((size_t)pool.hkv * pool.page_size * pool.d * (pool.dtype == GDN_BF16 ? 2 : 4) / 16);
    const int pieces = (page_vecs + kPieceVecs - 1) / kPieceVecs;
    const unsigned long long units = (unsigned long long)n * pool.layers * 2 * pieces;
    const unsigned long long most = 8ull * sm_count(); // eight CTAs of 256 threads fill an SM
    return launch_pdl(copy_kernel, dim3((unsigned)(units < most ? units : most)), dim3(kRowThreads), 0, s,
                      static_cast<uint4 *>(pool.k), static_cast<uint4 *>(pool.v), pool.num_pages, pool.layers,
                      page_vecs, pieces, src, dst, n, count, err);
}

} // namespace gdn
