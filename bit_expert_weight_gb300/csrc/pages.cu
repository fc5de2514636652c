// pages.cu -- upkeep of a paged cache's pages: smoe_pages_fork,
// smoe_pages_reserve, smoe_pages_compact (whole numbers only) and
// smoe_pages_copy.
//
// The first three change a few arrays of a pool at most of some MB, in steps
// that need one another's results.  Each runs as one thread-block cluster: its
// barrier is the hardware's and its words pass through shared memory, so a call
// is one launch, needs no workspace, and nothing of one launch is left for the
// next to find.
#include <atomic>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxKeys = 0x7fffffff - 511;  // of a sequence

__device__ __forceinline__ int log2_of(int power) { return 31 - __clz(power); }

// Pages of n keys.
__device__ __forceinline__ int pages_of(int n, int shift) { return (n + (1 << shift) - 1) >> shift; }

__device__ __forceinline__ bool valid_len(const smoe_page_pool &p, int len)
{
    return len >= 0 && len <= kMaxKeys && pages_of(len, log2_of(p.page_size)) <= p.table_stride;
}

// ------------------------------------------------------------------- fork

// Rows are rewritten in place, so one CTA owns some columns of the table for
// all sequences: it reads what moves, waits for its own threads, and writes.
// A page loses a holder with each sequence that used it and gains one with each
// child that does: for entry j of an old sequence the two come to (children
// with more than j pages) - 1, one atomic addition where that is not 0 (whole
// numbers: their order does not matter).
constexpr int kForkEntries = 8;  // of a thread and tile

struct ForkShared {
    int parent[SMOE_MAX_SEQS], was[SMOE_MAX_SEQS], len[SMOE_MAX_SEQS];
    int children[SMOE_MAX_SEQS], least[SMOE_MAX_SEQS];  // and the fewest pages of a child
};

__device__ int children_above(const ForkShared &sh, int n, int s, int j, int shift)
{
    int c = 0;
    for (int t = 0; t < n; ++t)
        c += sh.parent[t] == s && pages_of(sh.len[t], shift) > j;
    return c;
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const smoe_page_pool p, const int32_t *parent, const int32_t *keep, int *status)
{
    __shared__ ForkShared sh;
    const int tid = threadIdx.x, n = p.num_seqs, shift = log2_of(p.page_size);
    bool bad = false;
    int most = 0;
    for (int s = tid; s < n; s += kThreads) {
        const int a = parent[s], len = p.kv_len[s];
        sh.parent[s] = a;
        sh.was[s] = len;
        sh.children[s] = 0;
        sh.least[s] = 0x7fffffff;
        bad = bad || a < -1 || a >= n || !valid_len(p, len);
        if (!bad)
            most = max(most, pages_of(len, shift));
    }
    // (the same answer in every CTA: none of the arrays has been written yet)
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            set_status(status, kStatusBadArg);
        return;
    }
    for (int s = tid; s < n; s += kThreads) {
        const int a = sh.parent[s];
        int len = a < 0 ? 0 : sh.was[a];
        if (keep)
            len = min(len, max(keep[s], 0));
        sh.len[s] = len;
        if (a >= 0) {
            atomicAdd(&sh.children[a], 1);
            atomicMin(&sh.least[a], pages_of(len, shift));
        }
    }
    cluster_arrive();  // this CTA has read every length
    __shared__ int s_most;
    if (tid == 0)
        s_most = 0;
    __syncthreads();
    atomicMax(&s_most, most);
    __syncthreads();
    most = s_most;
    // columns of a tile: a power of two, so that a tile's entries fit the threads
    int width = 4;
    while (width * 2 * n <= kThreads * kForkEntries && width < 4096)
        width *= 2;
    const int wshift = log2_of(width);
    for (int j0 = cluster_rank() * width; j0 < most; j0 += cluster_size() * width) {
        // (first what is to be read, all at once; then what is done with it)
        int moved[kForkEntries], own[kForkEntries], by[kForkEntries];
        unsigned moves = 0;
#pragma unroll
        for (int i = 0; i < kForkEntries; ++i) {
            const int e = tid + i * kThreads, s = e >> wshift, j = j0 + (e & (width - 1));
            by[i] = moved[i] = own[i] = 0;
            if (s >= n)
                continue;
            const int a = sh.parent[s];
            if (a >= 0 && a != s && j < pages_of(sh.len[s], shift)) {
                moves |= 1u << i;
                moved[i] = p.page_table[(int64_t)a * p.table_stride + j];
            }
            if (j < pages_of(sh.was[s], shift)) {
                const int c = sh.children[s];
                by[i] = (j < sh.least[s] ? c : c == 1 ? 0 : children_above(sh, n, s, j, shift)) - 1;
                if (by[i] != 0)
                    own[i] = p.page_table[(int64_t)s * p.table_stride + j];
            }
        }
#pragma unroll
        for (int i = 0; i < kForkEntries; ++i)
            if (by[i] != 0) {
                if (own[i] >= 0 && own[i] < p.num_pages)
                    atomicAdd(p.refs + own[i], by[i]);
                else
                    set_status(status, kStatusBadArg);
            }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kForkEntries; ++i) {
            const int e = tid + i * kThreads, s = e >> wshift, j = j0 + (e & (width - 1));
            if (moves >> i & 1)
                p.page_table[(int64_t)s * p.table_stride + j] = moved[i];
        }
    }
    cluster_wait();
    if (cluster_rank() == 0)
        for (int s = tid; s < n; s += kThreads)
            p.kv_len[s] = sh.len[s];
}

// ------------------------------------------------- runs of a pool's pages

// Reserve and compact go over refs in runs: a CTA of the cluster has some
// consecutive pages, and each of its warps a run of them, 1024 pages (8 loads in
// flight) at a time.
constexpr int kChunk = 1024;

struct Runs {
    int64_t first, last;  // the warp's pages
};

__device__ __forceinline__ Runs run_of_warp(int num_pages)
{
    const int64_t runs = (int64_t)cluster_size() * kWarps;
    const int64_t len = (num_pages + runs * kChunk - 1) / (runs * kChunk) * kChunk;
    Runs r;
    r.first = ((int64_t)cluster_rank() * kWarps + (threadIdx.x >> 5)) * len;
    r.last = min(r.first + len, (int64_t)num_pages);
    return r;
}

// Four pages' holders from page `at` on (a multiple of 4); 0 past `last`.
__device__ __forceinline__ int4 refs_at(const int32_t *refs, int64_t at, int64_t last)
{
    if (at + 4 <= last)
        return __ldcg(reinterpret_cast<const int4 *>(refs + at));
    int4 v = make_int4(0, 0, 0, 0);
    if (at < last)
        v.x = __ldcg(refs + at);
    if (at + 1 < last)
        v.y = __ldcg(refs + at + 1);
    if (at + 2 < last)
        v.z = __ldcg(refs + at + 2);
    return v;
}

// Nibble i of a lane's word: which of pages at + 128 i + 4 lane + (0 .. 3) are held.
__device__ __forceinline__ uint32_t held_nibbles(const int32_t *refs, int64_t at, int64_t last, int lane)
{
    int4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = refs_at(refs, at + 128 * i + 4 * lane, last);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w |= static_cast<uint32_t>((v[i].x > 0) | (v[i].y > 0) << 1 | (v[i].z > 0) << 2 | (v[i].w > 0) << 3) << (4 * i);
    return w;
}

// Bit j of a lane's word: whether page at + 32 lane + j is held.
__device__ __forceinline__ uint32_t held_pages(const int32_t *refs, int64_t at, int64_t last, int lane)
{
    const uint32_t w = held_nibbles(refs, at, last, lane);
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < 8; ++t)
        m |= (__shfl_sync(0xffffffffu, w, 8 * (lane & 3) + t) >> (4 * (lane >> 2)) & 15u) << (4 * t);
    return m;
}

// Bit j: page at + j is below `end`.
__device__ __forceinline__ uint32_t below(int64_t at, int64_t end)
{
    return end - at >= 32 ? 0xffffffffu : end > at ? (1u << (end - at)) - 1u : 0u;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// The lanes' v before this one, and all lanes' in total.
__device__ __forceinline__ int lanes_before(int v, int lane, int *total)
{
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        x += lane >= o ? y : 0;
    }
    *total = __shfl_sync(0xffffffffu, x, 31);
    return x - v;
}

// Held pages of the warp's run.
__device__ __forceinline__ int count_held(const int32_t *refs, Runs r, int lane)
{
    int n = 0;
    for (int64_t at = r.first; at < r.last; at += kChunk)
        n += __popc(held_nibbles(refs, at, r.last, lane));
    return warp_sum(n);
}

// Counts of every warp of the cluster, and what comes before this warp's run.
struct RunCounts {
    int cta[kMaxCluster];  // by rank
    int warp[kWarps];      // of this CTA
};

// `mine`: the warp's count, the same in all its lanes.  The kernel has arrived
// at the cluster's barrier at its start (every CTA has begun where that ends).
// A barrier of the cluster.
__device__ __forceinline__ void share_counts(RunCounts &rc, int mine, int tid)
{
    if ((tid & 31) == 0)
        rc.warp[tid >> 5] = mine;
    __syncthreads();
    cluster_wait();
    if (tid < 32) {
        const int all = warp_sum(tid < kWarps ? rc.warp[tid] : 0);
        if (tid < static_cast<int>(cluster_size()))
            store_to_rank(&rc.cta[cluster_rank()], tid, all);
    }
    cluster_sync();
}

__device__ __forceinline__ int counted_before(const RunCounts &rc, int warp)
{
    int n = 0;
    for (unsigned r = 0; r < cluster_rank(); ++r)
        n += rc.cta[r];
    for (int w = 0; w < warp; ++w)
        n += rc.warp[w];
    return n;
}

__device__ __forceinline__ int counted(const RunCounts &rc)
{
    int n = 0;
    for (unsigned r = 0; r < cluster_size(); ++r)
        n += rc.cta[r];
    return n;
}

// ---------------------------------------------------------------- reserve

// Every CTA finds out for itself what each sequence needs, while the pool is
// counted in runs; then the free pages' ranks are known, and each one below
// the number needed looks up whose it is.
constexpr int kSlots = 2 * SMOE_MAX_SEQS;  // of the table of shared last pages

struct ReserveShared {
    RunCounts runs;
    int page[SMOE_MAX_SEQS];      // a partly filled last page that is to be written, else -1
    int holders[SMOE_MAX_SEQS];   // of it; later: the place of its copy in the list, else -1
    int had[SMOE_MAX_SEQS];       // pages
    int need[SMOE_MAX_SEQS];
    int base[SMOE_MAX_SEQS];      // free pages given to the sequences before
    int key[kSlots], writers[kSlots], first[kSlots];
    unsigned long long warp[kWarps], total;
};

// Sums over the threads before this one, and over all.
__device__ __forceinline__ unsigned long long threads_before(ReserveShared &sh, unsigned long long v, int tid)
{
    const int lane = tid & 31, w = tid >> 5;
    unsigned long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        x += lane >= o ? y : 0;
    }
    if (lane == 31)
        sh.warp[w] = x;
    __syncthreads();
    unsigned long long before = 0, all = 0;
    for (int i = 0; i < kWarps; ++i) {
        before += i < w ? sh.warp[i] : 0;
        all += sh.warp[i];
    }
    if (tid == 0)
        sh.total = all;
    __syncthreads();
    return before + x - v;
}

__device__ __forceinline__ int slot_of_page(ReserveShared &sh, int page)
{
    unsigned h = static_cast<unsigned>(page) * 2654435761u / (1u << 20) % kSlots;
    // (there are at most half as many pages as slots)
    for (int i = 0; i < kSlots; ++i) {
        const int was = atomicCAS(&sh.key[h], -1, page);
        if (was == -1 || was == page)
            break;
        h = (h + 1) % kSlots;
    }
    return static_cast<int>(h);
}

__global__ void __launch_bounds__(kThreads, 1)
    reserve_kernel(const smoe_page_pool p, const int32_t *row_start, int32_t *copies, int32_t *counts, int *status)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    ReserveShared &sh = *reinterpret_cast<ReserveShared *>(s_raw);
    const int tid = threadIdx.x, lane = tid & 31, n = p.num_seqs, shift = log2_of(p.page_size);
    const Runs run = run_of_warp(p.num_pages);
    cluster_arrive();
    bool bad = false;
    for (int i = tid; i < kSlots; i += kThreads) {
        sh.key[i] = -1;
        sh.writers[i] = 0;
        sh.first[i] = 0x7fffffff;
    }
    for (int s = tid; s < n; s += kThreads) {
        const int len = p.kv_len[s];
        const int64_t rows = (int64_t)row_start[s + 1] - row_start[s];
        int had = 0, need = 0, page = -1, holders = 0;
        if (!valid_len(p, len) || rows < 0 || rows > kMaxKeys - len || !valid_len(p, len + static_cast<int>(rows))) {
            bad = true;
        } else {
            had = pages_of(len, shift);
            need = pages_of(len + static_cast<int>(rows), shift) - had;
            if (rows > 0 && (len & (p.page_size - 1))) {
                page = p.page_table[(int64_t)s * p.table_stride + had - 1];
                if (page >= 0 && page < p.num_pages)
                    holders = __ldcg(p.refs + page);
                bad = bad || holders <= 0;
            }
        }
        sh.had[s] = had;
        sh.need[s] = need;
        sh.page[s] = page;
        sh.holders[s] = holders;
    }
    const int mine = static_cast<int>(max(run.last - run.first, (int64_t)0)) - count_held(p.refs, run, lane);
    bad = __syncthreads_or(bad);
    for (int s = tid; s < n && !bad; s += kThreads)
        if (sh.holders[s] > 1) {
            const int at = slot_of_page(sh, sh.page[s]);
            atomicAdd(&sh.writers[at], 1);
            atomicMin(&sh.first[at], s);
        }
    share_counts(sh.runs, mine, tid);  // (also: every CTA has read the lengths and the holders)
    // pages needed in the low 40 bits, copies above; a thread has two consecutive sequences
    unsigned long long own = 0;
    for (int s = 2 * tid; s < 2 * tid + 2 && s < n && !bad; ++s) {
        bool apart = false;
        if (sh.holders[s] > 1) {
            const int at = slot_of_page(sh, sh.page[s]);
            apart = sh.writers[at] < sh.holders[s] || sh.first[at] != s;
        }
        sh.need[s] += apart;
        sh.holders[s] = apart ? 0 : -1;
        own += sh.need[s] + (static_cast<unsigned long long>(apart) << 40);
    }
    unsigned long long before = threads_before(sh, own, tid);
    for (int s = 2 * tid; s < 2 * tid + 2 && s < n && !bad; ++s) {
        sh.base[s] = static_cast<int>(before & ((1ull << 40) - 1));
        const bool apart = sh.holders[s] == 0;
        sh.holders[s] = apart ? static_cast<int>(before >> 40) : -1;
        before += sh.need[s] + (static_cast<unsigned long long>(apart) << 40);
    }
    __syncthreads();
    // (row starts are of 32 bits: no more than 2^28 pages and one per sequence)
    const int needed = static_cast<int>(sh.total & ((1ull << 40) - 1));
    const int num_free = counted(sh.runs);
    const bool lead = cluster_rank() == 0;
    if (bad || needed > num_free) {
        if (lead && tid == 0) {
            set_status(status, kStatusBadArg);
            counts[0] = 0;
            counts[1] = bad ? -1 : num_free - needed;
        }
        return;
    }
    if (lead) {
        for (int s = tid; s < n; s += kThreads)
            p.kv_len[s] += row_start[s + 1] - row_start[s];
        if (tid == 0) {
            counts[0] = static_cast<int>(sh.total >> 40);
            counts[1] = num_free - needed;
        }
    }
    int rank = counted_before(sh.runs, tid >> 5);
    for (int64_t at = run.first; at < run.last && rank < needed; at += kChunk) {
        const int64_t page0 = at + 32 * lane;
        uint32_t free = ~held_pages(p.refs, at, run.last, lane) & below(page0, run.last);
        int all;
        int r = rank + lanes_before(__popc(free), lane, &all);
        rank += all;
        if (!free || r >= needed)
            continue;
        // the last sequence whose pages begin at rank r or before; the next ones follow
        int s = 0, end = n;
        while (end - s > 1) {
            const int mid = (s + end) / 2;
            if (sh.base[mid] <= r)
                s = mid;
            else
                end = mid;
        }
        int base = sh.base[s], next = base + sh.need[s];
        for (; free && r < needed; free &= free - 1, ++r) {
            const int page = static_cast<int>(page0) + __ffs(free) - 1;
            while (r >= next) {
                base = next;
                next += sh.need[++s];
            }
            const int copy = sh.holders[s];
            if (copy >= 0 && r == base) {
                copies[2 * copy] = sh.page[s];
                copies[2 * copy + 1] = page;
                atomicAdd(p.refs + sh.page[s], -1);
            }
            p.page_table[(int64_t)s * p.table_stride + sh.had[s] + (r - base) - (copy >= 0)] = page;
            p.refs[page] = 1;
        }
    }
}

// ---------------------------------------------------------------- compact

struct CompactShared {
    RunCounts runs;
    int under;                 // held pages below n
    int most;                  // pages of the longest sequence
    int pages[SMOE_MAX_SEQS];  // of each one
};

// The two ends of the moves are found by rank, each for itself; then the moves
// are gone through as a list.  While the tables are looked through, the entry
// of a moved page in refs_out (which will be 0) says where it went.
__device__ __forceinline__ int went_to(int page) { return -1 - page; }

__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(const smoe_page_pool p, int32_t *refs_out, int32_t *table_out, int32_t *copies,
                   int32_t *counts, int *status)
{
    __shared__ CompactShared sh;
    const int tid = threadIdx.x, lane = tid & 31, shift = log2_of(p.page_size);
    const Runs run = run_of_warp(p.num_pages);
    cluster_arrive();
    if (tid == 0)
        sh.most = 0;
    const int mine = count_held(p.refs, run, lane);
    share_counts(sh.runs, mine, tid);
    const int n = counted(sh.runs), before = counted_before(sh.runs, tid >> 5);
    // The free pages below n, by their rank among the free.
    int held_before = before;
    for (int64_t at = run.first; at < run.last && at < n; at += kChunk) {
        const int64_t page0 = at + 32 * lane;
        const uint32_t in = below(page0, min(run.last, (int64_t)n));
        const uint32_t held = held_pages(p.refs, at, run.last, lane) & in;
        int all;
        int64_t to = page0 - held_before - lanes_before(__popc(held), lane, &all);
        held_before += all;
        for (uint32_t free = ~held & in; free; free &= free - 1) {
            const int i = __ffs(free) - 1;
            copies[2 * (to + i - __popc(held & ((1u << i) - 1))) + 1] = static_cast<int>(page0) + i;
        }
    }
    // The run that page n lies in (or the end of the last one) tells how many are held below n.
    if (lane == 0 && run.first < run.last && n >= run.first && (n < run.last || run.last == p.num_pages))
        for (unsigned r = 0; r < cluster_size(); ++r)
            store_to_rank(&sh.under, r, held_before);
    for (int s = tid; s < p.num_seqs; s += kThreads) {
        const int len = p.kv_len[s];
        const bool ok = valid_len(p, len);
        sh.pages[s] = ok ? pages_of(len, shift) : 0;
        if (!ok)
            set_status(status, kStatusBadArg);
        atomicMax(&sh.most, sh.pages[s]);
    }
    cluster_sync();
    const int moves = n - sh.under;
    if (cluster_rank() == 0 && tid == 0) {
        counts[0] = moves;
        counts[1] = n;
    }
    // The held pages from n on, by their rank.
    int rank = max(before - sh.under, 0);
    for (int64_t at = run.first; at < run.last; at += kChunk) {
        if (at + kChunk <= n)
            continue;
        const int64_t page0 = at + 32 * lane;
        uint32_t held = held_pages(p.refs, at, run.last, lane) & ~below(page0, n);
        int all;
        int r = rank + lanes_before(__popc(held), lane, &all);
        rank += all;
        for (; held; held &= held - 1, ++r)
            copies[2 * (int64_t)r] = static_cast<int>(page0) + __ffs(held) - 1;
    }
    // What stays where it is (the free pages below n are written below).
    const int first = cluster_rank() * kThreads + tid, step = cluster_size() * kThreads;
    if (refs_out != p.refs)
        for (int64_t q = first; q < p.num_pages; q += step) {
            const int c = __ldcg(p.refs + q);
            if (q >= n || c > 0)
                refs_out[q] = q < n ? c : 0;
        }
    cluster_sync();
    for (int i = first; i < moves; i += step) {
        const int2 m = __ldcg(reinterpret_cast<const int2 *>(copies) + i);
        refs_out[m.y] = __ldcg(p.refs + m.x);
        refs_out[m.x] = went_to(m.y);
    }
    cluster_sync();
    // The tables: some columns of a row for each warp.
    constexpr int kEach = 8;
    const int warps = cluster_size() * kWarps, wide = (sh.most + 32 * kEach - 1) / (32 * kEach);
    for (int u = cluster_rank() * kWarps + (tid >> 5); u < wide * p.num_seqs; u += warps) {
        const int s = u % p.num_seqs, pages = sh.pages[s];
        const int j0 = u / p.num_seqs * 32 * kEach + lane;
        const int64_t row = (int64_t)s * p.table_stride;
        int page[kEach], to[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            page[i] = j0 + 32 * i < pages ? p.page_table[row + j0 + 32 * i] : 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            to[i] = -1;
            if (page[i] >= n && page[i] < p.num_pages)
                to[i] = __ldcg(refs_out + page[i]);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (j0 + 32 * i >= pages)
                continue;
            int now = page[i];
            if (now < 0 || now >= p.num_pages || (now >= n && to[i] >= 0))
                set_status(status, kStatusBadArg);
            else if (now >= n)
                now = went_to(to[i]);
            if (now != page[i] || table_out != p.page_table)
                table_out[row + j0 + 32 * i] = now;
        }
    }
    cluster_sync();
    for (int i = first; i < moves; i += step)
        refs_out[__ldcg(copies + 2 * (int64_t)i)] = 0;
}

// ------------------------------------------------------------------- copy

// Bound: HBM, each page is read and written once.  A unit is 16 KB of one
// page's keys or values in one cache.
constexpr int kCopyThreads = 256;
constexpr int kUnitWords = 1024;  // of 16 bytes

struct CopyArgs {
    const uint4 *k[SMOE_MAX_CACHES], *v[SMOE_MAX_CACHES];
    int64_t k_stride, v_stride;  // words
    int page_words, units;       // of a page's keys
    int num_caches, max_copies, num_pages;
};

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ CopyArgs a, const int32_t *copies, const int32_t *counts, int *status)
{
    const int asked = counts[0];
    const int n = min(max(asked, 0), a.max_copies);
    if (asked != n && blockIdx.x == 0 && threadIdx.x == 0)
        set_status(status, kStatusBadArg);
    const int64_t per_copy = (int64_t)a.num_caches * 2 * a.units;
    for (int64_t u = blockIdx.x; u < n * per_copy; u += gridDim.x) {
        const int i = static_cast<int>(u / per_copy);
        int rest = static_cast<int>(u - i * per_copy);
        const int unit = rest % a.units;
        rest /= a.units;
        const int cache = rest >> 1;
        const bool keys = (rest & 1) == 0;
        const int from = copies[2 * (int64_t)i], to = copies[2 * (int64_t)i + 1];
        if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages) {
            set_status(status, kStatusBadArg);
            continue;
        }
        uint4 *base = const_cast<uint4 *>(keys ? a.k[cache] : a.v[cache]);
        const int64_t stride = keys ? a.k_stride : a.v_stride;
        const uint4 *src = base + from * stride;
        uint4 *dst = base + to * stride;
        const int end = min((unit + 1) * kUnitWords, a.page_words);
        constexpr int kEach = kUnitWords / kCopyThreads;
        uint4 w[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int at = unit * kUnitWords + k * kCopyThreads + threadIdx.x;
            if (at < end)
                w[k] = __ldcs(src + at);
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int at = unit * kUnitWords + k * kCopyThreads + threadIdx.x;
            if (at < end)
                dst[at] = w[k];
        }
    }
}

// One cluster of at most kMaxCluster CTAs.
template <class... Params, class... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), int ctas, int smem, const DeviceFacts &dev, cudaStream_t stream,
                           Args... args)
{
    static std::atomic<bool> allowed[kMaxDeviceIndex];  // (of each kernel: they differ in their parameters)
    if (!allowed[dev.index].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && smem > 0)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess)
            return e;
        allowed[dev.index].store(true, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The power of two that n pieces of work keep busy.
int cluster_for(int64_t n)
{
    int c = 1;
    while (c < kMaxCluster && c < n)
        c *= 2;
    return c;
}

}  // namespace

cudaError_t launch_pages_fork(const smoe_page_pool &p, const int32_t *parent, const int32_t *keep,
                              const DeviceFacts &dev, cudaStream_t stream)
{
    const int64_t entries = (int64_t)p.num_seqs * p.table_stride;
    return launch_cluster(fork_kernel, cluster_for(entries / 4096), 0, dev, stream, p, parent, keep, dev.status);
}

cudaError_t launch_pages_reserve(const smoe_page_pool &p, const int32_t *row_start, int32_t *copies,
                                 int32_t *counts, const DeviceFacts &dev, cudaStream_t stream)
{
    return launch_cluster(reserve_kernel, cluster_for(p.num_pages / 8192), sizeof(ReserveShared), dev, stream, p,
                          row_start, copies, counts, dev.status);
}

cudaError_t launch_pages_compact(const smoe_page_pool &p, int32_t *refs_out, int32_t *table_out, int32_t *copies,
                                 int32_t *counts, const DeviceFacts &dev, cudaStream_t stream)
{
    const int64_t work = p.num_pages / 8192 + (int64_t)p.num_seqs * p.table_stride / 8192;
    return launch_cluster(compact_kernel, cluster_for(work), 0, dev, stream, p, refs_out, table_out, copies, counts,
                          dev.status);
}

cudaError_t launch_pages_copy(const smoe_kv_cache *caches, int num_caches, const int32_t *copies,
                              const int32_t *counts, int max_copies, const DeviceFacts &dev, cudaStream_t stream)
{
    CopyArgs a;
    const smoe_kv_cache &c = caches[0];
    for (int i = 0; i < num_caches; ++i) {
        a.k[i] = static_cast<const uint4 *>(caches[i].k_pages);
        a.v[i] = static_cast<const uint4 *>(caches[i].v_pages);
    }
    a.k_stride = c.k_page_stride / 8;
    a.v_stride = c.v_page_stride / 8;
    const int64_t words = (int64_t)c.num_kv_heads * c.page_size * c.head_dim / 8;
    a.page_words = static_cast<int>(words);
    a.units = static_cast<int>((words + kUnitWords - 1) / kUnitWords);
    a.num_caches = num_caches;
    a.max_copies = max_copies;
    a.num_pages = static_cast<int>(c.num_pages);
    const int64_t units = (int64_t)max_copies * num_caches * 2 * a.units;
    const int64_t wave = (int64_t)dev.sms * 8;
    copy_kernel<<<static_cast<unsigned>(units < wave ? units : wave), kCopyThreads, 0, stream>>>(a, copies, counts,
                                                                                              dev.status);
    return cudaGetLastError();
}

}  // namespace smoe
