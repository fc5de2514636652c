// pages.cu -- upkeep of a paged cache's pages: smoe_pages_fork,
// smoe_pages_reserve, smoe_pages_compact (whole numbers only) and
// smoe_pages_copy.
//
// The first three change a few arrays of a pool, at most of some MB, in steps
// that need one another's results.  Each runs as one thread-block cluster: its
// barrier is the hardware's and its words pass through shared memory, so a call
// is one launch (a large pool's compaction: four), needs no workspace, and nothing
// of one launch is left for the next to find.  Clusters have up to 16 CTAs (8 take
// 13.1 us instead of 10.0 for the chunks below, 17.4 instead of 14.1 for the larger
// compaction).
//
// Bound: chains of loads and barriers (an L2 load 700 to 1,000 cycles, a barrier
// of the cluster with what was written before it about as much), and issue
// slots where one cluster goes over a whole table.  Measured on the device:
// 4 sequences reordered 2.5 us, 512 of up to 16,001 keys 5.7 us; a step of 240
// beams cut back, reordered and extended 10.4 us in two calls (fork 3.9, reserve
// of no rows 4.0); chunks of 200 prompts in a pool of 430,000 pages 10.0 us in
// two calls; a pool of 1,100 pages compacted 7.1 us, one of 336,000 with 32,500
// moves 14.1 us.  A call's instructions are read from L2 once each, a latency at
// a time, so loops over chunks and passes are not unrolled (the smaller
// compaction 7.5 us unrolled).
#include <limits.h>

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
// all sequences: it reads what was there, waits for its own threads, and writes.
// An entry that changes takes a holder from its old page and gives one to the
// new (whole numbers: the order of the additions does not matter).  Beams share
// most of their pages, and entries that stay the same cost two reads only.
//
// The rows that may change are listed; of a tile of columns, their entries as
// they were and those of their parents come to shared memory together, by
// cp.async.
constexpr int kForkBytes = 96 << 10;  // of both, unless 8 columns take more

struct ForkRow {
    int seq, parent, was, now;  // pages
};

struct ForkShared {
    ForkRow row[SMOE_MAX_SEQS];
    int len[SMOE_MAX_SEQS];
    int rows, most;  // rows listed, pages of the longest of them
};

// Columns of a tile (its logarithm).
__host__ __device__ inline int fork_columns(int num_seqs)
{
    int shift = 3;
    while (shift < 9 && (8 * num_seqs << (shift + 1)) <= kForkBytes)
        ++shift;
    return shift;
}

__device__ __forceinline__ void copy_word(int *to, const int32_t *from)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

__device__ __forceinline__ void add_holder(const smoe_page_pool &p, int page, int by, int *status)
{
    if (page >= 0 && page < p.num_pages)
        atomicAdd(p.refs + page, by);
    else
        set_status(status, kStatusBadArg);
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const smoe_page_pool p, const int32_t *parent, const int32_t *keep, int *status)
{
    __shared__ ForkShared sh;
    extern __shared__ __align__(16) int s_entries[];
    const int tid = threadIdx.x, n = p.num_seqs, shift = log2_of(p.page_size);
    if (tid == 0)
        sh.rows = sh.most = 0;
    pdl_wait();
    pdl_launch_dependents();
    bool bad = false;
    int from_seq[2], was[2], len[2];  // a thread has sequences tid and tid + kThreads
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + i * kThreads;
        if (s >= n)
            continue;
        from_seq[i] = parent[s];
        was[i] = p.kv_len[s];
        len[i] = keep ? max(keep[s], 0) : 0x7fffffff;
        sh.len[s] = was[i];
        bad = bad || from_seq[i] < -1 || from_seq[i] >= n || !valid_len(p, was[i]);
    }
    // (the same answer in every CTA: none of the arrays has been written yet)
    if (__syncthreads_or(bad)) {
        if (tid == 0)
            set_status(status, kStatusBadArg);
        return;
    }
    cluster_arrive();  // this CTA has read every length
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + i * kThreads;
        if (s >= n)
            continue;
        len[i] = from_seq[i] < 0 ? 0 : min(sh.len[from_seq[i]], len[i]);
        const ForkRow r = {s, from_seq[i], pages_of(was[i], shift), pages_of(len[i], shift)};
        if (r.parent != s ? r.was + r.now > 0 : r.was > r.now) {
            sh.row[atomicAdd(&sh.rows, 1)] = r;
            atomicMax(&sh.most, max(r.was, r.now));
        }
    }
    __syncthreads();
    const int most = sh.most, wshift = fork_columns(n), width = 1 << wshift, entries = sh.rows << wshift;
    int *before = s_entries, *after = s_entries + (n << wshift);
    for (int j0 = cluster_rank() * width; j0 < most; j0 += cluster_size() * width) {
        for (int e = tid; e < entries; e += kThreads) {
            const ForkRow r = sh.row[e >> wshift];
            const int j = j0 + (e & (width - 1));
            if (j >= r.was && j >= r.now)
                continue;
            if (j < r.was && (r.parent != r.seq || j >= r.now))
                copy_word(before + e, p.page_table + (int64_t)r.seq * p.table_stride + j);
            if (j < r.now && r.parent != r.seq)
                copy_word(after + e, p.page_table + (int64_t)r.parent * p.table_stride + j);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // (every thread's entries are here, and nothing of these columns is written yet)
        for (int e = tid; e < entries; e += kThreads) {
            const ForkRow r = sh.row[e >> wshift];
            const int j = j0 + (e & (width - 1));
            const bool goes = j < r.was && (r.parent != r.seq || j >= r.now), comes = j < r.now && r.parent != r.seq;
            if (!goes && !comes)
                continue;
            const int from = before[e], to = after[e];
            if (goes && comes && from == to)
                continue;
            if (goes)
                add_holder(p, from, -1, status);
            if (comes) {
                add_holder(p, to, 1, status);
                p.page_table[(int64_t)r.seq * p.table_stride + j] = to;
            }
        }
        __syncthreads();
    }
    cluster_wait();
    if (cluster_rank() == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (tid + i * kThreads < n)
                p.kv_len[tid + i * kThreads] = len[i];
}

// ------------------------------------------------- runs of a pool's pages

// Reserve and compact go over refs in runs of consecutive pages, one for each
// warp of the cluster, dealt to its CTAs in turn (what is asked of pages is often
// asked of the lowest), and in each run in chunks of 128 pages (L = 1) or of 1024
// (L = 8 loads in flight), by the size of the pool: of up to two chunks of 128 for
// each warp, or more (a step of 240 beams in a pool of 100,000 pages: 10.4 us
// with 128, 11.2 with 1024; chunks of 200 prompts in one of 430,000: 17.5 and 10.0).
constexpr int chunk(int L) { return 128 * L; }

struct Run {
    int64_t first, last;  // pages
};

// The length of a run.
template <int L>
__device__ __forceinline__ int64_t run_length(int num_pages)
{
    const unsigned round = cluster_size() * kWarps * chunk(L);
    return (int64_t)((static_cast<unsigned>(num_pages) + round - 1) / round) * chunk(L);
}

// Run number r.
__device__ __forceinline__ Run run_at(int64_t length, int r, int num_pages)
{
    return {r * length, min((r + 1) * length, (int64_t)num_pages)};
}

// Warp w's run.
__device__ __forceinline__ int run_of_warp(int w) { return w * cluster_size() + cluster_rank(); }

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
template <int L>
__device__ __forceinline__ uint32_t held_nibbles(const int32_t *refs, int64_t at, int64_t last, int lane)
{
    int4 v[L];
    if (at + chunk(L) <= last) {  // (one condition for all loads)
#pragma unroll
        for (int i = 0; i < L; ++i)
            v[i] = __ldcg(reinterpret_cast<const int4 *>(refs + at) + 32 * i + lane);
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i)
            v[i] = refs_at(refs, at + 128 * i + 4 * lane, last);
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < L; ++i)
        w |= static_cast<uint32_t>((v[i].x > 0) | (v[i].y > 0) << 1 | (v[i].z > 0) << 2 | (v[i].w > 0) << 3) << (4 * i);
    return w;
}

// Those nibbles' pages that are below `end`.
template <int L>
__device__ __forceinline__ uint32_t nibbles_below(int64_t at, int64_t end, int lane)
{
    const int n = static_cast<int>(min(max(end - at, (int64_t)0), (int64_t)chunk(L)));
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int d = n - 128 * i - 4 * lane;
        w |= (d >= 4 ? 15u : d > 0 ? (1u << d) - 1u : 0u) << (4 * i);
    }
    return w;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// The lanes' v up to this one.
__device__ __forceinline__ int lanes_up_to(int v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        v += lane >= o ? y : 0;
    }
    return v;
}

// Where the set pages of a chunk stand among themselves, in the order of the
// pages: those of each nibble's word (32 lanes) one after the other.
template <int L>
struct Ranks {
    uint32_t before[2], total[2];  // a byte for each nibble: of the lanes before, of all lanes (at most 128)
    __device__ __forceinline__ Ranks(uint32_t w, int lane)
    {
#pragma unroll
        for (int h = 0; h < (L + 3) / 4; ++h) {
            uint32_t own = 0;
#pragma unroll
            for (int i = 4 * h; i < L && i < 4 * h + 4; ++i)
                own |= static_cast<uint32_t>(__popc(w >> (4 * i) & 15u)) << (8 * (i & 3));
            const uint32_t x = lanes_up_to(own, lane);
            before[h] = x - own;
            total[h] = __shfl_sync(0xffffffffu, x, 31);
        }
    }
    // Set pages before nibble i's first one of this lane.
    __device__ __forceinline__ int at(int i) const
    {
        const uint32_t low = i < 4 ? (1u << (8 * i)) - 1u : 0xffffffffu;
        const unsigned lanes = (L > 4 && i >= 4 ? before[1] : before[0]) >> (8 * (i & 3)) & 255u;
        const unsigned n = __dp4a(total[0] & low, 0x01010101u, lanes);
        return L > 4 && i > 4 ? __dp4a(total[1] & ((1u << (8 * (i - 4))) - 1u), 0x01010101u, n) : n;
    }
    __device__ __forceinline__ int all() const
    {
        const unsigned n = __dp4a(total[0], 0x01010101u, 0u);
        return L > 4 ? __dp4a(total[1], 0x01010101u, n) : n;
    }
};

// Held pages of a run, and (first_held) the nibbles of its first chunk.
template <int L>
__device__ __forceinline__ int count_held(const int32_t *refs, Run r, int lane, uint32_t &first_held)
{
    int n = 0;
    first_held = 0;
#pragma unroll 1
    for (int64_t at = r.first; at < r.last; at += chunk(L)) {
        const uint32_t w = held_nibbles<L>(refs, at, r.last, lane);
        first_held = at == r.first ? w : first_held;
        n += __popc(w);
    }
    return warp_sum(n);
}

// Counts of every run.
struct RunCounts {
    int own[kWarps];
    alignas(16) int run[kMaxCluster * kWarps];
};

// `mine`: the count of the warp's run, the same in all its lanes.  The kernel
// has arrived at the cluster's barrier at its start (every CTA has begun where
// that ends).  A barrier of the cluster.
__device__ __forceinline__ void share_counts(RunCounts &rc, int mine, int tid)
{
    if ((tid & 31) == 0)
        rc.own[tid >> 5] = mine;
    __syncthreads();
    cluster_wait();
    if (tid < static_cast<int>(cluster_size()) * kWarps)
        store_to_rank(&rc.run[run_of_warp(tid % kWarps)], tid / kWarps, rc.own[tid % kWarps]);
    cluster_sync();
}

// What the runs before r counted, and all of them, by a warp.
struct Counted {
    int before, all;
};
__device__ __forceinline__ Counted counted(const RunCounts &rc, int r, int lane)
{
    Counted c = {0, 0};
#pragma unroll
    for (int i = 4 * lane; i < kMaxCluster * kWarps; i += 128) {
        const int4 v = i < static_cast<int>(cluster_size()) * kWarps ? *reinterpret_cast<const int4 *>(rc.run + i)
                                                                       : make_int4(0, 0, 0, 0);
        c.all += v.x + v.y + v.z + v.w;
        c.before += (i < r ? v.x : 0) + (i + 1 < r ? v.y : 0) + (i + 2 < r ? v.z : 0) + (i + 3 < r ? v.w : 0);
    }
    return {warp_sum(c.before), warp_sum(c.all)};
}

// ---------------------------------------------------------------- reserve

// Every CTA finds out for itself what each sequence needs, while the pool is
// counted in runs; then the free pages' ranks are known, and each one below
// the number needed looks up whose it is.
constexpr int kSlots = 2 * SMOE_MAX_SEQS;  // of the table of shared last pages

// What a sequence gets, for those that get any.
struct Given {
    int end;    // free pages given to the sequences up to it
    int seq;
    int entry;  // of its row: the first one's
    int copy;   // the place of its copy in the list, -1: none
};

struct ReserveShared {
    RunCounts runs;
    Given given[SMOE_MAX_SEQS];
    int page[SMOE_MAX_SEQS];      // a partly filled last page that is to be written, else -1
    int holders[SMOE_MAX_SEQS];   // of it
    int had[SMOE_MAX_SEQS];       // pages
    int need[SMOE_MAX_SEQS];
    int key[kSlots], writers[kSlots], first[kSlots];
    int warp_need[kWarps], warp_copies[kWarps];
    uint32_t free[kWarps][32];    // of each run's chunk: the lanes' nibbles
    int rank[kWarps];             // of its first free page
};

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

template <int L>
__global__ void __launch_bounds__(kThreads, 1)
    reserve_kernel(const smoe_page_pool p, const int32_t *row_start, int32_t *copies, int32_t *counts, int *status)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    ReserveShared &sh = *reinterpret_cast<ReserveShared *>(s_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.num_seqs, shift = log2_of(p.page_size);
    const int64_t length = run_length<L>(p.num_pages);
    const Run run = run_at(length, run_of_warp(warp), p.num_pages);
    cluster_arrive();
    bool bad = false;
    for (int i = tid; i < kSlots; i += kThreads) {
        sh.key[i] = -1;
        sh.writers[i] = 0;
        sh.first[i] = 0x7fffffff;
    }
    pdl_wait();
    pdl_launch_dependents();
    // A thread has sequences tid and tid + kThreads.  Their lengths, last pages
    // and those pages' holders come one after the other; the pool is counted meanwhile.
    int had[2], page[2], new_pages[2], holders[2], grown[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + i * kThreads;
        had[i] = new_pages[i] = holders[i] = grown[i] = 0;
        page[i] = -1;
        if (s >= n)
            continue;
        const int len = p.kv_len[s];
        const int64_t rows = (int64_t)row_start[s + 1] - row_start[s];
        if (!valid_len(p, len) || rows < 0 || rows > kMaxKeys - len || !valid_len(p, len + static_cast<int>(rows))) {
            bad = true;
            continue;
        }
        grown[i] = len + static_cast<int>(rows);
        had[i] = pages_of(len, shift);
        new_pages[i] = pages_of(len + static_cast<int>(rows), shift) - had[i];
        if (rows > 0 && (len & (p.page_size - 1))) {
            page[i] = __ldcg(p.page_table + (int64_t)s * p.table_stride + had[i] - 1);
            holders[i] = -1;  // (to be looked up)
        }
    }
    uint32_t held;
    const int mine = static_cast<int>(max(run.last - run.first, (int64_t)0)) - count_held<L>(p.refs, run, lane, held);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (holders[i] < 0 && page[i] >= 0 && page[i] < p.num_pages)
            holders[i] = __ldcg(p.refs + page[i]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = tid + i * kThreads;
        if (s >= n)
            continue;
        bad = bad || holders[i] < 0 || (page[i] >= 0 && holders[i] == 0);
        sh.had[s] = had[i];
        sh.need[s] = new_pages[i];
        sh.page[s] = page[i];
        sh.holders[s] = holders[i];
    }
    bad = __syncthreads_or(bad);
    for (int s = tid; s < n && !bad; s += kThreads)
        if (sh.holders[s] > 1) {
            const int at = slot_of_page(sh, sh.page[s]);
            atomicAdd(&sh.writers[at], 1);
            atomicMin(&sh.first[at], s);
        }
    share_counts(sh.runs, mine, tid);  // (also: every CTA has read the lengths and the holders)
    // A thread has two consecutive sequences.
    int need[2] = {0, 0}, copy[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = 2 * tid + i;
        if (s < n && !bad) {
            if (sh.holders[s] > 1) {
                const int at = slot_of_page(sh, sh.page[s]);
                copy[i] = sh.writers[at] < sh.holders[s] || sh.first[at] != s;
            }
            need[i] = sh.need[s] + copy[i];
        }
    }
    // (row starts are of 32 bits: no more than 2^28 pages and one per sequence)
    // (copies, and above them in the same words, sequences that get pages)
    const int own = copy[0] + copy[1] + ((need[0] > 0) + (need[1] > 0) << 16);
    int end = lanes_up_to(need[0] + need[1], lane), place = lanes_up_to(own, lane);
    if (lane == 31) {
        sh.warp_need[warp] = end;
        sh.warp_copies[warp] = place;
    }
    __syncthreads();
    const int others = sh.warp_need[lane], other_copies = sh.warp_copies[lane];
    const int needed = warp_sum(others), counted_all = warp_sum(other_copies);
    const int num_copies = counted_all & 0xffff, num_given = counted_all >> 16;
    end += warp_sum(lane < warp ? others : 0);
    place += warp_sum(lane < warp ? other_copies : 0) - own;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = 2 * tid + i;
        if (need[i] > 0) {
            sh.given[place >> 16] = {i == 0 ? end - need[1] : end, s, sh.had[s] - copy[i],
                                     copy[i] ? place & 0xffff : -1};
            place += copy[i] + (1 << 16);
        }
    }
    __syncthreads();
    const Counted free_pages = counted(sh.runs, run_of_warp(warp), lane);
    const int num_free = free_pages.all;
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
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (tid + i * kThreads < n)
                p.kv_len[tid + i * kThreads] = grown[i];
        if (tid == 0) {
            counts[0] = num_copies;
            counts[1] = num_free - needed;
        }
    }
    // Gives the free pages of a chunk's slice away; w: the chunk's free ones,
    // the first of rank `rank`.
    const auto give = [&](int64_t at, int slice, uint32_t w, int rank) {
        int k = rank + Ranks<L>(w, lane).at(slice);
        unsigned free = w >> (4 * slice) & 15u;
        if (!free || k >= needed)
            return;
        // the first sequence whose pages end behind rank k; the next ones follow
        int at_given = 0;
        for (int hi = num_given - 1; at_given < hi;) {
            const int mid = (at_given + hi) / 2;
            if (sh.given[mid].end > k)
                hi = mid;
            else
                at_given = mid + 1;
        }
        Given g = sh.given[at_given];
        int begin = at_given > 0 ? sh.given[at_given - 1].end : 0;
        for (; free && k < needed; free &= free - 1, ++k) {
            const int page = static_cast<int>(at) + 128 * slice + 4 * lane + __ffs(free) - 1;
            if (k >= g.end) {
                begin = g.end;
                g = sh.given[++at_given];
            }
            if (g.copy >= 0 && k == begin) {
                const int old = sh.page[g.seq];
                copies[2 * g.copy] = old;
                copies[2 * g.copy + 1] = page;
                atomicAdd(p.refs + old, -1);
            }
            p.page_table[(int64_t)g.seq * p.table_stride + g.entry + (k - begin)] = page;
            p.refs[page] = 1;
        }
    };
    // Each warp looks at its own run, chunk by chunk, before any page of the
    // chunk is given away: what is given is held from then on.  With L > 1 the
    // chunks of the CTA's runs are then dealt out by slices, so that no lane has
    // more than 4 pages to give.
    int rank = free_pages.before;
    for (int64_t at = run.first;; at += chunk(L)) {
        const bool more = at < run.last && rank < needed;
        if (L > 1 ? !__syncthreads_or(more) : !more)
            break;
        if (more && at > run.first)
            held = held_nibbles<L>(p.refs, at, run.last, lane);
        const uint32_t free = more ? ~held & nibbles_below<L>(at, run.last, lane) : 0;
        const int first = rank;
        rank += warp_sum(__popc(free));
        if (L == 1) {
            give(at, 0, free, first);
            continue;
        }
        sh.free[warp][lane] = free;
        sh.rank[warp] = first;
        __syncthreads();
        for (int t = warp; t < kWarps * L && sh.rank[t / L] < needed; t += kWarps)
            give(run_of_warp(t / L) * length + (at - run.first), t % L, sh.free[t / L][lane], sh.rank[t / L]);
    }
}

// ---------------------------------------------------------------- compact

// The two ends of the moves are found by rank, each for itself, by a cluster;
// then the moves are gone through as a list, and the tables.  Meanwhile the
// entry of a moved page in refs_out (which will be 0) says where it went.  A
// small pool's are done with by the same cluster; a large one's by launches of
// the whole device (336,000 pages, 480 sequences: 14.1 us; by the cluster 24.9).
constexpr int kBatch = 4;  // loads of a thread that are in flight together
constexpr int kColumns = 128;

// (of a page that is free: no count is below -2^30, so that none is taken for this)
__device__ __forceinline__ int went_to(int page) { return INT_MIN + page; }
__device__ __forceinline__ bool is_told(int mark, int n) { return mark < INT_MIN + n; }
__device__ __forceinline__ int told(int mark) { return mark - INT_MIN; }

// What stays where it is, into other refs: a thread of `step` has number `first`.
__device__ __forceinline__ void stay_pass(const smoe_page_pool &p, int32_t *refs_out, int n, int64_t first, int64_t step)
{
    const bool whole = (reinterpret_cast<uintptr_t>(refs_out) & 15) == 0;
#pragma unroll 1
    for (int64_t q = 4 * first; q < p.num_pages; q += 4 * step) {
        const int4 v = refs_at(p.refs, q, p.num_pages);
        if (whole && q >= n && q + 4 <= p.num_pages && v.x <= 0 && v.y <= 0 && v.z <= 0 && v.w <= 0) {
            *reinterpret_cast<int4 *>(refs_out + q) = make_int4(0, 0, 0, 0);
            continue;
        }
        const int c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int d = 0; d < 4; ++d)  // (moved pages and those that they come to are told by move_pass)
            if (q + d < p.num_pages && (q + d < n) == (c[d] > 0))
                refs_out[q + d] = q + d < n ? c[d] : 0;
    }
}

__device__ __forceinline__ void move_pass(const smoe_page_pool &p, int32_t *refs_out, const int32_t *copies, int moves,
                                          int first, int step)
{
#pragma unroll 1
    for (int i0 = first; i0 < moves; i0 += kBatch * step) {
        int2 m[kBatch];
        int c[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            m[i] = __ldcg(reinterpret_cast<const int2 *>(copies) + min(i0 + i * step, moves - 1));
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            c[i] = __ldcg(p.refs + m[i].x);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (i0 + i * step < moves) {
                refs_out[m[i].y] = c[i];
                refs_out[m[i].x] = went_to(m[i].y);
            }
    }
}

// Entries j0 + 32 i of a row of `pages`, by a warp.  (Past the last entry the
// lanes do that one again.)
__device__ __forceinline__ void table_pass(const smoe_page_pool &p, const int32_t *refs_out, int32_t *table_out, int n,
                                           int s, int pages, int j0, int *status)
{
    const int64_t row = (int64_t)s * p.table_stride;
    const int32_t *from = p.page_table + row;
    int32_t *out = table_out + row;
    int page[kColumns / 32], to[kColumns / 32];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kColumns / 32; ++i)
        page[i] = __ldcg(from + min(j0 + 32 * i, pages - 1));
#pragma unroll
    for (int i = 0; i < kColumns / 32; ++i)
        to[i] = __ldcg(refs_out + (page[i] >= n && page[i] < p.num_pages ? page[i] : 0));
#pragma unroll
    for (int i = 0; i < kColumns / 32; ++i) {
        const bool above = page[i] >= n && page[i] < p.num_pages;
        bad = bad || static_cast<unsigned>(page[i]) >= static_cast<unsigned>(p.num_pages) || (above && !is_told(to[i], n));
        out[min(j0 + 32 * i, pages - 1)] = above && is_told(to[i], n) ? told(to[i]) : page[i];
    }
    if (bad)
        set_status(status, kStatusBadArg);
}

__device__ __forceinline__ void clear_pass(int32_t *refs_out, const int32_t *copies, int moves, int first, int step)
{
#pragma unroll 1
    for (int i0 = first; i0 < moves; i0 += kBatch * step) {
        int from[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            from[i] = __ldcg(copies + 2 * (int64_t)min(i0 + i * step, moves - 1));
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            refs_out[from[i]] = 0;  // (the last one more than once)
    }
}

struct CompactShared {
    RunCounts runs;
    int under;  // held pages below n
};

// ALONE: with the passes.
template <int L, bool ALONE>
__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(const smoe_page_pool p, int32_t *refs_out, int32_t *table_out, int32_t *copies,
                   int32_t *counts, int *status)
{
    __shared__ CompactShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Run run = run_at(run_length<L>(p.num_pages), run_of_warp(warp), p.num_pages);
    cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    uint32_t first_held;
    const int mine = count_held<L>(p.refs, run, lane, first_held);
    share_counts(sh.runs, mine, tid);
    const Counted held_pages = counted(sh.runs, run_of_warp(warp), lane);
    const int n = held_pages.all, before = held_pages.before;
    // The free pages below n, by their rank among the free.
    int64_t held_before = before;
#pragma unroll 1
    for (int64_t at = run.first; at < run.last && at < n; at += chunk(L)) {
        const uint32_t in = nibbles_below<L>(at, min(run.last, (int64_t)n), lane);
        const uint32_t held = (at == run.first ? first_held : held_nibbles<L>(p.refs, at, run.last, lane)) & in;
        const Ranks<L> ranks(~held & in, lane);
        const int64_t to = at - held_before;  // free pages before the chunk
#pragma unroll
        for (int i = 0; i < L; ++i) {
            int32_t *k = copies + 2 * (to + ranks.at(i)) + 1;
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if ((~held & in) >> (4 * i + d) & 1) {
                    *k = static_cast<int>(at) + 128 * i + 4 * lane + d;
                    k += 2;
                }
        }
        held_before += warp_sum(__popc(held));
    }
    // The run that page n lies in (or the end of the last one) tells how many are held below n.
    if (lane < static_cast<int>(cluster_size()) && run.first < run.last && n >= run.first &&
        (n < run.last || run.last == p.num_pages))
        store_to_rank(&sh.under, lane, static_cast<int>(held_before));
    cluster_sync();
    const int moves = n - sh.under;
    if (cluster_rank() == 0 && tid == 0) {
        counts[0] = moves;
        counts[1] = n;
    }
    // The held pages from n on, by their rank.
    int64_t rank = max(before - sh.under, 0);
#pragma unroll 1
    for (int64_t at = run.first; at < run.last; at += chunk(L)) {
        if (at + chunk(L) <= n)
            continue;
        const uint32_t held = (at == run.first ? first_held : held_nibbles<L>(p.refs, at, run.last, lane)) &
                              ~nibbles_below<L>(at, n, lane);
        const Ranks<L> ranks(held, lane);
#pragma unroll
        for (int i = 0; i < L; ++i) {
            int32_t *k = copies + 2 * (rank + ranks.at(i));
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (held >> (4 * i + d) & 1) {
                    *k = static_cast<int>(at) + 128 * i + 4 * lane + d;
                    k += 2;
                }
        }
        rank += ranks.all();
    }
    if (!ALONE)
        return;
    cluster_sync();
    const int first = cluster_rank() * kThreads + tid, step = cluster_size() * kThreads;
    if (refs_out != p.refs)
        stay_pass(p, refs_out, n, first, step);
    move_pass(p, refs_out, copies, moves, first, step);
    cluster_sync();
    const int shift = log2_of(p.page_size), warps = cluster_size() * kWarps;
    const int wide = max((p.table_stride + kColumns - 1) / kColumns, 1);  // (lengths are looked at without columns too)
#pragma unroll 1
    for (int u = cluster_rank() * kWarps + warp; u < wide * p.num_seqs; u += warps) {
        const int s = u / wide, j0 = u % wide * kColumns, len = p.kv_len[s];
        if (!valid_len(p, len))
            set_status(status, kStatusBadArg);
        else if (j0 < pages_of(len, shift))
            table_pass(p, refs_out, table_out, n, s, pages_of(len, shift), j0 + lane, status);
    }
    cluster_sync();
    clear_pass(refs_out, copies, moves, first, step);
}

constexpr int kPassThreads = 256;

// The passes of a large pool.
__global__ void __launch_bounds__(kPassThreads)
    move_kernel(const smoe_page_pool p, int32_t *refs_out, const int32_t *copies, const int32_t *counts)
{
    pdl_wait();
    pdl_launch_dependents();
    const int first = blockIdx.x * kPassThreads + threadIdx.x, step = gridDim.x * kPassThreads;
    if (refs_out != p.refs)
        stay_pass(p, refs_out, counts[1], first, step);
    move_pass(p, refs_out, copies, counts[0], first, step);
}

__global__ void __launch_bounds__(kPassThreads)
    table_kernel(const smoe_page_pool p, const int32_t *refs_out, int32_t *table_out, const int32_t *counts, int *status)
{
    pdl_wait();
    pdl_launch_dependents();
    const int s = blockIdx.y, len = p.kv_len[s], n = counts[1];
    if (!valid_len(p, len)) {
        set_status(status, kStatusBadArg);
        return;
    }
    const int pages = pages_of(len, log2_of(p.page_size)), lane = threadIdx.x & 31;
    const int warps = gridDim.x * (kPassThreads / 32);
    for (int j0 = (blockIdx.x * (kPassThreads / 32) + (threadIdx.x >> 5)) * kColumns; j0 < pages; j0 += warps * kColumns)
        table_pass(p, refs_out, table_out, n, s, pages, j0 + lane, status);
}

__global__ void __launch_bounds__(kPassThreads)
    clear_kernel(int32_t *refs_out, const int32_t *copies, const int32_t *counts)
{
    pdl_wait();
    pdl_launch_dependents();
    clear_pass(refs_out, copies, counts[0], blockIdx.x * kPassThreads + threadIdx.x, gridDim.x * kPassThreads);
}

// ------------------------------------------------------------------- copy

// Bound: HBM, each page is read and written once.  A unit is 16 KB of one
// page's keys or values in one cache.  Many CTAs of one to a few units each keep
// the most loads in flight: 601 pages in two layers (630 MB read and written) take
// 93.9 us, 6.7 TB/s, with 32 CTAs per SM, 103.8 us with 8 that go on and on, 93.2
// with 64.  12 pages in four layers: 2.2 us.
constexpr int kCopyThreads = 256;
constexpr int kUnitWords = 1024;  // of 16 bytes

// (arguments for 8 caches or for all: 2 KB of them make a launch longer)
template <int MOST>
struct CopyArgs {
    const uint4 *k[MOST], *v[MOST];
    int64_t k_stride, v_stride;  // words
    int page_words, units;       // of a page's keys
    int num_caches, max_copies, num_pages;
};

template <int MOST>
__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(const __grid_constant__ CopyArgs<MOST> a, const int32_t *copies, const int32_t *counts, int *status)
{
    pdl_wait();
    pdl_launch_dependents();
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
        const int first = unit * kUnitWords + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            w[k] = __ldcs(src + min(first + k * kCopyThreads, end - 1));
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (first + k * kCopyThreads < end)
                __stcs(dst + first + k * kCopyThreads, w[k]);
    }
}

// Dynamic shared memory of a CTA at most (fork: 8 columns of SMOE_MAX_SEQS rows).
constexpr int kMaxSmem = 64 * SMOE_MAX_SEQS;
static_assert(kForkBytes <= kMaxSmem && sizeof(ReserveShared) <= kMaxSmem, "shared memory");

// One cluster of at most kMaxCluster CTAs.
template <class... Params, class... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), int ctas, int smem, const DeviceFacts &dev,
                           std::atomic<bool> *allowed, cudaStream_t stream, Args... args)
{
    if (!allowed[dev.index].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) {
            (void)cudaGetLastError();
            return e;
        }
        allowed[dev.index].store(true, std::memory_order_release);
    }
    return launch_ahead(kernel, dim3(ctas), kThreads, smem, ctas, stream, args...);
}

// The power of two that n pieces of work keep busy.
int cluster_for(int64_t n)
{
    int c = 1;
    while (c < kMaxCluster && c < n)
        c *= 2;
    return c;
}

constexpr int kRound = kMaxCluster * kWarps * chunk(1);
bool small_chunks(const smoe_page_pool &p) { return p.num_pages <= 2 * kRound; }
// A pool of one round, with tables of few entries, is also compacted by the one
// launch: 1,100 pages take 7.3 us a call, and 13.4 by four launches, which the
// host takes longer for (7.5 us on the device).
bool compact_alone(const smoe_page_pool &p)
{
    return p.num_pages <= kRound && (int64_t)p.num_seqs * p.table_stride <= 1 << 16;
}
int pool_cluster(const smoe_page_pool &p)
{
    const int64_t pages = p.num_pages / (kWarps * chunk(1)), entries = (int64_t)p.num_seqs * p.table_stride / 8192;
    return cluster_for(pages > entries ? pages : entries);
}

}  // namespace

cudaError_t launch_pages_fork(const smoe_page_pool &p, const int32_t *parent, const int32_t *keep,
                              const DeviceFacts &dev, cudaStream_t stream)
{
    const int64_t entries = (int64_t)p.num_seqs * p.table_stride;
    static std::atomic<bool> allowed[kMaxDeviceIndex];
    const int smem = 8 * p.num_seqs << fork_columns(p.num_seqs);
    return launch_cluster(fork_kernel, cluster_for(entries / 4096), smem, dev, allowed, stream, p, parent, keep,
                          dev.status);
}

cudaError_t launch_pages_reserve(const smoe_page_pool &p, const int32_t *row_start, int32_t *copies,
                                 int32_t *counts, const DeviceFacts &dev, cudaStream_t stream)
{
    const auto go = [&](auto *kernel, std::atomic<bool> *allowed) {
        return launch_cluster(kernel, pool_cluster(p), sizeof(ReserveShared), dev, allowed, stream, p, row_start, copies,
                              counts, dev.status);
    };
    static std::atomic<bool> allowed[2][kMaxDeviceIndex];
    return small_chunks(p) ? go(reserve_kernel<1>, allowed[0]) : go(reserve_kernel<8>, allowed[1]);
}

cudaError_t launch_pages_compact(const smoe_page_pool &p, int32_t *refs_out, int32_t *table_out, int32_t *copies,
                                 int32_t *counts, const DeviceFacts &dev, cudaStream_t stream)
{
    const bool alone = compact_alone(p);
    const auto go = [&](auto *kernel, std::atomic<bool> *allowed) {
        return launch_cluster(kernel, pool_cluster(p), 0, dev, allowed, stream, p, refs_out, table_out, copies, counts,
                              dev.status);
    };
    static std::atomic<bool> allowed[3][kMaxDeviceIndex];
    cudaError_t e = alone             ? go(compact_kernel<1, true>, allowed[0])
                    : small_chunks(p) ? go(compact_kernel<1, false>, allowed[1])
                                      : go(compact_kernel<8, false>, allowed[2]);
    if (alone)
        return e;
    const auto pass = [&](dim3 grid, auto *kernel, auto... args) {
        if (e == cudaSuccess)
            e = launch_ahead(kernel, grid, kPassThreads, 0, 0, stream, args...);
    };
    pass(dim3(dev.sms * 2), move_kernel, p, refs_out, copies, counts);
    if (p.num_seqs > 0) {
        const int columns = kPassThreads / 32 * kColumns, wide = (p.table_stride + columns - 1) / columns;
        pass(dim3(wide < 1 ? 1 : wide < 64 ? wide : 64, p.num_seqs), table_kernel, p, refs_out, table_out, counts, dev.status);
    }
    pass(dim3(dev.sms), clear_kernel, refs_out, copies, counts);
    return e;
}

namespace {

template <int MOST>
cudaError_t launch_copy(const smoe_kv_cache *caches, int num_caches, const int32_t *copies, const int32_t *counts,
                        int max_copies, const DeviceFacts &dev, cudaStream_t stream)
{
    CopyArgs<MOST> a;
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
    const int64_t most = (int64_t)dev.sms * 32;
    return launch_ahead(copy_kernel<MOST>, dim3(static_cast<unsigned>(units < most ? units : most)), kCopyThreads, 0, 0,
                        stream, a, copies, counts, dev.status);
}

}  // namespace

cudaError_t launch_pages_copy(const smoe_kv_cache *caches, int num_caches, const int32_t *copies,
                              const int32_t *counts, int max_copies, const DeviceFacts &dev, cudaStream_t stream)
{
    return (num_caches <= 8 ? launch_copy<8> : launch_copy<SMOE_MAX_CACHES>)(caches, num_caches, copies, counts,
                                                                            max_copies, dev, stream);
}

}  // namespace smoe
