// attention.cu -- attention of new rows over a paged cache (smoe_attention).
//
// Mathematics: row with key index i, head h of kv head h / G:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q . k_j - m),
// over the keys i - window < j <= i, in one pass with a running maximum m
// and sum (an earlier part is multiplied by exp(m_old - m_new) where the
// maximum grows).  Exponents are taken in base 2: scale is multiplied by
// log2 e once.
//
// The G query heads of a kv head read the same keys, so the rows of one
// sequence and kv head are packed: packed row m is new row m / G, head m % G
// of the kv head.
#include <math.h>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kDecWarps = 8;   // warps per CTA, each with keys of its own
constexpr int kMmaRows = 16;   // packed rows of an mma tile (mma M)
constexpr int kDecKeys = 16;   // keys per warp and step (mma K of P V); a page holds them

// The kernel's instances by tiles per item, T: up to 16 packed rows, the
// queries in registers and three steps in flight per warp; or up to 32, the
// queries in shared memory and two steps in flight.
__host__ __device__ constexpr int dec_rows(int T) { return T * kMmaRows; }
__host__ __device__ constexpr int dec_stages(int T) { return T == 1 ? 3 : 2; }
__host__ __device__ constexpr int dec_step_bytes(int D) { return 2 * kDecKeys * D * 2; }
__host__ __device__ constexpr int dec_ring_bytes(int D, int T) { return dec_stages(T) * dec_step_bytes(D); }
__host__ __device__ constexpr int dec_query_bytes(int D, int T) { return T == 1 ? 0 : dec_rows(T) * D * 2; }
__host__ __device__ constexpr int dec_smem_bytes(int D, int T)
{
    return kDecWarps * (dec_ring_bytes(D, T) + dec_query_bytes(D, T)) + (SMOE_MAX_SEQS + 1) * 16;
}

// 16-byte chunk c of row r of a tile of 2 D bytes per row: the low three
// bits are mixed with the row's, so that the 8 rows of one ldmatrix matrix
// lie in distinct banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c)
{
    return static_cast<uint32_t>(r * (2 * D) + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;  // the rest is filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// ------------------------------------------------- few rows (decode steps)

// Sequences of at most 16 (or 32) packed rows: bound by reading the keys and
// values.  The work of a launch is one line of steps: for every sequence and
// kv head (an item) kItemSteps for its own cost (its queries, its output),
// then its keys in steps of kDecKeys.  Every warp of the grid is a worker
// with an equal share [w q, (w + 1) q) of that line, whatever the lengths,
// and copies its keys into a ring of its own that runs ahead over item
// borders; no warp waits for another one in the loop.  An item cut by shares
// is computed in parts.  Parts of one CTA are joined in shared memory, once,
// at its end; what still is a part then goes to the workspace, and the CTA
// that arrives last joins the item's parts, in CTA order.
// Bound: HBM, every visible key and value is read once.  Measured: one row on
// 500,003 keys, 32 query and 8 kv heads of 128: 320 us, 6.4 TB/s; 96 rows on 1 to
// 16,001 keys (137,853 in all), 64 and 4 heads of 128: 59 us, 4.8 TB/s, of which
// 44 stream at the copy rate and the plan, the first copies and the joins take
// the rest; 24 sequences of 5 rows on 25,667 keys, 32 and 8 heads of 128: 42.6 us,
// of which 18 stream at 5.8 TB/s (two tiles' products, a ring of two steps);
// one row on 777 keys: 12 us of latencies.
constexpr int kItemSteps = 8;
constexpr int kMaxCtas = 256;

// A sequence of the batch in shared memory, with the place of its first item
// on the line of steps.
struct RowSeq {
    int row0, rows, len;
    uint32_t at;
};

// Key steps of one item (0: no rows).  A row that sees nothing still takes a
// step: it writes its zeros.
__device__ __forceinline__ int item_steps(const smoe_attention_args &a, int rows, int len)
{
    if (rows == 0)
        return 0;
    int lo, hi, x, y;
    seen_from(a, len - rows, lo, x);
    seen_from(a, len - 1, y, hi);
    const int n = hi > lo ? (hi + kDecKeys - 1) / kDecKeys - lo / kDecKeys : 0;
    return n > 1 ? n : 1;
}

// How the line of steps is shared.
struct Share {
    uint32_t q, total;  // steps per worker, in all
    uint32_t unit;      // an item's length is rounded up to a multiple of this
};

__device__ __forceinline__ uint32_t item_length(int steps, uint32_t unit)
{
    return (steps + kItemSteps + unit - 1) / unit * unit;
}

// Steps per worker: an equal share, but no item in so many parts that the
// joining costs more than the sharing saves.  A CTA reads a part in about
// 1/8 of the time that it takes for 8 steps, so n steps are read and joined
// fastest by about sqrt(n) CTAs.
__device__ __forceinline__ uint32_t steps_per_worker(uint32_t total, int longest)
{
    const uint32_t workers = gridDim.x * kDecWarps;
    const uint32_t q = total / workers + (total % workers != 0);
    const uint32_t least = static_cast<uint32_t>(sqrtf(static_cast<float>(longest)) * 0.125f);
    return q > least ? q : (least > 1 ? least : 1);
}

// Steps of the longest line, with room below 2^32 for the rounding of a sum in
// fp32.
constexpr float kMaxLine = 4.2e9f;

// The batch into shared memory (n + 1 entries), and the shares.  Each thread
// takes `per` sequences in a row.  A batch whose line has more than kMaxLine
// steps is recorded and not worked on.
__device__ __forceinline__ Share plan(const smoe_attention_args &a, RowSeq *seqs, int *status)
{
    __shared__ uint32_t s_sum[2][kDecWarps];
    __shared__ int s_max[kDecWarps];
    __shared__ float s_all[kDecWarps];
    constexpr int kThreads = 32 * kDecWarps;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = a.batch.num_seqs, per = (n + kThreads - 1) / kThreads, Hkv = a.cache.num_kv_heads;
    // Lengths as they are, and rounded up to the steps that a CTA takes at one
    // per worker: where the grid has room for the latter, every CTA works on
    // one item only and has one join.
    uint32_t sum[2] = {0, 0};
    int mx = 0;
    float all = 0.f;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= n)
            break;
        const Seq s = seq_at(a, b, status);
        const int k = item_steps(a, s.rows, s.len);
        seqs[b].row0 = static_cast<int>(s.row0);
        seqs[b].rows = s.rows;
        seqs[b].len = s.len;
        seqs[b].at = k;
        if (k > 0) {
            sum[0] += item_length(k, 1);
            sum[1] += item_length(k, kDecWarps);
            all += static_cast<float>(item_length(k, kDecWarps)) * static_cast<float>(Hkv);
        }
        mx = k > mx ? k : mx;
    }
    uint32_t incl[2] = {sum[0], sum[1]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl[j], o);
            incl[j] += lane >= o ? v : 0;
        }
        const int m = __shfl_xor_sync(0xffffffffu, mx, o);
        mx = m > mx ? m : mx;
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    if (lane == 31) {
        s_sum[0][warp] = incl[0];
        s_sum[1][warp] = incl[1];
    }
    if (lane == 0) {
        s_max[warp] = mx;
        s_all[warp] = all;
    }
    __syncthreads();
    all = 0.f;
    uint32_t total[2] = {0, 0}, before[2] = {incl[0] - sum[0], incl[1] - sum[1]};
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            before[j] += w < warp ? s_sum[j][w] : 0;
            total[j] += s_sum[j][w];
        }
        mx = s_max[w] > mx ? s_max[w] : mx;
        all += s_all[w];
    }
    Share sh;
    sh.q = steps_per_worker(total[0] * Hkv, mx);
    const bool room = sh.q == 1 && total[1] * Hkv <= gridDim.x * kDecWarps;
    sh.unit = room ? kDecWarps : 1;
    sh.total = (room ? total[1] : total[0]) * Hkv;
    uint32_t at = (room ? before[1] : before[0]) * Hkv;
#pragma unroll 1
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= n)
            break;
        const int k = seqs[b].at;
        seqs[b].at = at;
        at += k > 0 ? item_length(k, sh.unit) * Hkv : 0;
    }
    if (tid == 0) {
        seqs[n].row0 = seqs[n].rows = seqs[n].len = 0;
        seqs[n].at = sh.total;
    }
    __syncthreads();
    if (all > kMaxLine) {  // the sums above may have wrapped
        set_status(status, kStatusBadArg);
        sh.total = 0;
    }
    return sh;
}

// A place on the line of steps, at an item.
struct Cursor {
    int row0, rows, len;  // its sequence (rows 0: past the last)
    int b, h, steps;      // key steps of the item
    uint32_t len_line;    // its length on the line
    uint32_t at;          // its first step on the line
    int k_lo, k_hi;       // keys seen by any of its rows
};

__device__ __forceinline__ void cursor_seq(const smoe_attention_args &a, const Share &sh, const RowSeq *seqs,
                                           Cursor &c)
{
    c.row0 = seqs[c.b].row0;
    c.rows = seqs[c.b].rows;
    c.len = seqs[c.b].len;
    c.steps = item_steps(a, c.rows, c.len);
    c.len_line = item_length(c.steps, sh.unit);
    int x, y;
    seen_from(a, c.len - c.rows, c.k_lo, x);
    seen_from(a, c.len - 1, y, c.k_hi);
}

__device__ __forceinline__ Cursor cursor_at(const smoe_attention_args &a, const Share &sh, const RowSeq *seqs,
                                            uint32_t w0)
{
    Cursor c;
    int lo = 0, hi = a.batch.num_seqs;  // the last sequence that begins at or before w0
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seqs[mid].at <= w0)
            lo = mid;
        else
            hi = mid - 1;
    }
    c.b = lo;
    cursor_seq(a, sh, seqs, c);
    c.h = c.rows ? (w0 - seqs[lo].at) / c.len_line : 0;
    c.at = seqs[lo].at + c.h * c.len_line;
    return c;
}

// Where the border between two shares that nominally lies at x, in the
// cursor's item, is drawn: at x, or at the nearer end of an item of at most
// half a share, which is not worth being cut.
__device__ __forceinline__ uint32_t border(const Share &sh, const Cursor &c, uint32_t x)
{
    if (x <= c.at || 2 * c.len_line > sh.q)
        return x;
    return 2 * (x - c.at) < c.len_line ? c.at : c.at + c.len_line;
}

// To the next item.
__device__ __forceinline__ void cursor_next(const smoe_attention_args &a, const Share &sh, const RowSeq *seqs,
                                            Cursor &c)
{
    c.at += c.len_line;
    if (++c.h < a.cache.num_kv_heads)
        return;
    c.h = 0;
    do
        ++c.b;
    while (seqs[c.b].rows == 0 && c.b < a.batch.num_seqs);
    cursor_seq(a, sh, seqs, c);
}

// Key steps [s0, s1) of the cursor's item that lie in the share [w0, w1).
__device__ __forceinline__ void steps_in(const Cursor &c, uint32_t w0, uint32_t w1, int &s0, int &s1)
{
    const uint32_t k = c.at + kItemSteps;
    s0 = w0 > k ? static_cast<int>(w0 - k) : 0;
    s1 = w1 <= k ? 0 : (w1 - k < static_cast<uint32_t>(c.steps) ? static_cast<int>(w1 - k) : c.steps);
}

// A part that a warp leaves for its CTA to join.
struct PartInfo {
    const float *at;       // outputs [rows][D], maxima [rows], sums [rows]
    int row0;
    int nrows, h;          // packed rows (0: no part)
    uint32_t first, last;  // the workers that share the item
};

__host__ __device__ constexpr int dec_part_floats(int D, int T) { return dec_rows(T) * (D + 2); }

// N consecutive outputs of a row, divided by the row's sum.
template <int N>
__device__ __forceinline__ void write_out(const smoe_attention_args &a, int G, int row0, int h, int r, int c,
                                          const float (&v)[N], float l)
{
    const float inv = l > 0.f ? 1.0f / l : 0.f;  // a row that sees no key: zeros
    const int64_t at = (row0 + static_cast<int64_t>(r / G)) * a.out_row_stride +
                       (int64_t)(h * G + r % G) * a.out_head_stride + c;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        if (a.out_dtype == SMOE_F32)
            *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at + i) =
                make_float2(v[i] * inv, v[i + 1] * inv);
        else
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + i) =
                pack_bf16x2(v[i] * inv, v[i + 1] * inv);
    }
}

// A row's maximum, sum and the D / 16 consecutive outputs of a lane: half a
// warp per row.
template <int D>
struct RowPart {
    float m, l, v[D / 16];

    __device__ __forceinline__ void clear()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            v[i] = 0.f;
    }
    // Adds a part: its maximum, sum and outputs.
    __device__ __forceinline__ void add(float pm, float pl, const float4 (&y)[D / 64])
    {
        const float mn = fmaxf(m, pm);
        const float mu = mn == -INFINITY ? 0.f : mn;  // nothing seen so far
        const float fo = ex2(m - mu), f = ex2(pm - mu);
        m = mn;
        l = fmaf(l, fo, pl * f);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            v[4 * i] = fmaf(v[4 * i], fo, y[i].x * f);
            v[4 * i + 1] = fmaf(v[4 * i + 1], fo, y[i].y * f);
            v[4 * i + 2] = fmaf(v[4 * i + 2], fo, y[i].z * f);
            v[4 * i + 3] = fmaf(v[4 * i + 3], fo, y[i].w * f);
        }
    }
};

// The joins run once per launch, so most of their time is the fetching of
// their code: the loop over a CTA's own parts stays a loop (8 parts unrolled
// took 3,900 cycles, this 1,300), the one over other CTAs' parts, which waits
// for the L2 cache, has the loads of four parts in flight.

// Rows r, r + 16, .. (T of them; those past nrows are not touched) of the
// parts that warps wa .. wb of this CTA left (`tail`: warp wa's is of an item
// begun in its share).
template <int D, int T>
__device__ __forceinline__ void join_near(RowPart<D> (&o)[T], const PartInfo (*parts)[2], int wa, int wb, bool tail,
                                          int r, int nrows, int l16)
{
#pragma unroll
    for (int t = 0; t < T; ++t)
        o[t].clear();
#pragma unroll 1
    for (int w = wa; w <= wb; ++w) {
        const float *p = parts[w][tail && w == wa ? 1 : 0].at;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int m = r + kMmaRows * t;
            if (m >= nrows)
                break;
            float4 y[D / 64];
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
                y[i] = *reinterpret_cast<const float4 *>(p + m * D + l16 * (D / 16) + 4 * i);
            o[t].add(p[dec_rows(T) * D + m], p[dec_rows(T) * (D + 1) + m], y);
        }
    }
}

// The same rows of n parts of other CTAs: the first at `first`, part k at
// rest + k step.  They are read past the L1 cache.
template <int D, int T>
__device__ __forceinline__ void join_far(RowPart<D> (&o)[T], const float *first, const float *rest, int64_t step,
                                         int n, int r, int nrows, int l16)
{
    constexpr int kBatch = 4 / T;
#pragma unroll
    for (int t = 0; t < T; ++t)
        o[t].clear();
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += kBatch) {
        float pm[kBatch][T], pl[kBatch][T];
        float4 y[kBatch][T][D / 64];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            // past the end: the last part again, with no weight
            const int at = k0 + k < n ? k0 + k : n - 1;
            const float *p = at == 0 ? first : rest + at * step;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int m = r + kMmaRows * t < nrows ? r + kMmaRows * t : r;
                pm[k][t] = __ldcg(p + dec_rows(T) * D + m);
                pl[k][t] = __ldcg(p + dec_rows(T) * (D + 1) + m);
#pragma unroll
                for (int i = 0; i < D / 64; ++i)
                    y[k][t][i] = __ldcg(reinterpret_cast<const float4 *>(p + m * D + l16 * (D / 16) + 4 * i));
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
#pragma unroll
            for (int t = 0; t < T; ++t)
                o[t].add(k0 + k < n ? pm[k][t] : -INFINITY, pl[k][t], y[k][t]);
    }
}

template <int D, int T>
__global__ void __launch_bounds__(32 * kDecWarps, 1)
    attend_rows_kernel(const smoe_attention_args a, uint8_t *workspace, int *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PartInfo s_part[kDecWarps][2];  // 0: of an item begun earlier, 1: begun here
    __shared__ int s_final[kDecWarps + 1];     // this CTA joins the item's parts of all CTAs
    constexpr int KB = D / 16;  // k blocks of Q K^T, pairs of column blocks of P V
    constexpr int kStages = dec_stages(T), kRows = dec_rows(T);
    static_assert(dec_part_floats(D, T) * 4 <= dec_ring_bytes(D, T) + dec_query_bytes(D, T),
                  "a part fits a ring and its queries");
    static_assert(kPartsAt + (size_t)kMaxCtas * (kDecWarps + 2) * dec_part_floats(D, T) * 4 <=
                      SMOE_ATTENTION_WORKSPACE_BYTES,
                  "workspace");
    static_assert(kMaxCtas <= kMaxCounters, "counters");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_heads / a.cache.num_kv_heads, page = a.cache.page_size;
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    const float sc = a.scale * 1.44269504088896341f;

    RowSeq *seqs = reinterpret_cast<RowSeq *>(smem + kDecWarps * (dec_ring_bytes(D, T) + dec_query_bytes(D, T)));
    const Share sh = plan(a, seqs, status);
    const uint32_t me = blockIdx.x * kDecWarps + warp;
    if ((uint64_t)blockIdx.x * kDecWarps * sh.q >= sh.total)
        return;  // nothing for the whole CTA
    if (lane == 0)
        s_part[warp][0].nrows = s_part[warp][1].nrows = 0;
    // the share's borders, one per half warp; shares end at the line's end
    const uint64_t nominal = (uint64_t)(me + (lane >> 4)) * sh.q;
    Cursor cc = cursor_at(a, sh, seqs, nominal < sh.total ? static_cast<uint32_t>(nominal) : sh.total);
    const uint32_t snapped = border(sh, cc, nominal < sh.total ? static_cast<uint32_t>(nominal) : sh.total);
    const uint32_t w0 = __shfl_sync(0xffffffffu, snapped, 0), w1 = __shfl_sync(0xffffffffu, snapped, 16);
    cc = cursor_at(a, sh, seqs, w0);
    Cursor ld = cc;
    // a warp's memory: its ring, then its queries (T > 1)
    const uint32_t ring = smem_u32(smem) + warp * (dec_ring_bytes(D, T) + dec_query_bytes(D, T));
    const uint32_t query = ring + dec_ring_bytes(D, T);
    unsigned *arrived = reinterpret_cast<unsigned *>(workspace);
    float *worker_parts = reinterpret_cast<float *>(workspace + kPartsAt);  // one per worker
    float *cta_parts = worker_parts + (int64_t)kMaxCtas * kDecWarps * dec_part_floats(D, T);  // two per CTA

    // The loading end of the ring: the next step to copy, its page id already
    // on the way.
    int ls, ls1, filled = 0, pg = 0;
    steps_in(ld, w0, w1, ls, ls1);
    auto seek = [&]() {  // to a step that exists, or past the share
        while (ld.rows > 0 && ls >= ls1) {
            if (ld.at + ld.len_line >= w1) {
                ld.rows = 0;
                break;
            }
            cursor_next(a, sh, seqs, ld);
            steps_in(ld, w0, w1, ls, ls1);
        }
        const int k0 = (ld.k_lo / kDecKeys + ls) * kDecKeys;
        pg = ld.rows > 0 && k0 < ld.k_hi
                 ? a.batch.page_table[(int64_t)ld.b * a.batch.table_stride + k0 / page]
                 : 0;
    };
    seek();
    auto issue = [&]() {
        if (ld.rows > 0) {
            const int k0 = (ld.k_lo / kDecKeys + ls) * kDecKeys;
            if (k0 < ld.k_hi) {
                const bool there = pg >= 0 && pg < a.cache.num_pages;
                if (!there && lane == 0)
                    set_status(status, kStatusBadArg);
                const int64_t at = ((int64_t)ld.h * page + k0 % page) * D;
                const uint16_t *ks = static_cast<const uint16_t *>(a.cache.k_pages) +
                                     (there ? pg * a.cache.k_page_stride + at : 0);
                const uint16_t *vs = static_cast<const uint16_t *>(a.cache.v_pages) +
                                     (there ? pg * a.cache.v_page_stride + at : 0);
                const uint32_t dk = ring + filled * dec_step_bytes(D), dv = dk + kDecKeys * D * 2;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int e = i * 32 + lane, r = e / (D / 8), c = e % (D / 8);
                    // slots of keys that no row sees are not read: zeros
                    const bool v = there && k0 + r >= ld.k_lo && k0 + r < ld.k_hi;
                    cp_async16(dk + chunk_at<D>(r, c), ks + (v ? r * D + c * 8 : 0), v);
                    cp_async16(dv + chunk_at<D>(r, c), vs + (v ? r * D + c * 8 : 0), v);
                }
            }
            filled = filled + 1 == kStages ? 0 : filled + 1;
            ++ls;
            seek();
        }
        cp_async_commit();
    };
    int used = 0, primed = 0;  // the ring's reading end, copies ahead of it
    for (; cc.rows > 0 && cc.at < w1; cursor_next(a, sh, seqs, cc)) {
        int s0, s1;
        steps_in(cc, w0, w1, s0, s1);
        if (s0 >= s1)
            continue;
        // ---- one item, or the part of it that lies in the share
        const int nrows = cc.rows * G;  // packed rows, kRows at most
        int lo[T][2], hi[T][2], t_lo, t_hi, x;  // [t_lo, t_hi) is seen by every row
        seen_from(a, cc.len - 1, t_lo, x);
        seen_from(a, cc.len - cc.rows, x, t_hi);
        // row m of the item in q
        auto query_at = [&](int m) {
            return static_cast<const uint16_t *>(a.q) + (cc.row0 + static_cast<int64_t>(m / G)) * a.q_row_stride +
                   (int64_t)(cc.h * G + m % G) * a.q_head_stride;
        };
        uint32_t q[T == 1 ? KB : 1][4];
        if (T == 1) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int m = g + 8 * r;
                const bool on = m < nrows;
                const uint16_t *src = query_at(m);
#pragma unroll
                for (int kb = 0; kb < (T == 1 ? KB : 0); ++kb) {
                    q[kb][r] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * kb + c2) : 0u;
                    q[kb][2 + r] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * kb + 8 + c2) : 0u;
                }
            }
        } else {
            __syncwarp();  // the queries before are no longer read
#pragma unroll 4
            for (int e = lane; e < kRows * (D / 8); e += 32) {
                const int m = e / (D / 8), c = e % (D / 8);
                cp_async16(query + chunk_at<D>(m, c), m < nrows ? query_at(m) + c * 8 : a.q, m < nrows);
            }
            // (they come with the copies of the next step)
        }
        float o[T][2 * KB][4], mx[T][2], sum[T][2];
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int m = kMmaRows * t + g + 8 * r;
                lo[t][r] = hi[t][r] = 0;
                if (m < nrows)
                    seen_from(a, cc.len - cc.rows + m / G, lo[t][r], hi[t][r]);
                mx[t][r] = -INFINITY;
                sum[t][r] = 0.f;
            }
#pragma unroll
            for (int n = 0; n < 2 * KB; ++n)
                o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
        }
        int k0 = (cc.k_lo / kDecKeys + s0) * kDecKeys;

        for (int st = s0; st < s1; ++st, k0 += kDecKeys) {
            // the first time as many as the ring holds
            do
                issue();
            while (primed++ < kStages - 1);
            primed = kStages;
            if (T > 1 && st == s0)
                cp_async_wait<0>();  // the queries too
            else
                cp_async_wait<kStages - 1>();
            __syncwarp();
            const uint32_t dk = ring + used * dec_step_bytes(D), dv = dk + kDecKeys * D * 2;
            used = used + 1 == kStages ? 0 : used + 1;
            if (k0 >= cc.k_hi)
                continue;  // no row sees a key: nothing was copied
            float p[T][2][4] = {};
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
                uint32_t b[4];
                ldm4(b, dk + chunk_at<D>((lane & 7) + ((lane >> 4) << 3), 2 * kb + ((lane >> 3) & 1)));
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    uint32_t qs[4];
                    if (T > 1)
                        ldm4(qs, query + chunk_at<D>(kMmaRows * t + (lane & 15), 2 * kb + (lane >> 4)));
                    const uint32_t (&qf)[4] = T > 1 ? qs : q[T == 1 ? kb : 0];
                    mma_bf16(p[t][0], qf, b[0], b[1]);
                    mma_bf16(p[t][1], qf, b[2], b[3]);
                }
            }
            // P as bf16 hi + lo: the loop waits for memory, not for the second
            // product, and the output keeps fp32 accuracy
            uint32_t hi4[T][4], lo4[T][4];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                if (k0 < t_lo || k0 + kDecKeys > t_hi) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = k0 + 8 * n + c2 + (e & 1), r = e >> 1;
                            if (key < lo[t][r] || key >= hi[t][r])
                                p[t][n][e] = -INFINITY;
                        }
                }
                float f[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = fmaxf(fmaxf(p[t][0][2 * r], p[t][0][2 * r + 1]),
                                    fmaxf(p[t][1][2 * r], p[t][1][2 * r + 1]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const float mn = fmaxf(mx[t][r], v * sc);
                    const float mu = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing yet
                    f[r] = ex2(mx[t][r] - mu);
                    mx[t][r] = mn;
                    float y = 0.f;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float &w = p[t][n][2 * r + e];
                            w = ex2(fmaf(w, sc, -mu));
                            y += w;
                        }
                    sum[t][r] = sum[t][r] * f[r] + y;
                }
                if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < 2 * KB; ++n) {
                        o[t][n][0] *= f[0];
                        o[t][n][1] *= f[0];
                        o[t][n][2] *= f[1];
                        o[t][n][3] *= f[1];
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        split_bf16x2(p[t][n][2 * r], p[t][n][2 * r + 1], hi4[t][2 * n + r], lo4[t][2 * n + r]);
            }
#pragma unroll
            for (int n = 0; n < KB; ++n) {
                uint32_t b[4];
                ldm4t(b, dv + chunk_at<D>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    mma_bf16(o[t][2 * n], hi4[t], b[0], b[1]);
                    mma_bf16(o[t][2 * n], lo4[t], b[0], b[1]);
                    mma_bf16(o[t][2 * n + 1], hi4[t], b[2], b[3]);
                    mma_bf16(o[t][2 * n + 1], lo4[t], b[2], b[3]);
                }
            }
            __syncwarp();
        }
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sum[t][r] += __shfl_xor_sync(0xffffffffu, sum[t][r], 1);
                sum[t][r] += __shfl_xor_sync(0xffffffffu, sum[t][r], 2);
            }
        if (s0 == 0 && s1 == cc.steps) {
            // the whole item
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int m = kMmaRows * t + g + 8 * r;
                    if (m < nrows)
#pragma unroll
                        for (int n = 0; n < 2 * KB; ++n) {
                            const float v[2] = {o[t][n][2 * r], o[t][n][2 * r + 1]};
                            write_out<2>(a, G, cc.row0, cc.h, m, 8 * n + c2, v, sum[t][r]);
                        }
                }
        } else {
            // a part: into the warp's ring where no later item has keys in the
            // share (every copy has been used then), else into the workspace,
            // while the ring works on
            const int which = s0 == 0 ? 1 : 0;
            const uint32_t after = cc.at + cc.len_line;
            const bool idle = after >= w1 || w1 - after <= kItemSteps;
            float *part = idle ? reinterpret_cast<float *>(smem + warp * (dec_ring_bytes(D, T) + dec_query_bytes(D, T)))
                               : worker_parts + (int64_t)me * dec_part_floats(D, T);
            if (lane == 0) {
                PartInfo &pi = s_part[warp][which];
                pi.at = part;
                pi.row0 = cc.row0;
                pi.nrows = nrows;
                pi.h = cc.h;
                pi.first = (cc.at + kItemSteps) / sh.q;
                pi.last = (cc.at + kItemSteps + cc.steps - 1) / sh.q;
            }
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int m = kMmaRows * t + g + 8 * r;
                    if (m >= nrows)
                        continue;
#pragma unroll
                    for (int n = 0; n < 2 * KB; ++n)
                        *reinterpret_cast<float2 *>(part + m * D + 8 * n + c2) =
                            make_float2(o[t][n][2 * r], o[t][n][2 * r + 1]);
                    if ((lane & 3) == 0) {
                        part[kRows * D + m] = mx[t][r];
                        part[kRows * (D + 1) + m] = sum[t][r];
                    }
                }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    // ---- join the CTA's parts: of the item begun before it, then of the items
    // begun by each warp.  Each half warp takes one row of one item at a time.
    constexpr int kPer = D / 16;  // outputs of a lane
    const uint32_t b0 = blockIdx.x * kDecWarps;
    const int hw = tid >> 4, l16 = lane & 15;
    static_assert(2 * kDecWarps == kMmaRows, "half a warp per row of a tile");
    int base = 0;  // rows of the items so far
#pragma unroll 1
    for (int j = -1; j < kDecWarps; ++j) {
        const PartInfo pi = s_part[j < 0 ? 0 : j][j < 0 ? 0 : 1];
        // rows go round over the half warps, whatever item they are of
        const int r0 = (hw - base) & (kMmaRows - 1);
        base += pi.nrows < kMmaRows ? pi.nrows : kMmaRows;
        const int wa = j < 0 ? 0 : j;
        const int wb = pi.last - b0 < kDecWarps ? static_cast<int>(pi.last - b0) : kDecWarps - 1;
        if (r0 >= pi.nrows)
            continue;
        RowPart<D> o[T];
        join_near<D, T>(o, s_part, wa, wb, j >= 0, r0, pi.nrows, l16);
        const bool whole = pi.first / kDecWarps == pi.last / kDecWarps;
        float *out = cta_parts + (2 * (int64_t)blockIdx.x + (j < 0 ? 0 : 1)) * dec_part_floats(D, T);
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const int r = r0 + kMmaRows * t;
            if (r >= pi.nrows)
                break;
            if (whole) {
                write_out<kPer>(a, G, pi.row0, pi.h, r, l16 * kPer, o[t].v, o[t].l);
                continue;
            }
            // the item goes over CTAs
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                __stcg(reinterpret_cast<float4 *>(out + r * D + l16 * kPer + i),
                       make_float4(o[t].v[i], o[t].v[i + 1], o[t].v[i + 2], o[t].v[i + 3]));
            if (l16 == 0) {
                __stcg(out + kRows * D + r, o[t].m);
                __stcg(out + kRows * (D + 1) + r, o[t].l);
            }
        }
    }
    // ---- of the items that go over CTAs (the one begun before this CTA, the
    // last one begun in it), the last CTA to arrive joins the parts
    __syncthreads();
    if (tid <= kDecWarps) {
        const PartInfo &pi = s_part[tid ? tid - 1 : 0][tid ? 1 : 0];
        const uint32_t c_first = pi.first / kDecWarps, c_last = pi.last / kDecWarps;
        s_final[tid] = pi.nrows > 0 && c_first != c_last && count_arrival(arrived + c_first) == c_last - c_first;
    }
    __syncthreads();
#pragma unroll 1
    for (int j = -1; j < kDecWarps; ++j) {
        if (!s_final[j + 1])
            continue;
        const PartInfo pi = s_part[j < 0 ? 0 : j][j < 0 ? 0 : 1];
        const int c_first = static_cast<int>(pi.first / kDecWarps), c_last = static_cast<int>(pi.last / kDecWarps);
        if (hw < pi.nrows) {
            // the first CTA's part, then those of the CTAs after it
            const float *of = cta_parts + 2 * (int64_t)c_first * dec_part_floats(D, T);
            RowPart<D> o[T];
            join_far<D, T>(o, of + dec_part_floats(D, T), of, 2 * dec_part_floats(D, T), c_last - c_first + 1, hw,
                           pi.nrows, l16);
#pragma unroll
            for (int t = 0; t < T; ++t)
                if (hw + kMmaRows * t < pi.nrows)
                    write_out<kPer>(a, G, pi.row0, pi.h, hw + kMmaRows * t, l16 * kPer, o[t].v, o[t].l);
        }
        if (tid == 0)
            arrived[c_first] = 0;  // for the next launch
    }
}

template <int D, int T>
cudaError_t launch_rows(const smoe_attention_args &a, uint8_t *workspace, const DeviceFacts &dev,
                        cudaStream_t stream)
{
    static std::atomic<bool> allowed[kMaxDeviceIndex];
    constexpr int smem = dec_smem_bytes(D, T);
    const cudaError_t e = allow_smem(attend_rows_kernel<D, T>, smem, dev, allowed);
    if (e != cudaSuccess)
        return e;
    attend_rows_kernel<D, T><<<dev.sms < kMaxCtas ? dev.sms : kMaxCtas, 32 * kDecWarps, smem, stream>>>(
        a, workspace, dev.status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const smoe_attention_args &a, void *workspace, const DeviceFacts &dev,
                             cudaStream_t stream)
{
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const int64_t rows = (int64_t)a.max_rows * (a.num_heads / a.cache.num_kv_heads);
    const bool wide = a.cache.head_dim == 128;
    if (rows <= dec_rows(1))
        return wide ? launch_rows<128, 1>(a, ws, dev, stream) : launch_rows<64, 1>(a, ws, dev, stream);
    if (rows <= dec_rows(2))
        return wide ? launch_rows<128, 2>(a, ws, dev, stream) : launch_rows<64, 2>(a, ws, dev, stream);
    return launch_attention_chunk(a, ws, dev, stream);
}

}  // namespace smoe
