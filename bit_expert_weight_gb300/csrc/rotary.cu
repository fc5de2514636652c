// rotary.cu -- position rotation of heads (smoe_rope) and its fusion with the
// write of new keys and values into the paged cache (smoe_kv_append).
//
// Mathematics: pair i of a head at position p turns by p * f_i.  The table
// holds f_i / (2 pi) as a 64-bit fixed-point fraction of a turn, so p times it
// modulo 2^64 is the angle reduced to one turn without any rounding: only the
// last conversion of that fraction to fp32 and sincospif round.  An fp32
// product p * f_i would be off by 0.03 rad at position one million, and fp64
// is slow on this part.
//
// Bound: HBM.  Both kernels read each head once and write it once.  A CTA
// takes some heads of some consecutive rows: it computes each row's sines and
// cosines once, into shared memory (with a set per lane and head they cost
// more than the copy: 102 us instead of 61 for 16,411 rows of 40 heads), then
// its threads go over the heads, 8 channels (4 pairs) at a time, four loads in
// flight.  Measured: 16,411 rows of 40 bf16 heads of 128 with 32 channels turned
// 60.6 us, 5.5 TB/s; an append of 11,011 rows of 32 + 8 + 8 fp32 heads of 128
// 66.4 us, 6.1 TB/s.  One row: 4.5 us, a launch and a chain of three loads.
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotRows = 16;        // rows of a CTA at most
// Runs of 8 channels that a thread loads together; the next ones are on their
// way while these are worked on.
template <bool F32>
constexpr int kRuns = F32 ? 2 : 4;

// 8 channels as they lie in memory: two runs of 4.
template <bool F32>
struct Raw {
    float4 u, v;
    __device__ __forceinline__ void load(const void *base, int64_t a, int64_t b)
    {
        u = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + a);
        v = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + b);
    }
    __device__ __forceinline__ void clear() { u = v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ float4 first() const { return u; }
    __device__ __forceinline__ float4 second() const { return v; }
};
__device__ __forceinline__ float4 widen(uint2 v)
{
    return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y), bf16hi_to_f32(v.y));
}
template <>
struct Raw<false> {
    uint2 u, v;
    __device__ __forceinline__ void load(const void *base, int64_t a, int64_t b)
    {
        u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + a);
        v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + b);
    }
    __device__ __forceinline__ void clear() { u = v = make_uint2(0, 0); }
    __device__ __forceinline__ float4 first() const { return widen(u); }
    __device__ __forceinline__ float4 second() const { return widen(v); }
};

template <bool F32>
__device__ __forceinline__ void store4(void *base, int64_t at, float4 v)
{
    if (F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + at) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// Where a lane's 8 channels of a head lie: two runs of 4, first channels o0
// and o1, one in each half of the channels that rotate (or of those that do
// not), so that it holds both halves of its 4 pairs and that each load of a
// warp covers whole sectors.
struct Lane {
    int o0, o1, t;
    bool on, turns, inter;  // it has channels; they rotate; (2i, 2i + 1) are pairs
};

__device__ __forceinline__ Lane lane_of(int t, int D, int R, int inter)
{
    Lane ln;
    ln.t = t;
    ln.on = 8 * t < D;
    ln.turns = 8 * t < R;
    ln.inter = inter != 0;
    ln.o0 = ln.turns ? 4 * t : R + 4 * (t - R / 8);
    ln.o1 = ln.o0 + (ln.turns ? R : D - R) / 2;
    return ln;
}

// (cosine, sine) times rot_scale of pair i at position pos.
__device__ __forceinline__ float2 turn_of(const int64_t *table, int i, int pos, float rot_scale)
{
    const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(pos)) *
                                     static_cast<unsigned long long>(table[i]);
    float sn, cs;
    // twice the signed fraction of a turn, in [-1, 1]
    sincospif(__ll2float_rn(static_cast<long long>(turns)) * 0x1p-63f, &sn, &cs);
    return make_float2(cs * rot_scale, sn * rot_scale);
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}

// cs: the row's (cosine, sine) of every pair.
__device__ __forceinline__ void turn_lane(const Lane &ln, const float2 *cs, float4 &u, float4 &v)
{
    if (!ln.turns)
        return;
    // pairs 4t .. 4t + 3; or, where (2i, 2i + 1) are pairs, two of each run
    const float2 *at = cs + (ln.inter ? ln.o0 / 2 : ln.o0);
    const float4 a = *reinterpret_cast<const float4 *>(at);
    const float4 b = *reinterpret_cast<const float4 *>(ln.inter ? cs + ln.o1 / 2 : at + 2);
    if (ln.inter) {
        turn(u.x, u.y, a.x, a.y);
        turn(u.z, u.w, a.z, a.w);
        turn(v.x, v.y, b.x, b.y);
        turn(v.z, v.w, b.z, b.w);
    } else {
        turn(u.x, v.x, a.x, a.y);
        turn(u.y, v.y, a.z, a.w);
        turn(u.z, v.z, b.x, b.y);
        turn(u.w, v.w, b.z, b.w);
    }
}

// x * rsqrt(mean(x^2) + eps) * w over the head that lph lanes share.  Every
// lane of the warp takes part in the shuffles; lanes without channels hold 0.
__device__ __forceinline__ void norm_lane(const Lane &ln, int lph, int D, float eps, const void *w, bool norm,
                                          float4 &u, float4 &v)
{
    float ss = u.x * u.x + u.y * u.y + u.z * u.z + u.w * u.w + v.x * v.x + v.y * v.y + v.z * v.z +
               v.w * v.w;
    for (int o = lph >> 1; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!norm || !ln.on)
        return;
    const float r = 1.0f / sqrtf(ss / static_cast<float>(D) + eps);
    Raw<false> weight;
    weight.load(w, ln.o0, ln.o1);
    const float4 a = weight.first(), b = weight.second();
    u = make_float4(u.x * r * a.x, u.y * r * a.y, u.z * r * a.z, u.w * r * a.w);
    v = make_float4(v.x * r * b.x, v.y * r * b.y, v.z * r * b.z, v.w * r * b.w);
}

// Lanes that share one head: the power of two that covers D / 8.
__host__ __device__ inline int lanes_per_head(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }

// How the heads of all rows are dealt to CTAs: `rows` consecutive rows and
// `heads` of their heads each.
struct Deal {
    int rows, heads, chunks;  // chunks: CTAs that share the heads of one row
};

// The place of a thread's next head: (row, head) of the CTA's block, stepping
// by `step` heads in row-major order.
struct Walk {
    int row, head;
    __device__ void go(int step, int heads)
    {
        head += step;
        while (head >= heads) {
            head -= heads;
            ++row;
        }
    }
};

template <bool F32>
__global__ void __launch_bounds__(kRotThreads) rope_kernel(const smoe_rope_args a, const Deal deal)
{
    __shared__ __align__(16) float2 s_cs[kRotRows * SMOE_MAX_HEAD_DIM / 2];
    const int D = a.head_dim, R = a.rot_dim, tid = threadIdx.x;
    const int lph = lanes_per_head(D), step = kRotThreads / lph;
    const int64_t row0 = (int64_t)(blockIdx.x / deal.chunks) * deal.rows;
    const int h0 = (blockIdx.x % deal.chunks) * deal.heads;
    const int rows = a.num_rows - row0 < deal.rows ? static_cast<int>(a.num_rows - row0) : deal.rows;
    const int heads = a.num_heads - h0 < deal.heads ? a.num_heads - h0 : deal.heads;
    const Lane ln = lane_of(tid & (lph - 1), D, R, a.interleaved);
    constexpr int kN = kRuns<F32>;
    Walk in = {0, tid / lph}, at = in;
    in.go(0, heads);
    at.go(0, heads);
    Raw<F32> raw[kN], next[kN];
    auto load = [&](Raw<F32> (&r)[kN]) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            r[i].clear();
            if (in.row < rows && ln.on) {
                const int64_t from = (row0 + in.row) * a.x_row_stride + (h0 + in.head) * a.x_head_stride;
                r[i].load(a.x, from + ln.o0, from + ln.o1);
            }
            in.go(step, heads);
        }
    };
    load(raw);  // the first heads are on their way while the turns are computed
    for (int i = tid; i < rows * (R / 2); i += kRotThreads)
        s_cs[i] = turn_of(a.table, i % (R / 2), a.positions[row0 + i / (R / 2)], a.rot_scale);
    __syncthreads();
    const int n = (rows * heads + step * kN - 1) / (step * kN);  // the same for every thread
    for (int k = 0; k < n; ++k) {
        load(next);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            float4 u = raw[i].first(), v = raw[i].second();
            if (a.norm_w)
                norm_lane(ln, lph, D, a.eps, a.norm_w, true, u, v);
            if (at.row < rows && ln.on) {
                turn_lane(ln, s_cs + at.row * (R / 2), u, v);
                const int64_t to = (row0 + at.row) * a.out_row_stride + (h0 + at.head) * a.out_head_stride;
                store4<F32>(a.out, to + ln.o0, u);
                store4<F32>(a.out, to + ln.o1, v);
            }
            at.go(step, heads);
            raw[i] = next[i];
        }
    }
}

// The sequence that owns `row` (row < row_start[n]): the number of starts
// 1 .. n that are <= row, found by all lanes of a warp together, 32 probes a
// round.  In range for any contents of row_start.
__device__ __forceinline__ int owner_of(const int32_t *row_start, int n, int64_t row, int lane)
{
    int lo = 0, hi = n;  // the count lies in [lo, hi)
    while (hi - lo > 1) {
        const int span = hi - lo, stride = (span + 31) / 32;
        const int at = lo + (lane + 1) * stride;  // the count is >= at where start[at] <= row
        const bool le = at < hi && row_start[at] <= row;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = __popc(m);
        const int nlo = lo + k * stride;
        hi = nlo + stride < hi ? nlo + stride : hi;
        lo = nlo < hi ? nlo : hi - 1;
    }
    return lo;
}

// Where a row's keys and values go.
struct Slot {
    int64_t k, v;  // element of kv head 0 (negative: nowhere)
};

// A row's place: its sequence (-1: none) and key index (negative: none).
struct Place {
    int seq, key;
};

// By one warp.
__device__ __forceinline__ Place place_of(const smoe_kv_append_args &a, int64_t row, int lane, int *status)
{
    const int n = a.batch.num_seqs;
    // In a batch of single rows the row's sequence is number `row`: all that
    // is needed then is asked for at once.
    int b = row < n ? static_cast<int>(row) : n - 1;
    int first = a.batch.row_start[b], last = a.batch.row_start[b + 1], len = a.batch.kv_len[b];
    if (row >= a.batch.row_start[n] || row < a.batch.row_start[0])
        return {-1, -1};
    if (row < first || row >= last) {
        b = owner_of(a.batch.row_start, n, row, lane);
        first = a.batch.row_start[b];
        last = a.batch.row_start[b + 1];
        len = a.batch.kv_len[b];
    }
    if (first < 0 || row < first || row >= last) {
        if (lane == 0)
            set_status(status, kStatusBadArg);
        return {-1, -1};
    }
    return {b, static_cast<int>((int64_t)len - last + row)};
}

__device__ __forceinline__ Slot slot_of(const smoe_kv_append_args &a, Place p, int *status)
{
    if (p.seq < 0 || p.key < 0)
        return {-1, -1};
    const int pi = p.key / a.cache.page_size, in = p.key % a.cache.page_size;
    const int pg = pi < a.batch.table_stride ? a.batch.page_table[(int64_t)p.seq * a.batch.table_stride + pi] : -1;
    if (pg < 0 || pg >= a.cache.num_pages) {
        set_status(status, kStatusBadArg);
        return {-1, -1};
    }
    return {pg * a.cache.k_page_stride + (int64_t)in * a.cache.head_dim,
            pg * a.cache.v_page_stride + (int64_t)in * a.cache.head_dim};
}

// The heads of a row: its q heads, k heads and v heads in this order.
template <bool F32>
__global__ void __launch_bounds__(kRotThreads)
    kv_append_kernel(const smoe_kv_append_args a, const Deal deal, int *status)
{
    __shared__ __align__(16) float2 s_cs[kRotRows * 128 / 2];
    __shared__ Slot s_slot[kRotRows];
    __shared__ Place s_place[kRotRows];
    const int D = a.cache.head_dim, R = a.rot_dim, tid = threadIdx.x;
    const int lph = lanes_per_head(D), step = kRotThreads / lph;
    const int Hq = a.q ? a.num_heads : 0, Hkv = a.cache.num_kv_heads;
    const int64_t row0 = (int64_t)(blockIdx.x / deal.chunks) * deal.rows;
    const int h0 = (blockIdx.x % deal.chunks) * deal.heads;
    const int rows = a.batch.num_rows - row0 < deal.rows ? static_cast<int>(a.batch.num_rows - row0) : deal.rows;
    const int heads = Hq + 2 * Hkv - h0 < deal.heads ? Hq + 2 * Hkv - h0 : deal.heads;
    const Lane ln = lane_of(tid & (lph - 1), D, R, a.interleaved);
    const Lane flat = lane_of(tid & (lph - 1), D, 0, 0);  // of values: not rotated
    constexpr int kN = kRuns<F32>;
    Walk in = {0, tid / lph}, at = in;
    in.go(0, heads);
    at.go(0, heads);
    Raw<F32> raw[kN], next[kN];
    auto load = [&](Raw<F32> (&x)[kN]) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            x[i].clear();
            if (in.row < rows && ln.on) {
                const int h = h0 + in.head, kh = h - Hq, vh = kh - Hkv;
                const int64_t r = row0 + in.row;
                const void *src = kh < 0 ? a.q : (vh < 0 ? a.k : a.v);
                const int64_t from = kh < 0   ? r * a.q_row_stride + h * a.q_head_stride
                                     : vh < 0 ? r * a.k_row_stride + kh * a.k_head_stride
                                              : r * a.v_row_stride + vh * a.v_head_stride;
                x[i].load(src, from + (vh < 0 ? ln.o0 : flat.o0), from + (vh < 0 ? ln.o1 : flat.o1));
            }
            in.go(step, heads);
        }
    };
    load(raw);  // the first heads are on their way while the rows' places are looked up
    // The first CTA looks whether the starts are in order; the loads are on
    // their way with those of its rows' places.
    const int seqs = a.batch.num_seqs;
    const bool look = blockIdx.x == 0;
    const int start = look && tid < seqs ? a.batch.row_start[tid] : 0;
    const int end = look && tid < seqs ? a.batch.row_start[tid + 1] : 0;
    for (int r = tid >> 5; r < rows; r += kRotThreads / 32) {
        const Place p = place_of(a, row0 + r, tid & 31, status);
        if ((tid & 31) == 0)
            s_place[r] = p;
    }
    if (look) {
        bool bad = end < start || start < 0 || end > a.batch.num_rows;
        for (int b = tid + kRotThreads; b < seqs; b += kRotThreads) {
            const int to = a.batch.row_start[b + 1];
            bad = bad || to < a.batch.row_start[b] || to > a.batch.num_rows;
        }
        if (bad)
            set_status(status, kStatusBadArg);
    }
    __syncthreads();
    if (tid >= kRotThreads - kRotRows && tid - (kRotThreads - kRotRows) < rows)
        s_slot[tid - (kRotThreads - kRotRows)] = slot_of(a, s_place[tid - (kRotThreads - kRotRows)], status);
    for (int i = tid; i < rows * (R / 2); i += kRotThreads) {
        const int r = i / (R / 2);
        s_cs[i] = turn_of(a.table, i % (R / 2), a.positions ? a.positions[row0 + r] : s_place[r].key, a.rot_scale);
    }
    __syncthreads();
    const int n = (rows * heads + step * kN - 1) / (step * kN);  // the same for every thread
    for (int k = 0; k < n; ++k) {
        load(next);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            float4 u = raw[i].first(), v = raw[i].second();
            raw[i] = next[i];
            const int row = at.row, h = h0 + at.head, kh = h - Hq, vh = kh - Hkv;
            at.go(step, heads);
            if (a.q_norm || a.k_norm) {
                const void *wn = kh < 0 ? a.q_norm : a.k_norm;
                norm_lane(ln, lph, D, a.eps, wn, wn && vh < 0, u, v);
            }
            if (row >= rows || !ln.on || s_place[row].seq < 0)
                continue;
            if (vh < 0)
                turn_lane(ln, s_cs + row * (R / 2), u, v);
            if (kh < 0) {
                const int64_t to = (row0 + row) * a.qo_row_stride + h * a.qo_head_stride;
                store4<false>(a.q_out, to + ln.o0, u);
                store4<false>(a.q_out, to + ln.o1, v);
                continue;
            }
            const int64_t slot = vh < 0 ? s_slot[row].k : s_slot[row].v;
            if (slot < 0)
                continue;
            const int64_t to = slot + (int64_t)(vh < 0 ? kh : vh) * a.cache.page_size * D;
            void *dst = vh < 0 ? a.cache.k_pages : a.cache.v_pages;
            store4<false>(dst, to + (vh < 0 ? ln.o0 : flat.o0), u);
            store4<false>(dst, to + (vh < 0 ? ln.o1 : flat.o1), v);
        }
    }
}

// Rounds of a CTA over its heads (a head per lane group and round): as few as
// put all CTAs on the device at once (three per SM fit for every type), at
// most 16.  More rounds share a row's turns and keep the loads in flight;
// fewer shorten a small call.  (128 rows of 72 heads: 15.4 us with 16 rounds;
// 16,411 rows of 40 heads: 63.8 us with 8 rounds, 60.6 with 16.)
Deal deal_heads(int64_t rows, int heads, int D, int sms, int64_t *blocks)
{
    const int per_round = kRotThreads / lanes_per_head(D);
    const int64_t wave = (int64_t)per_round * 3 * sms;
    const int64_t rounds = (rows * heads + wave - 1) / wave;
    const int want = per_round * static_cast<int>(rounds < 16 ? rounds : 16);
    Deal d;
    d.rows = want / heads < 1 ? 1 : (want / heads < kRotRows ? want / heads : kRotRows);
    d.heads = d.rows > 1 || heads < want ? heads : want;
    d.chunks = (heads + d.heads - 1) / d.heads;
    *blocks = (rows + d.rows - 1) / d.rows * d.chunks;
    return d;
}

}  // namespace

cudaError_t launch_rope(const smoe_rope_args &a, const DeviceFacts &dev, cudaStream_t stream)
{
    int64_t blocks;
    const Deal deal = deal_heads(a.num_rows, a.num_heads, a.head_dim, dev.sms, &blocks);
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    auto k = a.dtype == SMOE_F32 ? rope_kernel<true> : rope_kernel<false>;
    k<<<static_cast<unsigned>(blocks), kRotThreads, 0, stream>>>(a, deal);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const smoe_kv_append_args &a, const DeviceFacts &dev, cudaStream_t stream)
{
    int64_t blocks;
    const int heads = (a.q ? a.num_heads : 0) + 2 * a.cache.num_kv_heads;
    const Deal deal = deal_heads(a.batch.num_rows, heads, a.cache.head_dim, dev.sms, &blocks);
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    auto k = a.dtype == SMOE_F32 ? kv_append_kernel<true> : kv_append_kernel<false>;
    k<<<static_cast<unsigned>(blocks), kRotThreads, 0, stream>>>(a, deal, dev.status);
    return cudaGetLastError();
}

}  // namespace smoe
