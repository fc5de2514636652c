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
// Bound: HBM.  Both kernels read each head once and write it once; a lane
// holds 8 channels (4 pairs) of a head and computes its 4 sines and cosines
// once for the kHeadsPerLane heads of the same row that it rotates, whose
// loads are all issued before the first is used.
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kRotWarps = 8;        // warps per CTA
constexpr int kHeadsPerLane = 4;    // heads a lane works through

// 4 consecutive elements as fp32.
template <bool F32>
__device__ __forceinline__ float4 load4(const void *base, int64_t at)
{
    if (F32)
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    return make_float4(bf16lo_to_f32(v.x), bf16hi_to_f32(v.x), bf16lo_to_f32(v.y),
                       bf16hi_to_f32(v.y));
}

template <bool F32>
__device__ __forceinline__ void store4(void *base, int64_t at, float4 v)
{
    if (F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + at) = v;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// What a lane rotates: 8 channels as two runs of 4 (first channels o0, o1),
// and the cosines and sines of its 4 pairs (where it has any).
struct LanePairs {
    int o0, o1;
    bool on, turns;          // has channels; they rotate
    bool inter;
    float c[4], s[4];
};

__device__ __forceinline__ LanePairs lane_channels(int t, int D, int R, int inter)
{
    LanePairs lp;
    lp.on = 8 * t < D;
    lp.turns = 8 * t < R;
    lp.inter = inter != 0;
    const bool split = lp.turns && !lp.inter;
    lp.o0 = split ? 4 * t : 8 * t;
    lp.o1 = split ? R / 2 + 4 * t : 8 * t + 4;
    return lp;
}

// The lane's cosines and sines at position pos.
__device__ __forceinline__ void lane_turns(LanePairs &lp, int t, float rot_scale,
                                           const int64_t *table, int pos)
{
    if (!lp.turns)
        return;
    const longlong2 f0 = *reinterpret_cast<const longlong2 *>(table + 4 * t);
    const longlong2 f1 = *reinterpret_cast<const longlong2 *>(table + 4 * t + 2);
    const long long f[4] = {f0.x, f0.y, f1.x, f1.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned long long turns = static_cast<unsigned long long>(static_cast<long long>(pos)) *
                                         static_cast<unsigned long long>(f[j]);
        float sn, cs;
        // twice the signed fraction of a turn, in [-1, 1]
        sincospif(__ll2float_rn(static_cast<long long>(turns)) * 0x1p-63f, &sn, &cs);
        lp.c[j] = cs * rot_scale;
        lp.s[j] = sn * rot_scale;
    }
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a * c - b * s;
    b = b * c + a * s;
    a = x;
}

__device__ __forceinline__ void turn_lane(const LanePairs &lp, float4 &u, float4 &v)
{
    if (!lp.turns)
        return;
    if (lp.inter) {
        turn(u.x, u.y, lp.c[0], lp.s[0]);
        turn(u.z, u.w, lp.c[1], lp.s[1]);
        turn(v.x, v.y, lp.c[2], lp.s[2]);
        turn(v.z, v.w, lp.c[3], lp.s[3]);
    } else {
        turn(u.x, v.x, lp.c[0], lp.s[0]);
        turn(u.y, v.y, lp.c[1], lp.s[1]);
        turn(u.z, v.z, lp.c[2], lp.s[2]);
        turn(u.w, v.w, lp.c[3], lp.s[3]);
    }
}

// x * rsqrt(mean(x^2) + eps) * w over the head that lph lanes share.  Every
// lane of the warp takes part in the shuffles; lanes without channels hold 0.
__device__ __forceinline__ void norm_lane(const LanePairs &lp, int lph, int D, float eps,
                                          const void *w, bool norm, float4 &u, float4 &v)
{
    float ss = u.x * u.x + u.y * u.y + u.z * u.z + u.w * u.w + v.x * v.x + v.y * v.y + v.z * v.z +
               v.w * v.w;
    for (int o = lph >> 1; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!norm || !lp.on)
        return;
    const float r = 1.0f / sqrtf(ss / static_cast<float>(D) + eps);
    const float4 a = load4<false>(w, lp.o0), b = load4<false>(w, lp.o1);
    u = make_float4(u.x * r * a.x, u.y * r * a.y, u.z * r * a.z, u.w * r * a.w);
    v = make_float4(v.x * r * b.x, v.y * r * b.y, v.z * r * b.z, v.w * r * b.w);
}

// Lanes that share one head: the power of two that covers D / 8.
__host__ __device__ inline int lanes_per_head(int D) { return D <= 64 ? 8 : (D <= 128 ? 16 : 32); }
// Heads of one row that a warp rotates.
__host__ __device__ inline int heads_per_warp(int D) { return kHeadsPerLane * 32 / lanes_per_head(D); }

// One warp: heads_per_warp(D) heads of one row.
template <bool F32>
__global__ void __launch_bounds__(32 * kRotWarps) rope_kernel(const smoe_rope_args a, int chunks)
{
    const int64_t gw = (int64_t)blockIdx.x * kRotWarps + (threadIdx.x >> 5);
    const int64_t row = gw / chunks;
    if (row >= a.num_rows)
        return;
    const int lane = threadIdx.x & 31, D = a.head_dim;
    const int lph = lanes_per_head(D), t = lane & (lph - 1), step = 32 / lph;
    const int h0 = static_cast<int>(gw % chunks) * kHeadsPerLane * step + lane / lph;
    LanePairs lp = lane_channels(t, D, a.rot_dim, a.interleaved);
    float4 u[kHeadsPerLane], v[kHeadsPerLane];
#pragma unroll
    for (int i = 0; i < kHeadsPerLane; ++i) {
        const int h = h0 + i * step;
        u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lp.on && h < a.num_heads) {
            const int64_t at = row * a.x_row_stride + h * a.x_head_stride;
            u[i] = load4<F32>(a.x, at + lp.o0);
            v[i] = load4<F32>(a.x, at + lp.o1);
        }
    }
    lane_turns(lp, t, a.rot_scale, a.table, a.positions[row]);
#pragma unroll
    for (int i = 0; i < kHeadsPerLane; ++i) {
        const int h = h0 + i * step;
        if (a.norm_w)
            norm_lane(lp, lph, D, a.eps, a.norm_w, true, u[i], v[i]);
        turn_lane(lp, u[i], v[i]);
        if (lp.on && h < a.num_heads) {
            const int64_t at = row * a.out_row_stride + h * a.out_head_stride;
            store4<F32>(a.out, at + lp.o0, u[i]);
            store4<F32>(a.out, at + lp.o1, v[i]);
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

// One warp: heads_per_warp(D) heads of one row, out of its q heads, k heads
// and v heads in this order.
template <bool F32>
__global__ void __launch_bounds__(32 * kRotWarps)
    kv_append_kernel(const smoe_kv_append_args a, int chunks, int *status)
{
    const int64_t gw = (int64_t)blockIdx.x * kRotWarps + (threadIdx.x >> 5);
    const int64_t row = gw / chunks;
    const int n = a.batch.num_seqs;
    if (row >= a.batch.num_rows)
        return;
    const int lane = threadIdx.x & 31, D = a.cache.head_dim, page = a.cache.page_size;
    const int lph = lanes_per_head(D), t = lane & (lph - 1), step = 32 / lph;
    const int Hq = a.q ? a.num_heads : 0, Hkv = a.cache.num_kv_heads;
    const int h0 = static_cast<int>(gw % chunks) * kHeadsPerLane * step + lane / lph;

    // the heads' loads go out first: they need nothing of the row's place
    LanePairs lp = lane_channels(t, D, a.rot_dim, a.interleaved);
    float4 u[kHeadsPerLane], v[kHeadsPerLane];
#pragma unroll
    for (int i = 0; i < kHeadsPerLane; ++i) {
        const int h = h0 + i * step;
        u[i] = v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lp.on && h < Hq + 2 * Hkv) {
            const int kh = h - Hq, vh = kh - Hkv;
            const void *src = kh < 0 ? a.q : (vh < 0 ? a.k : a.v);
            const int64_t at = kh < 0 ? row * a.q_row_stride + h * a.q_head_stride
                               : vh < 0 ? row * a.k_row_stride + kh * a.k_head_stride
                                        : row * a.v_row_stride + vh * a.v_head_stride;
            // values are not rotated: their runs follow one another
            u[i] = load4<F32>(src, at + (vh < 0 ? lp.o0 : 8 * t));
            v[i] = load4<F32>(src, at + (vh < 0 ? lp.o1 : 8 * t + 4));
        }
    }

    // the row's sequence: in a batch of single rows it is number `row`
    int b = row < n ? static_cast<int>(row) : n - 1;
    int first = a.batch.row_start[b], last = a.batch.row_start[b + 1];
    if (row >= a.batch.row_start[n])
        return;
    if (row < first || row >= last) {
        b = owner_of(a.batch.row_start, n, row, lane);
        first = a.batch.row_start[b];
        last = a.batch.row_start[b + 1];
    }
    if (first < 0 || row < first || row >= last) {
        if (lane == 0)
            set_status(status, kStatusBadArg);
        return;
    }
    // its key index and slot
    const int64_t key = (int64_t)a.batch.kv_len[b] - (last - first) + (row - first);
    int64_t slot_k = -1, slot_v = -1;  // element of (kv head 0, this slot)
    if (key >= 0) {
        const int64_t pi = key / page;
        const int pg = pi < a.batch.table_stride
                           ? a.batch.page_table[(int64_t)b * a.batch.table_stride + pi]
                           : -1;
        if (pg < 0 || pg >= a.cache.num_pages) {
            if (lane == 0)
                set_status(status, kStatusBadArg);
        } else {
            slot_k = pg * a.cache.k_page_stride + (key % page) * D;
            slot_v = pg * a.cache.v_page_stride + (key % page) * D;
        }
    }
    const int pos = a.positions ? a.positions[row] : static_cast<int>(key);
    lane_turns(lp, t, a.rot_scale, a.table, pos);
#pragma unroll
    for (int i = 0; i < kHeadsPerLane; ++i) {
        const int h = h0 + i * step;
        const int kh = h - Hq, vh = kh - Hkv;
        if (a.q_norm || a.k_norm) {
            const void *w = kh < 0 ? a.q_norm : a.k_norm;
            norm_lane(lp, lph, D, a.eps, w, w && vh < 0, u[i], v[i]);
        }
        if (vh < 0)
            turn_lane(lp, u[i], v[i]);
        if (!lp.on || vh >= Hkv)
            continue;
        if (kh < 0) {
            const int64_t at = row * a.qo_row_stride + h * a.qo_head_stride;
            store4<false>(a.q_out, at + lp.o0, u[i]);
            store4<false>(a.q_out, at + lp.o1, v[i]);
        } else if (slot_k >= 0) {
            const int64_t head = (int64_t)page * D;
            const int64_t at = vh < 0 ? slot_k + kh * head : slot_v + vh * head;
            void *dst = vh < 0 ? a.cache.k_pages : a.cache.v_pages;
            store4<false>(dst, at + (vh < 0 ? lp.o0 : 8 * t), u[i]);
            store4<false>(dst, at + (vh < 0 ? lp.o1 : 8 * t + 4), v[i]);
        }
    }
}

}  // namespace

cudaError_t launch_rope(const smoe_rope_args &a, cudaStream_t stream)
{
    const int per = heads_per_warp(a.head_dim), chunks = (a.num_heads + per - 1) / per;
    const int64_t blocks = (a.num_rows * chunks + kRotWarps - 1) / kRotWarps;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    auto k = a.dtype == SMOE_F32 ? rope_kernel<true> : rope_kernel<false>;
    k<<<static_cast<unsigned>(blocks), 32 * kRotWarps, 0, stream>>>(a, chunks);
    return cudaGetLastError();
}

cudaError_t launch_kv_append(const smoe_kv_append_args &a, const DeviceFacts &dev, cudaStream_t stream)
{
    const int per = heads_per_warp(a.cache.head_dim);
    const int heads = (a.q ? a.num_heads : 0) + 2 * a.cache.num_kv_heads;
    const int chunks = (heads + per - 1) / per;
    const int64_t blocks = (a.batch.num_rows * chunks + kRotWarps - 1) / kRotWarps;
    if (blocks > 0x7fffffff)
        return cudaErrorInvalidConfiguration;
    auto k = a.dtype == SMOE_F32 ? kv_append_kernel<true> : kv_append_kernel<false>;
    k<<<static_cast<unsigned>(blocks), 32 * kRotWarps, 0, stream>>>(a, chunks, dev.status);
    return cudaGetLastError();
}

}  // namespace smoe
