// beam.cu -- the best continuations of beams (smoe_beam_select).
//
// Mathematics: value(k, v) = score_k + (x_kv - m_k) - log(sum_u exp(x_ku - m_k)),
// the num_out largest over a group's beams k and tokens v.  A row's normaliser
// moves all of its values alike, so its best tokens are those of its largest
// logits: one pass over a row finds them, and the sum, together.
//
// Work: a row is cut into parts, a CTA has one of them.  Each warp keeps its
// largest logits as a sorted list in its lanes (lane i the i-th), as 64-bit
// keys (logit, then the lower index), and an element enters the slow path only
// if it is larger than the list's last.  A part's sum and list go to the
// workspace; the CTA that arrives last of a group's joins its rows' parts in
// order, and then the rows' candidates by their values in 64 bits.
#include <float.h>
#include <math.h>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWords = 4;                         // of 16 bytes, of a thread and step
constexpr int kStepWords = kThreads * kWords;     // of a CTA and step
constexpr size_t kStatsAt = SMOE_MAX_SEQS * sizeof(unsigned);  // after the groups' counters
constexpr int kMaxWave = 4096;                    // CTAs that a launch is cut into, beyond one per row
static_assert(kStatsAt + (size_t)(SMOE_MAX_SEQS * SMOE_MAX_BEAMS + kMaxWave) *
                             (sizeof(float2) + SMOE_MAX_BEAMS * sizeof(unsigned long long)) <=
                  SMOE_BEAM_WORKSPACE_BYTES,
              "parts in the workspace");
constexpr float kLog2e = 1.4426950408889634f;
// The sum's reference may lie this far below the largest logit: 2^40 times
// what it holds still fits, and few steps have to rescale.
constexpr float kSlack = 27.0f;

using Key = unsigned long long;

// Larger logits have larger keys, and of equal ones the lower index.  0: none.
__device__ __forceinline__ Key key_of(float x, int index)
{
    const uint32_t b = __float_as_uint(x + 0.0f);  // (-0 is equal to 0)
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return static_cast<Key>(o) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ float logit_of(Key k)
{
    const uint32_t o = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int index_of(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

// Both lists sorted, largest first, one key a lane: the 32 largest of both.
__device__ __forceinline__ Key merged(Key a, Key b, int lane)
{
    const Key r = __shfl_sync(0xffffffffu, b, 31 - lane);
    a = a > r ? a : r;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Key y = __shfl_xor_sync(0xffffffffu, a, o);
        a = ((lane & o) == 0) == (a > y) ? a : y;
    }
    return a;
}

// k into the sorted list of the lanes.
__device__ __forceinline__ Key inserted(Key list, Key k, int lane)
{
    const int at = __popc(__ballot_sync(0xffffffffu, list > k));
    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
    return lane < at ? list : lane == at ? k : up;
}

struct BeamArgs {
    smoe_beam_args a;
    int parts;             // of a row
    int part_words;        // a multiple of kStepWords
    unsigned *arrivals;    // [groups], 0 between launches
    float2 *stats;         // [rows][parts]: reference and sum
    Key *keys;             // [rows][parts][num_out]
};

// What a beam does in this call.
enum : int { kDead, kFinished, kLive };

__device__ __forceinline__ int state_of(const smoe_beam_args &a, int64_t row)
{
    const float score = a.scores[row];
    if (!(fabsf(score) <= FLT_MAX))
        return kDead;
    return a.end_token >= 0 && a.last && a.last[row] == a.end_token ? kFinished : kLive;
}

// A logit as it counts: NaN as -inf, +inf as the largest finite one.
__device__ __forceinline__ float counted_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

template <bool F32>
constexpr int kPer = F32 ? 4 : 8;  // logits of a word

// The logits of word w of a row, -inf outside of it.
template <bool F32>
__device__ __forceinline__ void load_word(float (&x)[kPer<F32>], const uint8_t *base, int first, int vocab, int w,
                                          int words)
{
    const int at = w * kPer<F32> - first;  // index of the word's first logit
    if (w < words && at >= 0 && at + kPer<F32> <= vocab) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(base) + w);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (F32) {
                x[i] = __uint_as_float(u[i]);
            } else {
                x[2 * i] = bf16lo_to_f32(u[i]);
                x[2 * i + 1] = bf16hi_to_f32(u[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer<F32>; ++i) {
            x[i] = -INFINITY;
            if (w < words && at + i >= 0 && at + i < vocab)
                x[i] = F32 ? reinterpret_cast<const float *>(base)[w * kPer<F32> + i]
                           : __uint_as_float(static_cast<uint32_t>(
                                                 reinterpret_cast<const uint16_t *>(base)[w * kPer<F32> + i])
                                             << 16);
        }
    }
#pragma unroll
    for (int i = 0; i < kPer<F32>; ++i)
        x[i] = counted_logit(x[i]);
}

// A running sum of exp(x - ref).
struct Sum {
    float ref, sum;
    __device__ __forceinline__ void raise(float to)
    {
        if (to > ref + kSlack || (ref == -INFINITY && to > ref)) {
            sum = ref == -INFINITY ? 0.0f : sum * ex2((ref - to) * kLog2e);
            ref = to;
        }
    }
    __device__ __forceinline__ void add(float x) { sum += ex2((x - ref) * kLog2e); }
};

// Joins two sums exactly alike whichever way round they come.
__device__ __forceinline__ Sum joined(Sum a, Sum b)
{
    Sum r;
    r.ref = fmaxf(a.ref, b.ref);
    const float x = a.ref == r.ref ? a.sum : a.sum * ex2((a.ref - r.ref) * kLog2e);
    const float y = b.ref == r.ref ? b.sum : b.sum * ex2((b.ref - r.ref) * kLog2e);
    r.sum = x + y;
    return r;
}

struct PartShared {
    Sum sum[kWarps];
    Key list[kWarps][32];
};

// One part of one row: its sum and its largest logits, by the whole CTA.
template <bool F32>
__device__ __forceinline__ void scan_part(const BeamArgs &b, int64_t row, int part, PartShared &sh)
{
    const smoe_beam_args &a = b.a;
    constexpr int kP = kPer<F32>, kBytes = F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_out;
    // words of 16 bytes from the one that the row begins in
    const uint8_t *begin = static_cast<const uint8_t *>(a.logits) + row * a.row_stride * kBytes;
    const int first = static_cast<int>(reinterpret_cast<uintptr_t>(begin) & 15) / kBytes;
    const uint8_t *base = begin - first * kBytes;
    const int words = (first + a.vocab + kP - 1) / kP;
    const int w0 = part * b.part_words, w1 = min(w0 + b.part_words, words);
    Key list = 0;
    float last = -INFINITY;  // the list's last logit; what is not above it is out
    Sum s = {-INFINITY, 0.0f};
    for (int w = w0 + warp * 32 * kWords + lane; w - lane < w1; w += kStepWords) {
        float x[kWords][kP];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            load_word<F32>(x[i], base, first, a.vocab, w + 32 * i, w1);
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
            for (int e = 0; e < kP; ++e)
                top = fmaxf(top, x[i][e]);
        s.raise(top);
        if (s.ref > -INFINITY) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    s.add(x[i][e]);
        }
        if (!__any_sync(0xffffffffu, top > last))
            continue;
        Key bar = __shfl_sync(0xffffffffu, list, N - 1);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const int index = (w + 32 * i) * kP - first + e;
                const Key k = key_of(x[i][e], index);
                unsigned m = __ballot_sync(0xffffffffu, x[i][e] > -INFINITY && k > bar);
                while (m) {
                    const int from = __ffs(m) - 1;
                    list = inserted(list, __shfl_sync(0xffffffffu, k, from), lane);
                    bar = __shfl_sync(0xffffffffu, list, N - 1);
                    m &= m - 1;
                    m &= __ballot_sync(0xffffffffu, k > bar);
                }
            }
        last = bar ? logit_of(bar) : -INFINITY;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sum other;
        other.ref = __shfl_xor_sync(0xffffffffu, s.ref, o);
        other.sum = __shfl_xor_sync(0xffffffffu, s.sum, o);
        s = joined(s, other);
    }
    sh.list[warp][lane] = lane < N ? list : 0;
    if (lane == 0)
        sh.sum[warp] = s;
    __syncthreads();
    if (warp == 0) {
        for (int o = 1; o < kWarps; ++o) {
            s = joined(s, sh.sum[o]);
            list = merged(lane < N ? list : 0, sh.list[o][lane], lane);
        }
        const int64_t at = row * b.parts + part;
        if (lane == 0)
            b.stats[at] = make_float2(s.ref, s.sum);
        if (lane < N)
            b.keys[at * N + lane] = list;
    }
}

// A candidate of a group: its value, and 32 times its beam plus its rank there.
struct Candidate {
    double value;
    int place;
};
__device__ __forceinline__ bool before(const Candidate &x, const Candidate &y)
{
    return x.value > y.value || (x.value == y.value && x.place < y.place);
}

struct JoinShared {
    double value[SMOE_MAX_BEAMS][32];
    int token[SMOE_MAX_BEAMS][32];
};

__device__ __forceinline__ void join_group(const BeamArgs &b, int group, JoinShared &sh)
{
    const smoe_beam_args &a = b.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_out;
    for (int k = warp; k < a.beams; k += kWarps) {
        const int64_t row = (int64_t)group * a.beams + k;
        const int state = state_of(a, row);
        double value = -INFINITY;
        int token = -1;
        const double score = a.scores[row];
        if (state == kFinished && lane == 0) {
            value = score;
            token = a.end_token;
        } else if (state == kLive) {
            const float2 *stats = b.stats + row * b.parts;
            const Key *keys = b.keys + row * b.parts * N;
            float ref = -INFINITY;
            for (int p = lane; p < b.parts; p += 32)
                ref = fmaxf(ref, __ldcg(&stats[p].x));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
            double sum = 0.0;
            for (int p = lane; p < b.parts; p += 32) {
                const float2 s = __ldcg(stats + p);
                if (s.x > -INFINITY)
                    sum += s.y * exp(static_cast<double>(s.x) - ref);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            Key list = lane < N ? __ldcg(keys + lane) : 0;
            for (int p = 1; p < b.parts; ++p) {
                const Key other = lane < N ? __ldcg(keys + (int64_t)p * N + lane) : 0;
                list = merged(list, other, lane);
                list = lane < N ? list : 0;
            }
            if (list) {
                value = score + ((static_cast<double>(logit_of(list)) - ref) - log(sum));
                token = index_of(list);
            }
        }
        sh.value[k][lane] = value;
        sh.token[k][lane] = token;
    }
    __syncthreads();
    if (warp != 0)
        return;
    Candidate c = {sh.value[0][lane], lane};
    for (int k = 1; k < a.beams; ++k) {
        const Candidate r = {sh.value[k][31 - lane], 32 * k + 31 - lane};
        c = before(c, r) ? c : r;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Candidate y = {__shfl_xor_sync(0xffffffffu, c.value, o), __shfl_xor_sync(0xffffffffu, c.place, o)};
            c = ((lane & o) == 0) == before(c, y) ? c : y;
        }
    }
    if (lane < N) {
        const int64_t at = (int64_t)group * N + lane;
        const bool found = c.value > -INFINITY;
        a.scores_out[at] = static_cast<float>(c.value);
        a.parents[at] = found ? group * a.beams + (c.place >> 5) : -1;
        a.tokens[at] = found ? sh.token[c.place >> 5][c.place & 31] : -1;
    }
}

union BeamShared {
    PartShared part;
    JoinShared join;
};

template <bool F32>
__global__ void __launch_bounds__(kThreads) beam_kernel(const BeamArgs b)
{
    __shared__ BeamShared sh;
    __shared__ bool s_last;
    const int64_t row = blockIdx.x / b.parts;
    const int part = blockIdx.x % b.parts, group = static_cast<int>(row / b.a.beams);
    if (state_of(b.a, row) == kLive)
        scan_part<F32>(b, row, part, sh.part);
    __syncthreads();
    if (threadIdx.x == 0) {
        const unsigned all = b.a.beams * b.parts;
        s_last = count_arrival(b.arrivals + group) == all - 1;
        if (s_last)
            b.arrivals[group] = 0;
    }
    __syncthreads();
    if (s_last)
        join_group(b, group, sh.join);
}

}  // namespace

cudaError_t launch_beam_select(const smoe_beam_args &a, void *workspace, const DeviceFacts &dev, cudaStream_t stream)
{
    BeamArgs b;
    b.a = a;
    const bool f32 = a.dtype == SMOE_F32;
    const int64_t rows = (int64_t)a.num_groups * a.beams;
    // a row begins anywhere in its first word
    const int per = f32 ? 4 : 8;
    const int words = (a.vocab + 2 * per - 2) / per;
    const int steps = (words + kStepWords - 1) / kStepWords;
    // parts: about six CTAs per SM, of a step at least
    const int64_t wave = dev.sms * 6 < kMaxWave ? dev.sms * 6 : kMaxWave;
    int64_t parts = (wave + rows - 1) / rows;
    parts = parts < steps ? parts : steps;
    const int each = static_cast<int>((steps + parts - 1) / parts);
    b.part_words = each * kStepWords;
    b.parts = (steps + each - 1) / each;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    b.arrivals = reinterpret_cast<unsigned *>(ws);
    b.stats = reinterpret_cast<float2 *>(ws + kStatsAt);
    b.keys = reinterpret_cast<Key *>(ws + kStatsAt + rows * b.parts * sizeof(float2));
    auto k = f32 ? beam_kernel<true> : beam_kernel<false>;
    k<<<static_cast<unsigned>(rows * b.parts), kThreads, 0, stream>>>(b);
    return cudaGetLastError();
}

}  // namespace smoe
