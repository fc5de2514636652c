// beam.cu -- the best continuations of beams (smoe_beam_select).
//
// Mathematics: value(k, v) = score_k + (x_kv - m_k) - log(sum_u exp(x_ku - m_k)),
// the num_out largest over a group's beams k and tokens v.  A row's normaliser
// moves all of its values alike, so its best tokens are those of its largest
// logits: one pass over a row finds them, and the sum, together.
//
// Work: a row is cut into parts, a CTA has one of them.  A logit that may be
// among the part's largest goes to its warp's queue in shared memory, and from
// there, 32 at a time, sorted, into the warp's list (lane i the i-th largest),
// as 64-bit keys (logit, then the lower index).  A part's sum and list go to
// the workspace; the CTA that arrives last of a group's joins its rows' parts
// in order, and then the rows' candidates by their values in 64 bits.
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
// A sum's largest term may be 2^40: few steps have to rescale.
constexpr float kSlack = 40.0f;
// A sum's reference stays within this: sums of rows whose largest logit is
// beyond it come out as 0 or infinite, and are taken again (row_sum).
constexpr float kMaxRef = 2097152.0f;
// Warps tell their rank-th largest where rank is at most this (four steps of a
// few cycles); more is asked of parts of few warps with words only.
constexpr int kMaxRank = 4;

using Key = unsigned long long;

// Larger numbers as larger integers.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t o)
{
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// Larger logits have larger keys, and of equal ones the lower index.  0: none.
__device__ __forceinline__ Key key_of(float x, int index)
{
    // (-0 is equal to 0)
    return static_cast<Key>(ordered(x + 0.0f)) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}
__device__ __forceinline__ float logit_of(Key k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
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

// Next larger number (of a finite one or -inf).
__device__ __forceinline__ float next_up(float x)
{
    const int b = __float_as_int(x);
    return __int_as_float(x == 0.0f ? 1 : b > 0 ? b + 1 : b - 1);
}
template <bool F32>
constexpr int kPer = F32 ? 4 : 8;  // logits of a word

// Logit e of a word.
template <bool F32>
__device__ __forceinline__ float logit_at(const uint4 &v, int e)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    return F32 ? __uint_as_float(u[e]) : e & 1 ? bf16hi_to_f32(u[e / 2]) : bf16lo_to_f32(u[e / 2]);
}

// Word w of a row (from the aligned word that the row begins in), -inf in the
// places that are not the row's.
template <bool F32>
__device__ __forceinline__ uint4 load_word(const uint8_t *base, int first, int vocab, int w, int end)
{
    constexpr int kP = kPer<F32>;
    const int at = w * kP - first;  // index of the word's first logit
    if (w < end && at >= 0 && at + kP <= vocab)
        return __ldcs(reinterpret_cast<const uint4 *>(base) + w);
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
        for (int e = i * kP / 4; e < (i + 1) * kP / 4; ++e)
            if (w < end && at + e >= 0 && at + e < vocab) {
                if (F32) {
                    u[i] = reinterpret_cast<const uint32_t *>(base)[w * kP + e];
                } else {
                    const uint32_t h = reinterpret_cast<const uint16_t *>(base)[w * kP + e];
                    u[i] = e & 1 ? (u[i] & 0xffffu) | h << 16 : (u[i] & 0xffff0000u) | h;
                }
            }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // (of a NaN and a number: the number)
    return r;
}
// The largest logit of n words, NaN aside.
template <bool F32>
__device__ __forceinline__ float largest(const uint4 *v, int n)
{
    if (F32) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < n; ++i)
            m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[i].x)), fmaxf(__uint_as_float(v[i].y), __uint_as_float(v[i].z))),
                      __uint_as_float(v[i].w));
        return m;
    }
    uint32_t m = 0xff80ff80u;
#pragma unroll
    for (int i = 0; i < n; ++i)
        m = max_bf16x2(max_bf16x2(m, v[i].x), max_bf16x2(max_bf16x2(v[i].y, v[i].z), v[i].w));
    return fmaxf(bf16lo_to_f32(m), bf16hi_to_f32(m));
}

// Two fp32 numbers at once.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float lo, float hi)
{
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void halves(Pair p, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 2^n for a whole number n <= 127 (0 below 2^-126).
__device__ __forceinline__ float power_of_two(float n)
{
    return n < -126.0f ? 0.0f : __int_as_float((static_cast<int>(n) + 127) << 23);
}

// The sum of 2^(x log2 e - ref) over logits x, for a whole number ref, so that
// sums of different references are joined without any rounding but that of
// their addition.
struct Sum {
    float ref, sum;
    __device__ __forceinline__ void raise(float most)
    {
        const float to = fminf(fmaxf(ceilf(most * kLog2e), -kMaxRef), kMaxRef);
        if (to > ref + kSlack) {
            sum *= power_of_two(ref - to);
            ref = to;
        }
    }
};
__device__ __forceinline__ Sum joined(Sum a, Sum b)
{
    Sum r;
    r.ref = fmaxf(a.ref, b.ref);
    r.sum = a.sum * power_of_two(a.ref - r.ref) + b.sum * power_of_two(b.ref - r.ref);
    return r;
}

// log2 e as two numbers: with one, the exponents would be off by 2^-26 of
// x log2 e, all to one side.
constexpr float kLog2eRest = 1.9259629911266175e-8f;

// What a thread's words add to a sum.
template <bool F32>
__device__ __forceinline__ float sum_of(const uint4 (&v)[kWords], float ref)
{
    const Pair minus = pair_of(-ref, -ref), scale = pair_of(kLog2e, kLog2e), rest = pair_of(kLog2eRest, kLog2eRest);
    Pair p = 0;
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int e = 0; e < kPer<F32>; e += 2) {
            const Pair x = pair_of(logit_at<F32>(v[i], e), logit_at<F32>(v[i], e + 1));
            float a, b;
            halves(fma2(x, rest, fma2(x, scale, minus)), a, b);
            p = add2(p, pair_of(ex2(a), ex2(b)));
        }
    float a, b;
    halves(p, a, b);
    return a + b;
}

constexpr int kQueue = 31 + 32 * kPer<false>;  // what is left of a sort, and a word of every lane

struct PartShared {
    Sum sum[kWarps];
    Key list[kWarps][32];
    uint32_t rank[kWarps];   // see scan_part
    int queued[kWarps];
    Key queue[kWarps][kQueue];
};

// Sorted over the lanes, largest first.
__device__ __forceinline__ Key sorted(Key a, int lane)
{
#pragma unroll
    for (int n = 2; n <= 32; n *= 2)
#pragma unroll
        for (int o = n / 2; o > 0; o >>= 1) {
            const Key y = __shfl_xor_sync(0xffffffffu, a, o);
            const bool larger = ((lane & o) == 0) == ((lane & n) == 0);
            a = larger == (a > y) ? a : y;
        }
    return a;
}

// What waits in the warp's queue into its list, 32 keys at a time, until fewer
// than `keep` are left.
__device__ __forceinline__ void drain(PartShared &sh, int warp, int lane, int num_out, int keep, Key &list, Key &bar)
{
    int n = *static_cast<volatile int *>(&sh.queued[warp]);
    while (n >= keep) {
        const int m = n < 32 ? n : 32;
        Key k = lane < m ? sh.queue[warp][n - m + lane] : 0;
        n -= m;
        if (__any_sync(0xffffffffu, k > bar)) {
            list = merged(list, sorted(k, lane), lane);
            bar = __shfl_sync(0xffffffffu, list, num_out - 1);
        }
    }
    __syncwarp();
    if (lane == 0)
        sh.queued[warp] = n;
    __syncwarp();
}

// One part of one row: its sum and its largest logits, by the whole CTA.
//
// What may be among the row's num_out largest is at least `bar`:
// - strictly more than the last of the warp's own list, which is full of
//   logits of lower index (a warp meets its words in their order);
// - at least the least, over the warps, of their rank-th largest, where rank
//   times the warps is num_out: that many logits are not smaller.  A lane's
//   largest logit so far stands for the lane (other lanes' are other logits).
// The first words of a part are looked at only when every warp has told its
// own rank-th, so that nearly all of what passes from then on is wanted.
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
    const int busy = max(1, min(kWarps, (w1 - w0 + 32 * kWords - 1) / (32 * kWords)));  // warps with words
    const int rank = (N + busy - 1) / busy;
    if (lane == 0)
        sh.queued[warp] = 0;
    Key list = 0, bar = 0;
    float own = -FLT_MAX;     // what is not less may be among the list's largest
    float top = -INFINITY;    // the lane's largest
    Sum s = {-kMaxRef, 0.0f};
    int w = w0 + warp * 32 * kWords + lane;
    uint4 next[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i)
        next[i] = load_word<F32>(base, first, a.vocab, w + 32 * i, w1);
    for (int step = w0; step < w1; step += kStepWords, w += kStepWords) {
        uint4 v[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            v[i] = next[i];
        if (step + kStepWords < w1) {
#pragma unroll
            for (int i = 0; i < kWords; ++i)
                next[i] = load_word<F32>(base, first, a.vocab, w + kStepWords + 32 * i, w1);
        }
        const float most = largest<F32>(v, kWords);
        if (rank <= kMaxRank && (step == w0 || __any_sync(0xffffffffu, most > top))) {
            uint32_t o = ordered(fmaxf(top, most)), r = 0;
            for (int i = 0; i < rank; ++i) {
                r = __reduce_max_sync(0xffffffffu, o);
                const unsigned m = __ballot_sync(0xffffffffu, o == r);
                o = lane == __ffs(m) - 1 ? 0 : o;
            }
            if (lane == 0)
                sh.rank[warp] = r;
        }
        top = fmaxf(top, most);
        s.raise(most);
        s.sum += sum_of<F32>(v, s.ref);
        if (step == w0)
            __syncthreads();
        float least = own;
        if (rank <= kMaxRank) {
            const uint32_t r = lane < busy ? *static_cast<volatile uint32_t *>(&sh.rank[lane]) : 0xffffffffu;
            least = fmaxf(least, from_ordered(__reduce_min_sync(0xffffffffu, r)));
        }
        if (!__any_sync(0xffffffffu, most >= least))
            continue;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if (!__any_sync(0xffffffffu, largest<F32>(&v[i], 1) >= least))
                continue;
#pragma unroll
            for (int e = 0; e < kP; ++e) {
                const float x = logit_at<F32>(v[i], e);
                if (x >= least) {
                    const int at = atomicAdd(&sh.queued[warp], 1);
                    sh.queue[warp][at] = key_of(fminf(x, FLT_MAX), (w + 32 * i) * kP - first + e);
                }
            }
            __syncwarp();
            if (*static_cast<volatile int *>(&sh.queued[warp]) >= 32) {
                drain(sh, warp, lane, N, 32, list, bar);
                own = bar ? next_up(logit_of(bar)) : -FLT_MAX;
                least = fmaxf(least, own);
            }
        }
    }
    drain(sh, warp, lane, N, 1, list, bar);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Sum other;
        other.ref = __shfl_xor_sync(0xffffffffu, s.ref, o);
        other.sum = __shfl_xor_sync(0xffffffffu, s.sum, o);
        s = joined(s, other);
    }
    sh.list[warp][lane] = list;
    if (lane == 0)
        sh.sum[warp] = s;
    // the warps' lists are joined two by two
    for (int o = 1; o < kWarps; o *= 2) {
        __syncthreads();
        if (warp % (2 * o) == 0) {
            s = joined(s, sh.sum[warp + o]);
            list = merged(list, sh.list[warp + o][lane], lane);
            sh.list[warp][lane] = list;
            if (lane == 0)
                sh.sum[warp] = s;
        }
    }
    if (warp == 0) {
        const int64_t at = row * b.parts + part;
        if (lane == 0)
            b.stats[at] = make_float2(s.ref, s.sum);
        if (lane < N)
            b.keys[at * N + lane] = list;
    }
}

// A candidate of a group, as an integer that grows with its value in 64 bits
// (0: none), and 32 times its beam plus its rank there.
struct Candidate {
    unsigned long long value;
    int place;
};
__device__ __forceinline__ bool before(const Candidate &x, const Candidate &y)
{
    return x.value > y.value || (x.value == y.value && x.place < y.place);
}
__device__ __forceinline__ unsigned long long ordered_value(double x)
{
    const unsigned long long b = __double_as_longlong(x + 0.0);
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ double value_of(unsigned long long o)
{
    return __longlong_as_double(o >> 63 ? o & ~(1ull << 63) : ~o);
}

// c and the 32 of r, both sorted, in r's order reversed: the first 32 of both.
__device__ __forceinline__ Candidate merged(Candidate c, const Candidate &reversed, int lane)
{
    c = before(c, reversed) ? c : reversed;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const Candidate y = {__shfl_xor_sync(0xffffffffu, c.value, o), __shfl_xor_sync(0xffffffffu, c.place, o)};
        c = ((lane & o) == 0) == before(c, y) ? c : y;
    }
    return c;
}

struct JoinShared {
    Candidate best[kWarps][32];
    int token[SMOE_MAX_BEAMS][32];
    float sum[kWarps];
    int again;               // a beam whose sum has to be taken again
};

// The sum of exp(x - most) over a row, by the whole CTA: of rows with a NaN or
// +inf, or whose largest logit is out of the range of references.
template <bool F32>
__device__ float row_sum(const smoe_beam_args &a, int64_t row, float most, JoinShared &sh)
{
    const int tid = threadIdx.x;
    float s = 0.0f;
    for (int i = tid; i < a.vocab; i += kThreads) {
        const int64_t at = row * a.row_stride + i;
        const float x = F32 ? static_cast<const float *>(a.logits)[at]
                            : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[at]) << 16);
        s += ex2((counted_logit(x) - most) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if ((tid & 31) == 0)
        sh.sum[tid >> 5] = s;
    __syncthreads();
    s = 0.0f;
    for (int i = 0; i < kWarps; ++i)
        s += sh.sum[i];
    return s;
}

template <bool F32>
__device__ __forceinline__ void join_group(const BeamArgs &b, int group, JoinShared &sh)
{
    const smoe_beam_args &a = b.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_out;
    Candidate best = {0, 0x7fffffff};
    for (int k0 = 0; k0 < a.beams; k0 += kWarps) {
        const int k = k0 + warp;
        const int64_t row = (int64_t)group * a.beams + k;
        const int state = k < a.beams ? state_of(a, row) : kDead;
        double score = 0.0, base = 0.0, off = 0.0;  // off: the normaliser, less base
        Key list = 0;
        bool again = false;
        if (state == kLive) {
            score = a.scores[row];
            const float2 *stats = b.stats + row * b.parts;
            const Key *keys = b.keys + row * b.parts * N;
            list = lane < N ? __ldcg(keys + lane) : 0;
            float ref = -kMaxRef;
            for (int p = lane; p < b.parts; p += 32)
                ref = fmaxf(ref, __ldcg(&stats[p].x));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
            double sum = 0.0;
            for (int p = lane; p < b.parts; p += 32) {
                const float2 s = __ldcg(stats + p);
                sum += s.y * power_of_two(s.x - ref);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            for (int p = 1; p < b.parts; ++p) {
                const Key other = lane < N ? __ldcg(keys + (int64_t)p * N + lane) : 0;
                list = merged(list, other, lane);
            }
            list = lane < N ? list : 0;
            // in whole sums of normal numbers the largest logit's term is one of at least 2^-1
            again = !(sum >= 0.25 && sum <= FLT_MAX) && __shfl_sync(0xffffffffu, list, 0) != 0;
            off = (ref + log2(sum)) * 0.6931471805599453;
        }
        // (rare: rows one after the other, by all warps)
        if (__syncthreads_or(again)) {
            for (int w = 0; w < kWarps; ++w) {
                if (warp == w && lane == 0)
                    sh.again = again ? __float_as_int(logit_of(list)) : 0x7fffffff;
                __syncthreads();
                const int most = sh.again;
                __syncthreads();
                if (most == 0x7fffffff)  // (no logit's bits)
                    continue;
                const float s = row_sum<F32>(a, (int64_t)group * a.beams + k0 + w, __int_as_float(most), sh);
                if (warp == w) {
                    base = __int_as_float(most);
                    off = log(static_cast<double>(s));
                }
            }
        }
        Candidate c = {0, 0x7fffffff};
        int token = -1;
        if (list) {
            c.value = ordered_value(score + ((logit_of(list) - base) - off));
            token = index_of(list);
        } else if (state == kFinished && lane == 0) {
            c.value = ordered_value(a.scores[row]);
            token = a.end_token;
        }
        if (k < a.beams) {
            sh.token[k][lane] = token;
            c.place = 32 * k + lane;
        }
        const Candidate r = {__shfl_sync(0xffffffffu, c.value, 31 - lane), __shfl_sync(0xffffffffu, c.place, 31 - lane)};
        best = merged(best, r, lane);
    }
    __syncthreads();
    for (int o = 1; o < kWarps && o < a.beams; o *= 2) {
        sh.best[warp][lane] = best;
        __syncthreads();
        if (warp % (2 * o) == 0)
            best = merged(best, sh.best[warp + o][31 - lane], lane);
        __syncthreads();
    }
    if (warp == 0 && lane < N) {
        const int64_t at = (int64_t)group * N + lane;
        const bool found = best.value != 0;
        a.scores_out[at] = found ? static_cast<float>(value_of(best.value)) : -INFINITY;
        a.parents[at] = found ? group * a.beams + (best.place >> 5) : -1;
        a.tokens[at] = found ? sh.token[best.place >> 5][best.place & 31] : -1;
    }
}

union BeamShared {
    PartShared part;
    JoinShared join;
};

template <bool F32>
__global__ void __launch_bounds__(kThreads, 3) beam_kernel(const BeamArgs b)
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
        join_group<F32>(b, group, sh.join);
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
