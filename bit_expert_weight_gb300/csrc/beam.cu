// beam.cu -- the best continuations of beams (smoe_beam_select).
//
// Mathematics: value(k, v) = score_k + (x_kv - m_k) - log(sum_u exp(x_ku - m_k)),
// the num_out largest over a group's beams k and tokens v.  A row's normaliser
// moves all of its values alike, so its best tokens are those of its largest
// logits: one pass over a row finds them, and the sum, together.
//
// Work: a row is cut into parts, a CTA has one of them.  It reads its part once,
// adds the exponentials up and notes only the largest logit of every 32 (16 in
// fp32); the few words whose largest is among the part's are read again, and
// their logits ranked, as 64-bit keys (logit, then the lower index).  (Choosing
// while reading, by sorted lists or queues of each warp, took 52 to 127 us for 512
// rows of 151,936 instead of 31.)  A part's sum and its largest keys, in order,
// go to the workspace; the CTA that arrives last of a group's joins its rows'
// parts, and then the rows' candidates by their values.
//
// Bound: HBM while the rows are read (12 logits of bf16 per cycle and SM, all
// that comes), then a chain of latencies: words read again, the arrival, the
// join.  Measured: 512 rows of 151,936 bf16 logits, 16 of each group of 8, 433 of
// them read: 30.4 us, 4.3 TB/s; 60 fp32 rows of 100,003 11.1 us; 320 rows of 65,536
// of which 0.3 % are allowed 18.3 us; 4 rows of 32,000 6.4 us.  (Small calls wait
// for instructions too, each read once: loops that a call goes round in once or
// twice are not unrolled; with 92 KB of them, not 72, the fp32 rows took 11.5 us.)
// Rows with a NaN or +inf, and those whose logits above -inf are all the lowest
// value, are summed again by the CTA that joins their group, one after the other:
// a group of 32 such rows of 151,936 takes 1.01 ms instead of 25 us, one of 4 of
// 32,000 25 instead of 6.4.  Rows of few allowed tokens among the type's lowest
// value rank those too: 320 rows of 2,000, 32 of 16 beams, 1 % allowed 15.1 us (the
// rest -inf: 10.6), one token allowed 43.9 (10.1); of 1,000 84 and 121 us.
#include <float.h>
#include <math.h>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// (512 rows of 151,936: 30.4 us with three, 30.9 with four, whose threads have 64
// registers, not 74; two allow 80, of which three are resident all the same: 30.4)
constexpr int kCtasPerSm = 3;
constexpr int kWords = 4;                         // of 16 bytes, of a thread and step (4: 30.4 us, 3: 38.4, 8: 31.5)
constexpr int kStepWords = kThreads * kWords;     // of a CTA and step
constexpr size_t kStatsAt = SMOE_MAX_SEQS * sizeof(unsigned);  // after the groups' counters
constexpr int kMaxSteps = 24;                     // of a part
constexpr int kMaxWave = 4096;                    // CTAs that a launch is cut into, beyond what kMaxSteps asks
static_assert(kStatsAt + (size_t)(SMOE_MAX_SEQS * ((SMOE_MAX_VOCAB / 4 + 1) / (kStepWords * kMaxSteps) + 1) + kMaxWave) *
                             (sizeof(float2) + SMOE_MAX_BEAMS * sizeof(unsigned long long)) <=
                  SMOE_BEAM_WORKSPACE_BYTES,
              "parts in the workspace");
// Logits of more bytes than this are read as passing by (first to leave L2):
// those of less may lie there, from the product that made them, and the few
// words read again do (60 fp32 rows of 100,003: 11.1 us, 11.9 as passing by; 512
// rows of 151,936: 34.7 us, 30.4 as passing by).
constexpr int64_t kPassing = 32 << 20;
constexpr float kLog2e = 1.4426950408889634f;
// A sum's reference stays within this: sums of rows whose largest logit is
// beyond it come out as 0 or infinite, and are taken again (row_sum).
constexpr float kMaxRef = 2097152.0f;

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

struct BeamArgs {
    smoe_beam_args a;
    int parts;             // of a row
    int part_words;        // a multiple of kStepWords
    int depth;             // first values of a part that join_group's bar goes by
    unsigned *arrivals;    // [groups], 0 between launches
    float2 *stats;         // [rows][parts]: reference and sum
    Key *keys;             // [rows][parts][num_out]
};

// What a beam does in this call.
enum : int { kDead, kFinished, kLive };

__device__ __forceinline__ int state_of(const smoe_beam_args &a, int64_t row)
{
    const float score = a.scores[row];  // (both loads at once)
    const int last = a.last && a.end_token >= 0 ? a.last[row] : -1;
    if (!(fabsf(score) <= FLT_MAX))
        return kDead;
    return a.end_token >= 0 && last == a.end_token ? kFinished : kLive;
}

// A logit as it counts: NaN as -inf, +inf as the largest finite one.
__device__ __forceinline__ float counted_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }

template <bool F32>
constexpr int kPer = F32 ? 4 : 8;  // logits of a word

// Logit e of a word.
template <bool F32>
__device__ __forceinline__ float logit_at(const uint4 &v, int e)
{
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    return F32 ? __uint_as_float(u[e]) : e & 1 ? bf16hi_to_f32(u[e / 2]) : bf16lo_to_f32(u[e / 2]);
}

// A word that is not all the row's, its logits one by one; -inf in the other
// places.
template <bool F32>
__device__ __noinline__ uint4 edge_word(const uint8_t *base, int first, int vocab, int w)
{
    constexpr int kP = kPer<F32>;
    const int at = w * kP - first;  // index of the word's first logit
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = F32 ? 0xff800000u : 0xff80ff80u;
#pragma unroll
        for (int e = i * kP / 4; e < (i + 1) * kP / 4; ++e)
            if (at + e >= 0 && at + e < vocab) {
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

// Word w of a row (from the aligned word that the row begins in), -inf in the
// places that are not the row's.
template <bool F32>
__device__ __forceinline__ uint4 load_word(const uint8_t *base, int first, int vocab, int w, int end)
{
    constexpr int kP = kPer<F32>;
    constexpr uint32_t kNone = F32 ? 0xff800000u : 0xff80ff80u;
    const int at = w * kP - first;
    if (w < end && at >= 0 && at + kP <= vocab)
        return __ldcg(reinterpret_cast<const uint4 *>(base) + w);
    return w < end ? edge_word<F32>(base, first, vocab, w) : make_uint4(kNone, kNone, kNone, kNone);
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
// their addition.  The largest exponent is above -1 and at most 0, where its
// rounding is least.
struct Sum {
    float ref, sum;
    __device__ __forceinline__ void raise(float most)
    {
        const float to = fminf(fmaxf(ceilf(most * kLog2e), -kMaxRef), kMaxRef);
        if (to > ref) {
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

// Groups (a thread's words of one step) that are looked at again, and keys
// taken from them.  A part's num_out largest groups hold no more.
constexpr int kHits = 256;
constexpr int kKeys = 1024;
static_assert(SMOE_MAX_BEAMS * kWords * kPer<false> <= kKeys && SMOE_MAX_BEAMS <= kHits, "the largest groups fit");

struct PartShared {
    Sum sum[kWarps];
    uint32_t rank[kWarps];   // see scan_part
    int count[kWarps];
    int hits, queued;
    int hit[kHits];          // groups: step * kThreads + thread
    Key queue[kKeys];
    float most[kMaxSteps][kThreads];  // the largest logit of every group
};

// A part of a row, in words of 16 bytes from the one that the row begins in.
struct Part {
    const uint8_t *base;
    int first;      // logits of word 0 before the row
    int vocab;
    int w0, w1;     // words
    int steps;
};

template <bool F32>
__device__ __forceinline__ uint4 load_word(const Part &p, int w)
{
    return load_word<F32>(p.base, p.first, p.vocab, w, p.w1);
}

// A thread's words of the step that begins at word w.  Where all of the step's
// words are the row's, which is so but for its first and last ones, one
// condition does for all loads.
template <bool F32, bool PASSING>
__device__ __forceinline__ void load_step(uint4 (&v)[kWords], const Part &p, int w, int tid)
{
    if (w + kStepWords <= p.w1 && w * kPer<F32> >= p.first && (w + kStepWords) * kPer<F32> <= p.first + p.vocab) {
        const uint4 *from = reinterpret_cast<const uint4 *>(p.base) + w + tid;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            v[i] = PASSING ? __ldcs(from + kThreads * i) : __ldcg(from + kThreads * i);
    } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            v[i] = load_word<F32>(p, w + kThreads * i + tid);
    }
}

// Sum over the CTA, in every thread.
__device__ __forceinline__ int sum_over_cta(PartShared &sh, int v, int tid)
{
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((tid & 31) == 0)
        sh.count[tid >> 5] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
        v += sh.count[i];
    return v;
}

// The logits of a part that are not below `bar` (or, strictly, above it) into
// the queue, of the groups whose largest is: true if both had room.
template <bool F32>
__device__ __forceinline__ bool collect(PartShared &sh, const Part &p, float bar, bool strictly, int tid)
{
    constexpr int kP = kPer<F32>;
    unsigned mine = 0;  // by step
    for (int i = 0; i < p.steps; ++i) {
        const float m = sh.most[i][tid];
        mine |= (strictly ? m > bar : m >= bar) ? 1u << i : 0u;
    }
    if (mine) {
        int at = atomicAdd(&sh.hits, __popc(mine));
        for (; mine && at < kHits; mine &= mine - 1)
            sh.hit[at++] = (__ffs(mine) - 1) * kThreads + tid;
    }
    __syncthreads();
    const int hits = sh.hits;
    if (hits > kHits)
        return false;
#pragma unroll 1
    for (int u = tid; u < hits * kWords; u += kThreads) {
        const int g = sh.hit[u / kWords];
        const int w = p.w0 + g / kThreads * kStepWords + u % kWords * kThreads + g % kThreads;
        const uint4 v = load_word<F32>(p, w);
        unsigned pass = 0;
#pragma unroll
        for (int e = 0; e < kP; ++e) {
            const float x = logit_at<F32>(v, e);
            pass |= (strictly ? x > bar : x >= bar) ? 1u << e : 0u;
        }
        if (!pass)
            continue;
        int at = atomicAdd(&sh.queued, __popc(pass));
#pragma unroll
        for (int e = 0; e < kP; ++e)
            if ((pass >> e & 1) && at < kKeys)
                sh.queue[at++] = key_of(fminf(logit_at<F32>(v, e), FLT_MAX), w * kP - p.first + e);
    }
    __syncthreads();
    return sh.queued <= kKeys;
}

// What collect had no room for: logits of which very many are large, or alike.
// Where many are at the bar itself (masked ones), those above it are few.  Else
// the bar becomes the num_out-th largest group's (bit by bit): then fewer than
// num_out groups are above it.  Of the logits that are equal to the bar the
// first ones are taken in order, where they are needed (equal as they count: +inf
// is the largest number, a NaN none).
template <bool F32>
__device__ __noinline__ void collect_crowd(PartShared &sh, const Part &p, float bar, int num_out, int tid)
{
    constexpr int kP = kPer<F32>;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        if (turn == 1) {
            uint32_t o = 0;
#pragma unroll 1
            for (int bit = 31; bit >= 0; --bit) {
                const uint32_t t = o | 1u << bit;
                int n = 0;
                for (int i = 0; i < p.steps; ++i)
                    n += ordered(sh.most[i][tid]) >= t;
                if (sum_over_cta(sh, n, tid) >= num_out)
                    o = t;
            }
            bar = fmaxf(from_ordered(o), -FLT_MAX);
        }
        __syncthreads();
        if (tid == 0)
            sh.hits = sh.queued = 0;
        __syncthreads();
        if (collect<F32>(sh, p, bar, true, tid))
            break;
    }
    int need = num_out - sh.queued, found = sh.queued;
#pragma unroll 1
    for (int i = 0; i < p.steps && need > 0; ++i) {
        const bool maybe = sh.most[i][tid] >= bar;  // (if its largest is above, it may hold some too)
        if (!__syncthreads_or(maybe))
            continue;
#pragma unroll 1
        for (int j = 0; j < kWords && need > 0; ++j) {
            const int w = p.w0 + i * kStepWords + j * kThreads + tid;
            uint4 v = make_uint4(0, 0, 0, 0);
            int mine = 0;
            if (maybe) {
                v = load_word<F32>(p, w);
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    mine += counted_logit(logit_at<F32>(v, e)) == bar;
            }
            int at = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, at, d);
                at += lane >= d ? up : 0;
            }
            __syncthreads();
            if (lane == 31)
                sh.count[warp] = at;
            __syncthreads();
            at -= mine;
            int all = 0;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                at += x < warp ? sh.count[x] : 0;
                all += sh.count[x];
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < kP; ++e)
                    if (counted_logit(logit_at<F32>(v, e)) == bar && at++ < need)
                        sh.queue[found + at - 1] = key_of(bar, w * kP - p.first + e);
            }
            found += min(all, need);
            need -= min(all, need);
        }
    }
    __syncthreads();
    if (tid == 0)
        sh.queued = found;
    __syncthreads();
}

// The num_out largest of n keys to `out`, in order (0 where there are fewer): a
// key's place is the number of larger ones, for all keys differ.
__device__ __forceinline__ void rank_keys(const Key *keys, int n, int num_out, Key *out, int tid)
{
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
        const Key k = keys[i];
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            above += keys[j] > k;
        if (above < num_out)
            out[above] = k;
    }
    if (tid >= n && tid < num_out)
        out[tid] = 0;
}

// One part of one row: its sum and its largest logits, by the whole CTA.
//
// The part is read once, and nothing is chosen meanwhile: each thread only
// notes the largest logit of its words of every step.  Then a bar is set that
// num_out logits reach: the least, over the warps, of the rank-th largest of
// their threads' largest, where rank times the warps is num_out.  Few words
// reach it; they are read again (they lie in L2), and their logits ranked.
template <bool F32, bool PASSING>
__device__ __forceinline__ void scan_part(const BeamArgs &b, int64_t row, int part, PartShared &sh)
{
    const smoe_beam_args &a = b.a;
    constexpr int kP = kPer<F32>, kBytes = F32 ? 4 : 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_out;
    const uint8_t *begin = static_cast<const uint8_t *>(a.logits) + row * a.row_stride * kBytes;
    Part p;
    p.first = static_cast<int>(reinterpret_cast<uintptr_t>(begin) & 15) / kBytes;
    p.base = begin - p.first * kBytes;
    p.vocab = a.vocab;
    p.w0 = part * b.part_words;
    p.w1 = min(p.w0 + b.part_words, (p.first + a.vocab + kP - 1) / kP);
    p.steps = max(0, p.w1 - p.w0 + kStepWords - 1) / kStepWords;
    int w = p.w0;
    uint4 next[kWords];
    load_step<F32, PASSING>(next, p, w, tid);
    // (the first words are on their way while the beam's state is looked up)
    if (state_of(a, row) != kLive)
        return;
    float top = -INFINITY;
    Sum s = {-kMaxRef, 0.0f};
#pragma unroll 1
    for (int step = 0; step < p.steps; ++step, w += kStepWords) {
        uint4 v[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            v[i] = next[i];
        if (step + 1 < p.steps)
            load_step<F32, PASSING>(next, p, w + kStepWords, tid);
        const float most = fminf(largest<F32>(v, kWords), FLT_MAX);
        sh.most[step][tid] = most;
        top = fmaxf(top, most);
        s.raise(most);
        s.sum += sum_of<F32>(v, s.ref);
    }
    const int busy = max(1, min(kWarps, (p.w1 - p.w0 + 31) / 32));  // warps with words
    uint32_t o = ordered(top), r = 0;
#pragma unroll 1
    for (int i = 0; i < N; i += busy) {
        r = __reduce_max_sync(0xffffffffu, o);
        o = lane == __ffs(__ballot_sync(0xffffffffu, o == r)) - 1 ? 0 : o;
    }
    const float ref = static_cast<float>(__reduce_max_sync(0xffffffffu, static_cast<int>(s.ref)));
    s = {ref, s.sum * power_of_two(s.ref - ref)};
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
        s.sum += __shfl_xor_sync(0xffffffffu, s.sum, d);
    if (lane == 0) {
        sh.rank[warp] = r;
        sh.sum[warp] = s;
    }
    if (tid == 0)
        sh.hits = sh.queued = 0;
    __syncthreads();
    r = lane < busy ? sh.rank[lane] : 0xffffffffu;
    const float bar = fmaxf(from_ordered(__reduce_min_sync(0xffffffffu, r)), -FLT_MAX);
    if (!collect<F32>(sh, p, bar, false, tid))
        collect_crowd<F32>(sh, p, bar, N, tid);
    const int64_t at = row * b.parts + part;
    rank_keys(sh.queue, sh.queued, N, b.keys + at * N, tid);
    if (tid == kThreads - 32) {  // (a warp that seldom has keys to rank)
        s = sh.sum[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i)
            s = joined(s, sh.sum[i]);
        b.stats[at] = make_float2(s.ref, s.sum);
    }
}

// ------------------------------------------------- a group's candidates

// Values are sums of a large and a small fp32 number: the double format's
// units are so few on this part that a logarithm there takes 2,800 cycles.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b)  // exactly a + b
{
    Two r;
    r.hi = a + b;
    const float v = r.hi - a;
    r.lo = (a - (r.hi - v)) + (b - v);
    return r;
}
__device__ __forceinline__ Two settled(Two t)
{
    Two r;
    r.hi = t.hi + t.lo;
    r.lo = t.lo - (r.hi - t.hi);
    return r;
}

// c near 1 / (1 + (i + 1/2) / 32), of 8 bits, and -log c as two numbers.
__constant__ float kLogTable[32][3] = {
    {0.984375f, 0.015748357f, -4.3215895e-10f}, {0.95703125f, 0.043919235f, -1.5330752e-09f},
    {0.92578125f, 0.0771173f, 1.8207458e-09f}, {0.90234375f, 0.102759734f, 1.6164925e-10f},
    {0.875f, 0.13353139f, 1.0038866e-09f}, {0.8515625f, 0.16068238f, 1.4910411e-09f},
    {0.83203125f, 0.18388528f, 2.4525408e-09f}, {0.80859375f, 0.21245866f, -4.023958e-09f},
    {0.7890625f, 0.23690975f, -4.536055e-11f}, {0.76953125f, 0.2619737f, 6.873547e-09f},
    {0.75390625f, 0.28248724f, 1.21607515e-08f}, {0.734375f, 0.3087355f, -8.195663e-09f},
    {0.71875f, 0.33024168f, 6.725313e-09f}, {0.703125f, 0.3522206f, -1.293613e-09f},
    {0.6875f, 0.37469345f, -3.8705092e-09f}, {0.671875f, 0.39768296f, 2.8643212e-09f},
    {0.66015625f, 0.41527873f, -3.2201528e-09f}, {0.64453125f, 0.43923196f, 8.613421e-09f},
    {0.6328125f, 0.4575811f, 6.3991252e-09f}, {0.62109375f, 0.47627324f, 3.600426e-09f},
    {0.609375f, 0.49532142f, 1.4414702e-08f}, {0.59765625f, 0.5147395f, 9.68991e-09f},
    {0.5859375f, 0.53454214f, 7.0384276e-09f}, {0.578125f, 0.54796517f, 1.7625055e-09f},
    {0.56640625f, 0.5684437f, -1.3513369e-08f}, {0.5546875f, 0.5893504f, -1.5476893e-08f},
    {0.546875f, 0.603535f, 2.5360706e-08f}, {0.5390625f, 0.61792374f, 2.2750092e-08f},
    {0.52734375f, 0.63990265f, 1.4731166e-08f}, {0.51953125f, 0.6548283f, 6.244991e-09f},
    {0.51171875f, 0.6699801f, 1.25404656e-08f}, {0.50390625f, 0.685365f, 1.88891e-08f},
};

// The logarithm of (sum.hi + sum.lo) 2^ref, of a normal number and a whole one,
// to 2^-29 or so: by a table, as P. T. P. Tang's "Table-driven implementation
// of the logarithm function" has it: with m in [1, 2) and c m = 1 + r, |r| < 2^-5,
// log m = -log c + r - r^2 / 2 + r^3 / 3 - ...
__device__ __forceinline__ Two log_of(Two sum, float ref)
{
    const int bits = __float_as_int(sum.hi);
    const int e = (bits >> 23) - 127;
    const float m = __int_as_float((bits & 0x7fffff) | 0x3f800000);
    const float *t = kLogTable[(bits >> 18) & 31];
    const float r = fmaf(m, t[0], -1.0f);
    const float small = sum.lo * power_of_two(static_cast<float>(-e)) * t[0];
    const float q = r * r * fmaf(r, fmaf(r, fmaf(r, fmaf(r, -1.0f / 6, 0.2f), -0.25f), 1.0f / 3), -0.5f);
    const float n = ref + static_cast<float>(e), ln2 = 0.693147182464599609375f, rest = -1.904654323148236e-9f;
    const float p = n * ln2;
    float lo = fmaf(n, rest, fmaf(n, ln2, -p));
    Two s = two_sum(p, t[1]);
    lo += s.lo + t[2];
    s = two_sum(s.hi, r);
    s.lo += lo + (q + small);
    return settled(s);
}

// Integers that grow with a value, in 2^-45 of it or so; never 0.
using Value = unsigned long long;
__device__ __forceinline__ Value ordered_value(Two t)
{
    // (large enough, the rest is below what 64 bits would hold)
    const float lo = fabsf(t.hi) > 0x1p64f ? 0.0f : t.lo;
    return static_cast<Value>(ordered(t.hi + 0.0f)) << 32 | ordered(lo + 0.0f);
}

constexpr int kCands = 512;
constexpr int kSamples = 1024;
constexpr int kFirst = 4;  // candidates of a thread that are loaded ahead

// A candidate of a group, or none (0, 0): of equal values the one with the
// larger `tie` comes first: the lower beam, the larger logit, the lower token.
struct alignas(16) Candidate {
    Value value;
    unsigned long long tie;
};

struct JoinShared {
    // of each beam: a quarter of its score, and of its normaliser (base + off);
    // values may be three times fp32's largest number
    float score[SMOE_MAX_BEAMS], base[SMOE_MAX_BEAMS];
    Two off[SMOE_MAX_BEAMS];
    int state[SMOE_MAX_BEAMS];
    float again[SMOE_MAX_BEAMS];   // the largest logit where the sum has to be taken again, else NaN
    float sum[kWarps];
    int queued;
    uint32_t bar;                  // upper half of a value
    // upper halves of the first values of each part; 0: none, and of beams that are not live
    alignas(16) uint32_t sample[kSamples];
    Candidate queue[kCands];
    Candidate best[kWarps];        // of each warp (select_crowd)
};

__device__ __forceinline__ Value value_of(const JoinShared &sh, int k, Key key)
{
    Two t = two_sum(0.25f * logit_of(key), -sh.base[k]);
    const Two u = two_sum(t.hi, -sh.off[k].hi);
    const float lo = u.lo + (t.lo - sh.off[k].lo);
    t = two_sum(u.hi, sh.score[k]);
    t.lo += lo;
    return ordered_value(settled(t));
}
__device__ __forceinline__ float score_of(Value v) { return 4.0f * from_ordered(static_cast<uint32_t>(v >> 32)); }

// The parts of a candidate's tie.
constexpr int kTokenBits = 22, kBeamAt = 32 + kTokenBits;
static_assert(1 << kTokenBits == SMOE_MAX_VOCAB && SMOE_MAX_BEAMS <= 1 << (64 - kBeamAt), "bits of a tie");

__device__ __forceinline__ unsigned long long tie_of(int beam, Key key)
{
    return static_cast<unsigned long long>(SMOE_MAX_BEAMS - 1 - beam) << kBeamAt | (key >> 32) << kTokenBits |
           (SMOE_MAX_VOCAB - 1 - index_of(key));
}
__device__ __forceinline__ int beam_of(unsigned long long tie) { return SMOE_MAX_BEAMS - 1 - static_cast<int>(tie >> kBeamAt); }
__device__ __forceinline__ int token_of(unsigned long long tie)
{
    return SMOE_MAX_VOCAB - 1 - static_cast<int>(tie & (SMOE_MAX_VOCAB - 1));
}

__device__ __forceinline__ bool before(const Candidate &x, const Candidate &y)
{
    // (no branches: two threads of a warp hardly ever agree)
    return (x.value > y.value) | ((x.value == y.value) & (x.tie > y.tie));
}

// Output number `place` of a group: a candidate, or none where its value is 0.
__device__ __forceinline__ void put(const smoe_beam_args &a, int group, int place, const Candidate &c)
{
    const int64_t at = (int64_t)group * a.num_out + place;
    const bool found = c.value != 0;
    a.scores_out[at] = found ? score_of(c.value) : -INFINITY;
    a.parents[at] = found ? group * a.beams + beam_of(c.tie) : -1;
    a.tokens[at] = found ? token_of(c.tie) : -1;
}

// Candidate `rest` of a beam's parts * num_out, whose key was `key` (a finished
// beam has one, of its own).
__device__ __forceinline__ Candidate candidate(const smoe_beam_args &a, const JoinShared &sh, int beam, int rest, Key key)
{
    const int state = sh.state[beam];
    if (state == kFinished && rest == 0)
        return {ordered_value({sh.score[beam], 0.0f}), tie_of(beam, key_of(0.0f, a.end_token))};
    if (state != kLive || key == 0)
        return {0, 0};
    return {value_of(sh, beam, key), tie_of(beam, key)};
}

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

// The smallest of the lanes' keys.
__device__ __forceinline__ Key least_of(Key k)
{
    const uint32_t hi = __reduce_min_sync(0xffffffffu, static_cast<uint32_t>(k >> 32));
    const uint32_t lo =
        __reduce_min_sync(0xffffffffu, hi == static_cast<uint32_t>(k >> 32) ? static_cast<uint32_t>(k) : 0xffffffffu);
    return static_cast<Key>(hi) << 32 | lo;
}

// The outputs of a group with very many candidates that are alike: the best of
// all, then the best of what comes after it, and so on.
__device__ __noinline__ void select_crowd(const BeamArgs &b, int group, JoinShared &sh)
{
    const smoe_beam_args &a = b.a;
    const int tid = threadIdx.x, lane = tid & 31, per = b.parts * a.num_out, all = a.beams * per;
    const Key *keys = b.keys + (int64_t)group * all;
    Candidate last = {~0ull, ~0ull};
#pragma unroll 1
    for (int place = 0; place < a.num_out; ++place) {
        Candidate best = {0, 0};
#pragma unroll 1
        for (int i = tid; i < all; i += kThreads) {
            const int beam = i / per;
            const Candidate c = candidate(a, sh, beam, i - beam * per, __ldcg(keys + i));
            if (before(last, c) && before(c, best))
                best = c;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const Candidate c = {__shfl_xor_sync(0xffffffffu, best.value, o), __shfl_xor_sync(0xffffffffu, best.tie, o)};
            best = before(c, best) ? c : best;
        }
        __syncthreads();
        if (lane == 0)
            sh.best[tid >> 5] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w)
            best = before(sh.best[w], best) ? sh.best[w] : best;
        if (tid == 0)
            put(a, group, place, best);
        last = best;
    }
}

// A group's outputs from its rows' parts, by the CTA that arrived last.  As in
// a part: a bar that num_out candidates reach, and the few that do are ranked.
// The bar is the num_out-th largest of the first `depth` values of each part,
// four times as many as that in all.
template <bool F32>
__device__ __forceinline__ void join_group(const BeamArgs &b, int group, JoinShared &sh)
{
    const smoe_beam_args &a = b.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, N = a.num_out, P = b.parts;
    const int64_t row0 = (int64_t)group * a.beams;
    const int depth = b.depth, each = P * depth, samples = min(a.beams * each, kSamples);
    if (tid == 0) {
        sh.queued = 0;
        sh.bar = 0;
    }
    if (tid < 4 && samples + tid < kSamples)
        sh.sample[samples + tid] = 0;
    // All that a beam's warp needs is on its way at once, and so are the first
    // candidates of every thread (what belongs to beams that are not live means
    // nothing).
    const int per = P * N, all = a.beams * per;
    const Key *group_keys = b.keys + row0 * per;
    Key first[kFirst];
#pragma unroll
    for (int j = 0; j < kFirst; ++j)
        first[j] = __ldcg(group_keys + min(tid + j * kThreads, all - 1));
    bool again = false;
#pragma unroll 1
    for (int k = warp; k < a.beams; k += kWarps) {
        const float2 *stats = b.stats + (row0 + k) * P;
        const Key *keys = group_keys + k * per;
        const float score = a.scores[row0 + k];
        const int state = state_of(a, row0 + k);
        const int at = min(lane, each - 1);
        const Key sample = __ldcg(keys + at / depth * N + at % depth);
        Key top = 0;
        Two sum = {0.0f, 0.0f};
        float ref = -kMaxRef;
#pragma unroll 1
        for (int p = lane; p < P; p += 32) {
            const Key t = __ldcg(keys + p * N);
            const float2 s = __ldcg(stats + p);
            const float to = fmaxf(ref, s.x);
            sum.hi *= power_of_two(ref - to);
            sum.lo *= power_of_two(ref - to);
            const Two u = two_sum(sum.hi, s.y * power_of_two(s.x - to));
            sum = {u.hi, sum.lo + u.lo};
            ref = to;
            top = t > top ? t : top;
        }
        if (lane == 0) {
            sh.state[k] = state;
            sh.score[k] = 0.25f * score;
        }
        if (state != kLive) {
#pragma unroll 1
            for (int i = lane; i < each && k * each + i < kSamples; i += 32)
                sh.sample[k * each + i] = 0;
            continue;
        }
        const float to = static_cast<float>(__reduce_max_sync(0xffffffffu, static_cast<int>(ref)));
        sum.hi *= power_of_two(ref - to);
        sum.lo *= power_of_two(ref - to);
        for (int o = 16; o > 0; o >>= 1) {
            const Two t = two_sum(sum.hi, __shfl_xor_sync(0xffffffffu, sum.hi, o));
            sum = {t.hi, t.lo + (sum.lo + __shfl_xor_sync(0xffffffffu, sum.lo, o))};
        }
        top = ~least_of(~top);
        // the largest logit's term is at least 2^-1
        const bool wrong = !(sum.hi >= 0.25f && sum.hi <= FLT_MAX) && top != 0;
        const Two log = log_of(settled(sum), to);
        if (lane == 0) {
            sh.base[k] = 0.0f;
            sh.off[k] = {0.25f * log.hi, 0.25f * log.lo};
            sh.again[k] = wrong ? logit_of(top) : NAN;
        }
        again = again || wrong;
        __syncwarp();
        if (!wrong)
#pragma unroll 1
            for (int i = lane; i < each && k * each + i < kSamples; i += 32) {
                const Key t = i < 32 ? sample : __ldcg(keys + i / depth * N + i % depth);
                sh.sample[k * each + i] = t ? static_cast<uint32_t>(value_of(sh, k, t) >> 32) : 0;
            }
    }
    if (__syncthreads_or(again))
#pragma unroll 1
        for (int k = 0; k < a.beams; ++k) {
            const float most = sh.again[k];
            if (sh.state[k] != kLive || isnan(most))
                continue;
            const float s = row_sum<F32>(a, row0 + k, most, sh);
            const Two log = log_of({s, 0.0f}, 0.0f);
            if (tid == 0) {
                sh.base[k] = 0.25f * most;
                sh.off[k] = {0.25f * log.hi, 0.25f * log.lo};
            }
#pragma unroll 1
            for (int i = tid; i < each && k * each + i < kSamples; i += kThreads)
                sh.sample[k * each + i] = 0;
            __syncthreads();
        }
#pragma unroll 1
    for (int i = tid; i < samples; i += kThreads) {
        // (of equal ones the earlier comes first; what is behind the samples is 0)
        const uint32_t v = sh.sample[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < samples; j += 4) {
            const uint4 x = *reinterpret_cast<const uint4 *>(sh.sample + j);
            place += ((x.x > v) | ((x.x == v) & (j < i))) + ((x.y > v) | ((x.y == v) & (j + 1 < i))) +
                     ((x.z > v) | ((x.z == v) & (j + 2 < i))) + ((x.w > v) | ((x.w == v) & (j + 3 < i)));
        }
        if (place == N - 1)
            sh.bar = v;
    }
    __syncthreads();
    const Value bar = static_cast<Value>(sh.bar) << 32;
    const auto offer = [&](int i, Key key) {
        const int beam = i / per;
        const Candidate c = candidate(a, sh, beam, i - beam * per, key);
        if (c.value != 0 && c.value >= bar) {
            const int at = atomicAdd(&sh.queued, 1);
            if (at < kCands)
                sh.queue[at] = c;
        }
    };
#pragma unroll 1
    for (int i = tid; i < all; i += kThreads) {
        offer(i, first[0]);
#pragma unroll
        for (int j = 0; j + 1 < kFirst; ++j)
            first[j] = first[j + 1];
        const int ahead = i + kFirst * kThreads;
        first[kFirst - 1] = ahead < all ? __ldcg(group_keys + ahead) : 0;
    }
    __syncthreads();
    const int n = sh.queued;
    if (n > kCands) {
        select_crowd(b, group, sh);
        return;
    }
#pragma unroll 1
    for (int i = tid; i < n; i += kThreads) {
        const Candidate c = sh.queue[i];
        int place = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j)
            place += before(sh.queue[j], c);
        if (place < N)
            put(a, group, place, c);
    }
    if (tid >= n && tid < N)
        put(a, group, tid, {0, 0});
}

union BeamShared {
    PartShared part;
    JoinShared join;
};

template <bool F32, bool PASSING>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) beam_kernel(const BeamArgs b)
{
    __shared__ BeamShared sh;
    __shared__ bool s_last;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x / b.parts;
    const int part = blockIdx.x % b.parts, group = static_cast<int>(row / b.a.beams);
    scan_part<F32, PASSING>(b, row, part, sh.part);
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
    // parts: up to two CTAs per SM, of a step at least (60 fp32 rows of 100,003: 11.1 us with
    // two and with three, 14.0 with four: each part costs its end again)
    const int64_t wave = dev.sms * 2 < kMaxWave ? dev.sms * 2 : kMaxWave;
    int64_t parts = wave / rows;
    const int least = (steps + kMaxSteps - 1) / kMaxSteps;
    parts = parts < least ? least : parts < steps ? parts : steps;
    const int each = static_cast<int>((steps + parts - 1) / parts);
    b.part_words = each * kStepWords;
    b.parts = (steps + each - 1) / each;
    const int depth = (4 * a.num_out + a.beams * b.parts - 1) / (a.beams * b.parts);
    b.depth = depth < a.num_out ? depth : a.num_out;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    b.arrivals = reinterpret_cast<unsigned *>(ws);
    b.stats = reinterpret_cast<float2 *>(ws + kStatsAt);
    b.keys = reinterpret_cast<Key *>(ws + kStatsAt + rows * b.parts * sizeof(float2));
    const bool passing = rows * a.vocab * (f32 ? 4 : 2) > kPassing;
    auto k = f32 ? (passing ? beam_kernel<true, true> : beam_kernel<true, false>)
                 : (passing ? beam_kernel<false, true> : beam_kernel<false, false>);
    return launch_ahead(k, dim3(static_cast<unsigned>(rows * b.parts)), kThreads, 0, 0, stream, b);
}

}  // namespace smoe
