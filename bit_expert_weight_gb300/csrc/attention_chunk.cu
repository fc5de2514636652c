// attention_chunk.cu -- attention of chunks of new rows over a paged cache on
// the fifth-generation tensor cores (the mathematics: attention.cu).
//
// An item is one tile of 256 packed rows (row m of it: new row (m0 + m) / G,
// head (m0 + m) % G of the kv head), as two halves A and B of 128, over the
// keys that its rows see, loaded 128 keys (a unit) at a time.  Per half and
// 64 keys (a step):
//   S = Q K^T            tcgen05.mma, Q and K in shared memory, S in tensor
//                        memory (128 lanes = rows, 64 columns = keys)
//   P = exp2(S - m)      one thread per row: S from tensor memory to
//                        registers, P as bf16 back over the S columns
//   O += P V             tcgen05.mma, P from tensor memory, V in shared memory
// S has two buffers of 64 columns per half: the next step's S is computed
// while the threads work on this one's exponentials, so that they never wait
// for the tensor cores but at an item's start.  (With one buffer of 128
// columns a unit took 3,550 cycles instead of 2,600: the exponentials and the
// products took turns.)  m is set a factor 2^8 above the row's maximum and
// again once the maximum has passed it: P is at most 1, so that O stays in
// range wherever a plain sum does, and O is hardly ever rescaled; the final
// division by P's sum, kept in fp32, makes the choice of m drop out.  P is rounded to bf16
// (2^-8 of each p), the type that the tensor cores multiply V's bf16 with at
// their full rate; a second half as in attention.cu would double the products
// with V.  The sum is not rounded.
//
// Bounds, per unit of heads of 128: the queue of products.  One of Q and K
// (128 x 64 x 16) reads 4 KB of Q and 2 KB of K, 48 cycles of shared memory at
// 128 bytes a cycle against 32 of tensor cores, and there are 32: 1,536 cycles;
// the 16 with P and V (128 x 128 x 16) take 64 each: 1,024.  Of these 2,560 it
// takes 2,600.  Q in tensor memory would end the first bound, but S and O fill
// it.  Heads of 64 need half as much (1,280), and the softmax warps are the
// bound: two on each scheduler take 1,220 cycles for 64 keys of both (180 of
// waiting, 290 the maximum, 680 the exponentials), with 44 % of the issue slots
// and 36 % of the exponential unit in use: latencies that two warps don't fill.
// Measured: 608 rows on 33,376 keys, 64 query and 4 kv heads of 128: 403 to 419
// us (from GPU to GPU), 1,570 to 1,640 TFLOP/s; the same of 64: 377 us, 875
// TFLOP/s.  Prompts of 9,001 and 2,021 rows (the second on 6,559 keys), heads of
// 128: 1.06 to 1.10 ms, 1,540 to 1,600 TFLOP/s; the rest are items' starts and ends.
//
// Roles of the 16 warps of a CTA, one CTA per SM:
//   warps 0..3  half A, warps 4..7 half B: softmax, rescaling, output
//   warps 8, 9  issue the MMAs of half A and half B: with one warp for both,
//               its waits for one half kept the other's products back
//   warp 10     loads K and V by TMA, page by page, into rings of 3 and 2
//               units, 128-byte swizzle
//   warp 11     walks the line of items and hands them to the other warps
//               through a ring of records in shared memory
//   warps 12..15  load the queries, as soon as the products with the ones
//               before are done
// Work split: as in attention.cu, the items form a line of units, cut into
// equal shares, one per CTA; parts of an item are joined by the last of its
// CTAs to arrive.  Every wait is bounded; one that runs out is recorded as
// SMOE_ERR_TIMEOUT and ends the CTA's work.
#include <cuda.h>
#include <math.h>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace smoe {

namespace {

constexpr int kHalf = 128;              // rows of a half (MMA M)
constexpr int kTileRows2 = 2 * kHalf;   // packed rows of an item
constexpr int kKeys = 128;              // keys of a unit
constexpr int kStep = 64;               // keys of a step (MMA N of Q K^T, K of P V)
constexpr int kKStages = 3, kVStages = 2;  // units of K and of V in shared memory
constexpr int kFree = 4;                   // releases told apart
constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 10, kItemWarp = 11, kQueryWarp = 12;
constexpr int kItemSlots = 4;
constexpr int kThreads = 512;
// An item's own cost, in units (queries, first products, output).  Heads of 64:
// half the queries and output, while a unit takes about as long.  Measured at
// 20 sequences, half chunks, half single rows, and one chunk of 3,000 rows: heads
// of 64 with a cost of 4, 2, 1: 100.6, 95.7, 94.8 us and 45.8, 41.8, 41.5 us (two
// long chunks 824, 800, 807); two prompts of heads of 128 with 4, 3, 2, 1: 1,074,
// 1,078, 1,146, 1,332 us.
__host__ __device__ constexpr int item_units(int D) { return D == 128 ? 4 : 2; }
// Items of up to ten units are not cut: a cut costs about four units' time (a
// part written and read, the join), and a part more one unit to read.
constexpr int kWholeUnits = 10;
constexpr int kMaxCtas = 240;
// The longest run of one item in one CTA, in units: other warps wait for its
// end, and their waits are bounded at 4e9 cycles, 2.9 times as many.
constexpr int kMaxRun = 1 << 19;
// log2 of how far m is set above the maximum, which may grow by as much before
// sums are rescaled.  P is then between 2^-8 and 1 for the largest score, and
// bf16 and fp32 lose nothing by that.  Measured: without it every new maximum
// rescales, 1.74 ms instead of 1.07 for two prompts; 2^20 gains nothing more.
constexpr float kAhead = 8.0f;

__host__ __device__ constexpr int q_half_bytes(int D) { return kHalf * D * 2; }
__host__ __device__ constexpr int stage_bytes(int D) { return kKeys * D * 2; }
__host__ __device__ constexpr int smem_bytes(int D)
{
    return 2 * q_half_bytes(D) + (kKStages + kVStages) * stage_bytes(D) + 1024;  // slack for the alignment
}
// A part: outputs [D][rows], so that a warp's lanes, a row each, write and read
// whole sectors, then the rows' m, then their sums.
__host__ __device__ constexpr int part_floats(int D) { return (D + 2) * kTileRows2; }
static_assert(kPartsAt + (size_t)2 * kMaxCtas * part_floats(128) * 4 <= SMOE_ATTENTION_WORKSPACE_BYTES,
              "workspace");
static_assert((SMOE_MAX_SEQS + 1) * 16 <= (kKStages + kVStages) * stage_bytes(64), "sequence table");
static_assert(kMaxCtas <= kMaxCounters, "counters");

// Tensor memory columns: S (and P over it) and O of each half.
__device__ __forceinline__ constexpr uint32_t col_s(int half) { return half * kKeys; }
template <int D>
__device__ __forceinline__ constexpr uint32_t col_o(int half)
{
    return 2 * kKeys + half * D;
}

// One item, or the part of it in the CTA's share, as the item warp hands it
// on.  rows 0: there are no more.
struct Item {
    int64_t row0;           // the sequence's first row
    int b, h, m0, rows;     // sequence, kv head, first packed row, packed rows
    int i0;                 // key index of the sequence's first new row
    int u0, u1, kbase;      // units; unit u begins at key kbase + 128 u
    int k_lo, k_hi;         // keys seen by any of the rows
    int t_lo, t_hi;         // keys seen by every row
    int c_first, c_last;    // the CTAs that share the item (equal: it is whole)
};

struct Smem {
    uint64_t item_full[kItemSlots];   // item warp
    uint64_t item_empty[kItemSlots];  // all warps but the item warp
    Item item[kItemSlots];
    uint64_t k_first;            // loader: the first unit's K (1 arrival + bytes, as below)
    uint64_t kv_full[kVStages];  // loader: V of a unit and K of the next
    uint64_t v_raw;              // loader, for its own use: a V that it clears in part
    uint64_t unit_done[kFree];   // both MMA warps: the products of a unit
    uint64_t q_full[2];          // 2 query warps; the half's 4 warps: no wait of theirs on s_done is open
    uint64_t q_empty[2];         // 1 MMA commit
    uint64_t s_done[2][2];       // [half][buffer] 1 MMA commit: S, after the P V before it
    uint64_t p_full[2][2];       // [half][buffer] 4 warps
    uint64_t joined;             // 8 warps
    uint64_t drain;              // final commits of both MMA warps
    uint32_t tmem_base;
    uint32_t k_filled, kv_filled, raw_filled;  // phases of k_first, kv_full, v_raw (drain after a failure)
    int fail, last;
    // the work split
    uint32_t scan[kThreads / 32], grains[kThreads / 32];
    int scan_max[kThreads / 32];
    int64_t q, total, before;    // units per CTA, in all, before the CTA's first item's tile
    int64_t border[2];           // the CTA's share
    int unit;                    // an item's length is rounded up to a multiple of this
    int b, t;                    // that tile
    Seq seq, next;               // its sequence, and the one after it
};

// ------------------------------------------------------------ PTX helpers

// Shared-memory matrix descriptor: operand with its M or N dimension
// contiguous (64 elements = 128 bytes, 128-byte swizzle), 8 rows of K per
// 1024-byte atom; the next 64 elements of M or N lie `lead` bytes on.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr, uint32_t lead)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptors of kind::f16, bf16 in, fp32 out, M = 128: Q K^T
// (both K-major, N = keys) and P V (V with N = channels contiguous).
constexpr uint32_t kIdescBase = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kHalf >> 4) << 24);
constexpr uint32_t kIdescQK = kIdescBase | ((uint32_t)(kStep >> 3) << 17);
template <int D>
__device__ __forceinline__ constexpr uint32_t idesc_pv()
{
    return kIdescBase | (1u << 16) | ((uint32_t)(D >> 3) << 17);
}

// The warp's converged threads issue these together and one elected thread
// takes effect: with the operands the same in every lane they stay in uniform
// registers.  (Issued from a branch of one lane, each MMA took 70 to 80 cycles
// to move its descriptors there.)
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

#define SMOE_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                      "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SMOE_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                      "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
#define SMOE_U8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                      "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])

// 32 lanes x 32 consecutive columns of tensor memory into r[0..31].
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : SMOE_R8(r, 0), SMOE_R8(r, 8), SMOE_R8(r, 16), SMOE_R8(r, 24)
                 : "r"(addr));
}
// No use of r[0..31] moves above this point.
__device__ __forceinline__ void pin32(uint32_t *r)
{
    asm volatile("" : SMOE_U8(r, 0), SMOE_U8(r, 8));
    asm volatile("" : SMOE_U8(r, 16), SMOE_U8(r, 24));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::SMOE_W8(r, 0),
                 SMOE_W8(r, 8), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 bytes to global memory, in one piece where they are aligned to that: a
// warp's lanes write rows of their own here, and a store takes a cycle per row.
__device__ __forceinline__ void store32(void *p, const uint32_t *w, bool wide)
{
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), SMOE_W8(w, 0) : "memory");
    else
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            *reinterpret_cast<uint4 *>(static_cast<uint32_t *>(p) + i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// More bytes to come in the barrier's phase.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, unsigned bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}

// Bits lo .. hi - 1 of a word (any lo and hi).
__device__ __forceinline__ uint32_t bits_between(int lo, int hi)
{
    const uint32_t from = lo <= 0 ? ~0u : (lo < 32 ? ~0u << lo : 0u);
    const uint32_t to = hi >= 32 ? ~0u : (hi > 0 ? (1u << hi) - 1u : 0u);
    return from & to;
}

// Bounded wait that records a timeout in the CTA's fail flag.
__device__ __forceinline__ bool wait_for(Smem &sm, uint64_t *bar, unsigned parity, int *status)
{
    if (mbar_try_wait(bar, parity))
        return true;
    if (*reinterpret_cast<volatile int *>(&sm.fail))
        return false;
    if (mbar_wait_bounded(bar, parity))
        return true;
    set_status(status, kStatusTimeout);
    *reinterpret_cast<volatile int *>(&sm.fail) = 1;
    return false;
}

// ------------------------------------------------------------ work split

// A tile of a sequence's packed rows, and a place on the line of units.
struct Tile {
    Seq s, next;        // its sequence, and the one after it (loaded early)
    int b, t, h;
    int m0, rows;       // first packed row, packed rows (256 at most; 0: no tile)
    int units;
    int own;            // its own cost, in units
    int64_t at;         // its first unit on the line
    int k_lo, k_hi;     // keys seen by any of its rows; unit 0 begins at kbase
    int t_lo, t_hi;     // keys seen by every row
    int kbase;
};

// The keys of tile t of a sequence.
struct TileKeys {
    int rows, units, k_lo, k_hi, t_lo, t_hi;
};
__device__ __forceinline__ TileKeys keys_of(int window, int G, int seq_rows, int len, int t)
{
    const int m0 = t * kTileRows2, left = seq_rows * G - m0;
    TileKeys k;
    k.rows = left < kTileRows2 ? (left > 0 ? left : 0) : kTileRows2;
    k.k_lo = k.k_hi = k.t_lo = k.t_hi = 0;
    if (k.rows > 0) {
        const int i0 = len - seq_rows;  // key index of the first row
        seen_from(window, i0 + m0 / G, k.k_lo, k.t_hi);
        seen_from(window, i0 + (m0 + k.rows - 1) / G, k.t_lo, k.k_hi);
    }
    const int n = (k.k_hi - k.k_lo / kKeys * kKeys + kKeys - 1) / kKeys;
    // rows that see nothing still take a unit: they get their zeros
    k.units = k.rows == 0 ? 0 : (n > 1 ? n : 1);
    return k;
}

__device__ __forceinline__ void tile_keys(const smoe_attention_args &a, int G, Tile &c)
{
    const TileKeys k = keys_of(a.window, G, c.s.rows, c.s.len, c.t);
    c.own = item_units(a.cache.head_dim);
    c.m0 = c.t * kTileRows2;
    c.rows = k.rows;
    c.units = k.units;
    c.k_lo = k.k_lo;
    c.k_hi = k.k_hi;
    c.t_lo = k.t_lo;
    c.t_hi = k.t_hi;
    c.kbase = k.k_lo / kKeys * kKeys;
}

// An item's length on the line.
__device__ __forceinline__ int item_length(const Tile &c, int unit)
{
    return (c.units + c.own + unit - 1) / unit * unit;
}

// To the next item; past the last one it has no rows.
__device__ __forceinline__ void tile_next(const smoe_attention_args &a, int G, int unit, Tile &c, int *status)
{
    c.at += item_length(c, unit);
    if (++c.h < a.cache.num_kv_heads)
        return;
    c.h = 0;
    ++c.t;
    tile_keys(a, G, c);
    while (c.rows == 0 && c.b < a.batch.num_seqs) {
        ++c.b;
        c.s = c.next;
        c.next = seq_or_none(a, c.b + 1, status);
        c.t = 0;
        tile_keys(a, G, c);
    }
}

// Units [u0, u1) of the item that lie in the share [w0, w1).
__device__ __forceinline__ void units_in(const Tile &c, int64_t w0, int64_t w1, int &u0, int &u1)
{
    const int64_t k = c.at + c.own;
    u0 = w0 > k ? static_cast<int>(w0 - k) : 0;
    u1 = w1 - k < c.units ? static_cast<int>(w1 - k) : c.units;
}

__device__ __forceinline__ int tiles_of(const Seq &s, int G) { return (s.rows * G + kTileRows2 - 1) / kTileRows2; }

// Sums over the CTA's threads: before the thread's own, and of all; and the
// maximum of all.
struct Scan {
    uint32_t before, total;
    int most;
    bool over;  // the sum may not be below 2^32, and the two above have wrapped
};
// The line of one kv head must stay below 2^32 units.  That is seen from the
// threads' own sums in grains of 2^16, rounded up, which 32 bits hold whatever
// the batch: a thread has 2^14 tiles of 2^24 units at most.
constexpr int kGrainShift = 16;
constexpr uint32_t kMaxGrains = 1u << (32 - kGrainShift);
__device__ __forceinline__ Scan scan_all(Smem &sm, uint64_t own, int mx)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t v = static_cast<uint32_t>(own);
    const uint32_t grains = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(own >> kGrainShift) + 1u);
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? x : 0;
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    __syncthreads();
    if (lane == 31) {
        sm.scan[warp] = incl;
        sm.grains[warp] = grains;
        sm.scan_max[warp] = mx;
    }
    __syncthreads();
    // the warps' sums, a lane per warp
    const uint32_t w = lane < kThreads / 32 ? sm.scan[lane] : 0;
    Scan s;
    s.before = incl - v + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    s.total = __reduce_add_sync(0xffffffffu, w);
    s.most = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? sm.scan_max[lane] : 0);
    s.over = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? sm.grains[lane] : 0) > kMaxGrains;
    return s;
}

// A sequence of the batch in shared memory, with the tiles before it.
struct ChunkSeq {
    int row0, rows, len, tiles;
};

__device__ __forceinline__ Seq seq_of(const ChunkSeq &c)
{
    Seq s;
    s.row0 = c.row0;
    s.rows = c.rows;
    s.len = c.len;
    return s;
}

// The CTA's share, into shared memory: q, total, and the tile at its start.
// `seqs`: room for the batch and one more, in memory that is not in use yet.
__device__ __forceinline__ void find_share(const smoe_attention_args &a, int G, Smem &sm, ChunkSeq *seqs,
                                           int *status)
{
    const int tid = threadIdx.x, n = a.batch.num_seqs, Hkv = a.cache.num_kv_heads;
    // tiles before each sequence
    const int per = (n + kThreads - 1) / kThreads;
    uint32_t sum = 0;
#pragma unroll 1
    for (int b = tid * per; b < n && b < (tid + 1) * per; ++b) {
        const Seq s = seq_at(a, b, status);
        seqs[b].row0 = static_cast<int>(s.row0);
        seqs[b].rows = s.rows;
        seqs[b].len = s.len;
        seqs[b].tiles = tiles_of(s, G);
        sum += seqs[b].tiles;
    }
    Scan sc = scan_all(sm, sum, 0);
#pragma unroll 1
    for (int b = tid * per; b < n && b < (tid + 1) * per; ++b) {
        const int k = seqs[b].tiles;
        seqs[b].tiles = static_cast<int>(sc.before);
        sc.before += k;
    }
    const int all = static_cast<int>(sc.total);
    if (tid == 0) {
        seqs[n].row0 = seqs[n].rows = seqs[n].len = 0;
        seqs[n].tiles = all;
    }
    __syncthreads();
    // units of the tiles [i0, i1) of this thread
    const int pt = (all + kThreads - 1) / kThreads;
    const int i0 = tid * pt < all ? tid * pt : all, i1 = i0 + pt < all ? i0 + pt : all;
    Tile c;
    int b0 = 0, hi = n - 1;
    while (b0 < hi) {  // last sequence with as many tiles before it
        const int mid = (b0 + hi + 1) >> 1;
        if (seqs[mid].tiles <= i0)
            b0 = mid;
        else
            hi = mid - 1;
    }
    auto tile_at = [&](int i, int &b) {
        while (i >= seqs[b + 1].tiles)
            ++b;
        c.s = seq_of(seqs[b]);
        c.t = i - seqs[b].tiles;
        tile_keys(a, G, c);
    };
    // the length of this thread's tiles on the line of one kv head
    int mx = 0;
    auto length = [&](int unit) {
        uint64_t l = 0;
#pragma unroll 1
        for (int i = i0, b = b0; i < i1; ++i) {
            tile_at(i, b);
            l += item_length(c, unit);
            mx = c.units > mx ? c.units : mx;
        }
        return l;
    };
    int unit = 1;
    int64_t q;
    for (int pass = 0;; ++pass) {
        const uint64_t l = length(unit);
        const Scan s = scan_all(sm, l, mx);
        if (pass == 0) {
            // Equal shares, but no item in so many parts that the joining costs
            // more than the sharing saves.
            q = ceil_div((int64_t)s.total * Hkv, gridDim.x);
            const int64_t least = s.most <= kWholeUnits ? s.most + item_units(a.cache.head_dim)
                                               : static_cast<int64_t>(sqrtf(static_cast<float>(s.most)));
            q = q > least ? q : least;
            sum = static_cast<uint32_t>(l);
            sc = s;
            const int share = static_cast<int>(min(q, (int64_t)0x7fffffff));
            if (s.over || min(s.most, share) > kMaxRun) {  // recorded, and not worked on
                if (tid == 0)
                    set_status(status, kStatusBadArg);
                sum = sc.before = sc.total = 0;
                break;
            }
            // Where the grid has room for it, every item begins a CTA's share,
            // so that none is cut for the sake of its neighbours.
            if (all * Hkv > static_cast<int>(gridDim.x))
                break;
            unit = static_cast<int>(q);
        } else {
            if (!s.over && (int64_t)s.total * Hkv <= q * gridDim.x) {
                sum = static_cast<uint32_t>(l);
                sc = s;
            } else {
                unit = 1;
            }
            break;
        }
    }
    const int64_t before = (int64_t)sc.before * Hkv, all_units = (int64_t)sc.total * Hkv;
    if (tid == 0) {
        sm.q = q;
        sm.total = all_units;
        sm.unit = unit;
    }
    // The borders of the share: drawn at the nearer end of an item that is not
    // worth being cut.
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int64_t x = q * (blockIdx.x + side);
        if (x >= all_units && tid == 0)
            sm.border[side] = all_units;
        if (x < before || x >= before + (int64_t)sum * Hkv)
            continue;
        int64_t at = before;
#pragma unroll 1
        for (int i = i0, b = b0; i < i1; ++i) {
            tile_at(i, b);
            const int len = item_length(c, unit);
            const int64_t next = at + (int64_t)len * Hkv;
            if (x < next) {
                const int64_t item = at + (x - at) / len * len;
                sm.border[side] = x == item || c.units > kWholeUnits ? x
                                  : 2 * (x - item) < len             ? item
                                                                     : item + len;
                if (side == 0) {
                    sm.b = b;
                    sm.t = c.t;
                    sm.before = at;
                    sm.seq = c.s;
                    sm.next = seq_of(seqs[b + 1]);
                }
                break;
            }
            at = next;
        }
    }
    fence_async_smem();  // tensor copies will write where the batch lay
    __syncthreads();
}

__device__ __forceinline__ Tile first_tile(const smoe_attention_args &a, int G, const Smem &sm)
{
    Tile c;
    c.b = sm.b;
    c.t = sm.t;
    c.s = sm.seq;
    c.next = sm.next;
    tile_keys(a, G, c);
    const int len = item_length(c, sm.unit);
    // (a border drawn at an item's start lies in the item before it, or here)
    const int64_t x = sm.q * blockIdx.x;
    c.h = static_cast<int>((x - sm.before) / len);
    c.at = sm.before + (int64_t)c.h * len;
    return c;
}

// ------------------------------------------------------------ roles

// The items of the CTA's share, in order (warp 11).
__device__ void item_walker(const smoe_attention_args &a, int G, Smem &sm, int64_t w0, int64_t w1, int *status)
{
    const int lane = threadIdx.x & 31;
    uint32_t n = 0;
    for (Tile c = first_tile(a, G, sm);; tile_next(a, G, sm.unit, c, status)) {
        const bool end = c.rows == 0 || c.at >= w1;
        int u0 = 0, u1 = 0;
        if (!end) {
            units_in(c, w0, w1, u0, u1);
            if (u0 >= u1)
                continue;
        }
        const int slot = n % kItemSlots;
        if (!__all_sync(0xffffffffu, wait_for(sm, &sm.item_empty[slot], ((n / kItemSlots) & 1u) ^ 1u, status)))
            return;
        if (lane == 0) {
            Item &t = sm.item[slot];
            const int64_t k = c.at + c.own;
            t.row0 = c.s.row0;
            t.b = c.b;
            t.h = c.h;
            t.m0 = c.m0;
            t.rows = end ? 0 : c.rows;
            t.i0 = c.s.len - c.s.rows;
            t.u0 = u0;
            t.u1 = u1;
            t.kbase = c.kbase;
            t.k_lo = c.k_lo;
            t.k_hi = c.k_hi;
            t.t_lo = c.t_lo;
            t.t_hi = c.t_hi;
            const bool whole = u1 - u0 == c.units;
            t.c_first = whole ? 0 : static_cast<int>(k / sm.q);
            t.c_last = whole ? 0 : static_cast<int>((k + c.units - 1) / sm.q);
            mbar_arrive(&sm.item_full[slot]);
        }
        __syncwarp();
        ++n;
        if (end)
            return;
    }
}

// The next item of a role (n counts them).  False: there are no more, or a
// wait ran out.
__device__ __forceinline__ bool next_item(Smem &sm, uint32_t &n, Item &t, int *status)
{
    const int slot = n % kItemSlots;
    if (!__all_sync(0xffffffffu, wait_for(sm, &sm.item_full[slot], (n / kItemSlots) & 1u, status)))
        return false;
    t = sm.item[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(&sm.item_empty[slot]);
    ++n;
    return t.rows > 0;
}

// The queries of half of every item's half `half` (warps 12..15): row r as it
// is packed, into the swizzled layout that the MMA reads; rows past the
// item's are zeros.
template <int D>
__device__ void query_loader(const smoe_attention_args &a, int G, Smem &sm, uint8_t *sq, int half, int part,
                             int *status)
{
    const int lane = threadIdx.x & 31;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes per row, rows per round
    const uint32_t dst = smem_u32(sq + half * q_half_bytes(D));
    uint32_t n = 0, qn = 0;
    Item c;
    while (next_item(sm, n, c, status)) {
        if (c.rows <= kHalf * half)
            continue;
        int64_t at[kHalf / 2 / 32];  // of the rows 32 i + lane of this part
#pragma unroll
        for (int i = 0; i < kHalf / 2 / 32; ++i) {
            const int m = kHalf * half + kHalf / 2 * part + 32 * i + lane;
            const int pm = c.m0 + m;
            at[i] = m < c.rows ? (c.row0 + pm / G) * a.q_row_stride + (int64_t)(c.h * G + pm % G) * a.q_head_stride
                               : -1;
        }
        if (!__all_sync(0xffffffffu, wait_for(sm, &sm.q_empty[half], (qn++ & 1u) ^ 1u, status)))
            return;
#pragma unroll
        for (int i = 0; i < kHalf / 2 / 32; ++i) {
#pragma unroll 4
            for (int k = 0; k < 32 / kRows; ++k) {
                const int row = k * kRows + lane / kLanes, ch = lane % kLanes, r = kHalf / 2 * part + 32 * i + row;
                const int64_t from = __shfl_sync(0xffffffffu, at[i], row);
                const uint16_t *src = static_cast<const uint16_t *>(a.q) + (from >= 0 ? from + 8 * ch : 0);
                const int bytes = from >= 0 ? 16 : 0;  // the rest is filled with zeros
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 dst + (ch / 8) * (kHalf * 128) + r * 128 + (((ch % 8) ^ (r & 7)) << 4)),
                             "l"(src), "r"(bytes)
                             : "memory");
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.q_full[half]);
    }
}

struct Maps {
    CUtensorMap k, v;  // (channels, slots, kv heads, pages), boxes of 64 x box_rows x 1 x 1
};

// Zero the rows of a V stage whose keys the item does not see: their slots
// may hold anything, and 0 x NaN is NaN.
template <int D>
__device__ __forceinline__ void clear_unseen(uint8_t *stage, int key0, int lo, int hi)
{
    const int lane = threadIdx.x & 31;
    const int below = lo > key0 ? lo - key0 : 0, left = hi - key0 > 0 ? hi - key0 : 0;  // rows [below, left) stay
    constexpr int kLanes = D / 8;
    for (int i = lane / kLanes; i < kKeys; i += 32 / kLanes) {
        if (i >= below && i < left)
            continue;
        *reinterpret_cast<uint4 *>(stage + (lane % kLanes / 8) * (kKeys * 128) + i * 128 + (lane % 8) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
    __syncwarp();
}

// Keys and values (warp 10): V of each unit together with K of the next one,
// which take the places that one unit's products free.  A lane copies one
// 64-channel half of one page's share of the unit.  Pages without a key that
// the item sees are not read; the rest of V's first and last page is cleared
// before the MMA warps get it.
template <int D>
__device__ void loader(const smoe_attention_args &a, const Maps *maps, Smem &sm, uint8_t *ring, int *status)
{
    const int lane = threadIdx.x & 31, page = a.cache.page_size;
    const int box = page < kKeys ? page : kKeys, boxes = kKeys / box;
    const int i = lane / (D / 64), half = lane % (D / 64);
    const int at = half * (kKeys * 128) + i * box * 128;  // of the lane's box in a stage
    uint32_t n = 0, raw = 0;                              // items, cleared V
    auto ok = [&](uint64_t *bar, unsigned parity) {
        return __all_sync(0xffffffffu, wait_for(sm, bar, parity, status));
    };
    Item c = {};
    // a unit's keys, and the lane's page of them (-1: none)
    struct Unit {
        int key0, lo, hi, head, page;
        bool there;
    };
    auto unit_at = [&](int u) {
        Unit x;
        x.key0 = c.kbase + u * kKeys;
        x.lo = c.k_lo;
        x.hi = c.k_hi;
        x.head = c.h;
        x.there = true;
        x.page = -1;
        const int k0 = x.key0 + i * box;
        if (i < boxes && k0 < c.k_hi && k0 + box > c.k_lo) {
            x.page = a.batch.page_table[(int64_t)c.b * a.batch.table_stride + k0 / page];
            if (x.page < 0 || x.page >= a.cache.num_pages) {
                set_status(status, kStatusBadArg);
                x.page = -1;
            }
        }
        return x;
    };
    auto bytes_of = [&](const Unit &x) { return __popc(__ballot_sync(0xffffffffu, x.page >= 0)) * box * 128u; };
    auto copy = [&](uint8_t *stage, const CUtensorMap *map, const Unit &x, uint64_t *full) {
        if (x.page >= 0)
            tma_load_4d(stage + at, map, 64 * half, (x.key0 + i * box) % page, x.head, x.page, full);
    };
    if (!next_item(sm, n, c, status))
        return;
    int u = c.u0;
    Unit cur = unit_at(u);
    const uint32_t first = bytes_of(cur);
    if (lane == 0) {
        sm.k_filled = 1;
        mbar_arrive_expect_tx(&sm.k_first, first);
    }
    __syncwarp();
    copy(ring, &maps->k, cur, &sm.k_first);
    for (uint32_t g = 0;; ++g) {
        Unit next = cur;
        next.there = ++u < c.u1;
        if (!next.there && next_item(sm, n, c, status)) {
            u = c.u0;
            next.there = true;
        }
        next.page = -1;
        if (next.there)
            next = unit_at(u);
        if (g >= kVStages && !ok(&sm.unit_done[(g - kVStages) % kFree], ((g - kVStages) / kFree) & 1u))
            return;
        uint8_t *vs = ring + (kKStages + g % kVStages) * stage_bytes(D);
        uint64_t *full = &sm.kv_full[g % kVStages];
        const bool edge = cur.key0 < cur.lo || cur.key0 + kKeys > cur.hi;
        const uint32_t vbytes = bytes_of(cur), kbytes = bytes_of(next);
        if (lane == 0) {
            sm.kv_filled = g + 1;
            if (edge) {
                sm.raw_filled = raw + 1;
                mbar_arrive_expect_tx(&sm.v_raw, vbytes);
                mbar_expect_tx(full, kbytes);
            } else {
                mbar_arrive_expect_tx(full, vbytes + kbytes);
            }
        }
        __syncwarp();
        copy(vs, &maps->v, cur, edge ? &sm.v_raw : full);
        copy(ring + ((g + 1) % kKStages) * stage_bytes(D), &maps->k, next, full);
        if (edge) {
            const bool came = ok(&sm.v_raw, raw++ & 1u);
            if (came)
                clear_unseen<D>(vs, cur.key0, cur.lo, cur.hi);
            if (lane == 0)
                mbar_arrive(full);
            __syncwarp();
            if (!came)
                return;
        }
        if (!next.there)
            return;
        cur = next;
    }
}

// The MMAs of one half (warps 8 and 9).
template <int D>
__device__ void mma_issuer(Smem &sm, uint8_t *sq, uint8_t *ring, int half, int *status)
{
    const uint32_t base = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
    const uint32_t ts = base + col_s(half), to = base + col_o<D>(half);
    const uint64_t qd = sw128_desc(smem_u32(sq) + half * q_half_bytes(D)), kd = sw128_desc(smem_u32(ring));
    const uint64_t vd = sw128_desc_mn(smem_u32(ring) + kKStages * stage_bytes(D), kKeys * 128);
    constexpr uint64_t kStage = stage_bytes(D) >> 4;
    uint32_t g = 0, n = 0;    // units, items
    uint32_t qn = 0, pn = 0;  // items and units of this half
    const int lane = threadIdx.x & 31;
    auto ok = [&](uint64_t *bar, unsigned parity) {
        return __all_sync(0xffffffffu, wait_for(sm, bar, parity, status));
    };
    // S of step x of the CTA, into its buffer
    auto qk = [&](uint32_t x) {
        const uint64_t bd = kd + (x / 2 % kKStages) * kStage + (x & 1) * (kStep * 128 >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            // 16 channels: 32 bytes inside a 64-channel half, which is 16 KB
            const uint64_t off = (uint64_t)((k / 4) * (kHalf * 128 >> 4) + (k % 4) * 2);
            mma_ss(ts + (x & 1) * kStep, qd + off, bd + off, kIdescQK, k > 0);
        }
    };
    for (;; ++n) {
        const int slot = n % kItemSlots;
        if (!ok(&sm.item_full[slot], (n / kItemSlots) & 1u))
            return;
        // the same in every lane, and known to be
        const int rows = __shfl_sync(0xffffffffu, sm.item[slot].rows, 0);
        const int units = __shfl_sync(0xffffffffu, sm.item[slot].u1 - sm.item[slot].u0, 0);
        if (lane == 0)
            mbar_arrive(&sm.item_empty[slot]);
        if (rows == 0)
            return;
        if (rows <= kHalf * half) {
            // no rows in this half: nothing to wait for but the unit itself
            for (int i = 0; i < units; ++i, ++g) {
                if (!ok(&sm.kv_full[g % kVStages], (g / kVStages) & 1u))
                    return;
                if (lane == 0)
                    mbar_arrive(&sm.unit_done[g % kFree]);
            }
            continue;
        }
        // (K of a later item's first unit came with V of the unit before it)
        if (!ok(&sm.q_full[half], qn++ & 1u) || (g == 0 && !ok(&sm.k_first, 0)))
            return;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            qk(2 * g + b);
            commit_elected(&sm.s_done[half][b]);
        }
        for (int u = 0; u < units; ++u, ++g, ++pn) {
            const bool last = u + 1 == units;
            if (last)  // the item's last S are on their way: its queries are free after them
                commit_elected(&sm.q_empty[half]);
            if (!ok(&sm.kv_full[g % kVStages], (g / kVStages) & 1u))
                return;
            const uint64_t bd = vd + (g % kVStages) * kStage;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                if (!ok(&sm.p_full[half][b], pn & 1u))
                    return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k)  // 16 keys each
                    mma_ts(to, ts + b * kStep + 8 * k, bd + (uint64_t)((b * kStep + 16 * k) * 128 >> 4),
                           idesc_pv<D>(), u > 0 || b > 0 || k > 0);
                // the S after next over P, which the products above read first:
                // MMAs of one thread run in order
                if (!last)
                    qk(2 * (g + 1) + b);
                commit_elected(&sm.s_done[half][b]);
            }
            commit_elected(&sm.unit_done[g % kFree]);
        }
    }
}

// Softmax and output of half `half` (warps 4 half .. 4 half + 3).
template <int D>
__device__ void softmax(const smoe_attention_args &a, int G, Smem &sm, float *parts, unsigned *arrived,
                        int half, int *status)
{
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const int r = 32 * quarter + lane;  // row of the half, lane of tensor memory
    const uint32_t tl = sm.tmem_base + (static_cast<uint32_t>(32 * quarter) << 16);
    const float sc = a.scale * 1.44269504088896341f;
    const int64_t esize = a.out_dtype == SMOE_F32 ? 4 : 2;
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | a.out_row_stride * esize | a.out_head_stride * esize) & 31) == 0;
    uint32_t sn = 0, jn = 0;  // commits of each s_done of this half, joins
    auto ok = [&](uint64_t *bar, unsigned parity) {
        return __all_sync(0xffffffffu, wait_for(sm, bar, parity, status));
    };
    uint32_t n = 0;  // items
    if (lane == 0)
        mbar_arrive(&sm.q_full[half]);
    Item c;
    while (next_item(sm, n, c, status)) {
        const int u0 = c.u0, u1 = c.u1;
        const int m = kHalf * half + r;         // row of the item
        const bool on = m < c.rows;
        const bool active = c.rows > kHalf * half;  // the half has rows
        const int64_t token = c.row0 + (c.m0 + m) / G;
        const int head = c.h * G + (c.m0 + m) % G;
        int lo = 0, hi = 0;
        if (on)
            seen_from(a, c.i0 + (c.m0 + m) / G, lo, hi);
        float mr = -INFINITY, sum = 0.f;
        if (active) {
            const int steps = 2 * (u1 - u0);
#pragma unroll 1
            for (int v = 0; v < steps; ++v) {
                if (!ok(&sm.s_done[half][v & 1], (sn + v / 2) & 1u))
                    return;
                tc_fence_after();
                const uint32_t ts = tl + col_s(half) + (v & 1) * kStep;
                const int key0 = c.kbase + u0 * kKeys + v * kStep;
                uint32_t s[kStep];
                tmem_ld32(ts, s);
                tmem_ld32(ts + 32, s + 32);
                tmem_wait_ld();
                pin32(s);
                pin32(s + 32);
                if (key0 < c.t_lo || key0 + kStep > c.t_hi) {
                    // a bit per key: tested in place, it takes half the
                    // instructions of two comparisons
#pragma unroll
                    for (int h = 0; h < kStep; h += 32) {
                        const uint32_t unseen = ~bits_between(lo - key0 - h, hi - key0 - h);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (unseen & (1u << e))
                                s[h + e] = 0xff800000u;  // -infinity
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < kStep; e += 2)
                    mx[e / 2 & 3] = max3(mx[e / 2 & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                const bool raise = top > mr;
                if (__any_sync(0xffffffffu, raise)) {
                    // above the maximum; other rows of the warp keep theirs, so
                    // that a row's result does not depend on its neighbours
                    const float mn = raise ? top + kAhead : mr;
                    const float f = raise ? ex2(mr - mn) : 1.f;
                    mr = mn;
                    sum *= f;
                    if (v > 0) {
                        // O is at rest once the step before has been added
                        if (!ok(&sm.s_done[half][(v - 1) & 1], (sn + (v - 1) / 2 + 1) & 1u))
                            return;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < D; k += 16) {
                            uint32_t o[16];
                            tmem_ld16(tl + col_o<D>(half) + k, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                asm volatile("" : "+r"(o[e]));
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            }
                            tmem_st16(tl + col_o<D>(half) + k, o);
                        }
                    }
                }
                const float mu = mr == -INFINITY ? 0.f : mr;  // a row that has seen nothing yet
                const uint64_t sc2 = pair(sc, sc), mu2 = pair(-mu, -mu);
                uint64_t acc[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
                uint32_t p[kStep / 2];
#pragma unroll
                for (int e = 0; e < kStep / 2; ++e) {
                    float x, y;
                    unpair(fma2(pair(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, mu2), x, y);
                    x = ex2(x);
                    y = ex2(y);
                    acc[e & 1] = add2(acc[e & 1], pair(x, y));
                    p[e] = pack_bf16x2(x, y);
                    if ((e & 15) == 15)
                        tmem_st16(ts + (e & 16), p + (e & 16));
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sm.p_full[half][v & 1]);
                float x, y;
                unpair(add2(acc[0], acc[1]), x, y);
                sum += x + y;
            }
            // every step is in O
            sn += u1 - u0;
            if (!ok(&sm.s_done[half][0], sn & 1u) || !ok(&sm.s_done[half][1], sn & 1u))
                return;
            ++sn;
            tc_fence_after();
            // only now may the next item's S complete another phase of s_done
            if (lane == 0)
                mbar_arrive(&sm.q_full[half]);
        }
        const int c_first = c.c_first, c_last = c.c_last;
        const bool whole = c_first == c_last;
        auto write_out = [&](int col, const float *v, float inv) {  // 16 columns
            const int64_t at = token * a.out_row_stride + (int64_t)head * a.out_head_stride + col;
            uint32_t w[16];
            if (a.out_dtype == SMOE_F32) {
                float *dst = static_cast<float *>(a.out) + at;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    w[i] = __float_as_uint(v[i] * inv);
                store32(dst, w, wide);
                store32(dst + 8, w + 8, wide);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = pack_bf16x2(v[2 * i] * inv, v[2 * i + 1] * inv);
                store32(static_cast<uint16_t *>(a.out) + at, w, wide);
            }
        };
        float *part = parts + (2 * (int64_t)blockIdx.x + (static_cast<int>(blockIdx.x) == c_first ? 1 : 0)) *
                                  part_floats(D);
        if (active) {
            const float inv = sum > 0.f ? 1.0f / sum : 0.f;  // a row that sees no key: zeros
#pragma unroll 1
            for (int i = 0; i < D; i += 32) {
                uint32_t o[32];
                tmem_ld32(tl + col_o<D>(half) + i, o);
                tmem_wait_ld();
                pin32(o);
                if (whole) {
                    if (on) {
                        write_out(i, reinterpret_cast<const float *>(o), inv);
                        write_out(i + 16, reinterpret_cast<const float *>(o + 16), inv);
                    }
                } else if (on) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        __stcg(part + (i + j) * kTileRows2 + m, __uint_as_float(o[j]));
                }
            }
            if (!whole && on) {
                __stcg(part + D * kTileRows2 + m, mr);
                __stcg(part + (D + 1) * kTileRows2 + m, sum);
            }
            // the output is read before the next item's P lets P V overwrite it
            tc_fence_before();
        }
        if (whole)
            continue;
        // ---- the last of the item's CTAs to arrive joins its parts
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.joined);
        if (!ok(&sm.joined, jn & 1u))
            return;
        ++jn;
        if (threadIdx.x == 0)
            sm.last = count_arrival(arrived + c_first) == static_cast<unsigned>(c_last - c_first);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sm.joined);
        if (!ok(&sm.joined, jn & 1u))
            return;
        ++jn;
        if (*reinterpret_cast<volatile int *>(&sm.last)) {
            // part j of the item
            auto part_of = [&](int j) {
                return parts + (2 * (int64_t)j + (j == c_first ? 1 : 0)) * part_floats(D);
            };
            // a lane per row: the row's maximum and sum over the parts, then its
            // outputs, 32 of a part on their way together
            if (on) {
                float mj = -INFINITY, lj = 0.f;
#pragma unroll 4
                for (int j = c_first; j <= c_last; ++j)
                    mj = fmaxf(mj, __ldcg(part_of(j) + D * kTileRows2 + m));
                if (mj != -INFINITY)
#pragma unroll 4
                    for (int j = c_first; j <= c_last; ++j)
                        lj += __ldcg(part_of(j) + (D + 1) * kTileRows2 + m) *
                              ex2(__ldcg(part_of(j) + D * kTileRows2 + m) - mj);
                const float inv = lj > 0.f ? 1.0f / lj : 0.f;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    float v[32] = {};
#pragma unroll 1
                    for (int j = c_first; j <= c_last; ++j) {
                        const float *p = part_of(j) + i * kTileRows2 + m;
                        float y[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            y[e] = __ldcg(p + e * kTileRows2);
                        const float w = mj == -INFINITY ? 0.f : ex2(__ldcg(part_of(j) + D * kTileRows2 + m) - mj);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = fmaf(y[e], w, v[e]);
                    }
                    write_out(i, v, inv);
                    write_out(i + 16, v + 16, inv);
                }
            }
            if (threadIdx.x == 0)
                arrived[c_first] = 0;  // for the next launch
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const smoe_attention_args a, const __grid_constant__ Maps maps, uint8_t *workspace,
                        int *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ Smem sm;
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sq = base, *ring = base + 2 * q_half_bytes(D);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_heads / a.cache.num_kv_heads;
    if (tid == 0) {
        sm.fail = 0;
        sm.b = a.batch.num_seqs;
        sm.t = 0;
        sm.before = 0;
        sm.k_filled = sm.kv_filled = sm.raw_filled = 0;
        mbar_init(&sm.k_first, 1);
        for (int i = 0; i < kVStages; ++i)
            mbar_init(&sm.kv_full[i], 1);
        mbar_init(&sm.v_raw, 1);
        for (int i = 0; i < kFree; ++i)
            mbar_init(&sm.unit_done[i], 2);
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], kThreads / 32 - 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 2 + kSoftWarps / 2);
            mbar_init(&sm.q_empty[i], 1);
            for (int j = 0; j < 2; ++j) {
                mbar_init(&sm.s_done[i][j], 1);
                mbar_init(&sm.p_full[i][j], 4);
            }
        }
        mbar_init(&sm.joined, kSoftWarps);
        mbar_init(&sm.drain, 2);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm.tmem_base)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (the ring is not in use yet)
    find_share(a, G, sm, reinterpret_cast<ChunkSeq *>(ring), status);
    const int64_t w0 = sm.border[0], w1 = sm.border[1];
    if (w0 >= w1) {
        // nothing for this CTA
    } else if (warp < kSoftWarps) {
        softmax<D>(a, G, sm, reinterpret_cast<float *>(workspace + kPartsAt),
                   reinterpret_cast<unsigned *>(workspace), warp >> 2, status);
    } else if (warp == kLoadWarp) {
        loader<D>(a, &maps, sm, ring, status);
    } else if (warp == kItemWarp) {
        item_walker(a, G, sm, w0, w1, status);
    } else if (warp >= kQueryWarp) {
        query_loader<D>(a, G, sm, sq, (warp - kQueryWarp) / 2, (warp - kQueryWarp) % 2, status);
    } else {
        mma_issuer<D>(sm, sq, ring, __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp, status);
        __syncwarp();
        // every MMA issued so far has completed once this commit lands
        commit_elected(&sm.drain);
        if (!mbar_wait_bounded(&sm.drain, 0)) {
            set_status(status, kStatusTimeout);
            *reinterpret_cast<volatile int *>(&sm.fail) = 1;
        }
    }
    __syncwarp();
    // After a failure copies may be left unwaited: the loader waits (bounded)
    // for the last fill of every stage, so that none is in flight at the end.
    if (*reinterpret_cast<volatile int *>(&sm.fail) && warp == kLoadWarp && lane == 0) {
        bool done = true;
        if (sm.k_filled)
            done = mbar_wait_bounded(&sm.k_first, 0);
        for (uint32_t i = 0; i < kVStages && i < sm.kv_filled; ++i) {
            const uint32_t g = sm.kv_filled - 1 - i;
            done = mbar_wait_bounded(&sm.kv_full[g % kVStages], (g / kVStages) & 1u) && done;
        }
        if (sm.raw_filled)
            done = mbar_wait_bounded(&sm.v_raw, (sm.raw_filled - 1) & 1u) && done;
        if (!done)
            set_status(status, kStatusTimeout);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sm.tmem_base), "r"(512)
                     : "memory");
    }
}

// ------------------------------------------------------------ host side

// Tensor map of one of the cache's halves: (channels, slots, kv heads, pages),
// read in boxes of 64 channels x box_rows slots.
bool page_map(CUtensorMap *m, const void *pages, const smoe_kv_cache &c, int64_t page_stride, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn)
        return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                                static_cast<cuuint64_t>(c.num_kv_heads), static_cast<cuuint64_t>(c.num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.head_dim) * 2,
                                   static_cast<cuuint64_t>(c.page_size) * c.head_dim * 2,
                                   static_cast<cuuint64_t>(page_stride) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(box_rows), 1, 1};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pages), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const smoe_attention_args &a, uint8_t *workspace, const DeviceFacts &dev, cudaStream_t stream)
{
    static std::atomic<bool> allowed[kMaxDeviceIndex];
    Maps maps;
    const int box = a.cache.page_size < kKeys ? a.cache.page_size : kKeys;
    if (!page_map(&maps.k, a.cache.k_pages, a.cache, a.cache.k_page_stride, box) ||
        !page_map(&maps.v, a.cache.v_pages, a.cache, a.cache.v_page_stride, box))
        return cudaErrorInvalidValue;
    const cudaError_t e = allow_smem(attend_chunk_kernel<D>, smem_bytes(D), dev, allowed);
    if (e != cudaSuccess)
        return e;
    attend_chunk_kernel<D><<<dev.sms < kMaxCtas ? dev.sms : kMaxCtas, kThreads, smem_bytes(D), stream>>>(
        a, maps, workspace, dev.status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_chunk(const smoe_attention_args &a, uint8_t *workspace, const DeviceFacts &dev,
                                   cudaStream_t stream)
{
    return a.cache.head_dim == 64 ? launch<64>(a, workspace, dev, stream) : launch<128>(a, workspace, dev, stream);
}

}  // namespace smoe
