// attention.cuh -- what the attention kernels share: the sequences of a batch,
// the keys that a row sees, and the layout of the workspace.
#pragma once

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace smoe {

// Workspace: one arrival counter per CTA (zero between launches), then the
// parts of items that several CTAs share.
constexpr size_t kPartsAt = 4096;
constexpr int kMaxCounters = static_cast<int>(kPartsAt / sizeof(unsigned));

// Allow a kernel its dynamic shared memory, once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes, const DeviceFacts &dev, std::atomic<bool> *done)
{
    if (done[dev.index].load(std::memory_order_acquire))
        return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        done[dev.index].store(true, std::memory_order_release);
    return e;
}

// Counts an arrival at a counter in global memory: what the CTA's threads wrote
// before the barrier in front of it is visible to whoever sees the count, and
// what those who counted before wrote, to the threads behind the next barrier
// (no fence of theirs is needed: the order is transitive).
__device__ __forceinline__ unsigned count_arrival(unsigned *counter)
{
    unsigned v;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(v) : "l"(counter) : "memory");
    return v;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int kMaxLen = 0x7fffffff - 511;  // key indices and their roundings fit 31 bits

// A sequence of the batch as the kernels use it; an impossible one is
// recorded and gets what is left of it in range.
struct Seq {
    int64_t row0;  // first row
    int rows;      // new rows
    int len;       // keys
};

__device__ __forceinline__ Seq seq_at(const smoe_attention_args &a, int b, int *status)
{
    Seq s;
    const int r0 = a.batch.row_start[b], r1 = a.batch.row_start[b + 1];
    s.row0 = r0;
    s.rows = r1 - r0;
    s.len = a.batch.kv_len[b];
    bool bad = r0 < 0 || r1 < r0 || r1 > a.batch.num_rows || s.rows > a.max_rows || s.len < 0 ||
               s.len > kMaxLen || s.len > (int64_t)a.batch.table_stride * a.cache.page_size;
    if (bad) {
        set_status(status, kStatusBadArg);
        s.row0 = 0;
        s.rows = s.len = 0;
    }
    return s;
}

// Keys seen by a row with key index i (negative: none): [lo, hi).
__device__ __forceinline__ void seen_from(int window, int i, int &lo, int &hi)
{
    hi = i >= 0 ? i + 1 : 0;
    lo = window > 0 && hi > window ? hi - window : 0;
}
__device__ __forceinline__ void seen_from(const smoe_attention_args &a, int i, int &lo, int &hi)
{
    seen_from(a.window, i, lo, hi);
}

__device__ __forceinline__ Seq seq_or_none(const smoe_attention_args &a, int b, int *status)
{
    Seq s;
    s.row0 = 0;
    s.rows = s.len = 0;
    return b < a.batch.num_seqs ? seq_at(a, b, status) : s;
}

}  // namespace smoe
