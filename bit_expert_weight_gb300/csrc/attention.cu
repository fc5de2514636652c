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

#include "common.cuh"
#include "internal.h"

namespace smoe {

namespace {

constexpr int kDecWarps = 8;   // warps per CTA, each with keys of its own
constexpr int kDecRows = 16;   // packed rows per tile (mma M)
constexpr int kDecKeys = 16;   // keys per warp and step (mma K of P V); a page holds them
constexpr int kDecStages = 3;  // steps in flight per warp

__host__ __device__ constexpr int dec_step_bytes(int D) { return 2 * kDecKeys * D * 2; }
__host__ __device__ constexpr int dec_smem_bytes(int D)
{
    return kDecWarps * kDecStages * dec_step_bytes(D);
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

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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
    bool bad = r0 < 0 || s.rows < 0 || r1 > a.batch.num_rows || s.rows > a.max_rows || s.len < 0 ||
               s.len > (int64_t)a.batch.table_stride * a.cache.page_size;
    if (bad) {
        set_status(status, kStatusBadArg);
        s.row0 = 0;
        s.rows = s.len = 0;
    }
    return s;
}

// Keys seen by new row `token` of s: [lo, hi).
__device__ __forceinline__ void seen(const smoe_attention_args &a, const Seq &s, int token, int &lo,
                                     int &hi)
{
    const int64_t i = (int64_t)s.len - s.rows + token;
    hi = i + 1 > 0 ? static_cast<int>(i + 1) : 0;
    lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
}

// One tile of kDecRows packed rows: the warps take the keys in turn, 16 at a
// time, and their sums are joined at the end.
template <int D>
__global__ void __launch_bounds__(32 * kDecWarps, 1)
    attend_rows_kernel(const smoe_attention_args a, int *status)
{
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[kDecWarps][kDecRows], s_l[kDecWarps][kDecRows];
    constexpr int KB = D / 16;  // k blocks of Q K^T, pairs of column blocks of P V
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.num_heads / a.cache.num_kv_heads, h = blockIdx.y, page = a.cache.page_size;
    const Seq s = seq_at(a, blockIdx.z, status);
    const int m0 = blockIdx.x * kDecRows, nrows = s.rows * G;
    if (m0 >= nrows)
        return;
    const int mlast = m0 + kDecRows - 1 < nrows ? m0 + kDecRows - 1 : nrows - 1;
    int k_lo, k_hi, t_lo, t_hi;  // keys of the tile; [t_lo, t_hi) is seen by every row
    seen(a, s, mlast / G, t_lo, k_hi);
    seen(a, s, m0 / G, k_lo, t_hi);

    // this lane's two rows
    const int g = lane >> 2, c2 = 2 * (lane & 3);
    int lo[2], hi[2];
    uint32_t q[KB][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int m = m0 + g + 8 * r;
        lo[r] = hi[r] = 0;
        const bool on = m < nrows;
        if (on)
            seen(a, s, m / G, lo[r], hi[r]);
        const uint16_t *src = static_cast<const uint16_t *>(a.q) + (s.row0 + m / G) * a.q_row_stride +
                              (int64_t)(h * G + m % G) * a.q_head_stride;
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            q[kb][r] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * kb + c2) : 0u;
            q[kb][2 + r] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * kb + 8 + c2) : 0u;
        }
    }

    const float sc = a.scale * 1.44269504088896341f;
    float o[2 * KB][4];
#pragma unroll
    for (int n = 0; n < 2 * KB; ++n)
        o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    const int base = k_lo / kDecKeys * kDecKeys + warp * kDecKeys;
    constexpr int kStride = kDecWarps * kDecKeys;
    const int steps = k_hi > base ? (k_hi - base + kStride - 1) / kStride : 0;
    const uint32_t ring = smem_u32(smem) + warp * kDecStages * dec_step_bytes(D);
    const int32_t *table = a.batch.page_table + (int64_t)blockIdx.z * a.batch.table_stride;

    auto page_of = [&](int st) { return st < steps ? table[(base + st * kStride) / page] : 0; };
    auto issue = [&](int st, int pg) {
        if (st < steps) {
            const int k0 = base + st * kStride;
            const bool there = pg >= 0 && pg < a.cache.num_pages;
            if (!there && lane == 0)
                set_status(status, kStatusBadArg);
            const int64_t at = ((int64_t)h * page + k0 % page) * D;
            const uint16_t *ks = static_cast<const uint16_t *>(a.cache.k_pages) +
                                 (there ? pg * a.cache.k_page_stride + at : 0);
            const uint16_t *vs = static_cast<const uint16_t *>(a.cache.v_pages) +
                                 (there ? pg * a.cache.v_page_stride + at : 0);
            const uint32_t dk = ring + (st % kDecStages) * dec_step_bytes(D), dv = dk + kDecKeys * D * 2;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const int e = i * 32 + lane, r = e / (D / 8), c = e % (D / 8);
                const bool v = there && k0 + r >= k_lo && k0 + r < k_hi;
                cp_async16(dk + chunk_at<D>(r, c), ks + (v ? r * D + c * 8 : 0), v);
                cp_async16(dv + chunk_at<D>(r, c), vs + (v ? r * D + c * 8 : 0), v);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int st = 0; st < kDecStages - 1; ++st)
        issue(st, page_of(st));
    int next_page = page_of(kDecStages - 1);
    for (int st = 0; st < steps; ++st) {
        issue(st + kDecStages - 1, next_page);
        next_page = page_of(st + kDecStages);
        cp_async_wait<kDecStages - 1>();
        __syncwarp();
        const uint32_t dk = ring + (st % kDecStages) * dec_step_bytes(D), dv = dk + kDecKeys * D * 2;
        const int k0 = base + st * kStride;
        float p[2][4] = {};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            uint32_t b[4];
            ldm4(b, dk + chunk_at<D>((lane & 7) + ((lane >> 4) << 3), 2 * kb + ((lane >> 3) & 1)));
            mma_bf16(p[0], q[kb], b[0], b[1]);
            mma_bf16(p[1], q[kb], b[2], b[3]);
        }
        if (k0 < t_lo || k0 + kDecKeys > t_hi) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + 8 * n + c2 + (e & 1), r = e >> 1;
                    if (key < lo[r] || key >= hi[r])
                        p[n][e] = -INFINITY;
                }
        }
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float v = fmaxf(fmaxf(p[0][2 * r], p[0][2 * r + 1]), fmaxf(p[1][2 * r], p[1][2 * r + 1]));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
            const float mn = fmaxf(mx[r], v * sc);
            const float mu = mn == -INFINITY ? 0.f : mn;  // a row that has seen nothing yet
            f[r] = ex2(mx[r] - mu);
            mx[r] = mn;
            float t = 0.f;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = p[n][2 * r + e];
                    x = ex2(fmaf(x, sc, -mu));
                    t += x;
                }
            sum[r] = sum[r] * f[r] + t;
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
            for (int n = 0; n < 2 * KB; ++n) {
                o[n][0] *= f[0];
                o[n][1] *= f[0];
                o[n][2] *= f[1];
                o[n][3] *= f[1];
            }
        }
        // P as bf16 hi + lo: the loop waits for memory, not for the second
        // product, and the output keeps fp32 accuracy
        uint32_t hi4[4], lo4[4];
        split_bf16x2(p[0][0], p[0][1], hi4[0], lo4[0]);
        split_bf16x2(p[0][2], p[0][3], hi4[1], lo4[1]);
        split_bf16x2(p[1][0], p[1][1], hi4[2], lo4[2]);
        split_bf16x2(p[1][2], p[1][3], hi4[3], lo4[3]);
#pragma unroll
        for (int n = 0; n < KB; ++n) {
            uint32_t b[4];
            ldm4t(b, dv + chunk_at<D>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)));
            mma_bf16(o[2 * n], hi4, b[0], b[1]);
            mma_bf16(o[2 * n], lo4, b[0], b[1]);
            mma_bf16(o[2 * n + 1], hi4, b[2], b[3]);
            mma_bf16(o[2 * n + 1], lo4, b[2], b[3]);
        }
        __syncwarp();
    }
    cp_async_wait<0>();

    // join the warps: each scales its sums to the tile's maximum
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
        sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        if ((lane & 3) == 0) {
            s_m[warp][g + 8 * r] = mx[r];
            s_l[warp][g + 8 * r] = sum[r];
        }
    }
    __syncthreads();  // the rings are free as well
    float *part = reinterpret_cast<float *>(smem);  // [warps][rows][D]
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w)
            m = fmaxf(m, s_m[w][g + 8 * r]);
        const float f = m == -INFINITY ? 0.f : ex2(mx[r] - m);
#pragma unroll
        for (int n = 0; n < 2 * KB; ++n)
            *reinterpret_cast<float2 *>(part + (warp * kDecRows + g + 8 * r) * D + 8 * n + c2) =
                make_float2(o[n][2 * r] * f, o[n][2 * r + 1] * f);
    }
    __syncthreads();
    for (int e = tid; e < kDecRows * D / 2; e += 32 * kDecWarps) {
        const int r = e / (D / 2), c = 2 * (e % (D / 2)), mr = m0 + r;
        if (mr >= nrows)
            continue;
        float m = -INFINITY, l = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w)
            m = fmaxf(m, s_m[w][r]);
#pragma unroll
        for (int w = 0; w < kDecWarps; ++w) {
            const float2 v = *reinterpret_cast<const float2 *>(part + (w * kDecRows + r) * D + c);
            x += v.x;
            y += v.y;
            l += m == -INFINITY ? 0.f : s_l[w][r] * ex2(s_m[w][r] - m);
        }
        const float inv = l > 0.f ? 1.0f / l : 0.f;  // a row that sees no key: zeros
        const int64_t at = (s.row0 + mr / G) * a.out_row_stride +
                           (int64_t)(h * G + mr % G) * a.out_head_stride + c;
        if (a.out_dtype == SMOE_F32)
            *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(x * inv, y * inv);
        else
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at) =
                pack_bf16x2(x * inv, y * inv);
    }
}

template <int D>
cudaError_t launch_rows(const smoe_attention_args &a, cudaStream_t stream)
{
    const int G = a.num_heads / a.cache.num_kv_heads;
    const int64_t tiles = ((int64_t)a.max_rows * G + kDecRows - 1) / kDecRows;
    cudaError_t e = cudaFuncSetAttribute(attend_rows_kernel<D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         dec_smem_bytes(D));
    if (e != cudaSuccess)
        return e;
    const dim3 grid(static_cast<unsigned>(tiles), a.cache.num_kv_heads, a.batch.num_seqs);
    attend_rows_kernel<D><<<grid, 32 * kDecWarps, dec_smem_bytes(D), stream>>>(
        a, device_status_word());
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention(const smoe_attention_args &a, void *workspace, cudaStream_t stream)
{
    (void)workspace;
    return a.cache.head_dim == 64 ? launch_rows<64>(a, stream) : launch_rows<128>(a, stream);
}

}  // namespace smoe
