// decoder_api.cu -- the C ABI of the operators beside the expert layer
// (rotation, paged append, paged attention, beams and pages): argument
// validation, and the host's frequency table.
#include <math.h>

#include "common.cuh"
#include "internal.h"

using namespace smoe;

namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A [rows, heads, head_dim] view: 16-byte aligned, strides that keep every
// run of 8 channels aligned.
inline bool valid_view(const void *p, int64_t row_stride, int64_t head_stride)
{
    return p && aligned16(p) && row_stride >= 0 && head_stride >= 0 && row_stride % 8 == 0 &&
           head_stride % 8 == 0;
}

// Such a view to be written: its rows and its heads must not lie in one place.
inline bool valid_out(const void *p, int64_t row_stride, int64_t head_stride, int64_t rows, int heads, int dim)
{
    return valid_view(p, row_stride, head_stride) && (rows == 1 || row_stride >= dim) &&
           (heads == 1 || head_stride >= dim);
}

inline bool valid_dtype(int32_t t) { return t == SMOE_F32 || t == SMOE_BF16; }

bool valid_rotation(int32_t rot_dim, int32_t head_dim, const int64_t *table, float rot_scale,
                    float eps)
{
    return rot_dim >= 8 && rot_dim % 8 == 0 && rot_dim <= head_dim && table && aligned16(table) &&
           isfinite(rot_scale) && isfinite(eps) && eps >= 0.0f;
}

inline bool valid_page_size(int32_t n) { return n >= 16 && n <= 256 && !(n & (n - 1)); }

bool valid_cache(const smoe_kv_cache &c)
{
    if (!valid_page_size(c.page_size))
        return false;
    if (c.head_dim != 64 && c.head_dim != 128)
        return false;
    if (c.num_kv_heads < 1 || c.num_kv_heads > 65535 || c.num_pages < 1 ||
        c.num_pages > 0x7fffffff)
        return false;
    const int64_t page = (int64_t)c.num_kv_heads * c.page_size * c.head_dim;
    return c.k_pages && c.v_pages && aligned16(c.k_pages) && aligned16(c.v_pages) &&
           c.k_page_stride >= page && c.v_page_stride >= page && c.k_page_stride % 8 == 0 &&
           c.v_page_stride % 8 == 0;
}

bool valid_batch(const smoe_kv_batch &b)
{
    return b.num_rows >= 0 && b.num_rows <= 0x7fffffff && b.num_seqs >= 0 &&
           b.num_seqs <= SMOE_MAX_SEQS && b.table_stride >= 0;
}

bool batch_pointers(const smoe_kv_batch &b) { return b.row_start && b.kv_len && b.page_table; }

bool valid_pool(const smoe_page_pool &p)
{
    return p.num_pages >= 1 && p.num_pages <= (1 << 30) && valid_page_size(p.page_size) && p.num_seqs >= 0 &&
           p.num_seqs <= SMOE_MAX_SEQS && p.table_stride >= 0 && p.table_stride <= (1 << 27) && p.refs &&
           aligned16(p.refs) &&
           (p.num_seqs == 0 || (p.kv_len && (p.page_table || p.table_stride == 0)));
}

// b is a itself, or no part of it.
inline bool same_or_apart(const int32_t *a, const int32_t *b, int64_t n) { return a == b || a + n <= b || b + n <= a; }

smoe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SMOE_OK : SMOE_ERR_CUDA; }

}  // namespace

extern "C" {

smoe_status smoe_rope_table(int32_t rot_dim, double theta, const smoe_rope_scaling *scaling,
                            int64_t *table, float *rot_scale)
{
    const double kPi = 3.14159265358979323846;
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > SMOE_MAX_HEAD_DIM || !(theta > 1.0) ||
        !isfinite(theta) || !table || !rot_scale)
        return SMOE_ERR_INVALID_ARG;
    const int kind = scaling ? scaling->kind : SMOE_ROPE_PLAIN;
    if (kind < SMOE_ROPE_PLAIN || kind > SMOE_ROPE_BANDS)
        return SMOE_ERR_INVALID_ARG;
    if (kind != SMOE_ROPE_PLAIN && (!(scaling->factor >= 1.0) || !isfinite(scaling->factor)))
        return SMOE_ERR_INVALID_ARG;
    if (kind >= SMOE_ROPE_PARTS &&
        (!(scaling->original_len > 0.0) || !isfinite(scaling->original_len) ||
         !(scaling->slow > 0.0) || !(scaling->fast > scaling->slow) || !isfinite(scaling->fast)))
        return SMOE_ERR_INVALID_ARG;
    const double s = kind == SMOE_ROPE_PLAIN ? 1.0 : scaling->factor;
    double low = 0.0, high = 0.0;
    if (kind == SMOE_ROPE_PARTS) {
        // pair index at which a pair makes `turns` turns in original_len
        const auto at = [&](double turns) {
            return rot_dim * log(scaling->original_len / (2.0 * kPi * turns)) / (2.0 * log(theta));
        };
        low = fmax(0.0, floor(at(scaling->fast)));
        high = fmin(rot_dim - 1.0, ceil(at(scaling->slow)));
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(theta, -2.0 * i / rot_dim);
        if (kind == SMOE_ROPE_LINEAR) {
            f /= s;
        } else if (kind == SMOE_ROPE_PARTS) {
            const double ramp = fmin(1.0, fmax(0.0, (i - low) / fmax(high - low, 0.001)));
            f = f / s * ramp + f * (1.0 - ramp);
        } else if (kind == SMOE_ROPE_BANDS) {
            const double turns = scaling->original_len * f / (2.0 * kPi);
            const double keep =
                fmin(1.0, fmax(0.0, (turns - scaling->slow) / (scaling->fast - scaling->slow)));
            f = f / s * (1.0 - keep) + f * keep;
        }
        // f <= 1, so a pair makes at most 1 / (2 pi) turns per position
        table[i] = static_cast<int64_t>(llrint(f / (2.0 * kPi) * 0x1p64));
    }
    *rot_scale = kind == SMOE_ROPE_PARTS ? static_cast<float>(0.1 * log(s) + 1.0) : 1.0f;
    return SMOE_OK;
}

smoe_status smoe_rope(const smoe_rope_args *a, void *cuda_stream)
{
    if (!a || a->num_rows < 0 || a->num_rows > 0x7fffffff || a->num_heads < 0 ||
        a->num_heads > 65535 || a->head_dim < 8 || a->head_dim % 8 ||
        a->head_dim > SMOE_MAX_HEAD_DIM || !valid_dtype(a->dtype))
        return SMOE_ERR_INVALID_ARG;
    if (a->num_rows == 0 || a->num_heads == 0)
        return SMOE_OK;
    if (!valid_view(a->x, a->x_row_stride, a->x_head_stride) ||
        !valid_out(a->out, a->out_row_stride, a->out_head_stride, a->num_rows, a->num_heads, a->head_dim) ||
        !a->positions ||
        !valid_rotation(a->rot_dim, a->head_dim, a->table, a->rot_scale, a->eps) ||
        (a->norm_w && !aligned16(a->norm_w)))
        return SMOE_ERR_INVALID_ARG;
    if (a->out == a->x &&
        (a->x_row_stride != a->out_row_stride || a->x_head_stride != a->out_head_stride))
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_rope(*a, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_kv_append(const smoe_kv_append_args *a, void *cuda_stream)
{
    if (!a || !valid_cache(a->cache) || !valid_batch(a->batch) || !valid_dtype(a->dtype) ||
        a->num_heads < 0 || a->num_heads > 65535)
        return SMOE_ERR_INVALID_ARG;
    if (a->batch.num_rows == 0 || a->batch.num_seqs == 0)
        return SMOE_OK;
    if (!batch_pointers(a->batch) || !valid_view(a->k, a->k_row_stride, a->k_head_stride) ||
        !valid_view(a->v, a->v_row_stride, a->v_head_stride))
        return SMOE_ERR_INVALID_ARG;
    if (a->q && (a->num_heads < 1 || !valid_view(a->q, a->q_row_stride, a->q_head_stride) ||
                 !valid_out(a->q_out, a->qo_row_stride, a->qo_head_stride, a->batch.num_rows, a->num_heads,
                            a->cache.head_dim)))
        return SMOE_ERR_INVALID_ARG;
    if (a->q && a->q_out == a->q &&
        (a->dtype != SMOE_BF16 || a->q_row_stride != a->qo_row_stride ||
         a->q_head_stride != a->qo_head_stride))
        return SMOE_ERR_INVALID_ARG;
    if (a->rot_dim != 0 &&
        !valid_rotation(a->rot_dim, a->cache.head_dim, a->table, a->rot_scale, a->eps))
        return SMOE_ERR_INVALID_ARG;
    if (!(isfinite(a->eps) && a->eps >= 0.0f) || (a->q_norm && !aligned16(a->q_norm)) ||
        (a->k_norm && !aligned16(a->k_norm)))
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_kv_append(*a, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_attention(const smoe_attention_args *a, void *workspace, size_t workspace_bytes,
                           void *cuda_stream)
{
    if (!a || !valid_cache(a->cache) || !valid_batch(a->batch) || !valid_dtype(a->out_dtype))
        return SMOE_ERR_INVALID_ARG;
    if (a->num_heads < 1 || a->num_heads % a->cache.num_kv_heads ||
        a->num_heads / a->cache.num_kv_heads > 128 || a->window < 0 ||
        !isfinite(a->scale) || !(a->scale > 0.0f) ||
        a->batch.num_rows * a->num_heads > 0x7fffffff - 511)  // (rounded up to tiles, they fit 31 bits)
        return SMOE_ERR_INVALID_ARG;
    if (a->batch.num_rows == 0 || a->batch.num_seqs == 0)
        return SMOE_OK;
    if (a->max_rows < 1 || !batch_pointers(a->batch) || !valid_view(a->q, a->q_row_stride, a->q_head_stride) ||
        !valid_out(a->out, a->out_row_stride, a->out_head_stride, a->batch.num_rows, a->num_heads,
                   a->cache.head_dim) ||
        a->out == a->q)
        return SMOE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return SMOE_ERR_INVALID_ARG;
    if (workspace_bytes < SMOE_ATTENTION_WORKSPACE_BYTES)
        return SMOE_ERR_WORKSPACE;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_attention(*a, workspace, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_beam_select(const smoe_beam_args *a, void *workspace, size_t workspace_bytes, void *cuda_stream)
{
    if (!a || !valid_dtype(a->dtype) || a->vocab < 1 || a->vocab > SMOE_MAX_VOCAB || a->num_groups < 0 ||
        a->beams < 1 || a->beams > SMOE_MAX_BEAMS || a->num_groups > SMOE_MAX_SEQS / a->beams || a->num_out < 1 ||
        a->num_out > SMOE_MAX_BEAMS || a->end_token < -1 || a->end_token >= a->vocab || a->row_stride < 0 ||
        a->row_stride > (1ll << 40))
        return SMOE_ERR_INVALID_ARG;
    if (a->num_groups == 0)
        return SMOE_OK;
    const uintptr_t unit = a->dtype == SMOE_F32 ? 4 : 2;
    if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % unit || !a->scores || !a->scores_out ||
        !a->parents || !a->tokens || a->parents == a->tokens || a->parents == a->last)
        return SMOE_ERR_INVALID_ARG;
    // in place: a group is written when all of it has been read, so it has to lie where it was
    if (a->num_out != a->beams && (a->scores_out == a->scores || a->tokens == a->last))
        return SMOE_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return SMOE_ERR_INVALID_ARG;
    if (workspace_bytes < SMOE_BEAM_WORKSPACE_BYTES)
        return SMOE_ERR_WORKSPACE;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_beam_select(*a, workspace, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_pages_fork(const smoe_page_pool *pool, const int32_t *parent, const int32_t *keep,
                            void *cuda_stream)
{
    if (!pool || !valid_pool(*pool))
        return SMOE_ERR_INVALID_ARG;
    if (pool->num_seqs == 0)
        return SMOE_OK;
    if (!parent || parent == pool->kv_len || keep == pool->kv_len)
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_pages_fork(*pool, parent, keep, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_pages_reserve(const smoe_page_pool *pool, const int32_t *row_start, int32_t *copies,
                               int32_t *counts, void *cuda_stream)
{
    if (!pool || !valid_pool(*pool) || !counts)
        return SMOE_ERR_INVALID_ARG;
    if (pool->num_seqs > 0 && (!row_start || !copies))
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(
        launch_pages_reserve(*pool, row_start, copies, counts, dev, static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_pages_copy(const smoe_kv_cache *caches, int32_t num_caches, const int32_t *copies,
                            const int32_t *counts, int32_t max_copies, void *cuda_stream)
{
    if (num_caches < 0 || num_caches > SMOE_MAX_CACHES || max_copies < 0 || (num_caches > 0 && !caches))
        return SMOE_ERR_INVALID_ARG;
    for (int i = 0; i < num_caches; ++i) {
        const smoe_kv_cache &c = caches[i], &first = caches[0];
        if (!valid_cache(c) || c.num_pages != first.num_pages || c.k_page_stride != first.k_page_stride ||
            c.v_page_stride != first.v_page_stride || c.page_size != first.page_size ||
            c.num_kv_heads != first.num_kv_heads || c.head_dim != first.head_dim)
            return SMOE_ERR_INVALID_ARG;
    }
    if (num_caches == 0 || max_copies == 0)
        return SMOE_OK;
    if (!copies || !counts)
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_pages_copy(caches, num_caches, copies, counts, max_copies, dev,
                                         static_cast<cudaStream_t>(cuda_stream)));
}

smoe_status smoe_pages_compact(const smoe_page_pool *pool, int32_t *refs_out, int32_t *table_out, int32_t *copies,
                               int32_t max_copies, int32_t *counts, void *cuda_stream)
{
    if (!pool || !valid_pool(*pool) || !refs_out || !counts || max_copies < pool->num_pages / 2 ||
        (max_copies > 0 && !copies) || (reinterpret_cast<uintptr_t>(copies) & 7) || !same_or_apart(pool->refs, refs_out, pool->num_pages))
        return SMOE_ERR_INVALID_ARG;
    if (pool->num_seqs > 0 && pool->table_stride > 0 &&
        (!table_out ||
         !same_or_apart(pool->page_table, table_out, (int64_t)pool->num_seqs * pool->table_stride)))
        return SMOE_ERR_INVALID_ARG;
    const DeviceFacts &dev = device_facts();
    if (!dev.supported)
        return SMOE_ERR_UNSUPPORTED;
    return cuda_status(launch_pages_compact(*pool, refs_out, table_out, copies, counts, dev,
                                            static_cast<cudaStream_t>(cuda_stream)));
}

}  // extern "C"
