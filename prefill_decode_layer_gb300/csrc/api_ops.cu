// C ABI of the operators on device buffers beside the sampler's (include/ds4g.h): the
// paged K/V cache, rows of probabilities and draft verification.  Validation here, work
// in the kernel files; nothing is kept between calls.
#include <atomic>

#include "paged.h"

using namespace ds4g;

namespace {

bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
constexpr int kMaxHeads = 65536;  // element offsets within a token's row are 32-bit
size_t elem(int dtype) { return dtype == DS4G_BF16 ? 2 : 4; }
bool dtype_ok(int dtype) { return dtype == DS4G_BF16 || dtype == DS4G_F32; }
// A stride in elements of rows of at least `row` elements: whole 16-byte vectors.
bool stride_ok(int64_t s, int64_t row, int dtype) { return s >= row && s * (int64_t)elem(dtype) % 16 == 0; }

bool kv_ok(const ds4g_paged_kv *kv)
{
    if (!kv || !kv->k || !kv->v || !al16(kv->k) || !al16(kv->v) || !dtype_ok(kv->dtype)) return false;
    if (kv->n_pages < 1 || kv->page_size < 1 || kv->n_kv_heads < 1 || kv->n_kv_heads > kMaxHeads) return false;
    if (kv->head_dim < 8 || kv->head_dim > 256 || kv->head_dim % 8) return false;
    return stride_ok(kv->page_stride, kv->head_dim, kv->dtype) && stride_ok(kv->slot_stride, kv->head_dim, kv->dtype) &&
           stride_ok(kv->head_stride, kv->head_dim, kv->dtype);
}

bool batch_ok(const ds4g_paged_batch *b, int page_size)
{
    if (!b || b->n_seqs < 0 || b->n_tokens < 0) return false;
    if (b->n_seqs == 0) return b->n_tokens == 0 || b->start;
    if (!b->length || b->width < 0 || b->table_stride < b->width || (b->width > 0 && !b->table)) return false;
    if ((int64_t)b->width * page_size > 0x7fffff00) return false;   // positions are 32-bit
    if (b->max_new < 1) return false;
    return b->start || (b->max_new == 1 && b->n_tokens == b->n_seqs);
}

bool kv8_ok(const ds4g_paged_kv8 *kv)
{
    if (!kv || !kv->k || !kv->v || !al16(kv->k) || !al16(kv->v)) return false;
    if (!kv->k_scale || !kv->v_scale || ((uintptr_t)kv->k_scale & 3u) || ((uintptr_t)kv->v_scale & 3u)) return false;
    if (kv->n_pages < 1 || kv->page_size < 1 || kv->n_kv_heads < 1 || kv->n_kv_heads > kMaxHeads) return false;
    if (kv->head_dim < 8 || kv->head_dim > 256 || kv->head_dim % 8) return false;
    if (kv->block < 1 || kv->page_size % kv->block) return false;
    const int64_t scales = (int64_t)(kv->page_size / kv->block) * kv->n_kv_heads;
    if (scales > 0x7fffffff || kv->scale_stride < scales) return false;
    for (const int64_t s : {kv->page_stride, kv->slot_stride, kv->head_stride})
        if (s < kv->head_dim || s % 16) return false;
    return true;
}

PagedKV kv_of(const ds4g_paged_kv &kv)
{
    return {kv.k, kv.v, kv.page_stride, kv.slot_stride, kv.head_stride, kv.n_pages, kv.page_size, kv.n_kv_heads,
            kv.head_dim, nullptr, nullptr, 0, kv.page_size};
}
PagedKV kv_of(const ds4g_paged_kv8 &kv)
{
    return {kv.k, kv.v, kv.page_stride, kv.slot_stride, kv.head_stride, kv.n_pages, kv.page_size, kv.n_kv_heads,
            kv.head_dim, kv.k_scale, kv.v_scale, kv.scale_stride, kv.block};
}
PagedSeqs seqs_of(const ds4g_paged_batch &b)
{
    return {b.table, b.length, b.start, b.n_seqs, b.n_tokens, b.max_new, b.width, b.table_stride};
}

// SMs of the current device; 0 if there is none.  (Asked for once per device: a constant of
// the device, not of a call.)
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev)) return 0;
    const bool keep = dev >= 0 && dev < 64;
    if (keep && (n = known[dev].load(std::memory_order_relaxed))) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) return 0;
    if (keep) known[dev].store(n, std::memory_order_relaxed);
    return n;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? DS4G_OK : DS4G_ECUDA; }

constexpr int kMaxNew = 128;      // new tokens of one sequence in an attention call
constexpr int kMaxDraftsApi = 64;

bool heads_ok(int n_kv_heads, int n_heads)
{
    return n_heads >= 1 && n_heads <= kMaxHeads && n_heads % n_kv_heads == 0;
}

// The appends, behind the checks of the cache: `kv` its copy, dtype of the rows.
template <typename Go>
int append_to(const PagedKV &kv, const ds4g_paged_batch *batch, const void *k, int64_t k_stride, const void *v,
              int64_t v_stride, const ds4g_rope *rope, const void *q, int64_t q_stride, void *q_out,
              int64_t q_out_stride, int n_heads, int dtype, Go go)
{
    if (!batch_ok(batch, kv.page_size) || !dtype_ok(dtype)) return DS4G_EINVAL;
    if (batch->n_tokens == 0) return DS4G_OK;
    const int64_t row = (int64_t)kv.n_kv_heads * kv.head_dim;
    if (!k || !v || !al16(k) || !al16(v) || !stride_ok(k_stride, row, dtype) || !stride_ok(v_stride, row, dtype))
        return DS4G_EINVAL;
    if (rope && (!rope->cs || !al16(rope->cs) || rope->n_pos < 1 || rope->rot_dim < 2 || rope->rot_dim % 2 ||
                 rope->rot_dim > kv.head_dim))
        return DS4G_EINVAL;
    if (q) {
        if (!q_out || n_heads < 1 || n_heads > kMaxHeads || !al16(q) || !al16(q_out)) return DS4G_EINVAL;
        const int64_t qrow = (int64_t)n_heads * kv.head_dim;
        if (!stride_ok(q_stride, qrow, dtype) || !stride_ok(q_out_stride, qrow, dtype)) return DS4G_EINVAL;
        if (q == q_out && q_stride != q_out_stride) return DS4G_EINVAL;
    } else if (q_out) {
        return DS4G_EINVAL;
    }
    const int nsm = sm_count();
    if (!nsm) return DS4G_ECUDA;
    const AppendArgs a = {kv, seqs_of(*batch), k, v, q, q_out, k_stride, v_stride, q_stride, q_out_stride,
                          rope ? rope->cs : nullptr, rope ? rope->n_pos : 0, rope ? rope->rot_dim : 0, q ? n_heads : 0};
    return status_of(go(a, nsm));
}

size_t attention_ws_bytes(const PagedKV &kv, int kv_dtype, const ds4g_paged_batch *batch, int n_heads)
{
    if (!batch_ok(batch, kv.page_size) || !heads_ok(kv.n_kv_heads, n_heads) || batch->max_new > kMaxNew) return 0;
    return paged_attn_ws_bytes(kv, n_heads / kv.n_kv_heads, batch->n_seqs ? batch->max_new : 1, kv_dtype);
}

// The attention, behind the checks of the cache.
int attend_over(const PagedKV &kv, int kv_dtype, const ds4g_paged_batch *batch, const void *q, int64_t q_stride,
                void *out, int64_t out_stride, int n_heads, int dtype, float scale, int window, void *workspace,
                size_t workspace_bytes, void *stream)
{
    if (!batch_ok(batch, kv.page_size) || !dtype_ok(dtype) || !heads_ok(kv.n_kv_heads, n_heads)) return DS4G_EINVAL;
    if (!(scale >= 0.f && scale <= 1e38f)) return DS4G_EINVAL;   // (in powers of two it stays finite)
    if (batch->n_tokens == 0 || batch->n_seqs == 0) return DS4G_OK;
    if (batch->max_new > kMaxNew) return DS4G_EINVAL;
    // units of one sequence are counted in 32 bits (64 keys and 4 query rows a unit at least)
    if ((double)batch->width * kv.page_size / 64 * ((double)batch->max_new * n_heads / 4 + kv.n_kv_heads) > 2e9)
        return DS4G_EINVAL;
    const int64_t row = (int64_t)n_heads * kv.head_dim;
    if (!q || !out || q == out || !al16(q) || !al16(out) || !stride_ok(q_stride, row, dtype) || !stride_ok(out_stride, row, dtype))
        return DS4G_EINVAL;
    if (!workspace || ((uintptr_t)workspace & 255u)) return DS4G_EINVAL;
    if (workspace_bytes < attention_ws_bytes(kv, kv_dtype, batch, n_heads)) return DS4G_ESIZE;
    const int nsm = sm_count();
    if (!nsm) return DS4G_ECUDA;
    const float sc = scale != 0.f ? scale : 1.f / sqrtf((float)kv.head_dim);
    AttnArgs a = {kv, seqs_of(*batch), q, out, q_stride, out_stride, n_heads / kv.n_kv_heads, 0,
                  (float)((double)sc * 1.4426950408889634), window > 0 ? window : 0, 0, static_cast<char *>(workspace)};
    return status_of(paged_attention(a, dtype, kv_dtype, static_cast<cudaStream_t>(stream), nsm));
}

}  // namespace

extern "C" {

int ds4g_rope_fill(float *cs, int n_pos, int rot_dim, float base, void *stream)
{
    if (!cs || !al16(cs) || n_pos < 1 || rot_dim < 2 || rot_dim % 2 || !(base > 0.f)) return DS4G_EINVAL;
    return status_of(rope_fill(reinterpret_cast<float2 *>(cs), n_pos, rot_dim / 2, (double)base,
                               static_cast<cudaStream_t>(stream)));
}

int ds4g_paged_append(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, const ds4g_rope *rope, const void *q, int64_t q_stride,
                      void *q_out, int64_t q_out_stride, int n_heads, int dtype, void *stream)
{
    if (!kv_ok(kv)) return DS4G_EINVAL;
    return append_to(kv_of(*kv), batch, k, k_stride, v, v_stride, rope, q, q_stride, q_out, q_out_stride, n_heads, dtype,
                     [&](const AppendArgs &a, int nsm) {
                         return paged_append(a, dtype, kv->dtype, static_cast<cudaStream_t>(stream), nsm);
                     });
}

int ds4g_paged_append8(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, const ds4g_rope *rope, const void *q, int64_t q_stride,
                       void *q_out, int64_t q_out_stride, int n_heads, int dtype, void *stream)
{
    if (!kv8_ok(kv)) return DS4G_EINVAL;
    return append_to(kv_of(*kv), batch, k, k_stride, v, v_stride, rope, q, q_stride, q_out, q_out_stride, n_heads, dtype,
                     [&](const AppendArgs &a, int nsm) {
                         return paged_append8(a, dtype, static_cast<cudaStream_t>(stream), nsm);
                     });
}

size_t ds4g_paged_attention_workspace_bytes(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, int n_heads)
{
    return kv_ok(kv) ? attention_ws_bytes(kv_of(*kv), kv->dtype, batch, n_heads) : 0;
}

size_t ds4g_paged_attention8_workspace_bytes(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, int n_heads)
{
    return kv8_ok(kv) ? attention_ws_bytes(kv_of(*kv), kE4m3, batch, n_heads) : 0;
}

int ds4g_paged_attention(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, const void *q, int64_t q_stride,
                         void *out, int64_t out_stride, int n_heads, int dtype, float scale, int window,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    if (!kv_ok(kv)) return DS4G_EINVAL;
    return attend_over(kv_of(*kv), kv->dtype, batch, q, q_stride, out, out_stride, n_heads, dtype, scale, window,
                       workspace, workspace_bytes, stream);
}

int ds4g_paged_attention8(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, const void *q, int64_t q_stride,
                          void *out, int64_t out_stride, int n_heads, int dtype, float scale, int window,
                          void *workspace, size_t workspace_bytes, void *stream)
{
    if (!kv8_ok(kv)) return DS4G_EINVAL;
    return attend_over(kv_of(*kv), kE4m3, batch, q, q_stride, out, out_stride, n_heads, dtype, scale, window, workspace,
                       workspace_bytes, stream);
}

int ds4g_paged_attention_status(void *workspace, void *stream)
{
    if (!workspace || ((uintptr_t)workspace & 255u)) return DS4G_EINVAL;
    int status = DS4G_OK;
    const cudaError_t e = paged_attn_status(workspace, static_cast<cudaStream_t>(stream), &status);
    return e ? DS4G_ECUDA : status;
}

int ds4g_paged_resize(const ds4g_page_pool *pool, int32_t *table, int width, int table_stride, int32_t *length,
                      const int32_t *want, int n_seqs, int32_t *start, int64_t *slots, int max_tokens, void *stream)
{
    if (!pool || !pool->n_free || pool->capacity < 0 || pool->page_size < 1) return DS4G_EINVAL;
    if (pool->capacity > 0 && !pool->free_pages) return DS4G_EINVAL;
    if (n_seqs < 0 || max_tokens < 0 || !start) return DS4G_EINVAL;
    if (n_seqs > kResizeMaxSeqs) return DS4G_ESIZE;
    if (width < 0 || table_stride < width || (n_seqs > 0 && (!length || !want || (width > 0 && !table)))) return DS4G_EINVAL;
    if ((int64_t)width * pool->page_size > 0x7fffff00 || (int64_t)width * n_seqs > 0x7fffffff) return DS4G_EINVAL;
    if ((uintptr_t)slots & 7u) return DS4G_EINVAL;
    const ResizeArgs a = {pool->free_pages, pool->n_free, pool->capacity, pool->page_size, table, width, table_stride,
                          length, start, want, n_seqs, max_tokens, reinterpret_cast<long long *>(slots)};
    return status_of(paged_resize(a, static_cast<cudaStream_t>(stream)));
}

int ds4g_edit_logits(const float *logits, int64_t logits_stride, int n_rows, int n_vocab, const ds4g_logit_edits *e,
                     float *out, int64_t out_stride, void *stream)
{
    if (n_rows < 0 || n_vocab < 1 || !e) return DS4G_EINVAL;
    if (n_vocab > kMaxRowVocab) return DS4G_ESIZE;
    if (n_rows == 0) return DS4G_OK;
    if (!logits || !out || logits_stride < n_vocab || out_stride < n_vocab || n_rows > (1 << 24)) return DS4G_EINVAL;   // (items are 32-bit)
    if (logits == out && logits_stride != out_stride) return DS4G_EINVAL;
    // (a part without entries needs no array)
    if (e->max_history < 0 || (e->max_history > 0 && !e->history) || (n_rows > 1 && e->history_stride < e->max_history))
        return DS4G_EINVAL;
    if (e->max_bias < 0 || (e->max_bias > 0 && (!e->bias_ids || !e->bias)) || (n_rows > 1 && e->bias_stride < e->max_bias))
        return DS4G_EINVAL;
    if (e->max_bias > kEditMaxBias || e->max_history >= 1 << 30) return DS4G_ESIZE;
    if (e->allowed && n_rows > 1 && e->allowed_stride != 0 && e->allowed_stride < (n_vocab + 31) / 32) return DS4G_EINVAL;
    const int nsm = sm_count();
    if (!nsm) return DS4G_ECUDA;
    const EditArgs a = {logits, out, logits_stride, out_stride, n_rows, n_vocab,
                        e->max_history ? e->history : nullptr, e->n_history, e->n_prompt,
                        e->history_stride, e->max_history, e->repetition, e->frequency, e->presence, e->max_bias ? e->bias_ids : nullptr,
                        e->n_bias, e->bias, e->bias_stride, e->max_bias, e->allowed, e->allowed_stride};
    return status_of(edit_rows(a, static_cast<cudaStream_t>(stream), nsm));
}

int ds4g_probs(const float *logits, int64_t logits_stride, int n_rows, int n_vocab, float temperature, float *probs,
               int64_t probs_stride, void *stream)
{
    if (n_rows < 0 || n_vocab < 1 || temperature != temperature) return DS4G_EINVAL;
    if (n_vocab > kMaxRowVocab) return DS4G_ESIZE;
    if (n_rows == 0) return DS4G_OK;
    if (!logits || !probs || logits_stride < n_vocab || probs_stride < n_vocab || n_rows > (1 << 27)) return DS4G_EINVAL;
    if (logits == probs && logits_stride != probs_stride) return DS4G_EINVAL;
    const int nsm = sm_count();
    if (!nsm) return DS4G_ECUDA;
    return status_of(probs_rows(logits, logits_stride, n_rows, n_vocab, temperature, probs, probs_stride,
                                static_cast<cudaStream_t>(stream), nsm));
}

int ds4g_verify_draft(const float *p, int64_t p_seq_stride, int64_t p_stride, const float *q, int64_t q_seq_stride,
                      int64_t q_stride, const int32_t *drafts, const int32_t *n_drafts, const uint32_t *u24,
                      int n_seqs, int max_drafts, int n_vocab, int32_t *accepted, int32_t *tokens, void *stream)
{
    if (n_seqs < 0 || n_seqs > (1 << 27) || max_drafts < 0 || max_drafts > kMaxDraftsApi || n_vocab < 1)
        return DS4G_EINVAL;
    if (n_vocab > kMaxRowVocab) return DS4G_ESIZE;
    if (n_seqs == 0) return DS4G_OK;
    if (!p || !u24 || !accepted || !tokens || (max_drafts > 0 && !drafts)) return DS4G_EINVAL;
    if (p_stride < n_vocab || p_seq_stride < n_vocab) return DS4G_EINVAL;
    if (max_drafts == 0) q = nullptr;
    if (q && (q_stride < n_vocab || q_seq_stride < n_vocab)) return DS4G_EINVAL;
    const VerifyArgs a = {p, q, p_seq_stride, p_stride, q_seq_stride, q_stride, drafts, n_drafts,
                          u24, max_drafts, n_vocab, accepted, tokens};
    const int nsm = sm_count();
    if (!nsm) return DS4G_ECUDA;
    return status_of(verify_rows(a, n_seqs, static_cast<cudaStream_t>(stream), nsm));
}

}  // extern "C"
