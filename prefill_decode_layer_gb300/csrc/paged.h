// Operators on a paged K/V cache, probabilities and draft verification: arguments
// and host-side entry points of their kernel files (internal to the library).
#pragma once

#include <atomic>

#include "common.cuh"

namespace ds4g {

// Whether something has been set on the current device (function attributes last as long as
// the device's context, so they are set once per kernel and device).  Setting one twice, from
// two threads, does no harm.
struct PerDevice {
    std::atomic<bool> done[64];
    bool needs(int &dev) const
    {
        if (cudaGetDevice(&dev) || dev < 0 || dev >= 64) return dev = -1, true;
        return !done[dev].load(std::memory_order_acquire);
    }
    void set(int dev)
    {
        if (dev >= 0) done[dev].store(true, std::memory_order_release);
    }
};
// Let a kernel use `smem` bytes of dynamic shared memory (and clusters of 16), once per device.
template <typename K> inline cudaError_t allow_once(PerDevice &once, K kernel, size_t smem, bool wide_cluster = false)
{
    int dev = -1;
    if (!once.needs(dev)) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (!e && wide_cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (!e) once.set(dev);
    return e;
}

// Element type of a cache in 8 bits beside DS4G_F32 and DS4G_BF16 (the C interface has a struct of its own for it).
constexpr int kE4m3 = 2;
struct e4m3 {
    uint8_t bits;
};
// Bounds of an 8-bit cache's scales (ds4g_paged_kv8); anything else is taken as the nearer one, NaN as the lower.
constexpr float kScaleMin = 0x1p-64f, kScaleMax = 0x1p64f;
__device__ __forceinline__ float kv8_scale(float s) { return fminf(fmaxf(s, kScaleMin), kScaleMax); }

// A cache's pages, copied into kernel arguments (strides in elements).  In 8 bits: a scale for each
// `block` slots and head, [page][page_size / block][n_kv_heads] with `scale_stride` floats a page.
struct PagedKV {
    const void *k, *v;
    long long page_stride, slot_stride, head_stride;
    int n_pages, page_size, n_kv_heads, head_dim;
    const float *k_scale, *v_scale;
    long long scale_stride;
    int block;
};

// The sequences of a call, copied into kernel arguments.
struct PagedSeqs {
    const int *table, *length, *start;
    int n_seqs, n_tokens, max_new, width, table_stride;
};

struct AppendArgs {
    PagedKV kv;
    PagedSeqs s;
    const void *k, *v, *q;
    void *q_out;
    long long k_stride, v_stride, q_stride, q_out_stride;
    const float *cs;   // null: no rotation
    int n_pos, rot_dim;
    int n_heads;       // 0: no queries
};
cudaError_t paged_append(const AppendArgs &a, int in_dtype, int kv_dtype, cudaStream_t st, int nsm);
cudaError_t paged_append8(const AppendArgs &a, int in_dtype, cudaStream_t st, int nsm);

struct AttnArgs {
    PagedKV kv;
    PagedSeqs s;
    const void *q;
    void *out;
    long long q_stride, out_stride;
    int group;         // query heads per K/V head
    int rows;          // query rows of a row tile: (token, head of the group) pairs
    float scale_log2;  // scale * log2(e)
    int window;        // 0: no window
    int whole;         // items are not cut between CTAs
    char *ws;          // records, then parts (PartLayout)
};
// Whether the tensor-core form covers the call (paged_attn_tc.cu).
bool paged_attn_tc_ok(const PagedKV &kv, int group, int q_dtype, int kv_dtype);
// Query rows per tile of the tensor-core form: whole tokens, at most 128 rows.
int paged_attn_tc_rows(int group, int max_new);
cudaError_t paged_attn_tc(AttnArgs &a, cudaStream_t st, int nsm);
// The tensor-core form over a cache in 8 bits (paged_attn8_tc.cu): BF16 queries.
bool paged_attn8_tc_ok(const PagedKV &kv, int q_dtype);
int paged_attn8_tc_rows(int n_kv_heads, int group, int max_new);   // (of all K/V heads of a unit)
cudaError_t paged_attn8_tc(AttnArgs &a, cudaStream_t st, int nsm);
// Shared by the forms (paged_attn.cu): CTAs of a launch over units of kt keys (and
// a.whole), and the join of the tensor-core form's parts.
int paged_attn_grid(AttnArgs &a, int kt, int most);
cudaError_t paged_join_tc(const AttnArgs &a, int ctas, int nsm, cudaStream_t st);
size_t paged_attn_ws_bytes(const PagedKV &kv, int group, int max_new, int kv_dtype);
// DS4G_ETIMEOUT once after calls on the workspace in which a wait gave up (synchronises st).
cudaError_t paged_attn_status(void *ws, cudaStream_t st, int *status);
cudaError_t paged_attention(const AttnArgs &a, int q_dtype, int kv_dtype, cudaStream_t st, int nsm);

cudaError_t probs_rows(const float *logits, long long ls, int rows, int n, float temperature, float *out,
                       long long os, cudaStream_t st, int nsm);

struct VerifyArgs {
    const float *p, *q;
    long long ps, pstride, qs, qstride;
    const int *drafts, *n_drafts;
    const unsigned *u24;
    int max_drafts, n;
    int *accepted, *tokens;
};
cudaError_t verify_rows(const VerifyArgs &a, int n_seqs, cudaStream_t st, int nsm);

struct ResizeArgs {
    int *free, *n_free;
    int capacity, page_size;
    int *table;
    int width, table_stride;
    int *length, *start;
    const int *want;
    int n_seqs, max_tokens;
    long long *slots;   // or null
};
cudaError_t paged_resize(const ResizeArgs &a, cudaStream_t st);
constexpr int kResizeMaxSeqs = 65536;

struct EditArgs {
    const float *in;
    float *out;
    long long in_stride, out_stride;
    int rows, n;
    const int *history, *n_history, *n_prompt;
    long long history_stride;
    int max_history;
    const float *repetition, *frequency, *presence;
    const int *bias_ids, *n_bias;
    const float *bias;
    long long bias_stride;
    int max_bias;
    const uint32_t *allowed;
    long long allowed_stride;
};
cudaError_t edit_rows(const EditArgs &a, cudaStream_t st, int nsm);
constexpr int kEditMaxBias = 1024;

// Largest vocabulary of probs_rows, verify_rows and edit_rows.
constexpr int kMaxRowVocab = 1 << 20;

// api.cu's RoPE table fill: [n_pos][half] (cos, sin), angles in FP64.
cudaError_t rope_fill(float2 *t, int n_pos, int half, double base, cudaStream_t st);

}  // namespace ds4g
