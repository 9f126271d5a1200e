/*
 * ds4g.h -- C ABI of the GB300 (sm_103a) implementation of the ds4 per-token
 * layer step, its layer-major batched form for prefill, the lm_head and the
 * temperature / top-p sampler.
 *
 * Sources of the operations (cited by page title and section):
 *   [P3] "ds4.c 学习笔记 -- 端到端推理流程" (ds4-learning.pages.dev/inference-pipeline)
 *        阶段一  request_exceeds_context: a prompt with tokens >= context is rejected.
 *        阶段三  ds4_session_sync -> prefill_layer_major_cpu: reuse the cached prefix,
 *                then run every layer over the whole token batch before the next.
 *        阶段四  4.1 embed_token_f16; 4.2 the single-layer forward pseudocode
 *                (RMSNorm, low-rank Q/KV, RoPE, KV append, 64-head MQA over a
 *                128-token window, residual, RMSNorm, router over 256 experts,
 *                top-6, weighted experts plus a shared expert, residual),
 *                run once per layer per decoded token; 4.3 lm_head to 129280
 *                logits and sample_full_vocab (temperature, top-p, inverse CDF).
 *   [P1] "【#5】ds4.c を読み解く" (qiita.com/yoshiyakato) section 2: one worker owns
 *        the session and its KV; section 3: ds4_session_common_prefix and
 *        ds4_session_sync keep the KV of the common prefix and prefill the suffix.
 *
 * Conventions.
 *  - Every call returns an int status: DS4G_OK (0) or a negative DS4G_E* code;
 *    ds4g_sample returns the token id (>= 0) or a negative code.
 *  - Memory: the library never allocates device memory.  Weights are caller-owned
 *    device buffers that must outlive the model; a session lives inside one
 *    caller-owned device buffer of ds4g_session_bytes() bytes (KV cache, RoPE
 *    table, activations, logits).  Host-side bookkeeping (token history) is
 *    allocated with malloc and freed by the destroy calls.
 *  - Streams: every device operation of a session is issued on the stream
 *    given at ds4g_session_create, in call order.  Calls that return data to the
 *    host (ds4g_sample, ds4g_session_router) synchronise that stream.  A session
 *    of a model with the tensor-core prefill also owns one stream and two events
 *    of its own (created with the session, destroyed with it): each layer's shared
 *    expert GEMMs run on that stream, forked from and joined back into the
 *    session stream within the same ds4g_prefill call, so the ordering the caller
 *    sees is unchanged.
 *  - Threads: a session has one owner thread ([P1] section 2); the library is not
 *    thread-safe per session.  Different sessions may run on different threads.
 *  - Layouts are row-major [out][in] ("W x" is a dot product of each row with x).
 *    bf16 tensors hold raw bfloat16 bits; the embedding table is IEEE binary16.
 *  - Errors leave the session unchanged unless stated otherwise; DS4G_ECUDA
 *    reports a failed launch or CUDA call, after which the session is undefined.
 *  - The operators on device buffers (ds4g_sample*, ds4g_paged_*, ds4g_edit_logits,
 *    ds4g_probs, ds4g_verify_draft) run on the stream they are given, which belongs to the
 *    current device, and keep nothing between calls (but a time-out's report in the
 *    workspace of ds4g_paged_attention and ds4g_paged_attention8).  All but ds4g_sample* do not
 *    synchronise, that report's reading apart, and can be captured into a CUDA graph.  Calls that may overlap in
 *    time need workspaces of their own.
 */
#ifndef DS4G_H
#define DS4G_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum { DS4G_F32 = 0, DS4G_BF16 = 1 };

enum {
    DS4G_OK = 0,
    DS4G_EINVAL = -1,    /* bad argument, shape or handle */
    DS4G_ECONTEXT = -2,  /* the tokens would not fit: len + n >= n_ctx ([P3] 阶段一) */
    DS4G_ETOKEN = -3,    /* a token id outside [0, vocab) */
    DS4G_ECUDA = -4,     /* a CUDA call or kernel launch failed */
    DS4G_ETIMEOUT = -5,  /* a bounded device-side wait gave up */
    DS4G_ESIZE = -6,     /* a caller buffer is too small */
    DS4G_ENONFINITE = -7 /* a router score was NaN or infinite (the hidden state is not
                            finite); the step's results are invalid */
};

/* Model shape and formats.  The five synthetic workloads use hidden 4096,
 * 64 heads x 128, q_rank 1024, kv_rank 512, window 128, 256 experts top-6,
 * expert_inter 1024, vocab 129280 (and a tiny FP32 variant). */
typedef struct {
    int n_layers;
    int hidden;        /* H */
    int n_heads;       /* NH query heads; one shared K/V head (MQA) */
    int head_dim;      /* HD, even */
    int q_rank;        /* RQ: Q low-rank latent */
    int kv_rank;       /* RKV: KV low-rank latent */
    int window;        /* W: attention covers positions [pos-W+1, pos] */
    int n_experts;     /* E routed experts */
    int top_k;         /* K experts per token (<= 8) */
    int expert_inter;  /* I: SwiGLU inner width of every expert, shared one included */
    int vocab;         /* V */
    float rope_base;   /* RoPE base; pair (2i, 2i+1) turns by pos * base^(-2i/HD) */
    float rms_eps;     /* RMSNorm epsilon inside the square root */
    int weight_dtype;  /* DS4G_BF16 or DS4G_F32, all matrices including lm_head */
    int kv_dtype;      /* DS4G_BF16 or DS4G_F32, KV-cache storage */
    int prefill_chunk; /* tokens per layer-major pass (0: 4096); sets workspace size */
    int decode_kernel; /* DS4G_DECODE_AUTO: one persistent launch per decode step when
                          the device supports cooperative launch, else one kernel per
                          stage; DS4G_DECODE_STAGED forces one kernel per stage */
    int prefill_kernel; /* DS4G_PREFILL_AUTO: tensor-core GEMMs (tcgen05, BF16
                           activations times BF16 weights, FP32 accumulation and FP32
                           residual; the router's input as a BF16 hi/lo pair, so that its
                           scores carry about 16 significant bits of the normalised
                           residual) when the weights are BF16 and every weight piece is a
                           multiple of 128 rows (64 for expert gate/up) and every
                           reduction a multiple of 64, else SIMT GEMMs with FP32
                           activations; DS4G_PREFILL_HILO: the same tensor-core GEMMs
                           with every activation as a BF16 hi/lo pair (twice the tensor
                           work); DS4G_PREFILL_SIMT forces the SIMT GEMMs */
} ds4g_config;

enum { DS4G_DECODE_AUTO = 0, DS4G_DECODE_STAGED = 1 };
enum { DS4G_PREFILL_AUTO = 0, DS4G_PREFILL_SIMT = 1, DS4G_PREFILL_HILO = 2 };

/* One layer's weights (device pointers).  Gains are f32; matrices weight_dtype. */
typedef struct {
    const void *attn_norm; /* [H]          RMSNorm gain before attention */
    const void *wq_a;      /* [RQ][H]      Q down-projection */
    const void *wq_b;      /* [NH*HD][RQ]  Q up-projection, head-major rows */
    const void *wkv_a;     /* [RKV][H]     KV down-projection */
    const void *wk_b;      /* [HD][RKV]    K up-projection */
    const void *wv_b;      /* [HD][RKV]    V up-projection */
    const void *wo;        /* [H][NH*HD]   attention output projection */
    const void *ffn_norm;  /* [H]          RMSNorm gain before the MoE */
    const void *w_router;  /* [E][H]       router scores */
    const void *w_gate;    /* [E][I][H]    routed experts' gate projections */
    const void *w_up;      /* [E][I][H]    routed experts' up projections */
    const void *w_down;    /* [E][H][I]    routed experts' down projections */
    const void *ws_gate;   /* [I][H]       shared expert */
    const void *ws_up;     /* [I][H] */
    const void *ws_down;   /* [H][I] */
} ds4g_layer_weights;

typedef struct {
    const void *tok_embd;               /* f16 [V][H] */
    const void *lm_head;                /* [V][H] */
    const ds4g_layer_weights *layers;   /* host array of n_layers entries (copied) */
} ds4g_weights;

typedef struct ds4g_model ds4g_model;
typedef struct ds4g_session ds4g_session;

/* Validate the shape and record the weight pointers (copied; no device work
 * beyond setting kernel attributes).  DS4G_EINVAL if a dimension is unsupported:
 * H, RQ, RKV, I and HD must be multiples of 8, HD <= 256, W in [1, 1024],
 * top_k in [1, 8] and <= n_experts, n_experts <= 1024 and a multiple of 4, the
 * K/V window (2 W HD elements) and each activation vector must fit in 227 KB of
 * shared memory; or if a pointer is NULL or not 16-byte aligned. */
int ds4g_model_create(const ds4g_config *cfg, const ds4g_weights *w, ds4g_model **out);
void ds4g_model_destroy(ds4g_model *m);

/* Device bytes a session of context n_ctx needs (0 on a bad argument). */
size_t ds4g_session_bytes(const ds4g_config *cfg, int n_ctx);

/* Lay a session out in dev_mem (256-byte aligned, >= ds4g_session_bytes) and
 * fill its RoPE table on `cuda_stream` (a cudaStream_t; NULL = legacy stream).
 * The session starts empty (len 0).  DS4G_ESIZE if bytes is too small; DS4G_ECUDA
 * if its side stream or events cannot be created (tensor-core prefill). */
int ds4g_session_create(ds4g_model *m, int n_ctx, void *dev_mem, size_t bytes,
                        void *cuda_stream, ds4g_session **out);
void ds4g_session_destroy(ds4g_session *s);

/* [P3] 阶段三 / 阶段四: append n tokens (host array) at positions [len, len+n)
 * with layer-major prefill; afterwards every K/V of the context is cached and
 * the logits of the last token are at ds4g_session_logits.  n == 0 is a no-op.
 * DS4G_ECONTEXT if len + n >= n_ctx, DS4G_ETOKEN if a token is out of range. */
int ds4g_prefill(ds4g_session *s, const int32_t *tokens, int n);

/* [P3] 阶段四: one token through every layer (4.2, once per layer), then the
 * lm_head (4.3).  Same errors as ds4g_prefill with n = 1. */
int ds4g_decode_step(ds4g_session *s, int32_t token);

/* [P3] 阶段四 4.2 without 4.3: one token through every layer, no lm_head (for
 * callers that need the KV cache and the final hidden state but not the logits).
 * The final hidden state is at ds4g_session_hidden; the logits are not updated.
 * Same errors as ds4g_decode_step. */
int ds4g_decode_layers(ds4g_session *s, int32_t token);

/* ds4g_decode_layers with the final hidden state returned to the caller:
 * hidden_host (host memory, hidden floats) holds it when the call returns.  Pinned
 * (page-locked) memory is written by the persistent decode kernel itself through its
 * device view, and the kernel's last CTA signals completion through a pinned word of
 * the session (64 bytes of pinned host memory, allocated on first use and freed by
 * ds4g_session_destroy); the call returns on that signal, while the kernel may still
 * be exiting (later work on the session stream is ordered after it).  Other memory
 * gets a device-to-host copy and a stream synchronisation.  DS4G_ETIMEOUT if the
 * kernel gave up a wait (see ds4g_session_status).  One call per token for a host
 * loop that consumes the hidden state.  DS4G_EINVAL if
 * hidden_host is NULL; otherwise the errors of ds4g_decode_step (the session is
 * unchanged on DS4G_ETOKEN / DS4G_ECONTEXT). */
int ds4g_decode_layers_host(ds4g_session *s, int32_t token, float *hidden_host);

/* [P3] 阶段四 4.2 + 4.3 in one call: token through every layer and the lm_head
 * (as ds4g_decode_step), then the next token drawn from the logits (as
 * ds4g_sample, with its workspace, temperature, top_p and rng_state rules).
 * Returns the drawn token id (>= 0) or a negative DS4G_* code; the call
 * synchronises the session stream.  The one call per generated token of a
 * sampling loop. */
int32_t ds4g_decode_sample(ds4g_session *s, int32_t token, float temperature, float top_p,
                           uint64_t *rng_state, void *workspace, size_t workspace_bytes);

/* [P1] section 3 ds4_session_common_prefix: number of leading tokens shared by
 * the session's history and tokens[0..n). */
int ds4g_session_common_prefix(const ds4g_session *s, const int32_t *tokens, int n);

/* [P1] section 3 / [P3] 阶段三: keep the cached K/V of positions
 * [0, common_prefix); later positions become dead and are overwritten by the
 * next prefill.  0 <= common_prefix <= len, else DS4G_EINVAL; equal to len is a
 * no-op.  The logits are not recomputed. */
int ds4g_session_truncate(ds4g_session *s, int common_prefix);

/* [P1] section 3 ds4_session_sync / [P3] 阶段三: bring the session to the prompt
 * tokens[0..n) (host) in one call.  The cached K/V of the prompt's common prefix
 * with the history is kept, the rest is dropped, and the suffix is prefilled,
 * so that the session then holds exactly the prompt and the logits of its last
 * token.  The logits of a token are not kept once later tokens were processed,
 * so a prompt that the history already holds (whole, or as a prefix) runs its
 * last token again.  n == 0 empties the session.  *n_prefilled (may be NULL)
 * receives the number of tokens run through the layers.  Checked before the
 * session changes: DS4G_ECONTEXT if n >= n_ctx, DS4G_ETOKEN if a token is out of
 * range; then the errors of ds4g_prefill. */
int ds4g_session_sync(ds4g_session *s, const int32_t *tokens, int n, int *n_prefilled);

/* [P1] section 6 ds4_session_rewrite_from_common: rewrite the live checkpoint to
 * the prompt tokens[0..n) from a common prefix the caller found with
 * ds4g_session_common_prefix: positions [0, common) are kept and tokens[common..n)
 * are prefilled (when n > common; else the session is cut to n).  A prompt equal
 * to the history (common == n == len) changes nothing.  DS4G_EINVAL unless
 * 0 <= common <= ds4g_session_common_prefix(s, tokens, n); ECONTEXT and ETOKEN as
 * for ds4g_session_sync, checked before the session changes. */
int ds4g_session_rewrite_from_common(ds4g_session *s, const int32_t *tokens, int n, int common);

int ds4g_session_len(const ds4g_session *s);

/* Device pointer to the f32 [V] logits of the last processed token. */
const float *ds4g_session_logits(const ds4g_session *s);

/* Device pointer to the f32 [H] final hidden state (last layer's output) of the
 * last processed token. */
const float *ds4g_session_hidden(const ds4g_session *s);

/* Device pointers of layer `layer`'s K and V caches: [n_ctx][HD] of kv_dtype,
 * K stored after RoPE.  For tests and for restoring a saved cache. */
int ds4g_session_kv(ds4g_session *s, int layer, void **k, void **v);

/* Adopt K/V contents the caller wrote for positions [0, n) with the token
 * history tokens[0..n) (host): a restore of a saved cache.  DS4G_ECONTEXT if
 * n >= n_ctx. */
int ds4g_session_restore(ds4g_session *s, const int32_t *tokens, int n);

/* [P1] section 3 (steps 3-4: the disk KV cache, whose payload is restored before
 * only the suffix is prefilled): a checkpoint of a session's cached state, the
 * token history and the K/V rows of positions [0, len) of every layer, in a
 * caller-owned host buffer.  Layout (little-endian): a 64-byte header (magic
 * "DS4GKV01", format version, K/V element size, n_layers, head_dim, token count,
 * a digest of the configuration), the int32 tokens padded to 16 bytes, then per
 * layer the K rows and the V rows, [len][head_dim] each, as cached (K after RoPE).
 * The logits are not part of it: after a load, ds4g_session_sync with the prompt
 * runs the suffix (at least the last token) again. */
size_t ds4g_checkpoint_bytes(const ds4g_config *cfg, int n_tokens);
/* Write the checkpoint of s into buf (host memory of `bytes` bytes; pinned
 * memory copies faster).  Synchronises the session stream.  DS4G_ESIZE if bytes <
 * ds4g_checkpoint_bytes(cfg, len). */
int ds4g_session_save(ds4g_session *s, void *buf, size_t bytes);
/* Replace the state of s by a checkpoint written by ds4g_session_save for a model
 * of the same configuration: DS4G_EINVAL on a header or configuration mismatch,
 * DS4G_ESIZE if bytes is shorter than the checkpoint, DS4G_ECONTEXT if its length
 * is >= n_ctx, DS4G_ETOKEN if a token is out of range; the session is unchanged on
 * any of these.  If a copy to the device fails (DS4G_ECUDA), some layers' K/V rows
 * may already be overwritten, so the session is emptied (len 0).  Synchronises the
 * session stream. */
int ds4g_session_load(ds4g_session *s, const void *buf, size_t bytes);

/* Router decision of the last decoded token: ids (int32) and weights (f32) of
 * `layer`, top_k each, copied to host arrays (synchronises the stream). */
int ds4g_session_router(ds4g_session *s, int layer, int32_t *ids, float *weights);

/* Device pointer of one decode-step intermediate (the last layer's values of
 * the last ds4g_decode_step), for element-wise checks; NULL if unknown. */
enum {
    DS4G_DBG_X = 0,       /* f32 [H] residual after the step (layer output) */
    DS4G_DBG_CQKV = 1,    /* f32 [RQ+RKV] Q and KV latents */
    DS4G_DBG_Q = 2,       /* f32 [NH*HD] queries after RoPE */
    DS4G_DBG_ATTN = 3,    /* f32 [NH*HD] attention output, head-major */
    DS4G_DBG_XMID = 4,    /* f32 [H] residual after the attention half */
    DS4G_DBG_XN2 = 5,     /* f32 [H] normalised residual entering the MoE */
    DS4G_DBG_SCORES = 6,  /* f32 [E] router scores */
    DS4G_DBG_H = 7,       /* f32 [(K+1)*I] SwiGLU hidden, routed slots then shared */
    DS4G_DBG_HIDDEN = 8,  /* f32 [H] final hidden state (same as DS4G_DBG_X) */
    DS4G_DBG_PREFILL_X = 9, /* f32 [prefill_chunk][H] final hidden states of the last
                               prefill chunk (row t = t-th token of that chunk) */
    DS4G_DBG_STATUS = 10,   /* int32 raw device status word (0: no device-side error) */
    DS4G_DBG_PREFILL_LAYER_X = 11 /* f32 [L+1][H]: the last prefilled token's residual
                                     entering each layer, then its final hidden state */
};
const void *ds4g_session_debug(const ds4g_session *s, int which);

/* Record the residual stream at chosen positions, for teacher-forced checks of a
 * layer against a reference ([P3] 阶段四 4.2: each layer maps the residual x of a
 * position to the next layer's x).  positions: host array of n absolute session
 * positions (copied; 0 <= position < n_ctx; n <= 64).  buf: device memory owned by
 * the caller, n * (n_layers + 1) * hidden floats, which must outlive the setting.
 * Whenever a later ds4g_prefill, ds4g_decode_step or ds4g_decode_layers computes
 * positions[i], row i * (n_layers + 1) + l of buf receives the residual entering
 * layer l (row l = 0: the widened embedding), and row l = n_layers the final
 * hidden state.  n = 0 turns recording off.  DS4G_EINVAL on a bad argument; the
 * setting is then unchanged.  Recording adds device-to-device copies to a prefill
 * and one store per element to a decode step. */
int ds4g_session_set_probe(ds4g_session *s, const int32_t *positions, int n, float *buf);

/* Synchronise the session stream and report the first device-side error since the
 * last call: DS4G_ETIMEOUT (a bounded wait gave up) or DS4G_ENONFINITE (a router
 * score was not finite; the expert choice then falls back to the lowest unused
 * ids, so every access stays in bounds).  The step's results are then invalid.
 * The flag is cleared.  DS4G_ECUDA if the stream reports an error. */
int ds4g_session_status(ds4g_session *s);

/* Kernels this session has launched so far (all calls on it). */
uint64_t ds4g_session_launches(const ds4g_session *s);

/* Tracing: per-kernel timing.  While on, decode steps run one kernel per stage,
 * every kernel is bracketed by CUDA events on the session stream and the step
 * synchronises the stream at its end; a tensor-core prefill records an event after
 * every launch of each chunk, synchronises at the chunk's end and charges each
 * launch the time since the previous event (timing removes the overlap that
 * programmatic dependent launch gives consecutive kernels).  ds4g_session_timing
 * copies the accumulated milliseconds and launch counts of each kernel kind
 * (DS4G_K_*) into ms[0..n) and counts[0..n), then resets them. */
enum {
    DS4G_K_QKV_A = 0,      /* RMSNorm + Q/KV down-projections */
    DS4G_K_QKV_B = 1,      /* Q/K/V up-projections + RoPE + KV append */
    DS4G_K_ATTN = 2,       /* sliding-window MQA */
    DS4G_K_WO = 3,         /* output projection + residual */
    DS4G_K_ROUTER = 4,     /* RMSNorm + router + top-k */
    DS4G_K_EXPERT_GU = 5,  /* routed + shared gate/up with SwiGLU */
    DS4G_K_EXPERT_DOWN = 6,/* down projections + combine + residual */
    DS4G_K_LM_HEAD = 7,
    /* tensor-core prefill ([P3] 阶段三, layer-major) */
    DS4G_K_P_EMBED = 8,       /* embedding rows */
    DS4G_K_P_NORM = 9,        /* RMSNorm rows (the first layer's attention norm, every FFN norm) */
    DS4G_K_P_QKV_A = 10,      /* [W_qa; W_kva] GEMM */
    DS4G_K_P_Q_B = 11,        /* W_qb GEMM + RoPE */
    DS4G_K_P_KV_B = 12,       /* [W_kb; W_vb] GEMM + RoPE + K/V append */
    DS4G_K_P_ATTN = 13,       /* windowed attention */
    DS4G_K_P_WO = 14,         /* W_o GEMM + residual */
    DS4G_K_P_ROUTER = 15,     /* router GEMM */
    DS4G_K_P_TOPK = 16,       /* top-k + softmax of the selected scores */
    DS4G_K_P_GROUP = 17,      /* grouping of (token, slot) entries by expert */
    DS4G_K_P_GATE_UP = 18,    /* routed gate/up GEMM + SwiGLU */
    DS4G_K_P_SHARED_GU = 19,  /* shared expert gate/up GEMM + SwiGLU */
    DS4G_K_P_DOWN = 20,       /* routed down GEMM */
    DS4G_K_P_SHARED_DOWN = 21,/* shared expert down GEMM + residual */
    DS4G_K_P_COMBINE = 22,    /* slot-order combine + the next layer's RMSNorm */
    DS4G_K_COUNT = 23
};
int ds4g_session_set_timing(ds4g_session *s, int on);

/* Tracing of the single-launch decode step: when buf (device, caller-owned) is
 * not NULL, each later decode step writes the GPU global time (ns) at which every
 * CTA starts each stage: entry [e * n_cta + c] for event e = 7 * layer + stage
 * (stages: Q/KV down, up + RoPE + append, attention, output projection, router,
 * gate/up, down + combine), e = 7 * n_layers for the lm_head and 7 * n_layers + 1
 * for the end; n_cta is the number of SMs.  Events beyond bytes / (8 n_cta) are
 * dropped.  NULL turns tracing off. */
int ds4g_session_set_trace(ds4g_session *s, void *buf, size_t bytes);
int ds4g_session_timing(ds4g_session *s, double *ms, uint64_t *counts, int n);

/* Sampler workspace bytes for a vocabulary of n_vocab (device memory). */
size_t ds4g_sample_workspace_bytes(int n_vocab);

/* [P3] 阶段四 4.3 sample_full_vocab.  logits: device f32 [n_vocab].
 * temperature <= 0: argmax, lowest id on ties; rng_state untouched.
 * temperature > 0: z = logits / T, p = exp(z - max z); top-p keeps the most
 * probable tokens (ties to the lower id) until their sum reaches top_p of the
 * total (top_p >= 1 keeps all); one draw u = (xorshift64*(rng_state) >> 40) / 2^24
 * advances *rng_state (host, nonzero); the result is the first token, in
 * vocabulary order, at which the running sum of kept probabilities reaches
 * u * (their total).  Probabilities are summed exactly in 2^-40 fixed point, so
 * the result does not depend on the order of device reductions.
 * workspace: device, >= ds4g_sample_workspace_bytes(n_vocab) bytes, 256-byte
 * aligned.  Synchronises `cuda_stream`. */
int32_t ds4g_sample(const float *logits, int n_vocab, float temperature, float top_p,
                    uint64_t *rng_state, void *workspace, size_t workspace_bytes,
                    void *cuda_stream);

/* As ds4g_sample with the uniform draw given by the caller: u = u24 / 2^24,
 * u24 < 2^24 (else DS4G_EINVAL); no RNG state is used.  For callers that bring
 * their own random numbers. */
int32_t ds4g_sample_u(const float *logits, int n_vocab, float temperature, float top_p,
                      uint32_t u24, void *workspace, size_t workspace_bytes, void *cuda_stream);

/* [P3] 阶段四 sample_top_p_min_p (named there with top-p, without a definition):
 * ds4g_sample with a min-p filter as well.  Reading: of the top-p set, a token is
 * kept only if its probability is at least min_p times the largest probability;
 * min_p = 0 is ds4g_sample, min_p = 1 keeps the most probable token (and its exact
 * ties).  0 <= min_p <= 1, else DS4G_EINVAL.  Everything else as ds4g_sample. */
int32_t ds4g_sample_min_p(const float *logits, int n_vocab, float temperature, float top_p, float min_p,
                          uint64_t *rng_state, void *workspace, size_t workspace_bytes,
                          void *cuda_stream);
/* ds4g_sample_min_p with the uniform draw given by the caller, as ds4g_sample_u. */
int32_t ds4g_sample_u_min_p(const float *logits, int n_vocab, float temperature, float top_p, float min_p,
                            uint32_t u24, void *workspace, size_t workspace_bytes, void *cuda_stream);

/* Largest vocabulary ds4g_sample_static accepts. */
#define DS4G_SAMPLE_STATIC_MAX_VOCAB 262144

/* ds4g_sample without a caller workspace.  The pages have no counterpart: this is
 * a library convenience.  It is for callers that cannot allocate device memory
 * for a workspace: a host program that only holds a logits pointer produced by
 * another library (it owns no device allocator), or a decode loop that must not
 * call cudaMalloc between steps, because cudaMalloc can synchronise the device.
 * Its scratch is a fixed 16 KB array in the library's device image, which exists
 * once the module is loaded; the call allocates nothing.  n_vocab above
 * DS4G_SAMPLE_STATIC_MAX_VOCAB returns DS4G_ESIZE; other arguments and the result
 * are as for ds4g_sample.  Every call looks up the scratch's address on the
 * current device (cudaGetSymbolAddress, which allocates nothing), so a device reset
 * between calls is safe.  There is one scratch per device: calls that overlap in
 * time on one device (two host threads, or two streams whose calls are not
 * ordered) race on it and give undefined results.  The scratch keeps the last
 * call's contents; each call clears the part that must start at zero.
 * Synchronises `cuda_stream`. */
int32_t ds4g_sample_static(const float *logits, int n_vocab, float temperature, float top_p,
                           uint64_t *rng_state, void *cuda_stream);

/* ---------------------------------------------------------------- paged K/V cache
 *
 * Several sequences in one K/V cache ([P3] 阶段四 4.2 appends each token's K, after
 * RoPE, and V to the cache and attends over it; here the cache of many sequences is
 * cut into pages, so that they grow without moving).  Position p of a sequence lies
 * in the page its table names at p / page_size, slot p % page_size.  A session's own
 * cache (ds4g_session_kv) is the case of pages that follow one another. */

/* The cache of one layer.  Element d of head h of slot s of page g is at
 * k[g * page_stride + s * slot_stride + h * head_stride + d] (v alike); strides in
 * elements, each a multiple of 16 bytes, the pointers 16-byte aligned.  head_dim: a
 * multiple of 8, at most 256; at most 65536 heads. */
typedef struct {
    void *k, *v;
    int64_t page_stride, slot_stride, head_stride;
    int n_pages;
    int page_size;
    int n_kv_heads;
    int head_dim;
    int dtype; /* DS4G_BF16 or DS4G_F32 */
} ds4g_paged_kv;

/* The sequences of a call (device arrays).  Sequence b has length[b] tokens, its
 * newest ones, the call's new tokens, among them: n_b = start[b + 1] - start[b] of
 * them (at most max_new), rows start[b] .. of the call's token arrays, at positions
 * length[b] - n_b .. length[b] - 1.  start NULL: one token each, row b.  A table
 * entry outside [0, n_pages) is a page that is not there (nothing is stored to it and
 * its keys are left out), and so is everything at or past width * page_size.  Rows at or
 * past start[n_seqs] are left as they are.  start[0] is 0, start does not fall, and
 * start[n_seqs] <= n_tokens. */
typedef struct {
    const int32_t *table;  /* [n_seqs][table_stride], width entries used */
    const int32_t *length; /* [n_seqs] */
    const int32_t *start;  /* [n_seqs + 1] or NULL */
    int n_seqs;
    int n_tokens; /* rows of the token arrays; n_seqs when start is NULL */
    int max_new;  /* most new tokens of one sequence: 1 when start is NULL */
    int width;
    int table_stride;
} ds4g_paged_batch;

/* Rotation table: cs[(p * rot_dim / 2 + i) * 2] = cos and + 1 = sin of the angle of pair
 * (2i, 2i+1) at position p < n_pos (device, f32, 16-byte aligned).  The first rot_dim
 * dims of a head turn (even, at most head_dim); the rest pass through. */
typedef struct {
    const float *cs;
    int n_pos;
    int rot_dim;
} ds4g_rope;

/* Fill a rotation table: angle p * base^(-2i/rot_dim), computed in FP64 and stored
 * as FP32 (as the sessions' own tables).  cs: device, n_pos * rot_dim floats. */
int ds4g_rope_fill(float *cs, int n_pos, int rot_dim, float base, void *cuda_stream);

/* Store the new tokens' K and V rows into their pages, the keys rotated by their
 * positions on the way, rounded once (to nearest even) to the cache's type; with q
 * also rotate the queries into q_out (the same type; q_out == q is allowed with equal
 * strides, other overlaps are not).  k, v: [n_tokens][n_kv_heads][head_dim], q:
 * [n_tokens][n_heads][head_dim], each with its own token stride in elements (a
 * multiple of 16 bytes; heads and dims adjacent); dtype: their type, DS4G_BF16 or
 * DS4G_F32.  rope NULL: no rotation.  q NULL: keys and values only.  A token whose
 * position is outside the table or its page not there stores no K and V; one before
 * position 0, or at or past n_pos, stores none either and leaves its q_out row as it
 * was.  Two tokens of one
 * call must not share a slot.  One launch. */
int ds4g_paged_append(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, const ds4g_rope *rope, const void *q, int64_t q_stride,
                      void *q_out, int64_t q_out_stride, int n_heads, int dtype, void *cuda_stream);

/* Workspace bytes of ds4g_paged_attention (host arithmetic on the sizes alone); 0 on a
 * bad argument. */
size_t ds4g_paged_attention_workspace_bytes(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, int n_heads);

/* Attention of every sequence's new tokens over its cached positions (the new tokens'
 * rows already appended): token at position p attends to the positions max(0, p -
 * window + 1) .. p (window <= 0: 0 .. p), out = sum_j softmax_j(scale q . k_j) v_j, query
 * heads h * n_heads / n_kv_heads .. sharing K/V head h.  0 < scale <= 1e38, or 0: 1 / sqrt(head_dim).
 * A masked or missing key adds nothing, whatever its K and V hold; what is not finite in the V
 * of a key that a token sees leaves that place of its result infinite or NaN, however small
 * the key's weight.  A token without any key gets zeros.  q, out: [n_tokens][n_heads][head_dim] with token strides in elements
 * (multiples of 16 bytes, 16-byte aligned); dtype: their type.  q and out must not
 * overlap.  max_new <= 128.
 * BF16 queries over a BF16 cache with head_dim 64 or 128, pages of a multiple of 8 slots, heads
 * adjacent within a slot or whole heads within a page, and at most 128 query heads per K/V
 * head run on the tensor cores, the probabilities
 * rounded to BF16 for the product with V (FP32 sums); every other case runs in FP32.
 * The work is cut over the keys of all sequences by their lengths on the device, and
 * parts of one sequence are joined by a second launch in a fixed order: the same call gives the
 * same bits, but a sequence's last bits may depend on the others of its call.
 * workspace: device, >= ds4g_paged_attention_workspace_bytes, 256-byte aligned. */
int ds4g_paged_attention(const ds4g_paged_kv *kv, const ds4g_paged_batch *batch, const void *q, int64_t q_stride,
                         void *out, int64_t out_stride, int n_heads, int dtype, float scale, int window,
                         void *workspace, size_t workspace_bytes, void *cuda_stream);

/* The cache of one layer in 8 bits: element d of head h of slot s of page g is
 * code(k[g * page_stride + s * slot_stride + h * head_stride + d]) * k_scale[g * scale_stride +
 * (s / block) * n_kv_heads + h] (v alike), the codes E4M3 (a sign, 4 bits of exponent, 3 behind the first;
 * to 448, no infinities, NaN 0x7f and 0xff).  Strides in elements, those of the codes multiples of
 * 16, their pointers 16-byte aligned.  block: slots that share a scale, a divisor of page_size.
 * Scales lie in [2^-64, 2^64] (the attention takes others as the nearer bound, NaN as the lower). */
typedef struct {
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, slot_stride, head_stride;
    int64_t scale_stride;
    int n_pages;
    int page_size;
    int n_kv_heads;
    int head_dim;
    int block;
} ds4g_paged_kv8;

/* ds4g_paged_append to a cache in 8 bits; what it says of tokens, positions, pages and queries holds
 * here.  Where a block's first slot is among a sequence's new tokens its scale becomes the least
 * power of two s with |x| <= 448 s for the block's new rows x of that head (as rotated, in FP32; s
 * 2^-64 at least, 2^64 at most).  Otherwise the block keeps its scale, or takes the s that its new rows
 * ask for where that is larger; the rows that it holds already are then rounded again, which is exact
 * but for values below 2^-6 of the new scale.  Codes are rounded to nearest even from x / s; values above
 * 448 2^64 become 448, infinities and NaN become NaN and count for no scale.  Rows that are taken back (a length made
 * shorter, as after rejected drafts) leave their scale in the block until a call begins it again: the rows that it held stay
 * rounded to it, off by 2^-10 of that scale at most beside their own rounding, so that decoding with drafts is not bit-equal
 * to decoding without.  Two sequences of one call must not store into the same block.  One launch. */
int ds4g_paged_append8(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, const void *k, int64_t k_stride,
                       const void *v, int64_t v_stride, const ds4g_rope *rope, const void *q, int64_t q_stride,
                       void *q_out, int64_t q_out_stride, int n_heads, int dtype, void *cuda_stream);

/* ds4g_paged_attention over a cache in 8 bits: the same call, workspace rules and status, K and V
 * being the values that codes and scales stand for.  BF16 queries with head_dim 64 or 128, pages of a
 * multiple of 8 slots run on the tensor cores: the queries as pairs of E4M3 values (exact down to 2^-14 of
 * the row's largest, off by 2^-22 of it at most below), the probabilities times the V scales
 * as pairs of E4M3 values (up to 32 rows, new tokens times query heads, a K/V head: 2^-9 of each) or as FP16 (2^-11),
 * of what is very small 2^-32 of the largest; their sums in FP32 before that rounding; every other case runs in FP32.
 * scale times a K scale times a query's largest value has to stay below 2^126: scores beyond FP32 are not
 * infinities but NaN. */
size_t ds4g_paged_attention8_workspace_bytes(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, int n_heads);
int ds4g_paged_attention8(const ds4g_paged_kv8 *kv, const ds4g_paged_batch *batch, const void *q, int64_t q_stride,
                          void *out, int64_t out_stride, int n_heads, int dtype, float scale, int window,
                          void *workspace, size_t workspace_bytes, void *cuda_stream);

/* Pages that no sequence holds: a stack free_pages[0 .. n_free[0]) in an array of `capacity` (device). */
typedef struct {
    int32_t *free_pages;
    int32_t *n_free; /* [1] */
    int capacity;
    int page_size;
} ds4g_page_pool;

/* Bring every sequence's length to want[b] (below 0: 0) and its table with it.  First the pages that
 * shorter sequences no longer need go back to the pool, in the order of sequences and of their
 * tables, the first of them on top (what does not fit `capacity` is lost); their table entries become -1.
 * Then longer ones take theirs from the top of what is in the pool then, in the same order, so that giving back what the
 * last call took restores the pool.  A sequence whose pages exceed what is left after those that
 * all sequences before it asked for, whose new tokens exceed max_tokens behind theirs, or whose want exceeds
 * width * page_size is left as it was.  start [n_seqs + 1]: the new tokens of
 * the sequences one behind the other, as ds4g_paged_batch takes them (none where a sequence
 * became shorter).  slots, where not NULL, [max_tokens]: page * page_size + slot of each new token;
 * entries behind the last one stay as they are.  table [n_seqs][table_stride], length, start, slots and the pool are
 * device memory, read and written on the device: the pages of [0, ceil(length[b] / page_size)) of
 * a table are its sequence's (all of them go back to the pool in turn, also an entry that is no page).  n_seqs <=
 * 65536 (DS4G_ESIZE); want may not be length.  One launch. */
int ds4g_paged_resize(const ds4g_page_pool *pool, int32_t *table, int width, int table_stride, int32_t *length,
                      const int32_t *want, int n_seqs, int32_t *start, int64_t *slots, int max_tokens,
                      void *cuda_stream);

/* Synchronise the stream and report whether a bounded device-side wait gave up in any
 * ds4g_paged_attention or ds4g_paged_attention8 on this workspace since the last time it was reported:
 * DS4G_ETIMEOUT (the outputs of the calls since then are invalid; the report is cleared) or
 * DS4G_OK, also where there was no call or none with tokens. */
int ds4g_paged_attention_status(void *workspace, void *cuda_stream);

/* ---------------------------------------------------------------- drafted tokens */

/* Edits of rows of logits (device memory; each part may be NULL).  History: ids [n_rows]
 * [max_history] with a row stride, the first n_history[row] of a row (NULL: all), of them the
 * first n_prompt[row] the prompt's (NULL: none), the others generated; ids outside the vocabulary count for
 * nothing.  repetition, frequency, presence: [n_rows] (NULL: 1, 0, 0); repetition > 0; max_history < 2^30.  Biases:
 * ids and values [n_rows][max_bias] with a row stride, the first n_bias[row] (NULL: all); max_bias <= 1024.
 * allowed: bit i % 32 of word i / 32 of a row, rows allowed_stride words apart (0: the same for all). */
typedef struct {
    const int32_t *history, *n_history, *n_prompt;
    int64_t history_stride;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_ids, *n_bias;
    const float *bias;
    int64_t bias_stride;
    const uint32_t *allowed;
    int64_t allowed_stride;
    int max_history;
    int max_bias;
} ds4g_logit_edits;

/* Edit rows of logits before ds4g_probs or ds4g_sample ([P3] 阶段四 4.3).  For id i, in FP32 and in this
 * order: where i is in the row's history z <- z > 0 ? z / repetition : z * repetition (the quotient rounded once, off
 * by half a unit of its last place and 2^-20 of that at most, for repetition in [2^-60, 2^60] and quotients above
 * 2^-100; else a product with the rounded reciprocal); where it is c > 0 times in the generated part z <- z -
 * (frequency * c + presence); z <- z + the sum of the row's biases of i (in FP64, rounded once); where i is not allowed z <- -inf, whatever it was.  logits, out: device f32
 * [n_rows][n_vocab] with row strides in elements; out == logits is allowed with equal strides.
 * n_vocab <= 1048576 (DS4G_ESIZE).  One launch. */
int ds4g_edit_logits(const float *logits, int64_t logits_stride, int n_rows, int n_vocab, const ds4g_logit_edits *edits,
                     float *out, int64_t out_stride, void *cuda_stream);

/* Probabilities that ds4g_sample draws from (without top-p), one row of logits each:
 * p = softmax(logits / temperature); temperature <= 0: 1 at the largest logit (the lowest
 * id on ties), 0 elsewhere.  A NaN logit counts as -inf; if the largest is +inf, the ids
 * that have it share the whole; a row of -inf alone gives zeros.  logits, probs: device
 * f32 [n_rows][n_vocab] with row strides in elements; probs == logits is allowed with
 * equal strides.  n_vocab <= 1048576 (DS4G_ESIZE).  One launch. */
int ds4g_probs(const float *logits, int64_t logits_stride, int n_rows, int n_vocab, float temperature, float *probs,
               int64_t probs_stride, void *cuda_stream);

/* Verify drafted tokens ([P3] 阶段四 4.3 draws one token; here a draft's tokens are kept
 * while the target would have drawn them, so that the output is distributed as the
 * target's own draws).  For sequence b with n = n_drafts[b] drafts (NULL: max_drafts;
 * clamped to [0, max_drafts]): draft i is accepted while u_i * q_i(d_i) < p_i(d_i), u_i =
 * u24[b][i] / 2^24.  The token after the k accepted ones is drawn with the last number, u =
 * u24[b][max_drafts] / 2^24 (one that decided on a draft would not be independent of it):
 * from the weights max(p_k - q_k, 0) if draft k was rejected (p_k where these are all zero),
 * from p_n if k = n.  As in ds4g_sample the weights are rounded to 2^-40 and summed exactly: the
 * first token, in vocabulary order, at which the running sum reaches max(1, ceil(u *
 * total)).  q NULL: drafts without probabilities (each draft's own probability is 1: it is
 * accepted while u_i < p_i(d_i), and its weight is 0 when it was rejected).
 * p: device f32 [n_seqs][max_drafts + 1][n_vocab], q: [n_seqs][max_drafts][n_vocab], with
 * strides of a sequence and of a position in elements; a value below 0 or NaN counts as 0,
 * one above 1 as 1.  drafts: int32 [n_seqs][max_drafts] (an id outside the vocabulary is
 * rejected); u24: uint32 [n_seqs][max_drafts + 1] (the low 24 bits).
 * accepted: int32 [n_seqs], k; tokens: int32 [n_seqs][max_drafts + 1]: the accepted
 * drafts, the drawn token (-1 if p_k has no weight), then -1.  max_drafts in [0, 64];
 * n_vocab <= 1048576 (DS4G_ESIZE).  The outputs overlap no input.  One launch. */
int ds4g_verify_draft(const float *p, int64_t p_seq_stride, int64_t p_stride, const float *q, int64_t q_seq_stride,
                      int64_t q_stride, const int32_t *drafts, const int32_t *n_drafts, const uint32_t *u24,
                      int n_seqs, int max_drafts, int n_vocab, int32_t *accepted, int32_t *tokens,
                      void *cuda_stream);

const char *ds4g_strerror(int code);

#ifdef __cplusplus
}
#endif
#endif /* DS4G_H */
