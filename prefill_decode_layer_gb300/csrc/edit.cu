// Edits of logits before a token is drawn from them (the draw of page "ds4.c 学习笔记 --
// 端到端推理流程", 阶段四 4.3): for token i of a row, with `seen` = i is in the row's history and
// c = how often it is in the part of it that was generated,
//   z <- z / r if z > 0, else z r           where seen (repetition penalty r)
//   z <- z - (f c + p [c > 0])              (frequency and presence penalties f, p)
//   z <- z + the sum of the row's biases of i
//   z <- -inf                               where the row's mask has a 0 for i.
//
// A CTA takes a slice of a row, up to 32 logits a thread, which are on their way to registers while it looks through
// the row's history: a word a token in shared memory says whether the token was seen (bit 31) or has a bias (bit
// 30) and how often it was generated (whole numbers, so that the order of the atomics does not matter).  A warp
// adds up all entries of a biased token in FP64, in their order, for the token's thread to find.
// Bound: bytes (a logit read and written once, a bit of the mask), latency at one row (3.1 us).  Measured: 256 rows
// of 129280, 265 MB: 43 us without histories (0.92 of the copy); with histories of 2048 to 8192 ids 66 us, with 100
// biases as well 72: four CTAs an SM, whose chains of loads, counts and stores then leave the pipe idle.  (Eight
// ids in flight for four 66 us for 73; a cluster of eight CTAs that shares the history and counts in each other's
// shared memory 76; one CTA an SM with the next item's loads in registers 99.)
#include "paged.h"
#include "sm100.cuh"

namespace ds4g {

static constexpr int kEdThreads = 256;
static constexpr int kEdHold = 32, kEdHoldFew = 8;          // logits of a thread at most, and in short slices
static constexpr int kEdBatch = 8;                          // ids of a thread in flight
static constexpr uint32_t kEdSeen = 0x80000000u, kEdBias = 0x40000000u;

// A word of global memory to shared memory, complete after cp.async.wait_all.
__device__ __forceinline__ void copy_word(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int HOLD>
__global__ void __launch_bounds__(kEdThreads, 4) k_edit(const __grid_constant__ EditArgs a, int slice, int slices)
{
    extern __shared__ __align__(16) uint32_t s_word[];      // of the slice's tokens
    __shared__ int s_bias_id[kEditMaxBias];
    __shared__ float s_bias[kEditMaxBias];
    __shared__ int s_found[kEditMaxBias], s_n_found;        // the slice's biased tokens
    __shared__ float s_sum[kEditMaxBias];
    const int tid = threadIdx.x, lane = tid & 31;
    const int row = blockIdx.x / slices, v0 = (blockIdx.x - row * slices) * slice, n = max(min(slice, a.n - v0), 0);
    pdl_wait();
    pdl_trigger();
    const float *in = a.in + row * a.in_stride + v0;
    float *out = a.out + row * a.out_stride + v0;
    // the first ids of the history and the biases (whether they count is known later), then the logits and the
    // mask's words (lane k: of the warp's k-th 32 tokens): all on their way while the history is counted
    const int *ids = a.history + row * a.history_stride, *bias_ids = a.bias_ids + row * a.bias_stride;
    int id[kEdBatch];
    auto fetch = [&](int i0, int end) {
#pragma unroll
        for (int k = 0; k < kEdBatch; ++k) {
            const int i = i0 + k * kEdThreads;
            id[k] = i < end ? ids[i] : -1;
        }
    };
    int i0 = tid;
    if (a.history) fetch(i0, a.max_history);
    if (a.bias_ids)
        for (int i = tid; i < a.max_bias; i += kEdThreads) {
            copy_word(&s_bias_id[i], bias_ids + i);
            copy_word(&s_bias[i], a.bias + row * a.bias_stride + i);
        }
    float z[HOLD];
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int i = k * kEdThreads + tid;
        z[k] = i < n ? in[i] : 0.f;
    }
    uint32_t words = 0xffffffffu;
    if (a.allowed) {
        const int i = lane * kEdThreads + (tid & ~31);
        words = i < n ? a.allowed[row * a.allowed_stride + ((v0 + i) >> 5)] : 0u;
    }
    const int hist = a.history ? min(max(a.n_history ? a.n_history[row] : a.max_history, 0), a.max_history) : 0;
    const int prompt = hist && a.n_prompt ? min(max(a.n_prompt[row], 0), hist) : 0;
    const int biases = a.bias_ids ? min(max(a.n_bias ? a.n_bias[row] : a.max_bias, 0), a.max_bias) : 0;
    const float r = a.repetition ? a.repetition[row] : 1.f, f = a.frequency ? a.frequency[row] : 0.f,
                p = a.presence ? a.presence[row] : 0.f;
    // 1 / r in two parts, its rounded value and what that leaves: z / r = z inv + z inv_low is 2^-47 off before its one
    // rounding (256 rows: 73 us; z inv alone 71.5, divisions 81)
    const float inv = __frcp_rn(r), inv_low = r >= 0x1p-60f && r <= 0x1p60f ? __fmul_rn(__fmaf_rn(-r, inv, 1.f), inv) : 0.f;
    const bool counts = hist || biases;
    asm volatile("cp.async.wait_all;" ::: "memory");   // (also where none of them counts)
    if (counts) {
        for (int i = tid * 4; i < slice; i += kEdThreads * 4) *reinterpret_cast<uint4 *>(s_word + i) = make_uint4(0u, 0u, 0u, 0u);
        if (tid == 0) s_n_found = 0;
        __syncthreads();
#pragma unroll 1
        for (; i0 - tid < hist; fetch(i0, hist)) {
#pragma unroll
            for (int k = 0; k < kEdBatch; ++k) {
                const unsigned t = (unsigned)id[k] - (unsigned)v0;
                const int i = i0 + k * kEdThreads;
                if (i >= hist || id[k] < 0 || t >= (unsigned)n) continue;
                if (i >= prompt) atomicAdd(&s_word[t], 1u);
                else atomicOr(&s_word[t], kEdSeen);
            }
            i0 += kEdBatch * kEdThreads;
        }
        // a warp an entry of the slice, if no entry before it has its id
        for (int k = tid >> 5; k < biases; k += kEdThreads / 32) {
            const int token = s_bias_id[k];
            if (token < v0 || token >= v0 + n) continue;
            bool first = true;
            double sum = 0.0;
            for (int j0 = 0; first && j0 < biases; j0 += 32) {
                const int j = j0 + lane;
                uint32_t same = __ballot_sync(0xffffffffu, j < biases && s_bias_id[min(j, biases - 1)] == token);
                if (j0 <= k) first = (same & (k - j0 < 32 ? (1u << (k - j0)) - 1u : 0xffffffffu)) == 0u;
                for (; first && same; same &= same - 1) sum += (double)s_bias[j0 + __ffs(same) - 1];
            }
            if (lane == 0 && first) {
                const int at = atomicAdd(&s_n_found, 1);
                s_found[at] = token - v0;
                s_sum[at] = (float)sum;
                atomicOr(&s_word[token - v0], kEdBias);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int i = k * kEdThreads + tid;
        const uint32_t w = counts && i < n ? s_word[i] : 0u, allowed = __shfl_sync(0xffffffffu, words, k);
        // (without branches: of 32 tokens some are in the history as a rule)
        const float c = (float)(w & ~(kEdSeen | kEdBias));
        const float low = fmaxf(__fmul_rn(z[k], inv_low), -3.402823466e38f);   // (an infinite logit stays one)
        const float turned = z[k] > 0.f ? __fmaf_rn(z[k], inv, low) : __fmul_rn(z[k], r);
        z[k] = w & ~kEdBias ? turned : z[k];
        z[k] = c > 0.f ? __fsub_rn(z[k], __fadd_rn(__fmul_rn(f, c), p)) : z[k];
        if (w & kEdBias) {
            int j = 0;
            while (s_found[j] != i) ++j;   // (it is there)
            z[k] += s_sum[j];
        }
        if (i < n) out[i] = allowed >> lane & 1u ? z[k] : -INFINITY;
    }
}

cudaError_t edit_rows(const EditArgs &a, cudaStream_t st, int nsm)
{
    // slices of a row: as many as give every SM two CTAs, of 1024 tokens or more
    constexpr int most = kEdThreads * kEdHold, few = kEdThreads * kEdHoldFew;
    int slices = (a.n + most - 1) / most;
    while ((long long)slices * a.rows < 2 * nsm && a.n / (2 * slices) >= 1024) slices *= 2;
    const int slice = ((a.n + slices - 1) / slices + 31) & ~31;
    const size_t smem = a.history || a.bias_ids ? (size_t)slice * 4 : 0;
    const dim3 grid((unsigned)slices * a.rows), block(kEdThreads);
    if (slice <= few) return launch_pdl(k_edit<kEdHoldFew>, grid, block, smem, st, a, slice, slices);
    static PerDevice once;   // (with the static arrays more than 48 KB)
    const cudaError_t e = allow_once(once, k_edit<kEdHold>, 64 * 1024);
    if (e) return e;
    return launch_pdl(k_edit<kEdHold>, grid, block, smem, st, a, slice, slices);
}

}  // namespace ds4g
