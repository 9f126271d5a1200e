// Edits of logits before a token is drawn from them (the draw of page "ds4.c 学习笔记 --
// 端到端推理流程", 阶段四 4.3): for token i of a row, with `seen` = i is in the row's history and
// c = how often it is in the part of it that was generated,
//   z <- z / r if z > 0, else z r           where seen (repetition penalty r)
//   z <- z - (f c + p [c > 0])              (frequency and presence penalties f, p)
//   z <- z + the sum of the row's biases of i
//   z <- -inf                               where the row's mask has a 0 for i.
//
// A CTA takes a slice of a row: a word a token in shared memory, in which every id of the history
// that lies in the slice is counted (bit 31: seen; whole numbers, so that the order of the
// atomics does not matter), then one pass over the slice's logits.  Biases follow: a warp adds up all entries of an
// id in FP64, in their order.
// Bound: bytes (a logit read and written once, a bit of the mask), latency at one row.
#include "paged.h"

namespace ds4g {

static constexpr int kEdThreads = 256;
static constexpr int kEdHold = 32;                          // logits of a thread
static constexpr int kEdSlice = kEdThreads * kEdHold;       // tokens of a CTA at most
static constexpr int kEdBatch = 8;                          // ids of a thread in flight

__global__ void __launch_bounds__(kEdThreads, 4) k_edit(const __grid_constant__ EditArgs a, int slice, int slices)
{
    extern __shared__ __align__(16) uint32_t s_count[];
    __shared__ int s_bias[kEditMaxBias];
    const int tid = threadIdx.x, lane = tid & 31;
    const int row = blockIdx.x / slices, v0 = (blockIdx.x - row * slices) * slice, n = max(min(slice, a.n - v0), 0);
    pdl_wait();
    pdl_trigger();
    const float *in = a.in + row * a.in_stride + v0;
    float *out = a.out + row * a.out_stride + v0;
    // the logits and the mask's words (lane k: of the warp's k-th 32 tokens), on their way while the history is counted
    float z[kEdHold];
#pragma unroll
    for (int k = 0; k < kEdHold; ++k) {
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
    const int *ids = a.history + row * a.history_stride, *bias_ids = a.bias_ids + row * a.bias_stride;
    for (int i = tid; i < biases; i += kEdThreads) s_bias[i] = bias_ids[i];
    if (hist) {
        for (int i = tid * 4; i < slice; i += kEdThreads * 4) *reinterpret_cast<uint4 *>(s_count + i) = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
#pragma unroll 1
        for (int i0 = tid; i0 < hist; i0 += kEdBatch * kEdThreads) {
            int id[kEdBatch];
#pragma unroll
            for (int k = 0; k < kEdBatch; ++k) id[k] = i0 + k * kEdThreads < hist ? ids[i0 + k * kEdThreads] : -1;
#pragma unroll
            for (int k = 0; k < kEdBatch; ++k) {
                const unsigned t = (unsigned)id[k] - (unsigned)v0;
                if (id[k] < 0 || t >= (unsigned)n) continue;
                if (i0 + k * kEdThreads < prompt) atomicOr(&s_count[t], 0x80000000u);
                else atomicAdd(&s_count[t], 1u);
            }
        }
    }
    __syncthreads();
    const float r = a.repetition ? a.repetition[row] : 1.f, f = a.frequency ? a.frequency[row] : 0.f,
                p = a.presence ? a.presence[row] : 0.f;
#pragma unroll
    for (int k = 0; k < kEdHold; ++k) {
        const int i = k * kEdThreads + tid;
        const uint32_t w = hist && i < n ? s_count[i] : 0u, allowed = __shfl_sync(0xffffffffu, words, k);
        if (w) {
            z[k] = z[k] > 0.f ? __fdiv_rn(z[k], r) : __fmul_rn(z[k], r);
            const uint32_t c = w & 0x7fffffffu;
            if (c) z[k] = __fsub_rn(z[k], __fadd_rn(__fmul_rn(f, (float)c), p));
        }
        if (i < n) out[i] = allowed >> lane & 1u ? z[k] : -INFINITY;
    }
    if (!biases) return;
    __syncthreads();
    // a warp an entry of the slice, if no entry before it has its id
    for (int k = tid >> 5; k < biases; k += kEdThreads / 32) {
        const int id = s_bias[k];
        if (id < v0 || id >= v0 + n) continue;
        bool first = true;
        double sum = 0.0;
        for (int j0 = 0; first && j0 < biases; j0 += 32) {
            const int j = j0 + lane;
            uint32_t same = __ballot_sync(0xffffffffu, j < biases && s_bias[min(j, biases - 1)] == id);
            if (j0 <= k) first = (same & (k - j0 < 32 ? (1u << (k - j0)) - 1u : 0xffffffffu)) == 0u;
            for (; first && same; same &= same - 1) sum += (double)a.bias[row * a.bias_stride + j0 + __ffs(same) - 1];
        }
        if (lane == 0 && first && (!a.allowed || (a.allowed[row * a.allowed_stride + (id >> 5)] >> (id & 31) & 1u)))
            out[id - v0] += (float)sum;
    }
}

cudaError_t edit_rows(const EditArgs &a, cudaStream_t st, int nsm)
{
    // slices of a row: as many as give every SM two CTAs, of 1024 tokens or more
    int slices = (a.n + kEdSlice - 1) / kEdSlice;
    while ((long long)slices * a.rows < 2 * nsm && a.n / (2 * slices) >= 1024) slices *= 2;
    const int slice = ((a.n + slices - 1) / slices + 31) & ~31;
    const size_t smem = a.history ? (size_t)slice * 4 : 0;
    static PerDevice once;
    cudaError_t e = allow_once(once, k_edit, (size_t)kEdSlice * 4);
    if (e) return e;
    return launch_pdl(k_edit, dim3((unsigned)slices * a.rows), dim3(kEdThreads), smem, st, a, slice, slices);
}

}  // namespace ds4g
