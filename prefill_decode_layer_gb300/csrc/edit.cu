// Edits of logits before a token is drawn from them (the draw of page "ds4.c 学习笔记 --
// 端到端推理流程", 阶段四 4.3): for token i of a row, with `seen` = i is in the row's history and
// c = how often it is in the part of it that was generated,
//   z <- z / r if z > 0, else z r           where seen (repetition penalty r)
//   z <- z - (f c + p [c > 0])              (frequency and presence penalties f, p)
//   z <- z + the sum of the row's biases of i
//   z <- -inf                               where the row's mask has a 0 for i.
//
// A CTA takes a slice of a row, up to 32 logits a thread, which are on their way to registers while it looks through
// the row's history: a word a token in shared memory says whether the token was seen (bit 31) and how often it was
// generated (whole numbers, so that the order of the atomics does not matter).  The word of a biased token (bit 30)
// holds the place of its first entry instead, where its count and its sum of biases lie: the entries set it before the
// history is counted, and the token's thread finds both in one look.  A token of several entries has them added up by a
// thread in FP64, in their order.
// Bound: bytes (a logit read and written once, a bit of the mask), latency at one row (2.9 us).  Measured: 256 rows
// of 129280, 265 MB: 44 us without histories (0.89 of the copy); with histories of 2048 to 8192 ids 71 us, with 100
// biases as well 75: four CTAs an SM, whose chains of loads, counts and stores then leave the pipe idle.  1024 biases
// 53 us, side by side or not (with a search for each biased token's entry 480 to 810); each further entry of one token
// 0.1 us of its thread.  (Four ids in flight, not eight: 7 us more; a cluster of eight CTAs that shares the history and
// counts in each other's shared memory 10 more than that form; one CTA an SM with the next item's loads in registers 33.)
#include <type_traits>

#include "paged.h"
#include "sm100.cuh"

namespace ds4g {

static constexpr int kEdThreads = 256;
static constexpr int kEdHold = 32, kEdHoldFew = 8;          // logits of a thread at most, and in short slices
static constexpr int kEdBatch = 8;                          // ids of a thread in flight
static constexpr uint32_t kEdSeen = 0x80000000u, kEdBias = 0x40000000u, kEdTwice = 0x40000000u;   // (of a place's count)
static_assert((kEditMaxBias & (kEditMaxBias - 1)) == 0, "a word's low bits name an entry");

// A word of global memory to shared memory, complete after cp.async.wait_all.
__device__ __forceinline__ void copy_word(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

template <int HOLD>
__global__ void __launch_bounds__(kEdThreads, 4) k_edit(const __grid_constant__ EditArgs a, int slice, int slices)
{
    extern __shared__ __align__(16) uint32_t s_word[];      // of the slice's tokens
    __shared__ __align__(16) int s_bias_id[kEditMaxBias];
    __shared__ float s_bias[kEditMaxBias];
    __shared__ uint32_t s_count[kEditMaxBias];              // at the place of a biased token's first entry
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
        for (int k = tid; k < biases; k += kEdThreads) s_count[k] = 0u;
        __syncthreads();
        auto slot = [&](int k) { return (unsigned)s_bias_id[k] - (unsigned)v0; };   // n or more: not in the slice
        auto place = [&](uint32_t w) { return kEditMaxBias - 1 - (int)(w & (kEditMaxBias - 1)); };
        bool twice = false;
        if (biases) {
            for (int k = tid; k < biases; k += kEdThreads)
                if (slot(k) < (unsigned)n) atomicMax(&s_word[slot(k)], kEdBias | (unsigned)(kEditMaxBias - 1 - k));
            __syncthreads();
            for (int k = tid; k < biases; k += kEdThreads) {
                if (slot(k) >= (unsigned)n) continue;
                const int first = place(s_word[slot(k)]);
                if (first == k) continue;
                atomicOr(&s_count[first], kEdTwice);
                twice = true;
            }
        }
        auto count = [&](auto with_biases) {
#pragma unroll 1
            for (; i0 - tid < hist; fetch(i0, hist)) {
#pragma unroll
                for (int k = 0; k < kEdBatch; ++k) {
                    const unsigned t = (unsigned)id[k] - (unsigned)v0;
                    const int i = i0 + k * kEdThreads;
                    if (i >= hist || id[k] < 0 || t >= (unsigned)n) continue;
                    uint32_t *at = &s_word[t];
                    if (decltype(with_biases)::value && *at & kEdBias) at = &s_count[place(*at)];
                    if (i >= prompt) atomicAdd(at, 1u);
                    else atomicOr(at, kEdSeen);
                }
                i0 += kEdBatch * kEdThreads;
            }
        };
        if (biases) count(std::true_type{});
        else count(std::false_type{});
        if (__syncthreads_or(twice)) {
            for (int k = tid; k < biases; k += kEdThreads) {
                if (!(s_count[k] & kEdTwice)) continue;
                const int token = s_bias_id[k];
                double sum = 0.0;
#pragma unroll 2
                for (int j = k & ~7; j < biases; j += 8) {   // (FP64 is slow here: only where an entry is the token's)
                    const int4 u = *reinterpret_cast<const int4 *>(s_bias_id + j), v = *reinterpret_cast<const int4 *>(s_bias_id + j + 4);
                    uint32_t same = (u.x == token) | (u.y == token) << 1 | (u.z == token) << 2 | (u.w == token) << 3 |
                                    (v.x == token) << 4 | (v.y == token) << 5 | (v.z == token) << 6 | (v.w == token) << 7;
                    if (biases - j < 8) same &= (1u << (biases - j)) - 1u;   // (before k none is)
#pragma unroll 1
                    for (; same; same &= same - 1) sum += (double)s_bias[j + __ffs(same) - 1];
                }
                s_bias[k] = (float)sum;   // (no other thread looks at the token's entries)
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
        const int i = k * kEdThreads + tid;
        uint32_t w = counts && i < n ? s_word[i] : 0u;
        const uint32_t allowed = __shfl_sync(0xffffffffu, words, k);
        const bool biased = w & kEdBias;
        float bias = 0.f;
        if (biased) {
            const int first = kEditMaxBias - 1 - (int)(w & (kEditMaxBias - 1));
            w = s_count[first] & ~kEdTwice;
            bias = s_bias[first];
        }
        // (without branches: of 32 tokens some are in the history as a rule)
        const float c = (float)(w & ~kEdSeen);
        const float low = fmaxf(__fmul_rn(z[k], inv_low), -3.402823466e38f);   // (an infinite logit stays one)
        const float turned = z[k] > 0.f ? __fmaf_rn(z[k], inv, low) : __fmul_rn(z[k], r);
        z[k] = w ? turned : z[k];
        z[k] = c > 0.f ? __fsub_rn(z[k], __fadd_rn(__fmul_rn(f, c), p)) : z[k];
        if (biased) z[k] += bias;
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
    static_assert(most * 4 + kEditMaxBias * 12 <= 48 * 1024, "the words and the entries fit without an attribute");
    if (slice <= few) return launch_pdl(k_edit<kEdHoldFew>, grid, block, smem, st, a, slice, slices);
    return launch_pdl(k_edit<kEdHold>, grid, block, smem, st, a, slice, slices);
}

}  // namespace ds4g
