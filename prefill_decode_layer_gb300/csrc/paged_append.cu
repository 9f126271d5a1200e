// K/V append to a paged cache with the position rotation on the way: page "ds4.c
// 学习笔记 -- 端到端推理流程", 阶段四 4.2 (RoPE and KV append of the layer step), for the
// new tokens of many sequences.
//
// Token t of sequence b (start[b] <= t < start[b + 1]) has position
//   p = length[b] - (start[b + 1] - start[b]) + (t - start[b])
// and slot p % page_size of page table[b][p / page_size].  Pair (2i, 2i+1) of a key or
// query head turns by the table's (cos, sin) of (p, i) in FP32; every value is rounded
// once, to nearest even, to the type it is stored in.
//
// Bound: bytes (each row read once and written once).  A thread owns 8 adjacent dims (16
// bytes of BF16, 32 of FP32) of one token: it loads their (cos, sin) once and moves that part of
// one head after another, 128 bytes in flight.  The CTA's tokens are looked up first, by one
// warp each.
#include "paged_append.cuh"

namespace ds4g {

template <typename TI, typename TC, int U>
__global__ void __launch_bounds__(kApThreads) k_paged_append(const __grid_constant__ AppendArgs a, int tokens_per_cta)
{
    append_rows<TI, TC, U>(a, tokens_per_cta, blockIdx.x, blockIdx.y, gridDim.y, a.kv.n_kv_heads);
}

template <typename TI>
static cudaError_t append_from(const AppendArgs &a, int kv_dtype, dim3 grid, int tpc, int per_thread, cudaStream_t st)
{
    constexpr int U = 8 / sizeof(TI);
    const dim3 block(kApThreads);
    auto go = [&](auto to_bf16, auto to_f32) {
        return kv_dtype == DS4G_BF16 ? launch_pdl(to_bf16, grid, block, 0, st, a, tpc)
                                     : launch_pdl(to_f32, grid, block, 0, st, a, tpc);
    };
    if (per_thread <= 5) return go(k_paged_append<TI, bf16, 1>, k_paged_append<TI, float, 1>);
    return go(k_paged_append<TI, bf16, U>, k_paged_append<TI, float, U>);
}

cudaError_t paged_append(const AppendArgs &a, int in_dtype, int kv_dtype, cudaStream_t st, int nsm)
{
    if (a.s.n_tokens == 0) return cudaSuccess;
    const int groups = kApThreads / (a.kv.head_dim >> 3), heads = 2 * a.kv.n_kv_heads + a.n_heads;
    // Few tokens: a CTA for each and several for its heads, so that every SM has work; many:
    // up to kApTokens a CTA, whose look-ups of positions and pages run side by side.
    int tpc = 1;
    while (tpc < kApTokens && a.s.n_tokens / (2 * tpc) >= 4 * nsm) tpc *= 2;
    const int gx = (a.s.n_tokens + tpc - 1) / tpc;
    int gy = 1;
    while ((long long)gx * gy < 4 * nsm && gy * groups < heads * tpc) ++gy;
    const int per_thread = (heads * tpc + groups * gy - 1) / (groups * gy);
    return in_dtype == DS4G_BF16 ? append_from<bf16>(a, kv_dtype, dim3(gx, gy), tpc, per_thread, st)
                                 : append_from<float>(a, kv_dtype, dim3(gx, gy), tpc, per_thread, st);
}

}  // namespace ds4g
