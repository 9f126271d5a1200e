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
// Bound: bytes (each row read once and written once).  A thread moves 8 elements of
// one head at a time (16 bytes of BF16, 32 of FP32); the CTA's tokens are looked up
// first by one warp each, then all threads walk the (token, 8-element vector) pairs.
#include "paged.h"

namespace ds4g {

static constexpr int kApThreads = 256;
static constexpr int kApTokens = 8;   // tokens of a CTA at most: one warp looks up each

template <typename T> struct Row8;
template <> struct Row8<bf16> {
    static __device__ __forceinline__ void load(const bf16 *p, float (&x)[8])
    {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(bf16 *p, const float (&x)[8])
    {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            u[i] = pack_bf16x2(__float2bfloat16_rn(x[2 * i]), __float2bfloat16_rn(x[2 * i + 1]));
        *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Row8<float> {
    static __device__ __forceinline__ void load(const float *p, float (&x)[8])
    {
        const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// Turn the pairs of dims d .. d + 7 by the row cs of the table (rot_dim / 2 pairs).
__device__ __forceinline__ void turn8(float (&x)[8], const float *cs, int d, int rot_dim)
{
    float4 t[2][2];
    if (d + 8 <= rot_dim && (rot_dim & 3) == 0) {   // 16-byte aligned: rows of a multiple of 4 floats
        const float4 *p = reinterpret_cast<const float4 *>(cs + d);
        t[0][0] = p[0];
        t[0][1] = p[1];
    } else {
        float c[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = d + 2 * i < rot_dim;
            c[2 * i] = in ? cs[d + 2 * i] : 1.f;
            c[2 * i + 1] = in ? cs[d + 2 * i + 1] : 0.f;
        }
        t[0][0] = make_float4(c[0], c[1], c[2], c[3]);
        t[0][1] = make_float4(c[4], c[5], c[6], c[7]);
    }
    const float c[8] = {t[0][0].x, t[0][0].y, t[0][0].z, t[0][0].w, t[0][1].x, t[0][1].y, t[0][1].z, t[0][1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (d + 2 * i >= rot_dim) break;   // passes through unchanged, whatever it holds
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[2 * i] - b * c[2 * i + 1];
        x[2 * i + 1] = a * c[2 * i + 1] + b * c[2 * i];
    }
}

template <typename TI, typename TC>
__global__ void __launch_bounds__(kApThreads) k_paged_append(const __grid_constant__ AppendArgs a, int tokens_per_cta)
{
    __shared__ long long s_slot[kApTokens];   // element offset of the token's slot, or -1
    __shared__ int s_pos[kApTokens];          // its position, or -1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * tokens_per_cta;
    pdl_wait();
    pdl_trigger();
    if (warp < tokens_per_cta) {
        const int t = t0 + warp;
        int pos = -1;
        long long slot = -1;
        if (t < a.s.n_tokens) {
            int b = t, first = t, n = 1;
            if (a.s.start) {
                // the sequence of token t: as many sequences end at or before it
                int ended = 0;
                for (int i = lane; i < a.s.n_seqs; i += 32) ended += a.s.start[i + 1] <= t;
                b = __reduce_add_sync(0xffffffffu, ended);
                if (b < a.s.n_seqs) {
                    first = a.s.start[b];
                    n = a.s.start[b + 1] - first;
                }
            }
            if (b < a.s.n_seqs && t >= first) {
                const long long p = (long long)a.s.length[b] - n + (t - first);
                if (p >= 0 && p < (long long)a.s.width * a.kv.page_size) {
                    const int page = a.s.table[(long long)b * a.s.table_stride + (int)p / a.kv.page_size];
                    if (page >= 0 && page < a.kv.n_pages)
                        slot = page * a.kv.page_stride + ((int)p % a.kv.page_size) * a.kv.slot_stride;
                }
                if (p >= 0 && p < 0x7fffffff) pos = (int)p;
                if (a.cs && p >= a.n_pos) {   // no angle for it
                    pos = -1;
                    slot = -1;
                }
            }
        }
        if (lane == 0) {
            s_pos[warp] = pos;
            s_slot[warp] = slot;
        }
    }
    __syncthreads();
    const int hd = a.kv.head_dim, hv = hd >> 3, kvv = a.kv.n_kv_heads * hv;
    const int per = 2 * kvv + a.n_heads * hv;   // vectors of a token: K, V, then Q
    const int total = per * min(tokens_per_cta, a.s.n_tokens - t0);
    const TI *k = static_cast<const TI *>(a.k), *v = static_cast<const TI *>(a.v), *q = static_cast<const TI *>(a.q);
    TC *kc = static_cast<TC *>(const_cast<void *>(a.kv.k)), *vc = static_cast<TC *>(const_cast<void *>(a.kv.v));
    TI *qo = static_cast<TI *>(a.q_out);
    constexpr int U = 4;   // vectors in flight per thread
    const int stride = gridDim.y * kApThreads;
    for (int i0 = blockIdx.y * kApThreads + threadIdx.x; i0 < total; i0 += U * stride) {
        float x[U][8];
        int tt[U], vec[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * stride;
            tt[u] = -1;
            if (i >= total) continue;
            const int j = i / per;
            tt[u] = j;
            vec[u] = i - j * per;
            const long long t = t0 + j;
            const TI *src = vec[u] < kvv       ? k + t * a.k_stride + vec[u] * 8
                            : vec[u] < 2 * kvv ? v + t * a.v_stride + (vec[u] - kvv) * 8
                                               : q + t * a.q_stride + (vec[u] - 2 * kvv) * 8;
            Row8<TI>::load(src, x[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (tt[u] < 0) continue;
            const int pos = s_pos[tt[u]];
            const long long slot = s_slot[tt[u]];
            if (pos < 0) continue;
            const int c = vec[u];
            if (c < 2 * kvv) {
                if (slot < 0) continue;
                const int kv = c < kvv ? c : c - kvv, h = kv / hv, d = (kv - h * hv) * 8;
                if (c < kvv && a.cs && d < a.rot_dim) turn8(x[u], a.cs + (long long)pos * a.rot_dim, d, a.rot_dim);
                Row8<TC>::store((c < kvv ? kc : vc) + slot + h * a.kv.head_stride + d, x[u]);
            } else {
                const int d = (c - 2 * kvv) % hv * 8;
                if (a.cs && d < a.rot_dim) turn8(x[u], a.cs + (long long)pos * a.rot_dim, d, a.rot_dim);
                Row8<TI>::store(qo + (t0 + tt[u]) * a.q_out_stride + (c - 2 * kvv) * 8, x[u]);
            }
        }
    }
}

cudaError_t paged_append(const AppendArgs &a, int in_dtype, int kv_dtype, cudaStream_t st, int nsm)
{
    if (a.s.n_tokens == 0) return cudaSuccess;
    const int per = (2 * a.kv.n_kv_heads + a.n_heads) * (a.kv.head_dim >> 3);
    // Few tokens: a CTA for each and several for its vectors, so that every SM has work;
    // many: up to kApTokens a CTA, which share one look-up of positions and pages.
    int tpc = 1;
    while (tpc < kApTokens && a.s.n_tokens / (2 * tpc) >= 16 * nsm) tpc *= 2;
    const int gx = (a.s.n_tokens + tpc - 1) / tpc;
    int gy = 1;
    while ((long long)gx * gy < 8 * nsm && gy * kApThreads < per * tpc) ++gy;
    const dim3 grid(gx, gy), block(kApThreads);
    if (in_dtype == DS4G_BF16)
        return kv_dtype == DS4G_BF16 ? launch_pdl(k_paged_append<bf16, bf16>, grid, block, 0, st, a, tpc)
                                     : launch_pdl(k_paged_append<bf16, float>, grid, block, 0, st, a, tpc);
    return kv_dtype == DS4G_BF16 ? launch_pdl(k_paged_append<float, bf16>, grid, block, 0, st, a, tpc)
                                 : launch_pdl(k_paged_append<float, float>, grid, block, 0, st, a, tpc);
}

}  // namespace ds4g
