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
#include "paged.h"

namespace ds4g {

static constexpr int kApThreads = 256;
static constexpr int kApTokens = 8;   // tokens of a CTA at most: one warp looks up each

// 8 adjacent elements: as loaded, and as floats.
template <typename T> struct Row8;
template <> struct Row8<bf16> {
    uint4 w;
    __device__ __forceinline__ void load(const bf16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
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
    float4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const
    {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[8])
    {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// (cos, sin) of the pairs of dims d .. d + 7 from a row of the table (rot_dim / 2 pairs).
__device__ __forceinline__ void load_angles(float (&c)[8], const float *cs, int d, int rot_dim)
{
    if (d + 8 <= rot_dim && (rot_dim & 3) == 0) {   // 16-byte aligned: rows of a multiple of 4 floats
        Row8<float> r;
        r.load(cs + d);
        r.floats(c);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = d + (i & ~1) < rot_dim ? cs[d + i] : 0.f;
}
__device__ __forceinline__ void turn8(float (&x)[8], const float (&c)[8], int d, int rot_dim)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (d + 2 * i >= rot_dim) break;   // passes through unchanged, whatever it holds
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = a * c[2 * i] - b * c[2 * i + 1];
        x[2 * i + 1] = a * c[2 * i + 1] + b * c[2 * i];
    }
}

// U: heads in flight per thread, twice: the next U are loaded before these are stored (10k
// tokens of 66 heads: 72 us, 88 % of the copy rate).  One where a thread has up to five: more CTAs
// fit an SM, and the unrolled form's instructions take longer to fetch (1000 tokens: 10.2 us
// against 14.0).
template <typename TI, typename TC, int U>
__global__ void __launch_bounds__(kApThreads) k_paged_append(const __grid_constant__ AppendArgs a, int tokens_per_cta)
{
    __shared__ long long s_slot[kApTokens];   // element offset of the token's slot, or -1
    __shared__ int s_pos[kApTokens];          // its position, or -1
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * tokens_per_cta;
    const int hd = a.kv.head_dim, hv = hd >> 3, kvh = a.kv.n_kv_heads;
    // groups of hv threads; `per` of them share a token
    const int per = kApThreads / hv / tokens_per_cta, grp = threadIdx.x / hv, d = (threadIdx.x - grp * hv) * 8;
    const int j = grp / per;
    const bool mine = j < min(tokens_per_cta, a.s.n_tokens - t0);
    const long long t = t0 + j;
    const int heads = mine ? a.n_heads + 2 * kvh : 0;   // of a token: queries, keys, values
    const TI *k = static_cast<const TI *>(a.k) + t * a.k_stride + d;
    const TI *v = static_cast<const TI *>(a.v) + t * a.v_stride + d;
    const TI *q = static_cast<const TI *>(a.q) + t * a.q_stride + d;
    const int step = per * gridDim.y;
    auto load = [&](Row8<TI> (&w)[U], int h0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step, kh = h - a.n_heads;
            if (h < heads) w[u].load(kh < 0 ? q + h * hd : kh < kvh ? k + kh * hd : v + (kh - kvh) * hd);
        }
    };
    pdl_wait();
    pdl_trigger();
    int h0 = grp - j * per + per * blockIdx.y;
    Row8<TI> w[U];
    load(w, h0);   // on its way while the positions and pages are looked up
    if (warp < tokens_per_cta) {
        const int tk = t0 + warp;
        int pos = -1;
        long long slot = -1;
        if (tk < a.s.n_tokens) {
            int b = tk, first = tk, n = 1;
            if (a.s.start) {
                // the sequence of token tk: as many sequences end at or before it.  Of many, the
                // 32nd part in which the last of them lies first (start does not fall).
                int from = 0, left = a.s.n_seqs;
                while (left > 256) {
                    const int part = (left + 31) / 32, i = (lane + 1) * part;
                    const bool ends = i <= left && a.s.start[from + i] <= tk;
                    const int skip = __popc(__ballot_sync(0xffffffffu, ends)) * part;
                    from += skip;
                    left = min(part, left - skip);
                }
                int ended = 0;
                for (int i = lane; i < left; i += 32) ended += a.s.start[from + i + 1] <= tk;
                b = from + __reduce_add_sync(0xffffffffu, ended);
                if (b < a.s.n_seqs) {
                    first = a.s.start[b];
                    n = a.s.start[b + 1] - first;
                }
            }
            if (b < a.s.n_seqs && tk >= first) {
                const long long p = (long long)a.s.length[b] - n + (tk - first);
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
    if (!mine) return;
    const int pos = s_pos[j];
    if (pos < 0) return;
    const long long slot = s_slot[j];
    TC *kc = static_cast<TC *>(const_cast<void *>(a.kv.k)) + slot + d;
    TC *vc = static_cast<TC *>(const_cast<void *>(a.kv.v)) + slot + d;
    TI *qo = static_cast<TI *>(a.q_out) + t * a.q_out_stride + d;
    const bool turns = a.cs && d < a.rot_dim;
    float c[8];
    if (turns) load_angles(c, a.cs + (long long)pos * a.rot_dim, d, a.rot_dim);
#pragma unroll 1
    for (; h0 < heads; h0 += U * step) {
        Row8<TI> next[U];
        if (U > 1) load(next, h0 + U * step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u * step, kh = h - a.n_heads;
            if (h >= heads) continue;
            float x[8];
            w[u].floats(x);
            if (turns && kh < kvh) turn8(x, c, d, a.rot_dim);
            if (kh < 0) Row8<TI>::store(qo + h * hd, x);
            else if (slot >= 0) Row8<TC>::store(kh < kvh ? kc + kh * a.kv.head_stride : vc + (kh - kvh) * a.kv.head_stride, x);
        }
        if (U == 1) {
            load(w, h0 + step);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = next[u];
        }
    }
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
