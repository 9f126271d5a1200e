// K/V append to a paged cache in 8 bits, with the position rotation on the way: page "ds4.c
// 学习笔记 -- 端到端推理流程", 阶段四 4.2 (RoPE and KV append of the layer step), for a cache of
// E4M3 codes with a scale for each block of slots and head.
//
// For a block's new rows x of one head (rotated in FP32, products and sums rounded one by one):
//   top = max |x| over the rows and dims (of finite values),
//   ask = the least power of two with top <= 448 ask,
//   s   = ask where the block's first slot is among the new rows, else max(old s, ask),
//   code = E4M3(x / s), to nearest even; an infinity, which E4M3 has not, becomes NaN.
// A power of two costs no precision (E4M3 floats; 3 bits behind the first at every size) and
// makes division by it, and by it again, exact: where s grows, the rows that the block holds
// already, code E4M3(code old s / s), lose only what falls below E4M3's steps of 2^-9.
//
// One CTA has the block in hand: the CTA of a "leader", the first new token of its sequence or
// one at a block's first slot.  Warps take (head, K or V) pairs, a thread 8 dims of a row; where
// there are fewer pairs than warps, several share a pair's rows.  Up to eight rows a thread (FP32: four) stay in
// registers, as they came, between the maximum and the rounding, others are read again (from L2).  The
// queries' rotation is other CTAs' of the same launch.
//
// Bound: bytes (rows read once, codes written once), and latency where tokens are few: a chain of start, length,
// page, row, maximum, scale.  Measured: four prompts of 12,414 tokens in all, 64 + 16 heads of 128 (490 MB) 95 us, 0.76 of the
// copy's rate; 64 sequences' one token each 4.4 us; 33 sequences of FP32 rows 10.2 us.  (Without rows held between the
// maximum and the rounding the prompts took 123 us; with the blocks' CTAs in front of the queries' 97.)
#include <cuda_fp16.h>

#include "paged_append.cuh"

namespace ds4g {

static constexpr int kA8Tokens = 16;   // tokens of a K/V CTA at most
static constexpr int kA8Warps = kApThreads / 32;

// A block that one CTA stores into: rows tok .. tok + n - 1 of the token arrays at positions pos ..
// (n 0: none), slots `slot` .. of block `blk` of page `page`, which begin `skip` slots into the block.
struct BlockWork {
    int tok, n, pos, page, blk, slot, skip;
    bool begun;
};

// turn8 with every product and sum rounded for itself, so that the codes do not depend on
// what a compiler contracts.
__device__ __forceinline__ void turn8_rn(float (&x)[8], const float (&c)[8], int d, int rot_dim)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (d + 2 * i >= rot_dim) break;
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = __fsub_rn(__fmul_rn(a, c[2 * i]), __fmul_rn(b, c[2 * i + 1]));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(a, c[2 * i + 1]), __fmul_rn(b, c[2 * i]));
    }
}

// The least power of two s with top <= 448 s = 1.75 2^8 s, within the scales' bounds.
__device__ __forceinline__ float ask_scale(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);   // (denormal or 0: far below)
    return __uint_as_float((uint32_t)(min(max(e, -64), 64) + 127) << 23);
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Codes of x / s, 8 bytes.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s)
{
    float y[8];
    if ((__float_as_uint(s) & 0x7fffffu) == 0) {
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));   // a power of two: exact
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], 0.f, x[i] * inv);   // (0 * inf: NaN)
    } else {   // a caller's scale that was kept
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], 0.f, __fdiv_rn(x[i], s));
    }
    return make_uint2(to_e4m3x2(y[0], y[1]) | to_e4m3x2(y[2], y[3]) << 16,
                      to_e4m3x2(y[4], y[5]) | to_e4m3x2(y[6], y[7]) << 16);
}
__device__ __forceinline__ void floats8(uint2 w, float (&x)[8])
{
    const uint32_t u[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)u[i]));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The block that token tk leads, by one warp.
__device__ __forceinline__ BlockWork block_work(const AppendArgs &a, int tk)
{
    BlockWork w = {};
    if (tk >= a.s.n_tokens) return w;
    const TokenPlace at = find_token(a.s, tk);
    if (at.b >= a.s.n_seqs || tk < at.first) return w;
    const long long first = (long long)a.s.length[at.b] - at.n, p = first + (tk - at.first);
    const int block = a.kv.block, ps = a.kv.page_size;
    long long end = min(first + at.n, (long long)a.s.width * ps);   // fits 32 bits: checked by the host
    if (a.cs) end = min(end, (long long)a.n_pos);
    end = min(end, first + a.s.n_tokens - at.first);   // no row outside the token arrays, whatever start holds
    if (p < 0 || p >= end) return w;
    const int pos = (int)p, pi = pos / ps, slot = pos - pi * ps;
    w.skip = slot % block;
    if (p != max(first, 0ll) && w.skip != 0) return w;   // another token leads
    w.page = a.s.table[(long long)at.b * a.s.table_stride + pi];
    if (w.page < 0 || w.page >= a.kv.n_pages) return w;
    w.tok = tk;
    w.pos = pos;
    w.slot = slot;
    w.blk = slot / block;
    w.begun = pos - w.skip >= first;
    w.n = (int)min(end - p, (long long)(block - w.skip));
    return w;
}

template <typename TI>
__device__ __forceinline__ void append_blocks(const AppendArgs &a, int tokens_per_cta, int bx)
{
    __shared__ BlockWork s_work[kA8Tokens];
    __shared__ unsigned s_top[kA8Warps];   // of the pairs that several warps share
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    for (int i = warp; i < tokens_per_cta; i += kA8Warps) {
        const BlockWork w = block_work(a, bx * tokens_per_cta + i);
        if (lane == 0) s_work[i] = w;
    }
    if (threadIdx.x < kA8Warps) s_top[threadIdx.x] = 0u;
    __syncthreads();
    const int hd = a.kv.head_dim, hv = hd >> 3, kvh = a.kv.n_kv_heads, pairs = 2 * kvh;
    const int rpw = 32 / hv, row = lane / hv, d = (lane - row * hv) * 8;   // rows of a warp's step; this lane's
    int share = 1;   // warps of a pair
    while (2 * share * pairs <= kA8Warps) share *= 2;
    const int part = warp % share, stride = share * rpw;
    for (int i = 0; i < tokens_per_cta; ++i) {
        const BlockWork w = s_work[i];
        if (w.n == 0) continue;
        // (with share > 1 all pairs are in the first turn, where every warp comes to both barriers)
        for (int pair = warp / share; pair < pairs || share > 1; pair += kA8Warps / share) {
            const bool some = pair < pairs, is_k = pair < kvh;
            const int head = is_k ? pair : pair - kvh;
            const bool turns = is_k && a.cs && d < a.rot_dim;
            const TI *src = static_cast<const TI *>(is_k ? a.k : a.v) + head * hd + d;
            const long long ss = is_k ? a.k_stride : a.v_stride;
            const int r0 = part * rpw + row, n = some && row < rpw ? w.n : 0;
            auto turn = [&](int r, const Row8<TI> &v, float (&x)[8]) {   // (the angles: from L1 when they are read again)
                v.floats(x);
                if (turns) {
                    float c[8];
                    load_angles(c, a.cs + (long long)(w.pos + r) * a.rot_dim, d, a.rot_dim);
                    turn8_rn(x, c, d, a.rot_dim);
                }
            };
            auto value = [&](int r, float (&x)[8]) {
                Row8<TI> v;
                v.load(src + (long long)(w.tok + r) * ss);
                turn(r, v, x);
            };
            constexpr int kHold = 16 / sizeof(TI);
            Row8<TI> held[kHold];
            float top = 0.f;
            auto add = [&](const float (&y)[8]) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float m = fabsf(y[e]);
                    top = m <= 3.402823466e38f ? fmaxf(top, m) : top;   // (NaN: no)
                }
            };
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                const int r = r0 + h * stride;
                if (r < n) held[h].load(src + (long long)(w.tok + r) * ss);
            }
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                const int r = r0 + h * stride;
                float y[8];
                if (r < n) {
                    turn(r, held[h], y);
                    add(y);
                }
            }
            for (int r = r0 + kHold * stride; r < n; r += stride) {
                float y[8];
                value(r, y);
                add(y);
            }
            float *scale = const_cast<float *>(is_k ? a.kv.k_scale : a.kv.v_scale) + w.page * a.kv.scale_stride +
                           (long long)w.blk * kvh + head;
            unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            const float old = some && !w.begun ? kv8_scale(*scale) : 0.f;
            if (share > 1) {
                if (lane == 0 && some) atomicMax(&s_top[pair], bits);
                __syncthreads();
                bits = some ? s_top[pair] : 0u;
            } else {
                __syncwarp();   // every lane has read the old scale
            }
            const float s = fmaxf(old, ask_scale(__uint_as_float(bits)));
            if (some && part == 0 && lane == 0) *scale = s;
            uint8_t *dst = static_cast<uint8_t *>(const_cast<void *>(is_k ? a.kv.k : a.kv.v)) +
                           w.page * a.kv.page_stride + head * a.kv.head_stride + d;
            if (some && row < rpw && !w.begun && s > old) {   // the rows that the block holds already
                const float f = __fdiv_rn(old, s);
                for (int r = r0; r < w.skip; r += stride) {
                    uint2 *at = reinterpret_cast<uint2 *>(dst + (w.slot - w.skip + r) * a.kv.slot_stride);
                    float y[8];
                    floats8(*at, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= f;
                    *at = codes8(y, 1.f);
                }
            }
#pragma unroll
            for (int h = 0; h < kHold; ++h) {
                const int r = r0 + h * stride;
                float y[8];
                if (r < n) {
                    turn(r, held[h], y);
                    *reinterpret_cast<uint2 *>(dst + (w.slot + r) * a.kv.slot_stride) = codes8(y, s);
                }
            }
            for (int r = r0 + kHold * stride; r < n; r += stride) {
                float y[8];
                value(r, y);
                *reinterpret_cast<uint2 *>(dst + (w.slot + r) * a.kv.slot_stride) = codes8(y, s);
            }
            if (share > 1) {
                __syncthreads();   // the maxima have been read
                if (lane == 0 && some && part == 0) s_top[pair] = 0u;
                __syncthreads();
                break;
            }
        }
    }
}

// kv_ctas of the grid's CTAs, evenly spread, take blocks of K and V (a chain of look-ups, which the others' copies
// cover); the others the queries, ny of them a token group.
template <typename TI, int U>
__global__ void __launch_bounds__(kApThreads, 3) k_paged_append8(const __grid_constant__ AppendArgs a, int kv_ctas,
                                                                 int kv_tokens, int q_tokens, int ny)
{
    const unsigned long long n = gridDim.x, b = blockIdx.x;
    const int before = (int)(b * kv_ctas / n), upto = (int)((b + 1) * kv_ctas / n);   // CTAs of blocks
    const int bx = (int)b - before;
    if (upto > before) append_blocks<TI>(a, kv_tokens, before);
    else append_rows<TI, TI, U>(a, q_tokens, bx / ny, bx % ny, ny, 0);
}

cudaError_t paged_append8(const AppendArgs &a, int in_dtype, cudaStream_t st, int nsm)
{
    const int n = a.s.n_tokens, hd = a.kv.head_dim;
    if (n == 0) return cudaSuccess;
    int kv_tokens = 1;
    while (kv_tokens < kA8Tokens && 2 * kv_tokens <= a.kv.block && n / (2 * kv_tokens) >= 4 * nsm) kv_tokens *= 2;
    const int kv_ctas = (n + kv_tokens - 1) / kv_tokens;
    // the queries as the append without scales divides them
    int tpc = 1, ny = 0, gx = 0, per_thread = 0;
    if (a.n_heads) {
        const int groups = kApThreads / (hd >> 3);
        while (tpc < kApTokens && n / (2 * tpc) >= 4 * nsm) tpc *= 2;
        gx = (n + tpc - 1) / tpc;
        ny = 1;
        while ((long long)gx * ny < 4 * nsm && ny * groups < a.n_heads * tpc) ++ny;
        per_thread = (a.n_heads * tpc + groups * ny - 1) / (groups * ny);
    }
    const dim3 grid(kv_ctas + gx * ny), block(kApThreads);
    auto go = [&](auto few, auto many) {
        return launch_pdl(per_thread <= 5 ? few : many, grid, block, 0, st, a, kv_ctas, kv_tokens, tpc, ny > 0 ? ny : 1);
    };
    return in_dtype == DS4G_BF16 ? go(k_paged_append8<bf16, 1>, k_paged_append8<bf16, 4>)
                                 : go(k_paged_append8<float, 1>, k_paged_append8<float, 2>);
}

}  // namespace ds4g
