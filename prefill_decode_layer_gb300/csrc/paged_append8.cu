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
// One CTA has the rows of a block that its (head, K or V) pairs need: a CTA of the "leader", the first new token of its
// sequence or one at a block's first slot.  A warp has one pair, a thread 8 dims of a row; so many warps share a pair
// that its rows of a block stay in registers, as they came, between the maximum and the rounding: eight a thread (FP32:
// four; what is more is read again, from L2).  The other pairs are other CTAs' of the same leaders, and the queries'
// rotation that of others of the same launch.  Leaders are found first, a lane a token: what 32 sequences have for it
// in one round of loads, then its page.
//
// Bound: bytes (rows read once, codes written once), and latency where tokens are few: a chain of start and length,
// page, row, maximum, scale.  Measured: four prompts of 12,414 tokens in all, 64 + 16 heads of 128 (490 MB) 84 us, 0.86 of
// the copy's rate; 64 sequences' one token each 4.1 us; 768 FP32 rows of 33 sequences 7.9 us.  (All pairs of a block by one
// CTA, look-ups a warp a token: 95, 4.4 and 10.2 us; without rows held 123.  K and V of the prompts alone 34 us in blocks
// of 16 and 33 of 64, for 42 and 76; the angles are a third of it, but those of two rows at once did not fit registers.)
#include <cuda_fp16.h>

#include "paged_append.cuh"

namespace ds4g {

// Tokens of a K/V CTA at most: a lane looks up each.  (32: the prompts' K and V in blocks of 64 38.8 us for 32.8.)
static constexpr int kA8Tokens = 128;
static constexpr int kA8Warps = kApThreads / 32;
template <typename TI> constexpr int kA8Hold = 16 / sizeof(TI);   // rows of a thread in registers

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

// Codes of x / s, 8 bytes.  odd: some x may be infinite.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, bool odd)
{
    float y[8];
    if ((__float_as_uint(s) & 0x7fffffu) == 0) {
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));   // a power of two: exact
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    } else {   // a caller's scale that was kept
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], s);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], 0.f, y[i]);   // (0 * inf: NaN)
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

// The blocks that the first 32 of tokens t0 .. t0 + count - 1 lead, by one warp: a lane finds its token's.
__device__ __forceinline__ BlockWork block_work(const AppendArgs &a, int t0, int count)
{
    const int lane = threadIdx.x & 31, tk = t0 + lane;
    const bool mine = lane < count && tk < a.s.n_tokens;
    BlockWork w = {};
    int b = -1, begin = tk, n_new = 1, length = 0;
    if (!a.s.start) {
        if (mine) length = a.s.length[b = tk];
    } else {
        // lane i looks at sequence b0 + i: all that the tokens need of 32 sequences in one round of loads
        int b0 = a.s.n_seqs <= 32 ? 0 : find_token(a.s, min(t0, a.s.n_tokens - 1)).b;
        bool open = mine;
        for (; b0 < a.s.n_seqs && __any_sync(0xffffffffu, open); b0 += 32) {
            const int q = min(b0 + lane, a.s.n_seqs - 1);
            const int q_begin = a.s.start[q], q_end = a.s.start[q + 1], q_length = a.s.length[q];
            const int end = b0 + lane < a.s.n_seqs ? q_end : 0x7fffffff;
            int c = 0;   // as many of them end at or before the token
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (__shfl_sync(0xffffffffu, end, c + o - 1) <= tk) c += o;
            const bool found = __shfl_sync(0xffffffffu, end, c) > tk;
            const int f = __shfl_sync(0xffffffffu, q_begin, c), e = __shfl_sync(0xffffffffu, q_end, c),
                      l = __shfl_sync(0xffffffffu, q_length, c);
            if (open && found) {
                open = false;
                if (b0 + c < a.s.n_seqs) {
                    b = b0 + c;
                    begin = f;
                    n_new = e - f;
                    length = l;
                }
            }
        }
    }
    if (b < 0 || tk < begin) return w;
    const TokenPlace at = {b, begin, n_new};
    const long long first = (long long)length - at.n, p = first + (tk - at.first);
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

// by: which of the groups of (head, K or V) pairs; share: warps of a pair.
template <typename TI>
__device__ __forceinline__ void append_blocks(const AppendArgs &a, int tokens_per_cta, int bx, int by, int share)
{
    __shared__ BlockWork s_work[kA8Tokens];   // of the CTA's leaders, in any order
    __shared__ int s_n;
    __shared__ unsigned s_top[kA8Warps];   // of the pairs that several warps share
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    BlockWork found = {};
    if (warp * 32 < tokens_per_cta) found = block_work(a, bx * tokens_per_cta + warp * 32, tokens_per_cta - warp * 32);
    if (threadIdx.x < kA8Warps) s_top[threadIdx.x] = 0u;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    if (found.n > 0) s_work[atomicAdd(&s_n, 1)] = found;
    __syncthreads();
    const int leaders = s_n;
    const int hd = a.kv.head_dim, hv = hd >> 3, kvh = a.kv.n_kv_heads;
    const int rpw = 32 / hv, row = lane / hv, d = (lane - row * hv) * 8;   // rows of a warp's step; this lane's
    const int part = warp % share, stride = share * rpw, r0 = part * rpw + row;
    const int mine = warp / share, pair = by * (kA8Warps / share) + mine;
    const bool some = pair < 2 * kvh, is_k = pair < kvh;
    const int head = some ? is_k ? pair : pair - kvh : 0;
    const bool turns = is_k && a.cs && d < a.rot_dim;
    const TI *src = static_cast<const TI *>(is_k ? a.k : a.v) + head * hd + d;
    const long long ss = is_k ? a.k_stride : a.v_stride;
    for (int i = 0; i < leaders; ++i) {
        const BlockWork w = s_work[i];
        const int n = some && row < rpw ? w.n : 0;
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
        constexpr int kHold = kA8Hold<TI>;
        Row8<TI> held[kHold];
        unsigned top = 0u;   // magnitudes as bits, which order as they do
        auto add = [&](const float (&y)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
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
        const bool odd = top >= 0x7f800000u;   // infinities or NaN: the maximum of the others
        if (odd) {
            top = 0u;
#pragma unroll 1
            for (int r = r0; r < n; r += stride) {
                float y[8];
                value(r, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned m = __float_as_uint(y[e]) & 0x7fffffffu;
                    top = m < 0x7f800000u ? max(top, m) : top;
                }
            }
        }
        __syncwarp();
        float *scale = const_cast<float *>(is_k ? a.kv.k_scale : a.kv.v_scale) + w.page * a.kv.scale_stride +
                       (long long)w.blk * kvh + head;
        unsigned bits = __reduce_max_sync(0xffffffffu, top);
        const float old = some && !w.begun ? kv8_scale(*scale) : 0.f;
        if (share > 1) {
            if (lane == 0 && some) atomicMax(&s_top[mine], bits);
            __syncthreads();
            bits = s_top[mine];
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
                *at = codes8(y, 1.f, false);
            }
        }
#pragma unroll
        for (int h = 0; h < kHold; ++h) {
            const int r = r0 + h * stride;
            float y[8];
            if (r < n) {
                turn(r, held[h], y);
                *reinterpret_cast<uint2 *>(dst + (w.slot + r) * a.kv.slot_stride) = codes8(y, s, odd);
            }
        }
        for (int r = r0 + kHold * stride; r < n; r += stride) {
            float y[8];
            value(r, y);
            *reinterpret_cast<uint2 *>(dst + (w.slot + r) * a.kv.slot_stride) = codes8(y, s, odd);
        }
        if (share > 1) {
            __syncthreads();   // the maxima have been read
            if (lane == 0 && part == 0) s_top[mine] = 0u;
            __syncthreads();
        }
    }
}

// kv_ctas of the grid's CTAs, evenly spread, take blocks of K and V (a chain of look-ups, which the others' copies
// cover), nk of them a token group; the others the queries, ny of them a token group.
template <typename TI, int U>
__global__ void __launch_bounds__(kApThreads, 3) k_paged_append8(const __grid_constant__ AppendArgs a, int kv_ctas,
                                                                 int kv_tokens, int nk, int share, int q_tokens, int ny)
{
    const unsigned long long n = gridDim.x, b = blockIdx.x;
    const int before = (int)(b * kv_ctas / n), upto = (int)((b + 1) * kv_ctas / n);   // CTAs of blocks
    const int bx = (int)b - before;
    if (upto > before) append_blocks<TI>(a, kv_tokens, before / nk, before % nk, share);
    else append_rows<TI, TI, U>(a, q_tokens, bx / ny, bx % ny, ny, 0);
}

template <typename TI> static cudaError_t append8_from(const AppendArgs &a, cudaStream_t st, int nsm)
{
    const int n = a.s.n_tokens, hd = a.kv.head_dim, hv = hd >> 3, pairs = 2 * a.kv.n_kv_heads;
    // warps of a pair: as many as hold a block's rows in registers, more where there are fewer pairs than warps; a
    // warp has one pair
    int share = 1;
    while (share < kA8Warps && (share * kA8Hold<TI> * (32 / hv) < a.kv.block || 2 * share * pairs <= kA8Warps)) share *= 2;
    const int per_cta = kA8Warps / share, nk = (pairs + per_cta - 1) / per_cta;
    // (by tokens, of which few lead a block in calls of many: of 768 FP32 rows in blocks of 16 most CTAs find none, and
    // the grid takes two turns, 7.9 us for the chain's 4.1)
    int kv_tokens = 1;
    while (kv_tokens < kA8Tokens && 2 * kv_tokens <= a.kv.block && (long long)n * nk / (2 * kv_tokens) >= 4 * nsm) kv_tokens *= 2;
    // many tokens of tens of thousands of heads: a grid has 2^31 - 1 CTAs at most, of which the queries take up to 2^28
    auto ctas = [&]() { return ((long long)n + kv_tokens - 1) / kv_tokens * nk; };
    while (kv_tokens < kA8Tokens && ctas() > (1 << 24)) kv_tokens *= 2;
    if (ctas() > (1 << 30)) return cudaErrorInvalidValue;
    const int kv_ctas = (int)ctas();
    // the queries as the append without scales divides them
    int tpc = 1, ny = 0, gx = 0, per_thread = 0;
    if (a.n_heads) {
        const int groups = kApThreads / hv;
        while (tpc < kApTokens && n / (2 * tpc) >= 4 * nsm) tpc *= 2;
        gx = (n + tpc - 1) / tpc;
        ny = 1;
        while ((long long)gx * ny < 4 * nsm && ny * groups < a.n_heads * tpc) ++ny;
        per_thread = (a.n_heads * tpc + groups * ny - 1) / (groups * ny);
    }
    const dim3 grid(kv_ctas + gx * ny), block(kApThreads);
    auto kernel = per_thread <= 5 ? k_paged_append8<TI, 1> : k_paged_append8<TI, 8 / sizeof(TI)>;
    return launch_pdl(kernel, grid, block, 0, st, a, kv_ctas, kv_tokens, nk, share, tpc, ny > 0 ? ny : 1);
}

cudaError_t paged_append8(const AppendArgs &a, int in_dtype, cudaStream_t st, int nsm)
{
    if (a.s.n_tokens == 0) return cudaSuccess;
    return in_dtype == DS4G_BF16 ? append8_from<bf16>(a, st, nsm) : append8_from<float>(a, st, nsm);
}

}  // namespace ds4g
