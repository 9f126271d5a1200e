// Tensor-core form of the paged attention over a cache in 8 bits (tcgen05 MMAs with TMEM
// accumulators, TMA tiles of the cache's pages): page "ds4.c 学习笔记 -- 端到端推理流程", 阶段四
// 4.2.  The division of the work is paged_sched.cuh's; BF16 queries, head_dim 64 or 128.
//
// With K_j = ks_j k_j and V_j = vs_j v_j (codes k, v; scales ks, vs of key j's block), row r is
//   out_r = sum_j p_rj v_j / sum_j p_rj / vs_j,
//   p_rj = 2^(t_rj - m_r),  t_rj = (scale log2 e) ks_j (q_r . k_j) + log2 vs_j,
// so that the scales are two numbers a key, and m_r (the running maximum of t_rj, less 9) bounds what
// p_rj v_j adds to the row whatever the scales are.
//
// Both products have the keys on the MMA's M side, or the dims, and the query rows on its N
// side: with the few rows of a decode step the tensor cores' time then falls with the rows, and the
// softmax's work is spread over all 128 keys of a unit:
//   S^T = K Q^T    M 128 keys x N rows.  K's codes go from their TMA tile into the MMA as they are
//                  (kind::f8f6f4).  A BF16 query is the sum of two E4M3 values, exactly: of
//                  x in units of the row's power of two, hi = E4M3(x) holds 4 of its 8 bits and
//                  16 (x - hi) the others.  The two are 2 x rows columns of one MMA;
//   softmax        a thread owns a key and half of the rows; it adds the two halves, applies scales and
//                  masks and writes P^T as FP16 to shared memory.  FP16 (11 bits down to 2^-23 of the
//                  maximum, 2^-33 at least) and not E4M3, in which what is small beside the maximum,
//                  but counts because it is much, would vanish;
//   O^T += V^T P^T M 128 dims x N rows (kind::f16), of V's codes as FP16, which holds them exactly.
//                  Four warps convert each tile from its bytes.
// m_r moves only when a weight would exceed 2^15: nothing is reduced over keys in most units.
// Row sums are kept per key and thread in FP32 and added up when the item ends.
//
// Masked places: a key outside the item's keys or in a missing page, or hidden from a row, gets the
// weight 0; its row of V becomes zeros in the conversion.  NaN codes in V become 0 as well, and rows
// that see such a key get their NaN when the item ends.
//
// Roles (480 threads, one CTA per SM): warps 0-3 and 4-7 softmax and output of the two halves of
// the rows; warps 8-11 queries, scales and V's conversion; warp 12 the items and the TMA copies;
// warps 13 and 14 (one thread each) the MMAs of S and of O.  Every wait is bounded; a CTA that gives up
// says so in its status word, drains its copies and MMAs, frees its TMEM and returns.
#include <cuda.h>
#include <cuda_fp16.h>
#include <stddef.h>

#include "paged_sched.cuh"
#include "sm100.cuh"
#include "tc_gemm.cuh"

namespace ds4g {

static constexpr int kT8Keys = 128;                    // keys of a unit
static constexpr int kT8Rows = 64;                     // query rows of a tile at most
static constexpr int kT8Soft = 256, kT8Conv = 128;     // threads of the softmax, of the conversion
static constexpr int kT8Threads = kT8Soft + kT8Conv + 96;
static constexpr int kT8ConvWarp = kT8Soft / 32, kT8Tma = kT8ConvWarp + kT8Conv / 32, kT8Mma = kT8Tma + 1;
static constexpr int kT8MaxSlots = 4;                  // tiles of K, and of V, at most
static constexpr int kT8Items = 4;                     // items ahead of the softmax at most
static constexpr int kT8Scales = 4;                    // units whose scales are there at most
static constexpr int kT8Smem = 227 * 1024;
static constexpr float kT8Off = 9.f, kT8Most = 15.f;   // log2 of the largest weight when m is set, and before it moves

struct T8Misc {
    uint64_t k_full[kT8MaxSlots], k_empty[kT8MaxSlots], v_full[kT8MaxSlots], v_empty[kT8MaxSlots];
    uint64_t w_full[2], w_empty[2];                    // V tiles in FP16
    uint64_t sc_full[kT8Scales], sc_empty[kT8Scales];
    uint64_t q_full[2], q_empty[2];                    // of item i % 2
    uint64_t s_full[2], p_full[2], p_empty[2];         // of unit u % 2
    uint64_t o_free[2];                                // of item i % 2: its O has been read
    uint64_t item_full[kT8Items], item_empty[kT8Items];
    uint64_t done[2];
    PagedItem item[kT8Items];
    PagedCursor cur;
    long long scratch[kT8Threads / 32];
    float2 sc[kT8Scales][kT8Keys];                     // of a unit's keys: ks scale log2 e, log2 vs (-inf: masked)
    uint32_t valid[kT8Scales][4];                      // a bit per key of the unit
    int poison[kT8Items];                              // a V row of the item that counts has a NaN
    uint32_t tmem;
    int abort_flag;
    __align__(16) float q_scale[kT8Items][kT8Rows];      // of an item's rows (in item_full's slot: read until item_empty)
    __align__(16) float neg_m[kT8Rows], factor[kT8Rows];
    float part[8][32];                                 // of a softmax warp: a value of each row
    int pos[kT8Rows];
    long long off[kT8Rows];                            // of a row in the output
};

struct T8Geometry {
    int k_slots, v_slots;
    int box;         // slots of a page in one copy: gcd(page_size, 128)
    int page_shift;  // log2(page_size), or -1
};

bool paged_attn8_tc_ok(const PagedKV &kv, int q_dtype)
{
    return q_dtype == DS4G_BF16 && (kv.head_dim == 64 || kv.head_dim == 128) && kv.page_size % 8 == 0;
}

// Query rows of a tile: as few tiles as hold them, of equal size.
int paged_attn8_tc_rows(int group, int max_new)
{
    const int rows = group * max_new, tiles = (rows + kT8Rows - 1) / kT8Rows;
    return (rows + tiles - 1) / tiles;
}

__device__ __forceinline__ uint32_t t8_e4m3x2(float lo, float hi)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t t8_f16x2(uint32_t codes)   // of the low two bytes
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    return h;
}
// Barrier `id` of the n threads that use it, which tells each whether any of them says so.
template <int N> __device__ __forceinline__ bool t8_any(int id, bool yes)
{
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, %3, q;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)yes), "r"(id), "n"(N)
        : "memory");
    return any != 0;
}
template <int N> __device__ __forceinline__ void t8_sync(int id)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory");
}
__device__ __forceinline__ float t8_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// HD: head_dim.  NR: columns of query rows, the tile's rows or more.
template <int HD, int NR>
__global__ void __launch_bounds__(kT8Threads, 1)
    k_paged_attn8_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ AttnArgs a, const __grid_constant__ T8Geometry geo)
{
    constexpr int H = HD / 64;                          // 128-byte blocks of an FP16 row
    constexpr uint32_t kTile = HD * kT8Keys;            // bytes of a K or V tile of codes
    constexpr uint32_t kWide = 2 * kTile;               // of V in FP16
    constexpr uint32_t kQ = 2 * NR * HD, kP = kT8Keys * 128;
    constexpr uint32_t kCols = NR == 64 ? 512 : NR == 32 ? 256 : 128;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *wide = sm, *pbuf = wide + 2 * kWide, *qbuf = pbuf + 2 * kP, *kring = qbuf + 2 * kQ;
    unsigned char *vring = kring + (uint32_t)geo.k_slots * kTile;
    T8Misc &x = *reinterpret_cast<T8Misc *>(vring + (uint32_t)geo.v_slots * kTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PartLayout lay(kAttnMaxCtasTc, a.rows, HD);

    {   // one barrier per thread
        uint64_t *bars = x.k_full;
        constexpr int n = offsetof(T8Misc, item) / 8;
        const int i = threadIdx.x;
        auto in = [&](const uint64_t *b, int count) { return bars + i >= b && bars + i < b + count; };
        if (i < n) {
            int count = 1;
            if (in(x.v_empty, kT8MaxSlots) || in(x.w_full, 2) || in(x.sc_full, kT8Scales) || in(x.q_full, 2)) count = kT8Conv / 32;
            else if (in(x.sc_empty, kT8Scales) || in(x.p_full, 2) || in(x.o_free, 2)) count = kT8Soft / 32;
            else if (in(x.item_empty, kT8Items)) count = kT8Soft / 32 + kT8Conv / 32 + 2;
            mbar_init(bars + i, count);
        } else if (i == n) {
            x.abort_flag = 0;
        }
        mbar_fence_init();
    }
    if (warp == kT8Mma) tmem_alloc(&x.tmem, kCols);
    if (threadIdx.x == kT8Tma * 32) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_trigger();
    paged_begin(a, lay);
    const bool few = a.s.n_seqs <= 32;   // the copying warp finds the CTA's share by itself
    if (!few) paged_cursor<kT8Threads>(a, kT8Keys, &x.cur, x.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x.tmem;   // S of unit u: column (u % 2) 2 NR; O of item i: 4 NR + (i % 2) NR
    volatile int *ab = &x.abort_flag;
    auto give_up = [&]() {
        x.abort_flag = 1;
        reinterpret_cast<int *>(a.ws + lay.status)[blockIdx.x] = kAttnTimedOut;
    };
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab)) != 0;
    };
    // a place in a ring (kept up to date: no division at every use)
    struct Place {
        unsigned slot, phase;
        __device__ __forceinline__ void next(unsigned slots)
        {
            if (++slot == slots) {
                slot = 0;
                phase ^= 1u;
            }
        }
    };

    if (warp == kT8Tma) {
        // ---------------- items, page look-ups, copies
        PagedCursor cur;
        if (few) paged_cursor_warp(a, kT8Keys, cur);
        else cur = x.cur;
        const int boxes = kT8Keys / geo.box, ps = a.kv.page_size;
        int used_k = -1, used_v = -1;   // lane i: the phase of the last load into slot i
        Place kp = {0, 0}, vp = {0, 0};
        bool ok = true;
        for (unsigned i = 0; ok; ++i) {
            if (!warp_wait(&x.item_empty[i % kT8Items], (i / kT8Items & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            PagedItem &it = x.item[i % kT8Items];
            if (lane == 0) {
                paged_next(a, kT8Keys, cur, lay, it);
                x.poison[i % kT8Items] = 0;
                mbar_arrive(&x.item_full[i % kT8Items]);
            }
            __syncwarp();
            if (!it.more) break;
            const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
            const int lo = it.lo, hi = it.hi, head = it.head, t1 = it.t1;
            // this lane's box of tile t: whether it is copied, its page and first slot
            int page = -1, slot = 0;
            auto look = [&](int t) {
                const int j = t * kT8Keys + lane * geo.box;
                const bool load = t < t1 && lane < boxes && j < hi && j + geo.box > lo;
                if (load) {
                    const int p = geo.page_shift >= 0 ? j >> geo.page_shift : j / ps;
                    slot = j - p * ps;
                    page = table[p];
                }
                return load;
            };
            bool load = look(it.t0);
            for (int t = it.t0; ok && t < t1; ++t) {
                // a page that is not there: out of bounds, read as zeros
                const int at = page < 0 || page >= a.kv.n_pages ? a.kv.n_pages : page, from = slot;
                const bool mine = load;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, mine)) * geo.box * HD;
                load = look(t + 1);   // on its way while the slots become free
                auto copy = [&](uint64_t *full, uint64_t *empty, Place &p, unsigned slots, unsigned char *ring, const CUtensorMap *map,
                                int &used) {
                    if (!warp_wait(&empty[p.slot], p.phase ^ 1u)) return false;
                    if (lane == 0) mbar_expect_tx(&full[p.slot], bytes);
                    if (lane == (int)p.slot) used = (int)p.phase;
                    __syncwarp();
                    if (mine) tma_load_4d(ring + p.slot * kTile + lane * geo.box * HD, map, 0, from, head, at, &full[p.slot]);
                    p.next(slots);
                    return true;
                };
                ok = copy(x.k_full, x.k_empty, kp, geo.k_slots, kring, &kmap, used_k) &&
                     copy(x.v_full, x.v_empty, vp, geo.v_slots, vring, &vmap, used_v);
            }
        }
        if (!ok) give_up();
        // nothing may be in flight when the CTA exits
        volatile int never = 0;
        if (used_k >= 0) mbar_wait(&x.k_full[lane], (uint32_t)used_k, &never);
        if (used_v >= 0) mbar_wait(&x.v_full[lane], (uint32_t)used_v, &never);
    } else if (warp == kT8Mma) {
        // ---------------- S of every unit, up to two ahead of its softmax
        if (elect_one()) {
            const uint32_t id = idesc_e4m3_f32(kT8Keys, 2 * NR);
            unsigned u = 0, item = 0;
            int left = 0;
            Place kp = {0, 0};
            bool ok = true;
            while (ok) {
                if (left == 0) {
                    ok = mbar_wait(&x.item_full[item % kT8Items], item / kT8Items & 1u, ab);
                    if (!ok) break;
                    const PagedItem &it = x.item[item % kT8Items];
                    if (!it.more) break;
                    left = it.t1 - it.t0;
                    mbar_arrive(&x.item_empty[item % kT8Items]);
                    ok = mbar_wait(&x.q_full[item & 1], item >> 1 & 1u, ab);
                    ++item;
                }
                ok = ok && (u < 2 || mbar_wait(&x.p_full[u & 1], ((u - 2) >> 1) & 1u, ab)) &&   // S of unit u - 2 has been read
                     mbar_wait(&x.k_full[kp.slot], kp.phase, ab);
                if (!ok) break;
                tc_fence_after();
                const uint32_t ka = smem_u32(kring) + kp.slot * kTile, qa = smem_u32(qbuf) + ((item - 1) & 1) * kQ;
                const uint64_t kd = HD == 128 ? sdesc_kmajor_sw128(ka) : sdesc_kmajor_sw64(ka);
                const uint64_t qd = HD == 128 ? sdesc_kmajor_sw128(qa) : sdesc_kmajor_sw64(qa);
#pragma unroll
                for (int ks = 0; ks < HD / 32; ++ks)
                    tc_mma_e4m3(tmem + (u & 1) * 2 * NR, kd + (uint64_t)(ks * 2), qd + (uint64_t)(ks * 2), id, ks > 0);
                tc_commit(&x.s_full[u & 1]);
                tc_commit(&x.k_empty[kp.slot]);
                kp.next(geo.k_slots);
                ++u;
                if (--left == 0) tc_commit(&x.q_empty[(item - 1) & 1]);
            }
            if (!ok) give_up();
            volatile int never = 0;
            tc_commit(&x.done[0]);
            mbar_wait(&x.done[0], 0, &never);
        }
    } else if (warp == kT8Mma + 1) {
        // ---------------- O of every unit
        if (elect_one()) {
            const uint32_t id = idesc_f16_f32_mn(128, NR);
            unsigned u = 0, item = 0;
            int left = 0;
            bool ok = true, fresh = true;
            while (ok) {
                if (left == 0) {
                    ok = mbar_wait(&x.item_full[item % kT8Items], item / kT8Items & 1u, ab);
                    if (!ok) break;
                    const PagedItem &it = x.item[item % kT8Items];
                    if (!it.more) break;
                    left = it.t1 - it.t0;
                    mbar_arrive(&x.item_empty[item % kT8Items]);
                    ok = item < 2 || mbar_wait(&x.o_free[item & 1], ((item - 2) >> 1) & 1u, ab);
                    fresh = true;
                    ++item;
                }
                ok = ok && mbar_wait(&x.w_full[u & 1], u >> 1 & 1u, ab) && mbar_wait(&x.p_full[u & 1], u >> 1 & 1u, ab);
                if (!ok) break;
                tc_fence_after();
                // (64 dims: rows 64 .. 127 of the MMA repeat or run past the others, and are not read)
                const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(wide) + (u & 1) * kWide, 1024, H * 1024);
                const uint64_t pd = sdesc_mnmajor_sw128(smem_u32(pbuf) + (u & 1) * kP, 1024, 1024);
#pragma unroll
                for (int ks = 0; ks < kT8Keys / 16; ++ks)
                    tc_mma_bf16(tmem + 4 * NR + ((item - 1) & 1) * NR, vd + (uint64_t)(ks * 2 * H * 1024 >> 4),
                                pd + (uint64_t)(ks * 2 * 1024 >> 4), id, !fresh || ks > 0);
                fresh = false;
                tc_commit(&x.w_empty[u & 1]);
                tc_commit(&x.p_empty[u & 1]);
                ++u;
                --left;
            }
            if (!ok) give_up();
            volatile int never = 0;
            tc_commit(&x.done[1]);
            mbar_wait(&x.done[1], 0, &never);
        }
    } else if (warp >= kT8ConvWarp) {
        // ---------------- queries to pairs of codes; scales of every unit; V to FP16
        const int t = threadIdx.x - kT8Soft, cw = t >> 5, ps = a.kv.page_size;
        const bf16 *qp = static_cast<const bf16 *>(a.q);
        unsigned u0 = 0;   // units before this item
        Place vp = {0, 0};
        for (unsigned i = 0;; ++i) {
            bool ok = warp_wait(&x.item_full[i % kT8Items], i / kT8Items & 1u);
            if (t8_any<kT8Conv>(3, !ok)) {
                give_up();
                break;
            }
            const PagedItem &it = x.item[i % kT8Items];
            if (!it.more) break;
            const int units = it.t1 - it.t0, lo = it.lo, hi = it.hi, tile0 = it.t0, head = it.head;
            const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
            // queries: LPR threads a row, 8 dims each
            constexpr int LPR = HD / 8, RPP = kT8Conv / LPR, PASSES = NR / RPP > 0 ? NR / RPP : 1;
            const int sub = t % LPR;
            uint4 qw[PASSES];
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int r = p * RPP + t / LPR;
                qw[p] = make_uint4(0u, 0u, 0u, 0u);
                if (r < it.n_rows) {
                    const int row = it.row0 + r, tok = row / a.group, hd = row - tok * a.group;
                    qw[p] = *reinterpret_cast<const uint4 *>(qp + (long long)(it.token + tok) * a.q_stride +
                                                             (head * a.group + hd) * HD + sub * 8);
                }
            }
            // this thread's key of unit k: its page (-1: masked), its scales
            auto page_of = [&](int k) {
                const int j = (tile0 + k) * kT8Keys + t;
                if (k >= units || j < lo || j >= hi) return -1;
                const int p = table[geo.page_shift >= 0 ? j >> geo.page_shift : j / ps];
                return p < a.kv.n_pages ? p : -1;
            };
            struct Scales {
                float k, v;
                bool there;
            };
            auto scales = [&](int page, int k) {
                Scales s = {1.f, 1.f, page >= 0};
                if (page >= 0) {
                    const int j = (tile0 + k) * kT8Keys + t;
                    const int slot = geo.page_shift >= 0 ? j & (ps - 1) : j % ps;
                    const long long at = page * a.kv.scale_stride + slot / a.kv.block * a.kv.n_kv_heads + head;
                    s.k = a.kv.k_scale[at];
                    s.v = a.kv.v_scale[at];
                }
                return s;
            };
            auto publish = [&](const Scales &s, int k) {
                const unsigned u = u0 + k, slot = u % kT8Scales;
                ok = ok && warp_wait(&x.sc_empty[slot], (u / kT8Scales & 1u) ^ 1u);
                const float kc = fminf(kv8_scale(s.k) * a.scale_log2, 3.402823466e38f);
                x.sc[slot][t] = make_float2(kc, s.there ? log2f(kv8_scale(s.v)) : -INFINITY);
                const uint32_t bits = __ballot_sync(0xffffffffu, s.there);
                if (lane == 0) x.valid[slot][cw] = bits;
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.sc_full[slot]);
            };
            int page = page_of(0);
            Scales next = scales(page, 0);
            page = page_of(1);
            ok = ok && warp_wait(&x.q_empty[i & 1], (i >> 1 & 1u) ^ 1u);
            unsigned char *q8 = qbuf + (i & 1) * kQ;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int r = p * RPP + t / LPR;
                const uint32_t w[4] = {qw[p].x, qw[p].y, qw[p].z, qw[p].w};
                float y[8], top = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = __uint_as_float(w[e] << 16);
                    y[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fabsf(y[e]) <= 3.402823466e38f ? fmaxf(top, fabsf(y[e])) : top;
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                // the least power of two s with top <= 448 s
                const uint32_t b = __float_as_uint(top);
                const int ex = top > 0.f ? max((int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u), -126) : 0;
                const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
                uint32_t hi2[4], lo2[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y0 = fmaf(y[2 * e], 0.f, y[2 * e] * inv), y1 = fmaf(y[2 * e + 1], 0.f, y[2 * e + 1] * inv);   // (inf: NaN)
                    hi2[e] = t8_e4m3x2(y0, y1);
                    const uint32_t h = t8_f16x2(hi2[e]);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                    lo2[e] = t8_e4m3x2((y0 - f.x) * 16.f, (y1 - f.y) * 16.f);
                }
                if (r < NR) {   // (64 dims and 16 rows: one pass)
                    auto place = [&](int row) {   // of this thread's 8 bytes, in the swizzled tile
                        if (HD == 128) return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + (((sub >> 1) ^ (row & 7)) << 4) + (sub & 1) * 8);
                        return (uint32_t)((row >> 3) * 512 + (row & 7) * 64 + (((sub >> 1) ^ ((row >> 1) & 3)) << 4) + (sub & 1) * 8);
                    };
                    *reinterpret_cast<uint2 *>(q8 + place(r)) = make_uint2(hi2[0] | hi2[1] << 16, hi2[2] | hi2[3] << 16);
                    *reinterpret_cast<uint2 *>(q8 + place(NR + r)) = make_uint2(lo2[0] | lo2[1] << 16, lo2[2] | lo2[3] << 16);
                    if (sub == 0) x.q_scale[i % kT8Items][r] = __uint_as_float((uint32_t)(127 + ex) << 23);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.q_full[i & 1]);
            publish(next, 0);
            next = scales(page, 1);
            page = page_of(2);
            for (int k = 0; k < units; ++k) {
                const unsigned u = u0 + k;
                if (k + 1 < units) publish(next, k + 1);
                t8_sync<kT8Conv>(3);   // the valid keys of unit k are known
                next = scales(page, k + 2);   // on their way meanwhile
                page = page_of(k + 3);
                ok = ok && warp_wait(&x.v_full[vp.slot], vp.phase) && warp_wait(&x.w_empty[u & 1], (u >> 1 & 1u) ^ 1u);
                const unsigned char *src = vring + vp.slot * kTile;
                unsigned char *dst = wide + (u & 1) * kWide;
                constexpr int CPK = HD / 16, KPP = kT8Conv / CPK, TURNS = kT8Keys / KPP;   // 16-byte chunks of a key; keys of a turn
                const int c = t % CPK;
                uint4 in[TURNS];
#pragma unroll
                for (int y = 0; y < TURNS; ++y)
                    in[y] = *reinterpret_cast<const uint4 *>(src + (uint32_t)(y * KPP + t / CPK) * HD + c * 16);
#pragma unroll
                for (int y = 0; y < TURNS; ++y) {
                    const int key = y * KPP + t / CPK;
                    uint32_t w[4] = {in[y].x, in[y].y, in[y].z, in[y].w};
                    if (!(x.valid[u % kT8Scales][key >> 5] >> (key & 31) & 1u)) w[0] = w[1] = w[2] = w[3] = 0u;
                    uint32_t bad[4], any = 0u;   // NaN codes: 0x7f in the low seven bits
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        bad[e] = ((w[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                        any |= bad[e];
                    }
                    if (any) {
                        x.poison[i % kT8Items] = 1;
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] &= ~((bad[e] >> 7) * 0xffu);
                    }
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[2 * e] = t8_f16x2(w[e]);
                        h[2 * e + 1] = t8_f16x2(w[e] >> 16);
                    }
                    // rows of 128 bytes (64 dims), the second halves beside the first by groups of 8 keys; of
                    // the two 16-byte chunks the threads of the second half store the odd one first (banks)
                    const int half = c >> 2, c2 = (c & 3) * 2;
                    unsigned char *row = dst + (uint32_t)(key >> 3) * (H * 1024) + half * 1024 + (key & 7) * 128;
                    const uint4 h0 = make_uint4(h[0], h[1], h[2], h[3]), h1 = make_uint4(h[4], h[5], h[6], h[7]);
                    const bool odd = half != 0;
                    *reinterpret_cast<uint4 *>(row + (((c2 + odd) ^ (key & 7)) << 4)) = odd ? h1 : h0;
                    *reinterpret_cast<uint4 *>(row + (((c2 + !odd) ^ (key & 7)) << 4)) = odd ? h0 : h1;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&x.w_full[u & 1]);
                    mbar_arrive(&x.v_empty[vp.slot]);
                }
                vp.next(geo.v_slots);
            }
            u0 += units;
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.item_empty[i % kT8Items]);
            if (!ok) give_up();
        }
    } else {
        // ---------------- softmax and output: rows r0 .. r0 + NRH - 1; thread: key of S, dim of O
        constexpr int NRH = NR / 2, CH = NRH < 16 ? NRH : 16;   // rows of a read of TMEM
        const int g = warp >> 2, wq = warp & 3, key = 32 * wq + lane, r0 = g * NRH, bar = 1 + g, tg = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const int win = a.window > 0 ? a.window : 0x7fffffff;
        bf16 *out = static_cast<bf16 *>(a.out);
        auto load = [&](uint32_t at, uint32_t (&v)[CH]) {
            if constexpr (CH == 16) tmem_ld16_async(at, v);
            else tmem_ld8_async(at, v);
        };
        unsigned u0 = 0;   // units before this item
        for (unsigned i = 0;; ++i) {
            bool ok = warp_wait(&x.item_full[i % kT8Items], i / kT8Items & 1u);
            if (t8_any<128>(bar, !ok)) {
                give_up();
                break;
            }
            const PagedItem &it = x.item[i % kT8Items];
            if (!it.more) break;
            const int units = it.t1 - it.t0, tile0 = it.t0, n_rows = it.n_rows;
            const bool active = n_rows > r0;
            // the least and the greatest position of the tile's rows
            const int pos_a = max(it.pos0 + it.tok_a, -1), pos_b = max(it.pos0 + it.tok_b, -1);
            if (tg < NRH) {   // (rows that are not there are taken as the last one)
                const int r = r0 + tg, row = it.row0 + min(r, n_rows - 1), tok = row / a.group, hd = row - tok * a.group;
                x.pos[r] = max(it.pos0 + tok, -1);
                x.off[r] = (long long)(it.token + tok) * a.out_stride + (it.head * a.group + hd) * HD;
                x.neg_m[r] = INFINITY;
            }
            t8_sync<128>(bar);
            const float *qs = x.q_scale[i % kT8Items] + r0, *nm = x.neg_m + r0;
            const int *pos = x.pos + r0;
            const uint32_t t_o = tmem + lanes + 4 * NR + (i & 1) * NR + r0;
            uint64_t l[NRH / 2];
#pragma unroll
            for (int e = 0; e < NRH / 2; ++e) l[e] = 0ull;
#pragma unroll 1
            for (int k = 0; k < units; ++k) {
                const unsigned u = u0 + k;
                ok = ok && warp_wait(&x.sc_full[u % kT8Scales], u / kT8Scales & 1u);
                const float2 sc = x.sc[u % kT8Scales][key];
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.sc_empty[u % kT8Scales]);
                ok = ok && warp_wait(&x.s_full[u & 1], u >> 1 & 1u);
                if (active) {
                    tc_fence_after();
                    const int base = (tile0 + k) * kT8Keys, j = base + key;
                    const bool there = sc.y > -INFINITY;
                    // whether some rows see a key of the unit that others do not
                    const bool by_row = base + kT8Keys - 1 > pos_a || (a.window > 0 && base <= pos_b - win);
                    const bool mask = by_row || !__all_sync(0xffffffffu, there);
                    const uint32_t t_s = tmem + lanes + (u & 1) * 2 * NR + r0;
                    const uint64_t kc = pack_f32x2(sc.x, sc.x), lv = pack_f32x2(sc.y, sc.y), sixteenth = pack_f32x2(0.0625f, 0.0625f);
                    float y[NRH];
                    // t_rj, or with `less` t_rj - m_r
                    auto scores = [&](bool less) {
#pragma unroll
                        for (int q = 0; q < NRH; q += CH) {
                            uint32_t hi[CH], lo[CH];
                            load(t_s + q, hi);
                            load(t_s + NR + q, lo);
                            tmem_wait_ld<CH>(hi);
                            tmem_wait_ld<CH>(lo);
#pragma unroll
                            for (int e = 0; e < CH; e += 2) {
                                const uint64_t f = mul_f32x2(kc, *reinterpret_cast<const uint64_t *>(qs + q + e));
                                const uint64_t s = fma_f32x2(pack_f32x2(__uint_as_float(lo[e]), __uint_as_float(lo[e + 1])), sixteenth,
                                                             pack_f32x2(__uint_as_float(hi[e]), __uint_as_float(hi[e + 1])));
                                const uint64_t add = less ? add_f32x2(lv, *reinterpret_cast<const uint64_t *>(nm + q + e)) : lv;
                                const float2 v = unpack_f32x2(fma_f32x2(s, f, add));
                                y[q + e] = v.x;
                                y[q + e + 1] = v.y;
                            }
                        }
                        if (mask) {
#pragma unroll
                            for (int e = 0; e < NRH; ++e) {
                                const int p = pos[e];
                                const bool see = there && (!by_row || (j <= p && j > p - win));
                                y[e] = see ? y[e] : -INFINITY;
                            }
                        }
                    };
                    bool move = k == 0;
                    if (k > 0) {
                        scores(true);
                        float top = -INFINITY;
#pragma unroll
                        for (int e = 0; e < NRH; ++e) top = fmaxf(top, y[e]);
                        move = t8_any<128>(bar, top > kT8Most);
                    }
                    if (move) {   // some row's weights outgrow its m
                        scores(false);
                        int mine = 0;
#pragma unroll
                        for (int e = 0; e < NRH; ++e) {
                            // the largest over the warp's keys, as integers in the order of the floats (NaN as -inf)
                            const int b = __float_as_int(fmaxf(y[e], -INFINITY));
                            const int top = __reduce_max_sync(0xffffffffu, b ^ (b >> 31 & 0x7fffffff));
                            if (lane == e) mine = top;
                        }
                        if (lane < NRH) x.part[warp][lane] = __int_as_float(mine ^ (mine >> 31 & 0x7fffffff));
                        t8_sync<128>(bar);
                        if (tg < NRH) {
                            const int w0 = g * 4;
                            const float top = fmaxf(fmaxf(x.part[w0][tg], x.part[w0 + 1][tg]), fmaxf(x.part[w0 + 2][tg], x.part[w0 + 3][tg]));
                            const float old = -x.neg_m[r0 + tg];   // -inf: none yet
                            const bool up = top > -INFINITY && (k == 0 || top > old + kT8Most);
                            x.factor[r0 + tg] = up ? t8_ex2(old - (top - kT8Off)) : 1.f;
                            if (up) x.neg_m[r0 + tg] = kT8Off - top;
                        }
                        t8_sync<128>(bar);
                        if (k > 0) {
                            // O of the units before
                            ok = ok && warp_wait(&x.p_empty[(u - 1) & 1], ((u - 1) >> 1) & 1u);
                            tc_fence_after();
#pragma unroll
                            for (int q = 0; q < NRH; q += CH) {
                                uint32_t o[CH];
                                load(t_o + q, o);
                                tmem_wait_ld<CH>(o);
#pragma unroll
                                for (int e = 0; e < CH; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * x.factor[r0 + q + e]);
#pragma unroll
                                for (int e = 0; e < CH; e += 8) tmem_st8(t_o + q + e, o + e);
                            }
                            tmem_wait_st();
#pragma unroll
                            for (int e = 0; e < NRH; e += 2)
                                l[e / 2] = mul_f32x2(l[e / 2], *reinterpret_cast<const uint64_t *>(x.factor + r0 + e));
                        }
#pragma unroll
                        for (int e = 0; e < NRH; ++e) {
                            const float n = nm[e];
                            y[e] += n == INFINITY ? 0.f : n;   // (no key yet: every score is -inf or NaN)
                        }
                    }
                    const float r = there ? t8_ex2(-sc.y) : 0.f;   // 1 / vs
                    const uint64_t rr = pack_f32x2(r, r);
                    if (u >= 2) ok = ok && warp_wait(&x.p_empty[u & 1], ((u - 2) >> 1) & 1u);
                    unsigned char *prow = pbuf + (u & 1) * kP + (uint32_t)(key >> 3) * 1024 + (key & 7) * 128;
#pragma unroll
                    for (int q = 0; q < NRH; q += 8) {
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float p0 = t8_ex2(y[q + 2 * e]), p1 = t8_ex2(y[q + 2 * e + 1]);
                            l[q / 2 + e] = fma_f32x2(pack_f32x2(p0, p1), rr, l[q / 2 + e]);
                            const __half2 pk = __floats2half2_rn(p0, p1);
                            h[e] = *reinterpret_cast<const uint32_t *>(&pk);
                        }
                        *reinterpret_cast<uint4 *>(prow + ((((r0 + q) >> 3) ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    fence_proxy_async_smem();   // before the MMA reads them
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.p_full[u & 1]);
            }
            u0 += units;
            // ---- the item's rows.  O is complete with its last unit's (waited for by both halves: neither
            // runs ahead of the other by more than an item)
            const unsigned last = u0 - 1;
            if (active) {
                // row sums over the warp's keys: at each step a lane keeps half of its rows
                float v[NRH];
#pragma unroll
                for (int e = 0; e < NRH / 2; ++e) {
                    const float2 f = unpack_f32x2(l[e]);
                    v[2 * e] = f.x;
                    v[2 * e + 1] = f.y;
                }
#pragma unroll
                for (int n = NRH / 2, o = 16; n >= 1; n /= 2, o /= 2) {
                    const bool up = lane & o;
#pragma unroll
                    for (int e = 0; e < n; ++e) {
                        const float send = up ? v[e] : v[e + n], keep = up ? v[e + n] : v[e];
                        v[e] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                }
                constexpr int REP = 32 / NRH;   // lanes that hold the same row
#pragma unroll
                for (int o = REP / 2; o > 0; o >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                if (lane % REP == 0) x.part[warp][lane / REP] = v[0];
                t8_sync<128>(bar);
                const bool part = it.part >= 0;
                if (tg < NRH) {
                    const int w0 = g * 4, r = r0 + tg;
                    const float sum = (x.part[w0][tg] + x.part[w0 + 1][tg]) + (x.part[w0 + 2][tg] + x.part[w0 + 3][tg]);
                    if (part && r < n_rows) {
                        float *ml = reinterpret_cast<float *>(a.ws + lay.ml) + ((size_t)it.part * a.rows + r) * 2;
                        ml[0] = -x.neg_m[r];
                        ml[1] = sum;
                    }
                    x.factor[r] = part ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                }
                t8_sync<128>(bar);
                ok = ok && warp_wait(&x.p_empty[last & 1], last >> 1 & 1u);
                tc_fence_after();
                if (32 * wq < HD) {   // thread: dim `key`
                    uint32_t nan = 0u;   // rows that see a key whose V is NaN in this dim
                    if (*const_cast<volatile int *>(&x.poison[i % kT8Items])) {
                        const int j0 = max(it.lo, tile0 * kT8Keys), j1 = min(it.hi, it.t1 * kT8Keys);
#pragma unroll 1
                        for (int j = j0; j < j1; ++j) {
                            const int page = key_page(a, a.s.table + (long long)it.seq * a.s.table_stride, j);
                            if (page < 0) continue;
                            const uint8_t code = static_cast<const uint8_t *>(a.kv.v)[page * a.kv.page_stride + (j % a.kv.page_size) * a.kv.slot_stride +
                                                                                      it.head * a.kv.head_stride + key];
                            if ((code & 0x7fu) != 0x7fu) continue;
#pragma unroll 1
                            for (int e = 0; e < NRH; ++e)
                                if (j <= pos[e] && j > pos[e] - win) nan |= 1u << e;
                        }
                    }
                    float *po = reinterpret_cast<float *>(a.ws + lay.o) + ((size_t)it.part * a.rows + r0) * HD + key;
#pragma unroll
                    for (int q = 0; q < NRH; q += CH) {
                        uint32_t o[CH];
                        load(t_o + q, o);
                        tmem_wait_ld<CH>(o);
#pragma unroll
                        for (int e = 0; e < CH; ++e) {
                            const int r = r0 + q + e;
                            if (r >= n_rows) break;
                            float f = __uint_as_float(o[e]) * x.factor[r];
                            if (nan >> (q + e) & 1u) f = NAN;
                            if (part) po[(q + e) * HD] = f;
                            else out[x.off[r] + key] = __float2bfloat16_rn(f);
                        }
                    }
                }
            } else {
                ok = ok && warp_wait(&x.p_empty[last & 1], last >> 1 & 1u);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&x.o_free[i & 1]);
                mbar_arrive(&x.item_empty[i % kT8Items]);
            }
            if (!ok) give_up();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kT8Mma) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// ------------------------------------------------------------------ host side

static int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <int HD, int NR>
static cudaError_t t8_go(AttnArgs &a, T8Geometry &g, const CUtensorMap &km, const CUtensorMap &vm, int grid, cudaStream_t st)
{
    const int tile = HD * kT8Keys, fixed = 2 * 2 * tile + 2 * kT8Keys * 128 + 2 * 2 * NR * HD + (int)sizeof(T8Misc);
    static_assert(2 * 2 * HD * kT8Keys + 2 * kT8Keys * 128 + 2 * 2 * NR * HD + sizeof(T8Misc) + 4 * HD * kT8Keys <= kT8Smem,
                  "two tiles of K and of V beside the buffers");
    int slots = (kT8Smem - fixed) / tile;
    if (slots > 2 * kT8MaxSlots) slots = 2 * kT8MaxSlots;
    g.k_slots = (slots + 1) / 2;
    g.v_slots = slots / 2;
    static PerDevice once;
    auto kernel = k_paged_attn8_tc<HD, NR>;
    cudaError_t e = allow_once(once, kernel, kT8Smem);
    if (e) return e;
    return launch_pdl(kernel, dim3(grid), dim3(kT8Threads), (size_t)(fixed + slots * tile), st, km, vm, a, g);
}

cudaError_t paged_attn8_tc(AttnArgs &a, cudaStream_t st, int nsm)
{
    const int hd = a.kv.head_dim;
    T8Geometry g = {};
    g.box = gcd(a.kv.page_size, kT8Keys);
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (1 << i == a.kv.page_size) g.page_shift = i;
    CUtensorMap km, vm;
    const long long dims[4] = {hd, a.kv.page_size, a.kv.n_kv_heads, a.kv.n_pages};
    const long long strides[3] = {a.kv.slot_stride, a.kv.head_stride, a.kv.page_stride};
    const int box[4] = {hd, g.box, 1, 1};
    cudaError_t e = tc::make_map_u8_nd(&km, a.kv.k, 4, dims, strides, box, hd);
    if (!e) e = tc::make_map_u8_nd(&vm, a.kv.v, 4, dims, strides, box, 0);
    if (e) return e;
    const int grid = paged_attn_grid(a, kT8Keys, nsm < kAttnMaxCtasTc ? nsm : kAttnMaxCtasTc);
    if (hd == 64)
        e = a.rows <= 16   ? t8_go<64, 16>(a, g, km, vm, grid, st)
            : a.rows <= 32 ? t8_go<64, 32>(a, g, km, vm, grid, st)
                           : t8_go<64, 64>(a, g, km, vm, grid, st);
    else
        e = a.rows <= 16   ? t8_go<128, 16>(a, g, km, vm, grid, st)
            : a.rows <= 32 ? t8_go<128, 32>(a, g, km, vm, grid, st)
                           : t8_go<128, 64>(a, g, km, vm, grid, st);
    if (!e && !a.whole) e = paged_join_tc(a, grid, nsm, st);
    return e;
}

}  // namespace ds4g
