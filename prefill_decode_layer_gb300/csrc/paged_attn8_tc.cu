// Tensor-core form of the paged attention over a cache in 8 bits (tcgen05 MMAs with TMEM
// accumulators, TMA tiles of the cache's pages): page "ds4.c 学习笔记 -- 端到端推理流程", 阶段四
// 4.2.  The division of the work is paged_sched.cuh's; BF16 queries, head_dim 64 or 128.
//
// With K_j = ks_j k_j and V_j = vs_j v_j (codes k, v; scales ks, vs of key j's block), row r is
//   out_r = sum_j p_rj v_j / sum_j p_rj / vs_j,
//   p_rj = 2^(t_rj - m_r),  t_rj = (scale log2 e) ks_j (q_r . k_j) + log2 vs_j,
// so that the scales are two numbers a key, and m_r (the running maximum of t_rj, less an offset) bounds
// what p_rj v_j adds to the row whatever the scales are.
//
// Both products have the keys on the MMA's M side, or the dims, and the query rows on its N
// side: with the few rows of a decode step the tensor cores' time then falls with the rows, and the
// softmax's work is spread over all 128 keys of a unit:
//   S^T = K Q^T    M 128 keys x N rows.  K's codes go from their TMA tile into the MMA as they are
//                  (kind::f8f6f4).  A BF16 query is the sum of two E4M3 values, exactly: of
//                  x in units of the row's power of two, hi = E4M3(x) holds 4 of its 8 bits and
//                  16 (x - hi) the others.  The two are 2 x rows columns of one MMA;
//   softmax        a thread owns a key and 8 or 16 rows; it adds the two halves, applies scales and
//                  masks and writes P^T to shared memory.  m_r moves only when a weight would exceed
//                  the largest that fits: nothing is reduced over keys in most units.  Row sums are
//                  kept per key and thread in FP32 and added up when the item ends;
//   O^T += V^T P^T M 128 dims x N rows, in one of two ways.
// Up to 32 rows ("direct"): V's codes from their TMA tile as they are, and P as E4M3 too, four columns a
// row: a weight p as hi + lo / 16 like the queries, and weights below 2^-10 of the maximum in a pair of
// columns of their own, in units of 2^-13 (E4M3 alone has 2^-9 .. 448: many small weights beside a large one would
// vanish).  2^-9 of each weight, or 2^-32 of the largest.
// More rows: four times the columns of 64 rows, twice over, do not fit TMEM.  Four warps make FP16 of V's
// codes, which holds them exactly, and P is FP16 (2^-11, or 2^-34 of the largest).  (With that for every number of
// rows the batch below took 222 us, not 167, the long one 246, not 199.)
//
// Units of two K/V heads where their rows fit a group of softmax threads each: see paged_attn8_tc_heads.
//
// Bound and figures (device time, of a captured graph; the copy 6.79 TB/s):
//   one token of 64 sequences to 8191, 32 heads on 8 (0.69 GB)       114 us   DRAM, 6.0 TB/s
//   one token of 4 sequences to 131072, 64 heads on 8 (0.81 GB)      129 us   DRAM, 6.3 TB/s
//   1 to 5 tokens of 32 sequences to 16994, 64 heads on 1 (92 MB)     90 us   instruction issue (0.61 of the slots:
//     the softmax's 16 warps, V's conversion) and the chains of a unit, 2500 cycles for 128 keys and 64 rows;
//     shared memory, 176 KB of a unit, would take 1400, the MMAs 480
//   one token, 64 heads on 1, a window of 128                         9.8 us  latency: launch, item, page, K, softmax, O
// The K and V tiles are most of shared memory (five of two heads, 32 KB each, at eight rows; eleven of one), so that
// the copies run far ahead of the MMAs.
//
// Masked places: a key outside the item's keys or in a missing page, or hidden from a row, gets the
// weight 0.  In units at an edge (of the item's keys, or of what some rows see) the rows of V outside the
// item's keys are zeroed in the tile, and NaN codes of keys that only some rows see become 0; rows
// that see such a key get their NaN when the item ends.
//
// Roles (one CTA per SM): one to four groups of four warps, softmax and output of 8 or 16 rows each; four
// warps for the queries' codes and V's tiles; one warp each for the items and TMA copies, the MMAs of S, the
// MMAs of O (one thread each) and the scales.  Page look-ups and scales are fetched for 32 boxes or blocks at
// a time, one round ahead.  Every wait is bounded; a CTA that gives up says so in its status word, drains
// its copies and MMAs, frees its TMEM and returns.
//
// Code that runs once a unit is kept small (rolled loops, one place for each wait): in a first form with 32
// rows a thread, 174 KB of instructions, a fifth of the warps' time went to fetching them.
#include <cuda.h>
#include <cuda_fp16.h>
#include <stddef.h>

#include "paged_sched.cuh"
#include "sm100.cuh"
#include "tc_gemm.cuh"

namespace ds4g {

static constexpr int kT8Keys = 128;                    // keys of a unit
static constexpr int kT8Rows = 64;                     // query rows of a tile at most
static constexpr int kT8MaxSlots = 6;                  // tiles of K, and of V, at most
static constexpr int kT8Items = 4;                     // items ahead of the softmax at most
static constexpr int kT8Scales = 4;                    // rounds of scales that are there at most
static constexpr int kT8Smem = 227 * 1024;

// What follows from the columns of query rows NR (8, 16, 32 or 64) and the K/V heads HP of a kernel's units.
template <int NR, int HP> struct T8 {
    static constexpr bool direct = NR <= 32;
    static constexpr int own = NR < 16 ? NR : 16;      // rows of a softmax thread
    static constexpr int groups = HP * (NR / own);
    static constexpr int soft = groups * 128;          // softmax threads
    static constexpr int conv = groups * 4;            // warps: the first of the queries and V's tiles, then ..
    static constexpr int tma = conv + 4, mma_s = tma + 2, mma_o = tma + 3, scale = tma + 4;   // (tma: K's copies and the items, tma + 1: V's)
    static constexpr int threads = (scale + 1) * 32;
    static constexpr int s_head = 2 * NR, o_head = direct ? 4 * NR : NR;   // columns of a head: of a unit, of an item
    static constexpr int s_cols = HP * s_head, o_cols = HP * o_head;
    static constexpr int cols = 2 * s_cols + 2 * o_cols <= 128 ? 128 : 2 * s_cols + 2 * o_cols <= 256 ? 256 : 512;
    // log2 of the largest weight when m is set, and of the largest that fits
    static constexpr float off = direct ? 5.f : 9.f, most = direct ? 8.f : 15.f;
    static_assert(HP == 1 || (direct && NR == own), "of two heads each has a group");
};

struct T8Misc {
    uint64_t k_full[kT8MaxSlots], k_empty[kT8MaxSlots], v_full[kT8MaxSlots], v_empty[kT8MaxSlots];
    uint64_t w_full[kT8MaxSlots], w_empty[2];          // V's tile may be used: by slot, or of unit u % 2 in FP16
    uint64_t sc_full[kT8Scales], sc_empty[kT8Scales];
    uint64_t q_full[2], q_empty[2];                    // of item i % 2
    uint64_t s_full[2], p_full[2], p_empty[2];         // of unit u % 2
    uint64_t o_free[2];                                // of item i % 2: its O has been read
    uint64_t item_full[kT8Items], item_empty[kT8Items];
    uint64_t done[2];
    PagedItem item[kT8Items];
    PagedCursor cur;
    long long scratch[25];
    float2 sc[kT8Scales][2][kT8Keys];                  // of a round's blocks, by head: ks scale log2 e, log2 vs (-inf: no page)
    int poison[kT8Items];                              // a V row of the item has a NaN that was taken out
    uint32_t tmem;
    int abort_flag;
    __align__(16) float q_scale[kT8Items][kT8Rows];    // of an item's rows
    __align__(16) float neg_m[kT8Rows], factor[kT8Rows], delta[kT8Rows];
    __align__(16) float again[kT8Rows];                // the row sums' second factor
    float part[16][16];                                // of a softmax warp: a value of each row
    int pos[kT8Rows], set[kT8Rows], row[kT8Rows];      // of a row: its position; it has an m; its place among the item's
    long long off[kT8Rows], q_off[kT8Rows];            // of a row in the output; in the queries (-1: none)
};

struct T8Geometry {
    int k_slots, v_slots;
    int box;         // slots of a page in one copy: gcd(page_size, 128)
    int page_shift;  // log2(page_size), or -1
    // scales: one for every 2^gran keys of a unit at least (the part of the block size that divides 128), so
    // many a unit, and the units of a round: 32 scales, or one unit where it has more
    int gran, per_unit, round;
    int group, n_heads;   // query heads of a K/V head, K/V heads (AttnArgs' are those of a unit's heads taken as one)
};

bool paged_attn8_tc_ok(const PagedKV &kv, int q_dtype)
{
    return q_dtype == DS4G_BF16 && (kv.head_dim == 64 || kv.head_dim == 128) && kv.page_size % 8 == 0;
}

// K/V heads of a unit: two where their rows fit a group each.  A head's rows of a tile are 128 bytes (64) apart by all
// heads; two heads' are read side by side, which DRAM serves better, and a unit's waits serve twice the bytes.  (64
// sequences to 8191 with 32 heads on 8: 127 us with one head a unit, 116 with two; 4 to 131072 with 64 on 8: 157, and
// 136 to 163 on other devices, and 129.  More rows than a group's 16 would take a third and a fourth group beside them.)
int paged_attn8_tc_heads(int n_kv_heads, int group, int max_new)
{
    return n_kv_heads % 2 == 0 && group <= 16 && group * max_new <= 16 ? 2 : 1;
}
// Query rows of a tile: as few tiles as hold them, of equal size.
int paged_attn8_tc_rows(int n_kv_heads, int group, int max_new)
{
    const int rows = group * max_new, tiles = (rows + kT8Rows - 1) / kT8Rows;
    return paged_attn8_tc_heads(n_kv_heads, group, max_new) * ((rows + tiles - 1) / tiles);
}

// mbar_wait that looks once without sleeping (a wait that is over costs 60 cycles then, and 200 with the form
// that may sleep), and then sleeps for up to 0.1 ms at a time: warps that poll take issue slots from those that work.
__device__ __forceinline__ bool t8_wait(uint64_t *b, uint32_t parity, volatile int *abort_flag)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    if (ok) return true;
    const long long t0 = clock64();
    while (true) {
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
            " selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(smem_u32(b)), "r"(parity), "r"(100000u)
            : "memory");
        if (ok) return true;
        if (*abort_flag || clock64() - t0 > kWaitCycles) return false;
    }
}
__device__ __forceinline__ uint32_t t8_e4m3x2(float lo, float hi)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t t8_e4m3x2(__half2 v)
{
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&v)));
    return r;
}
__device__ __forceinline__ uint32_t t8_f16x2(uint32_t codes)   // of the low two bytes
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)codes));
    return h;
}
__device__ __forceinline__ float2 t8_floats(uint32_t codes)
{
    const uint32_t h = t8_f16x2(codes);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// NaN codes among four (0x7f in the low seven bits) become 0; true if there was one.
__device__ __forceinline__ bool t8_no_nan(uint32_t &w)
{
    const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    w &= ~((nan >> 7) * 0xffu);
    return nan != 0u;
}
__device__ __forceinline__ float t8_max3(float a, float b, float c)
{
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));   // (the number beside a NaN)
    return m;
}
// Two values as codes, and 16 times what the codes leave of them.
__device__ __forceinline__ void t8_split(float a, float b, uint32_t &hi, uint32_t &lo)
{
    hi = t8_e4m3x2(a, b);
    const float2 f = t8_floats(hi);
    lo = t8_e4m3x2((a - f.x) * 16.f, (b - f.y) * 16.f);
}
// Barrier `id` of the 128 threads that use it, which tells each whether any of them says so.
__device__ __forceinline__ bool t8_any(int id, bool yes)
{
    uint32_t any;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, 128, q;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(any)
        : "r"((uint32_t)yes), "r"(id)
        : "memory");
    return any != 0;
}
__device__ __forceinline__ void t8_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ float t8_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two rows' values of an array of floats in shared memory.
__device__ __forceinline__ ulonglong2 t8_rows4(const float *p) { return *reinterpret_cast<const ulonglong2 *>(p); }

// v[e] over the warp's lanes, the largest or the sum; at each step a lane keeps half of the rows, so that lane i
// ends with row i / (32 / N), in v[0].
template <bool MAX, int N> __device__ __forceinline__ void t8_over_warp(float (&v)[N])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = N / 2, o = 16; n >= 1; n /= 2, o /= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int e = 0; e < n; ++e) {
            const float send = up ? v[e] : v[e + n], keep = up ? v[e + n] : v[e], got = __shfl_xor_sync(0xffffffffu, send, o);
            v[e] = MAX ? fmaxf(keep, got) : keep + got;
        }
    }
#pragma unroll
    for (int o = 16 / N; o > 0; o >>= 1) {
        const float got = __shfl_xor_sync(0xffffffffu, v[0], o);
        v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
    }
}

// The least and the greatest position of an item's rows.
__device__ __forceinline__ int2 t8_ends(const PagedItem &it)
{
    return make_int2(max(it.pos0 + it.tok_a, -1), max(it.pos0 + it.tok_b, -1));
}
// Whether some of its rows see a key of the unit from `base` that others do not.  (Rows of one token: no.  Its
// keys are the item's.)
__device__ __forceinline__ bool t8_by_row(int2 ends, int base, int window)
{
    return ends.x != ends.y && (base + kT8Keys - 1 > ends.x || (window > 0 && base <= ends.y - window));
}

// A place in a ring (kept up to date: no division at every use).
struct T8Place {
    unsigned slot, phase;
    __device__ __forceinline__ void next(unsigned slots)
    {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// HD: head_dim.  NR: columns of a head's query rows, its rows of a tile or more.  HP: K/V heads of a unit.
template <int HD, int NR, int HP>
__global__ void __launch_bounds__(T8<NR, HP>::threads, 1)
    k_paged_attn8_tc(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ AttnArgs a, const __grid_constant__ T8Geometry geo)
{
    using P = T8<NR, HP>;
    constexpr bool kDirect = P::direct;
    constexpr int H = HD / 64;                          // 128-byte blocks of an FP16 row
    constexpr uint32_t kGroup = 8 * HD;                 // bytes of 8 keys of a head: [16 groups][HP heads][8 keys][HD] is ..
    constexpr uint32_t kTile = HP * HD * kT8Keys;       // .. a K or V tile of codes
    constexpr uint32_t kWide = kDirect ? 0 : 2 * kTile; // of V in FP16
    constexpr uint32_t kQhead = 2 * NR * HD, kQ = HP * kQhead, kP = kT8Keys * 128;
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
            if (in(x.w_full, kT8MaxSlots) || in(x.q_full, 2)) count = 4;
            else if (in(x.v_empty, kT8MaxSlots)) count = kDirect ? 5 : 4;
            else if (in(x.sc_empty, kT8Scales) || in(x.p_full, 2) || in(x.o_free, 2)) count = 4 * P::groups;
            else if (in(x.item_empty, kT8Items)) count = 4 * P::groups + 4 + 4;
            mbar_init(bars + i, count);
        } else if (i == n) {
            x.abort_flag = 0;
        }
        mbar_fence_init();
    }
    if (warp == P::mma_s) tmem_alloc(&x.tmem, P::cols);
    if (threadIdx.x == P::tma * 32) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_trigger();
    paged_begin(a, lay);
    const bool few = a.s.n_seqs <= 32;   // the copying warp finds the CTA's share by itself
    if (!few) paged_cursor<P::threads>(a, kT8Keys, &x.cur, x.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x.tmem, tmem_o = tmem + 2 * P::s_cols;   // S of unit u % 2; O of item i % 2
    volatile int *ab = &x.abort_flag;
    auto give_up = [&]() {
        x.abort_flag = 1;
        reinterpret_cast<int *>(a.ws + lay.status)[blockIdx.x] = kAttnTimedOut;
    };
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, t8_wait(bar, parity, ab)) != 0;
    };

    if (warp == P::tma || warp == P::tma + 1) {
        // ---------------- page look-ups and copies, of K or of V; the first of the two finds the items
        const bool is_v = warp != P::tma;
        PagedCursor cur;
        if (!is_v) {
            if (few) paged_cursor_warp(a, kT8Keys, cur);
            else cur = x.cur;
        }
        const int boxes = kT8Keys / geo.box, ps = a.kv.page_size;
        const CUtensorMap *map = is_v ? &vmap : &kmap;
        uint64_t *full = is_v ? x.v_full : x.k_full, *empty = is_v ? x.v_empty : x.k_empty;
        unsigned char *ring = is_v ? vring : kring;
        const unsigned slots = is_v ? geo.v_slots : geo.k_slots;
        int used = -1;   // lane i: the phase of the last load into slot i
        T8Place p = {0, 0};
        bool ok = true;
        for (unsigned i = 0; ok; ++i) {
            ok = warp_wait(is_v ? &x.item_full[i % kT8Items] : &x.item_empty[i % kT8Items], (i / kT8Items & 1u) ^ (is_v ? 0u : 1u));
            if (!ok) break;
            PagedItem &it = x.item[i % kT8Items];
            if (!is_v && lane == 0) {
                paged_next(a, kT8Keys, cur, lay, it);
                x.poison[i % kT8Items] = 0;
                mbar_arrive(&x.item_full[i % kT8Items]);
            }
            __syncwarp();
            if (!it.more) break;
            const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
            const int lo = it.lo, hi = it.hi, head = it.head * HP, t0 = it.t0, t1 = it.t1;
            if (is_v) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.item_empty[i % kT8Items]);
            }
            // a look-up is of 32 boxes: the lane's box of the group of tiles from tg, its page and first slot
            const int group = 32 / boxes, my_tile = lane / boxes, my_box = lane - my_tile * boxes;
            int page = -1, slot = 0, at = 0, from = 0, in_group = group;
            uint32_t loads = 0;
            bool load = false;
            // (two look-ups before the first tile, then one at the first tile of every group)
#pragma unroll 1
            for (int t = t0 - group; ok && t < t1; ++t, ++in_group) {
                if (in_group == group) {
                    // a page that is not there: out of bounds, read as zeros
                    at = page < 0 || page >= a.kv.n_pages ? a.kv.n_pages : page;
                    from = slot >> 3;
                    loads = __ballot_sync(0xffffffffu, load);
                    // the next group's, on its way meanwhile
                    const int tile = t + group + my_tile, j = tile * kT8Keys + my_box * geo.box;
                    load = tile < t1 && j < hi && j + geo.box > lo;
                    if (load) {
                        const int q = geo.page_shift >= 0 ? j >> geo.page_shift : j / ps;
                        slot = j - q * ps;
                        page = table[q];
                    }
                    in_group = 0;
                    if (t < t0) {
                        t = t0 - 1;
                        in_group = group - 1;
                        continue;
                    }
                }
                ok = warp_wait(empty + p.slot, p.phase ^ 1u);
                if (!ok) break;
                // one lane issues them all (the compiler then sees uniform operands), four at a time
                const uint32_t tile = loads >> (in_group * boxes) & ((1u << boxes) - 1u);
                if (lane == (int)p.slot) used = (int)p.phase;
                unsigned char *dst = ring + p.slot * kTile;
                const bool one = elect_one();
                if (one) mbar_expect_tx(full + p.slot, (uint32_t)__popc(tile) * geo.box * (HP * HD));
#pragma unroll 1
                for (int b = 0; b < boxes; b += 4) {
                    int at_b[4], from_b[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        at_b[z] = __shfl_sync(0xffffffffu, at, in_group * boxes + b + z);   // (past the tile's boxes: not used)
                        from_b[z] = __shfl_sync(0xffffffffu, from, in_group * boxes + b + z);
                    }
                    if (one) {
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            if (tile >> (b + z) & 1u)
                                tma_load_5d(dst + (b + z) * geo.box * (HP * HD), map, 0, 0, head, from_b[z], at_b[z], full + p.slot);
                    }
                }
                p.next(slots);
            }
        }
        if (!ok) give_up();
        // nothing may be in flight when the CTA exits
        volatile int never = 0;
        if (used >= 0) mbar_wait(full + lane, (uint32_t)used, &never);
    } else if (warp == P::mma_s) {
        // ---------------- S of every unit, up to two ahead of its softmax
        if (elect_one()) {
            const uint32_t id = idesc_e4m3_f32(kT8Keys, P::s_head);
            unsigned u = 0, item = 0;
            int left = 0;
            T8Place kp = {0, 0};
            bool ok = true;
            while (ok) {
                if (left == 0) {
                    ok = t8_wait(&x.item_full[item % kT8Items], item / kT8Items & 1u, ab);
                    if (!ok) break;
                    const PagedItem &it = x.item[item % kT8Items];
                    if (!it.more) break;
                    left = it.t1 - it.t0;
                    mbar_arrive(&x.item_empty[item % kT8Items]);
                    ok = t8_wait(&x.q_full[item & 1], item >> 1 & 1u, ab);
                    ++item;
                }
                ok = ok && (u < 2 || t8_wait(&x.p_full[u & 1], ((u - 2) >> 1) & 1u, ab)) &&   // S of unit u - 2 has been read
                     t8_wait(&x.k_full[kp.slot], kp.phase, ab);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    const uint32_t ka = smem_u32(kring) + kp.slot * kTile + h * kGroup, qa = smem_u32(qbuf) + ((item - 1) & 1) * kQ + h * kQhead;
                    const uint64_t kd = HD == 128 ? sdesc_kmajor_sw128(ka, HP * kGroup) : sdesc_kmajor_sw64(ka, HP * kGroup);
                    const uint64_t qd = HD == 128 ? sdesc_kmajor_sw128(qa, kGroup) : sdesc_kmajor_sw64(qa, kGroup);
#pragma unroll
                    for (int ks = 0; ks < HD / 32; ++ks)
                        tc_mma_e4m3(tmem + (u & 1) * P::s_cols + h * P::s_head, kd + (uint64_t)(ks * 2), qd + (uint64_t)(ks * 2), id, ks > 0);
                }
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
    } else if (warp == P::mma_o) {
        // ---------------- O of every unit
        if (elect_one()) {
            const uint32_t id = kDirect ? idesc_e4m3_f32_mn(128, P::o_head) : idesc_f16_f32_mn(128, P::o_head);
            unsigned u = 0, item = 0;
            int left = 0, base = 0, lo = 0, hi = 0;
            int2 ends = make_int2(0, 0);
            T8Place vp = {0, 0};
            bool ok = true, fresh = true;
            while (ok) {
                if (left == 0) {
                    ok = t8_wait(&x.item_full[item % kT8Items], item / kT8Items & 1u, ab);
                    if (!ok) break;
                    const PagedItem &it = x.item[item % kT8Items];
                    if (!it.more) break;
                    left = it.t1 - it.t0;
                    base = it.t0 * kT8Keys;
                    lo = it.lo;
                    hi = it.hi;
                    ends = t8_ends(it);
                    mbar_arrive(&x.item_empty[item % kT8Items]);
                    ok = item < 2 || t8_wait(&x.o_free[item & 1], ((item - 2) >> 1) & 1u, ab);
                    fresh = true;
                    ++item;
                }
                const uint32_t d = tmem_o + ((item - 1) & 1) * P::o_cols, pa = smem_u32(pbuf) + (u & 1) * kP;
                if (kDirect) {
                    const bool edge = base < lo || base + kT8Keys > hi || t8_by_row(ends, base, a.window);
                    ok = ok && t8_wait(&x.v_full[vp.slot], vp.phase, ab) &&
                         (!edge || t8_wait(&x.w_full[vp.slot], vp.phase, ab)) && t8_wait(&x.p_full[u & 1], u >> 1 & 1u, ab);
                    if (!ok) break;
                    tc_fence_after();
                    // (64 dims: rows 64 .. 127 of the MMA run on into what lies behind, and are not read)
#pragma unroll
                    for (int h = 0; h < HP; ++h) {
                        const uint32_t va = smem_u32(vring) + vp.slot * kTile + h * kGroup;
                        const uint64_t vd = HD == 128 ? sdesc_mnmajor_sw128(va, 1024, HP * kGroup) : sdesc_mnmajor_sw64(va, 512, HP * kGroup);
                        const uint64_t pd = sdesc_mnmajor_sw128(pa + h * P::o_head, 1024, 1024);   // a byte a column
#pragma unroll
                        for (int ks = 0; ks < kT8Keys / 32; ++ks)
                            tc_mma_e4m3(d + h * P::o_head, vd + (uint64_t)(ks * 4 * HP * kGroup >> 4), pd + (uint64_t)(ks * 32 * 128 >> 4), id,
                                        !fresh || ks > 0);
                    }
                    tc_commit(&x.v_empty[vp.slot]);
                } else {
                    ok = ok && t8_wait(&x.w_full[u & 1], u >> 1 & 1u, ab) && t8_wait(&x.p_full[u & 1], u >> 1 & 1u, ab);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t vd = sdesc_mnmajor_sw128(smem_u32(wide) + (u & 1) * kWide, 1024, H * 1024);
                    const uint64_t pd = sdesc_mnmajor_sw128(pa, 1024, 1024);
#pragma unroll
                    for (int ks = 0; ks < kT8Keys / 16; ++ks)
                        tc_mma_bf16(d, vd + (uint64_t)(ks * 2 * H * 1024 >> 4), pd + (uint64_t)(ks * 2 * 1024 >> 4), id, !fresh || ks > 0);
                    tc_commit(&x.w_empty[u & 1]);
                }
                fresh = false;
                tc_commit(&x.p_empty[u & 1]);
                vp.next(geo.v_slots);
                base += kT8Keys;
                ++u;
                --left;
            }
            if (!ok) give_up();
            volatile int never = 0;
            tc_commit(&x.done[1]);
            mbar_wait(&x.done[1], 0, &never);
        }
    } else if (warp == P::scale) {
        // ---------------- scales, 32 a step: fetched while those before them are stored, their pages a step earlier
        const int ps = a.kv.page_size, unit_shift = 7 - geo.gran, steps = geo.per_unit > 32 ? geo.per_unit / 32 : 1;   // of a round
        unsigned n = 0;   // rounds stored
        bool ok = true;
        for (unsigned i = 0; ok; ++i) {
            ok = warp_wait(&x.item_full[i % kT8Items], i / kT8Items & 1u);
            if (!ok) break;
            const PagedItem &it = x.item[i % kT8Items];
            if (!it.more) break;
            const int units = it.t1 - it.t0, lo = it.lo, hi = it.hi, tile0 = it.t0, head = it.head * HP;
            const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.item_empty[i % kT8Items]);
            const int all = (units + geo.round - 1) / geo.round * steps;
            int page = -1, next_slot = 0;
            float k[HP] = {}, v[HP] = {};
#pragma unroll 1
            for (int s = -2, in_round = 0; ok && s < all; ++s) {
                if (s >= 0) {
                    if (in_round == 0) ok = warp_wait(&x.sc_empty[n % kT8Scales], (n / kT8Scales & 1u) ^ 1u);
#pragma unroll
                    for (int h = 0; h < HP; ++h)
                        x.sc[n % kT8Scales][h][in_round * 32 + lane] =
                            make_float2(fminf(k[h] * a.scale_log2, 3.402823466e38f), v[h] > 0.f ? log2f(v[h]) : -INFINITY);
                    if (++in_round == steps) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&x.sc_full[n % kT8Scales]);
                        in_round = 0;
                        ++n;
                    }
                }
                const bool paged = page >= 0 && page < a.kv.n_pages;
                const long long at = paged ? page * a.kv.scale_stride + next_slot / a.kv.block * geo.n_heads + head : 0;
#pragma unroll
                for (int h = 0; h < HP; ++h) {
                    k[h] = paged ? kv8_scale(a.kv.k_scale[at + h]) : 0.f;   // (0: no page)
                    v[h] = paged ? kv8_scale(a.kv.v_scale[at + h]) : 0.f;
                }
                // the first key of this lane's scale of step s + 2
                page = -1;
                const int f = (s + 2) * 32 + lane, unit = f >> unit_shift;
                const int j = (tile0 + unit) * kT8Keys + ((f & (geo.per_unit - 1)) << geo.gran);
                if (unit < units && j < hi && j + (1 << geo.gran) > lo) {
                    const int p = geo.page_shift >= 0 ? j >> geo.page_shift : j / ps;
                    next_slot = j - p * ps;
                    page = table[p];
                }
            }
        }
        if (!ok) give_up();
    } else if (warp >= P::conv) {
        // ---------------- queries to pairs of codes; V's tiles
        const int t = threadIdx.x - P::soft, bar = 1 + P::groups;
        const bf16 *qp = static_cast<const bf16 *>(a.q);
        unsigned u = 0;
        T8Place vp = {0, 0};
        for (unsigned i = 0;; ++i) {
            bool ok = warp_wait(&x.item_full[i % kT8Items], i / kT8Items & 1u);
            if (t8_any(bar, !ok)) {
                give_up();
                break;
            }
            const PagedItem &it = x.item[i % kT8Items];
            if (!it.more) break;
            const int units = it.t1 - it.t0, lo = it.lo, hi = it.hi, tile0 = it.t0, n_rows = it.n_rows / HP;
            const int2 ends = t8_ends(it);
            // queries: LPR threads a row, 8 dims each, all rows in flight
            if (t < HP * NR) {
                const int h = t / NR, row = it.row0 + t % NR, tok = row / geo.group;
                x.q_off[t] = t % NR < n_rows ? (long long)(it.token + tok) * a.q_stride + (it.head * a.group + h * geo.group + row - tok * geo.group) * HD
                                             : -1;
            }
            t8_sync(bar);
            constexpr int LPR = HD / 8, RPP = 128 / LPR, ROWS = HP * NR, PASSES = ROWS > RPP ? ROWS / RPP : 1;
            const int sub = t % LPR, r_first = t / LPR;
            uint4 qw[PASSES];
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                qw[p] = make_uint4(0u, 0u, 0u, 0u);
                const int r = p * RPP + r_first;
                const long long off = r < ROWS ? x.q_off[r] : -1;   // (64 dims and 8 rows: half of the threads have none)
                if (off >= 0) qw[p] = *reinterpret_cast<const uint4 *>(qp + off + sub * 8);
            }
            ok = ok && warp_wait(&x.q_empty[i & 1], (i >> 1 & 1u) ^ 1u);
            unsigned char *q8 = qbuf + (i & 1) * kQ;
            uint32_t top[PASSES];   // a row's largest magnitude, as bits
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const uint32_t m2 = __vmaxu2(__vmaxu2(qw[p].x & 0x7fff7fffu, qw[p].y & 0x7fff7fffu),
                                             __vmaxu2(qw[p].z & 0x7fff7fffu, qw[p].w & 0x7fff7fffu));
                top[p] = max(m2 & 0xffffu, m2 >> 16);
            }
            auto over_row = [&]() {
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
                    for (int p = 0; p < PASSES; ++p) top[p] = max(top[p], __shfl_xor_sync(0xffffffffu, top[p], o));
            };
            over_row();
            uint32_t all = top[0];
#pragma unroll
            for (int p = 1; p < PASSES; ++p) all = max(all, top[p]);
            if (__any_sync(0xffffffffu, all >= 0x7f80u)) {   // of the finite ones
#pragma unroll
                for (int p = 0; p < PASSES; ++p) {
                    const uint32_t w[4] = {qw[p].x, qw[p].y, qw[p].z, qw[p].w};
                    top[p] = 0u;
#pragma unroll 1
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t v = w[e >> 1] >> (e & 1) * 16 & 0x7fffu;
                        if (v < 0x7f80u) top[p] = max(top[p], v);
                    }
                }
                over_row();
            }
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int r = p * RPP + r_first;
                const uint32_t w[4] = {qw[p].x, qw[p].y, qw[p].z, qw[p].w};
                // the least power of two s with top <= 448 s
                const int ex = top[p] ? max((int)(top[p] >> 7) - 127 - 8 + ((top[p] & 0x7fu) > 0x60u), -126) : 0;
                const float inv = __uint_as_float((uint32_t)(127 - ex) << 23);
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // as FP16, which holds 8 bits down to 2^-17; infinities become NaN
                    __half2 y = __floats2half2_rn(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xffff0000u) * inv);
                    y = __hfma2(y, __float2half2_rn(0.f), y);
                    h[e] = t8_e4m3x2(y);
                    const uint32_t f = t8_f16x2(h[e]);
                    l[e] = t8_e4m3x2(__hmul2(__hsub2(y, *reinterpret_cast<const __half2 *>(&f)), __float2half2_rn(16.f)));
                }
                if (r < ROWS) {
                    auto place = [&](int row) {   // of this thread's 8 bytes, in the swizzled tile
                        if (HD == 128) return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + (((sub >> 1) ^ (row & 7)) << 4) + (sub & 1) * 8);
                        return (uint32_t)((row >> 3) * 512 + (row & 7) * 64 + (((sub >> 1) ^ ((row >> 1) & 3)) << 4) + (sub & 1) * 8);
                    };
                    unsigned char *qh = q8 + r / NR * kQhead;   // of the row's head
                    *reinterpret_cast<uint2 *>(qh + place(r % NR)) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                    *reinterpret_cast<uint2 *>(qh + place(NR + r % NR)) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                    if (sub == 0) x.q_scale[i % kT8Items][r] = __uint_as_float((uint32_t)(127 + ex) << 23);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.q_full[i & 1]);
#pragma unroll 1
            for (int k = 0; k < units; ++k, ++u) {
                const int base = (tile0 + k) * kT8Keys;
                ok = ok && warp_wait(&x.v_full[vp.slot], vp.phase);
                unsigned char *src = vring + vp.slot * kTile;
                const bool by_row = t8_by_row(ends, base, a.window), edge = by_row || base < lo || base + kT8Keys > hi;
                // 16 codes of key j as they may be used
                auto mend = [&](uint4 &w4, int j) {
                    if (j < lo || j >= hi) {
                        w4 = make_uint4(0u, 0u, 0u, 0u);
                    } else if (by_row && (j > ends.x || (a.window > 0 && j <= ends.y - a.window))) {
                        if ((int)t8_no_nan(w4.x) | (int)t8_no_nan(w4.y) | (int)t8_no_nan(w4.z) | (int)t8_no_nan(w4.w)) x.poison[i % kT8Items] = 1;
                    }
                };
                if (kDirect) {
                    if (edge) {   // whole rows: the order of their chunks does not matter
#pragma unroll 1
                        for (int c = t; c < (int)kTile / 16; c += 128) {
                            uint4 *at = reinterpret_cast<uint4 *>(src) + c, w4 = *at;
                            const int row = c / (HD / 16);   // (of 8 keys of one head, then of the other)
                            mend(w4, base + row / (8 * HP) * 8 + row % 8);
                            *at = w4;
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&x.w_full[vp.slot]);
                        mbar_arrive(&x.v_empty[vp.slot]);
                    }
                } else {
                    ok = ok && warp_wait(&x.w_empty[u & 1], (u >> 1 & 1u) ^ 1u);
                    constexpr int CPK = HD / 16, KPP = 128 / CPK, TURNS = kT8Keys / KPP;   // 16-byte chunks of a key; keys of a turn
                    const int c = t % CPK, key0 = t / CPK;
                    // rows of 128 bytes (64 dims), the second halves beside the first by groups of 8 keys; of
                    // the two 16-byte chunks the threads of the second half store the odd one first (banks)
                    const int half = c >> 2, c2 = (c & 3) * 2, odd = half;
                    unsigned char *dst = wide + (u & 1) * kWide + half * 1024;
#pragma unroll 1
                    for (int y0 = 0; y0 < TURNS; y0 += 4) {
                        uint4 in[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            in[y] = *reinterpret_cast<const uint4 *>(src + (uint32_t)((y0 + y) * KPP + key0) * HD + c * 16);
                        if (edge) {
#pragma unroll
                            for (int y = 0; y < 4; ++y) mend(in[y], base + (y0 + y) * KPP + key0);
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const int key = (y0 + y) * KPP + key0;
                            unsigned char *row = dst + (uint32_t)(key >> 3) * (H * 1024) + (key & 7) * 128;
                            const uint4 h0 = make_uint4(t8_f16x2(in[y].x), t8_f16x2(in[y].x >> 16), t8_f16x2(in[y].y), t8_f16x2(in[y].y >> 16));
                            const uint4 h1 = make_uint4(t8_f16x2(in[y].z), t8_f16x2(in[y].z >> 16), t8_f16x2(in[y].w), t8_f16x2(in[y].w >> 16));
                            *reinterpret_cast<uint4 *>(row + (((c2 + odd) ^ (key & 7)) << 4)) = odd ? h1 : h0;
                            *reinterpret_cast<uint4 *>(row + (((c2 + 1 - odd) ^ (key & 7)) << 4)) = odd ? h0 : h1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&x.w_full[u & 1]);
                        mbar_arrive(&x.v_empty[vp.slot]);
                    }
                }
                vp.next(geo.v_slots);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&x.item_empty[i % kT8Items]);
            if (!ok) give_up();
        }
    } else {
        // ---------------- softmax and output: rows r0 .. r0 + OWN - 1; thread: key of S, dim of O
        constexpr int OWN = P::own;
        const int g = warp >> 2, wq = warp & 3, key = 32 * wq + lane, r0 = g * OWN, bar = 1 + g, tg = threadIdx.x & 127;
        const int head_row = HP > 1 ? r0 : 0;   // the first row of the group's head
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const int win = a.window > 0 ? a.window : 0x7fffffff;
        bf16 *out = static_cast<bf16 *>(a.out);
        const float *nm = x.neg_m + r0;
        const int *pos = x.pos + r0;
        unsigned u = 0, nr = 0;   // units, rounds of scales
        constexpr int REP = 32 / OWN;     // lanes that end with the same row
        for (unsigned i = 0;; ++i) {
            bool ok = warp_wait(&x.item_full[i % kT8Items], i / kT8Items & 1u);
            if (t8_any(bar, !ok)) {
                give_up();
                break;
            }
            const PagedItem &it = x.item[i % kT8Items];
            if (!it.more) break;
            const int units = it.t1 - it.t0, n_rows = it.n_rows / HP, lo = it.lo, hi = it.hi;   // (rows of a head)
            const bool active = n_rows > r0 - head_row;
            const int2 ends = t8_ends(it);
            if (tg < OWN) {   // (rows that are not there are taken as the last one)
                const int r = r0 + tg, row = min(r - head_row, n_rows - 1), tok = (it.row0 + row) / geo.group;
                const int hd = (HP > 1 ? g : 0) * geo.group + it.row0 + row - tok * geo.group;
                x.pos[r] = max(it.pos0 + tok, -1);
                x.off[r] = (long long)(it.token + tok) * a.out_stride + (it.head * a.group + hd) * HD;
                x.row[r] = HP > 1 ? tok * a.group + hd : row;
                x.neg_m[r] = 0.f;
                x.set[r] = 0;
            }
            t8_sync(bar);
            const float *qs = x.q_scale[i % kT8Items] + r0;
            const uint32_t t_o = tmem_o + lanes + (i & 1) * P::o_cols + (kDirect ? 4 : 1) * r0;
            uint64_t l[OWN / 2];
#pragma unroll
            for (int e = 0; e < OWN / 2; ++e) l[e] = 0ull;
            bool unset = true;   // some row has no m
            // (each lane looks for itself: a vote a wait cost 1.5 us of the drafts' 90)
            auto wait = [&](uint64_t *b, uint32_t parity) {
                ok = ok && t8_wait(b, parity, ab);
                __syncwarp();
            };
            int base = it.t0 * kT8Keys, in_round = 0;
#pragma unroll 1
            for (int k = 0; k < units; ++k, ++u, base += kT8Keys) {
                if (in_round == 0) wait(&x.sc_full[nr % kT8Scales], nr / kT8Scales & 1u);
                const float2 sc = x.sc[nr % kT8Scales][HP > 1 ? g : 0][in_round * geo.per_unit + (key >> geo.gran)];
                if (++in_round == geo.round || k == units - 1) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x.sc_empty[nr % kT8Scales]);
                    in_round = 0;
                    ++nr;
                }
                wait(&x.s_full[u & 1], u >> 1 & 1u);
                if (active) {
                    tc_fence_after();
                    const int j = base + key;
                    const bool there = j >= lo && j < hi && sc.y > -INFINITY;
                    const bool by_row = t8_by_row(ends, base, a.window);
                    const uint32_t t_s = tmem + lanes + (u & 1) * P::s_cols + head_row * 2 + r0 - head_row;
                    const uint64_t kc = pack_f32x2(sc.x, sc.x), lv = pack_f32x2(sc.y, sc.y), sixteenth = pack_f32x2(0.0625f, 0.0625f);
                    float y[OWN];   // t_rj - m_r
                    {
                        uint32_t h[OWN], s[OWN];
                        if constexpr (OWN == 16) {
                            tmem_ld16_async(t_s, h);
                            tmem_ld16_async(t_s + NR, s);
                        } else {
                            tmem_ld8_async(t_s, h);
                            tmem_ld8_async(t_s + NR, s);
                        }
                        tmem_wait_ld<OWN>(h);
                        tmem_wait_ld<OWN>(s);
#pragma unroll
                        for (int e = 0; e < OWN; e += 4) {
                            const ulonglong2 q4 = t8_rows4(qs + e), m4 = t8_rows4(nm + e);
#pragma unroll
                            for (int z = 0; z < 4; z += 2) {
                                const uint64_t f = mul_f32x2(kc, z ? q4.y : q4.x), b = add_f32x2(lv, z ? m4.y : m4.x);
                                const uint64_t w = fma_f32x2(pack_f32x2(__uint_as_float(s[e + z]), __uint_as_float(s[e + z + 1])), sixteenth,
                                                             pack_f32x2(__uint_as_float(h[e + z]), __uint_as_float(h[e + z + 1])));
                                const float2 v = unpack_f32x2(fma_f32x2(w, f, b));
                                y[e + z] = v.x;
                                y[e + z + 1] = v.y;
                            }
                        }
                    }
                    if (by_row || !__all_sync(0xffffffffu, there)) {
                        uint32_t see = 0u;   // a bit a row
                        if (there) {
                            see = 0xffffu;
                            if (by_row) {
                                see = 0u;
#pragma unroll 1
                                for (int e = 0; e < OWN; ++e) {
                                    const int p = pos[e];
                                    see |= (uint32_t)(j <= p && j > p - win) << e;
                                }
                            }
                        }
#pragma unroll
                        for (int e = 0; e < OWN; ++e) y[e] = see >> e & 1u ? y[e] : -INFINITY;
                    }
                    float top = y[0];
#pragma unroll
                    for (int e = 1; e < OWN - 1; e += 2) top = t8_max3(top, y[e], y[e + 1]);
                    top = fmaxf(top, y[OWN - 1]);
                    if (t8_any(bar, unset || top > P::most)) {   // some row's weights outgrow its m, or it has none
                        float v[OWN];
#pragma unroll
                        for (int e = 0; e < OWN; ++e) v[e] = y[e];
                        t8_over_warp<true>(v);   // (the number beside a NaN)
                        if (lane % REP == 0) x.part[warp][lane / REP] = fmaxf(v[0], -INFINITY);
                        t8_sync(bar);
                        bool none = false;
                        if (tg < OWN) {
                            const int w0 = g * 4, r = r0 + tg;
                            const float m = fmaxf(fmaxf(x.part[w0][tg], x.part[w0 + 1][tg]), fmaxf(x.part[w0 + 2][tg], x.part[w0 + 3][tg]));
                            const bool set = x.set[r] != 0, up = m > -INFINITY && (!set || m > P::most);
                            const float d = up ? P::off - m : 0.f;
                            none = !set && !up;
                            x.delta[r] = d;
                            // (Below 2^-126 the row sum may be as large as the factor is small, 2^64 for a key of zeros before one with
                            // a scale of 2^64, and takes its root twice.  O takes it once: the 2^-63 that stay of it are below what
                            // the weights hold.)
                            const bool tiny = set && d < -126.f;
                            const float f = set ? t8_ex2(tiny ? 0.5f * d : d) : 1.f;   // (a row without m has no sums)
                            x.factor[r] = f;
                            x.again[r] = tiny ? f : 1.f;
                            x.neg_m[r] += d;
                            if (up) x.set[r] = 1;
                        }
                        unset = t8_any(bar, none);
                        if (k > 0) {
                            // O of the units before
                            wait(&x.p_empty[(u - 1) & 1], ((u - 1) >> 1) & 1u);
                            tc_fence_after();
#pragma unroll 1
                            for (int q = 0; q < (kDirect ? 4 * OWN : OWN); q += 8) {   // (direct: eight rows have four times eight columns)
                                uint32_t o[8];
                                tmem_ld8_async(t_o + q, o);
                                tmem_wait_ld<8>(o);
                                const float *f = x.factor + r0 + (kDirect ? q >> 5 << 3 : q);
#pragma unroll
                                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
                                tmem_st8(t_o + q, o);
                            }
                            tmem_wait_st();
#pragma unroll
                            for (int e = 0; e < OWN; e += 4) {
                                const ulonglong2 f = t8_rows4(x.factor + r0 + e), f2 = t8_rows4(x.again + r0 + e);
                                l[e / 2] = mul_f32x2(mul_f32x2(l[e / 2], f.x), f2.x);
                                l[e / 2 + 1] = mul_f32x2(mul_f32x2(l[e / 2 + 1], f.y), f2.y);
                            }
                        }
#pragma unroll
                        for (int e = 0; e < OWN; ++e) y[e] += x.delta[r0 + e];
                    }
                    // Row sums: p / vs.  With a small vs, 2^-64 for a block of zeros, p may underflow beside a scale of up to 2^64
                    // although p / vs counts: then 2^(t - log2 vs - m), at the largest key 2^-59 or more.  (With that and the
                    // second factor of the sums the drafts take 90.1 us for 89.3; the two ways as the branches of each sum 91.6.)
                    const bool far = there && sc.y < -24.f;
                    const float r = there && !far ? t8_ex2(-sc.y) : 0.f;   // 1 / vs
                    const uint64_t rr = pack_f32x2(r, r);
                    if (u >= 2) wait(&x.p_empty[u & 1], ((u - 2) >> 1) & 1u);
                    unsigned char *prow = pbuf + (u & 1) * kP + (uint32_t)(key >> 3) * 1024 + (key & 7) * 128;
#pragma unroll
                    for (int q = 0; q < OWN; q += 8) {
                        float p[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] = t8_ex2(y[q + e]);
#pragma unroll
                        for (int e = 0; e < 8; e += 2) l[(q + e) / 2] = fma_f32x2(pack_f32x2(p[e], p[e + 1]), rr, l[(q + e) / 2]);
                        if (kDirect) {
                            // columns (r / 8) 32 + 8 s + r % 8: s 0, 1 the codes of the large weights and what they
                            // leave, 2, 3 those of the small ones, in units of 2^-13
                            uint32_t hi4[2], lo4[2], small[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                uint32_t h0, h1, l0, l1, m = 0u;
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (p[4 * z + e] < 0x1p-5f) {
                                        p[4 * z + e] *= 0x1p13f;
                                        m |= 0xffu << (8 * e);
                                    }
                                t8_split(p[4 * z], p[4 * z + 1], h0, l0);
                                t8_split(p[4 * z + 2], p[4 * z + 3], h1, l1);
                                hi4[z] = __byte_perm(h0, h1, 0x5410);
                                lo4[z] = __byte_perm(l0, l1, 0x5410);
                                small[z] = m;
                            }
                            const int c = (r0 + q) >> 2;   // 32 bytes: two of the row's 16-byte chunks
                            *reinterpret_cast<uint4 *>(prow + ((c ^ (key & 7)) << 4)) =
                                make_uint4(hi4[0] & ~small[0], hi4[1] & ~small[1], lo4[0] & ~small[0], lo4[1] & ~small[1]);
                            *reinterpret_cast<uint4 *>(prow + (((c + 1) ^ (key & 7)) << 4)) =
                                make_uint4(hi4[0] & small[0], hi4[1] & small[1], lo4[0] & small[0], lo4[1] & small[1]);
                        } else {
                            uint32_t h[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 pk = __floats2half2_rn(p[2 * e], p[2 * e + 1]);
                                h[e] = *reinterpret_cast<const uint32_t *>(&pk);
                            }
                            *reinterpret_cast<uint4 *>(prow + ((((r0 + q) >> 3) ^ (key & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    }
                    fence_proxy_async_smem();   // before the MMA reads them
                    if (__builtin_expect(far, 0)) {
#pragma unroll
                        for (int e = 0; e < OWN; e += 2)
                            l[e / 2] = add_f32x2(l[e / 2], pack_f32x2(t8_ex2(y[e] - sc.y), t8_ex2(y[e + 1] - sc.y)));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&x.p_full[u & 1]);
            }
            // ---- the item's rows: O is complete with its last unit's.  (All groups wait for it: none
            // runs ahead of the others by more than an item.)
            const unsigned last = u - 1;
            const bool part = it.part >= 0;
            if (active) {
                float v[OWN];   // row sums
#pragma unroll
                for (int e = 0; e < OWN / 2; ++e) {
                    const float2 f = unpack_f32x2(l[e]);
                    v[2 * e] = f.x;
                    v[2 * e + 1] = f.y;
                }
                t8_over_warp<false>(v);
                if (lane % REP == 0) x.part[warp][lane / REP] = v[0];
                t8_sync(bar);
                if (tg < OWN) {
                    const int w0 = g * 4, r = r0 + tg;
                    const float sum = (x.part[w0][tg] + x.part[w0 + 1][tg]) + (x.part[w0 + 2][tg] + x.part[w0 + 3][tg]);
                    if (part && r - head_row < n_rows) {
                        float *ml = reinterpret_cast<float *>(a.ws + lay.ml) + ((size_t)it.part * a.rows + x.row[r]) * 2;
                        ml[0] = x.set[r] ? -x.neg_m[r] : -INFINITY;
                        ml[1] = sum;
                    }
                    x.factor[r] = part ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
                }
                t8_sync(bar);
            }
            wait(&x.p_empty[last & 1], last >> 1 & 1u);
            if (active && 32 * wq < HD) {   // thread: dim `key`
                tc_fence_after();
                uint32_t nan = 0u;   // rows that see a key whose V is NaN in this dim
                if (*const_cast<volatile int *>(&x.poison[i % kT8Items])) {
                    // among the keys that only some rows see: those behind the first row's token, and those that left the
                    // last one's window
                    const int j0 = max(lo, it.t0 * kT8Keys), j1 = min(hi, it.t1 * kT8Keys);
#pragma unroll 1
                    for (int edge = 0; edge < 2; ++edge) {
                        const int from = edge ? j0 : max(j0, ends.x + 1);
                        const int upto = edge ? (a.window > 0 ? min(j1, min(ends.y - win, ends.x) + 1) : j0) : j1;
#pragma unroll 1
                        for (int j = from; j < upto; ++j) {
                            const int page = key_page(a, a.s.table + (long long)it.seq * a.s.table_stride, j);
                            if (page < 0) continue;
                            const uint8_t code =
                                static_cast<const uint8_t *>(a.kv.v)[page * a.kv.page_stride + (j % a.kv.page_size) * a.kv.slot_stride +
                                                                     (it.head * HP + (HP > 1 ? g : 0)) * a.kv.head_stride + key];
                            if ((code & 0x7fu) != 0x7fu) continue;
#pragma unroll 1
                            for (int e = 0; e < OWN; ++e)
                                if (j <= pos[e] && j > pos[e] - win) nan |= 1u << e;
                        }
                    }
                }
                float *po = reinterpret_cast<float *>(a.ws + lay.o) + (size_t)(part ? it.part : 0) * a.rows * HD + key;
#pragma unroll 1
                for (int q = 0; q < OWN; q += 8) {
                    float f[8];
                    if constexpr (kDirect) {
                        uint32_t o[32];
                        tmem_ld32_async(t_o + 4 * q, o);
                        tmem_wait_ld32(o);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[e] = fmaf(fmaf(__uint_as_float(o[24 + e]), 0.0625f, __uint_as_float(o[16 + e])), 0x1p-13f,
                                        fmaf(__uint_as_float(o[8 + e]), 0.0625f, __uint_as_float(o[e])));
                    } else {
                        uint32_t o[8];
                        tmem_ld8_async(t_o + q, o);
                        tmem_wait_ld<8>(o);
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[e]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int r = r0 + q + e;
                        if (r - head_row >= n_rows) break;
                        float v = f[e] * x.factor[r];
                        if (nan >> (q + e) & 1u) v = NAN;
                        if (part) po[x.row[r] * HD] = v;
                        else out[x.off[r] + key] = __float2bfloat16_rn(v);
                    }
                }
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
    if (warp == P::mma_s) {
        tc_fence_after();
        tmem_dealloc(tmem, P::cols);
    }
}

// ------------------------------------------------------------------ host side

static int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

template <int HD, int NR, int HP>
static cudaError_t t8_go(AttnArgs &a, T8Geometry &g, cudaStream_t st, int grid)
{
    constexpr bool direct = T8<NR, HP>::direct;
    CUtensorMap km, vm;
    // 8 slots, then the heads, then the groups of 8 slots of a page
    const long long dims[5] = {HD, 8, g.n_heads, a.kv.page_size / 8, a.kv.n_pages};
    const long long strides[4] = {a.kv.slot_stride, a.kv.head_stride, 8 * a.kv.slot_stride, a.kv.page_stride};
    const int box[5] = {HD, 8, HP, g.box / 8, 1};
    cudaError_t e = tc::make_map_u8_nd(&km, a.kv.k, 5, dims, strides, box, HD);
    if (!e) e = tc::make_map_u8_nd(&vm, a.kv.v, 5, dims, strides, box, direct ? HD : 0);
    if (e) return e;
    constexpr int tile = HP * HD * kT8Keys, fixed = (direct ? 0 : 4 * tile) + 2 * kT8Keys * 128 + 4 * HP * NR * HD + (int)sizeof(T8Misc);
    constexpr int room = (kT8Smem - fixed) / tile, slots = room > 2 * kT8MaxSlots ? 2 * kT8MaxSlots : room;
    static_assert(slots >= 4, "two tiles of K and of V beside the buffers");
    // the odd one is V's, whose tiles wait for the softmax (converted ones do not)
    g.v_slots = (slots + (direct ? 1 : 0)) / 2;
    g.k_slots = slots - g.v_slots;
    static PerDevice once;
    auto kernel = k_paged_attn8_tc<HD, NR, HP>;
    e = allow_once(once, kernel, kT8Smem);
    if (e) return e;
    return launch_pdl(kernel, dim3(grid), dim3(T8<NR, HP>::threads), (size_t)(fixed + slots * tile), st, km, vm, a, g);
}

template <int HD> static cudaError_t t8_dim(AttnArgs &a, T8Geometry &g, int heads, cudaStream_t st, int grid)
{
    const int rows = a.rows / heads;
    if (heads == 2) return rows <= 8 ? t8_go<HD, 8, 2>(a, g, st, grid) : t8_go<HD, 16, 2>(a, g, st, grid);
    if (rows <= 8) return t8_go<HD, 8, 1>(a, g, st, grid);
    if (rows <= 16) return t8_go<HD, 16, 1>(a, g, st, grid);
    return rows <= 32 ? t8_go<HD, 32, 1>(a, g, st, grid) : t8_go<HD, 64, 1>(a, g, st, grid);
}

cudaError_t paged_attn8_tc(AttnArgs &a, cudaStream_t st, int nsm)
{
    T8Geometry g = {};
    g.box = gcd(a.kv.page_size, kT8Keys);
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (1 << i == a.kv.page_size) g.page_shift = i;
    g.gran = 0;
    while (g.gran < 7 && a.kv.block % (2 << g.gran) == 0) ++g.gran;
    g.per_unit = kT8Keys >> g.gran;
    g.round = g.per_unit < 32 ? 32 / g.per_unit : 1;
    g.group = a.group;
    g.n_heads = a.kv.n_kv_heads;
    // two heads are taken as one with their query heads, for the division of the work and the join
    const int heads = paged_attn8_tc_heads(a.kv.n_kv_heads, a.group, a.s.max_new);
    a.group *= heads;
    a.kv.n_kv_heads /= heads;
    const int grid = paged_attn_grid(a, kT8Keys, nsm < kAttnMaxCtasTc ? nsm : kAttnMaxCtasTc);
    cudaError_t e = a.kv.head_dim == 64 ? t8_dim<64>(a, g, heads, st, grid) : t8_dim<128>(a, g, heads, st, grid);
    if (!e && !a.whole) e = paged_join_tc(a, grid, nsm, st);
    return e;
}

}  // namespace ds4g
