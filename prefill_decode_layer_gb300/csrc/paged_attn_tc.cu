// Tensor-core form of the paged attention (tcgen05 MMAs with TMEM accumulators, TMA tiles
// of the cache's pages): page "ds4.c 学习笔记 -- 端到端推理流程", 阶段四 4.2. The
// mathematics and the division of the work are paged_attn.cu's and paged_sched.cuh's; this
// form takes BF16 queries over a BF16 cache, head_dim 64 or 128.
//
// A unit is 128 keys of an item; the item's up to 128 query rows (new token, head of the
// K/V head's group) are the MMA's M side, also where there are fewer: at one new token the
// bound is the cache's bytes (128 keys of 128 dims are 64 KB, 1.46 us of an SM's share of
// the HBM bandwidth, against 0.57 us of padded MMA work).  Per unit:
//   S = Q K^T    M 128 x N 128 keys, from shared memory into TMEM;
//   softmax      a thread owns a row: it reads its 128 scores from TMEM, masks them, and
//                writes P = 2^(s c - m) as BF16 over them (the row sums stay FP32 and
//                unrounded; P's rounding, 2^-9 of a weight on average, is the price of the
//                BF16 tensor cores).  m is the row's running maximum, but moved only when a
//                tile exceeds it by 2^8: the rescale of O is then rare;
//   O += P V     A = P straight from TMEM, V read MN-major from its TMA tile.
// Units alternate between two streams, each with its own S/P and O columns, ring of tiles, MMA
// thread and four softmax warps, which are independent attentions over every other unit: the
// MMAs of one overlap the softmax of the other.  When the item ends both streams' O lie in the
// same TMEM lanes, so that merging them is a thread's own arithmetic.
//
// Masked places: rows of V outside the sequence's keys are zeroed in shared memory where a
// 16-key MMA step contains them; pages that are not there are read as zeros (a page
// coordinate out of bounds) and masked by a bit per 8 keys.  A key that only some rows
// see (several new tokens, or a window's edge) must not reach the others as 0 * NaN: what
// is not finite in its V row is replaced by 0 and added to the rows that see it when
// the item ends.
//
// Roles (352 threads, one CTA per SM): warps 0-3 and 4-7 softmax and output of streams 0
// and 1; warp 8 the items, the page look-ups and the TMA copies; warps 9 and 10 (one thread
// each) the MMAs of streams 0 and 1.  Every wait is bounded; a CTA that gives up says so in
// its status word, drains its copies and MMAs, frees its TMEM and returns.
//
// Measured (with the join; fractions of a copy's 6.78 TB/s): 64 sequences of up to 8191
// positions, 32 heads on 8 K/V heads of 128, 1.37 GB: 217-222 us, 0.91-0.93; four of up to 131072
// with 64 heads on 8, 1.63 GB: 250 us, 0.96; one token of 64 heads in a window of 128: 7.8
// us, latency (launch, page look-up, K, softmax, V); 32 sequences of up to 16994 with up to five new
// tokens and 64 heads on one K/V head, 181 MB and 34 GFLOP: 58 us, of which 19 do not grow with the
// length (launch, first tiles, output, join) and 32 units a CTA take 1.2 us each: 2500 cycles between
// two units, the streams in turn, so that a stream's chain S -> softmax -> P V takes 5000, 1024 of
// them MMAs (tensor pipe 40 % of the active cycles).  Each row tile reads K and V for itself: 64 KB a
// unit, 322 MB in all, 222 MB of them from DRAM.
#include <cuda.h>
#include <stddef.h>

#include "paged_sched.cuh"
#include "sm100.cuh"
#include "tc_gemm.cuh"

namespace ds4g {

static constexpr int kTcKeys = 128;                    // keys of a unit
static constexpr int kTcSoft = 256;                    // softmax threads
static constexpr int kTcThreads = kTcSoft + 96;
static constexpr int kTcTma = kTcSoft / 32, kTcMma = kTcTma + 1;   // warps of the copies and of stream 0's MMAs
static constexpr int kTcMaxSlots = 8;
static constexpr int kTcItems = 4;                     // items ahead of the softmax at most
static constexpr int kTcSmem = 227 * 1024;

struct TcMisc {
    uint64_t full[kTcMaxSlots], empty[kTcMaxSlots];    // K/V tiles of the ring
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[2], p_full[2];                     // of a stream
    uint64_t o_done, o_free;                           // O complete; O read by the softmax threads
    uint64_t item_full[kTcItems], item_empty[kTcItems];
    uint64_t done;
    PagedItem item[kTcItems];
    PagedCursor cur;
    long long scratch[kTcThreads / 32];
    uint32_t there[8];                                 // of unit u % 8: a bit per 8 keys whose page is there
    uint32_t tmem;
    int abort_flag;
    int poison[2];                                     // of item i % 2: a partly seen V row is not finite
    float2 ml[2][128];                                 // [stream][row] maximum (log2 units) and sum
};
// (a fifth tile would fit there, but no ring of three: a stream has one K and one V tile)
static_assert(4 * 2 * kTcKeys * 128 + 2 * 2 * 128 * 128 + sizeof(TcMisc) <= kTcSmem,
              "two rings of two tiles of 128 dims beside two query tiles of 128 rows");

struct TcGeometry {
    int q_half;      // bytes of 64 dims of the query tile
    int slots;
    int box;         // slots of a page in one copy: gcd(page_size, 128)
    int toks;        // tokens of the query box
    int page_shift;  // log2(page_size), or -1
    // coordinates of (page, head) in the cache's tensor map: 64-dim block head * block, index
    // page * page_mul + head * head_mul; `none` is an index out of bounds
    int block, page_mul, head_mul, none;
};

// The tensor map of a cache has five dimensions: 64 dims, 8 slots, the 64-dim blocks, the
// groups of 8 slots of a page, and the pages.  A copy then brings a page's rows as
// [8-slot group][64-dim block][8 rows of 128 bytes], whose 8-row groups lie evenly over
// all pages of a tile, and one copy suffices for both 64-dim halves.  Heads join the
// 64-dim blocks where they are adjacent, else the pages (heads outside the slots).
static bool heads_adjacent(const PagedKV &kv) { return kv.n_kv_heads == 1 || kv.head_stride == kv.head_dim; }
static bool heads_divide_pages(const PagedKV &kv)
{
    return kv.page_stride % kv.head_stride == 0 &&
           (kv.page_stride / kv.head_stride) * (kv.n_pages - 1) + kv.n_kv_heads < 0x7fffffff;
}

bool paged_attn_tc_ok(const PagedKV &kv, int group, int q_dtype, int kv_dtype)
{
    return q_dtype == DS4G_BF16 && kv_dtype == DS4G_BF16 && (kv.head_dim == 64 || kv.head_dim == 128) &&
           kv.page_size % 8 == 0 && group <= 128 && (heads_adjacent(kv) || heads_divide_pages(kv));
}

int paged_attn_tc_rows(int group, int max_new)
{
    const int toks = 128 / group;
    return group * (toks < max_new ? toks : max_new);
}

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1)
    k_paged_attn_tc(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AttnArgs a,
                    const __grid_constant__ TcGeometry geo)
{
    constexpr int H = HD / 64;                         // 64-dim boxes of a row
    constexpr uint32_t kTile = H * kTcKeys * 128;      // bytes of a K or V tile
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t qbytes = (uint32_t)H * geo.q_half;  // one of two query buffers
    unsigned char *ring = sm + 2 * qbytes;
    TcMisc &x = *reinterpret_cast<TcMisc *>(ring + (uint32_t)geo.slots * kTile);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PartLayout lay(kAttnMaxCtasTc, a.rows, HD);

    {   // one barrier per thread
        uint64_t *bars = x.full;
        constexpr int n = offsetof(TcMisc, item) / 8;
        const int i = threadIdx.x;
        if (i < n) {
            int count = 1;
            if (bars + i == &x.p_full[0] || bars + i == &x.p_full[1]) count = 4;
            else if (bars + i == &x.q_empty[0] || bars + i == &x.q_empty[1]) count = 2;
            else if (bars + i == &x.o_done || bars + i == &x.done) count = 2;
            else if (bars + i == &x.o_free) count = kTcSoft / 32;
            else if (bars + i >= x.item_empty && bars + i < x.item_empty + kTcItems) count = 2 + kTcSoft / 32;
            mbar_init(bars + i, count);
        } else if (i == n) {
            x.abort_flag = 0;
            x.poison[0] = x.poison[1] = 0;
        }
        mbar_fence_init();
    }
    if (warp == kTcMma) tmem_alloc(&x.tmem, 512);
    if (threadIdx.x == kTcTma * 32) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_trigger();
    paged_begin(a, lay);
    const bool few = a.s.n_seqs <= 32;   // the copying warp finds the CTA's share by itself
    if (!few) paged_cursor<kTcThreads>(a, kTcKeys, &x.cur, x.scratch);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x.tmem;
    volatile int *ab = &x.abort_flag;
    auto give_up = [&]() {
        x.abort_flag = 1;
        reinterpret_cast<int *>(a.ws + lay.status)[blockIdx.x] = kAttnTimedOut;
    };
    // stream s: scores (then P) at column 128 s, O at 256 + 128 s
    // Each stream has half of the slots as a ring of its own (who waits for the tiles of a ring must see
    // every phase of its barriers: a parity tells no more than two apart).  It holds K V K V .. of the
    // stream's units; tile i lies in slot i % ring, in the phase (i / ring) % 2 of its barriers
    // (kept up to date: a division at every poll cost more than the MMAs).
    struct Place {
        unsigned slot, phase;
    };
    const unsigned ring_slots = (unsigned)geo.slots / 2;
    auto next_unit = [&](Place &p) {   // two tiles on (a ring has two slots or more)
        p.slot += 2;
        if (p.slot >= ring_slots) {
            p.slot -= ring_slots;
            p.phase ^= 1u;
        }
    };
    const Place k_first = {0, 0}, v_first = {1, 0};

    if (warp == kTcTma) {
        // ---------------- items, page look-ups, copies
        PagedCursor cur;
        if (few) paged_cursor_warp(a, kTcKeys, cur);
        else cur = x.cur;
        auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab)) != 0;
        };
        const int boxes = kTcKeys / geo.box, per_page = a.kv.page_size;
        unsigned u = 0;      // units whose K is loaded
        unsigned nq = 0;     // query tiles loaded
        int used = -1;       // lane i: the phase of the last load into ring slot i
        Place kp = k_first, vp = v_first;
        bool ok = true;
        // this lane's box of a unit (the lane-th of its tile)
        struct Box {
            int block, slot8, at;
            bool load;
            uint32_t bytes;   // of the whole tile
        };
        auto copy = [&](const Place &p, unsigned stream, const CUtensorMap *map, const Box &b) {
            const unsigned sl = stream * ring_slots + p.slot;
            if (!warp_wait(&x.empty[sl], p.phase ^ 1u)) return false;
            if (lane == 0) mbar_expect_tx(&x.full[sl], b.bytes);
            if (lane == (int)sl) used = (int)p.phase;
            __syncwarp();
            if (b.load)
                tma_load_5d(ring + sl * kTile + lane * geo.box * 128 * H, map, 0, 0, b.block, b.slot8, b.at, &x.full[sl]);
            return true;
        };
        Box prev = {};       // of unit u - 1, whose V follows this unit's K
        for (unsigned i = 0; ok; ++i) {
            if (!warp_wait(&x.item_empty[i % kTcItems], (i / kTcItems & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            PagedItem &it = x.item[i % kTcItems];
            if (lane == 0) {
                paged_next(a, kTcKeys, cur, lay, it);
                mbar_arrive(&x.item_full[i % kTcItems]);
            }
            __syncwarp();
            if (!it.more) break;
            if (!warp_wait(&x.q_empty[i & 1], (i >> 1 & 1u) ^ 1u)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                mbar_expect_tx(&x.q_full[i & 1], (uint32_t)(H * a.group * geo.toks * 128));
                for (int h = 0; h < H; ++h)
                    tma_load_3d(sm + (i & 1) * qbytes + h * geo.q_half, &qmap, h * 64, it.head * a.group,
                                it.token + it.tok_a, &x.q_full[i & 1]);
            }
            ++nq;
            const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
            const int lo = it.lo, hi = it.hi, head = it.head, t1 = it.t1;
            for (int t = it.t0; ok && t < t1; ++t, ++u) {
                const int j = t * kTcKeys + lane * geo.box;
                Box b;
                b.load = lane < boxes && j < hi && j + geo.box > lo;
                int page = -1, slot = 0;
                if (b.load) {
                    const int p = geo.page_shift >= 0 ? j >> geo.page_shift : j / per_page;
                    slot = j - p * per_page;
                    page = table[p];
                    if (page >= a.kv.n_pages) page = -1;
                }
                const uint32_t bits = b.load && page >= 0 ? ((1u << (geo.box >> 3)) - 1u) << (lane * (geo.box >> 3)) : 0u;
                const uint32_t there = __reduce_or_sync(0xffffffffu, bits);
                b.bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, b.load)) * geo.box * 128 * H;
                b.block = head * geo.block;
                b.slot8 = slot >> 3;
                // a page that is not there: out of bounds, read as zeros
                b.at = page < 0 ? geo.none : page * geo.page_mul + head * geo.head_mul;
                if (lane == 0) x.there[u % 8] = there;   // read once the scores are there
                // (both streams' rings are at the same place)
                ok = copy(kp, u & 1, &kmap, b);
                if (u & 1) next_unit(kp);
                if (ok && u > 0) {
                    ok = copy(vp, (u - 1) & 1, &vmap, prev);
                    if (!(u & 1)) next_unit(vp);
                }
                prev = b;
            }
        }
        if (ok && u > 0) ok = copy(vp, (u - 1) & 1, &vmap, prev);
        if (!ok) give_up();
        // nothing may be in flight when the CTA exits
        volatile int never = 0;
        if (used >= 0) mbar_wait(&x.full[lane], (uint32_t)used, &never);
        if (lane == 0)
            for (unsigned k = nq > 2 ? nq - 2 : 0; k < nq; ++k) mbar_wait(&x.q_full[k & 1], k >> 1 & 1u, &never);
    } else if (warp > kTcTma) {
        // ---------------- MMAs of stream t, units t, t + 2, ..: S of the first, then P V of each and S
        // of the next.  (A thread for each stream: it runs no further ahead of its MMAs than a few,
        // and with one for both the tensor cores stood idle while it went from one group to the next.)
        if (elect_one()) {
            const unsigned t = warp - kTcMma;
            const uint32_t sbase = smem_u32(sm), rbase = smem_u32(ring);
            const uint32_t id_s = idesc_bf16_f32(128, kTcKeys), id_o = idesc_bf16_f32_bmn(128, HD);
            const uint32_t ss = tmem + t * 128, oo = tmem + 256 + t * 128;
            unsigned s_item = 0, p_item = 0, su = t, pu = t;   // items begun, units, of S and of P V
            unsigned s_end = 0, p_end = 0;                     // the first unit behind the item begun last
            bool s_over = false, ok = true;
            const unsigned slot0 = t * ring_slots;
            Place kp = k_first, vp = v_first;
            auto next_s = [&]() {   // the stream's next unit's scores, if there is one; false: gave up
                while (!s_over && su >= s_end) {
                    if (!mbar_wait(&x.item_full[s_item % kTcItems], s_item / kTcItems & 1u, ab)) return false;
                    const PagedItem &it = x.item[s_item % kTcItems];
                    if (!it.more) {
                        s_over = true;
                        break;
                    }
                    s_end += it.t1 - it.t0;
                    if (!mbar_wait(&x.q_full[s_item & 1], s_item >> 1 & 1u, ab)) return false;
                    if (su >= s_end) tc_commit(&x.q_empty[s_item & 1]);   // no unit of it is this stream's
                    ++s_item;
                }
                if (s_over) return true;
                const unsigned slot = slot0 + kp.slot;
                if (!mbar_wait(&x.full[slot], kp.phase, ab)) return false;
                tc_fence_after();
                const uint64_t qd = sdesc_kmajor_sw128(sbase + ((s_item - 1) & 1) * qbytes);
                const uint64_t kd = sdesc_kmajor_sw128(rbase + slot * kTile, H * 1024);
                const uint32_t qh = (uint32_t)geo.q_half >> 4;
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks)
                    tc_mma_bf16(ss, qd + (uint64_t)((ks >> 2) * qh + (ks & 3) * 2),
                                kd + (uint64_t)((ks >> 2) * 64 + (ks & 3) * 2), id_s, ks > 0);
                // (also: P V of the unit before is complete, so that the softmax may rescale O)
                tc_commit(&x.s_full[t]);
                tc_commit(&x.empty[slot]);
                next_unit(kp);
                su += 2;
                if (su >= s_end) tc_commit(&x.q_empty[(s_item - 1) & 1]);
                return true;
            };
            int p_tile = 0, p_lo = 0, p_hi = 0;
            bool fresh = true;   // no MMA of the item has written the stream's O
            ok = next_s();
            while (ok) {
                while (ok && pu >= p_end) {
                    ok = mbar_wait(&x.item_full[p_item % kTcItems], p_item / kTcItems & 1u, ab);
                    if (!ok) break;
                    const PagedItem &it = x.item[p_item % kTcItems];
                    if (!it.more) break;
                    p_tile = it.t0 + (int)(pu - p_end);
                    p_end += it.t1 - it.t0;
                    p_lo = it.lo;
                    p_hi = it.hi;
                    fresh = true;
                    ok = p_item == 0 || mbar_wait(&x.o_free, (p_item - 1) & 1u, ab);
                    if (ok && pu >= p_end) {   // no unit of it is this stream's
                        tc_commit(&x.o_done);
                        mbar_arrive(&x.item_empty[p_item % kTcItems]);
                    }
                    ++p_item;
                }
                if (!ok || pu >= p_end) break;
                ok = mbar_wait(&x.full[slot0 + vp.slot], vp.phase, ab) && mbar_wait(&x.p_full[t], pu >> 1 & 1u, ab);
                if (!ok) break;
                tc_fence_after();
                const int base = p_tile * kTcKeys;
                const int k0 = (max(p_lo - base, 0)) / 16, k1 = (min(p_hi - base, kTcKeys) + 15) / 16;
                const uint64_t vd = sdesc_mnmajor_sw128(rbase + (slot0 + vp.slot) * kTile, 1024, H * 1024);
#pragma unroll
                for (int ks = 0; ks < kTcKeys / 16; ++ks)   // 16 keys are 2 H KB of the tile
                    if (ks >= k0 && ks < k1)
                        tc_mma_bf16_ta(oo, ss + (uint32_t)ks * 8, vd + (uint64_t)(ks * 2 * H * 1024 >> 4), id_o,
                                       !fresh || ks > k0);
                if (k0 < k1) fresh = false;
                tc_commit(&x.empty[slot0 + vp.slot]);
                next_unit(vp);
                p_tile += 2;
                pu += 2;
                if (pu >= p_end) {
                    tc_commit(&x.o_done);
                    mbar_arrive(&x.item_empty[(p_item - 1) % kTcItems]);
                }
                ok = next_s();
            }
            if (!ok) give_up();
            volatile int never = 0;
            tc_commit(&x.done);
            mbar_wait(&x.done, 0, &never);
        }
    } else {
        // ---------------- softmax and output: stream s, row r = TMEM lane
        const int s = warp >> 2, wq = warp & 3, r = 32 * wq + lane;
        const uint32_t lanes = (uint32_t)(32 * wq) << 16;
        const uint32_t t_s = tmem + lanes + s * 128, t_o = tmem + lanes + 256;
        const float c = a.scale_log2;
        bf16 *out = static_cast<bf16 *>(a.out);
        const int win = a.window > 0 ? a.window : 0x7fffffff;
        auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab)) != 0;
        };
        // barrier of the softmax threads that also tells each of them whether any failed
        auto soft_sync_any = [&](bool fail) -> bool {
            uint32_t any;
            asm volatile(
                "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, 1, %2, q;\n"
                " selp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(any)
                : "r"((uint32_t)fail), "n"(kTcSoft)
                : "memory");
            return any != 0;
        };
        unsigned u0 = 0;   // the CTA's units before this item
        Place vp = v_first;   // of this stream's next unit
        for (unsigned i = 0;; ++i) {
            bool ok = warp_wait(&x.item_full[i % kTcItems], i / kTcItems & 1u);
            if (soft_sync_any(!ok)) {
                give_up();
                break;
            }
            const PagedItem it = x.item[i % kTcItems];
            if (!it.more) break;
            const int units = it.t1 - it.t0;
            const bool active = 32 * wq < it.n_rows;   // the warp has rows
            const int row = it.row0 + r, tok = row / a.group, hd = row - tok * a.group;
            const bool mine = r < it.n_rows;
            const int pos = mine ? max(it.pos0 + tok, -1) : -1;   // -1: sees no key
            const int see_lo = max(it.lo, pos - win + 1), see_hi = min(pos, it.hi - 1);
            // keys that some rows of the tile see and others do not
            const int pos_a = max(it.pos0 + it.tok_a, -1), pos_b = max(it.pos0 + it.tok_b, -1);
            const int win_a = max(pos_a - win + 1, 0), win_b = max(pos_b - win + 1, 0);
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int k = (int)((s ^ u0) & 1u); k < units; k += 2) {
                const unsigned u = u0 + k, nth = u >> 1;
                const int base = (it.t0 + k) * kTcKeys;
                const int end = min(it.hi - base, kTcKeys);   // columns [beg, end) are the item's keys
                const int beg = max(it.lo - base, 0);
                const int q0 = beg >> 5, q1 = (end + 31) >> 5;   // the 32-column parts they lie in
                ok = ok && warp_wait(&x.s_full[s], nth & 1u);
                if (ok && active) {
                    tc_fence_after();
                    // 32 scores at a time, read once for the maximum and again for the weights (P
                    // of columns 32 q .. covers columns 16 q .., which are read by then).  Loops
                    // that are not unrolled: the instructions of a fully unrolled unit took
                    // longer to fetch, in a short call, than to run.
                    uint32_t v[32];
                    const uint32_t there = *const_cast<volatile uint32_t *>(&x.there[u % 8]);
                    const int c0 = see_lo - base, c1 = see_hi - base;   // the row's keys, in columns
                    const bool whole = __all_sync(0xffffffffu, (c0 <= 0 && c1 >= kTcKeys - 1) || !mine) && there == 0xffffu;
                    auto load = [&](int q) {
                        tmem_ld32_async(t_s + 32 * q, v);
                        tmem_wait_ld32(v);
                        if (!whole) {
                            // the row's keys among these 32: bits c0 .. c1, and 8 for every page bit
                            const int f = max(c0 - 32 * q, 0), t = min(c1 - 32 * q, 31);
                            uint32_t in = t >= f ? (0xffffffffu >> (31 - t)) & (0xffffffffu << f) : 0u;
                            const uint32_t pg = there >> (4 * q) & 15u;
                            in &= (pg & 1u) * 0xffu | (pg >> 1 & 1u) * 0xff00u | (pg >> 2 & 1u) * 0xff0000u |
                                  (pg >> 3) * 0xff000000u;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(in >> e & 1u)) v[e] = 0xff800000u;   // -inf: its weight is 0
                        }
                    };
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int q = q0; q < q1; ++q) {
                        load(q);
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
#pragma unroll
                            for (int y = 0; y < 4; ++y)
                                mx4[y] = fmaxf(fmaxf(mx4[y], __uint_as_float(v[e + y])), __uint_as_float(v[e + y + 4]));
                    }
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                    const float top = mx * c;   // c > 0
                    if (first) {
                        m = top;
                        first = false;
                    } else {
                        const bool move = top > m + 8.f;   // (also from -inf)
                        if (__any_sync(0xffffffffu, move && mine)) {
                            const float f = move ? exp2f(m - top) : 1.f;   // m = -inf: 0, and O is 0
                            if (move) m = top;
                            l *= f;
                            // (O of the stream's unit before is complete: its MMAs precede this S)
#pragma unroll 1
                            for (int q = 0; q < HD / 32; ++q) {
                                uint32_t o[32];
                                tmem_ld32_async(t_o + s * 128 + 32 * q, o);
                                tmem_wait_ld32(o);
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st32(t_o + s * 128 + 32 * q, o);
                            }
                        }
                    }
                    const float off = m == -INFINITY ? 0.f : m;
                    const uint64_t cc = pack_f32x2(c, c), oo = pack_f32x2(-off, -off);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
                    for (int q = q0; q < q1; ++q) {
                        load(q);
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p0, p1;
                            const float2 y = unpack_f32x2(fma_f32x2(
                                pack_f32x2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), cc, oo));
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(y.x));
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(y.y));
                            sum[e & 1] = add_f32x2(sum[e & 1], pack_f32x2(p0, p1));
                            const __nv_bfloat162 pk = __floats2bfloat162_rn(p0, p1);
                            p[e] = *reinterpret_cast<const uint32_t *>(&pk);
                        }
                        tmem_st16(t_s + 16 * q, p);
                    }
                    const float2 s0 = unpack_f32x2(sum[0]), s1 = unpack_f32x2(sum[1]);
                    l += (s0.x + s1.x) + (s0.y + s1.y);
                    tmem_wait_st();
                }
                // ---- V rows of the tile that no row, or not every row, may take as they are
                const bool edge = ((beg | end) & 15) != 0 && end > beg;
                // columns only some rows see: keys pos_a + 1 .. pos_b, and win_a .. win_b - 1
                const int h0 = max(pos_a + 1 - base, beg), h1 = min(pos_b + 1 - base, end);
                const int g0 = max(win_a - base, beg), g1 = min(win_b - base, end);
                if (ok && (edge || h0 < h1 || g0 < g1)) {
                    const unsigned slot = s * ring_slots + vp.slot;
                    unsigned char *vt = ring + slot * kTile;
                    ok = warp_wait(&x.full[slot], vp.phase);
                    if (ok) {
                        const int t = threadIdx.x & 127;
                        auto chunk = [&](int key, int d16) {   // 16 bytes of dims 8 d16 .. of a V row
                            return reinterpret_cast<uint4 *>(vt + (uint32_t)(key >> 3) * (H * 1024) +
                                                             (uint32_t)(d16 >> 3) * 1024 + (uint32_t)(key & 7) * 128 +
                                                             (uint32_t)(((d16 & 7) ^ (key & 7)) * 16));
                        };
                        if (edge) {
                            const int b0 = beg & ~15, e1 = (end + 15) & ~15, n0 = beg - b0, n = n0 + e1 - end;
#pragma unroll 1
                            for (int y = t; y < n * (HD / 8); y += 128) {
                                const int z = y / (HD / 8);
                                *chunk(z < n0 ? b0 + z : end + z - n0, y % (HD / 8)) = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
                        auto finite_only = [&](int f0, int f1) {
#pragma unroll 1
                            for (int y = t; y < (f1 - f0) * (HD / 8); y += 128) {
                                uint4 *at = chunk(f0 + y / (HD / 8), y % (HD / 8));
                                uint4 w4 = *at;
                                uint32_t *w = reinterpret_cast<uint32_t *>(&w4);
                                bool bad = false;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    if ((w[e] & 0x7f80u) == 0x7f80u) {
                                        w[e] &= 0xffff0000u;
                                        bad = true;
                                    }
                                    if ((w[e] & 0x7f800000u) == 0x7f800000u) {
                                        w[e] &= 0xffffu;
                                        bad = true;
                                    }
                                }
                                if (bad) {
                                    *at = w4;
                                    x.poison[i & 1] = 1;
                                }
                            }
                        };
                        if (h0 < h1) finite_only(h0, h1);
                        if (g0 < g1) finite_only(g0, g1);
                        fence_proxy_async_smem();   // before the MMA reads the tile
                    }
                }
                next_unit(vp);
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&x.p_full[s]);
            }
            // ---- the item's rows: both streams' O, this warp's half of the dims
            x.ml[s][r] = make_float2(first ? -INFINITY : m, l);
            ok = ok && warp_wait(&x.o_done, i & 1u);
            if (soft_sync_any(!ok)) {
                give_up();
                break;
            }
            const float2 a0 = x.ml[0][r], a1 = x.ml[1][r];
            const bool poison = *const_cast<volatile int *>(&x.poison[i & 1]) != 0;
            if (threadIdx.x == 0) x.poison[(i + 1) & 1] = 0;
            asm volatile("bar.sync 1, %0;" ::"n"(kTcSoft) : "memory");   // ml may be rewritten
            if (active) {
                tc_fence_after();
                // the units that have a key: an MMA wrote the O of their streams
                const int ka = max(it.lo / kTcKeys - it.t0, 0);
                const int kb = it.hi > it.lo ? min((it.hi + kTcKeys - 1) / kTcKeys - it.t0, units) : 0;
                const bool has0 = kb - ka >= 2 || (kb - ka == 1 && ((u0 + ka) & 1u) == 0);
                const bool has1 = kb - ka >= 2 || (kb - ka == 1 && ((u0 + ka) & 1u) == 1);
                const float mm = fmaxf(a0.x, a1.x), ref = mm == -INFINITY ? 0.f : mm;
                float f0, f1;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f0) : "f"(a0.x - ref));
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f1) : "f"(a1.x - ref));
                const float sum = f0 * a0.y + f1 * a1.y;
                const bool part = it.part >= 0;
                if (!part) {   // the output's scale goes into the streams' factors
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    f0 *= inv;
                    f1 *= inv;
                }
                const size_t at = (size_t)it.part * a.rows + r;
                if (part && mine && s == 0) {
                    float *ml = reinterpret_cast<float *>(a.ws + lay.ml) + at * 2;
                    ml[0] = mm;
                    ml[1] = sum;
                }
                float *po = reinterpret_cast<float *>(a.ws + lay.o) + at * HD;
                bf16 *dst = out + (long long)(it.token + tok) * a.out_stride + (it.head * a.group + hd) * HD;
#pragma unroll 1
                for (int q = 0; q < HD / 64; ++q) {
                    const int d = s * (HD / 2) + 32 * q;
                    uint32_t o0[32], o1[32];
                    tmem_ld32_async(t_o + d, o0);
                    tmem_ld32_async(t_o + 128 + d, o1);
                    tmem_wait_ld32(o0);
                    tmem_wait_ld32(o1);
                    float o[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        o[e] = has0 ? f0 * __uint_as_float(o0[e]) : 0.f;
                        if (has1) o[e] = fmaf(f1, __uint_as_float(o1[e]), o[e]);
                    }
                    if (mine && part) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(po + d + 4 * e) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const __nv_bfloat162 pk = __floats2bfloat162_rn(o[8 * e + 2 * y], o[8 * e + 2 * y + 1]);
                                w[y] = *reinterpret_cast<const uint32_t *>(&pk);
                            }
                            *reinterpret_cast<uint4 *>(dst + d + 8 * e) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                }
                if (poison && mine) {
                    // what was taken out of the V rows that this row sees and others do not: an
                    // infinity or a NaN is added to what was just stored
                    auto add = [&](int j0, int j1) {
                        const int f = max(j0, max(see_lo, it.t0 * kTcKeys)), t = min(j1, min(see_hi + 1, it.t1 * kTcKeys));
#pragma unroll 1
                        for (int j = f; j < t; ++j) {
                            const int page = key_page(a, a.s.table + (long long)it.seq * a.s.table_stride, j);
                            if (page < 0) continue;
                            const bf16 *vr = static_cast<const bf16 *>(a.kv.v) + page * a.kv.page_stride +
                                             (j % a.kv.page_size) * a.kv.slot_stride + it.head * a.kv.head_stride;
#pragma unroll 1
                            for (int d = s * (HD / 2); d < (s + 1) * (HD / 2); ++d) {
                                const float vv = __bfloat162float(vr[d]);
                                if (isfinite(vv)) continue;
                                if (part) po[d] += vv;
                                else dst[d] = __float2bfloat16_rn(__bfloat162float(dst[d]) + vv);
                            }
                        }
                    };
                    add(pos_a + 1, pos_b + 1);
                    // a key of both ranges is added once
                    add(win_a, min(win_b, pos_a + 1));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&x.o_free);
                mbar_arrive(&x.item_empty[i % kTcItems]);
            }
            u0 += units;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kTcMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host side

static int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

cudaError_t paged_attn_tc(AttnArgs &a, cudaStream_t st, int nsm)
{
    const int hd = a.kv.head_dim, halves = hd / 64;
    TcGeometry g;
    g.toks = a.rows / a.group;
    g.q_half = (a.rows + 7) / 8 * 8 * 128;
    g.box = gcd(a.kv.page_size, kTcKeys);
    g.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (1 << i == a.kv.page_size) g.page_shift = i;
    const int tile = halves * kTcKeys * 128, qbytes = 2 * halves * g.q_half;
    g.slots = (kTcSmem - (int)sizeof(TcMisc) - qbytes) / tile;
    if (g.slots > kTcMaxSlots) g.slots = kTcMaxSlots;
    g.slots &= ~1;   // two rings
    const int smem = qbytes + g.slots * tile + (int)sizeof(TcMisc);

    CUtensorMap qm, km, vm;
    const int n_heads = a.group * a.kv.n_kv_heads;
    const long long qd[3] = {hd, n_heads, a.s.n_tokens}, qs[2] = {hd, a.q_stride};
    const int qb[3] = {64, a.group, g.toks};
    cudaError_t e = tc::make_map_bf16_nd(&qm, a.q, 3, qd, qs, qb);
    const bool adj = heads_adjacent(a.kv);
    const long long per = adj ? 1 : a.kv.page_stride / a.kv.head_stride;
    const long long n_at = adj ? a.kv.n_pages : per * (a.kv.n_pages - 1) + a.kv.n_kv_heads;
    g.block = adj ? halves : 0;
    g.page_mul = (int)per;
    g.head_mul = adj ? 0 : 1;
    g.none = (int)n_at;
    const long long cd[5] = {64, 8, adj ? halves * a.kv.n_kv_heads : halves, a.kv.page_size / 8, n_at};
    const long long cs[4] = {a.kv.slot_stride, 64, 8 * a.kv.slot_stride, adj ? a.kv.page_stride : a.kv.head_stride};
    const int cb[5] = {64, 8, halves, g.box / 8, 1};
    if (!e) e = tc::make_map_bf16_nd(&km, a.kv.k, 5, cd, cs, cb);
    if (!e) e = tc::make_map_bf16_nd(&vm, a.kv.v, 5, cd, cs, cb);
    if (e) return e;
    const int grid = paged_attn_grid(a, kTcKeys, nsm < kAttnMaxCtasTc ? nsm : kAttnMaxCtasTc);
    static PerDevice once[2];
    auto kernel = hd == 64 ? k_paged_attn_tc<64> : k_paged_attn_tc<128>;
    e = allow_once(once[hd == 64], kernel, kTcSmem);
    if (!e) e = launch_pdl(kernel, dim3(grid), dim3(kTcThreads), (size_t)smem, st, qm, km, vm, a, g);
    if (!e && !a.whole) e = paged_join_tc(a, grid, nsm, st);
    return e;
}

}  // namespace ds4g
