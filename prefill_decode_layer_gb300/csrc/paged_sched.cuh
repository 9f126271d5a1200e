// Division of paged attention's work among the CTAs of a launch, on the device.
//
// An item is one row tile of one sequence and K/V head: up to `rows` query rows
// (row r of a sequence: new token r / group, head r % group of the K/V head's group),
// all of them over the sequence's keys [lo, hi).  A unit is kt keys of an item.  With U
// units in all, CTA c of G takes units [c U / G, (c + 1) U / G), items in the order
// (sequence, K/V head, row tile), so that ragged lengths still give every CTA the same
// number of units.  An item that lies in one CTA is written to the output; a CTA's share
// of an item that others share goes to the workspace as a part (row maxima, row sums,
// unnormalised rows), and k_paged_join adds the parts in CTA order.  A CTA has at most
// two parts: of the item it begins in (slot 2c) and of the one it ends in (slot 2c + 1).
// Where no item can have more than a few units (a short window or table), items are not cut
// and the unit of the division is the item (a.whole).
#pragma once

#include "paged.h"

namespace ds4g {

// Most CTAs of the two forms (the workspace holds two parts for each).
constexpr int kAttnMaxCtas = 320;      // FP32 form: two CTAs per SM (a multiple of 64)
constexpr int kAttnMaxCtasTc = 160;    // tensor-core form: one
constexpr int kAttnRowsSimt = 4;       // query rows of an FP32 row tile
// Status word of a CTA in which a bounded wait gave up.  Any other word (memory that was never
// written) says that none has, and no call clears the words: a time-out stays until it is read,
// behind however many calls on the workspace.
constexpr int kAttnTimedOut = 0x54494d45;

struct PagedItem {
    int seq, head;          // sequence, K/V head
    int token;              // row of the token arrays of the sequence's first new token
    int pos0;               // position of its first new token
    int row0, n_rows;       // query rows of the tile
    int tok_a, tok_b;       // the new tokens (of the sequence) of its first and last row
    int lo, hi;             // keys that some row of the tile sees: [lo, hi)
    int t0, t1;             // this CTA's key tiles of the item
    int part;               // slot of the workspace, or -1: the whole item is here
    int more;               // 0: no item (the CTA is done)
};

// What the join needs of an item that begins in CTA c and ends in a later one.
struct __align__(16) PagedSplit {
    int last_cta, head, token, row0;
};

// Workspace: per CTA whether a bounded wait gave up (kAttnTimedOut), the rows of
// its split item (0: none begins in it) and that item's record; then the parts, [2 ctas][rows][2]
// maxima and sums and [2 ctas][rows][head_dim] rows.
struct PartLayout {
    size_t status, n_rows, split, ml, o, total;   // byte offsets
    __host__ __device__ PartLayout(int ctas, int rows, int head_dim)
    {
        status = 0;
        n_rows = (size_t)kAttnMaxCtas * 4;
        split = n_rows + (size_t)kAttnMaxCtas * 4;
        ml = split + (size_t)kAttnMaxCtas * sizeof(PagedSplit);
        o = (ml + (size_t)2 * ctas * rows * 2 * 4 + 255) & ~(size_t)255;
        total = o + (size_t)2 * ctas * rows * head_dim * 4;
    }
};
static_assert(kAttnMaxCtas * 4 % 256 == 0, "the arrays of the workspace are aligned");

// This CTA's count of rows in the workspace at the start of a launch (all threads; those of CTAs
// that the grid does not have are cleared too).
__device__ __forceinline__ void paged_begin(const AttnArgs &a, const PartLayout &lay)
{
    int *n_rows = reinterpret_cast<int *>(a.ws + lay.n_rows);
    for (int c = blockIdx.x + gridDim.x * threadIdx.x; c < kAttnMaxCtas; c += gridDim.x * blockDim.x) n_rows[c] = 0;
}

// A sequence's keys, new tokens and units.
struct SeqWork {
    int token, n_new, pos0, lo, hi, tiles, row_tiles;
    int units;   // fits: checked by the host
};
__device__ __forceinline__ SeqWork seq_work(const AttnArgs &a, int b, int kt)
{
    SeqWork w;
    const int length = a.s.length[b];
    int first = b, n = 1;
    if (a.s.start) {
        first = a.s.start[b];
        n = a.s.start[b + 1] - first;
    }
    // no row outside the token arrays, whatever start holds
    if (first < 0 || first > a.s.n_tokens) n = 0;
    n = min(min(n, a.s.max_new), a.s.n_tokens - first);
    n = max(n, 0);
    const int cap = a.s.width * a.kv.page_size;   // fits: checked by the host
    const int len = max(length, 0);
    w.token = first;
    w.n_new = n;
    w.pos0 = len - n;
    w.hi = min(len, cap);
    // (a token before position 0 sees no key; any window of 32 bits stays in range)
    w.lo = a.window > 0 ? min(max(max(w.pos0, 0) - a.window + 1, 0), w.hi) : 0;
    const int t = w.hi > w.lo ? (w.hi + kt - 1) / kt - w.lo / kt : 1;   // one empty unit still writes zeros
    w.tiles = t;
    w.row_tiles = a.rows >= a.s.max_new * a.group ? min(n, 1) : (n * a.group + a.rows - 1) / a.rows;
    w.units = a.kv.n_kv_heads * w.row_tiles * (a.whole ? 1 : t);
    return w;
}

// Where a CTA's units begin; found once by all its threads.
struct PagedCursor {
    long long total;        // units of the launch
    long long at, end;      // this CTA's remaining units
    int local;              // unit `at` within sequence seq
    int seq, ctas;          // ctas: those that have units
    SeqWork w;              // of sequence seq
};

// floor(c total / g) for c <= g (the quotient of 32-bit numbers where that is enough: a
// 64-bit division is a hundred instructions on the way to the first copy)
__device__ __forceinline__ long long share(long long total, int c, int g)
{
    if (total < (1ll << 22)) return (unsigned)total * (unsigned)c / (unsigned)g;   // c <= 512
    return total * c / g;
}

// All NT threads of the CTA (a multiple of 32); the result is in *cur (shared memory) after
// it returns.  scratch: NT / 32 shared 64-bit words.
template <int NT>
__device__ __forceinline__ void paged_cursor(const AttnArgs &a, int kt, PagedCursor *cur, long long *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.s.n_seqs + NT - 1) / NT;
    const int b0 = min(tid * per, a.s.n_seqs), b1 = min(b0 + per, a.s.n_seqs);
    long long mine = 0;
    SeqWork w;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
        w = seq_work(a, b, kt);
        mine += w.units;
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int k = 0; k < NT / 32; ++k) {
        const long long v = scratch[k];
        if (k < warp) base += v;
        total += v;
    }
    const int g = total < (long long)gridDim.x ? (int)total : (int)gridDim.x, c = (int)blockIdx.x;
    const long long u0 = c < g ? share(total, c, g) : total, u1 = c < g ? share(total, c + 1, g) : total;
    if (tid == 0) {
        cur->total = total;
        cur->at = u0;
        cur->end = u1;
        cur->ctas = g;
    }
    long long s = base + incl - mine;   // units before this thread's sequences
    if (u0 < u1 && s <= u0 && u0 < s + mine) {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            if (per > 1) w = seq_work(a, b, kt);
            if (u0 < s + w.units) {
                cur->seq = b;
                cur->local = (int)(u0 - s);
                cur->w = w;
                break;
            }
            s += w.units;
        }
    }
    __syncthreads();
}

// The same by one warp, for up to 32 sequences (one a lane): no barrier of the CTA lies on the way
// to its first copy.
__device__ __forceinline__ void paged_cursor_warp(const AttnArgs &a, int kt, PagedCursor &cur)
{
    const int lane = threadIdx.x & 31;
    SeqWork w;
    w.units = 0;
    if (lane < a.s.n_seqs) w = seq_work(a, lane, kt);
    long long incl = w.units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const long long total = __shfl_sync(0xffffffffu, incl, 31);
    const int g = total < (long long)gridDim.x ? (int)total : (int)gridDim.x, c = (int)blockIdx.x;
    cur.total = total;
    cur.at = c < g ? share(total, c, g) : total;
    cur.end = c < g ? share(total, c + 1, g) : total;
    cur.ctas = g;
    const unsigned has = __ballot_sync(0xffffffffu, cur.at < incl);
    const int src = has ? __ffs(has) - 1 : 0;
    cur.seq = src;
    cur.local = (int)(cur.at - __shfl_sync(0xffffffffu, incl - w.units, src));
    int *words = reinterpret_cast<int *>(&w), *to = reinterpret_cast<int *>(&cur.w);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(SeqWork) / 4); ++i) to[i] = __shfl_sync(0xffffffffu, words[i], src);
}

// The CTA's next item, one thread.  `cur` is the caller's copy, kept between calls.  Writes
// the CTA's split record.
__device__ __forceinline__ void paged_next(const AttnArgs &a, int kt, PagedCursor &cur, const PartLayout &lay, PagedItem &it)
{
    it.more = cur.at < cur.end;
    if (!it.more) return;
    SeqWork &w = cur.w;
    while (cur.local >= w.units) {   // ends: cur.at < total
        cur.local -= w.units;
        w = seq_work(a, ++cur.seq, kt);
    }
    const int item = a.whole ? cur.local : cur.local / w.tiles;
    const int x = a.whole ? 0 : cur.local - item * w.tiles;
    const long long left = cur.end - cur.at;
    const int take = a.whole ? w.tiles : (int)min((long long)(w.tiles - x), left);
    const int tile0 = w.lo / kt;
    it.seq = cur.seq;
    it.head = w.row_tiles == 1 ? item : item / w.row_tiles;
    it.token = w.token;
    it.pos0 = w.pos0;
    it.row0 = w.row_tiles == 1 ? 0 : (item - it.head * w.row_tiles) * a.rows;
    it.n_rows = min(a.rows, w.n_new * a.group - it.row0);
    // (one tile: all new tokens, no division)
    const int tok_a = w.row_tiles == 1 ? 0 : it.row0 / a.group;
    const int tok_b = w.row_tiles == 1 ? w.n_new - 1 : (it.row0 + it.n_rows - 1) / a.group;
    it.hi = min(w.hi, w.pos0 + tok_b + 1);
    it.lo = a.window > 0 ? max(w.lo, max(w.pos0 + tok_a, 0) - a.window + 1) : w.lo;
    it.tok_a = tok_a;
    it.tok_b = tok_b;
    it.t0 = tile0 + x;
    it.t1 = tile0 + x + take;
    const bool begins = x == 0, ends = x + take == w.tiles;
    it.part = begins && ends ? -1 : 2 * (int)blockIdx.x + (begins ? 1 : 0);
    if (begins && !ends) {
        // the CTA of the item's last unit e: the largest c with c total / ctas <= e
        const unsigned long long e = (unsigned long long)(cur.at + w.tiles - 1);
        const PagedSplit r = {(int)(((e + 1) * (unsigned long long)cur.ctas - 1) / (unsigned long long)cur.total),
                              it.head, it.token, it.row0};
        reinterpret_cast<PagedSplit *>(a.ws + lay.split)[blockIdx.x] = r;
        reinterpret_cast<int *>(a.ws + lay.n_rows)[blockIdx.x] = it.n_rows;
    }
    cur.at += a.whole ? 1 : take;
    cur.local += a.whole ? 1 : take;
}

// Page of key j of sequence b, or -1.
__device__ __forceinline__ int key_page(const AttnArgs &a, const int *table_row, int j)
{
    const int p = table_row[j / a.kv.page_size];
    return p >= 0 && p < a.kv.n_pages ? p : -1;
}

}  // namespace ds4g
