// Page tables, lengths, starts and slots of many sequences from the lengths they are to have:
// the bookkeeping in front of the appends of page "ds4.c 学习笔记 -- 端到端推理流程", 阶段四 4.2,
// for a cache that is cut into pages (a session's linear cache needs none).
//
// With P slots a page, sequence b holds h_b = ceil(length_b / P) pages and needs w_b = ceil(want_b
// / P).  Pages behind the w_b of a shorter one go back to the pool, a stack; then the longer
// ones take theirs from its top.  Both in the order (sequence, index in the table):
//   the r-th page given back of R lies at n_free + R - 1 - r (the first on top),
//   the k-th page taken comes from n_free + R - 1 - k (what lies beyond the stack's room is lost before),
// so that giving back what was just taken restores the stack.  All positions are prefix sums over
// the sequences: one of (pages back, pages wanted, tokens wanted), and, after those that do not fit
// the pool or the token rows are refused, one of (pages taken, tokens).
//
// One cluster does it all, an equal share of the sequences each CTA: its sums in registers and
// shared memory, the others' through distributed shared memory, a cluster barrier where pages
// given back may be taken and where the tables are complete.  Pages are moved one a thread, found
// by a binary search in the CTA's prefix sums; slots likewise, divided evenly over the cluster.
// Bound: latency.  Of a decode step a chain of loads and barriers: 64 sequences with drafts 4.8 us a call in one CTA, 4096
// sequences 12.4 in eight.  Of prompts the slots: each new token looks for its sequence in the starts, in global memory,
// and then for its length and page, by 512 threads or 4096.  4096 sequences, 256 prompts of up to 2000 among them
// (336,374 new tokens, 2.7 MB of slots) 262 us, 45 without slots; a prompt of 131072 among 16 sequences 275, among 64 356; one of 4096 16.
// (These with the launch and whatever waits for it; the stores alone would take half a microsecond.)
#include "paged.h"
#include "sm100.cuh"

namespace ds4g {

static constexpr int kRzThreads = 512;
static constexpr int kRzWarps = kRzThreads / 32;
static constexpr int kRzCluster = 8;

// Three sums that are scanned together (the pages of all tables fit 32 bits: checked by the host).
struct __align__(16) RzSums {
    int back, more;
    long long tokens;
    __device__ __forceinline__ void add(const RzSums &o)
    {
        back += o.back;
        more += o.more;
        tokens += o.tokens;
    }
};
// Inclusive prefix over the first `n` lanes of a warp (a power of two; the others' values have no meaning).
__device__ __forceinline__ RzSums rz_scan(RzSums v, int n)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o >= n) break;
        const RzSums y = {__shfl_up_sync(0xffffffffu, v.back, o), __shfl_up_sync(0xffffffffu, v.more, o),
                          __shfl_up_sync(0xffffffffu, v.tokens, o)};
        if (lane >= o) v.add(y);
    }
    return v;
}
__device__ __forceinline__ RzSums rz_from_lane(const RzSums &v, int lane)
{
    return {__shfl_sync(0xffffffffu, v.back, lane), __shfl_sync(0xffffffffu, v.more, lane), __shfl_sync(0xffffffffu, v.tokens, lane)};
}
__device__ __forceinline__ RzSums rz_remote(const RzSums *p, uint32_t rank)
{
    RzSums v;
    const uint32_t at = cluster_map(p, rank);
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.back), "=r"(v.more) : "r"(at) : "memory");
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v.tokens) : "r"(at + 8) : "memory");
    return v;
}

// What becomes of a sequence.
struct RzSeq {
    long long want;     // its new length, if that fits
    int now, held, need;
};
__device__ __forceinline__ RzSeq rz_seq(const ResizeArgs &a, int b)
{
    RzSeq s;
    const long long cap = (long long)a.width * a.page_size;
    s.now = max(a.length[b], 0);
    s.want = max(a.want[b], 0);
    if (s.want > cap) s.want = s.now;   // refused
    s.held = (int)min(((long long)s.now + a.page_size - 1) / a.page_size, (long long)a.width);
    s.need = (int)min((s.want + a.page_size - 1) / a.page_size, (long long)a.width);
    return s;
}

// Largest i with p[i] <= x, for p[0] <= x and p[0 .. n) that does not fall.
template <typename T> __device__ __forceinline__ int rz_find(const T *p, int n, T x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (p[m] <= x) lo = m;
        else hi = m;
    }
    return lo;
}

// Dynamic shared memory: back[share + 1], more[share + 1] (pages before each of the CTA's sequences).
__global__ void __launch_bounds__(kRzThreads) k_paged_resize(const __grid_constant__ ResizeArgs a, int share)
{
    extern __shared__ int sm[];
    __shared__ RzSums s_warp[2][kRzWarps], s_cta[2];
    int *s_back = sm, *s_more = sm + share + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), size = gridDim.x;   // one cluster
    const int b0 = min((int)rank * share, a.n_seqs), n = min(share, a.n_seqs - b0);
    const int per = (share + kRzThreads - 1) / kRzThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
    pdl_wait();
    pdl_trigger();
    auto sync_all = [&]() {   // of the cluster
        if (size == 1) __syncthreads();
        else cluster_sync_all();
    };
    // Exclusive prefix of `mine` over the CTA's threads; cta: before the CTA; total: over all.
    auto scan = [&](const RzSums &mine, int which, RzSums &cta, RzSums &total) {
        RzSums before = rz_scan(mine, 32);
        if (lane == 31) s_warp[which][warp] = before;
        __syncthreads();
        // the warps' and the CTAs' sums, by every warp
        const RzSums w = rz_scan(s_warp[which][lane % kRzWarps], kRzWarps);
        total = rz_from_lane(w, kRzWarps - 1);
        const RzSums ahead = rz_from_lane(w, max(warp - 1, 0));
        if (warp > 0) before.add(ahead);
        before.add({-mine.back, -mine.more, -mine.tokens});
        cta = RzSums{0, 0, 0};
        if (size > 1) {
            if (tid == 0) s_cta[which] = total;
            cluster_sync_all();
            const RzSums c = rz_scan(rz_remote(&s_cta[which], min((uint32_t)lane, size - 1)), kRzCluster);
            total = rz_from_lane(c, (int)size - 1);
            const RzSums earlier = rz_from_lane(c, max((int)rank - 1, 0));
            if (rank > 0) cta = earlier;
        }
        return before;
    };
    const int n_free = min(max(*a.n_free, 0), a.capacity);
    RzSums mine = {0, 0, 0};
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const RzSeq s = rz_seq(a, b0 + i);
        mine.add({max(s.held - s.need, 0), max(s.need - s.held, 0), max(s.want - s.now, 0ll)});
    }
    RzSums cta, total;
    RzSums at = scan(mine, 0, cta, total);
    const long long full = (long long)n_free + total.back, back0 = cta.back;   // the stack's height, had it room
    const long long top = min(full, (long long)a.capacity);
    // ---- who fits; pages given back
    RzSums taken = {0, 0, 0}, run = at;
    unsigned long long fit = 0;   // of this thread's sequences (64 at most: per <= kResizeMaxSeqs / kRzThreads / cluster)
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const RzSeq s = rz_seq(a, b0 + i);
        const int more = max(s.need - s.held, 0);
        const long long tokens = max(s.want - s.now, 0ll);
        s_back[i] = run.back;
        run.add({max(s.held - s.need, 0), more, tokens});
        const bool ok = (more == 0 || cta.more + run.more <= top) && (tokens == 0 || cta.tokens + run.tokens <= a.max_tokens);
        if (ok) {
            taken.add({0, more, tokens});
            fit |= 1ull << (i - i0);
        }
    }
    if (i1 == n && i0 < i1) s_back[n] = run.back;
    if (n == 0 && tid == 0) s_back[0] = 0;
    RzSums cta2, total2;
    at = scan(taken, 1, cta2, total2);
    // (s_back is complete: the scan has barriers)
    for (int r = tid; r < s_back[n]; r += kRzThreads) {
        const int i = rz_find(s_back, n, r);
        const RzSeq s = rz_seq(a, b0 + i);
        int *entry = a.table + (long long)(b0 + i) * a.table_stride + s.need + (r - s_back[i]);
        const long long to = full - 1 - (back0 + r);
        if (to < a.capacity) a.free[to] = *entry;
        *entry = -1;
    }
    sync_all();   // what was given back may be taken
    // ---- lengths, starts, and the pages before each sequence
    {
        RzSums run2 = at;
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const RzSeq s = rz_seq(a, b0 + i);
            const bool ok = fit >> (i - i0) & 1ull;
            s_more[i] = run2.more;
            a.start[b0 + i] = (int)(cta2.tokens + run2.tokens);
            if (ok) run2.add({0, max(s.need - s.held, 0), max(s.want - s.now, 0ll)});
        }
        if (i1 == n && i0 < i1) s_more[n] = run2.more;
        if (n == 0 && tid == 0) s_more[0] = 0;
        if (rank == 0 && tid == 0) {
            a.start[a.n_seqs] = (int)total2.tokens;
            *a.n_free = (int)(top - total2.more);
        }
    }
    __syncthreads();
    for (int k = tid; k < s_more[n]; k += kRzThreads) {
        const int i = rz_find(s_more, n, k);
        const RzSeq s = rz_seq(a, b0 + i);
        const long long from = top - 1 - (cta2.more + k);
        a.table[(long long)(b0 + i) * a.table_stride + s.held + (k - s_more[i])] = __ldcg(a.free + from);
    }
    __syncthreads();   // every thread has read the old lengths
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        const RzSeq s = rz_seq(a, b0 + i);
        if (s.want < s.now || (fit >> (i - i0) & 1ull)) a.length[b0 + i] = (int)s.want;
    }
    sync_all();   // tables, lengths and starts are complete
    if (!a.slots) return;
    const long long tokens = total2.tokens, chunk = (tokens + size - 1) / size;
    const long long t1 = min((rank + 1) * chunk, tokens);
    for (long long t = rank * chunk + tid; t < t1; t += kRzThreads) {
        int lo = 0, hi = a.n_seqs;   // the last sequence that starts at or before t has it
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (__ldcg(a.start + m) <= t) lo = m;
            else hi = m;
        }
        const int end = lo + 1 < a.n_seqs ? __ldcg(a.start + lo + 1) : (int)tokens;
        const int pos = __ldcg(a.length + lo) - end + (int)t;
        const int page = __ldcg(a.table + (long long)lo * a.table_stride + pos / a.page_size);
        a.slots[t] = (long long)page * a.page_size + pos % a.page_size;
    }
}

cudaError_t paged_resize(const ResizeArgs &a, cudaStream_t st)
{
    // One CTA where its threads have a sequence each, a cluster of eight for more: the barriers of eight cost 3 us
    // (decode steps, one CTA and eight: 64 sequences 4.9 and 7.8 us, 512 8.4 and 8.7, 1024 13.3 and 8.5, 4096 46.8 and
    // 12.3).  Eight would gain where few sequences bring long prompts: 64 with one of 4096 tokens 15.7 and 9.7, of 131072 356 and 54.
    const int cluster = a.n_seqs <= kRzThreads ? 1 : kRzCluster;
    const int share = (a.n_seqs + cluster - 1) / cluster;
    static PerDevice once;
    const size_t smem = 2 * (size_t)(share + 1) * 4;
    cudaError_t e = allow_once(once, k_paged_resize, 2 * (size_t)(kResizeMaxSeqs / kRzCluster + 1) * 4);
    if (e) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(kRzThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    ++launch_count();
    return cudaLaunchKernelEx(&cfg, k_paged_resize, a, share);
}

}  // namespace ds4g
