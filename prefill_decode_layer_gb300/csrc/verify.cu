// Rows of probabilities and the verification of drafted tokens: page "ds4.c 学习笔记 --
// 端到端推理流程", 阶段四 4.3 (temperature, then the inverse-CDF draw of
// sample_full_vocab), for many rows and for tokens that a draft proposed.
//
// A row of the vocabulary (0.5 MB at 129280 tokens) is the unit of work and one cluster's,
// whose CTAs take a contiguous chunk each and combine their maxima and sums through distributed
// shared memory; one launch, no workspace.  k_probs: 1 to 8 CTAs up to 131072 tokens, as few as hold
// the row, more where the rows leave SMs idle; 16 above.  k_verify: 1 to 8 by the vocabulary, up to
// 16 for up to four sequences.
//
// k_probs: p = 2^((z - max z) log2(e) / T) / sum.  A CTA's chunk comes into shared memory by a
// bulk copy and crosses HBM once each way.  Every thread takes 2^((z - m) c) of its values
// against a maximum m of its own, the (m, sum) pairs are combined over the CTA and then, in
// one exchange, over the cluster, and each thread scales its values by 2^((m - M) c) / S on the
// way out.  Three CTAs fit an SM, so that the copies of some overlap the arithmetic of others.
// Bound: bytes, at many rows (320 rows of 129280, 331 MB: 68 us, 0.72 of a copy's 6.78 TB/s; with
// the chunk in registers two CTAs fit, and 56 of a GPC's 57 places against 32 of 38: 94 us); the
// launch and two passes over a chunk at one (5.3 us).  k_probs_any holds the chunk in registers and
// reads what a larger vocabulary has beyond again: for rows that begin elsewhere in a 16-byte
// line than their results, and vocabularies above 262144.
//
// k_verify: draft i is accepted while u_i q_i(d_i) < p_i(d_i) (exact: products of two
// 24-bit numbers in FP64), which every CTA of the cluster evaluates for itself.  The
// draw's weights max(p - q, 0), or p, become integers w = round(weight 2^40), as the
// sampler's do, so that every order of summation gives the same total and the drawn
// token does not depend on the split: sums of 128 consecutive tokens are kept in shared
// memory, and only the segment that holds the target R is read a second time.  Bound: bytes
// and latency at many sequences (64 with up to 8 drafts, a row of each and the draft's where one
// was rejected: 50.3 MB in 17 us, 0.44 of the copy's rate, one wave of clusters), latency at one (6.8
// us: the drafts' probabilities, the rows, the segment).
#include <atomic>

#include "paged.h"
#include "sm100.cuh"

namespace ds4g {

static constexpr int kRowThreads = 512;
static constexpr int kRowWarps = kRowThreads / 32;
static constexpr int kRowTile = kRowThreads * 4;   // tokens of one round: 4 adjacent ones per thread
static constexpr int kRowHold = 8;                 // rounds a thread keeps in registers
static constexpr int kMaxCluster = 16;

__device__ __forceinline__ float ld_cluster_f32(const float *p, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long ld_cluster_u64(const unsigned long long *p, uint32_t rank)
{
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_map(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}

// A warp's 128 consecutive tokens from t0, four per lane: adjacent ones where the row is 16-byte
// aligned (VEC), else every 32nd, so that a warp's loads and stores stay whole lines.
template <bool VEC> __device__ __forceinline__ int row_token(int t0, int lane, int e)
{
    return VEC ? t0 + 4 * lane + e : t0 + 32 * e + lane;
}
// This lane's four of them, of a row of n (absent ones: `none`).
template <bool VEC> __device__ __forceinline__ float4 row_load4(const float *row, int t0, int lane, int n, float none)
{
    if (VEC && t0 + 4 * lane + 3 < n) return *reinterpret_cast<const float4 *>(row + t0 + 4 * lane);
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = row_token<VEC>(t0, lane, e);
        v[e] = i < n ? row[i] : none;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}
template <bool VEC> __device__ __forceinline__ void row_store4(float *row, int t0, int lane, int n, const float4 &x)
{
    if (VEC && t0 + 4 * lane + 3 < n) {
        *reinterpret_cast<float4 *>(row + t0 + 4 * lane) = x;
        return;
    }
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int i = row_token<VEC>(t0, lane, e);
        if (i < n) row[i] = v[e];
    }
}

// 2^((z - m) c), c = c_hi + c_lo.  The rounding of the product is carried to the result, so
// that what is left is that of the difference, 2^-24 of the exponent (a large one belongs to
// a small result), and of the hardware's 2^x.  Results below 2^-126 are 0, and so are those of
// -inf and NaN.
__device__ __forceinline__ float exp_scaled(float z, float m, float c_hi, float c_lo)
{
    const float d = z - m, y = d * c_hi;
    const float r = fmaf(d, c_lo, fmaf(d, c_hi, -y));
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
    e *= fmaf(r, 0.693147180559945f, 1.f);
    return y > -126.f ? e : 0.f;
}

struct ProbsArgs {
    const float *z;
    float *p;
    long long zs, ps;
    int n, chunk, rows;
    float c_hi, c_lo;   // log2(e) / T
    int greedy;
};

// The larger of two argmax candidates (key of the value, then the lower id); 0: none.
__device__ __forceinline__ unsigned long long arg_key(float v, int i)
{
    return v > -INFINITY ? ((unsigned long long)topk_key(v) << 32) | (0xffffffffu - (unsigned)i) : 0ull;
}
__device__ __forceinline__ unsigned long long max64(unsigned long long a, unsigned long long b) { return a > b ? a : b; }
__device__ __forceinline__ unsigned long long warp_max64(unsigned long long v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max64(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
// Values i, i + step, .. of the row that is 1 at id `win`.
__device__ __forceinline__ float4 one_hot4(int i, int step, int win)
{
    return make_float4(i == win ? 1.f : 0.f, i + step == win ? 1.f : 0.f, i + 2 * step == win ? 1.f : 0.f,
                       i + 3 * step == win ? 1.f : 0.f);
}
__device__ __forceinline__ unsigned long long arg_key4(const float4 &v, int i, int step)
{
    return max64(max64(arg_key(v.x, i), arg_key(v.y, i + step)),
                 max64(arg_key(v.z, i + 2 * step), arg_key(v.w, i + 3 * step)));
}
__device__ __forceinline__ int key_id(unsigned long long k) { return k ? (int)(0xffffffffu - (unsigned)(k & 0xffffffffull)) : -1; }

// Weight factor of values taken against maximum m once the maximum is M >= m (2^((m - M) c); 1
// for equal ones, infinite or absent as they may be).
__device__ __forceinline__ float rebase(float m, float M, float c_hi, float c_lo)
{
    return m == M ? 1.f : exp_scaled(m, M, c_hi, c_lo);
}

// Chunks of at most kRowHold rounds; cluster i of the grid takes rows i, i + clusters, ..  A row
// that begins `mis` floats behind a 16-byte boundary (as the rows of an odd vocabulary do) is taken
// as one that begins at the boundary, whose first `mis` values are not there; its result
// begins as far behind one.  Threads: 512, or 128 for short rows (twelve CTAs an SM).
template <int NT>
__global__ void __launch_bounds__(NT, 3 * kRowThreads / NT) k_probs(const __grid_constant__ ProbsArgs a)
{
    constexpr int kWarps = NT / 32;
    extern __shared__ __align__(16) float s_x[];   // the chunk: logits, then weights
    __shared__ float2 s_red[kWarps];
    __shared__ unsigned long long s_red64[kWarps];
    __shared__ unsigned long long s_all[2][kMaxCluster];   // what every CTA of the cluster has found, by row parity
    __shared__ uint64_t s_bar, s_all_bar[2];
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (int)rank * a.chunk;
    // of this CTA's chunk of a row: values [lo, len) are there, [bf, be) comes by the copy
    struct Span {
        const float *z;   // the chunk, 16-byte aligned
        int mis, lo, len, bf, be;
    };
    auto span = [&](int row) {
        Span s;
        const float *z = a.z + row * a.zs;
        s.mis = (int)((uintptr_t)z >> 2 & 3u);
        s.z = z - s.mis + c0;
        s.lo = max(s.mis - c0, 0);
        s.len = min(a.n + s.mis - c0, a.chunk);   // (none: a CTA without tokens)
        s.bf = (s.lo + 3) & ~3;
        s.be = max(s.len, 0) & ~3;
        return s;
    };
    const int clusters = gridDim.x / size;
    constexpr int kBatch = kRowHold / 2;   // vectors a thread holds at a time
    if (threadIdx.x == 0) {
        mbar_init(&s_bar, 1);
        mbar_init(&s_all_bar[0], 1);
        mbar_init(&s_all_bar[1], 1);
        mbar_fence_init();
    }
    cluster_sync_all();   // the barriers exist in every CTA
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](int row) {   // thread 0
        const Span s = span(row);
        const int n = max(s.be - s.bf, 0);
        mbar_expect_tx(&s_bar, (uint32_t)n * 4);
        if (n) bulk_g2s(s_x + s.bf, s.z + s.bf, (uint32_t)n * 4, &s_bar, policy_evict_first());
    };
    int row = blockIdx.x / size;
    if (threadIdx.x == 0 && row < a.rows) fetch(row);
    volatile int never = 0;
    // Warp 0 sends the CTA's word of this row to every CTA of the cluster; each thread returns
    // with word `lane` of the cluster's.  (A cluster barrier in its place waits for the stores of
    // the row before.)  A row's words are overwritten two rows later, by CTAs that have all words
    // of the row between, which this CTA sends after its threads have read these.
    auto exchange = [&](unsigned long long mine, int turn, bool &landed) {
        const int par = turn & 1;
        if (warp == 0) {
            if (lane == 0) mbar_expect_tx(&s_all_bar[par], size * 8);
            if (lane < (int)size)
                st_async_u64(cluster_map(&s_all[par][rank], lane), mine, cluster_map(&s_all_bar[par], lane));
        }
        landed = mbar_wait_cluster(&s_all_bar[par], (turn >> 1) & 1u) && landed;
        return lane < (int)size ? s_all[par][lane] : 0ull;
    };
    for (int turn = 0; row < a.rows; row += clusters, ++turn) {
        const Span sp = span(row);
        const int lo = sp.lo, len = sp.len, id0 = c0 - sp.mis;   // id of the chunk's value 0
        float *p = a.p + row * a.ps + id0;
        bool landed = mbar_wait(&s_bar, turn & 1u, &never);   // if the wait gave up, the row becomes NaN
        auto load4 = [&](int i) {   // (values that the copy does not bring: at most three at each end of a row)
            if (i >= sp.bf && i < sp.be) return *reinterpret_cast<const float4 *>(s_x + i);
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = i + e >= lo && i + e < len ? sp.z[i + e] : -INFINITY;
            return make_float4(v[0], v[1], v[2], v[3]);
        };
        auto store4 = [&](int i, const float4 &x) {
            if (i >= lo && i + 3 < len) {
                *reinterpret_cast<float4 *>(p + i) = x;
                return;
            }
            const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e >= lo && i + e < len) p[i + e] = v[e];
        };
        auto at = [&](int j) { return (j * NT + (int)threadIdx.x) * 4; };
        if (a.greedy) {   // one at the largest logit, lowest id on ties
            unsigned long long best = 0ull;
#pragma unroll
            for (int j = 0; j < kRowHold; ++j) {
                const int i = at(j);
                if (i >= len) break;
                const float4 v = load4(i);
                best = max64(best, arg_key4(v, id0 + i, 1));
            }
            best = warp_max64(best);
            if (lane == 0) s_red64[warp] = best;
            __syncthreads();   // (also: the buffer is free)
            if (threadIdx.x == 0 && row + clusters < a.rows) fetch(row + clusters);
            if (warp == 0) best = warp_max64(lane < kWarps ? s_red64[lane] : 0ull);
            const int win = key_id(warp_max64(exchange(best, turn, landed))) - id0;   // (none: below 0, or a value that is not there)
#pragma unroll
            for (int j = 0; j < kRowHold; ++j)
                if (at(j) < len)
                    store4(at(j), landed ? one_hot4(at(j), 1, win) : make_float4(NAN, NAN, NAN, NAN));
            continue;
        }
        // ---- weights against the maximum of each batch of the thread
        float m[2], s[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float4 x[kBatch];
            float mx = -INFINITY;   // fmaxf takes the number beside a NaN
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = at(b * kBatch + j);
                x[j] = i < len ? load4(i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                mx = fmaxf(fmaxf(mx, fmaxf(x[j].x, x[j].y)), fmaxf(x[j].z, x[j].w));
            }
            m[b] = mx;
            s[b] = 0.f;
            if (mx == INFINITY) {   // its ids have weight 1, the others none
                auto is = [](float v) { return v == INFINITY ? 0.f : -INFINITY; };
#pragma unroll
                for (int j = 0; j < kBatch; ++j) x[j] = make_float4(is(x[j].x), is(x[j].y), is(x[j].z), is(x[j].w));
                mx = 0.f;
            } else if (mx == -INFINITY) {
                mx = 0.f;   // no weight
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int i = at(b * kBatch + j);
                const float4 w = make_float4(exp_scaled(x[j].x, mx, a.c_hi, a.c_lo), exp_scaled(x[j].y, mx, a.c_hi, a.c_lo),
                                             exp_scaled(x[j].z, mx, a.c_hi, a.c_lo), exp_scaled(x[j].w, mx, a.c_hi, a.c_lo));
                s[b] += (w.x + w.y) + (w.z + w.w);
                if (i < len) *reinterpret_cast<float4 *>(s_x + i) = w;   // (the buffer holds whole vectors)
            }
        }
        // ---- (maximum, sum) of the CTA, then of the row
        float M = fmaxf(m[0], m[1]);
        const float wm = warp_max(M);
        float ws = warp_sum(s[0] * rebase(m[0], wm, a.c_hi, a.c_lo) + s[1] * rebase(m[1], wm, a.c_hi, a.c_lo));
        if (lane == 0) s_red[warp] = make_float2(wm, ws);
        __syncthreads();
        if (warp == 0) {
            const float2 v = lane < kWarps ? s_red[lane] : make_float2(-INFINITY, 0.f);
            M = warp_max(v.x);
            ws = warp_sum(v.y * rebase(v.x, M, a.c_hi, a.c_lo));
        }
        const unsigned long long word =
            exchange((unsigned long long)__float_as_uint(ws) << 32 | __float_as_uint(M), turn, landed);
        const float2 v = lane < (int)size ? make_float2(__uint_as_float((unsigned)word), __uint_as_float((unsigned)(word >> 32)))
                                          : make_float2(-INFINITY, 0.f);
        M = warp_max(v.x);
        const float total = warp_sum(v.y * rebase(v.x, M, a.c_hi, a.c_lo));
        const float inv = !landed ? NAN : total > 0.f ? 1.f / total : 0.f;
        const float f[2] = {rebase(m[0], M, a.c_hi, a.c_lo) * inv, rebase(m[1], M, a.c_hi, a.c_lo) * inv};
#pragma unroll
        for (int j = 0; j < kRowHold; ++j) {
            const int i = at(j);
            if (i >= len) break;
            const float4 w = *reinterpret_cast<const float4 *>(s_x + i);
            const float g = f[j / kBatch];
            store4(i, make_float4(w.x * g, w.y * g, w.z * g, w.w * g));
        }
        fence_proxy_async_smem();   // this thread's accesses of the buffer, before the next copy's
        __syncthreads();
        if (threadIdx.x == 0 && row + clusters < a.rows) fetch(row + clusters);
    }
    cluster_sync_all();   // no CTA leaves while another may still read its shared memory
}

// Rows of any alignment and any vocabulary, one cluster each.
template <bool VEC>
__global__ void __launch_bounds__(kRowThreads, 2) k_probs_any(const __grid_constant__ ProbsArgs a)
{
    __shared__ float s_red[kRowWarps], s_max, s_sum;
    __shared__ unsigned long long s_red64[kRowWarps], s_key;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (int)rank * a.chunk, c1 = min(a.n, c0 + a.chunk);
    const int rounds = c1 > c0 ? (c1 - c0 + kRowTile - 1) / kRowTile : 0;
    const long long row = blockIdx.x / size;
    const float *z = a.z + row * a.zs;
    float *p = a.p + row * a.ps;
    pdl_wait();
    pdl_trigger();
    auto at = [&](int j) { return c0 + (j * kRowThreads + 32 * warp) * 4; };   // the warp's 128 tokens of round j
    float4 x[kRowHold];
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) x[j] = row_load4<VEC>(z, at(j), lane, c1, -INFINITY);
    if (a.greedy) {
        unsigned long long best = 0ull;
        auto look4 = [&](const float4 &v, int t0) {   // (absent tokens are -inf)
            best = max64(best, arg_key4(v, row_token<VEC>(t0, lane, 0), VEC ? 1 : 32));
        };
#pragma unroll
        for (int j = 0; j < kRowHold; ++j) look4(x[j], at(j));
        for (int j = kRowHold; j < rounds; ++j) look4(row_load4<VEC>(z, at(j), lane, c1, -INFINITY), at(j));
        best = warp_max64(best);
        if (lane == 0) s_red64[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = warp_max64(lane < kRowWarps ? s_red64[lane] : 0ull);
            if (lane == 0) s_key = best;
        }
        cluster_sync_all();   // (in place: every CTA has read its part of the row)
        const int win = key_id(warp_max64(lane < (int)size ? ld_cluster_u64(&s_key, lane) : 0ull));
        for (int j = 0; j < rounds; ++j)
            row_store4<VEC>(p, at(j), lane, c1, one_hot4(row_token<VEC>(at(j), lane, 0), VEC ? 1 : 32, win));
        cluster_sync_all();   // no CTA leaves while another may still read its shared memory
        return;
    }
    float mx = -INFINITY;   // fmaxf takes the number beside a NaN
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) mx = fmaxf(fmaxf(mx, fmaxf(x[j].x, x[j].y)), fmaxf(x[j].z, x[j].w));
    for (int j = kRowHold; j < rounds; ++j) {
        const float4 v = row_load4<VEC>(z, at(j), lane, c1, -INFINITY);
        mx = fmaxf(fmaxf(mx, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
    }
    mx = warp_max(mx);
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
    if (warp == 0) {
        mx = warp_max(lane < kRowWarps ? s_red[lane] : -INFINITY);
        if (lane == 0) s_max = mx;
    }
    cluster_sync_all();
    mx = warp_max(lane < (int)size ? ld_cluster_f32(&s_max, lane) : -INFINITY);
    // an infinite maximum: its ids share the whole; no maximum: every weight is 0
    const bool top_inf = mx == INFINITY;
    if (top_inf || mx == -INFINITY) mx = 0.f;
    auto seen = [&](float v) { return !top_inf ? v : v == INFINITY ? 0.f : -INFINITY; };
    auto weight4 = [&](float4 v) {
        if (top_inf) v = make_float4(seen(v.x), seen(v.y), seen(v.z), seen(v.w));
        return make_float4(exp_scaled(v.x, mx, a.c_hi, a.c_lo), exp_scaled(v.y, mx, a.c_hi, a.c_lo),
                           exp_scaled(v.z, mx, a.c_hi, a.c_lo), exp_scaled(v.w, mx, a.c_hi, a.c_lo));
    };
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) {
        x[j] = weight4(x[j]);
        sum += (x[j].x + x[j].y) + (x[j].z + x[j].w);
    }
    for (int j = kRowHold; j < rounds; ++j) {
        const float4 v = weight4(row_load4<VEC>(z, at(j), lane, c1, -INFINITY));
        sum += (v.x + v.y) + (v.z + v.w);
    }
    sum = warp_sum(sum);
    if (lane == 0) s_red[warp] = sum;   // (the maxima in it were read before the cluster's barrier)
    __syncthreads();
    if (warp == 0) {
        sum = warp_sum(lane < kRowWarps ? s_red[lane] : 0.f);
        if (lane == 0) s_sum = sum;
    }
    cluster_sync_all();
    sum = warp_sum(lane < (int)size ? ld_cluster_f32(&s_sum, lane) : 0.f);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    auto store = [&](int j, const float4 &v) {
        row_store4<VEC>(p, at(j), lane, c1, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    };
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) store(j, x[j]);
    for (int j = kRowHold; j < rounds; ++j) store(j, weight4(row_load4<VEC>(z, at(j), lane, c1, -INFINITY)));
    cluster_sync_all();   // no CTA leaves while another may still read its shared memory
}

// CTAs of a row's cluster.  Probabilities: as few as hold the row, doubled while the rows leave
// SMs idle and 2048 tokens a CTA remain (4000 rows of 10000 tokens run 2.4 times as fast on one
// CTA each as on four).  Verification: as many as keep 2048 tokens each, at most 8, or 16 (more
// than the portable size) for up to four sequences: one of 129280 tokens takes 7.9 us on 16
// CTAs and 9.5 on 8, nine take 10.4 and 9.7.
static int probs_cluster(int n, int rows, int nsm)
{
    int c = 1;
    while (c < kMaxCluster && n > c * kRowHold * kRowTile) c *= 2;
    while (c < 8 && n >= 2 * c * kRowTile && (long long)rows * c < nsm) c *= 2;
    return c;
}
static int verify_cluster(int n, int seqs)
{
    const int most = seqs <= 4 ? kMaxCluster : 8;
    int c = 1;
    while (c < most && n >= 2 * c * kRowTile) c *= 2;
    return c;
}
static int row_chunk(int n, int c) { return ((n + c - 1) / c + 3) & ~3; }

template <typename A>
static cudaError_t launch_rows(PerDevice &once, void (*kernel)(A), int clusters, int cluster, int threads, size_t smem,
                               cudaStream_t st, const A &a)
{
    // (probs_go allows its buffer; clusters of 16)
    const cudaError_t e = allow_once(once, kernel, 0, true);
    if (e) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)clusters * cluster);
    cfg.blockDim = dim3((unsigned)threads);
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
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

static bool vec_ok(const void *p, long long s) { return ((uintptr_t)p & 15u) == 0 && (s & 3) == 0; }

// Clusters of c CTAs of k_probs<NT>, each with the largest buffer, that the current device holds at
// once (asked for once per device and size: whole clusters lie in one GPC, so that fewer fit
// than the SMs alone say).
template <int NT> static cudaError_t probs_go(const ProbsArgs &a, int c, int nsm, cudaStream_t st)
{
    static PerDevice once;
    static std::atomic<int> known[64][5];
    constexpr int smem = kRowHold * NT * 16;
    cudaError_t e = allow_once(once, k_probs<NT>, smem, true);
    int dev = 0, k = 0, n = 0;
    if (!e) e = cudaGetDevice(&dev);
    if (e) return e;
    while ((1 << k) < c) ++k;
    const bool keep = dev >= 0 && dev < 64;
    if (keep) n = known[dev][k].load(std::memory_order_relaxed);
    if (!n) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(nsm / c + 1) * c);
        cfg.blockDim = dim3(NT);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)c, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, k_probs<NT>, &cfg) || n < 1) {
            cudaGetLastError();
            n = nsm / c > 0 ? nsm / c : 1;
        }
        if (keep) known[dev][k].store(n, std::memory_order_relaxed);
    }
    // more rows than the GPU holds clusters take turns
    return launch_rows(once, k_probs<NT>, a.rows < n ? a.rows : n, c, NT, (size_t)a.chunk * 4, st, a);
}

cudaError_t probs_rows(const float *logits, long long ls, int rows, int n, float temperature, float *out,
                       long long os, cudaStream_t st, int nsm)
{
    if (rows == 0) return cudaSuccess;
    // rows that begin anywhere need up to three values more
    const bool vec = vec_ok(logits, ls) && vec_ok(out, os);
    const bool alike = (((uintptr_t)logits ^ (uintptr_t)out) & 15u) == 0 && ((ls ^ os) & 3) == 0;
    const int room = vec ? n : n + 3, c = probs_cluster(room, rows, nsm);
    ProbsArgs a = {logits, out, ls, os, n, row_chunk(room, c), rows, 0.f, 0.f, temperature <= 0.f};
    if (!a.greedy) {
        const double cc = 1.4426950408889634 / (double)temperature;
        a.c_hi = (float)(cc < 3e38 ? cc : 3e38);
        a.c_lo = cc < 3e38 ? (float)(cc - (double)a.c_hi) : 0.f;
    }
    // short rows: a CTA of 128 threads holds 4096 values (3700 rows of 2700 tokens: 53 us with 512)
    if (alike && c == 1 && a.chunk <= kRowHold * 128 * 4) return probs_go<128>(a, c, nsm, st);
    if (alike && a.chunk <= kRowHold * kRowTile) return probs_go<kRowThreads>(a, c, nsm, st);
    static PerDevice once[2];
    a.chunk = row_chunk(n, c);
    return vec ? launch_rows(once[1], k_probs_any<true>, rows, c, kRowThreads, 0, st, a)
               : launch_rows(once[0], k_probs_any<false>, rows, c, kRowThreads, 0, st, a);
}

// ------------------------------------------------------------------ verification

static constexpr int kVerifySegs = kMaxRowVocab / 8 / 128;   // 128-token segments of a chunk
static constexpr int kMaxDrafts = 64;

__device__ __forceinline__ float unit_prob(float v) { return v > 0.f ? fminf(v, 1.f) : 0.f; }   // NaN: 0

// round(w 2^40) of w in [0, 1] as hi 2^20 + lo (lo <= 2^20): w 2^20 and its fraction are exact, and
// so the second rounding, to nearest even, is the only one.  (One conversion to a 64-bit
// integer is the same number on a pipe of a fraction of the rate.)
__device__ __forceinline__ void weight_q(float w, unsigned &hi, unsigned &lo)
{
    const float s = w * 1048576.f;
    hi = (unsigned)s;
    lo = __float2uint_rn((s - (float)hi) * 1048576.f);
}

struct VerifyKArgs {
    VerifyArgs a;
    int chunk;
};

// Threads: 512 for few sequences (a chunk's loads all in flight at once), 256 for many (four CTAs
// an SM: 64 sequences of 8 CTAs run in one wave).
template <bool VEC, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_verify(const __grid_constant__ VerifyKArgs args)
{
    __shared__ unsigned long long s_seg[kVerifySegs];
    __shared__ unsigned long long s_warp[NT / 32], s_total[2];
    __shared__ unsigned s_ok[kMaxDrafts / 32];
    constexpr int kWarps = NT / 32, kTile = NT * 4;
    const VerifyArgs &a = args.a;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.x / size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.max_drafts;
    pdl_wait();
    pdl_trigger();

    // ---- the accepted drafts
    // (a draft is looked up whether or not the count, which comes with it, includes it)
    const int asked = a.n_drafts ? a.n_drafts[b] : D;
    const int *drafts = a.drafts + (long long)b * D;
    const unsigned *u24 = a.u24 + (long long)b * (D + 1);
    const float *pseq = a.p + (long long)b * a.ps;
    const float *qseq = a.q ? a.q + (long long)b * a.qs : nullptr;
    if (threadIdx.x < kMaxDrafts) {
        const int i = threadIdx.x;
        bool ok = false;
        if (i < D) {
            const int d = drafts[i];
            if (d >= 0 && d < a.n) {
                const float pd = unit_prob(pseq[i * a.pstride + d]);
                const float qd = qseq ? unit_prob(qseq[i * a.qstride + d]) : 1.f;
                ok = (double)(u24[i] & 0xffffffu) * (double)qd < (double)pd * 16777216.0;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) s_ok[warp] = m;
    }
    __syncthreads();
    const int nd = min(max(asked, 0), D);
    int k = 0;
    while (k < nd && (s_ok[k >> 5] >> (k & 31) & 1u)) ++k;
    const bool rejected = k < nd;
    const float *prow = pseq + k * a.pstride;
    const float *qrow = rejected && qseq ? qseq + k * a.qstride : nullptr;
    const int gone = rejected && !qseq ? drafts[k] : -1;   // without q: the rejected token's weight is 0

    // ---- the weights of tokens i .. i + 3 as integers; alone: those of p
    const int c0 = (int)rank * args.chunk, c1 = min(a.n, c0 + args.chunk);
    const int rounds = c1 > c0 ? (c1 - c0 + kTile - 1) / kTile : 0;
    // (t0: the warp's 128 tokens)
    auto weights4 = [&](const float4 &p, const float4 &q, int t0, bool alone, unsigned (&hi)[4], unsigned (&lo)[4]) {
        const float pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = unit_prob(pv[e]);
            if (!alone) {
                v = fmaxf(v - unit_prob(qv[e]), 0.f);
                if (row_token<VEC>(t0, lane, e) == gone) v = 0.f;
            }
            weight_q(v, hi[e], lo[e]);
        }
    };
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    unsigned long long before = 0ull, total = 0ull, mine = 0ull;
    bool alone = false;
    for (int mode = 0; mode < 2; ++mode) {
        alone = mode == 1;
        const bool with_q = qrow && !alone;
        unsigned long long wsum = 0ull;
        for (int j0 = 0; j0 < rounds; j0 += 4) {
            float4 p[4], q[4];
            const int first = c0 + (j0 * NT + 32 * warp) * 4;   // the warp's tokens of the four rounds
            if (VEC && first + 3 * kTile + 128 <= c1) {          // all there: eight loads without a branch
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    p[u] = *reinterpret_cast<const float4 *>(prow + first + u * kTile + 4 * lane);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    q[u] = with_q ? *reinterpret_cast<const float4 *>(qrow + first + u * kTile + 4 * lane) : zero4;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int t0 = first + u * kTile;
                    p[u] = j0 + u < rounds ? row_load4<VEC>(prow, t0, lane, c1, 0.f) : zero4;
                    q[u] = j0 + u < rounds && with_q ? row_load4<VEC>(qrow, t0, lane, c1, 0.f) : zero4;
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j0 + u >= rounds) break;
                const int t0 = c0 + ((j0 + u) * NT + 32 * warp) * 4;
                unsigned h4[4], l4[4];
                weights4(p[u], q[u], t0, alone, h4, l4);
                // 128 tokens: both halves stay below 2^28
                const unsigned lo = __reduce_add_sync(0xffffffffu, (l4[0] + l4[1]) + (l4[2] + l4[3]));
                const unsigned hi = __reduce_add_sync(0xffffffffu, (h4[0] + h4[1]) + (h4[2] + h4[3]));
                const unsigned long long seg = ((unsigned long long)hi << 20) + lo;
                if (lane == 0) s_seg[(j0 + u) * kWarps + warp] = seg;
                wsum += seg;
            }
        }
        if (lane == 0) s_warp[warp] = wsum;
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long t = 0ull;
            for (int w = 0; w < kWarps; ++w) t += s_warp[w];
            s_total[mode] = t;
        }
        cluster_sync_all();
        before = total = 0ull;
        for (uint32_t r = 0; r < size; ++r) {
            const unsigned long long t = ld_cluster_u64(&s_total[mode], r);
            if (r < rank) before += t;
            if (r == rank) mine = t;
            total += t;
        }
        if (total || !rejected) break;   // nothing left of the target: its own probabilities
    }
    cluster_sync_all();   // no CTA leaves while another may still read its total

    int *out = a.tokens + (long long)b * (D + 1);
    if (rank == 0) {
        if (threadIdx.x == 0) a.accepted[b] = k;
        if (threadIdx.x <= D) {
            const int i = threadIdx.x;
            if (i < k) out[i] = drafts[i];
            else if (i > k || !total) out[i] = -1;
        }
    }
    // target R = max(1, ceil(u24 total / 2^24)), exact in 64 bits (total < 2^61)
    const unsigned u = u24[D] & 0xffffffu;   // the draw's own number, whatever the drafts used
    unsigned long long R = u * (total >> 24) + ((u * (total & 0xffffffull) + 0xffffffull) >> 24);
    if (!R) R = 1ull;
    if (!(before < R && R <= before + mine) || warp != 0) return;

    // ---- the segment of 128 tokens in which the running sum reaches R, then the token
    unsigned long long need = R - before;
    const int nseg = rounds * kWarps, per = (nseg + 31) / 32;
    unsigned long long sum = 0ull;
    for (int i = lane * per; i < min(nseg, (lane + 1) * per); ++i) sum += s_seg[i];
    auto scan = [&](unsigned long long v) {   // inclusive over the lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    unsigned long long incl = scan(sum);
    const int src = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
    unsigned long long left = need - __shfl_sync(0xffffffffu, incl - sum, src);
    int seg = src * per;
    while (left > s_seg[seg]) left -= s_seg[seg++];   // ends: the lane's segments reach it
    const int j = seg / kWarps, w0 = seg - j * kWarps;
    const int t0 = c0 + (j * NT + w0 * 32) * 4;
    unsigned h4[4], l4[4];
    weights4(row_load4<VEC>(prow, t0, lane, c1, 0.f), qrow && !alone ? row_load4<VEC>(qrow, t0, lane, c1, 0.f) : zero4, t0,
             alone, h4, l4);
    unsigned long long w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ((unsigned long long)h4[e] << 20) + l4[e];
    if (VEC) {   // in vocabulary order: lane by lane
        sum = (w[0] + w[1]) + (w[2] + w[3]);
        incl = scan(sum);
        const int hit = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;
        if (lane == hit) {
            unsigned long long run = incl - sum;
            int e = 0;
            while (e < 3 && run + w[e] < left) run += w[e++];
            out[k] = row_token<VEC>(t0, lane, e);
        }
        return;
    }
    unsigned long long run = 0ull;   // 32 tokens by 32
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        incl = run + scan(w[e]);
        const unsigned reach = __ballot_sync(0xffffffffu, incl >= left);
        if (reach) {
            if (lane == __ffs(reach) - 1) out[k] = row_token<VEC>(t0, lane, e);
            return;
        }
        run = __shfl_sync(0xffffffffu, incl, 31);
    }
}

cudaError_t verify_rows(const VerifyArgs &a, int n_seqs, cudaStream_t st, int nsm)
{
    if (n_seqs == 0) return cudaSuccess;
    const int c = verify_cluster(a.n, n_seqs);
    const VerifyKArgs ka = {a, row_chunk(a.n, c)};
    bool vec = vec_ok(a.p, a.ps) && vec_ok(a.p, a.pstride);
    if (a.q) vec = vec && vec_ok(a.q, a.qs) && vec_ok(a.q, a.qstride);
    const bool few = (long long)n_seqs * c <= nsm;
    static PerDevice once[4];
    if (few)
        return vec ? launch_rows(once[0], k_verify<true, 512>, n_seqs, c, 512, 0, st, ka)
                   : launch_rows(once[1], k_verify<false, 512>, n_seqs, c, 512, 0, st, ka);
    return vec ? launch_rows(once[2], k_verify<true, 256>, n_seqs, c, 256, 0, st, ka)
               : launch_rows(once[3], k_verify<false, 256>, n_seqs, c, 256, 0, st, ka);
}

}  // namespace ds4g
