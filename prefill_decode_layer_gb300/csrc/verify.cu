// Rows of probabilities and the verification of drafted tokens: page "ds4.c 学习笔记 --
// 端到端推理流程", 阶段四 4.3 (temperature, then the inverse-CDF draw of
// sample_full_vocab), for many rows and for tokens that a draft proposed.
//
// A row of the vocabulary (0.5 MB at 129280 tokens) is the unit of work and one cluster's:
// up to 8 CTAs of 512 threads read a contiguous chunk each, so that one row alone
// already runs on 8 SMs, and combine their maxima and sums through distributed shared
// memory; one launch, no workspace.
//
// k_probs: p = 2^((z - max z) log2(e) / T) / sum.  The row stays in registers between
// the maximum, the sum and the store (32 values per thread, 131072 per cluster; a
// larger vocabulary is read again), so that it crosses HBM once each way.
//
// k_verify: draft i is accepted while u_i q_i(d_i) < p_i(d_i) (exact: products of two
// 24-bit numbers in FP64), which every CTA of the cluster evaluates for itself.  The
// draw's weights max(p - q, 0), or p, become integers w = round(weight 2^40), as the
// sampler's do, so that every order of summation gives the same total and the drawn
// token does not depend on the split: sums of 128 consecutive tokens are kept in shared
// memory, and only the segment that holds the target R is read a second time.
#include "paged.h"
#include "sm100.cuh"

namespace ds4g {

static constexpr int kRowThreads = 512;
static constexpr int kRowWarps = kRowThreads / 32;
static constexpr int kRowTile = kRowThreads * 4;   // tokens of one round: 4 adjacent ones per thread
static constexpr int kRowHold = 8;                 // rounds a thread keeps in registers

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

// Values i .. i + 3 of a row of n (absent ones: `none`).
template <bool VEC>
__device__ __forceinline__ float4 row_load4(const float *row, int i, int n, float none)
{
    if (VEC && i + 3 < n) return *reinterpret_cast<const float4 *>(row + i);
    return make_float4(i < n ? row[i] : none, i + 1 < n ? row[i + 1] : none, i + 2 < n ? row[i + 2] : none,
                       i + 3 < n ? row[i + 3] : none);
}
template <bool VEC> __device__ __forceinline__ void row_store4(float *row, int i, int n, const float4 &v)
{
    if (VEC && i + 3 < n) {
        *reinterpret_cast<float4 *>(row + i) = v;
        return;
    }
    if (i < n) row[i] = v.x;
    if (i + 1 < n) row[i + 1] = v.y;
    if (i + 2 < n) row[i + 2] = v.z;
    if (i + 3 < n) row[i + 3] = v.w;
}

// 2^((z - m) c), c = c_hi + c_lo: the rounding errors of the difference and of the
// product are carried to the result, so that its relative error stays near that of
// exp2f also where the exponent is large.
__device__ __forceinline__ float exp_scaled(float z, float m, float c_hi, float c_lo)
{
    const float d = z - m;
    const float y = d * c_hi;
    if (!(y > -160.f)) return 0.f;   // below the smallest FP32 value (also -inf logits and 0 * -inf)
    const float t = d - z;
    const float de = (z - (d - t)) + (-m - t);   // z - m = d + de exactly
    const float r = fmaf(d, c_hi, -y) + fmaf(d, c_lo, de * c_hi);
    return exp2f(y) * fmaf(r, 0.693147180559945f, 1.f);
}

struct ProbsArgs {
    const float *z;
    float *p;
    long long zs, ps;
    int n, chunk;
    float c_hi, c_lo;   // log2(e) / T
    int greedy;
};

template <bool VEC>
__global__ void __launch_bounds__(kRowThreads, 2) k_probs(const __grid_constant__ ProbsArgs a)
{
    __shared__ float s_red[kRowWarps], s_max, s_sum;
    __shared__ unsigned long long s_red64[kRowWarps], s_key;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const long long row = blockIdx.x / size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (int)rank * a.chunk, c1 = min(a.n, c0 + a.chunk);
    const float *z = a.z + row * a.zs;
    float *p = a.p + row * a.ps;
    const int rounds = c1 > c0 ? (c1 - c0 + kRowTile - 1) / kRowTile : 0;
    pdl_wait();
    pdl_trigger();
    auto at = [&](int j) { return c0 + (j * kRowThreads + (int)threadIdx.x) * 4; };
    auto clean = [](float v) { return v != v ? -INFINITY : v; };
    float4 x[kRowHold];
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) x[j] = row_load4<VEC>(z, at(j), c1, -INFINITY);
    float mx = -INFINITY;   // fmaxf takes the number beside a NaN
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) mx = fmaxf(fmaxf(mx, fmaxf(x[j].x, x[j].y)), fmaxf(x[j].z, x[j].w));
    for (int j = kRowHold; j < rounds; ++j) {
        const float4 v = row_load4<VEC>(z, at(j), c1, -INFINITY);
        mx = fmaxf(fmaxf(mx, fmaxf(v.x, v.y)), fmaxf(v.z, v.w));
    }
    mx = clean(mx);

    if (a.greedy) {   // one at the largest logit, lowest id on ties
        unsigned long long best = 0ull;
        auto look = [&](float v, int i) {
            if (i < c1 && clean(v) > -INFINITY) {
                const unsigned long long k = ((unsigned long long)topk_key(v) << 32) | (0xffffffffu - (unsigned)i);
                best = k > best ? k : best;
            }
        };
        for (int j = 0; j < rounds; ++j) {   // a second read: the chunk is in L2
            const int i = at(j);
            const float4 v = row_load4<VEC>(z, i, c1, -INFINITY);
            look(v.x, i); look(v.y, i + 1); look(v.z, i + 2); look(v.w, i + 3);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long k = __shfl_xor_sync(0xffffffffu, best, o);
            best = k > best ? k : best;
        }
        if (lane == 0) s_red64[warp] = best;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kRowWarps; ++w) best = s_red64[w] > best ? s_red64[w] : best;
            s_key = best;
        }
        cluster_sync_all();
        best = 0ull;
        for (uint32_t r = 0; r < size; ++r) {
            const unsigned long long k = ld_cluster_u64(&s_key, r);
            best = k > best ? k : best;
        }
        cluster_sync_all();   // every CTA has read the others' key (and, in place, the row)
        const int win = best ? (int)(0xffffffffu - (unsigned)(best & 0xffffffffull)) : -1;
        for (int j = 0; j < rounds; ++j) {
            const int i = at(j);
            row_store4<VEC>(p, i, c1,
                            make_float4(i == win ? 1.f : 0.f, i + 1 == win ? 1.f : 0.f, i + 2 == win ? 1.f : 0.f,
                                        i + 3 == win ? 1.f : 0.f));
        }
        return;
    }

    mx = warp_max(mx);
    if (lane == 0) s_red[warp] = mx;
    __syncthreads();
    if (warp == 0) {
        mx = warp_max(lane < kRowWarps ? s_red[lane] : -INFINITY);
        if (lane == 0) s_max = mx;
    }
    cluster_sync_all();
    mx = -INFINITY;
    for (uint32_t r = 0; r < size; ++r) mx = fmaxf(mx, ld_cluster_f32(&s_max, r));
    const float c_hi = a.c_hi, c_lo = a.c_lo;
    const bool top_inf = mx == INFINITY, none = mx == -INFINITY;
    auto weight = [&](float v) {
        if (none || top_inf) return top_inf && v == mx ? 1.f : 0.f;
        return exp_scaled(clean(v), mx, c_hi, c_lo);
    };
    auto weight4 = [&](const float4 &v) { return make_float4(weight(v.x), weight(v.y), weight(v.z), weight(v.w)); };
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) {
        x[j] = weight4(x[j]);
        sum += (x[j].x + x[j].y) + (x[j].z + x[j].w);
    }
    for (int j = kRowHold; j < rounds; ++j) {
        const float4 v = weight4(row_load4<VEC>(z, at(j), c1, -INFINITY));
        sum += (v.x + v.y) + (v.z + v.w);
    }
    sum = warp_sum(sum);
    __syncthreads();   // s_red holds the maxima until here
    if (lane == 0) s_red[warp] = sum;
    __syncthreads();
    if (warp == 0) {
        sum = warp_sum(lane < kRowWarps ? s_red[lane] : 0.f);
        if (lane == 0) s_sum = sum;
    }
    cluster_sync_all();
    sum = 0.f;
    for (uint32_t r = 0; r < size; ++r) sum += ld_cluster_f32(&s_sum, r);
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    auto store = [&](int j, const float4 &v) {
        row_store4<VEC>(p, at(j), c1, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
    };
#pragma unroll
    for (int j = 0; j < kRowHold; ++j) store(j, x[j]);
    for (int j = kRowHold; j < rounds; ++j) store(j, weight4(row_load4<VEC>(z, at(j), c1, -INFINITY)));
    cluster_sync_all();   // no CTA leaves while another may still read its shared memory
}

// CTAs of a row's cluster: as many as keep 2048 tokens each, at most 8 (the portable
// size), so that a single row's latency is that of an eighth of it.
static int row_cluster(int n)
{
    int c = 1;
    while (c < 8 && n >= 2 * c * kRowTile) c *= 2;
    return c;
}
static int row_chunk(int n, int c) { return ((n + c - 1) / c + 3) & ~3; }

template <typename A>
static cudaError_t launch_rows(void (*kernel)(A), int rows, int cluster, cudaStream_t st, const A &a)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * cluster);
    cfg.blockDim = dim3(kRowThreads);
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

cudaError_t probs_rows(const float *logits, long long ls, int rows, int n, float temperature, float *out,
                       long long os, cudaStream_t st)
{
    if (rows == 0) return cudaSuccess;
    const int c = row_cluster(n);
    ProbsArgs a = {logits, out, ls, os, n, row_chunk(n, c), 0.f, 0.f, temperature <= 0.f};
    if (!a.greedy) {
        const double cc = 1.4426950408889634 / (double)temperature;
        a.c_hi = (float)(cc < 3e38 ? cc : 3e38);
        a.c_lo = cc < 3e38 ? (float)(cc - (double)a.c_hi) : 0.f;
    }
    const bool vec = vec_ok(logits, ls) && vec_ok(out, os);
    return vec ? launch_rows(k_probs<true>, rows, c, st, a) : launch_rows(k_probs<false>, rows, c, st, a);
}

// ------------------------------------------------------------------ verification

static constexpr int kVerifySegs = kMaxRowVocab / 8 / kRowTile * kRowWarps;   // 128-token segments of a chunk
static constexpr int kMaxDrafts = 64;

__device__ __forceinline__ float unit_prob(float v) { return v > 0.f ? fminf(v, 1.f) : 0.f; }   // NaN: 0

__device__ __forceinline__ unsigned long long weight_q(float w)
{
    return (unsigned long long)__float2ll_rn(w * 1099511627776.f);   // 2^40, exact scaling
}

struct VerifyKArgs {
    VerifyArgs a;
    int chunk;
};

template <bool VEC>
__global__ void __launch_bounds__(kRowThreads, 2) k_verify(const __grid_constant__ VerifyKArgs args)
{
    __shared__ unsigned long long s_seg[kVerifySegs];
    __shared__ unsigned long long s_warp[kRowWarps], s_total[2];
    __shared__ unsigned s_ok[kMaxDrafts / 32];
    const VerifyArgs &a = args.a;
    const uint32_t rank = cluster_rank(), size = cluster_size();
    const int b = blockIdx.x / size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int D = a.max_drafts;
    pdl_wait();
    pdl_trigger();

    // ---- the accepted drafts
    const int nd = a.n_drafts ? min(max(a.n_drafts[b], 0), D) : D;
    const int *drafts = a.drafts + (long long)b * D;
    const unsigned *u24 = a.u24 + (long long)b * (D + 1);
    const float *pseq = a.p + (long long)b * a.ps;
    const float *qseq = a.q ? a.q + (long long)b * a.qs : nullptr;
    if (threadIdx.x < kMaxDrafts) {
        const int i = threadIdx.x;
        bool ok = false;
        if (i < nd) {
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
    int k = 0;
    while (k < nd && (s_ok[k >> 5] >> (k & 31) & 1u)) ++k;
    const bool rejected = k < nd;
    const float *prow = pseq + k * a.pstride;
    const float *qrow = rejected && qseq ? qseq + k * a.qstride : nullptr;
    const int gone = rejected && !qseq ? drafts[k] : -1;   // without q: the rejected token's weight is 0

    // ---- the weights of tokens i .. i + 3 as integers; alone: those of p
    const int c0 = (int)rank * args.chunk, c1 = min(a.n, c0 + args.chunk);
    const int rounds = c1 > c0 ? (c1 - c0 + kRowTile - 1) / kRowTile : 0;
    auto weights4 = [&](const float4 &p, const float4 &q, int i, bool alone, unsigned long long (&w)[4]) {
        const float pv[4] = {p.x, p.y, p.z, p.w}, qv[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float v = unit_prob(pv[e]);
            if (!alone) {
                v = fmaxf(v - unit_prob(qv[e]), 0.f);
                if (i + e == gone) v = 0.f;
            }
            w[e] = weight_q(v);
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
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = c0 + ((j0 + u) * kRowThreads + (int)threadIdx.x) * 4;
                p[u] = j0 + u < rounds ? row_load4<VEC>(prow, i, c1, 0.f) : zero4;
                q[u] = j0 + u < rounds && with_q ? row_load4<VEC>(qrow, i, c1, 0.f) : zero4;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (j0 + u >= rounds) break;
                const int i = c0 + ((j0 + u) * kRowThreads + (int)threadIdx.x) * 4;
                unsigned long long w[4];
                weights4(p[u], q[u], i, alone, w);
                const unsigned long long s = (w[0] + w[1]) + (w[2] + w[3]);   // at most 2^42
                const unsigned lo = __reduce_add_sync(0xffffffffu, (unsigned)(s & 0x1fffffull));
                const unsigned hi = __reduce_add_sync(0xffffffffu, (unsigned)(s >> 21));
                const unsigned long long seg = ((unsigned long long)hi << 21) + lo;
                if (lane == 0) s_seg[(j0 + u) * kRowWarps + warp] = seg;
                wsum += seg;
            }
        }
        if (lane == 0) s_warp[warp] = wsum;
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned long long t = 0ull;
            for (int w = 0; w < kRowWarps; ++w) t += s_warp[w];
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
    const int nseg = rounds * kRowWarps, per = (nseg + 31) / 32;
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
    const int j = seg / kRowWarps, w0 = seg - j * kRowWarps;
    const int i = c0 + (j * kRowThreads + w0 * 32 + lane) * 4;
    unsigned long long w[4];
    weights4(row_load4<VEC>(prow, i, c1, 0.f), qrow && !alone ? row_load4<VEC>(qrow, i, c1, 0.f) : zero4, i, alone, w);
    sum = (w[0] + w[1]) + (w[2] + w[3]);
    incl = scan(sum);
    const int hit = __ffs(__ballot_sync(0xffffffffu, incl >= left)) - 1;
    if (lane == hit) {
        unsigned long long run = incl - sum;
        int e = 0;
        while (e < 3 && run + w[e] < left) run += w[e++];
        out[k] = i + e;
    }
}

cudaError_t verify_rows(const VerifyArgs &a, int n_seqs, cudaStream_t st)
{
    if (n_seqs == 0) return cudaSuccess;
    const int c = row_cluster(a.n);
    const VerifyKArgs ka = {a, row_chunk(a.n, c)};
    bool vec = vec_ok(a.p, a.ps) && vec_ok(a.p, a.pstride);
    if (a.q) vec = vec && vec_ok(a.q, a.qs) && vec_ok(a.q, a.qstride);
    return vec ? launch_rows(k_verify<true>, n_seqs, c, st, ka) : launch_rows(k_verify<false>, n_seqs, c, st, ka);
}

}  // namespace ds4g
