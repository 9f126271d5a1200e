// Attention of the newest tokens of many sequences over a paged K/V cache: page "ds4.c
// 学习笔记 -- 端到端推理流程", 阶段四 4.2 (the layer step's attention of one token over
// its cached keys), with grouped heads, several new tokens, an optional window and a
// cache cut into pages.  This file holds the FP32 form, the join of split items and
// the host side; paged_attn_tc.cu holds the tensor-core form.
//
// out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(s (q_r . k_j) - m_r),  s = scale log2 e,
// over the keys j visible to row r; m_r is the running maximum (online softmax), so
// that K and V are read once.
//
// FP32 form (k_paged_attn): for FP32 queries or caches and for head sizes and page sizes
// the tensor-core form does not take.  Lanes are split into groups of LPK that own D dims
// each, and every group is a stream of its own through the CTA's keys: it loads KB keys'
// K and V straight into registers (coalesced 16-byte loads, no shared memory).  The R x KB dot
// products of R query rows are summed over the lanes by exchanging halves, so that a lane
// ends with one of them: R KB - 1 exchanges where summing each over all lanes takes log2(LPK)
// R KB, and one 2^x a lane.  The weights then go round once (a shuffle each) for O += P V in
// registers.  The streams of an item are merged when it ends, those of a warp by shuffles, the
// eight warps through shared memory.  Bound: the cache's bytes at few rows (two CTAs an SM keep
// 64 KB of loads in flight), the issue of instructions at many: K and V pass once per four rows, and
// 15 exchanges with their selects and 16 broadcasts go with the 128 FMAs of a batch.  Measured: 16
// sequences of up to 2000 positions, 8 heads on 2 of 64, FP32, 20.8 MB: 16.3 us with the join, a
// chain of latencies (two launches, lengths, pages, keys, merge, parts); 32 sequences of 4000, 64
// heads on 8 of 64, 335 MB: 138 us, an instruction in 64 % of the issue slots (21 M of the 99 M are the
// products' FMAs), 604 MB read from DRAM because both row tiles of a K/V head read it.
#include "paged_sched.cuh"

namespace ds4g {

static constexpr int kPaThreads = 256;
static constexpr int kPaWarps = kPaThreads / 32;
static constexpr int kPaKeys = 64;    // keys of a unit

// D consecutive elements as floats (D 4 or 8; 8- or 16-byte loads of BF16, 16-byte of FP32).
template <typename T, int D> struct Load;
template <> struct Load<float, 4> {
    static __device__ __forceinline__ void run(const float *p, float (&x)[4])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    }
};
template <> struct Load<float, 8> {
    static __device__ __forceinline__ void run(const float *p, float (&x)[8])
    {
        const float4 v = *reinterpret_cast<const float4 *>(p), w = *reinterpret_cast<const float4 *>(p + 4);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
    }
};
template <> struct Load<bf16, 4> {
    static __device__ __forceinline__ void run(const bf16 *p, float (&x)[4])
    {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x[0] = __uint_as_float(v.x << 16);
        x[1] = __uint_as_float(v.x & 0xffff0000u);
        x[2] = __uint_as_float(v.y << 16);
        x[3] = __uint_as_float(v.y & 0xffff0000u);
    }
};
template <> struct Load<bf16, 8> {
    static __device__ __forceinline__ void run(const bf16 *p, float (&x)[8])
    {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
};

template <typename T> __device__ __forceinline__ void store_out(T *p, float v);
template <> __device__ __forceinline__ void store_out<float>(float *p, float v) { *p = v; }
template <> __device__ __forceinline__ void store_out<bf16>(bf16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Finite stand-in of a maximum over no key, for the exponents.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ float pa_ex2(float x)   // 2^x (hardware approximation, 2 ulp)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Dynamic shared memory: [warps][R] maxima and sums, then [warps][R][head_dim].
static size_t pa_smem(int rows, int hd) { return (size_t)kPaWarps * rows * (2 + hd) * 4; }

template <typename TQ, typename TKV, int LPK, int D, int R, int KB>
__global__ void __launch_bounds__(kPaThreads, R * D <= 16 ? 2 : 1) k_paged_attn(const __grid_constant__ AttnArgs a)
{
    constexpr int S = kPaThreads / LPK;   // streams
    constexpr int NV = R * KB;            // dot products of a batch
    constexpr int REP = LPK / NV;         // lanes that hold the same one
    static_assert(NV <= LPK, "a lane holds one dot product");
    extern __shared__ float sm[];
    __shared__ PagedCursor s_cur;
    __shared__ PagedItem s_item;
    __shared__ long long s_scratch[kPaWarps];
    const PartLayout lay(kAttnMaxCtas, kAttnRowsSimt, a.kv.head_dim);
    pdl_wait();
    pdl_trigger();
    paged_begin(a, lay);
    paged_cursor<kPaThreads>(a, kPaKeys, &s_cur, s_scratch);
    PagedCursor cur = s_cur;

    const int hd = a.kv.head_dim, ps = a.kv.page_size;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stream = threadIdx.x / LPK, sub = threadIdx.x % LPK;
    const int d0 = sub * D;
    const bool own = d0 < hd;   // head_dim is a multiple of 8: whole vectors of D
    const unsigned lanes = LPK == 32 ? 0xffffffffu : ((1u << (LPK & 31)) - 1u) << (lane / LPK * LPK);
    const int my_row = sub / REP / KB, my_key = sub / REP % KB;   // the dot product this lane ends with
    const bool one_page = ps % KB == 0;   // a batch's keys lie in one page
    float *s_m = sm, *s_l = sm + kPaWarps * R, *s_o = sm + 2 * kPaWarps * R;
    const TKV *kc = static_cast<const TKV *>(a.kv.k) + d0, *vc = static_cast<const TKV *>(a.kv.v) + d0;
    const TQ *qp = static_cast<const TQ *>(a.q) + d0;
    TQ *out = static_cast<TQ *>(a.out);
    const int win = a.window > 0 ? a.window : 0x7fffffff;

    while (true) {
        if (threadIdx.x == 0) paged_next(a, kPaKeys, cur, lay, s_item);
        __syncthreads();
        if (!s_item.more) return;
        const PagedItem it = s_item;
        const int *table = a.s.table + (long long)it.seq * a.s.table_stride;
        float q[R][D], o[R][D], m = -INFINITY, l = 0.f;   // m, l: of this lane's row (l: of its keys)
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < D; ++e) q[r][e] = o[r][e] = 0.f;
            if (r < it.n_rows && own) {
                const int row = it.row0 + r, t = row / a.group, h = row - t * a.group;
                Load<TQ, D>::run(qp + (long long)(it.token + t) * a.q_stride + (it.head * a.group + h) * hd, q[r]);
#pragma unroll
                for (int e = 0; e < D; ++e) q[r][e] *= a.scale_log2;
            }
        }
        // the keys this lane's row sees: [see_lo, see_hi]
        const int pos = my_row < it.n_rows ? it.pos0 + (it.row0 + my_row) / a.group : -1;
        const int k0 = max(it.lo, it.t0 * kPaKeys), k1 = min(it.hi, it.t1 * kPaKeys);
        const int see_lo = max(max(pos, -1) - win + 1, k0), see_hi = min(pos, k1 - 1);
        // element offset of key j in its page, or -1: outside the CTA's keys or no page
        auto place = [&](int j) -> long long {
            if (j < k0 || j >= k1) return -1;
            const int pi = j / ps, page = table[pi];
            if (page < 0 || page >= a.kv.n_pages) return -1;
            return page * a.kv.page_stride + (j - pi * ps) * a.kv.slot_stride + it.head * a.kv.head_stride;
        };
        auto places = [&](int j0, long long (&at)[KB]) {
            if (one_page) {
                const int jv = min(max(j0, k0), k1 - 1);   // a key of the batch that is the CTA's, if one is
                const long long p = j0 < k1 ? place(jv) : -1;
#pragma unroll
                for (int u = 0; u < KB; ++u) {
                    const int j = j0 + u;
                    at[u] = p < 0 || j < k0 || j >= k1 ? -1 : p + (j - jv) * a.kv.slot_stride;
                }
            } else {
#pragma unroll
                for (int u = 0; u < KB; ++u) at[u] = place(j0 + u);
            }
        };
        long long at[KB];
        int j0 = k0 / KB * KB + stream * KB;
        if (j0 < k1) places(j0, at);
#pragma unroll 1
        for (; j0 < k1; j0 += S * KB) {
            float k[KB][D], v[KB][D];
            bool there = false;   // of this lane's key
#pragma unroll
            for (int u = 0; u < KB; ++u) {
#pragma unroll
                for (int e = 0; e < D; ++e) k[u][e] = v[u][e] = 0.f;
                if (at[u] >= 0 && own) Load<TKV, D>::run(kc + at[u], k[u]);
                if (u == my_key) there = at[u] >= 0;
            }
#pragma unroll
            for (int u = 0; u < KB; ++u)
                if (at[u] >= 0 && own) Load<TKV, D>::run(vc + at[u], v[u]);
            places(j0 + S * KB, at);   // the next batch's pages, while these keys are on their way
            float s[NV];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < KB; ++u) {
                    float x = 0.f;
#pragma unroll
                    for (int e = 0; e < D; ++e) x = fmaf(q[r][e], k[u][e], x);
                    s[r * KB + u] = x;
                }
            // sums over the lanes: at each step a lane keeps half of its values
#pragma unroll
            for (int n = NV / 2, x = LPK / 2; n >= 1; n /= 2, x /= 2) {
                const bool up = sub & x;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const float send = up ? s[i] : s[i + n], keep = up ? s[i + n] : s[i];
                    s[i] = keep + __shfl_xor_sync(lanes, send, x);
                }
            }
#pragma unroll
            for (int x = REP / 2; x > 0; x >>= 1) s[0] += __shfl_xor_sync(lanes, s[0], x);
            const int j = j0 + my_key;
            const bool see = there && j >= see_lo && j <= see_hi;
            float top = see ? s[0] : -INFINITY;
#pragma unroll
            for (int x = REP; x < REP * KB; x *= 2) top = fmaxf(top, __shfl_xor_sync(lanes, top, x));
            // the reference moves only when it is exceeded by 2^8 (or was no key's)
            if (__any_sync(lanes, top > m + 8.f)) {
                const bool move = top > m + 8.f;
                const float f = move ? pa_ex2(m - top) : 1.f;   // m = -inf: 0
                if (move) m = top;
                l *= f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float fr = __shfl_sync(lanes, f, r * KB * REP, LPK);
#pragma unroll
                    for (int e = 0; e < D; ++e) o[r][e] *= fr;
                }
            }
            // (-1: masked.  A weight of 0 counts: it may meet an infinity or a NaN)
            const float p = see ? pa_ex2(s[0] - finite_max(m)) : -1.f;
            l += see ? p : 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < KB; ++u) {
                    const float pr = __shfl_sync(lanes, p, (r * KB + u) * REP, LPK);
                    if (!(pr < 0.f)) {   // (NaN: yes) a masked key adds nothing, whatever its V holds
#pragma unroll
                        for (int e = 0; e < D; ++e) o[r][e] = fmaf(pr, v[u][e], o[r][e]);
                    }
                }
        }
        // ---- merge the streams of the warp, then the warps, in order
        __syncwarp();
#pragma unroll
        for (int x = REP; x < REP * KB; x *= 2) l += __shfl_xor_sync(0xffffffffu, l, x);
#pragma unroll
        for (int x = LPK; x < 32; x *= 2) {
            const float mo = __shfl_xor_sync(0xffffffffu, m, x), lo = __shfl_xor_sync(0xffffffffu, l, x);
            const float mn = fmaxf(m, mo), ref = finite_max(mn);
            const float f = pa_ex2(m - ref), fo = pa_ex2(mo - ref);
            l = l * f + lo * fo;
            m = mn;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float fr = __shfl_sync(0xffffffffu, f, r * KB * REP, LPK);
                const float fro = __shfl_sync(0xffffffffu, fo, r * KB * REP, LPK);
#pragma unroll
                for (int e = 0; e < D; ++e)
                    o[r][e] = o[r][e] * fr + __shfl_xor_sync(0xffffffffu, o[r][e], x) * fro;
            }
        }
        if (lane < LPK) {
            if (sub % (REP * KB) == 0) {
                s_m[warp * R + my_row] = m;
                s_l[warp * R + my_row] = l;
            }
            if (own) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < D; ++e) s_o[(warp * R + r) * hd + d0 + e] = o[r][e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < it.n_rows * hd; i += kPaThreads) {
            const int r = i / hd, d = i - r * hd;
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < kPaWarps; ++w) mx = fmaxf(mx, s_m[w * R + r]);
            const float ref = finite_max(mx);
            float acc = 0.f, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kPaWarps; ++w) {
                const float f = pa_ex2(s_m[w * R + r] - ref);
                sum = fmaf(f, s_l[w * R + r], sum);
                acc = fmaf(f, s_o[(w * R + r) * hd + d], acc);
            }
            if (it.part < 0) {
                const int row = it.row0 + r, t = row / a.group, h = row - t * a.group;
                store_out<TQ>(out + (long long)(it.token + t) * a.out_stride + (it.head * a.group + h) * hd + d,
                              sum == 0.f ? 0.f : acc / sum);
            } else {
                const size_t part = (size_t)it.part * kAttnRowsSimt + r;
                float *ml = reinterpret_cast<float *>(a.ws + lay.ml) + part * 2;
                if (d == 0) {
                    ml[0] = mx;
                    ml[1] = sum;
                }
                reinterpret_cast<float *>(a.ws + lay.o)[part * hd + d] = acc;
            }
        }
        __syncthreads();   // s_item and the merge buffers are rewritten
    }
}

// ------------------------------------------------------------------ join

// Rows of split items: out = sum_i f_i o_i / sum_i f_i l_i over the row's parts i, f_i = 2^(m_i -
// max m).  Every warp reads how many rows each CTA's split item has and finds its rows itself.
// Where items are many, a row has few parts and is one warp's; where they are few (a long
// sequence alone), a row is a CTA's, warp w adding the parts w, w + 8, .. and the eight partial
// sums then added in order.  Bound: latency (KBs to a few MB of parts from L2): three
// loads that wait for one another, the rows' counts, the item's record, its parts.
static constexpr int kJoinThreads = 256;
static constexpr int kJoinWarps = kJoinThreads / 32;

// V consecutive floats, 4 V bytes aligned (V 2, 4 or 8).
template <int V> __device__ __forceinline__ void ld_part(const float *p, float (&x)[V])
{
    if constexpr (V == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x; x[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    }
}
template <typename T, int V> __device__ __forceinline__ void st_row(T *p, const float (&x)[V])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 2) *reinterpret_cast<float2 *>(p + i) = make_float2(x[i], x[i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            *reinterpret_cast<uint32_t *>(p + i) =
                pack_bf16x2(__float2bfloat16_rn(x[i]), __float2bfloat16_rn(x[i + 1]));
    }
}

template <typename T, int ROWS, int CTAS, int V>   // V: adjacent dims per lane
__global__ void __launch_bounds__(kJoinThreads) k_paged_join(const __grid_constant__ AttnArgs a, int wide)
{
    __shared__ float s_o[kJoinWarps][32 * V], s_l[kJoinWarps];
    const int hd = a.kv.head_dim;
    const int stride = ROWS > 0 ? ROWS : a.rows;
    const PartLayout lay(CTAS, stride, hd);
    const int *n_rows = reinterpret_cast<const int *>(a.ws + lay.n_rows);
    const PagedSplit *split = reinterpret_cast<const PagedSplit *>(a.ws + lay.split);
    const float2 *ml = reinterpret_cast<const float2 *>(a.ws + lay.ml);
    const float *po = reinterpret_cast<const float *>(a.ws + lay.o);
    T *out = static_cast<T *>(a.out);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d = lane * V;
    pdl_wait();
    pdl_trigger();
    // lane i: rows of the split items of CTAs K i .. K i + K - 1, and the rows before them
    constexpr int K = CTAS / 32;
    static_assert(CTAS % 32 == 0 && CTAS <= kAttnMaxCtas, "a lane looks at whole groups");
    int nr[K], mine = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        nr[k] = n_rows[K * lane + k];
        mine += nr[k];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    const int rows = __shfl_sync(0xffffffffu, incl, 31);
    const int first = wide ? blockIdx.x : blockIdx.x * kJoinWarps + warp, step = wide ? gridDim.x : gridDim.x * kJoinWarps;
    for (int job = first; job < rows; job += step) {
        // the CTA whose item has row `job`, and the row in the item
        const int src = __ffs(__ballot_sync(0xffffffffu, job < incl)) - 1;
        int c = 0, r = job - (incl - mine);
        if (lane == src) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (c == k && r >= nr[k]) {
                    r -= nr[k];
                    c = k + 1;
                }
            c += K * lane;
        }
        c = __shfl_sync(0xffffffffu, c, src);
        r = __shfl_sync(0xffffffffu, r, src);
        const PagedSplit sp = split[c];
        const int parts = sp.last_cta - c + 1;
        // part i: the CTA's own tail, then the head parts of the CTAs after it
        auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * stride + r; };
        float mx = -INFINITY, acc[V], sum;
        const float2 m0 = lane < parts ? ml[slot(lane)] : make_float2(-INFINITY, 0.f);
        mx = m0.x;
        for (int i = lane + 32; i < parts; i += 32) mx = fmaxf(mx, ml[slot(i)].x);
        mx = warp_max(mx);
        const float ref = finite_max(mx);
        const int w0 = wide ? warp : 0, ws = wide ? kJoinWarps : 1;
        auto add_parts = [&](auto weigh) {
            sum = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 4
            for (int i = w0; i < parts; i += ws) {
                float2 m2 = make_float2(__shfl_sync(0xffffffffu, m0.x, i & 31), __shfl_sync(0xffffffffu, m0.y, i & 31));
                if (i >= 32) m2 = ml[slot(i)];
                const float f = pa_ex2(m2.x - ref);
                sum = fmaf(f, m2.y, sum);
                if (d < hd) {
                    float x[V];
                    ld_part<V>(po + slot(i) * hd + d, x);
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] = weigh(f, x[e], acc[e]);
                }
            }
        };
        add_parts([](float f, float x, float s) { return fmaf(f, x, s); });
        bool odd = false;
#pragma unroll
        for (int e = 0; e < V; ++e) odd |= isnan(acc[e]);
        // An infinity stays one where the factor of its part underflows.  (In a pass of its own: in the
        // first one it cost 0.9 us of 24.2 at one sequence of 54310.)
        if (__any_sync(0xffffffffu, odd))
            add_parts([](float f, float x, float s) { return f == 0.f && isinf(x) ? s + x : fmaf(f, x, s); });
        if (wide) {
#pragma unroll
            for (int e = 0; e < V; ++e) s_o[warp][d + e] = acc[e];
            if (lane == 0) s_l[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
                for (int w = 0; w < kJoinWarps; ++w) {
                    sum += s_l[w];
#pragma unroll
                    for (int e = 0; e < V; ++e) acc[e] += s_o[w][d + e];
                }
            }
            __syncthreads();
        }
        if (d < hd && (!wide || warp == 0)) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const int row = sp.row0 + r, tk = row / a.group, h = row - tk * a.group;
#pragma unroll
            for (int e = 0; e < V; ++e) acc[e] *= inv;
            st_row<T, V>(out + (long long)(sp.token + tk) * a.out_stride + (sp.head * a.group + h) * hd + d, acc);
        }
    }
}

// ------------------------------------------------------------------ host side

size_t paged_attn_ws_bytes(const PagedKV &kv, int group, int max_new, int kv_dtype)
{
    size_t n = PartLayout(kAttnMaxCtas, kAttnRowsSimt, kv.head_dim).total;
    if (paged_attn_tc_ok(kv, group, DS4G_BF16, kv_dtype)) {
        const size_t t = PartLayout(kAttnMaxCtasTc, paged_attn_tc_rows(group, max_new), kv.head_dim).total;
        n = t > n ? t : n;
    }
    return n;
}

cudaError_t paged_attn_status(void *ws, cudaStream_t st, int *status)
{
    int word[kAttnMaxCtas];
    cudaError_t e = cudaMemcpyAsync(word, ws, sizeof(word), cudaMemcpyDeviceToHost, st);   // PartLayout::status
    if (!e) e = cudaStreamSynchronize(st);
    *status = DS4G_OK;
    for (int c = 0; !e && c < kAttnMaxCtas; ++c)
        if (word[c] == kAttnTimedOut) *status = DS4G_ETIMEOUT;
    if (!e && *status != DS4G_OK) {   // read: the words are cleared
        e = cudaMemsetAsync(ws, 0, sizeof(word), st);
        if (!e) e = cudaStreamSynchronize(st);
    }
    return e;
}

static long long most_items(const AttnArgs &a);

// Launches the join behind a grid of `ctas`: one row a CTA where the items are so few that a
// row has eight parts or more on average.
template <typename T, int ROWS, int CTAS>
static cudaError_t join(const AttnArgs &a, int ctas, int nsm, cudaStream_t st)
{
    const long long items = most_items(a), rows = (items < ctas ? items : ctas) * a.rows;   // a cut item begins in a CTA of its own
    const int wide = items * 8 <= ctas, most = 8 * nsm;
    const long long jobs = wide ? rows : (rows + kJoinWarps - 1) / kJoinWarps;
    const int grid = (int)(jobs < most ? jobs : most);
    const dim3 block(kJoinThreads);
    if (a.kv.head_dim <= 64) return launch_pdl(k_paged_join<T, ROWS, CTAS, 2>, dim3(grid), block, 0, st, a, wide);
    if (a.kv.head_dim <= 128) return launch_pdl(k_paged_join<T, ROWS, CTAS, 4>, dim3(grid), block, 0, st, a, wide);
    return launch_pdl(k_paged_join<T, ROWS, CTAS, 8>, dim3(grid), block, 0, st, a, wide);
}
cudaError_t paged_join_tc(const AttnArgs &a, int ctas, int nsm, cudaStream_t st)
{
    return join<bf16, 0, kAttnMaxCtasTc>(a, ctas, nsm, st);
}

// Most items of a call and most units of an item, by the sizes the host knows.
static long long most_items(const AttnArgs &a)
{
    return (long long)a.s.n_seqs * a.kv.n_kv_heads * (((long long)a.s.max_new * a.group + a.rows - 1) / a.rows);
}
static long long most_tiles(const AttnArgs &a, int kt)
{
    long long keys = (long long)a.s.width * a.kv.page_size;
    if (a.window > 0) {
        const long long seen = (long long)a.window + a.s.max_new - 1;   // may begin inside a unit
        keys = seen + kt - 1 < keys ? seen + kt - 1 : keys;
    }
    return keys > 0 ? (keys + kt - 1) / kt : 1;
}
// Items stay whole where cutting them gains less than the join costs (about 3 us, two or three
// units): up to four units (one sequence of 384 positions: 9.0 us whole, 10.8 cut; 64 with 8 K/V
// heads 28.8 and 37.2), and up to eight where the items alone occupy a quarter of the CTAs or
// more, but no CTA has two (768 positions: 8 x 8 heads 11.5 us whole, 13.8 cut; one sequence 12.8 and
// 11.1; 24 x 8 heads, in two turns, 21.6 and 20.5).  The last condition gains where the items are
// little more than one turn (8 K/V heads, 40 of 1024 39.8 -> 33.3 us, 24 of 640 20.7 -> 18.5) and loses
// where they fill two (32 of 640 21.8 -> 23.3, of 768 23.6 -> 26.4, of 1024 28.1 -> 29.5).
// The host knows the table's width and the window, not the lengths: under a table four times as
// wide as the longest sequence items of three units are cut (384 positions: one sequence 8.9 -> 10.1
// us, 64 with 8 K/V heads 27.7 -> 35.6; 100 positions, whole at four times the width, 7.6 -> 8.7 at 16).
int paged_attn_grid(AttnArgs &a, int kt, int most)
{
    const long long tiles = most_tiles(a, kt), items = most_items(a);
    a.whole = tiles <= 4 || (tiles <= 8 && items * 4 >= most && items <= most);
    const long long u = items * (a.whole ? 1 : tiles);
    return (int)(u < most ? u : most);
}

template <typename TQ, typename TKV, int LPK, int D, int R, int KB>
static cudaError_t simt(AttnArgs &a, int nsm, cudaStream_t st)
{
    auto kernel = k_paged_attn<TQ, TKV, LPK, D, R, KB>;
    const size_t smem = pa_smem(R, a.kv.head_dim);
    static PerDevice once;
    cudaError_t e = allow_once(once, kernel, pa_smem(R, 256));
    if (e) return e;
    a.rows = R;
    const int resident = (R * D <= 16 ? 2 : 1) * nsm;
    const int grid = paged_attn_grid(a, kPaKeys, resident < kAttnMaxCtas ? resident : kAttnMaxCtas);
    e = launch_pdl(kernel, dim3(grid), dim3(kPaThreads), smem, st, a);
    if (!e && !a.whole) e = join<TQ, kAttnRowsSimt, kAttnMaxCtas>(a, grid, nsm, st);
    return e;
}
// Four query rows a tile.  (Eight, with half as many warps an SM: 186 us against 138 for 32
// sequences of 4000 positions with eight rows a K/V head of 64; at 128 dims the two are even.)
template <typename TQ, typename TKV> static cudaError_t simt_dim(AttnArgs &a, int nsm, cudaStream_t st)
{
    if (a.kv.head_dim <= 32) return simt<TQ, TKV, 8, 4, 4, 2>(a, nsm, st);
    if (a.kv.head_dim <= 64) return simt<TQ, TKV, 16, 4, 4, 4>(a, nsm, st);
    if (a.kv.head_dim <= 128) return simt<TQ, TKV, 32, 4, 4, 4>(a, nsm, st);
    return simt<TQ, TKV, 32, 8, 4, 4>(a, nsm, st);
}

cudaError_t paged_attention(const AttnArgs &in, int q_dtype, int kv_dtype, cudaStream_t st, int nsm)
{
    if (in.s.n_seqs == 0 || in.s.n_tokens == 0) return cudaSuccess;
    AttnArgs a = in;
    if (paged_attn_tc_ok(a.kv, a.group, q_dtype, kv_dtype)) {
        a.rows = paged_attn_tc_rows(a.group, a.s.max_new);
        return paged_attn_tc(a, st, nsm);
    }
    if (q_dtype == DS4G_F32)
        return kv_dtype == DS4G_F32 ? simt_dim<float, float>(a, nsm, st) : simt_dim<float, bf16>(a, nsm, st);
    return kv_dtype == DS4G_F32 ? simt_dim<bf16, float>(a, nsm, st) : simt_dim<bf16, bf16>(a, nsm, st);
}

}  // namespace ds4g
