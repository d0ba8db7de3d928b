// The pages worth reading of the paged cache: per (row, KV head) a score per page from its mean key,
// the top_k best by it, written ascending between the pages that are always read.
//
// A score is sum_d s_d mean_d, s_d the sum of the group's queries: s is held as an f32 pair (hi + lo,
// its sum taken in 64 bits), the products' and sums' rounding errors are carried along (Ogita, Rump
// and Oishi, "Accurate sum and dot product", 2005: Dot2), and the result is rounded to f32 once.
// Pages whose exact scores differ by less than an f32 step then compare as any evaluation in 64 bits
// rounded to f32 would have them, whatever the summation order.
//
// A cluster of CTAs shares the pages of a (row, KV head) where there are few of these; each score goes
// to the first CTA's shared memory, which selects: the take-th largest by three histograms of 11, 11
// and 10 bits, then one scan.
//
// One long sequence is bound by latencies (131072 keys, 2048 pages: 9.2 us; the scores 3, the threshold 2,
// the list 1.3, the rest start and end); many by the scores' instructions, 11 packed ones to two channels
// besides the conversion: 32 sequences of up to 512 pages 16.8 us, the longest's CTA last.  Eight lanes a
// page: sixteen (fewer registers, more warps) spend more on the sums over lanes (4 us more).
#include <cmath>

#include "dl_async.cuh"
#include "paged_kv.cuh"

namespace {

struct SelectArgs {
    const float *q;
    int64_t q_stride;
    const __half *mean;
    const int32_t *tables;
    int64_t table_stride;
    int width;
    const int32_t *seqlen;
    int32_t *pages, *status;
    int n_q, n_kv, page, n_pages, top_k, sink, local;
};

constexpr int kGroup = 8;                    // lanes that share a page
constexpr int kFlight = 4;                   // pages a group has in flight (two lanes a page in the end)
constexpr int kBins = 2048;

// f32 scores as unsigned keys of the same order; NaN below every number.
__device__ __forceinline__ uint32_t order_key(float x)
{
    if (x != x) return 0u;
    if (x == 0.f) x = 0.f;                   // -0 ties with +0
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// a + b = s + e exactly, for both halves of a pair.
__device__ __forceinline__ void two_sum(float2 a, float2 b, float2 &s, float2 &e)
{
    const float2 minus = make_float2(-1.f, -1.f);
    s = __fadd2_rn(a, b);
    const float2 z = __ffma2_rn(a, minus, s);                        // s - a
    const float2 y = __ffma2_rn(z, minus, s);                        // s - z
    e = __fadd2_rn(__ffma2_rn(y, minus, a), __ffma2_rn(z, minus, b));
}

// a + b, its error and those of a and b in `e`.
__device__ __forceinline__ float sum_carried(float a, float b, float ea, float eb, float &e)
{
    const float s = a + b, z = s - a, y = s - z;
    e = ea + eb + ((a - y) + (b - z));
    return s;
}

__device__ __forceinline__ float2 shfl_xor(float2 x, int o)
{
    return make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o));
}

// Inclusive sum over the CTA's threads (every thread calls it; s_warp is the call's own).
template <int kWarps>
__device__ __forceinline__ int cta_scan(int v, int *s_warp)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        if (w < warp) x += s_warp[w];
    return x;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads, 512 / kThreads) paged_select_kernel(const __grid_constant__ SelectArgs a)
{
    constexpr int kWarps = kThreads / 32;
    extern __shared__ __align__(16) uint32_t hist_keys[];    // [3][kBins] of the histograms, then the candidates' keys
    int *hist = reinterpret_cast<int *>(hist_keys);
    uint32_t *keys = hist_keys + 3 * kBins;
    __shared__ float s_hi[D], s_lo[D];
    __shared__ int s_warp[3][kWarps], s_pick[3][2];
    __shared__ int2 s_count[kWarps];
    const int r = blockIdx.y, h = blockIdx.z, G = a.n_q / a.n_kv, C = gridDim.x;
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t rank = C > 1 ? cluster_rank() : 0;
    const int cap = a.sink + a.top_k + a.local;
    int32_t *dst = a.pages + ((int64_t)r * a.n_kv + h) * cap;
    // The sequence's pages np and its candidates [lo, lo + nc), from its length.
    auto pages_of = [&](int len, int &np, int &lo) {
        const int64_t most = (int64_t)a.width * a.page;
        len = (int)min((int64_t)max(len, 0), most);
        np = (len + a.page - 1) / a.page;
        lo = min(a.sink, np);
        return max(lo, np - a.local) - lo;
    };
    int np, lo, nc = pages_of(__ldcg(a.seqlen + r), np, lo);

    // ---- scores: eight lanes a page, D/8 channels a lane.  The first pages' table entries are read
    // before the wait on the previous kernel, which may still write lengths and tables: their means are
    // asked for, and if the entries or the length read after the wait differ, asked for anew.  All that
    // threads have to agree on comes from the length read after the wait.
    constexpr int E = D / kGroup;
    const int gl = lane % kGroup, groups = kThreads / kGroup, step = groups * C;
    uint4 m[kFlight][E / 8];
    int phys[kFlight];
    auto entries = [&](int c0) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int c = c0 + f * step;
            phys[f] = c < nc ? __ldcg(a.tables + r * a.table_stride + lo + c) : 0;
        }
    };
    auto means = [&](int c0) {
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const bool ok = phys[f] >= 0 && phys[f] < a.n_pages;
            const uint4 *p = reinterpret_cast<const uint4 *>(a.mean + ((int64_t)(ok ? phys[f] : 0) * a.n_kv + h) * D + gl * E);
#pragma unroll
            for (int i = 0; i < E / 8; ++i)
                if (c0 + f * step < nc) m[f][i] = p[i];
        }
    };
    int c0 = (int)rank * groups + tid / kGroup;
    entries(c0);
    dl_pdl_wait();
    dl_pdl_launch_dependents();
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    means(c0);
    {
        const int seen = nc, from = lo, len = __ldcg(a.seqlen + r);
        int was[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) was[f] = phys[f];
        entries(c0);
        nc = pages_of(len, np, lo);
        bool changed = seen != nc || from != lo;
#pragma unroll
        for (int f = 0; f < kFlight; ++f) changed |= was[f] != phys[f];
        if (changed) {
            entries(c0);
            means(c0);
        }
        if ((len < 0 || len > (int64_t)a.width * a.page) && tid == 0 && h == 0 && rank == 0)
            dl_status_or(a.status, DL_STATUS_SEQLEN_RANGE);
    }
    const int take = min(a.top_k, nc), hi = lo + nc;
    if (take == nc || take == 0) {           // all of them or none: no scores (the same for the whole cluster)
        if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        const int skip = nc - take;
        if (rank == 0)
            for (int i = tid; i < cap; i += kThreads) dst[i] = i < lo ? i : i < np - skip ? i + skip : -1;
        return;
    }
    if (rank == 0)
        for (int i = tid; i < 3 * kBins / 4; i += kThreads) reinterpret_cast<int4 *>(hist)[i] = make_int4(0, 0, 0, 0);
    static_assert(D <= kThreads, "a channel a thread");
    bool mine = false;                       // the thread's channel passes 2^100
    if (tid < D) {
        const float *src = a.q + r * a.q_stride + (int64_t)h * G * D + tid;
        double s = 0.0;
        for (int g0 = 0; g0 < G; g0 += 8) {          // (eight loads in flight)
            float v[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) v[g] = g0 + g < G ? src[(g0 + g) * D] : 0.f;
#pragma unroll
            for (int g = 0; g < 8; ++g)
                if (g0 + g < G) s += (double)v[g];
        }
        float hi = (float)s;
        mine = fabsf(hi) >= 0x1p100f;
        if (mine) {
            s *= 0x1p-64;
            hi = (float)s;
        }
        s_hi[tid] = hi;
        s_lo[tid] = isfinite(hi) ? (float)(s - (double)hi) : 0.f;
    }
    // from 2^100 on sums, products or their sums might pass f32 where the score does not: they are taken 2^-64
    // as large, and the scores, rounded, brought back (1 x 131072 keys 0.3 us more)
    const bool large = __syncthreads_or(mine);
    if (large) {
        if (tid < D && !mine) {
            s_hi[tid] *= 0x1p-64f;
            s_lo[tid] *= 0x1p-64f;
        }
        __syncthreads();
    }
    // (the first CTA of the cluster runs: its shared memory may be written)
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    float2 qh[E / 2], ql[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
        qh[i] = make_float2(s_hi[gl * E + 2 * i], s_hi[gl * E + 2 * i + 1]);
        ql[i] = make_float2(s_lo[gl * E + 2 * i], s_lo[gl * E + 2 * i + 1]);
    }
    uint32_t keys0 = dla::smem_u32(keys);
    if (C > 1) asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(keys0) : "r"(dla::smem_u32(keys)), "r"(0));
    // (whole warps run the loops together: their bounds are the warp's first group's)
    for (int w0 = c0 - lane / kGroup; w0 < nc; w0 += step * kFlight, c0 += step * kFlight) {
        float2 sum[kFlight], err[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            float2 s = make_float2(0.f, 0.f), e = s;
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                const uint32_t w[4] = {m[f][i].x, m[f][i].y, m[f][i].z, m[f][i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                    const float2 p = __fmul2_rn(qh[4 * i + k], x);
                    const float2 pe = __ffma2_rn(qh[4 * i + k], x, make_float2(-p.x, -p.y));
                    float2 te;
                    two_sum(s, p, s, te);
                    e = __fadd2_rn(e, __fadd2_rn(te, __ffma2_rn(ql[4 * i + k], x, pe)));
                }
            }
            sum[f] = s;
            err[f] = e;
        }
        // even and odd channels of pages 0, 1 and 2, 3; then the lanes, which halve their pages on the way:
        // a pair of lanes ends with one page's score
        float2 te, s[2], e[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 u = sum[2 * i], v = sum[2 * i + 1], x = err[2 * i], y = err[2 * i + 1];
            two_sum(make_float2(u.x, v.x), make_float2(u.y, v.y), s[i], te);
            e[i] = __fadd2_rn(__fadd2_rn(make_float2(x.x, y.x), make_float2(x.y, y.y)), te);
        }
        const bool b4 = gl & 4, b2 = gl & 2;
        const float2 s4 = b4 ? s[1] : s[0], t4 = b4 ? s[0] : s[1], e4 = b4 ? e[1] : e[0], f4 = b4 ? e[0] : e[1];
        two_sum(s4, shfl_xor(t4, 4), s[0], te);
        e[0] = __fadd2_rn(__fadd2_rn(e4, shfl_xor(f4, 4)), te);
        float s1 = b2 ? s[0].y : s[0].x, e1 = b2 ? e[0].y : e[0].x;
        s1 = sum_carried(s1, __shfl_xor_sync(0xffffffffu, b2 ? s[0].x : s[0].y, 2),
                         e1, __shfl_xor_sync(0xffffffffu, b2 ? e[0].x : e[0].y, 2), e1);
        s1 = sum_carried(s1, __shfl_xor_sync(0xffffffffu, s1, 1), e1, __shfl_xor_sync(0xffffffffu, e1, 1), e1);
        const int c = c0 + (gl >> 1) * step;
        if ((gl & 1) == 0 && c < nc) {
            float score = isfinite(s1) ? s1 + e1 : s1;       // (an infinite term leaves NaN in e1)
            if (large) score *= 0x1p64f;
            const int page = b4 ? b2 ? phys[3] : phys[2] : b2 ? phys[1] : phys[0];
            if (page < 0 || page >= a.n_pages) {
                score = NAN;
                dl_status_or(a.status, DL_STATUS_PAGE_RANGE);
            }
            const uint32_t key = order_key(score);
            if (C > 1)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(keys0 + 4u * c), "r"(key) : "memory");
            else
                keys[c] = key;
        }
        if (w0 + step * kFlight < nc) {
            entries(c0 + step * kFlight);
            means(c0 + step * kFlight);
        }
    }
    if (C > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank != 0) return;
    }
    __syncthreads();

    // ---- the take-th largest key: `prefix` under `mask`, `need` of the keys that match it
    uint32_t prefix = 0, mask = 0;
    int need = take;
    bool cut = true;                         // some of the matching keys stay out
#pragma unroll
    for (int pass = 0; pass < 3; ++pass, hist += kBins) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1023u : 2047u;
        for (int c = tid; c < nc; c += kThreads)
            if ((keys[c] & mask) == prefix) atomicAdd(&hist[(keys[c] >> shift) & digits], 1);
        __syncthreads();
        // bins from the top, `per` a thread: the one the need-th key falls in
        constexpr int per = kBins / kThreads;
        int n[per], mine = 0;
#pragma unroll
        for (int i = 0; i < per / 4; ++i) {
            const int4 b = reinterpret_cast<const int4 *>(hist)[kBins / 4 - 1 - i - per / 4 * tid];
            n[4 * i] = b.w; n[4 * i + 1] = b.z; n[4 * i + 2] = b.y; n[4 * i + 3] = b.x;
        }
#pragma unroll
        for (int i = 0; i < per; ++i) mine += n[i];
        int before = cta_scan<kWarps>(mine, s_warp[pass]) - mine;
        if (before < need && need <= before + mine) {
#pragma unroll
            for (int i = 0; i < per; ++i) {
                if (before < need && need <= before + n[i]) {
                    s_pick[pass][0] = kBins - 1 - (tid * per + i);
                    s_pick[pass][1] = need - before - (need - before == n[i] ? 1 << 30 : 0);
                }
                before += n[i];
            }
        }
        __syncthreads();
        prefix |= (uint32_t)s_pick[pass][0] << shift;
        mask |= digits << shift;
        need = s_pick[pass][1];
        if (need < 0) {                      // every key that matches is in
            cut = false;
            break;
        }
    }
    // ---- the chosen, in index order: a run of candidates a warp, 32 at a time
    const int warp = tid >> 5, run = ((nc + kThreads - 1) / kThreads) * 32, k0 = min(warp * run, nc), k1 = min(k0 + run, nc);
    const unsigned below = (1u << lane) - 1u;
    int above = 0, equal = 0;
    for (int c = k0 + lane; c - lane < k1; c += 32) {
        const uint32_t k = c < k1 ? keys[c] & mask : 0u;
        above += __popc(__ballot_sync(0xffffffffu, c < k1 && k > prefix));
        equal += __popc(__ballot_sync(0xffffffffu, c < k1 && k == prefix));
    }
    if (lane == 0) s_count[warp] = make_int2(above, equal);
    __syncthreads();
    int at = lo, eq = 0;                     // of the warps before: chosen, and equal keys seen
    const int most_eq = cut ? need : nc;
    for (int w = 0; w < warp; ++w) {
        at += s_count[w].x + min(s_count[w].y, max(0, most_eq - eq));
        eq += s_count[w].y;
    }
    for (int c = k0 + lane; c - lane < k1; c += 32) {
        const uint32_t k = c < k1 ? keys[c] & mask : 0u;
        const unsigned eqs = __ballot_sync(0xffffffffu, c < k1 && k == prefix);
        const bool in = c < k1 && (k > prefix || (k == prefix && eq + __popc(eqs & below) < most_eq));
        const unsigned ins = __ballot_sync(0xffffffffu, in);
        if (in) dst[at + __popc(ins & below)] = lo + c;
        at += __popc(ins);
        eq += __popc(eqs);
    }
    for (int i = tid; i < lo; i += kThreads) dst[i] = i;
    for (int i = tid; i < np - hi; i += kThreads) dst[lo + take + i] = hi + i;
    for (int i = lo + take + np - hi + tid; i < cap; i += kThreads) dst[i] = -1;
}

constexpr int smem_bytes(int width) { return width * 4 + 3 * kBins * 4; }

template <int D, int kThreads>
int launch(const SelectArgs &a, int rows, int C, cudaStream_t st)
{
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)C, (unsigned)rows, (unsigned)a.n_kv);
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = (size_t)smem_bytes(a.width);
    lc.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    lc.attrs = attr;
    lc.numAttrs = C > 1 ? 2 : 1;
    auto go = [&]() {
        cudaError_t e = cudaLaunchKernelEx(&lc, paged_select_kernel<D, kThreads>, a);
        return e == cudaSuccess ? DL_OK : dl::cuda_fail(e, "dl_paged_select: launch");
    };
    if (smem_bytes(a.width) <= 40 * 1024) return go();   // (the default limit is 48 KB with the static part)
    static std::atomic<uint64_t> asked{0};
    return dlp::launch_wide(reinterpret_cast<const void *>(paged_select_kernel<D, kThreads>),
                            smem_bytes(DL_PAGED_MAX_WIDTH), asked, "dl_paged_select: shared memory", go);
}

}  // namespace

extern "C" {

int dl_paged_select(const float *q, int64_t q_stride, const dl_paged_kv *kv, const dl_block_tables *tables,
                    const int32_t *seqlen, int rows, int n_q, int top_k, int n_sink, int n_local,
                    int32_t *pages, int32_t *status, dl_stream_t stream)
{
    dl::clear_error();
    if (rows != 0 && (!q || !seqlen || !pages)) return dl::fail(DL_E_ARG, "dl_paged_select: null pointer");
    int rc = dlp::check_cache("dl_paged_select", kv, tables, n_q, true);
    if (rc != DL_OK) return rc;
    if (rows != tables->n_seqs)
        return dl::fail(DL_E_ARG, "dl_paged_select: %d rows of %d sequences (one row each)", rows, tables->n_seqs);
    if (top_k < 0 || n_sink < 0 || n_local < 1 || (int64_t)top_k + n_sink + n_local > 0x7fffffff)
        return dl::fail(DL_E_ARG, "dl_paged_select: top_k=%d n_sink=%d n_local=%d", top_k, n_sink, n_local);
    if (tables->width > DL_PAGED_MAX_WIDTH)
        return dl::fail(DL_E_SHAPE, "dl_paged_select: tables of %d entries (at most %d)", tables->width, DL_PAGED_MAX_WIDTH);
    if (q_stride < (int64_t)n_q * kv->head_dim) return dl::fail(DL_E_ARG, "dl_paged_select: stride below the row width");
    if (kv->n_kv > 65535 || rows > 65535)
        return dl::fail(DL_E_SHAPE, "dl_paged_select: rows=%d n_kv=%d (at most 65535)", rows, kv->n_kv);
    if (rows == 0) return DL_OK;
    SelectArgs a{};
    a.q = q; a.q_stride = q_stride; a.mean = static_cast<const __half *>(kv->k_mean);
    a.tables = tables->pages; a.table_stride = tables->stride; a.width = tables->width; a.seqlen = seqlen;
    a.pages = pages; a.status = status;
    a.n_q = n_q; a.n_kv = kv->n_kv; a.page = kv->page; a.n_pages = kv->n_pages;
    a.top_k = top_k; a.sink = n_sink; a.local = n_local;
    int sms = 0;
    rc = dl::device_sm_count(&sms);
    if (rc != DL_OK) return rc;
    // CTAs of a (row, KV head): up to three an SM in all, each at least 64 pages (48 sequences of 4 KV heads:
    // two CTAs 9.1 us, four 11.3; 32 of 8: one 16.0 us, two 18.5); of 512 threads where that leaves SMs idle
    // (1 x 131072 keys: 256 threads took 1.1 us more)
    int C = 1;
    while (C < 8 && (int64_t)rows * kv->n_kv * C * 2 <= 3 * (int64_t)sms && tables->width >= C * 2 * 64) C *= 2;
    const int threads = (int64_t)rows * kv->n_kv * C <= sms ? 512 : 256;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (kv->head_dim == 128) return threads == 512 ? launch<128, 512>(a, rows, C, st) : launch<128, 256>(a, rows, C, st);
    return threads == 512 ? launch<64, 512>(a, rows, C, st) : launch<64, 256>(a, rows, C, st);
}

}  // extern "C"
