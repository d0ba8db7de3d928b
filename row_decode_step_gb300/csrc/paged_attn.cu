// Attention over the paged 4-bit cache.
//
// Work.  An item is (sequence, KV head, tile of 4 or 8 queries); its keys are taken in chunks of 32
// (two cells).  The chunks of all items, kItemCost units for each item's own cost before them, stand
// in one line, which is cut into equal ranges, a CTA each: ragged lengths and few sequences alike
// load every SM, and no plan is made on the host.  A CTA finds its range by a scan over the lengths.
// Items a cut falls into leave (O, reference, sum) in the workspace; the CTA that completes an
// item's count joins its parts in their order, so that results do not depend on which one that is.
//
// Products.  Keys are the 16-row side of 16x8x16 f16 products: S^T = K Q^T and O^T = V^T P^T, so
// that 8 queries fill the narrow side.  The codes are used as they lie in the cell:
//   a nibble pair OR'ed into the mantissas of 1024 (or 64, for the second nibble), less 1032 (72):
//   two instructions for two codes u - 8, exact.  (A nibble alone is the f16 subnormal u 2^-24 and
//   needs no OR, but products of subnormals are cut at the subnormals' own scale: outputs 7e-6 off 64
//   bits instead of 5e-7.)
//   K  the block's scale multiplies the block's sum of 32 channels in f32
//   V  the scale multiplies the weights: P d, per block of 32 channels
// q and P d enter as two f16 terms each (hi + lo, 22 bits), because the results are f32: with one term
// they would carry 11 bits.  q is scaled by a power of two per row, P through the softmax's reference
// (its largest at 2^8 to 2^15) and, where the V scales are small or large, d by a power of two, so
// that P d stays under 2^15 and keeps its low terms; P is split once, turned to the operand's layout,
// and (P d)'s terms follow in f16 from hi = r(P_hi d), lo = r(P_lo d + (P_hi d - hi)), the difference
// being exact.  With four queries the terms lie side by side in one product: columns 0-3 the hi terms,
// 4-7 the lo terms.  Tiles of 16 queries would decode a key once for both halves, but their 255
// registers leave two CTAs an SM (24 sequences of 1 to 5 drafted rows 70 us, in tiles of eight 68).
//
// Bound by a warp's own chain of instructions (740 for 32 keys, 0.6 a cycle and scheduler): 16 sequences
// of 32768 keys run at 4.5 TB/s (133 us), with the codes used undecoded (wrong, to see) at 5.3.
#include <cmath>

#include "dl_async.cuh"
#include "paged_kv.cuh"
#include "paged_layout.h"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 2 * dlp::kCell;       // keys a warp takes at a time
constexpr int kItemCost = 12;                // an item's queries, join and output, in chunks
// Items of at most kUncut chunks are not cut: their parts' join would cost more than the balance gains (333
// keys 7.1 us, cut 10.6; 256 short sequences 20.0 and 21.0; with 40 chunks 18.9, but 64 ragged sequences 52.2 ->
// 53.9 and 48 sequences of 1088 chosen keys 22.8 -> 25.2).
constexpr int kUncut = 24;
constexpr int kKept = 512;                   // sequences whose lengths a CTA copies; more are planned after the wait
                                             // (256 short sequences: 20.0 us, after the wait 21.0)
constexpr int kLeastChunks = kWarps;         // a chunk a warp: 333 keys 7.1 us, with 16 chunks 12.1

// Ring stages a warp, a power of two: three of 32 keys were no faster than two.
constexpr int stages(int D) { return 2 * (128 / D); }

struct PagedAttnArgs {
    const float *q;
    int64_t q_stride;
    const uint8_t *pool;
    const int32_t *tables;
    int64_t table_stride;
    int n_seqs, width;
    const int32_t *seqlen, *row_begin;
    const int32_t *list;
    int n_list;
    float *out, *lse;
    int64_t out_stride;
    int32_t *status;
    float *parts;             // [grid][2] of QT x (D + 2) floats
    int *counters;            // [3][grid]: arrivals at an item's first group, at its others, groups done
    int rows, max_rows, n_q, n_kv, page, page_shift, n_pages;
    float qk_scale;           // log2(e) / sqrt(D)
};

// a / b of numbers that mostly fit 32 bits (a >= 0, b > 0).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return (a | b) >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// A sequence as the work line sees it.
struct Seq {
    int len, row0, rows, tiles, chunks;      // keys, its rows, query tiles, chunks of an item
    int items, work;                         // its items and their chunks (the host keeps both in 31 bits)
};

// Where the plan reads lengths and rows: the caller's arrays, or the CTA's copies of them.
struct Lens {
    const int32_t *len, *row_begin;
};

template <int QT>
__device__ __forceinline__ Seq seq_at(const PagedAttnArgs &a, const Lens &src, int s)
{
    Seq q;
    const int64_t most = (int64_t)a.width << a.page_shift;
    q.len = (int)min((int64_t)max(src.len[s], 0), most);
    q.row0 = s;
    q.rows = 1;
    if (src.row_begin) {
        q.row0 = src.row_begin[s];
        q.rows = min(max(src.row_begin[s + 1] - q.row0, 0), a.max_rows);
        // row indexes outside q are never followed
        if (q.row0 < 0 || q.row0 > a.rows) q.rows = 0;
        else q.rows = min(q.rows, a.rows - q.row0);
    }
    const int G = a.n_q / a.n_kv;
    q.tiles = (q.rows * G + QT - 1) / QT;
    int keys = q.len;
    if (a.list) keys = min((q.len + a.page - 1) >> a.page_shift, a.n_list) << a.page_shift;
    q.chunks = max(1, (keys + kChunk - 1) / kChunk);
    q.items = q.tiles * a.n_kv;
    q.work = q.items * q.chunks;
    return q;
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                    float c2, float c3)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%10,%11,%12,%13};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    mma(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (x, y) as f16 pairs hi + lo.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 r = __ffma2_rn(__half22float2(h), make_float2(-1.f, -1.f), make_float2(x, y));
    const __half2 l = __float22half2_rn(r);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// f16 pairs: x y, x y + z, x y - z.
__device__ __forceinline__ __half2 h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) { return bits(__hmul2(h2(x), h2(y))); }
__device__ __forceinline__ uint32_t times_plus(uint32_t x, uint32_t y, uint32_t z) { return bits(__hfma2(h2(x), h2(y), h2(z))); }
__device__ __forceinline__ uint32_t times_minus(uint32_t x, uint32_t y, uint32_t z)
{
    return bits(__hfma2(h2(x), h2(y), __hneg2(h2(z))));
}

// u - 8 of nibble 0 of each half, and of nibble 1.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t y, uint32_t z)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(y), "r"(z));
    return r;
}
__device__ __forceinline__ uint32_t code_low(uint32_t w) { return bits(__hadd2(h2(and_or(w, 0x000F000Fu, 0x64006400u)), h2(0xE408E408u))); }
__device__ __forceinline__ uint32_t code_high(uint32_t w) { return bits(__hadd2(h2(and_or(w, 0x00F000F0u, 0x54005400u)), h2(0xD480D480u))); }

template <int D>
__device__ __forceinline__ void load_words(uint32_t (&w)[D / 32], const uint8_t *p)
{
    if constexpr (D == 128) {
        const uint4 t = *reinterpret_cast<const uint4 *>(p);
        w[0] = t.x; w[1] = t.y; w[2] = t.z; w[3] = t.w;
    } else {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        w[0] = t.x; w[1] = t.y;
    }
}

// The D/32 scales of a key, as packed pairs.
template <int D>
__device__ __forceinline__ void load_scales(uint32_t (&w)[D / 64], const uint8_t *p)
{
    if constexpr (D == 128) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        w[0] = t.x; w[1] = t.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}
__device__ __forceinline__ float scale_of(const uint32_t *w, int b)
{
    const __half2 h = *reinterpret_cast<const __half2 *>(&w[b / 2]);
    return b & 1 ? __high2float(h) : __low2float(h);
}

constexpr float kFar = 4194304.f;            // 2^22

constexpr int kDesc = 32;                    // chunks of a warp that are described at a time, in two halves

// Shared memory: the warps' rings, the warps' outputs (whose room the references of an item's parts take
// when it is joined), the tile's queries as operands.
__host__ __device__ constexpr int ring_bytes(int D) { return kWarps * stages(D) * 2 * dlp::cell_bytes(D); }
__host__ __device__ constexpr int out_bytes(int D, int QT) { return kWarps * QT * (D + 4) * 4; }
__host__ __device__ constexpr int query_bytes(int D, int QT) { return D / 32 * 32 * (QT == 4 ? 16 : 32); }
template <int D, int QT>
constexpr int smem_bytes() { return ring_bytes(D) + out_bytes(D, QT) + query_bytes(D, QT); }

template <int D, int QT>
__host__ __device__ constexpr size_t part_floats() { return (size_t)QT * (D + 2); }

// The output row and lse of query qi of a tile: O over its sum of weights.  (Without a reference the sum
// is 0, or NaN for a query that is NaN itself: lse is then -inf or NaN.)
struct Target {
    float *out, *lse;                        // of the tile's first row and head; lse may be null
    int64_t out_stride;
    int n_q, G, q0;                          // q0: the tile's first query counted from that row's first head
};
template <int D>
__device__ __forceinline__ void store_query(const Target &w, int qi, int d, float R, float L, float4 v)
{
    const int row = (w.q0 + qi) / w.G, head = (w.q0 + qi) - row * w.G;
    const float n = R == -INFINITY ? 0.f : 1.0f / L;
    *reinterpret_cast<float4 *>(w.out + (int64_t)row * w.out_stride + (int64_t)head * D + d) =
        make_float4(v.x * n, v.y * n, v.z * n, v.w * n);
    if (d == 0 && w.lse)
        w.lse[(int64_t)row * w.n_q + head] = R == -INFINITY ? fmaf(0.f, L, R) : (R + log2f(L)) * 0.69314718056f;
}

// A part of a cut item: O [QT][D], references [QT], sums [QT].
template <int D, int QT>
__device__ __forceinline__ void store_part(float *p, int qi, int d, float R, float L, float4 v)
{
    *reinterpret_cast<float4 *>(p + qi * D + d) = v;
    if (d == 0) {
        p[QT * D + qi] = R;
        p[QT * D + QT + qi] = L;
    }
}

// The most parts joined at once; an item of more is joined in groups of about its square root first.
constexpr int kJoinMost = 12;
inline int group_size_most(int n) { return n <= kJoinMost ? n : (int)sqrtf((float)n) + 1 + kJoinMost; }
__device__ __forceinline__ int group_size(int n)
{
    if (n <= kJoinMost) return n;
    int w = (int)sqrtf((float)n);
    return w * w < n ? w + 1 : w;
}

// n parts in their order (part(i), i < n): the warps take each query's reference and sum from all of
// them (the references stay in s_w), then emit(query, channel, reference, sum, O) gets the weighted
// sums.  The first four parts are on their way meanwhile.  (With six or eight in flight this rare code's
// registers slowed the loop over the chunks, 64 ragged sequences 51 -> 52 and 54 us.)
template <int D, int QT, typename Part, typename Emit>
__device__ __forceinline__ void join_parts(Part part, int n, int nq, float *s_w, float *s_ref, float *s_sum, Emit emit)
{
    constexpr int kFlight = 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float4 u[kFlight];
    auto fetch = [&](int i0, int e) {
#pragma unroll
        for (int i = 0; i < kFlight; ++i)
            if (i0 + i < n) u[i] = __ldcg(reinterpret_cast<const float4 *>(part(i0 + i)) + e);
    };
    int e = tid;                             // query e / (D/4), channels 4 (e % (D/4)) ..
    if (e < nq * (D / 4)) fetch(0, e);
    for (int qi = warp; qi < nq; qi += kWarps) {
        float R = -INFINITY, L = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float r = __ldcg(part(i) + QT * D + qi), l = __ldcg(part(i) + QT * D + QT + qi);
            s_w[i * QT + qi] = r;
            const float m = fmaxf(R, r);
            // (no reference yet: the sums are 0, or the NaN of a query that is none)
            L = m == -INFINITY ? L + l : L * exp2_approx(R - m) + l * exp2_approx(r - m);
            R = m;
        }
        float m = R;
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
        if (m != -INFINITY) L *= exp2_approx(R - m);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
        if (lane == 0) {
            s_ref[qi] = m;
            s_sum[qi] = L;
        }
    }
    __syncthreads();
    for (; e < nq * (D / 4); e += kThreads) {
        const int qi = e / (D / 4);
        const float R = s_ref[qi];
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < n; i0 += kFlight) {
            if (i0 || e != tid) fetch(i0, e);
#pragma unroll
            for (int i = 0; i < kFlight; ++i)
                if (i0 + i < n) {
                    const float f = R == -INFINITY ? 0.f : exp2_approx(s_w[(i0 + i) * QT + qi] - R);
                    v.x = fmaf(f, u[i].x, v.x);
                    v.y = fmaf(f, u[i].y, v.y);
                    v.z = fmaf(f, u[i].z, v.z);
                    v.w = fmaf(f, u[i].w, v.w);
                }
        }
        emit(qi, (e - qi * (D / 4)) * 4, R, s_sum[qi], v);
    }
}

template <int D, int QT>
__global__ void __launch_bounds__(kThreads, dlp::attn_ctas_per_sm(D, QT)) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a)
{
    constexpr int NB = D / 32;               // blocks of 32 channels
    constexpr int S = stages(D), CB = dlp::cell_bytes(D), OS = D + 4;
    constexpr bool PK = QT == 4;             // columns 0-3 the queries' hi terms, 4-7 their lo terms
    constexpr int PF = (int)part_floats<D, QT>();
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ __align__(8) uint64_t s_full[kWarps][S];
    __shared__ float s_ref[kWarps][QT], s_sum[kWarps][QT];
    __shared__ __align__(16) int4 s_desc[kWarps][kDesc];      // a chunk's cells (-1: none) and their first keys
    __shared__ long long s_scan[kWarps][2], s_chunk[2], s_unit;
    __shared__ int s_seq, s_last, s_len[kKept], s_rows[kKept + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    unsigned char *ring = smem + (size_t)warp * S * 2 * CB;
    float *s_o = reinterpret_cast<float *>(smem + ring_bytes(D));    // [warp][query][OS]
    uint4 *s_q = reinterpret_cast<uint4 *>(smem + ring_bytes(D) + out_bytes(D, QT));  // [block][hi, lo][lane]
    const int G = a.n_q / a.n_kv;

    if (lane == 0) {
        for (int i = 0; i < S; ++i) dla::mbar_init(&s_full[warp][i], 1);
        dla::mbar_init_fence();
    }

    // ---- the work line: its length, this CTA's range of it, the sequence the range starts in; the first
    // chunks' cells.  All this comes from lengths and tables that the caller keeps, and is mostly done while
    // the previous kernel runs.  That kernel may still write them: up to kKept sequences' lengths are copied
    // once, so that every thread plans from the same numbers, whatever they are, and after the wait lengths and
    // table entries are read again; had any changed, the plan is made anew.  (333 keys 7.1 us among others, all
    // of it after the wait 9.2.)
    const bool kept = a.n_seqs <= kKept;
    const Lens src = {kept ? s_len : a.seqlen, !a.row_begin ? nullptr : kept ? s_rows : a.row_begin};
    const int s_lo = (int)((int64_t)a.n_seqs * tid / kThreads), s_hi = (int)((int64_t)a.n_seqs * (tid + 1) / kThreads);
    bool early = kept;                       // the previous kernel may be running
    bool odd = false, held = false;          // a length out of range, an entry out of range of an early look
    long long per;
    int n_range, mine_n, d_seq, d_base;
    uint32_t open;                           // bit i: every query of chunk i's tile sees all 32 keys
    const int32_t *entry;                    // the table entry the lane looked at last, and what it held
    int entry_was;
    // the warp's chunks: every kWarps-th of the range, described 16 at a time, a cell a lane
    auto describe = [&](int j0) {
        const int t = lane >> 4, ji = j0 + (lane & 15);
        int cell = -1, pos = 0;
        bool all = false;
        if (ji < mine_n) {
            const int x = warp + kWarps * ji;
            Seq q = seq_at<QT>(a, src, d_seq);
            while (x >= d_base + q.work) {
                d_base += q.work;
                q = seq_at<QT>(a, src, ++d_seq);
            }
            const int r = x - d_base, item = r / q.chunks, h = item / q.tiles;
            const int key = (r - item * q.chunks) * kChunk + t * dlp::kCell, in = key & (a.page - 1);
            const int np = (q.len + a.page - 1) >> a.page_shift;
            int lp = key >> a.page_shift;
            bool ok = true, bad = false;
            if (a.list) {
                ok = lp < min(np, a.n_list);
                if (ok) {
                    lp = a.list[((int64_t)q.row0 * a.n_kv + h) * a.n_list + lp];
                    bad = lp < 0 || lp >= np;
                }
            }
            if (ok && !bad && (lp << a.page_shift) + in < q.len) {
                entry = a.tables + d_seq * a.table_stride + lp;
                const int phys = entry_was = __ldcg(entry);
                bad = phys < 0 || phys >= a.n_pages;
                if (!bad) {
                    cell = (phys * a.n_kv + h) * (a.page / dlp::kCell) + in / dlp::kCell;
                    pos = (lp << a.page_shift) + in;
                    const int n_rows = src.row_begin ? src.row_begin[d_seq + 1] - q.row0 : 1;
                    all = pos + dlp::kCell <= q.len - (n_rows - 1 - (item - h * q.tiles) * QT / G);
                }
            }
            if (bad && !early) dl_status_or(a.status, DL_STATUS_PAGE_RANGE);
            held |= bad;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, all);
        const int sh = j0 & 16;
        open = (open & ~(0xffffu << sh)) | ((m & (m >> 16) & 0xffffu) << sh);
        int *d = reinterpret_cast<int *>(&s_desc[warp][ji & (kDesc - 1)]);
        d[t] = cell;
        d[2 + t] = pos;
        __syncwarp();
    };
    bool bad = false;                        // a wait gave up, at chunk `stuck`
    int issued = 0, stuck = 0;
    auto issue = [&]() {                     // fetch the warp's next chunk into its slot
        if (issued >= mine_n) return;
        if ((issued & 15) == 0 && (issued || a.list)) describe(issued);
        if (lane == 0) {
            const int2 d = *reinterpret_cast<const int2 *>(&s_desc[warp][issued & (kDesc - 1)]);
            unsigned char *dst = ring + (issued & (S - 1)) * 2 * CB;
            uint64_t *bar = &s_full[warp][issued & (S - 1)];
            if ((d.x ^ -1) && d.y == d.x + 1) {
                dla::mbar_expect_tx(bar, 2 * CB);
                dla::bulk_g2s(dst, a.pool + (int64_t)d.x * CB, 2 * CB, bar);
            } else {
                dla::mbar_expect_tx(bar, (uint32_t)(((d.x >= 0) + (d.y >= 0)) * CB));
                if (d.x >= 0) dla::bulk_g2s(dst, a.pool + (int64_t)d.x * CB, CB, bar);
                if (d.y >= 0) dla::bulk_g2s(dst + CB, a.pool + (int64_t)d.y * CB, CB, bar);
            }
        }
        ++issued;
    };
    // ---- segments: the part of one item in this range
    struct Segment {
        Seq q;
        int item, h, ch0, n, q0, nq, n_rows;     // item of its sequence, first chunk, chunks, queries
        int fb, lb;                          // the CTAs that share the item, where it is cut
    };
    int x = 0, sq, base;
    long long ubase;                         // the sequence's first unit on the whole line
    float qv[NB][8];                         // the lane's share of the tile's queries as they are
    auto open_segment = [&](Segment &z) {
        z.q = seq_at<QT>(a, src, sq);
        while (x >= base + z.q.work) {
            base += z.q.work;
            ubase += z.q.work + (long long)kItemCost * z.q.items;
            z.q = seq_at<QT>(a, src, ++sq);
        }
        const int r = x - base;
        z.item = r / z.q.chunks;
        z.ch0 = r - z.item * z.q.chunks;
        z.h = z.item / z.q.tiles;
        z.n = min(z.q.chunks - z.ch0, n_range - x);
        z.q0 = (z.item - z.h * z.q.tiles) * QT;
        z.nq = min(QT, z.q.rows * G - z.q0);
        z.n_rows = src.row_begin ? src.row_begin[sq + 1] - z.q.row0 : 1;
        z.fb = z.lb = 0;
        if (z.n < z.q.chunks) {
            const long long unit = ubase + (long long)z.item * (z.q.chunks + kItemCost) + kItemCost;
            z.fb = (int)quotient(unit, per);
            z.lb = (int)quotient(unit + z.q.chunks - 1, per);
        }
    };
    auto load_queries = [&](const Segment &z) {
        const int col = PK ? g & 3 : g, qi = z.q0 + col, hq = z.h * G + qi % G;
        const bool has = col < z.nq;
        const float *src = a.q + (int64_t)(z.q.row0 + qi / G) * a.q_stride + (int64_t)hq * D + 8 * c;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float4 u0 = make_float4(0.f, 0.f, 0.f, 0.f), u1 = u0;
            if (has) {
                u0 = *reinterpret_cast<const float4 *>(src + 32 * b);
                u1 = *reinterpret_cast<const float4 *>(src + 32 * b + 4);
            }
            qv[b][0] = u0.x; qv[b][1] = u0.y; qv[b][2] = u0.z; qv[b][3] = u0.w;
            qv[b][4] = u1.x; qv[b][5] = u1.y; qv[b][6] = u1.z; qv[b][7] = u1.w;
        }
    };
    int j = 0;
    Segment z;
    if (!kept) {
        dl_pdl_wait();
        dl_pdl_launch_dependents();
    }
    while (true) {
        if (kept) {
            for (int s = s_lo; s < s_hi; ++s) {
                s_len[s] = __ldcg(a.seqlen + s);
                if (a.row_begin) s_rows[s] = __ldcg(a.row_begin + s);
            }
            if (a.row_begin && tid == kThreads - 1) s_rows[a.n_seqs] = __ldcg(a.row_begin + a.n_seqs);
            __syncthreads();
        }
        odd = held = false;
        entry = nullptr;
        long long n_chunk = 0, n_item = 0;       // of the thread's sequences
        for (int s = s_lo; s < s_hi; ++s) {
            const Seq q = seq_at<QT>(a, src, s);
            n_chunk += q.work;
            n_item += q.items;
            const int raw = src.len[s];
            odd |= raw < 0 || raw > ((int64_t)a.width << a.page_shift) ||
                   (src.row_begin && src.row_begin[s + 1] - src.row_begin[s] > a.max_rows);
        }
        long long chunk0 = n_chunk, item0 = n_item;     // inclusive, then exclusive sums
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, chunk0, o), u = __shfl_up_sync(0xffffffffu, item0, o);
            if (lane >= o) {
                chunk0 += t;
                item0 += u;
            }
        }
        if (lane == 31) {
            s_scan[warp][0] = chunk0;
            s_scan[warp][1] = item0;
        }
        __syncthreads();
        long long chunks = 0, items = 0;
        chunk0 -= n_chunk;
        item0 -= n_item;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) {
                chunk0 += s_scan[w][0];
                item0 += s_scan[w][1];
            }
            chunks += s_scan[w][0];
            items += s_scan[w][1];
        }
        const long long units = chunks + kItemCost * items;
        per = max(quotient(units + gridDim.x - 1, gridDim.x), (long long)(kLeastChunks + kItemCost));
        n_range = 0;
        if (per * blockIdx.x < units) {
            // chunk k of an item stands at unit kItemCost + k of it; a cut before that leaves the item whole
            if (tid == 0) s_chunk[1] = chunks;
            __syncthreads();
#pragma unroll
            for (int end = 0; end < 2; ++end) {
                const long long at = per * (blockIdx.x + end), u0 = chunk0 + kItemCost * item0;
                if (u0 <= at && at < u0 + n_chunk + kItemCost * n_item) {
                    long long u = u0, ch = chunk0;
                    for (int s = s_lo;; ++s) {
                        const Seq q = seq_at<QT>(a, src, s);
                        const long long n = q.work + (long long)kItemCost * q.items;
                        if (at < u + n) {
                            const long long r = at - u, item = quotient(r, q.chunks + kItemCost);
                            int k = max((int)(r - item * (q.chunks + kItemCost)) - kItemCost, 0);
                            if (q.chunks <= kUncut) k = 2 * k > q.chunks ? q.chunks : 0;     // short items stay whole
                            s_chunk[end] = ch + item * q.chunks + k;
                            if (end == 0) {
                                s_seq = s;
                                s_unit = u;
                                s_scan[0][0] = ch;
                            }
                            break;
                        }
                        u += n;
                        ch += q.work;
                    }
                }
            }
            __syncthreads();
            // from here on chunks are counted from the range's first
            n_range = (int)(s_chunk[1] - s_chunk[0]);
            base = d_base = (int)(s_scan[0][0] - s_chunk[0]);    // the first sequence's first chunk
            sq = d_seq = s_seq;
            ubase = s_unit;
            mine_n = (n_range - warp + kWarps - 1) / kWarps;
            open = 0;
            if (n_range > 0) open_segment(z);
            __syncwarp();
            if (!a.list && mine_n > 0) describe(0);  // (a list comes from the previous kernel)
        }
        if (!early) break;
        early = false;
        dl_pdl_wait();
        dl_pdl_launch_dependents();
        bool changed = entry && __ldcg(entry) != entry_was;
        for (int s = s_lo; s < s_hi; ++s) {
            changed |= __ldcg(a.seqlen + s) != s_len[s];
            if (a.row_begin) changed |= __ldcg(a.row_begin + s) != s_rows[s];
        }
        if (a.row_begin && tid == kThreads - 1) changed |= __ldcg(a.row_begin + a.n_seqs) != s_rows[a.n_seqs];
        if (!__syncthreads_or(changed)) {
            if (held) dl_status_or(a.status, DL_STATUS_PAGE_RANGE);
            break;
        }
    }
    if (odd && blockIdx.x == 0) dl_status_or(a.status, DL_STATUS_SEQLEN_RANGE);
    if (n_range == 0) return;
    load_queries(z);                         // (on their way while the first chunks are asked for)
    for (int i = 0; i < S - 1; ++i) issue();
    while (x < n_range) {
        const int j_end = (x + z.n - warp + kWarps - 1) / kWarps;    // the warp's chunks of it
        // ---- the tile's queries as B operands, hi + lo, a block a warp (all warps have left the segment before)
        float top = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(qv[b][i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // power of two that brings the largest |q| into [2^14, 2^15) (-113: that of the largest number)
        const int e = min(100, max(-113, 14 - ((int)(__float_as_uint(top) >> 23) - 127)));
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const float back = a.qk_scale * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int b = 0; b < NB; ++b)
            if (b % kWarps == warp) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int p = 0; p < 4; ++p)      // nibbles (p, p + 4) of the lane's word
                    split2(qv[b][p] * up, qv[b][p + 4] * up, hi[p], lo[p]);
                uint4 *dst = s_q + b * (PK ? 1 : 2) * 32 + lane;
                if (PK && g >= 4) {
                    dst[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                } else {
                    dst[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    if constexpr (!PK) dst[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
        const float2 cq = make_float2(__shfl_sync(0xffffffffu, back, 8 * c), __shfl_sync(0xffffffffu, back, 8 * c + 4));
        __syncthreads();

        // ---- the chunks
        float o[D / 16][4], mraw[2];
        float2 sum, ref;                     // by the lane's two queries; ref 0 while nothing is seen
        uint32_t dtop = 0;                   // largest V scale so far (f16 bits)
        float kshift = 0.f;                  // P carries 2^kshift and d 2^dshift: together they put P d
        int dshift = 0;                      // under 2^15
        bool started = false;                // every query of the tile has seen a key, none a far one
#pragma unroll
        for (int m = 0; m < D / 16; ++m) o[m][0] = o[m][1] = o[m][2] = o[m][3] = 0.f;
        mraw[0] = mraw[1] = -INFINITY;
        ref = sum = make_float2(0.f, 0.f);
        for (; j < j_end && !bad; ++j) {
            issue();
            unsigned char *ck = ring + (j & (S - 1)) * 2 * CB;
            if (__any_sync(0xffffffffu, !dla::mbar_wait(&s_full[warp][j & (S - 1)], (uint32_t)(j / S) & 1u))) {
                if (lane == 0) dl_status_or(a.status, DL_STATUS_SYNC_TIMEOUT);
                bad = true;
                stuck = j;
                break;
            }

            // the largest V scale of the lane's key (scales are not negative: their bits compare as numbers)
            uint32_t dk[D / 64], dmine = 0;
            load_scales<D>(dk, ck + (lane >> 4) * CB + dlp::v_scale_off(D) + (lane & 15) * (D / 16));
#pragma unroll
            for (int i = 0; i < D / 64; ++i) dmine = __vmaxu2(dmine, dk[i]);
            dmine = max(dmine & 0xffffu, dmine >> 16);

            // scores of both cells
            float2 sc[2][2];                 // [cell][key g, g + 8], by the lane's two queries
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const unsigned char *cell = ck + t * CB;
                uint32_t w0[NB], w1[NB], ks[2][D / 64];
                load_words<D>(w0, cell + g * (D / 2) + c * (D / 8));
                load_words<D>(w1, cell + (g + 8) * (D / 2) + c * (D / 8));
                load_scales<D>(ks[0], cell + dlp::k_scale_off(D) + g * (D / 16));
                load_scales<D>(ks[1], cell + dlp::k_scale_off(D) + (g + 8) * (D / 16));
                sc[t][0] = sc[t][1] = make_float2(0.f, 0.f);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t x0 = w0[b] >> 8, x1 = w1[b] >> 8;
                    const uint32_t a0[4] = {code_low(w0[b]), code_low(w1[b]), code_high(w0[b]), code_high(w1[b])};
                    const uint32_t a1[4] = {code_low(x0), code_low(x1), code_high(x0), code_high(x1)};
                    const float d0 = scale_of(ks[0], b), d1 = scale_of(ks[1], b);
                    float acc[4];
                    const uint4 *qb = s_q + b * (PK ? 1 : 2) * 32 + lane;
                    const uint4 qh = qb[0];
                    if constexpr (PK) {
                        mma(acc, a0, qh.x, qh.y, 0.f, 0.f, 0.f, 0.f);
                    } else {
                        const uint4 ql = qb[32];
                        mma(acc, a0, ql.x, ql.y, 0.f, 0.f, 0.f, 0.f);
                        mma(acc, a1, ql.z, ql.w);
                        mma(acc, a0, qh.x, qh.y);
                    }
                    mma(acc, a1, qh.z, qh.w);
                    sc[t][0].x = fmaf(acc[0], d0, sc[t][0].x);
                    sc[t][0].y = fmaf(acc[1], d0, sc[t][0].y);
                    sc[t][1].x = fmaf(acc[2], d1, sc[t][1].x);
                    sc[t][1].y = fmaf(acc[3], d1, sc[t][1].y);
                }
                if constexpr (PK)            // hi + lo: the lane two columns on holds the other half
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        sc[t][i].x += __shfl_xor_sync(0xffffffffu, sc[t][i].x, 2);
                        sc[t][i].y += __shfl_xor_sync(0xffffffffu, sc[t][i].y, 2);
                    }
            }
            if (!(open >> (j & 31) & 1)) {   // some query does not see all keys
                const int4 d = s_desc[warp][j & (kDesc - 1)];
                // keys that nobody wrote may hold any scale: make V's 0 (their scores are replaced)
                const int cell = lane < 16 ? d.x : d.y, pos = (lane < 16 ? d.z : d.w) + (lane & 15);
                if (cell < 0 || pos >= z.q.len) {
                    uint32_t *v = reinterpret_cast<uint32_t *>(ck + (lane >> 4) * CB + dlp::v_scale_off(D) + (lane & 15) * (D / 16));
#pragma unroll
                    for (int i = 0; i < D / 64; ++i) v[i] = 0;
                    dla::fence_proxy_async();            // (the slot's next fetch comes after this store)
                    dmine = 0;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // keys the query of column 2c + i sees: row r of n sees len - (n - 1 - r)
                    const int col = PK ? (2 * c + i) & 3 : 2 * c + i;
                    const int see = col < z.nq ? z.q.len - (z.n_rows - 1 - (z.q0 + col) / G) : 0;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int p = (t ? d.y : d.x) < 0 ? 0x7fffff00 : (t ? d.w : d.z) + g;
                        float2 &lo = sc[t][0], &hi = sc[t][1];
                        if (p >= see) (i ? lo.y : lo.x) = -INFINITY;
                        if (p + 8 >= see) (i ? hi.y : hi.x) = -INFINITY;
                    }
                }
                __syncwarp();
            }
            // exponents of the weights.  The references stay as they are while no weight passes twice the
            // largest that they were set for, no V scale passes its largest so far and every query of the
            // tile has seen a key
            float most = -INFINITY;
            const float2 minus = make_float2(-ref.x, -ref.y);
            float2 ex[2][2];                 // the exponents
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ex[t][i] = __ffma2_rn(sc[t][i], cq, minus);
                    most = fmaxf(most, fmaxf(ex[t][i].x, ex[t][i].y));
                }
            const bool stale = most > kshift + 1.f || dmine > dtop || !started;
            if (__any_sync(0xffffffffu, stale)) {
                float od = 1.f;              // what the outputs' factor 2^dshift changes by
                const uint32_t dm = __reduce_max_sync(0xffffffffu, dmine);
                if (dm > dtop) {
                    dtop = dm;
                    const float d = __half2float(__ushort_as_half((unsigned short)dm));
                    const int k = 13 - ((int)(__float_as_uint(d) >> 23) - 127), kp = max(min(k, 14), 8);
                    od = exp2f((float)(k - kp - dshift));
                    kshift = (float)kp;
                    dshift = k - kp;
                }
                bool seen = true;
                float mx = fmaxf(fmaxf(sc[0][0].x, sc[0][1].x), fmaxf(sc[1][0].x, sc[1][1].x));
                float my = fmaxf(fmaxf(sc[0][0].y, sc[0][1].y), fmaxf(sc[1][0].y, sc[1][1].y));
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                    my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, w));
                }
                mraw[0] = fmaxf(mx, mraw[0]);
                mraw[1] = fmaxf(my, mraw[1]);
                seen = seen && mraw[0] != -INFINITY && mraw[1] != -INFINITY;
                float2 nref = make_float2(mraw[0] == -INFINITY ? 0.f : fmaf(mraw[0], cq.x, -kshift),
                                          mraw[1] == -INFINITY ? 0.f : fmaf(mraw[1], cq.y, -kshift));
                // References as large as this are off by a quarter of an exponent and more, so that the products'
                // exact differences from them are nobody's weights (past f16 from 2^25 on): here the scores are
                // rounded first and the largest weight is 1, chunk by chunk.  (The exponents pass on from here, which costs
                // 24 drafted sequences 67.7 -> 68.2 us; computed again below, with a factor for these, 69.8.)
                const bool far_x = fabsf(nref.x) >= kFar, far_y = fabsf(nref.y) >= kFar;
                if (far_x) nref.x = __fmul_rn(mraw[0], cq.x);
                if (far_y) nref.y = __fmul_rn(mraw[1], cq.y);
                seen = seen && !far_x && !far_y;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        ex[t][i].x = far_x ? __fsub_rn(__fmul_rn(sc[t][i].x, cq.x), nref.x) : fmaf(sc[t][i].x, cq.x, -nref.x);
                        ex[t][i].y = far_y ? __fsub_rn(__fmul_rn(sc[t][i].y, cq.y), nref.y) : fmaf(sc[t][i].y, cq.y, -nref.y);
                    }
                // (a query that has seen nothing has sums of zero: any finite factor will do)
                const float2 f = make_float2(exp2_approx(fminf(ref.x - nref.x, 100.f)),
                                             exp2_approx(fminf(ref.y - nref.y, 100.f)));
                ref = nref;
                sum = __fmul2_rn(sum, f);
                const float fx = f.x * od, fy = f.y * od;
#pragma unroll
                for (int m = 0; m < D / 16; ++m) {
                    o[m][0] *= fx;
                    o[m][1] *= fy;
                    o[m][2] *= fx;
                    o[m][3] *= fy;
                }
                started = __all_sync(0xffffffffu, seen);
            }
            if (dshift) {                    // small or large scales: d 2^dshift, in place
                const float f = exp2f((float)dshift);
                __half *v = reinterpret_cast<__half *>(ck + (lane >> 4) * CB + dlp::v_scale_off(D) + (lane & 15) * (D / 16));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) v[i] = __float2half_rn(__half2float(v[i]) * f);
                dla::fence_proxy_async();
                __syncwarp();
            }
            // weights 2^(s - ref), their terms in the operand's layout: keys 2c, 2c + 1 and 2c + 8, 2c + 9 of
            // query column g.  (QT = 4: columns 0-3 get P d rounded, from pa d + 0; columns 4-7 what that
            // leaves, from pa d + (ph d - r(ph d)).)
            uint32_t ph[2][2], pa[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 w = make_float2(exp2_approx(ex[t][i].x), exp2_approx(ex[t][i].y));
                    sum = __fadd2_rn(sum, w);
                    uint32_t hi, lo;
                    split2(w.x, w.y, hi, lo);
                    ph[t][i] = transpose8x8(PK && c < 2 ? 0u : hi);
                    pa[t][i] = transpose8x8(PK && c < 2 ? hi : lo);
                }
            // O += (P d) V
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const unsigned char *cell = ck + t * CB;
                uint32_t w0[NB], w1[NB], k0[D / 32], k1[D / 32];     // codes; scales of the keys 2c, 2c + 1 (+ 8)
                const int place = (g ^ dlp::v_swizzle(D, c)) * (D / 8);
                load_words<D>(w0, cell + dlp::v_code_off(D) + c * D + place);
                load_words<D>(w1, cell + dlp::v_code_off(D) + (c + 4) * D + place);
                load_words<D>(k0, cell + dlp::v_scale_off(D) + c * (D / 8));
                load_words<D>(k1, cell + dlp::v_scale_off(D) + (c + 4) * (D / 8));
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t x0 = w0[b] >> 8, x1 = w1[b] >> 8;
                    const uint32_t a0[4] = {code_low(w0[b]), code_high(w0[b]), code_low(w1[b]), code_high(w1[b])};
                    const uint32_t a1[4] = {code_low(x0), code_high(x0), code_low(x1), code_high(x1)};
                    // (d of the even key, d of the odd key), D/64 words a key
                    const uint32_t d0 = __byte_perm(k0[b / 2], k0[D / 64 + b / 2], b & 1 ? 0x7632 : 0x5410);
                    const uint32_t d1 = __byte_perm(k1[b / 2], k1[D / 64 + b / 2], b & 1 ? 0x7632 : 0x5410);
                    const uint32_t h0 = times(ph[t][0], d0), h1 = times(ph[t][1], d1);
                    const uint32_t l0 = times_plus(pa[t][0], d0, times_minus(ph[t][0], d0, h0));
                    const uint32_t l1 = times_plus(pa[t][1], d1, times_minus(ph[t][1], d1, h1));
                    mma(o[2 * b], a0, l0, l1);
                    mma(o[2 * b + 1], a1, l0, l1);
                    if constexpr (!PK) {
                        mma(o[2 * b], a0, h0, h1);
                        mma(o[2 * b + 1], a1, h0, h1);
                    }
                }
            }
            __syncwarp();                    // the slot's readers are done: it may be filled again
        }

        // ---- join the warps
        if (dshift) {
            const float f = exp2f((float)-dshift);
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][i] *= f;
        }
        if constexpr (PK)
#pragma unroll
            for (int m = 0; m < D / 16; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][i] += __shfl_xor_sync(0xffffffffu, o[m][i], 2);
        x += z.n;
        const bool whole = z.n == z.q.chunks;
        const int nq = z.nq, fb = z.fb;
        // the item's first part lies in the second slot of its CTA, the others in the first
        float *mine = a.parts + ((int64_t)blockIdx.x * 2 + ((int)blockIdx.x == fb)) * PF;
        Target to;
        to.out = a.out + (int64_t)z.q.row0 * a.out_stride + (int64_t)z.h * G * D;
        to.lse = a.lse ? a.lse + (int64_t)z.q.row0 * a.n_q + z.h * G : nullptr;
        to.out_stride = a.out_stride;
        to.n_q = a.n_q;
        to.G = G;
        to.q0 = z.q0;
        __syncthreads();                     // s_o, s_ref and s_sum have been read
        // query 2c + i of the lane, channels 32 b + 4 g .. + 3
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float t = i ? sum.y : sum.x;
            t += __shfl_xor_sync(0xffffffffu, t, 4);
            t += __shfl_xor_sync(0xffffffffu, t, 8);
            t += __shfl_xor_sync(0xffffffffu, t, 16);
            if (PK && c >= 2) continue;
            if (g == 0) {
                s_ref[warp][2 * c + i] = mraw[i] == -INFINITY ? -INFINITY : i ? ref.y : ref.x;
                s_sum[warp][2 * c + i] = t;
            }
            float *dst = s_o + (warp * QT + 2 * c + i) * OS + 4 * g;
#pragma unroll
            for (int b = 0; b < NB; ++b)
                *reinterpret_cast<float4 *>(dst + 32 * b) =
                    make_float4(o[2 * b][i], o[2 * b][i + 2], o[2 * b + 1][i], o[2 * b + 1][i + 2]);
        }
        __syncthreads();
        for (int e = tid; e < nq * (D / 4); e += kThreads) {
            const int qi = e / (D / 4), d = (e - qi * (D / 4)) * 4;
            float R = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) R = fmaxf(R, s_ref[w][qi]);
            float L = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_ref[w][qi] == -INFINITY ? 0.f : exp2_approx(s_ref[w][qi] - R);
                const float4 u = *reinterpret_cast<const float4 *>(s_o + (w * QT + qi) * OS + d);
                L = fmaf(f, s_sum[w][qi], L);
                v.x = fmaf(f, u.x, v.x);
                v.y = fmaf(f, u.y, v.y);
                v.z = fmaf(f, u.z, v.z);
                v.w = fmaf(f, u.w, v.w);
            }
            if (whole) store_query<D>(to, qi, d, R, L, v);
            else store_part<D, QT>(mine, qi, d, R, L, v);
        }
        if (!whole) {
            // the CTA that completes a group of parts joins them, into the place of the group's first; the
            // one that completes the groups joins those (s_o is read out and free)
            const int n = z.lb - fb + 1;
            auto part = [&](int i) { return a.parts + ((int64_t)(fb + i) * 2 + (i == 0)) * PF; };
            const int W = group_size(n), first = ((int)blockIdx.x - fb) / W * W;
            int from = first, count = min(W, n - first), step = 1;
            int *counter = first ? a.counters + gridDim.x + fb + first : a.counters + fb;
            while (true) {
                __syncthreads();             // (before thread 0's release, as its acquire before the reads)
                if (tid == 0) {
                    int old;
                    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
                    s_last = old == count - 1;
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                if (!s_last) break;
                const bool done = step > 1 || W == n;
                join_parts<D, QT>([&](int i) { return part(from + i * step); }, count, nq, s_o, s_ref[0], s_sum[0],
                                  [&](int qi, int d, float R, float L, float4 v) {
                                      if (done) store_query<D>(to, qi, d, R, L, v);
                                      else store_part<D, QT>(part(from), qi, d, R, L, v);
                                  });
                if (done) break;
                from = 0;
                count = (n + W - 1) / W;
                step = W;
                counter = a.counters + 2 * gridDim.x + fb;
            }
        }
        if (x < n_range) {
            open_segment(z);
            load_queries(z);
        }
    }
    // a wait that gave up: leave no copy of this warp in flight
    if (bad)
        for (j = stuck; j < issued; ++j)
            if (!dla::mbar_wait(&s_full[warp][j & (S - 1)], (uint32_t)(j / S) & 1u)) break;
}

template <int D, int QT>
int launch(PagedAttnArgs &a, int sms, int64_t most_chunks, unsigned char *workspace, cudaStream_t st)
{
    static_assert(dlp::attn_ctas_per_sm(D, QT) <= dlp::kMostCtasPerSm, "counters of more CTAs");
    const dlp::AttnLayout layout = dlp::attn_layout(sms, D, QT);
    const int full = layout.grid;
    a.counters = reinterpret_cast<int *>(workspace);
    a.parts = reinterpret_cast<float *>(workspace + layout.counters);
    const int G = a.n_q / a.n_kv;
    const int64_t tiles = dl::ceil_div((int64_t)a.max_rows * G, QT);
    if (tiles * a.n_kv * most_chunks > 0x7fffffff)
        return dl::fail(DL_E_SHAPE, "dl_paged_attn: %lld query tiles x %d KV heads x %lld chunks of keys of a sequence pass 2^31 - 1",
                        (long long)tiles, a.n_kv, (long long)most_chunks);
    // no more CTAs than the longest possible work line can fill
    const int64_t items = (int64_t)a.n_seqs * a.n_kv * tiles;
    int64_t grid = full;
    if (items < full && most_chunks < (1 << 20))
        grid = dl::ceil_div(items * (most_chunks + kItemCost), kLeastChunks + kItemCost);
    if (grid > full) grid = full;
    constexpr int smem = smem_bytes<D, QT>();
    // the references of a group's parts lie where the warps' outputs did
    if ((int64_t)(group_size_most(full) + 1) * QT * 4 > out_bytes(D, QT))
        return dl::fail(DL_E_SHAPE, "dl_paged_attn: %d CTAs are more parts than an item's join holds", full);
    auto go = [&]() {
        return dl::launch_pdl(paged_attn_kernel<D, QT>, dim3((unsigned)grid), dim3(kThreads), smem, st,
                              "dl_paged_attn: launch", a);
    };
    if constexpr (smem <= 41 * 1024) return go();        // (48 KB with the kernel's 7 KB of static shared memory)
    static std::atomic<uint64_t> asked{0};
    return dlp::launch_wide(reinterpret_cast<const void *>(paged_attn_kernel<D, QT>), smem, asked,
                            "dl_paged_attn: shared memory", go);
}

int check_heads(const char *who, int n_q, int n_kv, int D)
{
    if (n_kv <= 0 || n_q <= 0 || n_q % n_kv != 0 || n_q / n_kv > 16 || (D != 64 && D != 128))
        return dl::fail(DL_E_SHAPE, "%s: n_q=%d n_kv=%d head_dim=%d (at most 16 query heads a KV head; 64 or 128)", who, n_q,
                        n_kv, D);
    return DL_OK;
}

size_t workspace_bytes_for(int sms, int D)
{
    size_t most = 0;
    for (int QT = 4; QT <= 8; QT *= 2) {
        const size_t total = dlp::attn_layout(sms, D, QT).total();
        if (total > most) most = total;
    }
    return most;
}

}  // namespace

extern "C" {

int dl_paged_attn_workspace_size(int n_q, int n_kv, int head_dim, size_t *bytes)
{
    dl::clear_error();
    if (!bytes) return dl::fail(DL_E_ARG, "dl_paged_attn_workspace_size: null pointer");
    int rc = check_heads("dl_paged_attn_workspace_size", n_q, n_kv, head_dim);
    if (rc != DL_OK) return rc;
    int sms = 0;
    rc = dl::device_sm_count(&sms);
    if (rc != DL_OK) return rc;
    *bytes = workspace_bytes_for(sms, head_dim);
    return DL_OK;
}

int dl_paged_attn(const float *q, int64_t q_stride, const dl_paged_kv *kv, const dl_block_tables *tables,
                  const int32_t *seqlen, const int32_t *row_begin, int rows, int max_rows, int n_q,
                  const int32_t *pages, int n_list, float *out, int64_t out_stride, float *lse,
                  void *workspace, size_t workspace_bytes, int32_t *status, dl_stream_t stream)
{
    dl::clear_error();
    if ((rows != 0 && (!q || !out)) || (!seqlen && tables && tables->n_seqs != 0) || !workspace)
        return dl::fail(DL_E_ARG, "dl_paged_attn: null pointer");
    int rc = dlp::check_cache("dl_paged_attn", kv, tables, n_q, false);
    if (rc != DL_OK) return rc;
    rc = check_heads("dl_paged_attn", n_q, kv->n_kv, kv->head_dim);
    if (rc != DL_OK) return rc;
    if (rows < 0 || max_rows < 1 || (pages && n_list < 1))
        return dl::fail(DL_E_ARG, "dl_paged_attn: rows=%d max_rows=%d n_list=%d", rows, max_rows, n_list);
    if (!row_begin && (rows != tables->n_seqs || max_rows != 1))
        return dl::fail(DL_E_ARG, "dl_paged_attn: %d rows of %d sequences, max_rows=%d, want row_begin", rows,
                        tables->n_seqs, max_rows);
    if (pages && row_begin) return dl::fail(DL_E_ARG, "dl_paged_attn: a page list wants one row per sequence");
    if (q_stride < (int64_t)n_q * kv->head_dim || out_stride < (int64_t)n_q * kv->head_dim)
        return dl::fail(DL_E_ARG, "dl_paged_attn: strides below the row widths");
    if (!dl::aligned16(q) || !dl::aligned16(out) || q_stride % 4 != 0 || out_stride % 4 != 0 || !dl::aligned16(workspace))
        return dl::fail(DL_E_ALIGN, "dl_paged_attn: q, out and the workspace must be 16-byte aligned, strides multiples of 4");
    if (rows == 0 || tables->n_seqs == 0) return DL_OK;
    int sms = 0;
    rc = dl::device_sm_count(&sms);
    if (rc != DL_OK) return rc;
    const size_t need = workspace_bytes_for(sms, kv->head_dim);
    if (workspace_bytes < need)
        return dl::fail(DL_E_WORKSPACE, "dl_paged_attn: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    PagedAttnArgs a{};
    a.q = q; a.q_stride = q_stride;
    a.pool = static_cast<const uint8_t *>(kv->pool);
    a.tables = tables->pages; a.table_stride = tables->stride; a.n_seqs = tables->n_seqs; a.width = tables->width;
    a.seqlen = seqlen; a.row_begin = row_begin; a.list = pages; a.n_list = n_list;
    a.out = out; a.out_stride = out_stride; a.lse = lse; a.status = status;
    a.rows = rows; a.max_rows = max_rows; a.n_q = n_q; a.n_kv = kv->n_kv; a.page = kv->page; a.n_pages = kv->n_pages;
    while ((1 << a.page_shift) < kv->page) ++a.page_shift;
    a.qk_scale = 1.44269504089f / sqrtf((float)kv->head_dim);
    int64_t listed = tables->width;
    if (pages && n_list < listed) listed = n_list;
    const int64_t most_chunks = dl::ceil_div(listed * kv->page, kChunk) > 0 ? dl::ceil_div(listed * kv->page, kChunk) : 1;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // tiles of four queries where a sequence's rows have no more to a KV head, else of eight
    const bool four = (int64_t)max_rows * (n_q / kv->n_kv) <= 4;
    if (kv->head_dim == 128) return four ? launch<128, 4>(a, sms, most_chunks, ws, st) : launch<128, 8>(a, sms, most_chunks, ws, st);
    return four ? launch<64, 4>(a, sms, most_chunks, ws, st) : launch<64, 8>(a, sms, most_chunks, ws, st);
}

}  // extern "C"
