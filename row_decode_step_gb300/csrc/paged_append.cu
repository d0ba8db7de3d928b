// RoPE of a step's rows and their k and v into the pages of the paged 4-bit cache, and the mean
// key of every page a step fills.
//
// A group of D/8 lanes owns a k or v head of a row, eight consecutive channels a lane: that is one
// word of the K cell (eight nibbles) and two halves of the V cell, and a block of 32 channels is
// four neighbouring lanes, whose maximum two shuffles give; or two q heads, whose angles are the same.
// A thread asks for its heads' values before it knows its row's position, so that only the angles and
// the page wait for it.  Bound by that chain (position, table and angles, store) times the rounds of CTAs:
// a prompt of 4099 rows of 32 + 2 x 8 heads of 64 takes 22.7 us (105 MB: 4.6 TB/s, 68 % of a copy's rate),
// of 128 channels 40.8 us (4.6 TB/s); the q heads alone run at 5.8 TB/s.
#include "paged_kv.cuh"

namespace dlp {

int check_cache(const char *who, const dl_paged_kv *kv, const dl_block_tables *t, int n_q, bool want_mean)
{
    // (an empty batch may have no address for what it has no elements of)
    if (!kv || !t || !kv->pool || (!t->pages && t->n_seqs > 0)) return dl::fail(DL_E_ARG, "%s: null pointer", who);
    if (kv->head_dim != 64 && kv->head_dim != 128)
        return dl::fail(DL_E_SHAPE, "%s: head_dim=%d (64 or 128)", who, kv->head_dim);
    if (!page_ok(kv->page)) return dl::fail(DL_E_SHAPE, "%s: page=%d (16, 32, 64, 128 or 256)", who, kv->page);
    if (kv->n_kv <= 0 || n_q <= 0 || n_q % kv->n_kv != 0)
        return dl::fail(DL_E_SHAPE, "%s: n_q=%d n_kv=%d", who, n_q, kv->n_kv);
    if (kv->n_pages <= 0) return dl::fail(DL_E_ARG, "%s: n_pages=%d", who, kv->n_pages);
    if (t->n_seqs < 0 || t->width <= 0 || t->stride < t->width)
        return dl::fail(DL_E_ARG, "%s: tables of %d sequences, width %d, stride %lld", who, t->n_seqs, t->width,
                        (long long)t->stride);
    if ((int64_t)t->width * kv->page > 0x7fffff00)       // (positions and a page more fit 31 bits)
        return dl::fail(DL_E_SHAPE, "%s: width * page = %lld keys pass 2^31 - 256", who, (long long)t->width * kv->page);
    if (!dl::aligned16(kv->pool) || !dl::aligned16(kv->k_mean))
        return dl::fail(DL_E_ALIGN, "%s: the pool and the mean plane must be 16-byte aligned", who);
    if (want_mean && !kv->k_mean) return dl::fail(DL_E_ARG, "%s: the cache has no mean plane", who);
    return DL_OK;
}

}  // namespace dlp

namespace {

struct AppendArgs {
    const float *q, *k, *v, *bias;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *pos, *row_seq, *tables;
    int64_t table_stride;
    int n_seqs, width;
    const float2 *cs;
    uint8_t *pool;
    __half *mean;
    float *q_out, *k_out, *v_out;
    int64_t q_out_stride, k_out_stride, v_out_stride;
    int32_t *status;
    int rows, n_q, n_kv, page, page_shift, n_pages, rot, neox, max_pos;
    int vec;                  // float4 accesses throughout (see dl_paged_append)
    int own_pages;            // no two rows of the call write one page: its mean needs no second launch
};

// Where row r goes: its position p, its sequence's table entry `phys` and the status bit that refuses
// it (0: none; -1: padding).  Reads the table only where it may.
__device__ __forceinline__ int locate(const AppendArgs &a, int r, int &p, int &phys)
{
    p = a.pos[r];
    const int s = a.row_seq ? a.row_seq[r] : r;
    if (p < 0) return -1;
    if (s < 0 || s >= a.n_seqs) return DL_STATUS_REGION_RANGE;
    if (p >= a.max_pos || p >> a.page_shift >= a.width) return DL_STATUS_POS_RANGE;
    phys = a.tables[s * a.table_stride + (p >> a.page_shift)];
    return phys < 0 || phys >= a.n_pages ? DL_STATUS_PAGE_RANGE : 0;
}

// Channel c of a head at x (bias at b or NULL), rotated: the f32 operations of dl_rope_kv_store.
__device__ __forceinline__ float rotated(const AppendArgs &a, const float *x, const float *b, int c, const float2 *cs)
{
    float v = x[c] + (b ? b[c] : 0.f);
    if (c < a.rot) {
        const int rh = a.rot >> 1;
        const int j = a.neox ? (c < rh ? c : c - rh) : c >> 1;
        const int i0 = a.neox ? j : 2 * j, i1 = a.neox ? j + rh : 2 * j + 1;
        const float x0 = x[i0] + (b ? b[i0] : 0.f), x1 = x[i1] + (b ? b[i1] : 0.f);
        const float2 t = cs[j];
        v = c == i0 ? fmaf(x0, t.x, -x1 * t.y) : fmaf(x0, t.y, x1 * t.x);
    }
    return v;
}

// The mean key of a page of one KV head, by a warp: the decoded keys of each cell summed in f32 in
// their order, the cells' sums in theirs.  `stage`: 4 * 9 D bytes of shared memory of the warp's own,
// through which the cells' K halves pass (wide loads, all in flight at once).
template <int D>
__device__ __forceinline__ void store_mean(const AppendArgs &a, int phys, int h, unsigned char *stage)
{
    constexpr int KB = 9 * D, U = KB / 16;   // bytes, and 16-byte units, of a cell's K half
    constexpr int LG = D / 8, NG = 32 / LG;  // lanes of a cell (8 channels each), cells at a time
    const int lane = threadIdx.x & 31, l = lane % LG, grp = lane / LG, n_cells = a.page / dlp::kCell;
    const uint8_t *cells = a.pool + ((int64_t)phys * a.n_kv + h) * n_cells * dlp::cell_bytes(D);
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c0 = 0; c0 < n_cells; c0 += 4) {
        const int n = min(4, n_cells - c0);
        for (int u = lane; u < n * U; u += 32)
            reinterpret_cast<uint4 *>(stage)[u] = __ldcg(
                reinterpret_cast<const uint4 *>(cells + (int64_t)(c0 + u / U) * dlp::cell_bytes(D)) + u % U);
        __syncwarp();
        for (int k0 = 0; k0 < n; k0 += NG) {
            float part[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (k0 + grp < n) {
                const unsigned char *cell = stage + (k0 + grp) * KB;
#pragma unroll 4
                for (int t = 0; t < dlp::kCell; ++t) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(cell + dlp::k_word_off(D, t, 8 * l));
                    const float f = __half2float(
                        reinterpret_cast<const __half *>(cell + dlp::k_scale_off(D))[t * (D / 32) + l / 4]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) part[i] += (float)((int)((w >> (4 * i)) & 15u) - 8) * f;
                }
            }
#pragma unroll
            for (int k = 0; k < NG; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += __shfl_sync(0xffffffffu, part[i], k * LG + l);
        }
        __syncwarp();
    }
    if (grp) return;
    const float f = 1.0f / (float)a.page;    // (a power of two)
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 t = __floats2half2_rn(sum[2 * i] * f, sum[2 * i + 1] * f);
        m[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    *reinterpret_cast<uint4 *>(a.mean + ((int64_t)phys * a.n_kv + h) * D + 8 * l) = make_uint4(m[0], m[1], m[2], m[3]);
}

// The codes of eight values in steps of d > 0 (x / d in f32, rounded half away from zero, within +-7)
// as nibbles code + 8, and the values they stand for.  x * (1 / d), off by a few units of the last
// place of 7, rounds as x / d does but next to a half: there the quotient itself is taken.
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], float d, float (&y)[8])
{
    constexpr float kRound = 12582912.f;     // 1.5 * 2^23: sums with it hold whole numbers, in their low bits
    const float inv = __frcp_rn(d);
    uint32_t w = 0;
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fminf(fmaxf(x[i] * inv, -7.f), 7.f), u = t + kRound, n = u - kRound;
        near |= fabsf(t - n) > 0.49999f;
        y[i] = n * d;
        w |= (__float_as_uint(u) & 15u) << (4 * i);
    }
    if (near) {
        w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = fminf(floorf(__fdiv_rn(fabsf(x[i]), d) + 0.5f), 7.f), s = x[i] < 0.f ? -n : n;
            y[i] = s * d;
            w |= ((uint32_t)(int)s & 15u) << (4 * i);
        }
    }
    return w ^ 0x88888888u;
}

__device__ __forceinline__ void load8(float (&x)[8], const float *p)
{
    const float4 u = *reinterpret_cast<const float4 *>(p), v = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}

// N q heads, from `head` on, by a group of lanes.  A lane takes the same four pairs of each (or, past the
// rotated width, eight channels): their angles are read once, and nothing twice.
template <int D, int N>
__device__ __forceinline__ void append_q(const AppendArgs &a, int r, int head)
{
    constexpr int L = D / 8;
    const int l = threadIdx.x % L, rh = a.rot >> 1;
    const bool turn = 8 * l < a.rot, apart = turn && a.neox;
    const int c0 = apart ? 4 * l : 8 * l, c1 = apart ? c0 + rh : c0 + 4;
    const float *src = a.q + r * a.q_stride + head * D;
    float4 x[N], z[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i == 0 || head + i < a.n_q) {
            x[i] = *reinterpret_cast<const float4 *>(src + i * D + c0);
            z[i] = *reinterpret_cast<const float4 *>(src + i * D + c1);
        }
    int p, phys;
    const int refused = locate(a, r, p, phys);
    // (the angles are asked for beside the table entry: their address does not depend on it)
    const float4 *cs = reinterpret_cast<const float4 *>(a.cs + (int64_t)min(max(p, 0), a.max_pos - 1) * rh +
                                                        (turn ? 4 * l : 0));
    float4 u, w;                             // (cos, sin) of two pairs each
    if (turn) {
        u = cs[0];
        w = cs[1];
    }
    if (refused) {
        if (refused > 0 && head == 0 && l == 0) dl_status_or(a.status, refused);
        return;
    }
    float *dst = a.q_out + r * a.q_out_stride + head * D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i && head + i >= a.n_q) break;
        float4 s = x[i], t = z[i];
        if (a.bias) {
            const float4 bs = *reinterpret_cast<const float4 *>(a.bias + (head + i) * D + c0);
            const float4 bt = *reinterpret_cast<const float4 *>(a.bias + (head + i) * D + c1);
            s.x += bs.x; s.y += bs.y; s.z += bs.z; s.w += bs.w;
            t.x += bt.x; t.y += bt.y; t.z += bt.z; t.w += bt.w;
        }
        float4 o = s, m = t;
        if (apart) {
            o.x = fmaf(s.x, u.x, -t.x * u.y); m.x = fmaf(s.x, u.y, t.x * u.x);
            o.y = fmaf(s.y, u.z, -t.y * u.w); m.y = fmaf(s.y, u.w, t.y * u.z);
            o.z = fmaf(s.z, w.x, -t.z * w.y); m.z = fmaf(s.z, w.y, t.z * w.x);
            o.w = fmaf(s.w, w.z, -t.w * w.w); m.w = fmaf(s.w, w.w, t.w * w.z);
        } else if (turn) {
            o.x = fmaf(s.x, u.x, -s.y * u.y); o.y = fmaf(s.x, u.y, s.y * u.x);
            o.z = fmaf(s.z, u.z, -s.w * u.w); o.w = fmaf(s.z, u.w, s.w * u.z);
            m.x = fmaf(t.x, w.x, -t.y * w.y); m.y = fmaf(t.x, w.y, t.y * w.x);
            m.z = fmaf(t.z, w.z, -t.w * w.w); m.w = fmaf(t.z, w.w, t.w * w.z);
        }
        *reinterpret_cast<float4 *>(dst + i * D + c0) = o;
        *reinterpret_cast<float4 *>(dst + i * D + c1) = m;
    }
}

// Eight channels of a k or v head by a lane, encoded into slot `slot` of page `phys`.
template <int D, bool VEC>
__device__ __forceinline__ void store_kv(const AppendArgs &a, int r, int h, bool isv, int phys, int slot, float (&x)[8])
{
    const int l = threadIdx.x % (D / 8), c0 = 8 * l, s = slot % dlp::kCell;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -65504.f), 65504.f);
        m = fmaxf(m, fabsf(x[i]));
    }
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
    m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
    // the scale that is stored is the one the codes are counted in
    const __half dh = __float2half_rn(__fdiv_rn(m, 7.0f));
    const float d = __half2float(dh);
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint32_t w = d > 0.f ? encode8(x, d, y) : 0x88888888u;
    uint8_t *cell = a.pool +
                    (((int64_t)phys * a.n_kv + h) * (a.page / dlp::kCell) + slot / dlp::kCell) * dlp::cell_bytes(D);
    if (isv) {
        *reinterpret_cast<uint16_t *>(cell + dlp::v_half_off(D, s, c0)) = (uint16_t)w;
        *reinterpret_cast<uint16_t *>(cell + dlp::v_half_off(D, s, c0 + 4)) = (uint16_t)(w >> 16);
    } else {
        *reinterpret_cast<uint32_t *>(cell + dlp::k_word_off(D, s, c0)) = w;
    }
    if ((l & 3) == 0)
        reinterpret_cast<__half *>(cell + (isv ? dlp::v_scale_off(D) : dlp::k_scale_off(D)))[s * (D / 32) + l / 4] = dh;
    float *out = isv ? a.v_out : a.k_out;
    if (out) {
        out += r * (isv ? a.v_out_stride : a.k_out_stride) + h * D + c0;
        if constexpr (VEC) {
            *reinterpret_cast<float4 *>(out) = make_float4(y[0], y[1], y[2], y[3]);
            *reinterpret_cast<float4 *>(out + 4) = make_float4(y[4], y[5], y[6], y[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) out[i] = y[i];
        }
    }
}

// k or v head `head` (of the 2 n_kv: k, then v) of row r by a group of lanes; true for the lanes of a k head
// that fills its page.  16-byte accesses; the rotary pairs of a lane's channels are all in the lane
// (interleaved) or in one other lane (NeoX).
template <int D>
__device__ __forceinline__ bool append_kv(const AppendArgs &a, int r, int head, int &phys)
{
    const int l = threadIdx.x % (D / 8), c0 = 8 * l, rh = a.rot >> 1;
    const bool isv = head >= a.n_kv, turn = !isv && c0 < a.rot, apart = turn && a.neox, first = c0 < rh;
    const int h = isv ? head - a.n_kv : head;
    const int cz = !apart ? c0 : first ? c0 + rh : c0 - rh;       // the other channels of the lane's pairs
    const float *src = (isv ? a.v + r * a.v_stride : a.k + r * a.k_stride) + h * D;
    float x[8], z[8];
    load8(x, src + c0);
    int p;
    const int refused = locate(a, r, p, phys);
    // (the angles are asked for beside the table entry: their address does not depend on it)
    const float4 *t = reinterpret_cast<const float4 *>(a.cs + (int64_t)min(max(p, 0), a.max_pos - 1) * rh +
                                                       (apart ? min(c0, cz) : turn ? c0 / 2 : 0));
    float4 angle[4];
    if (turn) {
        angle[0] = t[0];
        angle[1] = t[1];
        if (apart) {
            angle[2] = t[2];
            angle[3] = t[3];
        }
    }
    if (refused) return false;               // (the lanes of q report it)
    if (apart) load8(z, src + cz);           // (another lane has asked for them: they come from L1)
    if (a.bias) {
        const float *b = a.bias + (int64_t)(a.n_q + head) * D;
        float u[8];
        load8(u, b + c0);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += u[i];
        if (apart) {
            load8(u, b + cz);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] += u[i];
        }
    }
    if (apart) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {        // (cos, sin) of two pairs: x cos - z sin, or z sin + x cos
            const float4 u = angle[i];
            const int e = 2 * i, o = e + 1;
            x[e] = fmaf(first ? x[e] : z[e], first ? u.x : u.y, (first ? z[e] : x[e]) * (first ? -u.y : u.x));
            x[o] = fmaf(first ? x[o] : z[o], first ? u.z : u.w, (first ? z[o] : x[o]) * (first ? -u.w : u.z));
        }
    } else if (turn) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 u = angle[i];
            const float x0 = x[4 * i], x1 = x[4 * i + 1], x2 = x[4 * i + 2], x3 = x[4 * i + 3];
            x[4 * i] = fmaf(x0, u.x, -x1 * u.y);
            x[4 * i + 1] = fmaf(x0, u.y, x1 * u.x);
            x[4 * i + 2] = fmaf(x2, u.z, -x3 * u.w);
            x[4 * i + 3] = fmaf(x2, u.w, x3 * u.z);
        }
    }
    const int slot = p & (a.page - 1);
    store_kv<D, true>(a, r, h, isv, phys, slot, x);
    return !isv && slot == a.page - 1;       // this key fills its page
}

// One head of row r by a group of lanes, whatever its alignment; true for the lanes of a k head that
// fills its page.
template <int D>
__device__ __forceinline__ bool append_head(const AppendArgs &a, int r, int head, int &phys)
{
    constexpr int L = D / 8;                 // lanes of a head
    const int l = threadIdx.x % L, c0 = 8 * l;
    const unsigned lanes = ((1u << L) - 1u) << ((threadIdx.x & 31) / L * L);
    const bool isq = head < a.n_q, isv = head >= a.n_q + a.n_kv;
    const int h = isq ? head : head - a.n_q - (isv ? a.n_kv : 0);
    const float *src = (isq ? a.q + r * a.q_stride : isv ? a.v + r * a.v_stride : a.k + r * a.k_stride) + h * D;
    const float *b = a.bias ? a.bias + head * D : nullptr;
    int p;
    const int refused = locate(a, r, p, phys);
    if (refused) {
        if (refused > 0 && head == 0 && l == 0) dl_status_or(a.status, refused);
        return false;
    }
    const float2 *cs = a.cs + (int64_t)p * (a.rot >> 1);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = isv ? src[c0 + i] + (b ? b[c0 + i] : 0.f) : rotated(a, src, b, c0 + i, cs);
    if (isq) {
        __syncwarp(lanes);                   // q may be rotated in place: every lane has read its pairs
        float *dst = a.q_out + r * a.q_out_stride + h * D + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = x[i];
        return false;
    }
    const int slot = p & (a.page - 1);
    store_kv<D, false>(a, r, h, isv, phys, slot, x);
    return !isv && slot == a.page - 1;       // this key fills its page
}

// Grid: (row, set of blockDim.x / (D/8) groups of lanes).  A group takes N q heads, or a k or v head; N = 0:
// a head, without 16-byte accesses.  MEAN: no two rows of the call write one page, so that a CTA that stores
// a page's last key finds the others stored and takes the mean itself.
template <int D, int N, bool MEAN>
__global__ void __launch_bounds__(256, MEAN ? 4 : 5) paged_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int L = D / 8;
    dl_pdl_wait();
    dl_pdl_launch_dependents();
    const int group = (int)((blockIdx.y * blockDim.x + threadIdx.x) / L), r = (int)blockIdx.x;
    int phys = 0, head;                      // of the k and v heads, if it is one
    bool full = false;
    if constexpr (N > 0) {
        head = group - (a.n_q + N - 1) / N;
        if (head < 0) append_q<D, N>(a, r, group * N);
        else if (head < 2 * a.n_kv) full = append_kv<D>(a, r, head, phys);
    } else {
        head = group - a.n_q;
        if (head < 2 * a.n_kv) full = append_head<D>(a, r, group, phys);
    }
    if constexpr (MEAN) {
        __shared__ __align__(16) unsigned char s_stage[8][4 * 9 * D];
        __shared__ int s_full[256 / L][2];   // (page, KV head) of each group of lanes that fills one
        if (threadIdx.x % L == 0) {
            s_full[threadIdx.x / L][0] = full ? phys : -1;
            s_full[threadIdx.x / L][1] = head;
        }
        if (!__syncthreads_or(full)) return;
        const int warp = threadIdx.x >> 5;
        for (int i = warp; i < (int)blockDim.x / L; i += blockDim.x >> 5)
            if (s_full[i][0] >= 0) store_mean<D>(a, s_full[i][0], s_full[i][1], s_stage[warp]);
    }
}

// Mean keys of the pages that the launch before filled, each by a CTA of 256 threads: a thread takes two
// channels of a cell, the cells' sums pass through shared memory to be added in their order.  (A page and
// head by a warp, eight channels a lane, cost 3 to 8 us more: 96 rows 7.2 us instead of 4.6.)  Grid: (sets
// of `per` rows, KV heads); the rows that wrote a page's last key are found before the wait: the launch before
// is this call's store, which lets this one start only after its own wait, so that whatever wrote positions,
// sequences and tables has finished, and it writes none of them itself.
template <int D>
__global__ void __launch_bounds__(256) paged_mean_kernel(const __grid_constant__ AppendArgs a, int per)
{
    constexpr int P = D / 2, NC = 256 / P;   // threads of a cell, cells at a time
    __shared__ float2 s_part[NC][P];
    const int tid = threadIdx.x, lane = tid & 31, r = (int)blockIdx.x * per + lane;
    int p = 0, phys = 0;
    const bool full = lane < per && r < a.rows && locate(a, r, p, phys) == 0 && (p & (a.page - 1)) == a.page - 1;
    unsigned todo = __ballot_sync(0xffffffffu, full);
    dl_pdl_wait();
    dl_pdl_launch_dependents();
    const int e = tid % P, c = tid / P, shift = 8 * (e & 3), n_cells = a.page / dlp::kCell;
    for (; todo; todo &= todo - 1) {
        const int pg = __shfl_sync(0xffffffffu, phys, __ffs(todo) - 1);
        for (int h = (int)blockIdx.y; h < a.n_kv; h += (int)gridDim.y) {
            const uint8_t *cells = a.pool + ((int64_t)pg * a.n_kv + h) * n_cells * dlp::cell_bytes(D);
            float2 sum = make_float2(0.f, 0.f);
            for (int c0 = 0; c0 < n_cells; c0 += NC) {
                float2 part = make_float2(0.f, 0.f);
                if (c0 + c < n_cells) {
                    const uint8_t *cell = cells + (int64_t)(c0 + c) * dlp::cell_bytes(D);
                    uint32_t w[dlp::kCell];
                    unsigned short f[dlp::kCell];
#pragma unroll
                    for (int t = 0; t < dlp::kCell; ++t) {
                        w[t] = __ldcg(reinterpret_cast<const uint32_t *>(cell + dlp::k_word_off(D, t, e / 4 * 8)));
                        f[t] = __ldcg(reinterpret_cast<const unsigned short *>(cell + dlp::k_scale_off(D)) +
                                      t * (D / 32) + e / 16);
                    }
#pragma unroll
                    for (int t = 0; t < dlp::kCell; ++t) {
                        const uint32_t u = w[t] >> shift;
                        const float d = __half2float(__ushort_as_half(f[t]));
                        part.x += (float)((int)(u & 15u) - 8) * d;
                        part.y += (float)((int)((u >> 4) & 15u) - 8) * d;
                    }
                }
                s_part[c][e] = part;
                __syncthreads();
                if (c == 0)
                    for (int k = 0; k < min(NC, n_cells - c0); ++k) {
                        sum.x += s_part[k][e].x;
                        sum.y += s_part[k][e].y;
                    }
                __syncthreads();
            }
            const float f = 1.0f / (float)a.page;    // (a power of two)
            if (c == 0)
                *reinterpret_cast<__half2 *>(a.mean + ((int64_t)pg * a.n_kv + h) * D + 2 * e) =
                    __floats2half2_rn(sum.x * f, sum.y * f);
        }
    }
}

// q heads of a group of lanes: with one, a prompt of 4099 rows (heads of 128, bias) takes 63 us, with two 44,
// with four (64 registers) 44; 96 rows 4.6 with two, 5.7 with four.
constexpr int kHeads = 2;

template <int D>
int launch_append(const AppendArgs &a, cudaStream_t st)
{
    // the groups of a row over equal sets of at most 256 threads
    const int64_t groups = (a.vec ? dl::ceil_div(a.n_q, kHeads) : a.n_q) + 2 * (int64_t)a.n_kv;
    const int64_t lanes = groups * (D / 8), sets = dl::ceil_div(lanes, 256);
    if (sets > 65535)
        return dl::fail(DL_E_SHAPE, "dl_paged_append: n_q=%d n_kv=%d pass the grid", a.n_q, a.n_kv);
    const unsigned threads = (unsigned)(dl::ceil_div(dl::ceil_div(lanes, sets), 32) * 32);
    const bool mean = a.mean && a.own_pages;
    void (*kern)(AppendArgs) = a.vec ? (mean ? paged_append_kernel<D, kHeads, true> : paged_append_kernel<D, kHeads, false>)
                                     : (mean ? paged_append_kernel<D, 0, true> : paged_append_kernel<D, 0, false>);
    int rc = dl::launch_pdl(kern, dim3((unsigned)a.rows, (unsigned)sets), dim3(threads), 0, st,
                            "dl_paged_append: launch", a);
    if (rc != DL_OK || !a.mean || mean) return rc;
    // about two CTAs an SM, of at most a warp's rows
    int sms = 0;
    if ((rc = dl::device_sm_count(&sms)) != DL_OK) return rc;
    const int64_t most = dl::ceil_div((int64_t)a.rows * a.n_kv, (int64_t)2 * sms);
    const int per = (int)(most < 32 ? most : 32);
    const dim3 grid((unsigned)dl::ceil_div(a.rows, per), (unsigned)(a.n_kv < 65535 ? a.n_kv : 65535));
    return dl::launch_pdl(paged_mean_kernel<D>, grid, dim3(256), 0, st, "dl_paged_append: mean launch", a, per);
}

}  // namespace

extern "C" {

int dl_paged_kv_bytes(int n_pages, int page, int n_kv, int head_dim, size_t *pool_bytes, size_t *mean_bytes)
{
    dl::clear_error();
    if (n_pages <= 0 || n_kv <= 0 || !pool_bytes || !mean_bytes)
        return dl::fail(DL_E_ARG, "dl_paged_kv_bytes: n_pages=%d n_kv=%d", n_pages, n_kv);
    if (!dlp::page_ok(page) || (head_dim != 64 && head_dim != 128))
        return dl::fail(DL_E_SHAPE, "dl_paged_kv_bytes: page=%d head_dim=%d", page, head_dim);
    *pool_bytes = (size_t)n_pages * n_kv * (page / dlp::kCell) * dlp::cell_bytes(head_dim);
    *mean_bytes = (size_t)n_pages * n_kv * head_dim * 2;
    return DL_OK;
}

int dl_paged_append(const float *q, int64_t q_stride, const float *k, int64_t k_stride,
                    const float *v, int64_t v_stride, const float *bias, const int32_t *pos,
                    const int32_t *row_seq, int rows, int n_q, const dl_block_tables *tables,
                    const dl_rope *rope, const dl_paged_kv *kv, float *q_out, int64_t q_out_stride,
                    float *k_out, int64_t k_out_stride, float *v_out, int64_t v_out_stride,
                    int32_t *status, dl_stream_t stream)
{
    dl::clear_error();
    if ((rows != 0 && (!q || !k || !v || !pos)) || !rope || (!rope->cos_sin && rope->rot_dim > 0))
        return dl::fail(DL_E_ARG, "dl_paged_append: null pointer");
    int rc = dlp::check_cache("dl_paged_append", kv, tables, n_q, false);
    if (rc != DL_OK) return rc;
    const int D = kv->head_dim;
    if (rows < 0) return dl::fail(DL_E_ARG, "dl_paged_append: rows=%d", rows);
    if (!row_seq && rows > tables->n_seqs)
        return dl::fail(DL_E_ARG, "dl_paged_append: %d rows of %d sequences want row_seq", rows, tables->n_seqs);
    if (rope->rot_dim < 0 || rope->rot_dim % 2 != 0 || rope->rot_dim > D || rope->max_pos <= 0)
        return dl::fail(DL_E_SHAPE, "dl_paged_append: rot_dim=%d head_dim=%d", rope->rot_dim, D);
    const int64_t qw = (int64_t)n_q * D, kw = (int64_t)kv->n_kv * D;
    if (q_stride < qw || k_stride < kw || v_stride < kw || (q_out && q_out_stride < qw) ||
        (k_out && k_out_stride < kw) || (v_out && v_out_stride < kw))
        return dl::fail(DL_E_ARG, "dl_paged_append: strides below the row widths");
    if ((k_out && k_out == k) || (v_out && v_out == v))
        return dl::fail(DL_E_ARG, "dl_paged_append: only q may be its own output");
    if (q_out == q && q_out && q_out_stride != q_stride)
        return dl::fail(DL_E_ARG, "dl_paged_append: q rotated in place has one stride");
    if (rows == 0) return DL_OK;

    AppendArgs a{};
    a.q = q; a.k = k; a.v = v; a.bias = bias;
    a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.pos = pos; a.row_seq = row_seq; a.tables = tables->pages;
    a.table_stride = tables->stride; a.n_seqs = tables->n_seqs; a.width = tables->width;
    a.cs = reinterpret_cast<const float2 *>(rope->cos_sin);
    a.pool = static_cast<uint8_t *>(kv->pool);
    a.mean = static_cast<__half *>(kv->k_mean);
    a.q_out = q_out ? q_out : const_cast<float *>(q);
    a.q_out_stride = q_out ? q_out_stride : q_stride;
    a.k_out = k_out; a.k_out_stride = k_out_stride;
    a.v_out = v_out; a.v_out_stride = v_out_stride;
    a.status = status;
    a.rows = rows; a.n_q = n_q; a.n_kv = kv->n_kv; a.page = kv->page; a.n_pages = kv->n_pages;
    while ((1 << a.page_shift) < kv->page) ++a.page_shift;
    a.rot = rope->rot_dim; a.neox = rope->neox ? 1 : 0; a.max_pos = rope->max_pos;
    a.own_pages = rows == 1 || !row_seq;
    auto vec = [](const void *ptr, int64_t stride) { return dl::aligned16(ptr) && stride % 4 == 0; };
    const int unit = a.neox ? 16 : 8;        // a lane's pairs lie in it or in one other lane
    a.vec = vec(q, q_stride) && vec(k, k_stride) && vec(v, v_stride) && vec(a.q_out, a.q_out_stride) &&
            vec(k_out, k_out_stride) && vec(v_out, v_out_stride) && vec(bias, 0) && vec(a.cs, 0) && a.rot % unit == 0;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return D == 128 ? launch_append<128>(a, st) : launch_append<64>(a, st);
}

}  // extern "C"
