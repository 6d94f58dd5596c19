// kv_append.cu -- new tokens' keys (normalised and rotated) and values into a paged cache, their queries
// normalised and rotated on the way (declared in include/dr.h).  The row's mathematics: qk_norm_rope.cu.
//
// One pass, bound by HBM bandwidth (32768 rows, 19876 of them of a live sequence, H16/4 d128: 244 MB of reads and writes in 51 us,
// 4.8 TB/s; the same with fp32 rows, 16384, 9938 live: 244 MB in 50 us; 64 tokens: 6 us).
// A group of d / 8 lanes takes a token and a run of its heads (queries, keys, values, one behind another), 8 values a
// lane, so a warp's accesses are whole rows.  (Its tokens lie in the grid's x, its run in y: with 64-bit divisions for
// those and for the page the kernel was bound by issue, 70 %.)  A token finds its sequence in the offsets by bisection
// (they stay in L1), its position from the sequence's length before the call, and its page in the table.
#include <math.h>

#include "../../include/dr.h"
#include "common.cuh"
#include "linrec.h"
#include "rope.cuh"
#include "spans.h"

namespace dr {
namespace {

struct AppendArgs {
    const void *x[3];            // q, k, v: rows of `stride` elements a token
    int64_t stride[3], out_stride;
    void *q_out, *cache[2];      // keys, values: [pages][Hk][page][d]
    const float *w[2];
    const uint64_t *table;
    const int *pages;
    const int64_t *cu, *start;
    int64_t n_tok, N, n_pages, max_pages, room;   // room: tokens of a sequence's pages
    int page, Hq, Hk, rot, run, zero_rest;        // run: heads (of queries, keys, values, one behind another) a block takes
    float eps, scale;
};

// The row's sequence and position in it; false for a row of no sequence or of an inactive one.
__device__ __forceinline__ bool place(const AppendArgs &a, int64_t tok, int64_t &n, int64_t &pos) {
    n = tok;
    int64_t first = tok;
    if (a.cu) {
        int64_t lo = 0, hi = a.N - 1;        // the last sequence that begins at or before the row
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            if (__ldg(a.cu + mid) <= tok) lo = mid;
            else hi = mid - 1;
        }
        n = lo;
        first = __ldg(a.cu + n);
        if (first > tok || __ldg(a.cu + n + 1) <= tok) return false;
        first = max(first, (int64_t)0);
    }
    const int64_t s = __ldg(a.start + n);
    pos = (int64_t)((uint64_t)s + (uint64_t)(tok - first));
    return s >= 0 && pos >= 0;       // (a start near 2^63 wraps)
}

template <int D, bool HALF, typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3)
kv_append_kernel(const AppendArgs a, int norm) {
    constexpr int LPR = D / 8, U = 4;
    const int lane = threadIdx.x & 31, l = lane % LPR, src = partner<HALF>(a, lane, l), lp = l + src - lane;
    const bool rotated = 8 * l < a.rot;
    const int64_t tok = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
    const int run0 = blockIdx.y * a.run, run1 = run0 + a.run;      // this block's heads
    const bool there = tok < a.n_tok;
    int64_t n = 0, pos = 0;
    const bool live = there && place(a, tok, n, pos);
    // the token's slot: element of its row in head 0 of the cache, or -1
    int64_t slot = -1;
    if (live && pos < a.room) {
        const int64_t at = pos >> 32 ? pos / a.page : (int64_t)((uint32_t)pos / (uint32_t)a.page);   // (64-bit divisions are long)
        const int64_t pg = __ldg(a.pages + n * a.max_pages + at);
        if (pg >= 0 && pg < a.n_pages) slot = (pg * a.Hk * a.page + (pos - at * a.page)) * D;
    }
    float co[8], si[8];
    angles<HALF>(a, pos, l, false, co, si);
#pragma unroll 1
    for (int s = 0; s < 3; ++s) {
        const int first = s == 0 ? 0 : a.Hq + (s - 1) * a.Hk, last = s == 0 ? a.Hq : first + a.Hk;
        const int h0 = max(run0, first), h1 = min(run1, last);
        const bool mine = s == 0 ? there && (live || a.zero_rest) : slot >= 0;
        const int rows = mine && h1 > h0 ? h1 - h0 : 0, most = __reduce_max_sync(0xffffffffu, rows);
        if (most == 0) continue;
        const T *x0 = (const T *)a.x[s] + tok * a.stride[s] + (int64_t)(h0 - first) * D + 8 * l;
        const int64_t step = s == 0 ? D : (int64_t)a.page * D;
        T *y0 = s == 0 ? (T *)a.q_out + tok * a.out_stride + (int64_t)(h0 - first) * D + 8 * l
                       : (T *)a.cache[s - 1] + slot + (int64_t)(h0 - first) * step + 8 * l;
        float A[8], B[8];
        if (s < 2) {
            const float *w = a.w[s];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                A[e] = co[e] * (w ? __ldg(w + 8 * l + e) : 1.f);
                B[e] = si[e] * (w ? __ldg(w + (HALF ? 8 * lp + e : 8 * l + (e ^ 1))) : 1.f);
            }
        }
#pragma unroll 1
        for (int i = 0; i < most; i += U) {
            Vec8<T> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = i + u < rows && live ? ld8(x0 + (int64_t)(i + u) * D) : Vec8<T>{};
            if (s == 2) {      // values go as they are
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + u < rows) *reinterpret_cast<Vec8<T> *>(y0 + (int64_t)(i + u) * step) = raw[u];
                continue;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[8], o[8];
                unpack(raw[u], x);
                others<HALF>(raw[u], x, src, o);
                float r = 1.f;
                if (norm != DR_NORM_NONE) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
                    ss = row_sum<LPR>(ss);
                    r = rsqrtf(norm == DR_NORM_RMS ? fmaf(ss, 1.f / D, a.eps) : ss + a.eps);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {   // (0 times an infinity would be NaN where there is no pair)
                    float y = A[e] * x[e];
                    if (rotated) y = fmaf(B[e], o[e], y);
                    x[e] = live ? r * y : 0.f;   // (eps 0: a row of no sequence is 0 times infinity)
                }
                if (i + u < rows) st8(y0 + (int64_t)(i + u) * step, x);
            }
        }
    }
}

template <int D, typename T>
int launch(const AppendArgs &a, int norm, bool half, cudaStream_t s) {
    const dim3 blocks((unsigned)((a.n_tok * (D / 8) + 255) / 256), (unsigned)((a.Hq + 2 * a.Hk + a.run - 1) / a.run));
    if (half) kv_append_kernel<D, true, T><<<blocks, 256, 0, s>>>(a, norm);
    else kv_append_kernel<D, false, T><<<blocks, 256, 0, s>>>(a, norm);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

int check_desc(const dr_kv_append_desc *d) {
    if (!d) return kErrInvalid;
    if (d->n_tok < 0 || d->N < 1 || d->Hq < 0 || d->Hk < 1 || d->d < 1 || d->rot < 0 || d->rot > d->d) return kErrInvalid;
    if (d->n_pages < 1 || d->page < 1 || d->max_pages < 1) return kErrInvalid;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return kErrInvalid;
    if (d->norm < DR_NORM_NONE || d->norm > DR_NORM_RMS || d->layout < DR_ROPE_HALF || d->layout > DR_ROPE_INTERLEAVED)
        return kErrInvalid;
    if (!(d->eps >= 0.f) || !(d->rot_scale == d->rot_scale) || d->reserved != 0) return kErrInvalid;
    if (d->zero_rest != 0 && d->zero_rest != 1) return kErrInvalid;
    if ((d->d != 64 && d->d != 128) || d->rot % 16 != 0) return kErrUnsupported;
    if (d->page % 16 != 0 || d->page > 1024) return kErrUnsupported;
    if (d->Hq > (1 << 16) || d->Hk > (1 << 16) || d->n_tok > ((int64_t)1 << 31) || d->N > ((int64_t)1 << 31)) return kErrUnsupported;
    if (d->max_pages > ((int64_t)1 << 31) || d->n_pages > ((int64_t)1 << 31) || d->n_pages * d->Hk > (((int64_t)1 << 31) - 1) / d->page)
        return kErrUnsupported;
    const int64_t unit = d->dtype == DR_BF16 ? 8 : 4;   // rows start on 16-byte boundaries
    const int64_t strides[4] = {d->q_stride, d->q_out_stride, d->k_stride, d->v_stride};
    for (int i = 0; i < 4; ++i) {
        if (strides[i] == 0) continue;
        if (strides[i] < (i < 2 ? d->Hq : d->Hk) * d->d || strides[i] % unit != 0) return kErrInvalid;
        if (strides[i] > ((int64_t)1 << 31)) return kErrUnsupported;
    }
    return kOk;
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" int dr_kv_append(const dr_kv_append_desc *desc, const void *q, const void *k, const void *v, const float *wq,
                            const float *wk, const uint64_t *table, const int32_t *pages, const int64_t *start,
                            const int64_t *cu_seqlens, void *q_out, void *k_cache, void *v_cache, dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_kv_append_desc &d = *desc;
    if (!cu_seqlens && d.n_tok != d.N) return kErrInvalid;   // one row a sequence
    if (d.n_tok == 0) return kOk;
    if ((d.Hq > 0 && (!q || !q_out)) || !k || !v || !k_cache || !v_cache || !pages || !start || (d.rot > 0 && !table)) return kErrInvalid;
    if (d.norm == DR_NORM_NONE && (wq || wk)) return kErrInvalid;
    const void *ptrs[] = {q, k, v, q_out, k_cache, v_cache};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    if (!aligned(wq, 4) || !aligned(wk, 4) || !aligned(pages, 4) || !aligned(table, 8) || !aligned(start, 8) || !aligned(cu_seqlens, 8))
        return kErrInvalid;
    AppendArgs a{};
    const int64_t e = d.dtype == DR_BF16 ? 2 : 4, wide[3] = {d.Hq * d.d, d.Hk * d.d, d.Hk * d.d};
    a.x[0] = d.Hq > 0 ? q : nullptr; a.x[1] = k; a.x[2] = v;
    a.stride[0] = d.q_stride ? d.q_stride : wide[0];
    a.stride[1] = d.k_stride ? d.k_stride : wide[1];
    a.stride[2] = d.v_stride ? d.v_stride : wide[2];
    a.out_stride = d.q_out_stride ? d.q_out_stride : wide[0];
    a.q_out = d.Hq > 0 ? q_out : nullptr; a.cache[0] = k_cache; a.cache[1] = v_cache;
    a.w[0] = wq; a.w[1] = wk; a.table = table; a.pages = pages; a.cu = cu_seqlens; a.start = start;
    a.n_tok = d.n_tok; a.N = d.N; a.n_pages = d.n_pages; a.max_pages = d.max_pages;
    a.page = (int)d.page; a.Hq = (int)d.Hq; a.Hk = (int)d.Hk; a.rot = (int)d.rot; a.zero_rest = d.zero_rest;
    a.eps = d.eps; a.scale = d.rot_scale;
    // Nothing written meets another buffer; q_out may be q (every row is read before it is written).
    const size_t cache = (size_t)(d.n_pages * d.Hk * d.page * d.d * e);
    const Block written[2] = {{k_cache, cache}, {v_cache, cache}};
    const Block read[6] = {{wq, sizeof(float) * (size_t)d.d}, {wk, sizeof(float) * (size_t)d.d}, {table, sizeof(uint64_t) * (size_t)(d.rot / 2)},
                           {pages, sizeof(int32_t) * (size_t)(d.N * d.max_pages)}, {start, sizeof(int64_t) * (size_t)d.N},
                           {cu_seqlens, sizeof(int64_t) * (size_t)(d.N + 1)}};
    const Rows out{a.q_out, wide[0], a.out_stride};
    if (meet(written[0], written[1])) return kErrInvalid;
    for (int i = 0; i < 3; ++i) {
        const Rows x{a.x[i], wide[i], a.stride[i]};
        if (meet(out, x, d.n_tok, e) && !(i == 0 && same(out, x))) return kErrInvalid;
        for (const Block &w : written)
            if (meet(x, w, d.n_tok, e)) return kErrInvalid;
    }
    for (const Block &w : written)
        if (meet(out, w, d.n_tok, e)) return kErrInvalid;
    for (const Block &r : read)
        if (meet(out, r, d.n_tok, e) || meet(written[0], r) || meet(written[1], r)) return kErrInvalid;
    // runs of heads a token's rows are split into: one while the tokens alone give every SM its 2048 threads
    const int64_t threads = d.n_tok * (d.d / 8), all = d.Hq + 2 * d.Hk, want = (int64_t)152 * 2048;
    const int64_t groups = threads >= want ? 1 : (want + threads - 1) / threads;
    a.run = (int)(groups < all ? (all + groups - 1) / groups : 1);
    if (a.run < (all + 65534) / 65535) a.run = (int)((all + 65534) / 65535);      // (the grid's second extent)
    a.room = d.max_pages * d.page;
    const bool half = d.layout == DR_ROPE_HALF;
    cudaStream_t s = (cudaStream_t)stream;
    if (d.dtype == DR_BF16)
        return d.d == 64 ? launch<64, __nv_bfloat16>(a, d.norm, half, s) : launch<128, __nv_bfloat16>(a, d.norm, half, s);
    return d.d == 64 ? launch<64, float>(a, d.norm, half, s) : launch<128, float>(a, d.norm, half, s);
}
