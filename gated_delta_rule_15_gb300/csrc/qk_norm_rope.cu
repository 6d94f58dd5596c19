// qk_norm_rope.cu -- norm of every query and key head and the rotation by its position, in
// one pass over q and k, and the gradients (declared in include/dr.h).
//
// Per row x of d values, with weights w (1 without), n = d (RMS) or 1 (L2):
//     r = 1 / sqrt(sum x^2 / n + eps)   (1 without a norm),   y = w x r,
//     the pairs (y_a, y_b) of the first rot values are rotated by pos * f_i and scaled by c.
// Gradient, with u the output gradient rotated back (and scaled by c) and g = w u:
//     dx = r g - x r^3 (g . x) / n,    dw = sum over rows of u x r.
//
// Angles: f_i enters as turns per position in units of 2^-64 turns (dr_rope_table), so the
// 64-bit product with the position wraps to the exact fraction of a turn of the table's frequency,
// however far the position; its upper 32 bits go to sincospi in fp32, which keeps 2^-26 of a turn (1e-7
// rad).  The table's own 53 bits add at most |position| f_i 2^-52.6 turns.
//
// Both directions stream q and k once and are bound by HBM bandwidth.  A row is held by
// d / 8 lanes with 8 values each, so a warp's accesses are whole rows; a group of lanes takes
// one token and runs over its heads, so that sines and cosines are computed once for all of
// them.  A pair's other half sits in the same lane (interleaved) or rot / 16 lanes away
// (half): its raw values come by shuffle.
// Measured, bf16, 16 + 16 heads of 128, half layout, RMS: forward of 32768 rows 95 us (537 MB, 83 % of
// the copy bandwidth; 197 us while every row read its weights again and formed sine, sign and
// weight apart), gradient of 16384 rows 88 us (403 MB, 67 %; 54 % while a thread kept the weight
// gradients of both kinds).  The gradient is bound by issue (67 %): two shuffle trees and the
// rotation, norm and weight sums on 8 values a lane.
#include <math.h>

#include <array>

#include "../../include/dr.h"
#include "common.cuh"
#include "rope.cuh"
#include "spans.h"

namespace dr {
namespace {

struct RopeArgs {
    const void *x[2];        // q, k: rows of `stride` elements per token, heads d apart
    const void *dy[2];       // (gradient) of the outputs, contiguous
    void *y[2];              // outputs, or gradients of x
    int64_t stride[2], out_stride[2];
    const float *w[2];
    const uint64_t *table;
    const int64_t *pos;
    int64_t n_tok, seq_len, pos0;
    int heads[2], rot, groups;   // groups: runs of heads a token's rows are split into
    int blocks[2];           // (gradient) blocks of q, of k
    float eps, scale;
    float *partial;          // (gradient) [d][blocks of q], [d][blocks of k] partial weight gradients, or NULL
};

// A group of lanes' unit of work: a token and a run of its q and k heads (numbered behind one
// another).  Of each kind s (q, k) every row is
//     y_e = r (A_e x_e + B_e x_e'),    A = w cos, B = +- w' sin
// (x' the pair's other value), so weights, sines and signs are folded once a token.  Shuffles are
// by whole warps: its groups make as many turns as the longest, the rest of them on no row.
template <int D, bool HALF, typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3)
qk_rope_kernel(const RopeArgs a, int norm) {
    constexpr int LPR = D / 8, U = 4;
    const int lane = threadIdx.x & 31, l = lane % LPR, src = partner<HALF>(a, lane, l), lp = l + src - lane;
    const bool rotated = 8 * l < a.rot;
    const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LPR;
    const int64_t tok = unit / a.groups;
    const int g = (int)(unit % a.groups), all = a.heads[0] + a.heads[1];
    const bool live = tok < a.n_tok;
    const int64_t pos = !live ? 0 : a.pos ? a.pos[tok] : a.pos0 + tok % a.seq_len;
    float co[8], si[8];
    angles<HALF>(a, pos, l, false, co, si);
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
        const int first = s ? a.heads[0] : 0, last = s ? all : a.heads[0];
        const int h0 = max((int)((int64_t)all * g / a.groups), first), h1 = min((int)((int64_t)all * (g + 1) / a.groups), last);
        const int rows = live && h1 > h0 ? h1 - h0 : 0, most = __reduce_max_sync(0xffffffffu, rows);
        if (most == 0) continue;
        const float *w = a.w[s];
        float A[8], B[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            A[e] = co[e] * (w ? __ldg(w + 8 * l + e) : 1.f);
            B[e] = si[e] * (w ? __ldg(w + (HALF ? 8 * lp + e : 8 * l + (e ^ 1))) : 1.f);
        }
        const T *x0 = (const T *)a.x[s] + tok * a.stride[s] + (int64_t)(h0 - first) * D + 8 * l;
        T *y0 = (T *)a.y[s] + tok * a.out_stride[s] + (int64_t)(h0 - first) * D + 8 * l;
#pragma unroll 1
        for (int i = 0; i < most; i += U) {
            Vec8<T> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u] = i + u < rows ? ld8(x0 + (int64_t)(i + u) * D) : Vec8<T>{};
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
                    x[e] = r * y;
                }
                if (i + u < rows) st8(y0 + (int64_t)(i + u) * D, x);
            }
        }
    }
}

// Gradient: a block takes rows of one kind (q or k), its groups of lanes run over the tokens, the
// weight gradients of a lane's 8 values in registers, summed over the block at the end (a
// fixed order: no atomics).  The next row is loaded while one is worked on.
template <int D, bool HALF, typename T>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2)
qk_rope_bwd_kernel(const RopeArgs a, int norm) {
    constexpr int LPR = D / 8, RPB = 256 / LPR;
    const int lane = threadIdx.x & 31, l = lane % LPR, src = partner<HALF>(a, lane, l);
    const bool rotated = 8 * l < a.rot;
    const int s = (int)blockIdx.x >= a.blocks[0], blocks = a.blocks[s], block = (int)blockIdx.x - s * a.blocks[0], heads = a.heads[s];
    const int groups = a.groups < heads ? a.groups : heads;   // runs of heads a token's rows are split into
    const int64_t units = a.n_tok * groups;
    float dw[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        dw[e] = 0.f;
        w[e] = a.w[s] ? a.w[s][8 * l + e] : 1.f;
    }
#pragma unroll 1
    for (int64_t u0 = (int64_t)block * RPB; u0 < units; u0 += (int64_t)blocks * RPB) {
        const int64_t unit = u0 + threadIdx.x / LPR, tok = unit / groups;
        const bool live = unit < units;
        const int g = (int)(unit % groups);
        const int64_t pos = !live ? 0 : a.pos ? a.pos[tok] : a.pos0 + tok % a.seq_len;
        const int h0 = (int)((int64_t)heads * g / groups), h1 = (int)((int64_t)heads * (g + 1) / groups);
        const int rows = live ? h1 - h0 : 0, most = __reduce_max_sync(0xffffffffu, rows);
        const int64_t row = (int64_t)h0 * D + 8 * l;
        const T *x0 = (const T *)a.x[s] + tok * a.stride[s] + row, *d0 = (const T *)a.dy[s] + tok * (int64_t)heads * D + row;
        T *y0 = (T *)a.y[s] + tok * a.out_stride[s] + row;
        Vec8<T> nx{}, nd{};
        if (rows > 0) {
            nx = ld8(x0);
            nd = ld8(d0);
        }
        float co[8], si[8];
        angles<HALF>(a, pos, l, true, co, si);
#pragma unroll 1
        for (int i = 0; i < most; ++i) {
            const Vec8<T> vx = nx, vd = nd;
            if (i + 1 < rows) {
                nx = ld8(x0 + (int64_t)(i + 1) * D);
                nd = ld8(d0 + (int64_t)(i + 1) * D);
            } else {
                nx = nd = Vec8<T>{};
            }
            float x[8], u[8], o[8];
            unpack(vx, x);
            unpack(vd, u);
            others<HALF>(vd, u, src, o);
            float r = 1.f, gx = 0.f, ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(x[e], x[e], ss);
                u[e] *= co[e];   // rotated back
                if (rotated) u[e] = fmaf(si[e], o[e], u[e]);
                o[e] = u[e] * x[e];
                u[e] *= w[e];
                gx = fmaf(o[e], w[e], gx);
            }
            if (norm != DR_NORM_NONE) {
#pragma unroll
                for (int k = 1; k < LPR; k <<= 1) {   // both sums of the row side by side
                    ss += __shfl_xor_sync(0xffffffffu, ss, k);
                    gx += __shfl_xor_sync(0xffffffffu, gx, k);
                }
                r = rsqrtf(norm == DR_NORM_RMS ? fmaf(ss, 1.f / D, a.eps) : ss + a.eps);
                const float f = -r * r * gx * (norm == DR_NORM_RMS ? 1.f / D : 1.f);
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] = r * fmaf(x[e], f, u[e]);
            }
            if (i < rows) {   // a turn on no row has sums of 0, and r is infinite there without eps
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[e] = fmaf(o[e], r, dw[e]);
                st8(y0 + (int64_t)i * D, u);
            }
        }
    }
    if (!a.partial) return;
    __shared__ float sum[RPB][D];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[threadIdx.x / LPR][8 * l + e] = dw[e];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 256) {
        float t = 0.f;
        for (int k = 0; k < RPB; ++k) t += sum[k][c];
        a.partial[((size_t)s * a.blocks[0] * D) + (size_t)c * blocks + block] = t;
    }
}

// dw[s][c] = sum of the blocks' partial sums, in a fixed order: one warp per value.
__global__ void __launch_bounds__(256)
rope_weight_sum_kernel(const float *__restrict__ partial, int blocks_q, int blocks_k, int d, float *__restrict__ dwq,
                       float *__restrict__ dwk) {
    const int c = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;   // of 2 d
    if (c >= 2 * d) return;
    const bool k = c >= d;
    const int blocks = k ? blocks_k : blocks_q;
    const float *p = partial + (k ? (size_t)blocks_q * d + (size_t)(c - d) * blocks : (size_t)c * blocks);
    float t = 0.f;
    for (int b = lane; b < blocks; b += 32) t += p[b];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    float *dst = k ? dwk : dwq;
    if (lane == 0 && dst) dst[k ? c - d : c] = t;
}

constexpr int kGradBlocks = 456;   // three per SM, of q and k together

template <int D, typename T>
int launch_fwd(const RopeArgs &a, int norm, bool half, cudaStream_t s) {
    const int64_t threads = a.n_tok * a.groups * (D / 8);
    const unsigned blocks = (unsigned)((threads + 255) / 256);
    if (half) qk_rope_kernel<D, true, T><<<blocks, 256, 0, s>>>(a, norm);
    else qk_rope_kernel<D, false, T><<<blocks, 256, 0, s>>>(a, norm);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}
template <int D, typename T>
int launch_bwd(const RopeArgs &a, int norm, bool half, float *dwq, float *dwk, cudaStream_t s) {
    const int blocks = a.blocks[0] + a.blocks[1];
    if (half) qk_rope_bwd_kernel<D, true, T><<<blocks, 256, 0, s>>>(a, norm);
    else qk_rope_bwd_kernel<D, false, T><<<blocks, 256, 0, s>>>(a, norm);
    if (cudaGetLastError() != cudaSuccess) return kErrCuda;
    if (!a.partial) return kOk;
    rope_weight_sum_kernel<<<(2 * D + 7) / 8, 256, 0, s>>>(a.partial, a.blocks[0], a.blocks[1], D, dwq, dwk);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

int check_desc(const dr_qk_norm_rope_desc *d) {
    if (!d) return kErrInvalid;
    if (d->n_tok < 0 || d->Hq < 1 || d->Hk < 0 || d->d < 1 || d->rot < 0 || d->rot > d->d || d->seq_len < 0)
        return kErrInvalid;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return kErrInvalid;
    if (d->norm < DR_NORM_NONE || d->norm > DR_NORM_RMS || d->layout < DR_ROPE_HALF || d->layout > DR_ROPE_INTERLEAVED)
        return kErrInvalid;
    if (!(d->eps >= 0.f) || !(d->rot_scale == d->rot_scale) || d->reserved != 0) return kErrInvalid;
    if (d->d != 64 && d->d != 128 && d->d != 256) return kErrUnsupported;
    if (d->rot % 16 != 0) return kErrUnsupported;
    if (d->Hq > (1 << 16) || d->Hk > (1 << 16) || d->n_tok > ((int64_t)1 << 31)) return kErrUnsupported;
    const int64_t unit = d->dtype == DR_BF16 ? 8 : 4;   // rows start on 16-byte boundaries
    const int64_t strides[4] = {d->q_stride, d->q_out_stride, d->k_stride, d->k_out_stride};
    for (int i = 0; i < 4; ++i) {
        if (strides[i] == 0) continue;
        if (strides[i] < (i < 2 ? d->Hq : d->Hk) * d->d || strides[i] % unit != 0) return kErrInvalid;
        if (strides[i] > ((int64_t)1 << 31)) return kErrUnsupported;
    }
    return kOk;
}

// Runs of heads a token's rows are split into: one while the tokens alone give every SM its
// 2048 threads (the sines are then computed once a token), more for few tokens.
int head_groups(const dr_qk_norm_rope_desc &d) {
    const int64_t threads = d.n_tok * (d.d / 8), all = d.Hq + d.Hk, want = (int64_t)152 * 2048;
    int64_t g = threads >= want ? 1 : (want + threads - 1) / (threads > 0 ? threads : 1);
    return (int)(g < all ? g : all);
}

RopeArgs common_args(const dr_qk_norm_rope_desc &d, const void *q, const void *k, const float *wq, const float *wk,
                     const uint64_t *table, const int64_t *positions) {
    RopeArgs a{};
    a.x[0] = q; a.x[1] = k;
    a.stride[0] = d.q_stride ? d.q_stride : d.Hq * d.d;
    a.stride[1] = d.k_stride ? d.k_stride : d.Hk * d.d;
    a.out_stride[0] = d.q_out_stride ? d.q_out_stride : d.Hq * d.d;
    a.out_stride[1] = d.k_out_stride ? d.k_out_stride : d.Hk * d.d;
    a.w[0] = wq; a.w[1] = wk;
    a.table = table; a.pos = positions;
    a.n_tok = d.n_tok; a.seq_len = d.seq_len > 0 ? d.seq_len : (d.n_tok > 0 ? d.n_tok : 1); a.pos0 = d.pos0;
    a.heads[0] = (int)d.Hq; a.heads[1] = (int)d.Hk; a.rot = (int)d.rot;
    a.eps = d.eps; a.scale = d.rot_scale;
    a.groups = head_groups(d);
    return a;
}

// Blocks of q and of k: shares of kGradBlocks by their heads, no more than there are units of work.
void grad_blocks(const dr_qk_norm_rope_desc &d, int (&blocks)[2]) {
    const int64_t rpb = 256 / (d.d / 8), heads[2] = {d.Hq, d.Hk}, split = head_groups(d);
    for (int s = 0; s < 2; ++s) {
        const int64_t groups = split < heads[s] ? split : heads[s], need = (d.n_tok * groups + rpb - 1) / rpb;
        int64_t share = kGradBlocks * heads[s] / (d.Hq + d.Hk);
        if (share < 1) share = 1;
        blocks[s] = heads[s] == 0 ? 0 : (int)(need < 1 ? 1 : need < share ? need : share);
    }
}
size_t partial_bytes(const dr_qk_norm_rope_desc &d) {
    int b[2];
    grad_blocks(d, b);
    return sizeof(float) * (size_t)d.d * (b[0] + b[1]);
}

// What every block may read beside its rows.
using Operands = std::array<Block, 4>;
Operands operands(const dr_qk_norm_rope_desc &d, const RopeArgs &a) {
    const size_t w = sizeof(float) * (size_t)d.d;
    return {Block{a.w[0], w}, Block{a.w[1], w}, Block{a.table, sizeof(uint64_t) * (size_t)(d.rot / 2)},
            Block{a.pos, sizeof(int64_t) * (size_t)d.n_tok}};
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" int dr_rope_table(int64_t rot, double base, int32_t scaling, double factor, double original, double low,
                             double high, uint64_t *table) {
    if (!table || rot < 0 || rot > 256 || !(base > 1.0) || !isfinite(base)) return kErrInvalid;
    if (scaling < DR_ROPE_PLAIN || scaling > DR_ROPE_BY_PARTS) return kErrInvalid;
    if (scaling != DR_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return kErrInvalid;
    if (scaling == DR_ROPE_BY_PARTS && (!(original > 0.0) || !(high > low) || !isfinite(original) || !isfinite(low) || !isfinite(high)))
        return kErrInvalid;
    if (rot % 16 != 0) return kErrUnsupported;
    const double two_pi = 6.283185307179586476925286766559;
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * (double)i / (double)rot);   // radians a position
        if (scaling == DR_ROPE_LINEAR) f /= factor;
        if (scaling == DR_ROPE_BY_PARTS) {
            double w = (original * f / two_pi - low) / (high - low);
            w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
            f *= w + (1.0 - w) / factor;
        }
        table[i] = (uint64_t)(f / two_pi * 18446744073709551616.0 + 0.5);   // 2^64; f <= 1, so below 2^62
    }
    return kOk;
}

extern "C" int dr_qk_norm_rope(const dr_qk_norm_rope_desc *desc, const void *q, const void *k, const float *wq,
                               const float *wk, const uint64_t *table, const int64_t *positions, void *q_out, void *k_out,
                               dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_qk_norm_rope_desc &d = *desc;
    if (d.n_tok == 0) return kOk;
    if (!q || !q_out || (d.Hk > 0 && (!k || !k_out)) || (d.rot > 0 && !table)) return kErrInvalid;
    if (d.norm == DR_NORM_NONE && (wq || wk)) return kErrInvalid;
    const void *ptrs[] = {q, k, q_out, k_out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    if (!aligned(wq, 4) || !aligned(wk, 4) || !aligned(table, 8) || !aligned(positions, 8)) return kErrInvalid;
    RopeArgs a = common_args(d, q, k, wq, wk, table, positions);
    a.y[0] = q_out; a.y[1] = k_out;
    // an output is its own input (every row is read before it is written) or meets neither
    // input nor the other output
    const int64_t e = d.dtype == DR_BF16 ? 2 : 4, wide[2] = {d.Hq * d.d, d.Hk * d.d};
    if (meet(Rows{q_out, wide[0], a.out_stride[0]}, Rows{k_out, wide[1], a.out_stride[1]}, d.n_tok, e)) return kErrInvalid;
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 2; ++i) {
            const Rows y{a.y[o], wide[o], a.out_stride[o]}, x{a.x[i], wide[i], a.stride[i]};
            if (meet(y, x, d.n_tok, e) && !(o == i && same(y, x))) return kErrInvalid;
        }
    for (const Block &x : operands(d, a))
        for (int o = 0; o < 2; ++o)
            if (meet({a.y[o], wide[o], a.out_stride[o]}, x, d.n_tok, e)) return kErrInvalid;
    const bool half = d.layout == DR_ROPE_HALF;
    cudaStream_t s = (cudaStream_t)stream;
    using bf = __nv_bfloat16;
    if (d.n_tok * a.groups * (d.d / 8) > (int64_t)256 * 0x7fffffff) return kErrUnsupported;
    if (d.dtype == DR_BF16)
        return d.d == 64 ? launch_fwd<64, bf>(a, d.norm, half, s) : d.d == 128 ? launch_fwd<128, bf>(a, d.norm, half, s)
                                                                               : launch_fwd<256, bf>(a, d.norm, half, s);
    return d.d == 64 ? launch_fwd<64, float>(a, d.norm, half, s) : d.d == 128 ? launch_fwd<128, float>(a, d.norm, half, s)
                                                                              : launch_fwd<256, float>(a, d.norm, half, s);
}

extern "C" int dr_qk_norm_rope_bwd_workspace_bytes(const dr_qk_norm_rope_desc *desc, size_t *bytes) {
    if (!bytes) return kErrInvalid;
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    *bytes = desc->norm == DR_NORM_NONE ? 0 : partial_bytes(*desc);
    return kOk;
}

extern "C" int dr_qk_norm_rope_bwd(const dr_qk_norm_rope_desc *desc, const void *q, const void *k, const float *wq,
                                   const float *wk, const uint64_t *table, const int64_t *positions, const void *dq_out,
                                   const void *dk_out, void *dq, void *dk, float *dwq, float *dwk, void *workspace,
                                   size_t workspace_bytes, dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_qk_norm_rope_desc &d = *desc;
    if (d.n_tok > 0 && (!q || !dq_out || !dq || (d.Hk > 0 && (!k || !dk_out || !dk)) || (d.rot > 0 && !table))) return kErrInvalid;
    if (d.norm == DR_NORM_NONE && (wq || wk)) return kErrInvalid;
    if ((dwq && !wq) || (dwk && !wk)) return kErrInvalid;   // no weights, no gradient of them
    const void *ptrs[] = {q, k, dq_out, dk_out, dq, dk, workspace};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    const void *words[] = {wq, wk, dwq, dwk};
    for (const void *p : words)
        if (!aligned(p, 4)) return kErrInvalid;
    if (!aligned(table, 8) || !aligned(positions, 8)) return kErrInvalid;
    RopeArgs a = common_args(d, q, k, wq, wk, table, positions);
    a.dy[0] = dq_out; a.dy[1] = dk_out;
    a.y[0] = dq; a.y[1] = dk;
    // dq may be q and dk may be k; otherwise no written row meets another or an input's
    const int64_t e = d.dtype == DR_BF16 ? 2 : 4, wide[2] = {d.Hq * d.d, d.Hk * d.d};
    if (meet(Rows{dq, wide[0], a.out_stride[0]}, Rows{dk, wide[1], a.out_stride[1]}, d.n_tok, e)) return kErrInvalid;
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 2; ++i) {
            const Rows y{a.y[o], wide[o], a.out_stride[o]}, x{a.x[i], wide[i], a.stride[i]};
            if (meet(y, x, d.n_tok, e) && !(o == i && same(y, x))) return kErrInvalid;
            if (meet(y, Rows{a.dy[i], wide[i], wide[i]}, d.n_tok, e)) return kErrInvalid;
        }
    const Operands ins = operands(d, a);
    const Block dw[2] = {{dwq, sizeof(float) * (size_t)d.d}, {dwk, sizeof(float) * (size_t)d.d}};
    for (int o = 0; o < 2; ++o) {
        const Rows y{a.y[o], wide[o], a.out_stride[o]};
        for (const Block &x : ins)
            if (meet(y, x, d.n_tok, e)) return kErrInvalid;
        if (meet(y, dw[0], d.n_tok, e) || meet(y, dw[1], d.n_tok, e)) return kErrInvalid;
    }
    if (meet(dw[0], dw[1])) return kErrInvalid;
    const bool weights = dwq || dwk;
    grad_blocks(d, a.blocks);
    if (weights && (!workspace || workspace_bytes < partial_bytes(d))) return kErrWorkspace;
    if (weights) {   // the partial sums meet nothing that is read or written beside them
        const Block ws{workspace, partial_bytes(d)};
        for (int o = 0; o < 2; ++o)
            if (meet({a.y[o], wide[o], a.out_stride[o]}, ws, d.n_tok, e) || meet({a.x[o], wide[o], a.stride[o]}, ws, d.n_tok, e) ||
                meet({a.dy[o], wide[o], wide[o]}, ws, d.n_tok, e) || meet(dw[o], ws))
                return kErrInvalid;
        for (const Block &x : ins)
            if (meet(ws, x)) return kErrInvalid;
    }
    if (d.n_tok == 0 && !weights) return kOk;
    a.partial = weights ? (float *)workspace : nullptr;
    const bool half = d.layout == DR_ROPE_HALF;
    cudaStream_t s = (cudaStream_t)stream;
    using bf = __nv_bfloat16;
    if (d.dtype == DR_BF16)
        return d.d == 64    ? launch_bwd<64, bf>(a, d.norm, half, dwq, dwk, s)
               : d.d == 128 ? launch_bwd<128, bf>(a, d.norm, half, dwq, dwk, s)
                            : launch_bwd<256, bf>(a, d.norm, half, dwq, dwk, s);
    return d.d == 64    ? launch_bwd<64, float>(a, d.norm, half, dwq, dwk, s)
           : d.d == 128 ? launch_bwd<128, float>(a, d.norm, half, dwq, dwk, s)
                        : launch_bwd<256, float>(a, d.norm, half, dwq, dwk, s);
}
