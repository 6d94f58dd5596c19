// linrec_simt.cu -- the additive gated linear recurrence on the CUDA cores: a token
// recurrence in fp32 for every type and width, the log-decay gradient's last step, and the
// single-token step.  The passes and their use for the gradients: linrec.h.
#include "common.cuh"
#include "linrec.h"
#include "umma.cuh"

namespace dr {
namespace {

using umma::fma2;
using umma::mul2;

// ---------------------------------------------------------------- token recurrence
// One CTA per (sequence, head, 64 value columns): four warps, each with the state's 16
// columns in registers.  A thread holds two columns of the rows 16 m + 4 rg + e (rg = lane / 8,
// e < 4), so the key and query rows of a token are read from shared memory as float4s whose
// four addresses per warp lie side by side, two adjacent rows form the operand of one packed
// fma.rn.f32x2, and a column's read-out is a register sum and two shuffles.  Per token and
// element: one multiply (decay), two fused multiply-adds.  Many chains: bound by the packed FP32
// rate, 3 dk dv / 2 instructions a head-token.  Few chains: by one token's latency, 0.14 us (64 x 64) and
// 0.2 us (128 x 128).
// Rows come by asynchronous copies, a tile ahead.
// kGroup tokens' read-outs are summed over the lanes at a time; kTile tokens (kTokenAnchor is a multiple) are staged
// in shared memory, of which 48 KB hold two tiles.  One fp32 chain of 256 tokens of 64 x 64 / 128 x 128, us on
// the GPU, by kTile and kGroup: 8 and 4 48 / 65, 16 and 4 37 / 57, 8 and 8 46 / 57, 16 and 8 37 / 50.
constexpr int kGroup = 8;
template <typename Tin, int DK, bool DOT> constexpr int kTileOf = DK == 128 && sizeof(Tin) == 4 && DOT ? 8 : 16;

template <int DK, int DV, bool REV, bool DOT, typename Tin, typename Tout>
__global__ void __launch_bounds__(128)
linrec_token_kernel(const LinrecPass p) {
    constexpr int M = DK / 16, PARTS = DV / kSimtCols, kTile = kTileOf<Tin, DK, DOT>;
    __shared__ __align__(16) Tin sQ_[2][kTile][DK], sK_[2][kTile][DK], sV_[2][kTile][kSimtCols], sY_[2][DOT ? kTile : 1][kSimtCols];
    __shared__ __align__(16) float sO[kTile][kSimtCols];
    __shared__ float sA_[2][kTile], sDot[4][kTile], sRed[4];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rg = lane >> 3;
    const int part = blockIdx.x % PARTS, c0 = part * kSimtCols;
    const int64_t chain = blockIdx.x / PARTS, n = chain / p.H;
    const int h = (int)(chain % p.H), H = p.H;
    int64_t lo, hi;
    seq_range(p.seqs, n, lo, hi);
    const int64_t len = hi - lo, tiles = (len + kTile - 1) / kTile;
    const int wc = 16 * warp + 2 * (lane & 7);   // this thread's columns within the part

    // element (row, part column) of the caller's state
    auto at = [&](int i, int c) {
        return (size_t)chain * (DK * DV) + (p.state_t ? (size_t)(c0 + c) * DK + i : (size_t)i * DV + c0 + c);
    };
    float2 S[2][2 * M];   // [column][row pair]
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 2 * M; ++j) {
            const int i = 16 * (j >> 1) + 4 * rg + 2 * (j & 1);
            S[c][j] = p.init ? make_float2(p.init[at(i, wc + c)], p.init[at(i + 1, wc + c)]) : make_float2(0.f, 0.f);
        }
    const Tin *q = (const Tin *)p.q, *k = (const Tin *)p.k, *v = (const Tin *)p.v, *y = (const Tin *)p.y;
    Tout *out = (Tout *)p.out;
    // the stored states of this (head, part): one float2 per thread and register
    auto slot_ptr = [&](int64_t j) {
        const int64_t s = linrec_slot(kTokenAnchor, lo, n, j);
        return reinterpret_cast<float2 *>(p.anchor) + ((size_t)(s * H + h) * PARTS + part) * (DK * kSimtCols / 2) + tid;
    };
    auto store_anchor = [&](int64_t j) {
        float2 *d = slot_ptr(j);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 2 * M; ++r) __stcs(d + (c * 2 * M + r) * 128, S[c][r]);
    };
    auto inner_product = [&](int64_t j, float decay) {
        const float2 *d = slot_ptr(j);
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 2 * M; ++r) {
                const float2 s = __ldcs(d + (c * 2 * M + r) * 128);
                x = fmaf(s.x, S[c][r].x, x);
                x = fmaf(s.y, S[c][r].y, x);
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) sRed[warp] = x;
        __syncthreads();
        if (tid == 0)
            p.inner[((size_t)part * linrec_slots(kTokenAnchor, p.seqs) + linrec_slot(kTokenAnchor, lo, n, j)) * H + h] =
                decay * ((sRed[0] + sRed[1]) + (sRed[2] + sRed[3]));
        __syncthreads();
    };

    float la = 0.f;   // this thread's token's log decay of the tile that was issued last
    auto tile_of = [&](int64_t it) { return REV ? tiles - 1 - it : it; };
    auto issue = [&](int64_t it) {
        if (it < tiles) {
            constexpr int E = 16 / sizeof(Tin);   // elements of a 16-byte copy
            const int64_t base = lo + tile_of(it) * kTile;
            const int cnt = (int)min((int64_t)kTile, hi - base), b = (int)(it & 1);
            for (int i = tid; i < cnt * (DK / E); i += 128) {
                const int r = i / (DK / E), c = E * (i % (DK / E));
                const size_t g = ((size_t)(base + r) * H + h) * DK + c;
                umma::cp_async16(&sQ_[b][r][c], q + g);
                umma::cp_async16(&sK_[b][r][c], k + g);
            }
            for (int i = tid; i < cnt * (kSimtCols / E); i += 128) {
                const int r = i / (kSimtCols / E), c = E * (i % (kSimtCols / E));
                const size_t g = ((size_t)(base + r) * H + h) * DV + c0 + c;
                umma::cp_async16(&sV_[b][r][c], v + g);
                if (DOT) umma::cp_async16(&sY_[b][r][c], y + g);
            }
            // the decay in front of each token; backwards that of the next token
            const int64_t t = base + tid + (REV ? 1 : 0);
            la = p.la && tid < cnt && t < hi ? p.la[t * H + h] : 0.f;
        }
        umma::cp_async_commit();   // (empty behind the last tile)
    };
    issue(0);
    for (int64_t it = 0; it < tiles; ++it) {
        const int64_t tile = tile_of(it), base = lo + tile * kTile;
        const int cnt = (int)min((int64_t)kTile, hi - base);
        const auto &sQ = sQ_[it & 1];
        const auto &sK = sK_[it & 1];
        const auto &sV = sV_[it & 1];
        const auto &sY = sY_[it & 1];
        float *sA = sA_[it & 1];
        if (tid < cnt) sA[tid] = p.la ? expf(la) : 1.f;
        issue(it + 1);   // the other buffer's readers have passed the barrier behind their tile
        umma::cp_async_wait_group1();
        __syncthreads();
        if (DOT && REV && (tile + 1) * kTile % kTokenAnchor == 0 || DOT && REV && it == 0)
            inner_product(((tile + 1) * kTile - 1) / kTokenAnchor, sA[cnt - 1]);
        // kGroup tokens' read-outs are summed over the lanes together: the shuffles' latency is paid
        // once (rows behind the tile's end take no part; the condition is the block's)
        for (int x0 = 0; x0 < cnt; x0 += kGroup) {
            float o[kGroup][2], w[kGroup];
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                o[g][0] = o[g][1] = w[g] = 0.f;
                if (x0 + g >= cnt) continue;
                const int t = REV ? cnt - 1 - (x0 + g) : x0 + g;
                const float2 a2 = make_float2(sA[t], sA[t]);
                const float v0 = to_f32(sV[t][wc]), v1 = to_f32(sV[t][wc + 1]);
                const float2 v2[2] = {make_float2(v0, v0), make_float2(v1, v1)};
                float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}, qk = make_float2(0.f, 0.f);
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float4 k4 = load4(&sK[t][16 * m + 4 * rg]), q4 = load4(&sQ[t][16 * m + 4 * rg]);
                    const float2 kk[2] = {make_float2(k4.x, k4.y), make_float2(k4.z, k4.w)};
                    const float2 qq[2] = {make_float2(q4.x, q4.y), make_float2(q4.z, q4.w)};
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float2 &s = S[c][2 * m + e];
                            s = mul2(a2, s);
                            if (DOT) acc[c] = fma2(qq[e], s, acc[c]);
                            s = fma2(kk[e], v2[c], s);
                            if (!DOT) acc[c] = fma2(qq[e], s, acc[c]);
                        }
                        if (DOT) qk = fma2(qq[e], kk[e], qk);
                    }
                }
                o[g][0] = acc[0].x + acc[0].y;
                o[g][1] = acc[1].x + acc[1].y;
                w[g] = qk.x + qk.y;
            }
#pragma unroll
            for (int off = 8; off < 32; off <<= 1) {
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    o[g][0] += __shfl_xor_sync(0xffffffffu, o[g][0], off);
                    o[g][1] += __shfl_xor_sync(0xffffffffu, o[g][1], off);
                    if (DOT) w[g] += __shfl_xor_sync(0xffffffffu, w[g], off);
                }
            }
            if (DOT) {   // the other tokens' part of out . y, then the token's own term of out
                float d[kGroup];
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    const int t = x0 + g < cnt ? (REV ? cnt - 1 - (x0 + g) : x0 + g) : 0;
                    d[g] = fmaf(o[g][0], to_f32(sY[t][wc]), o[g][1] * to_f32(sY[t][wc + 1]));
                    o[g][0] = fmaf(w[g], to_f32(sV[t][wc]), o[g][0]);
                    o[g][1] = fmaf(w[g], to_f32(sV[t][wc + 1]), o[g][1]);
                }
#pragma unroll
                for (int off = 1; off < 8; off <<= 1) {
#pragma unroll
                    for (int g = 0; g < kGroup; ++g) d[g] += __shfl_xor_sync(0xffffffffu, d[g], off);
                }
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    if (lane == 0 && x0 + g < cnt) sDot[warp][REV ? cnt - 1 - (x0 + g) : x0 + g] = d[g];
            }
#pragma unroll
            for (int g = 0; g < kGroup; ++g)
                if (rg == 0 && x0 + g < cnt)
                    *reinterpret_cast<float2 *>(&sO[REV ? cnt - 1 - (x0 + g) : x0 + g][wc]) = make_float2(o[g][0], o[g][1]);
        }
        __syncthreads();
        for (int i = tid; i < cnt * (kSimtCols / 4); i += 128) {
            const int r = i / (kSimtCols / 4), c = 4 * (i % (kSimtCols / 4));
            store4(out + ((size_t)(base + r) * H + h) * DV + c0 + c, *reinterpret_cast<const float4 *>(&sO[r][c]));
        }
        if (DOT && tid < cnt)
            p.dot[((size_t)part * H + h) * p.seqs.total + base + tid] =
                (sDot[0][tid] + sDot[1][tid]) + (sDot[2][tid] + sDot[3][tid]);
        if (DOT && !REV && ((tile + 1) * kTile % kTokenAnchor == 0 || it == tiles - 1))
            store_anchor(((tile + 1) * kTile - 1) / kTokenAnchor);
    }
    if (p.fin) {
        const float a = REV && len > 0 && p.la ? expf(p.la[lo * H + h]) : 1.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 2 * M; ++j) {
                const int i = 16 * (j >> 1) + 4 * rg + 2 * (j & 1);
                p.fin[at(i, wc + c)] = a * S[c][j].x;
                p.fin[at(i + 1, wc + c)] = a * S[c][j].y;
            }
    }
}

template <int DK, int DV, typename Tin, typename Tout>
int launch_token(const LinrecPass &p, cudaStream_t s) {
    const int64_t ctas = p.seqs.N * p.H * (DV / kSimtCols);
    if (p.rev && p.dot) linrec_token_kernel<DK, DV, true, true, Tin, Tout><<<(unsigned)ctas, 128, 0, s>>>(p);
    else if (p.rev) linrec_token_kernel<DK, DV, true, false, Tin, Tout><<<(unsigned)ctas, 128, 0, s>>>(p);
    else if (p.dot) linrec_token_kernel<DK, DV, false, true, Tin, Tout><<<(unsigned)ctas, 128, 0, s>>>(p);
    else linrec_token_kernel<DK, DV, false, false, Tin, Tout><<<(unsigned)ctas, 128, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

template <int DK, int DV>
int launch_token_types(const LinrecPass &p, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (p.in_bf16 && p.out_bf16) return launch_token<DK, DV, bf, bf>(p, s);
    if (p.in_bf16) return launch_token<DK, DV, bf, float>(p, s);
    if (p.out_bf16) return launch_token<DK, DV, float, bf>(p, s);
    return launch_token<DK, DV, float, float>(p, s);
}

// ---------------------------------------------------------------- log-decay gradient
// One warp per run of 32 E tokens of a chain: E consecutive tokens a lane, a suffix sum
// over the lanes, the run's inner product added.  Where alpha is 0 (a reset) so is the gradient,
// alpha <S, dS>: the sums would leave their rounding there.  Reads 12 and writes 4 bytes a head-token.
template <int E>
__global__ void __launch_bounds__(256)
linrec_gate_grad_kernel(const LinrecSeqs seqs, int H, int parts, const float *__restrict__ la, const float *__restrict__ dot_q,
                        const float *__restrict__ dot_k, const float *__restrict__ inner, float *__restrict__ dla) {
    const int64_t chain = blockIdx.x, n = chain / H;
    const int h = (int)(chain % H), lane = threadIdx.x & 31;
    int64_t lo, hi;
    seq_range(seqs, n, lo, hi);
    constexpr int RUN = 32 * E;
    const int64_t runs = (hi - lo + RUN - 1) / RUN, slots = linrec_slots(RUN, seqs);
    for (int64_t j = blockIdx.y * 8 + (threadIdx.x >> 5); j < runs; j += (int64_t)gridDim.y * 8) {
        const int64_t t0 = lo + j * RUN + E * lane;
        float x[E], a[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = 0.f;
            a[e] = t0 + e < hi ? la[(t0 + e) * H + h] : 0.f;
        }
        float d = 0.f;
        for (int part = 0; part < parts; ++part) {
            const size_t row = ((size_t)part * H + h) * seqs.total;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (t0 + e < hi) x[e] += dot_q[row + t0 + e] - dot_k[row + t0 + e];
            d += inner[((size_t)part * slots + linrec_slot(RUN, lo, n, j)) * H + h];
        }
#pragma unroll
        for (int e = E - 2; e >= 0; --e) x[e] += x[e + 1];
        float later = x[0];   // inclusive suffix sum over the lanes, then without the own part
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float z = __shfl_down_sync(0xffffffffu, later, o);
            if (lane + o < 32) later += z;
        }
        later = __shfl_down_sync(0xffffffffu, later, 1);
        if (lane == 31) later = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (t0 + e < hi) dla[(t0 + e) * H + h] = expf(a[e]) == 0.f ? 0.f : x[e] + later + d;
    }
}

// ---------------------------------------------------------------- rows of no sequence
// Packed sequences lie behind one another, so the rest is in front of the first and behind the last.
__global__ void __launch_bounds__(256)
linrec_zero_rest_kernel(const LinrecSeqs seqs, const LinrecRest rest) {
    int64_t lo, last, hi;
    seq_range(seqs, 0, lo, hi);
    seq_range(seqs, seqs.N - 1, last, hi);
    const int64_t t0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        if (!rest.rows[b]) continue;
        uint4 *p = static_cast<uint4 *>(rest.rows[b]);
        const int64_t w = rest.row_bytes[b] / 16;
        for (int64_t i = t0; i < lo * w; i += step) p[i] = make_uint4(0, 0, 0, 0);
        for (int64_t i = hi * w + t0; i < seqs.total * w; i += step) p[i] = make_uint4(0, 0, 0, 0);
    }
    if (!rest.gates) return;
    for (int64_t i = t0; i < lo * rest.gate_words; i += step) rest.gates[i] = 0.f;
    for (int64_t i = hi * rest.gate_words + t0; i < seqs.total * rest.gate_words; i += step) rest.gates[i] = 0.f;
}

// ---------------------------------------------------------------- single token
// S <- a S + k v^T in place, o = S^T q: a stream of the state through the SM, bound by HBM
// bandwidth.  A CTA holds COLS value columns of one chain; lane (rr, cq) = (lane / 4, lane % 4)
// owns the float4 at columns 4 cq of its warp's 16 and rows rr + 8 m, so a warp's load touches
// whole 32-byte sectors and a column's read-out is a register sum and three shuffles.  32 columns
// a CTA: 8192 chains of 128 x 128 take 157 us, 6.9 TB/s; 16 chains spread over 64 SMs.
template <int DK, int DV, int COLS, typename Tin, typename Tout>
__global__ void __launch_bounds__(COLS * 2)
linrec_step_kernel(const Tin *__restrict__ q, const Tin *__restrict__ k, const Tin *__restrict__ v,
                   const float *__restrict__ la, float *__restrict__ state, Tout *__restrict__ out) {
    constexpr int RPL = DK / 8, PARTS = DV / COLS;
    const int64_t chain = blockIdx.x / PARTS;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cq = lane & 3, rr = lane >> 2;
    const int col = (int)(blockIdx.x % PARTS) * COLS + warp * 16 + cq * 4;
    float *S = state + (size_t)chain * DK * DV;
    float4 s[RPL];   // the only long-latency loads, issued first
#pragma unroll
    for (int m = 0; m < RPL; ++m)
        s[m] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(rr + 8 * m) * DV + col));
    __shared__ float sk[DK], sq[DK];
    for (int i = tid; i < DK; i += COLS * 2) {
        sk[i] = to_f32(k[(size_t)chain * DK + i]);
        sq[i] = to_f32(q[(size_t)chain * DK + i]);
    }
    const float a = la ? expf(la[chain]) : 1.f;
    const float4 vv = load4(v + (size_t)chain * DV + col);
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < RPL; ++m) {
        const int i = rr + 8 * m;
        const float ki = sk[i], qi = sq[i];
        float4 x;
        x.x = fmaf(a, s[m].x, ki * vv.x); x.y = fmaf(a, s[m].y, ki * vv.y);
        x.z = fmaf(a, s[m].z, ki * vv.z); x.w = fmaf(a, s[m].w, ki * vv.w);
        o.x = fmaf(qi, x.x, o.x); o.y = fmaf(qi, x.y, o.y);
        o.z = fmaf(qi, x.z, o.z); o.w = fmaf(qi, x.w, o.w);
        __stcs(reinterpret_cast<float4 *>(S + (size_t)i * DV + col), x);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    if (rr == 0) store4(out + (size_t)chain * DV + col, o);
}

template <int DK, int DV, typename Tin, typename Tout>
int launch_step(int64_t chains, const void *q, const void *k, const void *v, const float *la, float *state, void *out,
                cudaStream_t s) {
    linrec_step_kernel<DK, DV, 32, Tin, Tout><<<(unsigned)(chains * (DV / 32)), 64, 0, s>>>(
        (const Tin *)q, (const Tin *)k, (const Tin *)v, la, state, (Tout *)out);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

template <int DK, int DV>
int launch_step_types(int64_t n, bool ib, bool ob, const void *q, const void *k, const void *v, const float *la,
                      float *state, void *out, cudaStream_t s) {
    using bf = __nv_bfloat16;
    if (ib && ob) return launch_step<DK, DV, bf, bf>(n, q, k, v, la, state, out, s);
    if (ib) return launch_step<DK, DV, bf, float>(n, q, k, v, la, state, out, s);
    if (ob) return launch_step<DK, DV, float, bf>(n, q, k, v, la, state, out, s);
    return launch_step<DK, DV, float, float>(n, q, k, v, la, state, out, s);
}

}  // namespace

int launch_linrec_simt(const LinrecPass &p, cudaStream_t s) {
    if (p.dk == 128 && p.dv == 128) return launch_token_types<128, 128>(p, s);
    if (p.dk == 128 && p.dv == 64) return launch_token_types<128, 64>(p, s);
    if (p.dk == 64 && p.dv == 128) return launch_token_types<64, 128>(p, s);
    if (p.dk == 64 && p.dv == 64) return launch_token_types<64, 64>(p, s);
    return kErrUnsupported;
}

int launch_linrec_gate_grad(const LinrecSeqs &seqs, int H, int run, int parts, const float *la, const float *dot_q,
                            const float *dot_k, const float *inner, float *dla, cudaStream_t s) {
    const int64_t runs = ((seqs.cu ? seqs.total : seqs.T) + run - 1) / run;
    const int64_t y = runs < 8 ? 1 : (runs + 7) / 8 < 1024 ? (runs + 7) / 8 : 1024;
    const dim3 grid((unsigned)(seqs.N * H), (unsigned)y);
    if (run == kAnchor) linrec_gate_grad_kernel<kAnchor / 32><<<grid, 256, 0, s>>>(seqs, H, parts, la, dot_q, dot_k, inner, dla);
    else linrec_gate_grad_kernel<kTokenAnchor / 32><<<grid, 256, 0, s>>>(seqs, H, parts, la, dot_q, dot_k, inner, dla);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

int launch_linrec_zero_rest(const LinrecSeqs &seqs, const LinrecRest &r, cudaStream_t s) {
    linrec_zero_rest_kernel<<<304, 256, 0, s>>>(seqs, r);   // two blocks an SM
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

int launch_linrec_step(int64_t n, int dk, int dv, bool ib, bool ob, const void *q, const void *k, const void *v,
                       const float *la, float *state, void *out, cudaStream_t s) {
    if (dk == 128 && dv == 128) return launch_step_types<128, 128>(n, ib, ob, q, k, v, la, state, out, s);
    if (dk == 128 && dv == 64) return launch_step_types<128, 64>(n, ib, ob, q, k, v, la, state, out, s);
    if (dk == 64 && dv == 128) return launch_step_types<64, 128>(n, ib, ob, q, k, v, la, state, out, s);
    if (dk == 64 && dv == 64) return launch_step_types<64, 64>(n, ib, ob, q, k, v, la, state, out, s);
    return kErrUnsupported;
}

}  // namespace dr
