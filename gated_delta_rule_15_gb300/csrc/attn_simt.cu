// attn_simt.cu -- window attention on the CUDA cores (fp32 rows): forward, gradients.  The
// mathematics: attn.h; the blocks of dk and dv: attn_sinks.cuh.
//
// Tiles of 16 R rows (queries; of dk, dv keys) by 64 others, 256 threads as 16 x 16: a thread holds R x 4 scores (rows
// R ty + r, others tx + 16 c) and R rows x d / 16 columns of what is summed.  Products run over rows in
// shared memory as float4 of both operands and two FMAs an instruction (R = 4: 32 of them to 8 loads); the
// row stride of d + 4 floats keeps the 16 rows of a load on different banks.  What is summed over tiles is first summed
// within one, so that sums of a thousand terms are less off than one chain of them would be.
// The 64 others come by asynchronous copies a tile ahead.  A query's keys: first the sinks in front of its tile's window, then the
// window, with the running maximum and sum of the softmax in registers.
// R = 4, or 1 where tiles of 64 rows would leave more than half of the SMs without one.  Measured with R = 1 and 4, by the
// number of tiles of 64: forward 8 (T256 H2 d64 w64) 10.3 and 18.5 us, 32 (T512 H4 d128) 51 and 74, 80 (T300 H16 d64 w64) 14.3 and
// 16.4, 102 (T1037 H6 d64 w200) 39 and 31, 128 (T2048 H4 d128) 414 and 275; dq 32 35 us less, 80 18 and 102 30 us more; dk, dv 51 25
// us less, 64 (B2 T1024 H8/2) 8 us less, 128 (T4096 H2 d64 w256) 40 us more.
// What bounds it: issue and shared memory (R = 4: 12 of its cycles to 16 of FMAs; R = 1: 9 to 4), and
// for the few blocks of small problems the longest one's tiles, one behind another.
#include "../../include/dr.h"
#include "attn.h"
#include "attn_sinks.cuh"
#include "common.cuh"
#include "launch_chain.cuh"
#include "umma.cuh"

namespace dr {
namespace {

using umma::add2;
using umma::fma2;
using umma::mul2;

constexpr int kTile = 64, kThreads = 256, kPs = kTile + 4;

template <int D> constexpr int row_floats() { return D + 4; }

// Rows 0 .. ROWS - 1 of one head as at(r) says, zeros where that is NULL, on their way.  `any`: some address of the rows.
template <int D, int ROWS, class At>
__device__ __forceinline__ void fetch(float *dst, const void *any, At at) {
    constexpr int PER = D / 4;
#pragma unroll
    for (int i = threadIdx.x; i < ROWS * PER; i += kThreads) {
        const int r = i / PER, c = i % PER;
        const float *src = at(r);
        umma::cp_async16(dst + r * row_floats<D>() + 4 * c, src ? src + 4 * c : any, src ? 16u : 0u);
    }
}

// acc[r][c] = sum over d of A[R ty + r] B[tx + 16 c], in sums of 8 of the even and 8 of the odd channels (a score's error is
// its weight's)
template <int D, int R>
__device__ __forceinline__ void rows_by_rows(float (&acc)[R][4], const float *A, const float *B, int ty, int tx) {
    constexpr int S = row_floats<D>();
    float2 sum[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[r][c] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < D; k0 += 16) {
        float2 x[R][4];
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            float4 a[R], b[4];
#pragma unroll
            for (int r = 0; r < R; ++r) a[r] = load4(A + (R * ty + r) * S + k0 + k);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = load4(B + (tx + 16 * c) * S + k0 + k);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 a0 = make_float2(a[r].x, a[r].y), b0 = make_float2(b[c].x, b[c].y);
                    x[r][c] = k == 0 ? mul2(a0, b0) : fma2(a0, b0, x[r][c]);
                    x[r][c] = fma2(make_float2(a[r].z, a[r].w), make_float2(b[c].z, b[c].w), x[r][c]);
                }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) sum[r][c] = add2(sum[r][c], x[r][c]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = sum[r][c].x + sum[r][c].y;
}

// acc[r][2 u + h] += sum over `n` k (a multiple of 4) of P[R ty + r][k] X[k][64 u + 4 tx + 2 h, + 1]
template <int D, int R>
__device__ __forceinline__ void rows_by_cols(float2 (&acc)[R][D / 32], const float *P, const float *X, int n, int ty, int tx) {
    constexpr int S = row_floats<D>(), U = D / 64;
    float2 sum[R][D / 32];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) sum[r][u] = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < n; k += 4) {
        float p[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 x = load4(P + (R * ty + r) * kPs + k);
            p[r][0] = x.x; p[r][1] = x.y; p[r][2] = x.z; p[r][3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 x = load4(X + (k + e) * S + 64 * u + 4 * tx);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    sum[r][2 * u] = fma2(make_float2(p[r][e], p[r][e]), make_float2(x.x, x.y), sum[r][2 * u]);
                    sum[r][2 * u + 1] = fma2(make_float2(p[r][e], p[r][e]), make_float2(x.z, x.w), sum[r][2 * u + 1]);
                }
            }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < D / 32; ++u) acc[r][u] = add2(acc[r][u], sum[r][u]);
}

// A thread's scores where the 16 threads of its rows, which are in its warp, read them.
template <int R>
__device__ __forceinline__ void put_scores(float *P, const float (&s)[R][4], int ty, int tx) {
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) P[(R * ty + r) * kPs + tx + 16 * c] = s[r][c];
    __syncwarp();
}

__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ bool sees(const AttnProblem &p, int i, int j) {
    return j <= i && (i - j < p.window || j < p.sinks);
}

// The keys of the queries q0 .. q0 + rows - 1, one behind another: sinks in front of the first one's window, then the keys
// from there to the last one.
struct Keys {
    int sinks, near0, total;
    __device__ __forceinline__ Keys(const AttnProblem &p, int q0, int rows, int len) {
        near0 = max(0, q0 - p.window + 1);
        sinks = min(p.sinks, near0);
        total = sinks + min(len, q0 + rows) - near0;
    }
    __device__ __forceinline__ int at(int v) const { return v < sinks ? v : near0 + v - sinks; }
};

template <int D, int R>
__device__ __forceinline__ void put_rows(float *dst, int64_t stride, int n, const float2 (&x)[R][D / 32], float f, int ty, int tx) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (R * ty + r >= n) continue;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            store4(dst + (int64_t)(R * ty + r) * stride + 64 * u + 4 * tx,
                   make_float4(f * x[r][2 * u].x, f * x[r][2 * u].y, f * x[r][2 * u + 1].x, f * x[r][2 * u + 1].y));
    }
}

// A query tile's block: (sequence tile, head).
template <int ROWS>
__device__ __forceinline__ bool query_tile(const AttnProblem &p, int &h, int &hk, int64_t &lo, int &len, int &q0) {
    int64_t n;
    int j;
    h = blockIdx.x % p.Hq;
    hk = h / (p.Hq / p.Hk);
    if (!find_tile(p.seqs, ROWS, blockIdx.x / p.Hq, n, j, lo, len)) return false;
    q0 = j * ROWS;
    return true;
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads) attn_simt_fwd_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>(), ROWS = 16 * R;
    extern __shared__ float sm[];
    float *Q = sm, *KV = Q + ROWS * S, *P = KV + 4 * kTile * S;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    int64_t lo;
    int h, hk, len, q0;
    if (!query_tile<ROWS>(p, h, hk, lo, len, q0)) return;
    const Keys keys(p, q0, ROWS, len);
    const float *q = (const float *)p.q + (lo + q0) * p.qs + h * D, *k = (const float *)p.k + lo * p.ks + hk * D,
                *v = (const float *)p.v + lo * p.vs + hk * D;
    auto fetch_keys = [&](int t) {
        float *dst = KV + (t & 1) * 2 * kTile * S;
        fetch<D, kTile>(dst, k, [&](int r) { return kTile * t + r < keys.total ? k + (int64_t)keys.at(kTile * t + r) * p.ks : nullptr; });
        fetch<D, kTile>(dst + kTile * S, v, [&](int r) { return kTile * t + r < keys.total ? v + (int64_t)keys.at(kTile * t + r) * p.vs : nullptr; });
    };
    fetch<D, ROWS>(Q, p.q, [&](int r) { return q0 + r < len ? q + (int64_t)r * p.qs : nullptr; });
    fetch_keys(0);
    umma::cp_async_commit();
    float m[R], l[R];
    float2 o[R][D / 32];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[r][c] = make_float2(0.f, 0.f);
    }
    const int tiles = (keys.total + kTile - 1) / kTile;
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_keys(t + 1);
        umma::cp_async_commit();
        const float *K = KV + (t & 1) * 2 * kTile * S;
        float s[R][4];
        rows_by_rows<D, R>(s, Q, K, ty, tx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = q0 + R * ty + r;
            float top = m[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int at = kTile * t + tx + 16 * c;
                s[r][c] = at < keys.total && sees(p, i, keys.at(at)) ? p.scale * s[r][c] : -INFINITY;
                top = fmaxf(top, s[r][c]);
            }
            top = max16(top);
            const float base = top == -INFINITY ? 0.f : top, turn = expf(m[r] - base);
            m[r] = top;
            float sum = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] = expf(s[r][c] - base);
                sum += s[r][c];
            }
            l[r] = fmaf(l[r], turn, sum);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[r][c] = mul2(o[r][c], make_float2(turn, turn));
        }
        put_scores<R>(P, s, ty, tx);
        rows_by_cols<D, R>(o, P, K + kTile * S, min(kTile, (keys.total - kTile * t + 3) & ~3), ty, tx);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float sum = sum16(l[r]), inv = 1.f / sum;
        const int i = q0 + R * ty + r;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[r][c] = mul2(o[r][c], make_float2(inv, inv));
        if (i < len && tx == 0) p.lse[(lo + i) * p.Hq + h] = m[r] + logf(sum);
    }
    put_rows<D, R>((float *)p.out + ((lo + q0) * p.Hq + h) * D, (int64_t)p.Hq * D, len - q0, o, 1.f, ty, tx);
}

// dq of a query tile, and of its rows l and delta.  lse and out are rounded, and results of other sums than this kernel's:
// with w_ij = exp(s_ij - lse_i), l = sum_j w_ij is not quite 1 and sum_j w_ij (do_i.v_j - do_i.o_i) not quite 0, which what
// the keys have in common magnifies.  So
//     x_ij = w_ij (do_i.v_j - do_i.o_i),   e = sum_j x_ij / l,   delta_i = do_i.o_i + e,
//     dq_i = scale (sum_j x_ij k_j - e sum_j w_ij k_j) / l,
// a fourth product to three (keys with a common direction of 3 times their spread, sequences of 10 tokens: dq off by 2.5e-6
// without, where all in one arithmetic is off by 1.1e-6).
template <int D, int R>
__global__ void __launch_bounds__(kThreads) attn_simt_dq_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>(), ROWS = 16 * R;
    extern __shared__ float sm[];
    float *Q = sm, *O = Q + ROWS * S, *KV = O + ROWS * S, *P = KV + 4 * kTile * S;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    int64_t lo;
    int h, hk, len, q0;
    let_next_start();
    if (!query_tile<ROWS>(p, h, hk, lo, len, q0)) return;
    const int rows = len - q0;
    const Keys keys(p, q0, ROWS, len);
    const float *q = (const float *)p.q + (lo + q0) * p.qs + h * D, *k = (const float *)p.k + lo * p.ks + hk * D,
                *v = (const float *)p.v + lo * p.vs + hk * D;
    const int64_t at0 = ((lo + q0) * p.Hq + h) * D, step = (int64_t)p.Hq * D;
    auto fetch_keys = [&](int t) {
        float *dst = KV + (t & 1) * 2 * kTile * S;
        fetch<D, kTile>(dst, k, [&](int r) { return kTile * t + r < keys.total ? k + (int64_t)keys.at(kTile * t + r) * p.ks : nullptr; });
        fetch<D, kTile>(dst + kTile * S, v, [&](int r) { return kTile * t + r < keys.total ? v + (int64_t)keys.at(kTile * t + r) * p.vs : nullptr; });
    };
    fetch<D, ROWS>(O, p.d_out, [&](int r) { return r < rows ? (const float *)p.d_out + at0 + r * step : nullptr; });
    fetch<D, ROWS>(Q, p.q, [&](int r) { return r < rows ? q + (int64_t)r * p.qs : nullptr; });
    fetch_keys(0);
    umma::cp_async_commit();
    float delta[R], lse[R], l[R], e[R];
    float2 dq[R][D / 32], wk[R][D / 32];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = R * ty + r;
        float x = 0.f;
        if (i < rows) {
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const float4 a = load4((const float *)p.out + at0 + i * step + 64 * u + 4 * tx),
                             b = load4((const float *)p.d_out + at0 + i * step + 64 * u + 4 * tx);
                x += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
            }
        }
        delta[r] = sum16(x);
        lse[r] = i < rows ? p.lse[(lo + q0 + i) * p.Hq + h] : 0.f;
        l[r] = e[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) dq[r][c] = wk[r][c] = make_float2(0.f, 0.f);
    }
    const int tiles = (keys.total + kTile - 1) / kTile;
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_keys(t + 1);
        umma::cp_async_commit();
        const float *K = KV + (t & 1) * 2 * kTile * S;
        float s[R][4], dp[R][4];
        rows_by_rows<D, R>(s, Q, K, ty, tx);
        rows_by_rows<D, R>(dp, O, K + kTile * S, ty, tx);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float sw = 0.f, sx = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int at = kTile * t + tx + 16 * c;
                const bool in = at < keys.total && sees(p, q0 + R * ty + r, keys.at(at));
                s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -lse[r])) : 0.f;
                dp[r][c] = in ? s[r][c] * (dp[r][c] - delta[r]) : 0.f;
                sw += s[r][c];
                sx += dp[r][c];
            }
            l[r] += sw;
            e[r] += sx;
        }
        const int n = min(kTile, (keys.total - kTile * t + 3) & ~3);
        put_scores<R>(P, s, ty, tx);
        rows_by_cols<D, R>(wk, P, K, n, ty, tx);
        put_scores<R>(P, dp, ty, tx);
        rows_by_cols<D, R>(dq, P, K, n, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = R * ty + r;
        const float inv = 1.f / sum16(l[r]), x = sum16(e[r]) * inv;
        if (tx == 0 && i < rows) {
            const int64_t at = h * p.seqs.total + lo + q0 + i;
            p.delta[at] = delta[r] + x;
            p.inv_l[at] = inv;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) dq[r][c] = mul2(fma2(make_float2(-x, -x), wk[r][c], dq[r][c]), make_float2(inv, inv));
    }
    put_rows<D, R>((float *)p.dq + (lo + q0) * p.dqs + h * D, p.dqs, rows, dq, p.scale, ty, tx);
}

// dk and dv of a key tile, over the block's queries and all heads that share the keys.
template <int D, int R>
__global__ void __launch_bounds__(kThreads) attn_simt_dkv_kernel(const AttnProblem p, const attn::SinkPlan plan) {
    constexpr int S = row_floats<D>(), ROWS = 16 * R;
    extern __shared__ float sm[];
    float *K = sm, *V = K + ROWS * S, *QO = V + ROWS * S, *P = QO + 4 * kTile * S, *stat = P + ROWS * kPs;   // [2][lse, delta, 1 / l][64]
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, g = p.Hq / p.Hk;
    attn::KeyBlock kb;
    let_next_start();
    if (!kb.find(p, plan, blockIdx.x)) {
        wait_for_last();
        return;
    }
    const int64_t lo = kb.lo;
    const int len = kb.len, hk = kb.hk, k0 = kb.k0, rows = len - k0;
    const int nt = (kb.qb - kb.qa + kTile - 1) / kTile, tiles = nt * g;
    auto fetch_queries = [&](int t) {
        const int h = hk * g + t / nt, q0 = kb.qa + t % nt * kTile, n = kb.qb - q0;
        float *dst = QO + (t & 1) * 2 * kTile * S, *st = stat + (t & 1) * 3 * kTile;
        const float *q = (const float *)p.q + (lo + q0) * p.qs + h * D, *d = (const float *)p.d_out + ((lo + q0) * p.Hq + h) * D;
        fetch<D, kTile>(dst, p.q, [&](int r) { return r < n ? q + (int64_t)r * p.qs : nullptr; });
        fetch<D, kTile>(dst + kTile * S, p.d_out, [&](int r) { return r < n ? d + (int64_t)r * p.Hq * D : nullptr; });
        const int r = threadIdx.x & (kTile - 1);
        if (threadIdx.x < kTile) umma::cp_async4(st + r, r < n ? p.lse + (lo + q0 + r) * p.Hq + h : p.lse, r < n ? 4u : 0u);
        else if (threadIdx.x < 3 * kTile) {
            const float *from = threadIdx.x < 2 * kTile ? p.delta : p.inv_l;
            umma::cp_async4(st + threadIdx.x, r < n ? from + h * p.seqs.total + lo + q0 + r : from, r < n ? 4u : 0u);
        }
    };
    fetch<D, ROWS>(K, p.k, [&](int r) { return r < rows ? (const float *)p.k + (lo + k0 + r) * p.ks + hk * D : nullptr; });
    fetch<D, ROWS>(V, p.v, [&](int r) { return r < rows ? (const float *)p.v + (lo + k0 + r) * p.vs + hk * D : nullptr; });
    wait_for_last();       // delta, 1 / l
    fetch_queries(0);
    umma::cp_async_commit();
    float2 dk[R][D / 32], dv[R][D / 32];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < D / 32; ++c) dk[r][c] = dv[r][c] = make_float2(0.f, 0.f);
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_queries(t + 1);
        umma::cp_async_commit();
        const int q0 = kb.qa + t % nt * kTile, n = min(kTile, (kb.qb - q0 + 3) & ~3);
        const float *Q = QO + (t & 1) * 2 * kTile * S, *O = Q + kTile * S, *st = stat + (t & 1) * 3 * kTile;
        float s[R][4], dp[R][4];
        rows_by_rows<D, R>(s, K, Q, ty, tx);
        rows_by_rows<D, R>(dp, V, O, ty, tx);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int qi = tx + 16 * c, j = k0 + R * ty + r;
                const bool in = q0 + qi < kb.qb && sees(p, q0 + qi, j) && (kb.chunk < 0 || j < p.sinks);
                s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -st[qi])) * st[2 * kTile + qi] : 0.f;
                dp[r][c] = in ? s[r][c] * (dp[r][c] - st[kTile + qi]) : 0.f;
            }
        put_scores<R>(P, s, ty, tx);
        rows_by_cols<D, R>(dv, P, O, n, ty, tx);
        put_scores<R>(P, dp, ty, tx);
        rows_by_cols<D, R>(dk, P, Q, n, ty, tx);
    }
    // a sink's row is a part of a sum where its queries are cut
    const int sinks = kb.cut ? min(p.sinks - k0, rows) : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = R * ty + r;
        const bool part = row < sinks;
        if (row >= rows || (kb.chunk >= 0 && !part)) continue;
        float *to_k = part ? kb.sum(p, plan, k0 + row) : (float *)p.dk + (lo + k0 + row) * p.dks + hk * D;
        float *to_v = part ? to_k + D : (float *)p.dv + (lo + k0 + row) * p.dvs + hk * D;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float2 a = mul2(dk[r][2 * u], make_float2(p.scale, p.scale)), b = mul2(dk[r][2 * u + 1], make_float2(p.scale, p.scale));
            store4(to_k + 64 * u + 4 * tx, make_float4(a.x, a.y, b.x, b.y));
            store4(to_v + 64 * u + 4 * tx, make_float4(dv[r][2 * u].x, dv[r][2 * u].y, dv[r][2 * u + 1].x, dv[r][2 * u + 1].y));
        }
    }
}

// Rows in front of the first sequence and behind the last.
__global__ void __launch_bounds__(256) attn_zero_rest_kernel(const LinrecSeqs s, const AttnRest r) {
    const int64_t first = min(max(s.cu[0], (int64_t)0), s.total), last = min(max(s.cu[s.N], first), s.total);
    const int64_t rows = first + s.total - last;
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        if (!r.p[b]) continue;
        const int64_t words = r.bytes[b] / 4;
        for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * words; i += (int64_t)gridDim.x * 256) {
            const int64_t row = i / words < first ? i / words : i / words - first + last;
            reinterpret_cast<uint32_t *>(static_cast<char *>(r.p[b]) + row * r.stride[b])[i % words] = 0u;
        }
    }
}

constexpr int kSms = 152;

// Whether to take tiles of 16 rows (above).
bool few(const AttnProblem &p, int heads) { return attn_tile_slots(p.seqs, kTile) * heads < kSms / 2; }

template <class F, class... A>
int launch(F *kernel, size_t floats, int64_t blocks, cudaStream_t s, const A &...args) {
    const size_t smem = sizeof(float) * floats;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return kErrCuda;
    kernel<<<(unsigned)blocks, kThreads, smem, s>>>(args...);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}
template <class F, class... A>
int launch_next(F *kernel, size_t floats, int64_t blocks, cudaStream_t s, const A &...args) {
    const size_t smem = sizeof(float) * floats;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return kErrCuda;
    return launch_after(kernel, (unsigned)blocks, kThreads, smem, s, args...);
}
// a block's own tiles of ROWS rows, the four of 64, the scores
template <int D> constexpr size_t floats(int own, int rows) { return (size_t)(own * rows + 4 * kTile) * row_floats<D>() + (size_t)rows * kPs; }

template <int D, int R>
int fwd(const AttnProblem &p, cudaStream_t s) {
    return launch(attn_simt_fwd_kernel<D, R>, floats<D>(1, 16 * R), attn_tile_slots(p.seqs, 16 * R) * p.Hq, s, p);
}
template <int D, int R>
int bwd_q(const AttnProblem &p, cudaStream_t s) {
    return launch(attn_simt_dq_kernel<D, R>, floats<D>(2, 16 * R), attn_tile_slots(p.seqs, 16 * R) * p.Hq, s, p);
}

int key_rows(const AttnProblem &p) { return few(p, p.Hk) ? 16 : 64; }
// delta, or 1 / l
size_t stat_bytes(const AttnProblem &p) { return attn::round256(sizeof(float) * (size_t)(p.seqs.total * p.Hq)); }

template <int D>
int bwd(const AttnProblem &p, void *workspace, cudaStream_t s) {
    int rc = few(p, p.Hq) ? bwd_q<D, 1>(p, s) : bwd_q<D, 4>(p, s);
    if (rc != kOk) return rc;
    attn::SinkPlan plan;
    attn::plan_sinks(p, key_rows(p), 256, (char *)workspace + 2 * stat_bytes(p), plan);
    const int64_t blocks = attn::key_blocks(p, plan);
    rc = plan.tile == 16 ? launch_next(attn_simt_dkv_kernel<D, 1>, floats<D>(2, 16) + 6 * kTile, blocks, s, p, plan)
                         : launch_next(attn_simt_dkv_kernel<D, 4>, floats<D>(2, 64) + 6 * kTile, blocks, s, p, plan);
    return rc != kOk ? rc : attn::launch_sink_sum<D, float>(p, plan, s);
}

}  // namespace

int launch_attn_simt_fwd(const AttnProblem &p, cudaStream_t s) {
    if (few(p, p.Hq)) return p.d == 64 ? fwd<64, 1>(p, s) : fwd<128, 1>(p, s);
    return p.d == 64 ? fwd<64, 4>(p, s) : fwd<128, 4>(p, s);
}

size_t attn_simt_bwd_workspace_bytes(const AttnProblem &p) {
    attn::SinkPlan plan;
    return 2 * stat_bytes(p) + attn::plan_sinks(p, key_rows(p), 256, nullptr, plan);
}

int launch_attn_simt_bwd(const AttnProblem &p, void *workspace, cudaStream_t s) {
    AttnProblem x = p;
    x.delta = (float *)workspace;
    x.inv_l = (float *)((char *)workspace + stat_bytes(p));
    return p.d == 64 ? bwd<64>(x, workspace, s) : bwd<128>(x, workspace, s);
}

int launch_attn_zero_rest(const LinrecSeqs &s, const AttnRest &r, cudaStream_t stream) {
    attn_zero_rest_kernel<<<152, 256, 0, stream>>>(s, r);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace dr
