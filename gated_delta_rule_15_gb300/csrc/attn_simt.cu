// attn_simt.cu -- window attention on the CUDA cores (fp32 rows): forward, gradients.  The
// mathematics: attn.h; the blocks of dk and dv: attn_sinks.cuh.
//
// A block takes a tile of 64 or 16 rows (queries; of dk, dv keys) and 64 others at a time, with 256 threads: Across and Patches below say who
// has which scores and sums.  Products run over rows in shared memory as float4 of both operands and two FMAs an
// instruction; the row stride of d + 4 floats keeps the rows of a load on different banks.  What is summed
// over tiles is first summed within one, so that sums of a thousand terms are less off than one chain of them would be.
// The 64 others come by asynchronous copies a tile ahead.  A query's keys: first the sinks in front of its tile's window, then
// the window, with the running maximum and sum of the softmax in registers.
//
// Tiles of 16 rows where those of 64 would leave more than half of the SMs without one.  Measured with 16 and 64, by the
// number of tiles of 64: forward 8 (T256 H2 d64 w64) 10.3 and 18.5 us, 32 (T512 H4 d128) 51 and 74, 80 (T300 H16 d64 w64) 14.3
// and 16.4, 102 (T1037 H6 d64 w200) 39 and 31, 128 (T2048 H4 d128) 414 and 275; all of the backward, dq's tiles: 32 (T512 H4 d128) 119 and
// 182, 80 (T300 H16/4) 55 and 57, 102 (T1037 H6/3) 105 and 99; dk's and dv's: 20 (T300 H16/4) 57 and 94, 51 (T1037 H6/3) 99 and 150, 64 (B2
// T1024 H8/2) 158 and 211, 128 (B4 T512 H4 d128 w256) 172 and 156.  So the sides cross between 80 tiles and 102; near there they are
// two microseconds apart, and the border stays at 76, where the rule's reason ends.
// What bounds it: loads from shared memory, 16 bytes a lane take as long as two paired FMAs of every scheduler, and Across<D, 4> has 8 for 32
// (backward of B4 T2048 H8/2 d128 w512: 1,974 us, 30 TFLOP/s of some 77 with the eight products that it forms for five).  Small problems: the longest block's
// tiles, one behind another (T1037 H6/3 d64 w200, 0.73 GFLOP: 99 us, 102 and 210 blocks of four to six tiles).
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

// Which scores and sums a thread has, of a block's rows by 64 others.  Across: 16 x 16 threads, a row's 64 scores in one warp.
template <int D, int R>
struct Across {
    static constexpr int ROWS = 16 * R, NR = R, NC = 4, NU = D / 64;      // rows, scores a row, float4 columns a row
    static constexpr int LANES = 16;                                      // neighbours with the same rows
    static constexpr bool ALONE = true;                                   // no other warp needs a row's scores
    static constexpr int PARTS = 1;                                       // threads that each sum over a part of the 64
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    __device__ __forceinline__ int lane() const { return tx; }
    __device__ __forceinline__ int row(int r) const { return R * ty + r; }
    __device__ __forceinline__ int other(int c) const { return tx + 16 * c; }
    __device__ __forceinline__ int col(int u) const { return 64 * u + 4 * tx; }
    __device__ __forceinline__ int part() const { return 0; }
    __device__ __forceinline__ int group() const { return 0; }
};
// Patches: 16 rows; a warp takes 8 rows by 16 others, and by 32 columns of what is summed (d = 64: over half of the
// others).  A thread loads 4 times for 8 paired FMAs of a product over rows and 6 times for 16 of one over columns, where Across<D, 1> loads
// 5 times for 8, and a load's 8 rows, or columns, are all different (the backward of T1037 H6/3 d64 100 us, 125 with that for
// dk and dv).
template <int D>
struct Patches {
    static constexpr int ROWS = 16, NR = 2, NC = 2, NU = 1, LANES = 8;
    static constexpr bool ALONE = false;
    static constexpr int PARTS = 128 / D;
    const int w = threadIdx.x / 32, lr = threadIdx.x / 8 % 4, lc = threadIdx.x % 8;
    __device__ __forceinline__ int lane() const { return lc; }
    __device__ __forceinline__ int row(int r) const { return 8 * (w & 1) + lr + 4 * r; }
    __device__ __forceinline__ int other(int c) const { return 16 * (w >> 1) + lc + 8 * c; }
    __device__ __forceinline__ int col(int) const { return 32 * ((w >> 1) % (D / 32)) + 4 * lc; }
    __device__ __forceinline__ int part() const { return (w >> 1) / (D / 32); }
    __device__ __forceinline__ int group() const { return w >> 1; }       // of the four with the same rows
};

// acc[r][c] = sum over d of A[row r] B[other c], in sums of 8 of the even and 8 of the odd channels (a score's error is
// its weight's)
template <int D, class M>
__device__ __forceinline__ void rows_by_rows(float (&acc)[M::NR][M::NC], const float *A, const float *B, const M &m) {
    constexpr int S = row_floats<D>(), R = M::NR, C = M::NC;
    float2 sum[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) sum[r][c] = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < D; k0 += 16) {
        float2 x[R][C];
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            float4 a[R], b[C];
#pragma unroll
            for (int r = 0; r < R; ++r) a[r] = load4(A + m.row(r) * S + k0 + k);
#pragma unroll
            for (int c = 0; c < C; ++c) b[c] = load4(B + m.other(c) * S + k0 + k);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float2 a0 = make_float2(a[r].x, a[r].y), b0 = make_float2(b[c].x, b[c].y);
                    x[r][c] = k == 0 ? mul2(a0, b0) : fma2(a0, b0, x[r][c]);
                    x[r][c] = fma2(make_float2(a[r].z, a[r].w), make_float2(b[c].z, b[c].w), x[r][c]);
                }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) sum[r][c] = add2(sum[r][c], x[r][c]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = sum[r][c].x + sum[r][c].y;
}

template <class M> using Sums = float2[M::NR][2 * M::NU];     // of a thread: its rows' columns col(u) .. col(u) + 3

template <class M>
__device__ __forceinline__ void clear(Sums<M> &x) {
#pragma unroll
    for (int r = 0; r < M::NR; ++r)
#pragma unroll
        for (int u = 0; u < 2 * M::NU; ++u) x[r][u] = make_float2(0.f, 0.f);
}

// acc[r][columns] += sum over `n` k (a multiple of 4) of P[row r][k] X[k][columns]
template <int D, class M>
__device__ __forceinline__ void rows_by_cols(Sums<M> &acc, const float *P, const float *X, int n, const M &m) {
    constexpr int S = row_floats<D>(), R = M::NR, U = M::NU, PART = kTile / M::PARTS;
    Sums<M> sum;
    clear<M>(sum);
    const int k0 = PART * m.part(), k1 = min(n, k0 + PART);
#pragma unroll 2
    for (int k = k0; k < k1; k += 4) {
        float p[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 x = load4(P + m.row(r) * kPs + k);
            p[r][0] = x.x; p[r][1] = x.y; p[r][2] = x.z; p[r][3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 x = load4(X + (k + e) * S + m.col(u));
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
        for (int u = 0; u < 2 * U; ++u) acc[r][u] = add2(acc[r][u], sum[r][u]);
}

// The parts' sums added up in those of part 0, by way of shared memory (a block's rows, no longer read).
template <int D, class M>
__device__ __forceinline__ void join_parts(Sums<M> &x, float *sm, const M &m) {
    if constexpr (M::PARTS == 2) {
        __syncthreads();
        if (m.part())
#pragma unroll
            for (int r = 0; r < M::NR; ++r) store4(sm + m.row(r) * row_floats<D>() + m.col(0), make_float4(x[r][0].x, x[r][0].y, x[r][1].x, x[r][1].y));
        __syncthreads();
        if (!m.part())
#pragma unroll
            for (int r = 0; r < M::NR; ++r) {
                const float4 y = load4(sm + m.row(r) * row_floats<D>() + m.col(0));
                x[r][0] = add2(x[r][0], make_float2(y.x, y.y));
                x[r][1] = add2(x[r][1], make_float2(y.z, y.w));
            }
    }
}

// A thread's scores where the others of its rows read them.
template <class M>
__device__ __forceinline__ void put_scores(float *P, const float (&s)[M::NR][M::NC], const M &m) {
#pragma unroll
    for (int r = 0; r < M::NR; ++r)
#pragma unroll
        for (int c = 0; c < M::NC; ++c) P[m.row(r) * kPs + m.other(c)] = s[r][c];
}
// x += P X, y += P2 Y with scores s and s2.
template <int D, class M>
__device__ __forceinline__ void two_sums(Sums<M> &x, const float (&s)[M::NR][M::NC], const float *X, Sums<M> &y,
                                         const float (&s2)[M::NR][M::NC], const float *Y, float *P, int n, const M &m) {
    if constexpr (M::ALONE) {
        __syncwarp();
        put_scores(P, s, m);
        __syncwarp();
        rows_by_cols<D>(x, P, X, n, m);
        __syncwarp();
        put_scores(P, s2, m);
        __syncwarp();
        rows_by_cols<D>(y, P, Y, n, m);
    } else {                                  // (the tile's barrier is behind the last ones' reads)
        put_scores(P, s, m);
        put_scores(P + M::ROWS * kPs, s2, m);
        __syncthreads();
        rows_by_cols<D>(x, P, X, n, m);
        rows_by_cols<D>(y, P + M::ROWS * kPs, Y, n, m);
    }
}

// Over the neighbours with the same rows.
template <class M>
__device__ __forceinline__ float sum_lanes(float x) {
#pragma unroll
    for (int o = M::LANES / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ float max16(float x) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
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

template <class M>
__device__ __forceinline__ void put_rows(float *dst, int64_t stride, int n, const Sums<M> &x, float f, const M &m) {
#pragma unroll
    for (int r = 0; r < M::NR; ++r) {
        if (m.row(r) >= n || m.part()) continue;
#pragma unroll
        for (int u = 0; u < M::NU; ++u)
            store4(dst + m.row(r) * stride + m.col(u), make_float4(f * x[r][2 * u].x, f * x[r][2 * u].y, f * x[r][2 * u + 1].x, f * x[r][2 * u + 1].y));
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
    constexpr int S = row_floats<D>(), ROWS = Across<D, R>::ROWS;
    extern __shared__ float sm[];
    float *Q = sm, *KV = Q + ROWS * S, *P = KV + 4 * kTile * S;
    using M = Across<D, R>;
    static_assert(M::ALONE, "the maxima are a warp's own");
    const M mine;
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
    Sums<M> o;
    clear<M>(o);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
    }
    const int tiles = (keys.total + kTile - 1) / kTile;
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_keys(t + 1);
        umma::cp_async_commit();
        const float *K = KV + (t & 1) * 2 * kTile * S;
        float s[R][4];
        rows_by_rows<D>(s, Q, K, mine);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = q0 + mine.row(r);
            float top = m[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int at = kTile * t + mine.other(c);
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
        __syncwarp();
        put_scores(P, s, mine);
        __syncwarp();
        rows_by_cols<D>(o, P, K + kTile * S, min(kTile, (keys.total - kTile * t + 3) & ~3), mine);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float sum = sum_lanes<M>(l[r]), inv = 1.f / sum;
        const int i = q0 + mine.row(r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[r][c] = mul2(o[r][c], make_float2(inv, inv));
        if (i < len && mine.lane() == 0) p.lse[(lo + i) * p.Hq + h] = m[r] + logf(sum);
    }
    put_rows((float *)p.out + ((lo + q0) * p.Hq + h) * D, (int64_t)p.Hq * D, len - q0, o, 1.f, mine);
}

// dq of a query tile, and of its rows l and delta.  lse and out are rounded, and results of other sums than this kernel's:
// with w_ij = exp(s_ij - lse_i), l = sum_j w_ij is not quite 1 and sum_j w_ij (do_i.v_j - do_i.o_i) not quite 0, which what
// the keys have in common magnifies.  So
//     x_ij = w_ij (do_i.v_j - do_i.o_i),   e = sum_j x_ij / l,   delta_i = do_i.o_i + e,
//     dq_i = scale (sum_j x_ij k_j - e sum_j w_ij k_j) / l,
// a fourth product to three (keys with a common direction of 3 times their spread, sequences of 10 tokens: dq off by 2.5e-6
// without, where all in one arithmetic is off by 1.1e-6).
template <int D, class M>
__global__ void __launch_bounds__(kThreads) attn_simt_dq_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>(), ROWS = M::ROWS, R = M::NR, C = M::NC;
    extern __shared__ float sm[];
    float *Q = sm, *O = Q + ROWS * S, *KV = O + ROWS * S, *P = KV + 4 * kTile * S;
    const M mine;
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
    Sums<M> dq, wk;
    clear<M>(dq);
    clear<M>(wk);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = mine.row(r);
        float x = 0.f;
        if (i < rows) {
#pragma unroll
            for (int c = 4 * mine.lane(); c < D; c += 4 * M::LANES) {
                const float4 a = load4((const float *)p.out + at0 + i * step + c), b = load4((const float *)p.d_out + at0 + i * step + c);
                x += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
            }
        }
        delta[r] = sum_lanes<M>(x);
        lse[r] = i < rows ? p.lse[(lo + q0 + i) * p.Hq + h] : 0.f;
        l[r] = e[r] = 0.f;
    }
    const int tiles = (keys.total + kTile - 1) / kTile;
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_keys(t + 1);
        umma::cp_async_commit();
        const float *K = KV + (t & 1) * 2 * kTile * S;
        float s[R][C], dp[R][C];
        rows_by_rows<D>(s, Q, K, mine);
        rows_by_rows<D>(dp, O, K + kTile * S, mine);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float sw = 0.f, sx = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int at = kTile * t + mine.other(c);
                const bool in = at < keys.total && sees(p, q0 + mine.row(r), keys.at(at));
                s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -lse[r])) : 0.f;
                dp[r][c] = in ? s[r][c] * (dp[r][c] - delta[r]) : 0.f;
                sw += s[r][c];
                sx += dp[r][c];
            }
            l[r] += sw;
            e[r] += sx;
        }
        two_sums<D>(wk, s, K, dq, dp, K, P, min(kTile, (keys.total - kTile * t + 3) & ~3), mine);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        l[r] = sum_lanes<M>(l[r]);
        e[r] = sum_lanes<M>(e[r]);
    }
    if constexpr (!M::ALONE) {                // over the warps with the same rows
        __syncthreads();
        float2 *all = reinterpret_cast<float2 *>(P);
        if (mine.lane() == 0)
#pragma unroll
            for (int r = 0; r < R; ++r) all[4 * mine.row(r) + mine.group()] = make_float2(l[r], e[r]);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 *a = all + 4 * mine.row(r);
            l[r] = (a[0].x + a[1].x) + (a[2].x + a[3].x);
            e[r] = (a[0].y + a[1].y) + (a[2].y + a[3].y);
        }
    }
    join_parts<D>(dq, KV, mine);
    join_parts<D>(wk, KV, mine);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int i = mine.row(r);
        const float inv = 1.f / l[r], x = e[r] * inv;
        if (mine.lane() == 0 && mine.group() == 0 && i < rows) {
            const int64_t at = h * p.seqs.total + lo + q0 + i;
            p.delta[at] = delta[r] + x;
            p.inv_l[at] = inv;
        }
#pragma unroll
        for (int c = 0; c < 2 * M::NU; ++c) dq[r][c] = mul2(fma2(make_float2(-x, -x), wk[r][c], dq[r][c]), make_float2(inv, inv));
    }
    put_rows((float *)p.dq + (lo + q0) * p.dqs + h * D, p.dqs, rows, dq, p.scale, mine);
}

// dk and dv of a key tile, over the block's queries and all heads that share the keys.
template <int D, class M>
__global__ void __launch_bounds__(kThreads) attn_simt_dkv_kernel(const AttnProblem p, const attn::SinkPlan plan) {
    constexpr int S = row_floats<D>(), ROWS = M::ROWS, R = M::NR, C = M::NC;
    extern __shared__ float sm[];
    float *K = sm, *V = K + ROWS * S, *QO = V + ROWS * S, *P = QO + 4 * kTile * S, *stat = P + (M::ALONE ? 1 : 2) * ROWS * kPs;   // [2][lse, delta, 1 / l][64]
    const M mine;
    const int g = p.Hq / p.Hk;
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
    Sums<M> dk, dv;
    clear<M>(dk);
    clear<M>(dv);
    for (int t = 0; t < tiles; ++t) {
        umma::cp_async_wait_all();
        __syncthreads();
        if (t + 1 < tiles) fetch_queries(t + 1);
        umma::cp_async_commit();
        const int q0 = kb.qa + t % nt * kTile, n = min(kTile, (kb.qb - q0 + 3) & ~3);
        const float *Q = QO + (t & 1) * 2 * kTile * S, *O = Q + kTile * S, *st = stat + (t & 1) * 3 * kTile;
        float s[R][C], dp[R][C];
        rows_by_rows<D>(s, K, Q, mine);
        rows_by_rows<D>(dp, V, O, mine);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int qi = mine.other(c), j = k0 + mine.row(r);
                const bool in = q0 + qi < kb.qb && sees(p, q0 + qi, j) && (kb.chunk < 0 || j < p.sinks);
                s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -st[qi])) * st[2 * kTile + qi] : 0.f;
                dp[r][c] = in ? s[r][c] * (dp[r][c] - st[kTile + qi]) : 0.f;
            }
        two_sums<D>(dv, s, O, dk, dp, Q, P, n, mine);
    }
    join_parts<D>(dk, QO, mine);
    join_parts<D>(dv, QO, mine);
    // a sink's row is a part of a sum where its queries are cut
    const int sinks = kb.cut ? min(p.sinks - k0, rows) : 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = mine.row(r);
        const bool part = row < sinks;
        if (row >= rows || (kb.chunk >= 0 && !part) || mine.part()) continue;
        float *to_k = part ? kb.sum(p, plan, k0 + row) : (float *)p.dk + (lo + k0 + row) * p.dks + hk * D;
        float *to_v = part ? to_k + D : (float *)p.dv + (lo + k0 + row) * p.dvs + hk * D;
#pragma unroll
        for (int u = 0; u < M::NU; ++u) {
            const float2 a = mul2(dk[r][2 * u], make_float2(p.scale, p.scale)), b = mul2(dk[r][2 * u + 1], make_float2(p.scale, p.scale));
            store4(to_k + mine.col(u), make_float4(a.x, a.y, b.x, b.y));
            store4(to_v + mine.col(u), make_float4(dv[r][2 * u].x, dv[r][2 * u].y, dv[r][2 * u + 1].x, dv[r][2 * u + 1].y));
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
template <int D, class M>
int bwd_q(const AttnProblem &p, cudaStream_t s) {
    return launch(attn_simt_dq_kernel<D, M>, floats<D>(2, M::ROWS) + (M::ALONE ? 0 : M::ROWS * kPs), attn_tile_slots(p.seqs, M::ROWS) * p.Hq, s, p);
}

int key_rows(const AttnProblem &p) { return few(p, p.Hk) ? 16 : 64; }
// delta, or 1 / l
size_t stat_bytes(const AttnProblem &p) { return attn::round256(sizeof(float) * (size_t)(p.seqs.total * p.Hq)); }

template <int D>
int bwd(const AttnProblem &p, void *workspace, cudaStream_t s) {
    int rc = few(p, p.Hq) ? bwd_q<D, Patches<D>>(p, s) : bwd_q<D, Across<D, 4>>(p, s);
    if (rc != kOk) return rc;
    attn::SinkPlan plan;
    attn::plan_sinks(p, key_rows(p), 256, (char *)workspace + 2 * stat_bytes(p), plan);
    const int64_t blocks = attn::key_blocks(p, plan);
    rc = plan.tile == 16 ? launch_next(attn_simt_dkv_kernel<D, Patches<D>>, floats<D>(2, 16) + 16 * kPs + 6 * kTile, blocks, s, p, plan)
                         : launch_next(attn_simt_dkv_kernel<D, Across<D, 4>>, floats<D>(2, 64) + 6 * kTile, blocks, s, p, plan);
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
