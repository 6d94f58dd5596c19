// attn_simt.cu -- window attention on the CUDA cores (fp32 rows): forward, gradients.  The
// mathematics: attn.h.
//
// Tiles of 64 queries by 64 keys, 256 threads as 16 x 16: a thread holds 4 x 4 scores (queries
// 4 ty + r, keys tx + 16 c) and 4 rows x d / 16 columns of what is summed.  Products run over rows in
// shared memory as float4 of both operands (64 FMAs per 8 loads of 16 bytes), whose row stride of
// d + 4 floats keeps the 16 keys of a load on different banks.
// A query's keys come in one pass, first the sinks in front of its tile's window, then the window,
// with the running maximum and sum of the softmax in registers.
#include "../../include/dr.h"
#include "attn.h"
#include "common.cuh"

namespace dr {
namespace {

constexpr int kTile = 64, kThreads = 256, kPs = kTile + 4;

template <int D> constexpr int row_floats() { return D + 4; }

// Rows row0 .. row0 + n - 1 of one head as fp32, zeros behind them.
template <int D, typename T>
__device__ __forceinline__ void load_tile(float *dst, const T *src, int64_t stride, int n) {
    constexpr int PER = D / 4;
#pragma unroll
    for (int i = threadIdx.x; i < kTile * PER; i += kThreads) {
        const int r = i / PER, c = i % PER;
        const float4 x = r < n ? load4(src + (int64_t)r * stride + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        store4(dst + r * row_floats<D>() + 4 * c, x);
    }
}

// acc[r][c] = sum over d of A[4 ty + r] B[tx + 16 c]
template <int D>
__device__ __forceinline__ void rows_by_rows(float (&acc)[4][4], const float *A, const float *B, int ty, int tx) {
    constexpr int S = row_floats<D>();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[r][c] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = load4(A + (4 * ty + r) * S + k);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = load4(B + (tx + 16 * c) * S + k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                acc[r][c] = fmaf(a[r].x, b[c].x, acc[r][c]);
                acc[r][c] = fmaf(a[r].y, b[c].y, acc[r][c]);
                acc[r][c] = fmaf(a[r].z, b[c].z, acc[r][c]);
                acc[r][c] = fmaf(a[r].w, b[c].w, acc[r][c]);
            }
    }
}

// acc[r][4 u + e] += sum over 64 k of P[4 ty + r][k] X[k][64 u + 4 tx + e]
template <int D>
__device__ __forceinline__ void rows_by_cols(float (&acc)[4][D / 16], const float *P, const float *X, int ty, int tx) {
    constexpr int S = row_floats<D>(), U = D / 64;
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        float p[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 x = load4(P + (4 * ty + r) * kPs + k);
            p[r][0] = x.x; p[r][1] = x.y; p[r][2] = x.z; p[r][3] = x.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 x = load4(X + (k + e) * S + 64 * u + 4 * tx);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[r][4 * u] = fmaf(p[r][e], x.x, acc[r][4 * u]);
                    acc[r][4 * u + 1] = fmaf(p[r][e], x.y, acc[r][4 * u + 1]);
                    acc[r][4 * u + 2] = fmaf(p[r][e], x.z, acc[r][4 * u + 2]);
                    acc[r][4 * u + 3] = fmaf(p[r][e], x.w, acc[r][4 * u + 3]);
                }
            }
    }
}

__device__ __forceinline__ void put_scores(float *P, const float (&s)[4][4], int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) P[(4 * ty + r) * kPs + tx + 16 * c] = s[r][c];
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

// The key tiles of a query tile: sinks in front of the window of its first query, then the keys
// from there to its last query.
struct KeyTiles {
    int sinks, n_sink, near0, end, n;
    __device__ KeyTiles(const AttnProblem &p, int q0, int len) {
        near0 = max(0, q0 - p.window + 1);
        sinks = min(p.sinks, near0);
        end = min(len, q0 + kTile);
        n_sink = (sinks + kTile - 1) / kTile;
        n = n_sink + (end - near0 + kTile - 1) / kTile;
    }
    __device__ void get(int t, int &k0, int &count) const {
        k0 = t < n_sink ? t * kTile : near0 + (t - n_sink) * kTile;
        count = min(kTile, (t < n_sink ? sinks : end) - k0);
    }
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) attn_simt_fwd_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>();
    extern __shared__ float sm[];
    float *Q = sm, *KV = Q + kTile * S, *P = KV + kTile * S;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, h = blockIdx.x % p.Hq, hk = h / (p.Hq / p.Hk);
    int64_t n, lo;
    int j, len;
    if (!find_tile(p.seqs, kTile, blockIdx.x / p.Hq, n, j, lo, len)) return;
    const int q0 = j * kTile;
    load_tile<D>(Q, (const T *)p.q + (lo + q0) * p.qs + h * D, p.qs, len - q0);
    float m[4], l[4], o[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[r][c] = 0.f;
    }
    const KeyTiles tiles(p, q0, len);
    for (int t = 0; t < tiles.n; ++t) {
        int k0, count;
        tiles.get(t, k0, count);
        __syncthreads();
        load_tile<D>(KV, (const T *)p.k + (lo + k0) * p.ks + hk * D, p.ks, count);
        __syncthreads();
        float s[4][4];
        rows_by_rows<D>(s, Q, KV, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = q0 + 4 * ty + r;
            float top = m[r];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int kj = tx + 16 * c;
                s[r][c] = kj < count && sees(p, i, k0 + kj) ? p.scale * s[r][c] : -INFINITY;
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
            for (int c = 0; c < D / 16; ++c) o[r][c] *= turn;
        }
        put_scores(P, s, ty, tx);
        __syncthreads();
        load_tile<D>(KV, (const T *)p.v + (lo + k0) * p.vs + hk * D, p.vs, count);
        __syncthreads();
        rows_by_cols<D>(o, P, KV, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float sum = sum16(l[r]), inv = 1.f / sum;
        const int i = q0 + 4 * ty + r;
        if (i >= len) continue;
        T *dst = (T *)p.out + ((lo + i) * p.Hq + h) * D;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            store4(dst + 64 * u + 4 * tx, make_float4(o[r][4 * u] * inv, o[r][4 * u + 1] * inv, o[r][4 * u + 2] * inv, o[r][4 * u + 3] * inv));
        if (tx == 0) p.lse[(lo + i) * p.Hq + h] = m[r] + logf(sum);
    }
}

template <int D, typename T>
__device__ __forceinline__ void put_rows(T *dst, int64_t stride, int n, const float (&x)[4][D / 16], float f, int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (4 * ty + r >= n) continue;
#pragma unroll
        for (int u = 0; u < D / 64; ++u)
            store4(dst + (int64_t)(4 * ty + r) * stride + 64 * u + 4 * tx,
                   make_float4(f * x[r][4 * u], f * x[r][4 * u + 1], f * x[r][4 * u + 2], f * x[r][4 * u + 3]));
    }
}

// dq of a query tile, and delta of its rows.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) attn_simt_dq_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>();
    extern __shared__ float sm[];
    float *Q = sm, *O = Q + kTile * S, *K = O + kTile * S, *V = K + kTile * S, *P = V + kTile * S;
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, h = blockIdx.x % p.Hq, hk = h / (p.Hq / p.Hk);
    int64_t n, lo;
    int j, len;
    if (!find_tile(p.seqs, kTile, blockIdx.x / p.Hq, n, j, lo, len)) return;
    const int q0 = j * kTile, rows = len - q0;
    load_tile<D>(K, (const T *)p.out + ((lo + q0) * p.Hq + h) * D, (int64_t)p.Hq * D, rows);   // (K's place is free)
    load_tile<D>(O, (const T *)p.d_out + ((lo + q0) * p.Hq + h) * D, (int64_t)p.Hq * D, rows);
    load_tile<D>(Q, (const T *)p.q + (lo + q0) * p.qs + h * D, p.qs, rows);
    __syncthreads();
    float delta[4], lse[4], dq[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 4 * ty + r;
        float x = 0.f;
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
            const float4 a = load4(K + i * S + 64 * u + 4 * tx), b = load4(O + i * S + 64 * u + 4 * tx);
            x += a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
        }
        delta[r] = sum16(x);
        lse[r] = 0.f;
        if (i < rows) {
            lse[r] = p.lse[(lo + q0 + i) * p.Hq + h];
            if (tx == 0) p.delta[h * p.seqs.total + lo + q0 + i] = delta[r];
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dq[r][c] = 0.f;
    }
    const KeyTiles tiles(p, q0, len);
    for (int t = 0; t < tiles.n; ++t) {
        int k0, count;
        tiles.get(t, k0, count);
        __syncthreads();
        load_tile<D>(K, (const T *)p.k + (lo + k0) * p.ks + hk * D, p.ks, count);
        load_tile<D>(V, (const T *)p.v + (lo + k0) * p.vs + hk * D, p.vs, count);
        __syncthreads();
        float s[4][4], dp[4][4];
        rows_by_rows<D>(s, Q, K, ty, tx);
        rows_by_rows<D>(dp, O, V, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int kj = tx + 16 * c;
                const bool in = kj < count && sees(p, q0 + 4 * ty + r, k0 + kj);
                s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -lse[r])) * (dp[r][c] - delta[r]) : 0.f;
            }
        put_scores(P, s, ty, tx);
        __syncthreads();
        rows_by_cols<D>(dq, P, K, ty, tx);
    }
    put_rows<D>((T *)p.dq + (lo + q0) * p.dqs + h * D, p.dqs, rows, dq, p.scale, ty, tx);
}

// dk and dv of a key tile, over all queries that see a key of it and all heads that share it.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads) attn_simt_dkv_kernel(const AttnProblem p) {
    constexpr int S = row_floats<D>();
    extern __shared__ float sm[];
    float *Q = sm, *O = Q + kTile * S, *K = O + kTile * S, *V = K + kTile * S, *P = V + kTile * S;
    __shared__ float lse[kTile], delta[kTile];
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16, hk = blockIdx.x % p.Hk, g = p.Hq / p.Hk;
    int64_t n, lo;
    int j, len;
    if (!find_tile(p.seqs, kTile, blockIdx.x / p.Hk, n, j, lo, len)) return;
    const int k0 = j * kTile, rows = len - k0;
    load_tile<D>(K, (const T *)p.k + (lo + k0) * p.ks + hk * D, p.ks, rows);
    load_tile<D>(V, (const T *)p.v + (lo + k0) * p.vs + hk * D, p.vs, rows);
    float dk[4][D / 16], dv[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < D / 16; ++c) dk[r][c] = dv[r][c] = 0.f;
    const int end = k0 < p.sinks ? len : min(len, k0 + kTile - 1 + p.window);
    for (int h = hk * g; h < (hk + 1) * g; ++h)
        for (int q0 = k0; q0 < end; q0 += kTile) {
            const int count = len - q0;
            __syncthreads();
            load_tile<D>(Q, (const T *)p.q + (lo + q0) * p.qs + h * D, p.qs, count);
            load_tile<D>(O, (const T *)p.d_out + ((lo + q0) * p.Hq + h) * D, (int64_t)p.Hq * D, count);
            if (threadIdx.x < kTile) {
                const bool in = (int)threadIdx.x < count;
                lse[threadIdx.x] = in ? p.lse[(lo + q0 + threadIdx.x) * p.Hq + h] : 0.f;
                delta[threadIdx.x] = in ? p.delta[h * p.seqs.total + lo + q0 + threadIdx.x] : 0.f;
            }
            __syncthreads();
            float s[4][4], dp[4][4];
            rows_by_rows<D>(s, K, Q, ty, tx);
            rows_by_rows<D>(dp, V, O, ty, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int qi = tx + 16 * c;
                    const bool in = qi < count && sees(p, q0 + qi, k0 + 4 * ty + r);
                    s[r][c] = in ? expf(fmaf(s[r][c], p.scale, -lse[qi])) : 0.f;
                    dp[r][c] = s[r][c] * (dp[r][c] - delta[qi]);
                }
            put_scores(P, s, ty, tx);
            __syncthreads();
            rows_by_cols<D>(dv, P, O, ty, tx);
            __syncthreads();
            put_scores(P, dp, ty, tx);
            __syncthreads();
            rows_by_cols<D>(dk, P, Q, ty, tx);
        }
    put_rows<D>((T *)p.dk + (lo + k0) * p.dks + hk * D, p.dks, rows, dk, p.scale, ty, tx);
    put_rows<D>((T *)p.dv + (lo + k0) * p.dvs + hk * D, p.dvs, rows, dv, 1.f, ty, tx);
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

template <class F>
int launch(F *kernel, size_t smem, int64_t blocks, const AttnProblem &p, cudaStream_t s) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return kErrCuda;
    kernel<<<(unsigned)blocks, kThreads, smem, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}
template <int D> constexpr size_t smem_bytes(int tiles) { return sizeof(float) * (tiles * kTile * row_floats<D>() + kTile * kPs); }

template <int D, typename T>
int bwd(const AttnProblem &p, cudaStream_t s) {
    const int64_t slots = attn_tile_slots(p.seqs, kTile);
    const int rc = launch(attn_simt_dq_kernel<D, T>, smem_bytes<D>(4), slots * p.Hq, p, s);
    return rc != kOk ? rc : launch(attn_simt_dkv_kernel<D, T>, smem_bytes<D>(4), slots * p.Hk, p, s);
}

}  // namespace

int launch_attn_simt_fwd(const AttnProblem &p, cudaStream_t s) {
    const int64_t blocks = attn_tile_slots(p.seqs, kTile) * p.Hq;
    return p.d == 64 ? launch(attn_simt_fwd_kernel<64, float>, smem_bytes<64>(2), blocks, p, s)
                     : launch(attn_simt_fwd_kernel<128, float>, smem_bytes<128>(2), blocks, p, s);
}

int launch_attn_simt_bwd(const AttnProblem &p, cudaStream_t s) {
    return p.d == 64 ? bwd<64, float>(p, s) : bwd<128, float>(p, s);
}

int launch_attn_zero_rest(const LinrecSeqs &s, const AttnRest &r, cudaStream_t stream) {
    attn_zero_rest_kernel<<<152, 256, 0, stream>>>(s, r);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace dr
