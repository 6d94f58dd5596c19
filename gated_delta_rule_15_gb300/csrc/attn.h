// attn.h -- what the kernels and the C ABI of the window attention share.
//
// Of a sequence, query i sees key j when
//     j <= i  and  (i - j < window  or  j < sinks),
// and with s_ij = scale q_i.k_j over the visible keys
//     lse_i = log sum_j exp s_ij,   p_ij = exp(s_ij - lse_i),   o_i = sum_j p_ij v_j.
// Gradients, with delta_i = do_i.o_i:
//     ds_ij = p_ij (do_i.v_j - delta_i),
//     dq_i = scale sum_j ds_ij k_j,   dk_j = scale sum_i ds_ij q_i,   dv_j = sum_i p_ij do_i,
// the last two also over the query heads that share the key head.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "linrec.h"   // LinrecSeqs, seq_range

namespace dr {

constexpr int kNoWindow = 1 << 30;   // above any distance within a sequence of this library's calls
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttnProblem {
    LinrecSeqs seqs;
    int Hq, Hk, d, window, sinks;      // window kNoWindow: none
    float scale;
    bool bf16;
    const void *q, *k, *v;             // rows qs, ks, vs elements apart
    int64_t qs, ks, vs;
    void *out;                         // [rows, Hq, d]; read by the backward
    float *lse;                        // [rows, Hq]; read by the backward
    const void *d_out;                 // [rows, Hq, d]
    void *dq, *dk, *dv;                // rows dqs, dks, dvs elements apart
    int64_t dqs, dks, dvs;
    float *delta, *inv_l;              // (workspace, fp32 rows) [Hq][rows]; inv_l: attn_simt.cu
};

#ifdef __CUDACC__
// The sequences are cut into tiles of TILE tokens; tile j of sequence n has the slot
// lo / TILE + n + j (packed; lo its first row) or n * tiles + j, which no other has.
__host__ __device__ inline int64_t attn_tile_slots(const LinrecSeqs &s, int tile) {
    return s.cu ? s.total / tile + s.N : s.N * ((s.T + tile - 1) / tile);
}
// The last of the packed sequences whose key(n, first row) is at most `slot`, and its rows; keys do not fall.  By
// whole warps: 32 sequences are asked at a time.
template <class Key>
__device__ __forceinline__ int64_t last_sequence(const LinrecSeqs &s, int slot, Key key, int64_t &lo, int &len) {
    int64_t a = 0, b = s.N - 1, hi;
    while (a < b) {
        const int64_t step = (b - a + 31) >> 5, m = a + 1 + (threadIdx.x & 31) * step;
        bool in = false;
        if (m <= b) {
            seq_range(s, m, lo, hi);
            in = key(m, lo) <= slot;
        }
        const int k = __popc(__ballot_sync(0xffffffffu, in));
        b = min(b, a + k * step);
        if (k > 0) a += 1 + (k - 1) * step;
    }
    seq_range(s, a, lo, hi);
    len = (int)(hi - lo);
    return a;
}
// Finds (n, j) of a slot and the sequence's rows, or false where the slot has no tile.  By whole
// warps.  Rows and slots fit in 31 bits.
__device__ __forceinline__ bool find_tile(const LinrecSeqs &s, int tile, int slot, int64_t &n, int &j, int64_t &lo, int &len) {
    if (!s.cu) {
        const int per = (int)((s.T + tile - 1) / tile);
        n = slot / per;
        j = slot - (int)n * per;
        lo = n * s.T;
        len = (int)s.T;
        return true;
    }
    // the first slot of a sequence is lo / tile + n
    n = last_sequence(s, slot, [&](int64_t m, int64_t at) { return (uint32_t)at / (uint32_t)tile + m; }, lo, len);
    j = slot - (int)((uint32_t)lo / (uint32_t)tile + n);
    return j >= 0 && (int64_t)j * tile < len;
}
#endif

// CUDA cores: fp32 rows.
int launch_attn_simt_fwd(const AttnProblem &p, cudaStream_t stream);
size_t attn_simt_bwd_workspace_bytes(const AttnProblem &p);   // (by seqs.cu being NULL or not, not what it holds)
int launch_attn_simt_bwd(const AttnProblem &p, void *workspace, cudaStream_t stream);

// Zeroes the rows of no sequence of a packed problem: `n` buffers of `bytes[i]` bytes a row,
// `stride[i]` bytes apart (both multiples of 4; a NULL buffer is passed over).
struct AttnRest {
    void *p[3];
    int64_t bytes[3], stride[3];
};
int launch_attn_zero_rest(const LinrecSeqs &s, const AttnRest &r, cudaStream_t stream);

// One token for each sequence over a paged cache.
struct AttnStep {
    int64_t B;
    int Hq, Hk, d, page, max_pages, window, sinks;
    int64_t n_pages;
    float scale;
    bool bf16;
    const void *q, *kc, *vc;
    const int *pages;
    const int64_t *lens;
    void *out;
    float *lse;
};
size_t attn_step_workspace_bytes(const AttnStep &p);
int launch_attn_step(const AttnStep &p, void *workspace, int *status, cudaStream_t stream);

}  // namespace dr
