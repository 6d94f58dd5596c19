// linrec.h -- what the kernels and the C ABI of the additive gated linear recurrence
//     S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t        (a_t = exp(log_alpha_t) or 1)
// share.
//
// One pass serves the forward and all three token gradients.  With dS_t = dL/dS_t,
//     dS_t = a_{t+1} dS_{t+1} + q_t do_t^T,
//     dq_t = S_t do_t,   dk_t = dS_t v_t,   dv_t = dS_t^T k_t,   dS_0 = a_1 dS_1,
// so with (q, k, v) standing for the pass's queries, keys and values
//     out: pass(q, k, v)          forwards,  state S
//     dq:  pass(do, v, k)         forwards,  state S^T
//     dk:  pass(v, do, q)         backwards, state dS^T
//     dv:  pass(k, q, do)         backwards, state dS
// where a backwards pass decays by a_{t+1} in front of token t.
//
// The log-decay gradient is <a_t S_{t-1}, dS_t>.  Scaling every S_t behind a token by a
// common factor shows that it telescopes: with x_r = q_r.dq_r - k_r.dk_r,
//     dlog a_t = x_t + ... + x_{e-1} + <S_{e-1}, dL/dS_{e-1}>
// for any e > t (dL/dS_{e-1} without the output of token e-1).  Both dot products hold the
// same term (do_r.v_r)(q_r.k_r) of the token itself; it is left out of both, so that a
// strong decay's small gradient is no difference of large numbers.  The sums run over at
// most `run` tokens: the dq pass stores S at every such boundary and the dk pass, which
// holds the same entries of dS there, adds the inner product.  Where a_t is 0 the gradient is set
// to 0: the sums are 0 there in exact arithmetic only.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dr {

// Tokens between two stored states of the log-decay gradient, on the tensor cores and in the token
// recurrence.  The sums' rounding grows with the root of it: of fp32 rows the gradient is 0.3e-6 to 0.8e-6 off
// in the 2-norm (256 tokens: up to 1.1e-6); the chunks, for which the states' traffic counts, are 0.5e-6 to
// 0.9e-6 off with 256.
constexpr int kAnchor = 256, kTokenAnchor = 128;

// The sequences of a problem: N of them, packed by `cu` (N + 1 device offsets into `total`
// rows) or T rows each.  Offsets from the device are clamped into the rows that exist.
struct LinrecSeqs {
    const int64_t *cu;
    int64_t N, T, total;
};

#ifdef __CUDACC__
__device__ __forceinline__ void seq_range(const LinrecSeqs &s, int64_t n, int64_t &lo, int64_t &hi) {
    if (s.cu) {
        lo = min(max(s.cu[n], (int64_t)0), s.total);
        hi = min(max(s.cu[n + 1], lo), s.total);
    } else {
        lo = n * s.T;
        hi = lo + s.T;
    }
}
#endif
// Slot of the stored state at the end of sequence n's `j`-th run of `run` tokens; two
// sequences never share one, and there are linrec_slots() of them.
__host__ __device__ inline int64_t linrec_slot(int run, int64_t lo, int64_t n, int64_t j) { return lo / run + n + j; }
__host__ __device__ inline int64_t linrec_slots(int run, const LinrecSeqs &s) { return s.total / run + s.N + 1; }

struct LinrecPass {
    LinrecSeqs seqs;
    int H, dk, dv;               // the pass's own key and value widths
    bool in_bf16, out_bf16, rev;
    const void *q, *k, *v;       // [rows, H, dk | dk | dv]
    const float *la;             // [rows, H] or NULL
    const float *init;           // state before the first (backwards: after the last) token, or NULL
    float *fin;                  // state at the other end, or NULL
    bool state_t;                // init and fin hold the transposed state
    bool chained;                // the workspace still holds the segments' start states: the pass before had this state
    void *out;                   // [rows, H, dv]
    // log-decay gradient, in the dq and dk passes: dot[part][h][row] = sum over the part's
    // value columns of out without the row's own term, times y [rows, H, dv]
    const void *y;
    float *dot;
    float *anchor;               // the stored states; written forwards, read backwards
    float *inner;                // backwards: [part][slot][h] inner products
};

// CUDA-core token recurrence: every type and width.
constexpr int kSimtCols = 64;    // value columns of one CTA (one "part" of dot and inner)
int launch_linrec_simt(const LinrecPass &p, cudaStream_t stream);

// Tensor cores: bf16 rows and outputs.  One part.  `status`: the library's device status word.
bool linrec_tc_supported(const LinrecSeqs &s, int64_t H, bool in_bf16, bool out_bf16);
size_t linrec_tc_workspace_bytes(const LinrecSeqs &s, int64_t H, int dk, int dv);
int launch_linrec_tc(const LinrecPass &p, void *workspace, int *status, cudaStream_t stream);

// dlog a from the two passes' dot products and the inner products of runs of `run` tokens; `parts` of each.
int launch_linrec_gate_grad(const LinrecSeqs &s, int H, int run, int parts, const float *la, const float *dot_q,
                            const float *dot_k, const float *inner, float *dla, cudaStream_t stream);

// Zeroes the rows of no sequence of `rows` (row_bytes a multiple of 16) and `gates` (words a row), where given.
struct LinrecRest {
    void *rows[3];
    int64_t row_bytes[3];
    float *gates;
    int64_t gate_words;
};
int launch_linrec_zero_rest(const LinrecSeqs &s, const LinrecRest &r, cudaStream_t stream);

int launch_linrec_step(int64_t chains, int dk, int dv, bool in_bf16, bool out_bf16, const void *q, const void *k,
                       const void *v, const float *la, float *state, void *out, cudaStream_t stream);

}  // namespace dr
