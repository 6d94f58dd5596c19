/*
 * dr.h -- C ABI of the GB300 (sm_103a) gated delta rule library, libdr.so.
 *
 * The operation (page "NLP: linear attention summary", sections "DeltaNet", "Gated
 * DeltaNet" and "Kimi Delta Attention"):
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T,
 *     o_t = S_t^T q_t,
 *
 * per (batch b, head h), with the state S in R^{dk x dv}.  alpha_t is a scalar per head and
 * token (Gated DeltaNet), a dk-vector (KDA, per-channel gate) or 1 (DeltaNet).  The order
 * is decay, predict with the decayed state, write the beta-scaled residual, read after the
 * write (teaching loop `gated_delta_rule`, page "linear-attention gated-deltanet guide",
 * section 4).  The chunkwise-parallel form evaluated by dr_chunk_fwd (section 5 of the same
 * page; the WY representation and triangular solve named on the page "Transformer notes
 * (5): linear attention optimisations") reaches the same result up to rounding.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers (cudaMalloc / torch CUDA memory) on the
 *     current device, contiguous, row-major, 16-byte aligned.  The caller owns every
 *     buffer; the library never allocates, frees or synchronises (except
 *     dr_get_device_status) and keeps no host-side state between calls.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream).  A status of DR_OK means the work was validated and enqueued.
 *   - Token-major layouts, the layout a projection GEMM writes:
 *       q, k        [B, T, H, dk]    in_dtype
 *       v           [B, T, H, dv]    in_dtype
 *       beta        [B, T, H]        in_dtype, values in [0, 1] (logits under
 *                                    DR_FUSE_BETA_SIGMOID)
 *       log_alpha   [B, T, H] (DR_GATE_SCALAR) or [B, T, H, dk] (DR_GATE_CHANNEL), fp32,
 *                   values <= 0; NULL for DR_GATE_NONE
 *       out         [B, T, H, dv]    out_dtype
 *       states      [B, H, dk, dv]   fp32 (row i = key channel, column j = value channel)
 *     The decode entry point drops the T axis.
 *   - Inputs are assumed finite; log_alpha <= 0 and beta in [0, 1] are not checked.
 *   - Errors are returned before anything is enqueued: nothing is launched on a
 *     negative status.
 */
#ifndef DR_H_
#define DR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle as cudaStream_t. */
typedef struct CUstream_st *dr_stream_t;

/* Storage dtypes. */
enum { DR_F32 = 0, DR_BF16 = 1 };

/* Gate kinds: no gate (DeltaNet), scalar per head and token (Gated DeltaNet),
   per key channel (KDA). */
enum { DR_GATE_NONE = 0, DR_GATE_SCALAR = 1, DR_GATE_CHANNEL = 2 };

/* Status codes. */
enum {
    DR_OK = 0,
    DR_ERR_INVALID = -1,      /* null pointer, bad size, misaligned pointer, bad enum   */
    DR_ERR_UNSUPPORTED = -2,  /* valid but not built: dk, dv not in {64, 128}, chunk    */
    DR_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed                   */
    DR_ERR_TIMEOUT = -4,      /* a bounded device-side wait expired (device status)     */
    DR_ERR_WORKSPACE = -5     /* workspace missing or smaller than the query's answer   */
};

/* Problem descriptor of the chunkwise forward. */
typedef struct {
    int64_t B, T, H, dk, dv;  /* B, H >= 1; T >= 0; dk, dv in {64, 128}                */
    int32_t in_dtype;         /* DR_F32 or DR_BF16: q, k, v, beta                       */
    int32_t out_dtype;        /* DR_F32 or DR_BF16: out                                 */
    int32_t gate;             /* DR_GATE_*                                              */
    int32_t chunk;            /* chunk length C: 16, 32 or 64; 0 selects 64             */
} dr_chunk_desc;

/* Problem descriptor of one decode step. */
typedef struct {
    int64_t B, H, dk, dv;     /* B, H >= 1; dk, dv in {64, 128}                         */
    int32_t in_dtype;         /* DR_F32 or DR_BF16: q, k, v, beta                       */
    int32_t out_dtype;        /* DR_F32 or DR_BF16: out                                 */
    int32_t gate;             /* DR_GATE_*                                              */
    int32_t reserved;         /* must be 0                                              */
} dr_step_desc;

/*
 * Fused neighbours of the operation: the steps on either side of it in a Gated DeltaNet
 * layer (page "linear-attention gated-deltanet guide", section 4: the write gate beta, the
 * read-out gated by SiLU; q and k enter L2-normalised), applied inside the kernels of
 * dr_chunk_fwd_ex and dr_recurrent_step_ex, with no extra pass over memory.  OR-ed into
 * their `fuse` argument:
 *   DR_FUSE_QK_L2NORM      every q and k row (dk values) is divided by
 *                          sqrt(sum of squares + DR_L2NORM_EPS), in fp32, before use
 *   DR_FUSE_BETA_SIGMOID   `beta` holds logits (any finite value, in_dtype); the kernels
 *                          use beta = 1 / (1 + exp(-logit)) rounded to in_dtype, the
 *                          value a beta stored before the call would hold
 *   DR_FUSE_OUT_SILU_GATE  out = o * z * sigmoid(z), elementwise, with `z` laid out as
 *                          out ([B, T, H, dv], or [B, H, dv] for a step) in in_dtype
 * The state (init_state, final_state, the decode state) is never gated: only `out` is.
 */
enum { DR_FUSE_QK_L2NORM = 1, DR_FUSE_BETA_SIGMOID = 2, DR_FUSE_OUT_SILU_GATE = 4 };
#define DR_FUSE_ALL 7u
#define DR_L2NORM_EPS 1e-6f

/* Library version, (major << 16) | minor. */
int dr_version(void);

/* Bytes of device workspace dr_chunk_fwd takes for *desc on its fastest path; written to
   *bytes.  The answer depends only on the descriptor.  Returns DR_OK, DR_ERR_INVALID or
   DR_ERR_UNSUPPORTED.
   Few long chains (at most 76 for the tensor-core paths, at least 32 chunks each) are split
   into segments that run side by side; each (b, h, segment) then takes three dk x dv fp32
   states (the segment's transition dk x dk, its end state from a zero start, its start
   state).  Besides those:
     - bf16 inputs, dk = dv = 128, chunk 64, scalar or no gate: nothing for many chains; for
       chains split into segments, also 16.5 KB per (b, h, chunk): every chunk's
       triangular-solve operands (T = (I + A)^-1 of the WY form, page "Transformer notes
       (5): linear attention optimisations", KDA paragraph), formed for all chunks at once,
       and the row norms of the fused L2 norm;
     - the same with the per-channel gate: 131,584 bytes of tensor-core operands per
       (b, h, chunk);
     - every other configuration (the CUDA-core path): the fp32 operands W, Q*G, K*G_C/G
       [C][dk], U [C][dv], P [C][C] and G_C [dk] per (b, h, chunk). */
int dr_chunk_fwd_workspace_bytes(const dr_chunk_desc *desc, size_t *bytes);

/* The least workspace dr_chunk_fwd accepts for *desc; written to *bytes.  Equal to
   dr_chunk_fwd_workspace_bytes() except for the scalar / no-gate tensor-core configuration
   with chains split into segments, where a workspace below that size (but at least this
   one: the segments' states alone) selects a single kernel that solves inside each chain,
   with the same results up to rounding.  Returns as dr_chunk_fwd_workspace_bytes. */
int dr_chunk_fwd_min_workspace_bytes(const dr_chunk_desc *desc, size_t *bytes);

/*
 * Chunkwise forward over T tokens for all B x H chains.
 *
 *   init_state   NULL = zero initial state, else [B, H, dk, dv] fp32 (read only)
 *   out          [B, T, H, dv] out_dtype (written)
 *   final_state  NULL = not returned, else [B, H, dk, dv] fp32 (written); may equal
 *                init_state for an in-place carry, must not overlap it otherwise
 *   workspace    device scratch of at least dr_chunk_fwd_min_workspace_bytes() bytes
 *                (dr_chunk_fwd_workspace_bytes() for the fastest path); may be NULL when
 *                that size is 0.  Contents on entry are ignored; it must not be used by
 *                other work until this call's kernels finish on `stream`.
 *
 * The chunk length C only changes rounding, never the result's definition.  A tail chunk
 * (T not a multiple of C) is padded with identity steps (k = 0, beta = 0, log_alpha = 0),
 * which leave S unchanged; their outputs are not written.
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED, DR_ERR_WORKSPACE or DR_ERR_CUDA.
 */
int dr_chunk_fwd(const dr_chunk_desc *desc,
                 const void *q, const void *k, const void *v,
                 const float *log_alpha, const void *beta,
                 const float *init_state, void *out, float *final_state,
                 void *workspace, size_t workspace_bytes, dr_stream_t stream);

/*
 * dr_chunk_fwd for callers holding HOST buffers (the end-to-end path): q, k, v, log_alpha,
 * beta, init_state are HOST pointers (layouts and dtypes as for dr_chunk_fwd), and so are
 * out and final_state (NULL = not returned).  The call copies the inputs host -> device,
 * runs the forward and copies the results device -> host, all enqueued behind `stream`
 * (the results are in place once `stream` has completed; the host buffers must not be
 * touched before).  The sequence is split into `pieces` time ranges of whole chunks (1 ..
 * 16, at most the number of chunks), the state carried from one to the next on the device:
 * one piece's kernels overlap the next piece's input copies and the previous piece's output
 * copies (the two directions also overlap each other).  Host buffers should be page-locked
 * (cudaHostAlloc / pinned) for the copies to be asynchronous.  `dev` is a device buffer of
 * at least dr_chunk_fwd_host_dev_bytes() bytes, 256-byte aligned, holding the staging
 * copies, the state and the workspace; it must not be used by other work until `stream`
 * completes.  Streams and events are created for the call and released behind its work.
 * Returns the statuses of dr_chunk_fwd (DR_ERR_WORKSPACE for a missing or short `dev`); on
 * DR_ERR_CUDA part of the work may have been enqueued; `stream` then still waits for all of it.
 */
int dr_chunk_fwd_host_dev_bytes(const dr_chunk_desc *desc, int pieces, size_t *bytes);
int dr_chunk_fwd_host(const dr_chunk_desc *desc, int pieces,
                      const void *q, const void *k, const void *v,
                      const float *log_alpha, const void *beta,
                      const float *init_state, void *out, float *final_state,
                      void *dev, size_t dev_bytes, dr_stream_t stream);

/*
 * dr_chunk_fwd with fused neighbours: `fuse` is an OR of DR_FUSE_* (0 makes the call
 * identical to dr_chunk_fwd); `z` is the output gate's input, [B, T, H, dv] in_dtype, read
 * only, required (non-NULL, 16-byte aligned, not overlapping `out`) when DR_FUSE_OUT_SILU_GATE
 * is set and ignored otherwise.  Every configuration dr_chunk_fwd accepts takes every flag.
 * The least workspace is dr_chunk_fwd_min_workspace_bytes() whatever the flags; the fastest
 * path with flags set may take more, dr_chunk_fwd_ex_workspace_bytes().  Returns the
 * statuses of dr_chunk_fwd; DR_ERR_INVALID also for bits outside DR_FUSE_ALL or a missing z.
 */
/* Bytes of device workspace dr_chunk_fwd_ex takes for *desc and the flags `fuse` on its
   fastest path; written to *bytes.  With fuse = 0, dr_chunk_fwd_workspace_bytes().  For bf16
   inputs, dk = dv = 128, chunk 64 and a scalar or no gate, with any flag set (and bf16
   outputs when the output gate is fused): the two-kernel path's 16 KB of triangular-solve
   operands plus 512 bytes of row norms per (b, h, chunk), and the segments' states when few
   long chains are split.  Returns DR_OK, DR_ERR_INVALID (also for bits outside DR_FUSE_ALL)
   or DR_ERR_UNSUPPORTED. */
int dr_chunk_fwd_ex_workspace_bytes(const dr_chunk_desc *desc, uint32_t fuse, size_t *bytes);

int dr_chunk_fwd_ex(const dr_chunk_desc *desc, uint32_t fuse,
                    const void *q, const void *k, const void *v,
                    const float *log_alpha, const void *beta, const void *z,
                    const float *init_state, void *out, float *final_state,
                    void *workspace, size_t workspace_bytes, dr_stream_t stream);

/*
 * One decode step for B x H chains, one token each (the loop body of the recurrence
 * once).  Streams the fp32 state through HBM once: it is read, decayed, updated and
 * written back in place.
 *
 *   q, k   [B, H, dk] in_dtype;  v [B, H, dv] in_dtype;  beta [B, H] in_dtype
 *   log_alpha  NULL (DR_GATE_NONE), [B, H] (scalar) or [B, H, dk] (channel), fp32
 *   state  [B, H, dk, dv] fp32, read and overwritten
 *   out    [B, H, dv] out_dtype (must not overlap state)
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED or DR_ERR_CUDA.
 */
int dr_recurrent_step(const dr_step_desc *desc,
                      const void *q, const void *k, const void *v,
                      const float *log_alpha, const void *beta,
                      float *state, void *out, dr_stream_t stream);

/*
 * Backward of dr_chunk_fwd (training): the gradients of
 *     L = <d_out, out> + <d_final_state, final_state>
 * with respect to every input, for the same descriptor (any gate, dk, dv in {64, 128},
 * chunk 16, 32 or 64, fp32 or bf16), computed chunkwise with fp32 sums: the forward's
 * per-chunk operands and chunk-start states are recomputed into the workspace, a reverse
 * pass carries the state gradient from the last chunk to the first, and every chunk's
 * token gradients follow in parallel.  Products of rows run on the tensor cores as TF32
 * tiles, split into three products (fp32 accuracy) for fp32 inputs and single products
 * for bf16 inputs; the chunk-start states of bf16 problems that the tensor-core forward
 * serves come from it (bf16 operands).  Accuracy: fp32 inputs within 1e-4 of the exact
 * gradients (unit-scale values), bf16 inputs within the forward's bf16 bound.  The pages ask for chunkwise kernels for
 * training (page "linear-attention gated-deltanet guide", section 5) without printing a
 * backward; this is the derivative of the chunk form.
 *
 *   inputs         as for dr_chunk_fwd (q, k, v, log_alpha, beta, init_state)
 *   d_out          [B, T, H, dv] out_dtype
 *   d_final_state  NULL (zero) or [B, H, dk, dv] fp32
 *   dq, dk         [B, T, H, dk] in_dtype (written)
 *   dv             [B, T, H, dv] in_dtype (written)
 *   d_log_alpha    log_alpha's shape, fp32 (written); NULL exactly when gate is NONE
 *   d_beta         [B, T, H] in_dtype (written)
 *   d_init_state   NULL (not returned) or [B, H, dk, dv] fp32 (written)
 *   workspace      at least dr_chunk_bwd_workspace_bytes() (295,424 bytes per
 *                  (b, h, chunk) at dk = dv = 128, C = 64); contents on entry ignored
 * Written buffers must not overlap each other or any input.  The fused-neighbour flags
 * are not taken here.  Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED,
 * DR_ERR_WORKSPACE or DR_ERR_CUDA.
 */
int dr_chunk_bwd_workspace_bytes(const dr_chunk_desc *desc, size_t *bytes);
int dr_chunk_bwd(const dr_chunk_desc *desc,
                 const void *q, const void *k, const void *v,
                 const float *log_alpha, const void *beta, const float *init_state,
                 const void *d_out, const float *d_final_state,
                 void *dq, void *dk, void *dv, float *d_log_alpha, void *d_beta,
                 float *d_init_state, void *workspace, size_t workspace_bytes,
                 dr_stream_t stream);

/*
 * dr_recurrent_step with fused neighbours (flags as for dr_chunk_fwd_ex); `z` is
 * [B, H, dv] in_dtype, required when DR_FUSE_OUT_SILU_GATE is set, and must not overlap
 * `state` or `out`.  Returns the statuses of dr_recurrent_step.
 */
int dr_recurrent_step_ex(const dr_step_desc *desc, uint32_t fuse,
                         const void *q, const void *k, const void *v,
                         const float *log_alpha, const void *beta, const void *z,
                         float *state, void *out, dr_stream_t stream);

/*
 * dr_chunk_fwd without a caller-provided workspace.  The pages have no counterpart of
 * this entry point: it exists for callers that cannot allocate device memory -- code
 * whose host framework owns all device memory through a pre-reserved pool, plugin
 * interfaces whose execute callback must not allocate, latency-bound loops that cannot
 * pay cudaMalloc's implicit synchronisation.  They still pass inputs and outputs exactly
 * as for dr_chunk_fwd; the scratch comes from one static device array of
 * DR_NOALLOC_SCRATCH_BYTES that libdr.so holds on every GPU it is loaded on until exit.
 *
 *   - Problems whose dr_chunk_fwd_min_workspace_bytes() exceeds DR_NOALLOC_SCRATCH_BYTES
 *     are rejected with DR_ERR_WORKSPACE before anything is enqueued; the fastest path is
 *     taken whenever dr_chunk_fwd_workspace_bytes() fits.  At bf16 inputs,
 *     dk = dv = 128, C = 64: the tensor-core path (scalar or no gate) needs none
 *     unless few long chains are split into segments; the per-channel gate needs 131,584
 *     bytes per (b, h, chunk), so there B * H * ceil(T / 64) <= 510.  The CUDA-core path
 *     (fp32 inputs, other sizes) needs 147,968 bytes per (b, h, chunk) at dk = dv = 128,
 *     C = 64, so there B * H * ceil(T / 64) <= 453.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress
 *     with that device current); make that first call before any stream capture.
 *   - Every call shares the array.  Calls whose work overlaps on the GPU (other streams,
 *     other host threads) race on it; the caller must serialise them.  No contents need
 *     clearing between calls: every scratch element read is first written by the call.
 *   - Allocates nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 * Returns the statuses of dr_chunk_fwd, and DR_ERR_CUDA if the address lookup fails.
 */
#define DR_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int dr_chunk_fwd_noalloc(const dr_chunk_desc *desc,
                         const void *q, const void *k, const void *v,
                         const float *log_alpha, const void *beta,
                         const float *init_state, void *out, float *final_state,
                         dr_stream_t stream);

/*
 * The additive gated linear recurrence: the members of the family without the delta rule's
 * correction ("Linear attention" on the page "NLP: linear attention summary"; the scalar
 * decay of "Transformer notes (5): linear attention optimisations", summary and Q&A),
 *
 *     S_t = alpha_t S_{t-1} + k_t v_t^T,      o_t = S_t^T q_t,
 *
 * alpha_t = exp(log_alpha_t) a scalar per head and token (DR_GATE_SCALAR) or 1
 * (DR_GATE_NONE).  It is no case of dr_chunk_fwd: there one beta scales both the write and
 * the correction.  The per-channel gate is not built for it (DR_ERR_UNSUPPORTED).
 *
 *   - B sequences of T tokens, laid out as for dr_chunk_fwd; or (N >= 1, B = 1) N sequences
 *     packed behind one another in the T rows: sequence n has the rows cu_seqlens[n] ..
 *     cu_seqlens[n + 1] - 1.  cu_seqlens is a device array of N + 1 non-decreasing values in
 *     0 .. T (values outside are clamped; the sequences must not share rows: where decreasing
 *     offsets make them, those rows' results are undefined, and no other memory is touched); a
 *     sequence may be empty: its state passes through.  Rows of no sequence are neither read for
 *     another row's sake nor written.  States are [N, H, dk, dv] (N = B if not packed).
 *   - The first call on a device looks up device addresses: make it before a stream capture.
 *   - log_alpha and d_log_alpha need 4-byte, cu_seqlens 8-byte alignment.
 *   - Two ways of computing, chosen by types and lengths alone.  bf16 inputs with bf16 results of
 *     more than 16 tokens (packed: rows in all) run on the tensor cores in chunks of 64 tokens.
 *     Everything else (fp32 inputs, fp32 results of bf16 inputs, up to 16 tokens) runs token
 *     by token in fp32 arithmetic, in 15 (many chains) to 100 (few long ones) times the other's time.
 *   - Precision.  Sums are fp32 everywhere.  On the tensor cores the state's products are exact,
 *     and scores and states are read out as two bf16 terms (2^-17 of a value at most is lost): bf16
 *     results are off by their own rounding, d_log_alpha (three terms) by 1e-6 of its 2-norm, states by 3e-7.
 *     Who wants fp32 arithmetic asks for fp32 results (forward) or hands in fp32 rows (backward).
 *   - log_alpha = -inf is a full reset (alpha = 0; from -120 on it is one in fp32).  On the tensor
 *     cores out and dv hold their sums divided by the row's decay within its chunk, 2^-60 at least: the
 *     state in front of the chunk enters them with no less than 2^-60, and values beyond 3.4e38
 *     times the divisor (2.9e20 behind strong decays) overflow to infinity or NaN.  dq, dk, states
 *     and d_log_alpha know neither limit.
 *     Inputs of the sequences' rows are otherwise finite; a NaN or infinity may reach every
 *     output of its chunk.  Values in rows of no sequence do not matter.
 */
typedef struct {
    int64_t B, T, H, dk, dv;  /* B, H >= 1; T >= 0; dk, dv in {64, 128}                */
    int64_t N;                /* 0: B sequences of T tokens; >= 1: packed sequences     */
    int32_t in_dtype;         /* DR_F32 or DR_BF16: q, k, v and their gradients         */
    int32_t out_dtype;        /* DR_F32 or DR_BF16: out, d_out                          */
    int32_t gate;             /* DR_GATE_NONE or DR_GATE_SCALAR                         */
    int32_t reserved;         /* must be 0                                              */
} dr_linrec_desc;

/*
 * Forward.  q, k, v, log_alpha, init_state, out, final_state as for dr_chunk_fwd (final_state
 * may equal init_state); cu_seqlens NULL unless N >= 1.  out overlaps no input or state,
 * final_state no input other than init_state, workspace nothing (DR_ERR_INVALID).
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED, DR_ERR_WORKSPACE or DR_ERR_CUDA.  Workspace
 * rules as for dr_chunk_fwd; its size depends only on the descriptor.
 */
int dr_linrec_fwd_workspace_bytes(const dr_linrec_desc *desc, size_t *bytes);
int dr_linrec_fwd(const dr_linrec_desc *desc, const void *q, const void *k, const void *v,
                  const float *log_alpha, const int64_t *cu_seqlens, const float *init_state,
                  void *out, float *final_state, void *workspace, size_t workspace_bytes,
                  dr_stream_t stream);

/*
 * Backward: the gradients of <d_out, out> + <d_final_state, final_state>.
 *   d_out          [B, T, H, dv]; in_dtype = out_dtype here (DR_ERR_UNSUPPORTED otherwise)
 *   d_final_state  NULL (zero) or fp32 [N, H, dk, dv]
 *   dq, dk, dv     in_dtype (written);  d_log_alpha fp32 [B, T, H] (written), NULL exactly
 *                  when gate is NONE;  d_init_state NULL or fp32 [N, H, dk, dv] (written),
 *                  may equal d_final_state
 * d_log_alpha_t = alpha_t <S_{t-1}, dL/dS_t> comes as a sum of q.dq - k.dk over the up to 256 tokens
 * behind t (128 where the call runs token by token) and one inner product of states.  It is 0 where
 * alpha is; where a strong decay makes it small against those terms, it carries their rounding
 * (some 1e-6 of the largest).
 * Written buffers, workspace among them, overlap neither each other nor an input otherwise
 * (DR_ERR_INVALID).  Results do not depend on the order in which the GPU runs its blocks.
 * Statuses as for dr_linrec_fwd.
 */
int dr_linrec_bwd_workspace_bytes(const dr_linrec_desc *desc, size_t *bytes);
int dr_linrec_bwd(const dr_linrec_desc *desc, const void *q, const void *k, const void *v,
                  const float *log_alpha, const int64_t *cu_seqlens, const float *init_state,
                  const void *d_out, const float *d_final_state, void *dq, void *dk, void *dv,
                  float *d_log_alpha, float *d_init_state, void *workspace,
                  size_t workspace_bytes, dr_stream_t stream);

/*
 * Zeroes what dr_linrec_fwd and dr_linrec_bwd leave alone, the rows of no sequence of a packed
 * problem (N >= 1; those in front of cu_seqlens[0] and from cu_seqlens[N] on), in any of dq, dk
 * [T, H, dk] in_dtype, out [T, H, dv] out_dtype (or dv) and d_log_alpha [T, H] (NULL: not given),
 * for callers whose buffers are new and may be summed over all rows.  Returns DR_OK,
 * DR_ERR_INVALID, DR_ERR_UNSUPPORTED or DR_ERR_CUDA.
 */
int dr_linrec_zero_rest(const dr_linrec_desc *desc, const int64_t *cu_seqlens, void *dq, void *dk, void *out,
                        float *d_log_alpha, dr_stream_t stream);

/*
 * One token for B x H chains, the state updated in place: layouts and checks of
 * dr_recurrent_step, without beta (gate NONE or SCALAR).  log_alpha needs 4-byte alignment.
 */
int dr_linrec_step(const dr_step_desc *desc, const void *q, const void *k, const void *v,
                   const float *log_alpha, float *state, void *out, dr_stream_t stream);

/*
 * Queries and keys as a layer hands them to the recurrences (or to an attention layer
 * between them): every head's row normalised and rotated by its position, in one pass.
 *
 *     y = w x / sqrt(sum(x^2) / n + eps)    n = d (DR_NORM_RMS) or 1 (DR_NORM_L2);
 *                                           y = x without a norm
 *     (y_a, y_b) -> s (y_a cos p f_i - y_b sin p f_i,  y_b cos p f_i + y_a sin p f_i)
 *
 * for the pairs i < rot / 2 of the first rot values: (a, b) = (i, i + rot / 2) in the half
 * layout, (2 i, 2 i + 1) in the interleaved one; p is the row's position, s rot_scale.  The
 * other d - rot values are not rotated.  Statistics are fp32.  Angles: position times table
 * entry (dr_rope_table) is exact modulo a turn at any position, then rounded to fp32: off by at
 * most 2^-26 of a turn (1e-7 rad).  A table entry is within 2^-50 of its frequency, which against
 * f_i itself adds at most |p| f_i 2^-52.6 turns: as much again at |p| = 2^26, below 2^-21 of a turn up
 * to 2^31, where positions are meant to stay.
 */
enum { DR_NORM_NONE = 0, DR_NORM_L2 = 1, DR_NORM_RMS = 2 };
enum { DR_ROPE_HALF = 0, DR_ROPE_INTERLEAVED = 1 };
/* How the frequencies f_i = base^(-2 i / rot) are scaled for contexts longer than the
   trained one: not at all; f_i / factor; or by parts, f_i (w + (1 - w) / factor) with
   w = clamp((r - low) / (high - low), 0, 1) and r = original f_i / (2 pi), the turns within
   the original context: fast pairs stay, slow ones are interpolated. */
enum { DR_ROPE_PLAIN = 0, DR_ROPE_LINEAR = 1, DR_ROPE_BY_PARTS = 2 };

typedef struct {
    int64_t n_tok;            /* rows (tokens) of all sequences, >= 0                    */
    int64_t seq_len, pos0;    /* without positions: row t is at pos0 + t mod seq_len
                                 (seq_len 0: n_tok)                                      */
    int64_t Hq, Hk;           /* query heads >= 1, key heads >= 0 (0: no k)              */
    int64_t d, rot;           /* head width 64, 128 or 256; rotated part, a multiple of
                                 16 in 0 .. d                                            */
    int64_t q_stride, k_stride; /* elements between the rows of q, k: 0 for contiguous,
                                 else at least Hq d (Hk d), multiples of 16 bytes        */
    int64_t q_out_stride, k_out_stride; /* the same of what is written: q_out, k_out, or
                                 dq, dk of the gradient                                  */
    int32_t dtype;            /* DR_F32 or DR_BF16                                       */
    int32_t norm, layout;     /* DR_NORM_*, DR_ROPE_HALF or DR_ROPE_INTERLEAVED          */
    int32_t reserved;         /* must be 0                                               */
    float eps, rot_scale;     /* eps >= 0                                                */
} dr_qk_norm_rope_desc;

/* HOST function: the rot / 2 frequencies as turns a position in units of 2^-64 turns, into
   the host array `table`, which the caller copies to the device and keeps.  base > 1,
   factor >= 1 (ignored for PLAIN); original, low < high for BY_PARTS only.  Returns DR_OK,
   DR_ERR_INVALID or DR_ERR_UNSUPPORTED (rot no multiple of 16). */
int dr_rope_table(int64_t rot, double base, int32_t scaling, double factor, double original,
                  double low, double high, uint64_t *table);

/*
 *   q, k           [n_tok, Hq | Hk, d] dtype, rows q_stride, k_stride apart
 *   wq, wk         NULL (ones) or fp32 [d]; NULL without a norm
 *   table          device copy of dr_rope_table's array (NULL when rot is 0)
 *   positions      NULL or int64 [n_tok] (device), any values (angles: above)
 *   q_out, k_out   [n_tok, Hq | Hk, d], rows q_out_stride, k_out_stride apart (written);
 *                  may be q, k themselves, with their strides; no written row shares a
 *                  byte with another or an input otherwise (DR_ERR_INVALID)
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED or DR_ERR_CUDA.
 */
int dr_qk_norm_rope(const dr_qk_norm_rope_desc *desc, const void *q, const void *k,
                    const float *wq, const float *wk, const uint64_t *table,
                    const int64_t *positions, void *q_out, void *k_out, dr_stream_t stream);

/*
 * Its gradients, from the inputs of the forward and the outputs' gradients dq_out, dk_out
 * (contiguous, dtype).  dq, dk are rows q_out_stride, k_out_stride apart (parts of one fused
 * gradient's rows, for instance) and may be q, k themselves; dwq, dwk fp32 [d] or NULL
 * (not returned; only with wq, wk), which overlap no other written buffer.  Workspace as for
 * dr_chunk_fwd, needed for dwq or dwk only; it overlaps nothing (DR_ERR_INVALID).
 * The sums' order is fixed: equal inputs give equal results.
 */
int dr_qk_norm_rope_bwd_workspace_bytes(const dr_qk_norm_rope_desc *desc, size_t *bytes);
int dr_qk_norm_rope_bwd(const dr_qk_norm_rope_desc *desc, const void *q, const void *k,
                        const float *wq, const float *wk, const uint64_t *table,
                        const int64_t *positions, const void *dq_out, const void *dk_out,
                        void *dq, void *dk, float *dwq, float *dwk, void *workspace,
                        size_t workspace_bytes, dr_stream_t stream);

/*
 * Attention over a window, for the layers of softmax attention that stand between recurrent ones: of
 * a sequence, token i sees token j when
 *
 *     j <= i  and  (i - j < window  or  j < sinks),
 *
 * the last `window` tokens (itself among them; 0: all before it) and the first `sinks` ones, which stay
 * visible.  Over the visible tokens, with s_ij = scale q_i.k_j,
 *
 *     lse_i = log sum_j exp(s_ij),    out_i = sum_j exp(s_ij - lse_i) v_j.
 *
 * Query head h reads key and value head h / (Hq / Hk).
 *   - Sequences as for dr_linrec_fwd: B of T tokens, or (N >= 1, B = 1) N packed ones by cu_seqlens
 *     (clamped; decreasing offsets make results undefined and touch no other memory).  Rows of no
 *     sequence are left as they are, or zeroed (out, lse, gradients) with zero_rest.  They and
 *     other sequences' rows do not enter a result whatever they hold; the sequence's own rows are finite (a NaN
 *     or infinity may reach every row whose tile of 128 tokens meets it, visible or not).
 *   - Sums, maxima and products' accumulators are fp32.  fp32 rows are computed in fp32 arithmetic.  Of bf16
 *     rows the weights exp(s_ij - m) and, backwards, the score gradients enter their products rounded to bf16 (half
 *     a step of 2^-8 each, at random), which leaves a result about as far off as its own rounding does.
 *   - The first call on a device looks up device addresses: make it before a stream capture.
 */
typedef struct {
    int64_t B, T, Hq, Hk, d;  /* B >= 1, T >= 0; Hq a multiple of Hk; d 64 or 128       */
    int64_t N;                /* 0: B sequences of T tokens; >= 1: packed sequences     */
    int64_t window, sinks;    /* >= 0                                                   */
    int64_t q_stride, k_stride, v_stride; /* elements between the rows of q, k, v: 0 for
                                 contiguous, else at least a row, multiples of 16 bytes */
    int64_t dq_stride, dk_stride, dv_stride; /* (backward) the same of what is written  */
    int32_t dtype;            /* DR_F32 or DR_BF16: every row                           */
    int32_t zero_rest;        /* packed: 1 zeroes the rows of no sequence, 0 leaves them */
    int32_t reserved;         /* must be 0                                              */
    float scale;              /* of the scores, > 0                                     */
} dr_attn_desc;

/*
 *   q          [B, T, Hq, d], rows q_stride apart;  k, v  [B, T, Hk, d], rows k_stride, v_stride apart
 *   out        [B, T, Hq, d] contiguous (written);  lse  fp32 [B, T, Hq] (written), natural log
 * out and lse meet neither each other nor an input (DR_ERR_INVALID).
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED or DR_ERR_CUDA.
 */
int dr_window_attn_fwd(const dr_attn_desc *desc, const void *q, const void *k, const void *v,
                       const int64_t *cu_seqlens, void *out, float *lse, dr_stream_t stream);

/*
 * Gradients of <d_out, out> from the forward's inputs, its results out and lse, and d_out [B, T, Hq, d]
 * (contiguous).  dq, dk, dv: rows dq_stride, dk_stride, dv_stride apart (written); they meet
 * neither each other nor an input.  fp32 rows: weights and delta_i are summed anew, so out and lse may come from
 * a forward with other roundings.  Results do not depend on the order in which the GPU runs its blocks.
 * A token that sees itself alone has dq = 0 up to the rounding of d_out.out.
 * Workspace rules as for dr_chunk_fwd; its size depends only on the descriptor: 8 bytes a row and query head and, with
 * a window and sinks, sums of the sinks' rows that follow the rows / window, not N: at most 16 bytes a value of dq, dk, dv.
 */
int dr_window_attn_bwd_workspace_bytes(const dr_attn_desc *desc, size_t *bytes);
int dr_window_attn_bwd(const dr_attn_desc *desc, const void *q, const void *k, const void *v,
                       const int64_t *cu_seqlens, const void *out, const float *lse, const void *d_out,
                       void *dq, void *dk, void *dv, void *workspace, size_t workspace_bytes,
                       dr_stream_t stream);

/*
 * Its paged cache.  k_cache, v_cache [n_pages, Hk, page, d]; sequence n keeps the token at position p
 * in slot p % page of the page pages[n][p / page].  Entries outside 0 .. n_pages - 1 stand for
 * pages that are not there (given back, since their tokens left the window, or not yet given).
 *
 * dr_kv_append writes new tokens: keys normalised and rotated by their position as dr_qk_norm_rope
 * does, values as they are, and on the way (Hq > 0) the same tokens' queries normalised and rotated into
 * q_out.  Row t of sequence n is its token at position start[n] + t, start[n] the tokens it had before.
 *   q, k, v      [n_tok, Hq | Hk | Hk, d], rows q_stride, k_stride, v_stride apart
 *   wq, wk, table  as for dr_qk_norm_rope
 *   pages        int32 [N, max_pages];  start  int64 [N] (device)
 *   cu_seqlens   NULL: one row for each sequence (n_tok = N); else int64 [N + 1], rows
 *                cu_seqlens[n] .. cu_seqlens[n + 1] - 1 are sequence n's
 *   q_out        [n_tok, Hq, d], rows q_out_stride apart (written); may be q itself
 * start[n] < 0: a slot of the batch without a sequence; its rows and rows of no sequence are not
 * written anywhere (q_out: zeroed with zero_rest).  Keys and values of tokens whose page is not there,
 * or behind max_pages pages, are dropped.  Rows of one call for the same slot (a page in two
 * sequences' tables): every value there is one of theirs.  Written buffers meet no other one (DR_ERR_INVALID).
 * Returns DR_OK, DR_ERR_INVALID, DR_ERR_UNSUPPORTED or DR_ERR_CUDA.
 */
typedef struct {
    int64_t n_tok, N;         /* rows >= 0; sequences >= 1                              */
    int64_t Hq, Hk;           /* query heads >= 0 (0: no q), key heads >= 1             */
    int64_t d, rot;           /* head width 64 or 128; rotated part, a multiple of 16   */
    int64_t q_stride, k_stride, v_stride, q_out_stride; /* as in dr_qk_norm_rope_desc   */
    int64_t n_pages, page, max_pages; /* pages of the cache; tokens a page, a multiple of
                                 16 up to 1024; pages a sequence                        */
    int32_t dtype;            /* DR_F32 or DR_BF16: rows and cache                      */
    int32_t norm, layout;     /* DR_NORM_*, DR_ROPE_HALF or DR_ROPE_INTERLEAVED         */
    int32_t zero_rest;        /* 1 zeroes q_out's rows of no sequence, 0 leaves them    */
    int32_t reserved;         /* must be 0                                              */
    float eps, rot_scale;     /* eps >= 0                                               */
} dr_kv_append_desc;
int dr_kv_append(const dr_kv_append_desc *desc, const void *q, const void *k, const void *v,
                 const float *wq, const float *wk, const uint64_t *table, const int32_t *pages,
                 const int64_t *start, const int64_t *cu_seqlens, void *q_out, void *k_cache,
                 void *v_cache, dr_stream_t stream);

/*
 * The attention of one new token for each of B sequences over that cache (the token itself has been
 * appended).
 *   q       [B, Hq, d] contiguous;  pages  int32 [B, max_pages];  lens  int64 [B]: tokens of each
 *           sequence, the new one among them (<= 0: none; from 2^30 on: taken as 2^30)
 *   out     [B, Hq, d] (written);  lse  NULL or fp32 [B, Hq] (written)
 * Visible are the last `window` of lens tokens and the first `sinks`, as far as their pages are there;
 * without any, out is 0 and lse -infinity.  What invisible slots of a page hold does not matter.
 * bf16: scores in fp32, weights as two bf16 terms (2^-17 of one is lost): out is off by its own rounding.
 * Workspace rules as for dr_chunk_fwd (some MB whatever the lengths); results do not depend
 * on the order in which the GPU runs its blocks.
 */
typedef struct {
    int64_t B, Hq, Hk, d;     /* as in dr_attn_desc                                     */
    int64_t n_pages, page, max_pages; /* as in dr_kv_append_desc                        */
    int64_t window, sinks;    /* as in dr_attn_desc                                     */
    int32_t dtype;            /* DR_F32 or DR_BF16: q, cache, out                       */
    int32_t reserved;         /* must be 0                                              */
    float scale;              /* > 0                                                    */
} dr_attn_step_desc;
int dr_window_attn_step_workspace_bytes(const dr_attn_step_desc *desc, size_t *bytes);
int dr_window_attn_step(const dr_attn_step_desc *desc, const void *q, const void *k_cache,
                        const void *v_cache, const int32_t *pages, const int64_t *lens, void *out,
                        float *lse, void *workspace, size_t workspace_bytes, dr_stream_t stream);

/* Synchronises `stream`, then returns and clears the library's sticky device status word
   on the current device (DR_OK, or DR_ERR_TIMEOUT if a bounded device wait expired), or
   DR_ERR_CUDA if the synchronisation itself failed. */
int dr_get_device_status(dr_stream_t stream);

/* Self-test of failure detection, with no GPU fault: launches one kernel whose thread waits
   on a barrier that nothing completes, with the chunk kernels' bounded-wait loop and a
   budget of `cycles` SM clock cycles (1 .. 4e9); on expiry it records DR_ERR_TIMEOUT in
   the status word that dr_get_device_status returns, and exits.  Returns DR_OK once
   enqueued, DR_ERR_INVALID for a budget out of range, DR_ERR_CUDA on a launch failure. */
int dr_selftest_bounded_wait(long long cycles, dr_stream_t stream);

/* Static, human-readable text of a status code (never NULL). */
const char *dr_strerror(int status);

#ifdef __cplusplus
}
#endif

#endif /* DR_H_ */
