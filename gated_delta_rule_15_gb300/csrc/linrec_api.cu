// linrec_api.cu -- the C ABI of the additive gated linear recurrence (declared in
// include/dr.h): argument validation, workspace layout and dispatch to the kernels.
#include "../../include/dr.h"
#include "common.cuh"
#include "linrec.h"

namespace dr {

int *device_status_ptr();   // dr_api.cu

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const char *a0 = (const char *)a, *b0 = (const char *)b;
    return a && b && na && nb && a0 < b0 + nb && b0 < a0 + na;
}

int check_desc(const dr_linrec_desc *d) {
    if (!d) return kErrInvalid;
    if (d->B < 1 || d->H < 1 || d->T < 0 || d->N < 0 || d->dk < 1 || d->dv < 1 || d->reserved != 0) return kErrInvalid;
    if ((d->in_dtype != DR_F32 && d->in_dtype != DR_BF16) || (d->out_dtype != DR_F32 && d->out_dtype != DR_BF16))
        return kErrInvalid;
    if (d->gate < DR_GATE_NONE || d->gate > DR_GATE_CHANNEL) return kErrInvalid;
    if (d->N > 0 && d->B != 1) return kErrInvalid;
    if (d->gate == DR_GATE_CHANNEL) return kErrUnsupported;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128)) return kErrUnsupported;
    // rows, chains and runs index 32-bit grids; rows * H * 128 stays below 2^63 by far
    if (d->B > (1 << 20) || d->N > (1 << 20) || d->H > (1 << 16) || d->T >= ((int64_t)1 << 31)) return kErrUnsupported;
    if ((d->N > 0 ? d->N : d->B) * d->H > (1 << 28) || d->B * d->T >= ((int64_t)1 << 40) / d->H) return kErrUnsupported;
    return kOk;
}

LinrecSeqs seqs_of(const dr_linrec_desc *d, const int64_t *cu) {
    LinrecSeqs s;
    s.cu = d->N > 0 ? cu : nullptr;
    s.N = d->N > 0 ? d->N : d->B;
    s.T = d->T;
    s.total = d->B * d->T;
    return s;
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

bool on_tensor_cores(const dr_linrec_desc *d, const LinrecSeqs &s) {
    return linrec_tc_supported(s, d->H, d->in_dtype == DR_BF16, d->out_dtype == DR_BF16);
}
// What the size of a workspace goes by: packed or not, not where the offsets lie.
LinrecSeqs shape_of(const dr_linrec_desc *d) {
    static const int64_t packed = 0;
    return seqs_of(d, &packed);
}

// Workspace of the backward: the segments' states; with a gate the two dot products, the
// stored states and their inner products.
struct BwdSpace {
    size_t dot_q, dot_k, inner, anchor, bytes;
    int parts, run;
};
BwdSpace bwd_space(const dr_linrec_desc *d) {
    BwdSpace w{};
    const LinrecSeqs s = shape_of(d);
    const bool tc = on_tensor_cores(d, s);
    const size_t segs = tc ? round256(linrec_tc_workspace_bytes(s, d->H, (int)d->dk, (int)d->dv)) : 0;
    w.bytes = segs;
    if (d->gate == DR_GATE_NONE) return w;
    w.parts = tc ? 1 : (int)d->dk / kSimtCols;   // the dq and dk passes' value width is dk
    w.run = tc ? kAnchor : kTokenAnchor;
    const size_t slots = (size_t)linrec_slots(w.run, s);
    const size_t dot = round256(sizeof(float) * (size_t)w.parts * d->H * s.total);
    w.dot_q = segs;
    w.dot_k = segs + dot;
    w.inner = segs + 2 * dot;
    w.anchor = w.inner + round256(sizeof(float) * (size_t)w.parts * slots * d->H);
    w.bytes = w.anchor + round256(sizeof(float) * slots * d->H * d->dk * d->dv);
    return w;
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" int dr_linrec_fwd_workspace_bytes(const dr_linrec_desc *desc, size_t *bytes) {
    if (!bytes) return kErrInvalid;
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const LinrecSeqs s = shape_of(desc);
    *bytes = on_tensor_cores(desc, s) ? linrec_tc_workspace_bytes(s, desc->H, (int)desc->dk, (int)desc->dv) : 0;
    return kOk;
}

extern "C" int dr_linrec_bwd_workspace_bytes(const dr_linrec_desc *desc, size_t *bytes) {
    if (!bytes) return kErrInvalid;
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    *bytes = bwd_space(desc).bytes;
    return kOk;
}

extern "C" int dr_linrec_fwd(const dr_linrec_desc *desc, const void *q, const void *k, const void *v,
                             const float *log_alpha, const int64_t *cu_seqlens, const float *init_state, void *out,
                             float *final_state, void *workspace, size_t workspace_bytes, dr_stream_t stream) {
    int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_linrec_desc &d = *desc;
    if (d.T > 0 && (!q || !k || !v || !out)) return kErrInvalid;
    if (d.gate != DR_GATE_NONE && d.T > 0 && !log_alpha) return kErrInvalid;
    if (d.N > 0 && !cu_seqlens) return kErrInvalid;
    const void *ptrs[] = {q, k, v, init_state, out, final_state, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return kErrInvalid;
    if (((uintptr_t)cu_seqlens & 7u) || ((uintptr_t)log_alpha & 3u)) return kErrInvalid;
    const LinrecSeqs seqs = seqs_of(desc, cu_seqlens);
    const size_t sb = sizeof(float) * (size_t)seqs.N * d.H * d.dk * d.dv, rows = (size_t)seqs.total * d.H;
    const size_t ie = d.in_dtype == DR_BF16 ? 2 : 4, ob = rows * d.dv * (d.out_dtype == DR_BF16 ? 2 : 4);
    if (final_state != init_state && overlaps(final_state, sb, init_state, sb)) return kErrInvalid;
    const struct { const void *p; size_t n; } read[] = {
        {q, rows * d.dk * ie}, {k, rows * d.dk * ie}, {v, rows * d.dv * ie}, {log_alpha, rows * sizeof(float)},
        {seqs.cu, sizeof(int64_t) * (size_t)(d.N + 1)}};
    for (const auto &r : read)
        if (overlaps(out, ob, r.p, r.n) || overlaps(final_state, sb, r.p, r.n)) return kErrInvalid;
    if (overlaps(out, ob, init_state, sb) || overlaps(out, ob, final_state, sb)) return kErrInvalid;
    size_t need = 0;
    dr_linrec_fwd_workspace_bytes(desc, &need);
    if (need > 0 && (!workspace || workspace_bytes < need)) return kErrWorkspace;
    for (const auto &r : read)
        if (overlaps(workspace, need, r.p, r.n)) return kErrInvalid;
    if (overlaps(workspace, need, init_state, sb) || overlaps(workspace, need, out, ob) || overlaps(workspace, need, final_state, sb))
        return kErrInvalid;
    if (d.T == 0 && !final_state) return kOk;
    LinrecPass p{};
    p.seqs = seqs;
    p.H = (int)d.H; p.dk = (int)d.dk; p.dv = (int)d.dv;
    p.in_bf16 = d.in_dtype == DR_BF16; p.out_bf16 = d.out_dtype == DR_BF16;
    p.q = q; p.k = k; p.v = v; p.la = d.gate == DR_GATE_NONE ? nullptr : log_alpha;
    p.init = init_state; p.fin = final_state; p.out = out;
    if (!on_tensor_cores(desc, seqs)) return launch_linrec_simt(p, (cudaStream_t)stream);
    int *status = device_status_ptr();
    if (!status) return kErrCuda;
    return launch_linrec_tc(p, workspace, status, (cudaStream_t)stream);
}

extern "C" int dr_linrec_bwd(const dr_linrec_desc *desc, const void *q, const void *k, const void *v,
                             const float *log_alpha, const int64_t *cu_seqlens, const float *init_state,
                             const void *d_out, const float *d_final_state, void *dq, void *dk, void *dv,
                             float *d_log_alpha, float *d_init_state, void *workspace, size_t workspace_bytes,
                             dr_stream_t stream) {
    int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_linrec_desc &d = *desc;
    if (d.in_dtype != d.out_dtype) return kErrUnsupported;
    if (d.T > 0 && (!q || !k || !v || !d_out || !dq || !dk || !dv)) return kErrInvalid;
    if (d.gate != DR_GATE_NONE && d.T > 0 && (!log_alpha || !d_log_alpha)) return kErrInvalid;
    if (d.gate == DR_GATE_NONE && d_log_alpha) return kErrInvalid;
    if (d.N > 0 && !cu_seqlens) return kErrInvalid;
    const void *ptrs[] = {q, k, v, init_state, d_out, d_final_state, dq, dk, dv, d_init_state, workspace};
    for (const void *p : ptrs)
        if (!aligned16(p)) return kErrInvalid;
    if (((uintptr_t)cu_seqlens & 7u) || (((uintptr_t)log_alpha | (uintptr_t)d_log_alpha) & 3u)) return kErrInvalid;
    const LinrecSeqs seqs = seqs_of(desc, cu_seqlens);
    const size_t sb = sizeof(float) * (size_t)seqs.N * d.H * d.dk * d.dv, rows = (size_t)seqs.total * d.H;
    const size_t e = d.in_dtype == DR_BF16 ? 2 : 4, kb = rows * d.dk * e, vb = rows * d.dv * e, gb = rows * sizeof(float);
    // no written buffer overlaps another one or an input; only d_init_state may be d_final_state
    const struct { const void *p; size_t n; } written[] = {{dq, kb}, {dk, kb}, {dv, vb}, {d_log_alpha, gb}, {d_init_state, sb}},
        read[] = {{q, kb}, {k, kb}, {v, vb}, {log_alpha, gb}, {init_state, sb}, {d_out, vb}, {d_final_state, sb},
                  {seqs.cu, sizeof(int64_t) * (size_t)(d.N + 1)}};
    for (int i = 0; i < 5; ++i) {
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(written[i].p, written[i].n, written[j].p, written[j].n)) return kErrInvalid;
        for (int j = 0; j < 8; ++j)
            if (overlaps(written[i].p, written[i].n, read[j].p, read[j].n) && !(i == 4 && j == 6 && d_init_state == d_final_state))
                return kErrInvalid;
    }
    const BwdSpace w = bwd_space(desc);
    if (w.bytes > 0 && d.T > 0 && (!workspace || workspace_bytes < w.bytes)) return kErrWorkspace;
    if (d.T > 0) {
        for (const auto &x : written)
            if (overlaps(workspace, w.bytes, x.p, x.n)) return kErrInvalid;
        for (const auto &x : read)
            if (overlaps(workspace, w.bytes, x.p, x.n)) return kErrInvalid;
    }
    if (d.T == 0 && !d_init_state) return kOk;
    char *ws = (char *)workspace;
    const bool tc = on_tensor_cores(desc, seqs);
    int *status = tc ? device_status_ptr() : nullptr;
    if (tc && !status) return kErrCuda;
    auto pass = [&](const LinrecPass &x) {
        return tc ? launch_linrec_tc(x, workspace, status, (cudaStream_t)stream) : launch_linrec_simt(x, (cudaStream_t)stream);
    };
    const bool gate = d.gate != DR_GATE_NONE && d.T > 0;
    LinrecPass p{};
    p.seqs = seqs;
    p.H = (int)d.H;
    p.in_bf16 = d.in_dtype == DR_BF16; p.out_bf16 = d.out_dtype == DR_BF16;
    p.la = d.gate == DR_GATE_NONE ? nullptr : log_alpha;
    if (d.T > 0) {
        // dq forwards over S^T, storing S for the log-decay gradient
        p.dk = (int)d.dv; p.dv = (int)d.dk; p.rev = false; p.state_t = true;
        p.q = d_out; p.k = v; p.v = k; p.init = init_state; p.fin = nullptr; p.out = dq;
        if (gate) {
            p.y = q; p.dot = (float *)(ws + w.dot_q); p.anchor = (float *)(ws + w.anchor);
        }
        if ((rc = pass(p)) != kOk) return rc;
        // dk backwards over dS^T, multiplying it with the stored S
        p.rev = true; p.q = v; p.k = d_out; p.v = q; p.init = d_final_state; p.out = dk;
        if (gate) {
            p.y = k; p.dot = (float *)(ws + w.dot_k); p.inner = (float *)(ws + w.inner);
        }
        if ((rc = pass(p)) != kOk) return rc;
    }
    // dv backwards over dS, and the initial state's gradient; its segments start from the dk
    // pass's states, which lie in the workspace in the caller's orientation
    p.dk = (int)d.dk; p.dv = (int)d.dv; p.rev = true; p.state_t = false;
    p.q = k; p.k = q; p.v = d_out; p.init = d_final_state; p.fin = d_init_state; p.out = dv;
    p.chained = d.T > 0;
    p.y = nullptr; p.dot = p.anchor = p.inner = nullptr;
    if ((rc = pass(p)) != kOk) return rc;
    if (!gate) return kOk;
    return launch_linrec_gate_grad(seqs, (int)d.H, w.run, w.parts, log_alpha, (const float *)(ws + w.dot_q),
                                   (const float *)(ws + w.dot_k), (const float *)(ws + w.inner), d_log_alpha,
                                   (cudaStream_t)stream);
}

extern "C" int dr_linrec_zero_rest(const dr_linrec_desc *desc, const int64_t *cu_seqlens, void *dq, void *dk, void *out,
                                   float *d_log_alpha, dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_linrec_desc &d = *desc;
    if (d.N < 1 || !cu_seqlens || ((uintptr_t)cu_seqlens & 7u) || ((uintptr_t)d_log_alpha & 3u)) return kErrInvalid;
    const LinrecSeqs seqs = seqs_of(desc, cu_seqlens);
    LinrecRest r{};
    const int64_t ie = d.in_dtype == DR_BF16 ? 2 : 4, oe = d.out_dtype == DR_BF16 ? 2 : 4;
    r.rows[0] = dq; r.rows[1] = dk; r.rows[2] = out;
    r.row_bytes[0] = r.row_bytes[1] = d.H * d.dk * ie;
    r.row_bytes[2] = d.H * d.dv * oe;
    r.gates = d_log_alpha;
    r.gate_words = d.H;
    const size_t cu = sizeof(int64_t) * (size_t)(d.N + 1);
    for (int i = 0; i < 3; ++i)
        if (!aligned16(r.rows[i]) || overlaps(r.rows[i], (size_t)(r.row_bytes[i] * d.T), cu_seqlens, cu)) return kErrInvalid;
    if (overlaps(d_log_alpha, sizeof(float) * (size_t)(d.T * d.H), cu_seqlens, cu)) return kErrInvalid;
    if (d.T == 0) return kOk;
    return launch_linrec_zero_rest(seqs, r, (cudaStream_t)stream);
}

extern "C" int dr_linrec_step(const dr_step_desc *d, const void *q, const void *k, const void *v, const float *log_alpha,
                              float *state, void *out, dr_stream_t stream) {
    if (!d) return kErrInvalid;
    if (d->B < 1 || d->H < 1 || d->dk < 1 || d->dv < 1 || d->reserved != 0) return kErrInvalid;
    if ((d->in_dtype != DR_F32 && d->in_dtype != DR_BF16) || (d->out_dtype != DR_F32 && d->out_dtype != DR_BF16))
        return kErrInvalid;
    if (d->gate < DR_GATE_NONE || d->gate > DR_GATE_CHANNEL) return kErrInvalid;
    if (d->gate == DR_GATE_CHANNEL) return kErrUnsupported;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128)) return kErrUnsupported;
    if (d->B > (1 << 28) || d->H > (1 << 28) || d->B * d->H > (1 << 28)) return kErrUnsupported;
    if (!q || !k || !v || !state || !out || (d->gate != DR_GATE_NONE && !log_alpha)) return kErrInvalid;
    const void *ptrs[] = {q, k, v, state, out};
    for (const void *p : ptrs)
        if (!aligned16(p)) return kErrInvalid;
    if ((uintptr_t)log_alpha & 3u) return kErrInvalid;
    const size_t n = (size_t)(d->B * d->H), sb = sizeof(float) * n * d->dk * d->dv;
    const size_t ie = d->in_dtype == DR_BF16 ? 2 : 4, ob = n * d->dv * (d->out_dtype == DR_BF16 ? 2 : 4);
    const struct { const void *p; size_t n; } read[] = {
        {q, n * d->dk * ie}, {k, n * d->dk * ie}, {v, n * d->dv * ie}, {log_alpha, n * sizeof(float)}};
    for (const auto &r : read)
        if (overlaps(out, ob, r.p, r.n) || overlaps(state, sb, r.p, r.n)) return kErrInvalid;
    if (overlaps(state, sb, out, ob)) return kErrInvalid;
    return launch_linrec_step((int64_t)n, (int)d->dk, (int)d->dv, d->in_dtype == DR_BF16, d->out_dtype == DR_BF16, q, k,
                              v, d->gate == DR_GATE_NONE ? nullptr : log_alpha, state, out, (cudaStream_t)stream);
}
