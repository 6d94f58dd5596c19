// attn_api.cu -- the C ABI of the window attention (declared in include/dr.h): argument
// validation, workspace layout and dispatch to the kernels.
#include <math.h>

#include "../../include/dr.h"
#include "attn.h"
#include "attn_tc.cuh"
#include "common.cuh"
#include "spans.h"

namespace dr {

int *device_status_ptr();   // dr_api.cu

namespace {

int check_desc(const dr_attn_desc *d) {
    if (!d) return kErrInvalid;
    if (d->B < 1 || d->T < 0 || d->N < 0 || d->Hq < 1 || d->Hk < 1 || d->d < 1 || d->reserved != 0) return kErrInvalid;
    if (d->Hq % d->Hk != 0 || d->window < 0 || d->sinks < 0 || (d->N > 0 && d->B != 1)) return kErrInvalid;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return kErrInvalid;
    if (!(d->scale > 0.f) || isinf(d->scale) || (d->zero_rest != 0 && d->zero_rest != 1)) return kErrInvalid;
    if (d->d != 64 && d->d != 128) return kErrUnsupported;
    if (d->B > (1 << 20) || d->N > (1 << 20) || d->Hq > (1 << 16) || d->T > kNoWindow) return kErrUnsupported;
    if (d->B * d->T >= ((int64_t)1 << 31) - 256 || (d->B * (d->T / 64 + 1) + d->N) * d->Hq >= ((int64_t)1 << 31)) return kErrUnsupported;
    const int64_t unit = d->dtype == DR_BF16 ? 8 : 4;   // rows start on 16-byte boundaries
    const int64_t strides[6] = {d->q_stride, d->dq_stride, d->k_stride, d->v_stride, d->dk_stride, d->dv_stride};
    for (int i = 0; i < 6; ++i) {
        if (strides[i] == 0) continue;
        if (strides[i] < (i < 2 ? d->Hq : d->Hk) * d->d || strides[i] % unit != 0) return kErrInvalid;
        if (strides[i] > ((int64_t)1 << 31)) return kErrUnsupported;
    }
    return kOk;
}

AttnProblem problem_of(const dr_attn_desc &d, const int64_t *cu) {
    AttnProblem p{};
    p.seqs.cu = d.N > 0 ? cu : nullptr;
    p.seqs.N = d.N > 0 ? d.N : d.B;
    p.seqs.T = d.T;
    p.seqs.total = d.B * d.T;
    p.Hq = (int)d.Hq; p.Hk = (int)d.Hk; p.d = (int)d.d;
    p.window = d.window == 0 || d.window > kNoWindow ? kNoWindow : (int)d.window;
    p.sinks = d.sinks > kNoWindow ? kNoWindow : (int)d.sinks;
    p.scale = d.scale;
    p.bf16 = d.dtype == DR_BF16;
    const int64_t wq = d.Hq * d.d, wk = d.Hk * d.d;
    p.qs = d.q_stride ? d.q_stride : wq;
    p.ks = d.k_stride ? d.k_stride : wk;
    p.vs = d.v_stride ? d.v_stride : wk;
    p.dqs = d.dq_stride ? d.dq_stride : wq;
    p.dks = d.dk_stride ? d.dk_stride : wk;
    p.dvs = d.dv_stride ? d.dv_stride : wk;
    return p;
}

size_t bwd_bytes(const dr_attn_desc &d) {
    static const int64_t packed = 0;     // packed or not, not where the offsets lie
    const AttnProblem p = problem_of(d, &packed);
    return p.bf16 ? attn_tc_bwd_workspace_bytes(p) : attn_simt_bwd_workspace_bytes(p);
}

int check_step(const dr_attn_step_desc *d) {
    if (!d) return kErrInvalid;
    if (d->B < 1 || d->Hq < 1 || d->Hk < 1 || d->d < 1 || d->reserved != 0) return kErrInvalid;
    if (d->Hq % d->Hk != 0 || d->window < 0 || d->sinks < 0 || d->n_pages < 1 || d->page < 1 || d->max_pages < 1) return kErrInvalid;
    if (d->dtype != DR_F32 && d->dtype != DR_BF16) return kErrInvalid;
    if (!(d->scale > 0.f) || isinf(d->scale)) return kErrInvalid;
    if ((d->d != 64 && d->d != 128) || d->page % 16 != 0 || d->page > 1024) return kErrUnsupported;
    if (d->B > (1 << 20) || d->Hq > (1 << 16) || d->max_pages > kNoWindow / d->page) return kErrUnsupported;
    // a cache's rows are coordinates of 31 bits
    if (d->n_pages > ((int64_t)1 << 31) || d->n_pages * d->Hk > (((int64_t)1 << 31) - 1) / d->page) return kErrUnsupported;
    return kOk;
}

AttnStep step_of(const dr_attn_step_desc &d) {
    AttnStep p{};
    p.B = d.B; p.Hq = (int)d.Hq; p.Hk = (int)d.Hk; p.d = (int)d.d;
    p.page = (int)d.page; p.max_pages = (int)d.max_pages; p.n_pages = d.n_pages;
    p.window = d.window == 0 || d.window > kNoWindow ? kNoWindow : (int)d.window;
    p.sinks = d.sinks > kNoWindow ? kNoWindow : (int)d.sinks;
    p.scale = d.scale;
    p.bf16 = d.dtype == DR_BF16;
    return p;
}

}  // namespace
}  // namespace dr

using namespace dr;

extern "C" int dr_window_attn_fwd(const dr_attn_desc *desc, const void *q, const void *k, const void *v, const int64_t *cu_seqlens,
                                  void *out, float *lse, dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_attn_desc &d = *desc;
    if (d.T > 0 && (!q || !k || !v || !out || !lse)) return kErrInvalid;
    if (d.N > 0 && !cu_seqlens) return kErrInvalid;
    const void *ptrs[] = {q, k, v, out};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    if (!aligned(lse, 4) || !aligned(cu_seqlens, 8)) return kErrInvalid;
    if (d.T == 0) return kOk;
    AttnProblem p = problem_of(d, cu_seqlens);
    p.q = q; p.k = k; p.v = v; p.out = out; p.lse = lse;
    const int64_t e = p.bf16 ? 2 : 4, n = p.seqs.total;
    const Block written[2] = {{out, (size_t)(n * d.Hq * d.d * e)}, {lse, sizeof(float) * (size_t)(n * d.Hq)}};
    const Rows read[3] = {{q, d.Hq * d.d, p.qs}, {k, d.Hk * d.d, p.ks}, {v, d.Hk * d.d, p.vs}};
    const Block cu{p.seqs.cu, sizeof(int64_t) * (size_t)(d.N + 1)};
    if (meet(written[0], written[1])) return kErrInvalid;
    for (const Block &w : written) {
        if (meet(w, cu)) return kErrInvalid;
        for (const Rows &r : read)
            if (meet(r, w, n, e)) return kErrInvalid;
    }
    if (d.zero_rest && d.N > 0) {
        const AttnRest r{{out, lse, nullptr}, {d.Hq * d.d * e, d.Hq * 4, 0}, {d.Hq * d.d * e, d.Hq * 4, 0}};
        const int rz = launch_attn_zero_rest(p.seqs, r, (cudaStream_t)stream);
        if (rz != kOk) return rz;
    }
    if (!p.bf16) return launch_attn_simt_fwd(p, (cudaStream_t)stream);
    int *status = device_status_ptr();
    if (!status) return kErrCuda;
    return launch_attn_tc_fwd(p, status, (cudaStream_t)stream);
}

extern "C" int dr_window_attn_bwd_workspace_bytes(const dr_attn_desc *desc, size_t *bytes) {
    if (!bytes) return kErrInvalid;
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    *bytes = bwd_bytes(*desc);
    return kOk;
}

extern "C" int dr_window_attn_bwd(const dr_attn_desc *desc, const void *q, const void *k, const void *v, const int64_t *cu_seqlens,
                                  const void *out, const float *lse, const void *d_out, void *dq, void *dk, void *dv, void *workspace,
                                  size_t workspace_bytes, dr_stream_t stream) {
    const int rc = check_desc(desc);
    if (rc != kOk) return rc;
    const dr_attn_desc &d = *desc;
    if (d.T > 0 && (!q || !k || !v || !out || !lse || !d_out || !dq || !dk || !dv)) return kErrInvalid;
    if (d.N > 0 && !cu_seqlens) return kErrInvalid;
    const void *ptrs[] = {q, k, v, out, d_out, dq, dk, dv, workspace};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    if (!aligned(lse, 4) || !aligned(cu_seqlens, 8)) return kErrInvalid;
    if (d.T == 0) return kOk;
    const size_t need = bwd_bytes(d);
    if (!workspace || workspace_bytes < need) return kErrWorkspace;
    AttnProblem p = problem_of(d, cu_seqlens);
    p.q = q; p.k = k; p.v = v; p.out = const_cast<void *>(out); p.lse = const_cast<float *>(lse); p.d_out = d_out;
    p.dq = dq; p.dk = dk; p.dv = dv;
    const int64_t e = p.bf16 ? 2 : 4, n = p.seqs.total, wq = d.Hq * d.d, wk = d.Hk * d.d;
    // no written row meets another one, an input or the workspace
    const Rows written[3] = {{dq, wq, p.dqs}, {dk, wk, p.dks}, {dv, wk, p.dvs}};
    const Rows read[5] = {{q, wq, p.qs}, {k, wk, p.ks}, {v, wk, p.vs}, {out, wq, wq}, {d_out, wq, wq}};
    const Block small[2] = {{lse, sizeof(float) * (size_t)(n * d.Hq)}, {p.seqs.cu, sizeof(int64_t) * (size_t)(d.N + 1)}}, ws{workspace, need};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (meet(written[i], written[j], n, e)) return kErrInvalid;
        for (const Rows &r : read)
            if (meet(written[i], r, n, e)) return kErrInvalid;
        for (const Block &b : small)
            if (meet(written[i], b, n, e)) return kErrInvalid;
        if (meet(written[i], ws, n, e)) return kErrInvalid;
    }
    for (const Rows &r : read)
        if (meet(r, ws, n, e)) return kErrInvalid;
    for (const Block &b : small)
        if (meet(b, ws)) return kErrInvalid;
    if (d.zero_rest && d.N > 0) {
        const AttnRest r{{dq, dk, dv}, {wq * e, wk * e, wk * e}, {p.dqs * e, p.dks * e, p.dvs * e}};
        const int rz = launch_attn_zero_rest(p.seqs, r, (cudaStream_t)stream);
        if (rz != kOk) return rz;
    }
    if (!p.bf16) return launch_attn_simt_bwd(p, workspace, (cudaStream_t)stream);
    int *status = device_status_ptr();
    if (!status) return kErrCuda;
    return launch_attn_tc_bwd(p, workspace, status, (cudaStream_t)stream);
}

extern "C" int dr_window_attn_step_workspace_bytes(const dr_attn_step_desc *desc, size_t *bytes) {
    if (!bytes) return kErrInvalid;
    const int rc = check_step(desc);
    if (rc != kOk) return rc;
    *bytes = attn_step_workspace_bytes(step_of(*desc));
    return kOk;
}

extern "C" int dr_window_attn_step(const dr_attn_step_desc *desc, const void *q, const void *k_cache, const void *v_cache,
                                   const int32_t *pages, const int64_t *lens, void *out, float *lse, void *workspace,
                                   size_t workspace_bytes, dr_stream_t stream) {
    const int rc = check_step(desc);
    if (rc != kOk) return rc;
    const dr_attn_step_desc &d = *desc;
    if (!q || !k_cache || !v_cache || !pages || !lens || !out) return kErrInvalid;
    const void *ptrs[] = {q, k_cache, v_cache, out, workspace};
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return kErrInvalid;
    if (!aligned(lse, 4) || !aligned(pages, 4) || !aligned(lens, 8)) return kErrInvalid;
    AttnStep p = step_of(d);
    p.q = q; p.kc = k_cache; p.vc = v_cache; p.pages = pages; p.lens = lens; p.out = out; p.lse = lse;
    const size_t need = attn_step_workspace_bytes(p);
    if (!workspace || workspace_bytes < need) return kErrWorkspace;
    const size_t e = p.bf16 ? 2 : 4, rows = (size_t)(d.B * d.Hq * d.d) * e, cache = (size_t)(d.n_pages * d.Hk * d.page * d.d) * e;
    const Block written[3] = {{out, rows}, {lse, sizeof(float) * (size_t)(d.B * d.Hq)}, {workspace, need}};
    const Block read[5] = {{q, rows}, {k_cache, cache}, {v_cache, cache}, {pages, sizeof(int32_t) * (size_t)(d.B * d.max_pages)},
                           {lens, sizeof(int64_t) * (size_t)d.B}};
    for (int i = 0; i < 3; ++i) {
        for (int j = i + 1; j < 3; ++j)
            if (meet(written[i], written[j])) return kErrInvalid;
        for (const Block &r : read)
            if (meet(written[i], r)) return kErrInvalid;
    }
    int *status = device_status_ptr();
    if (!status) return kErrCuda;
    return launch_attn_step(p, workspace, status, (cudaStream_t)stream);
}
