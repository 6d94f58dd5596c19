// linrec_tc.cu -- launches of the additive gated linear recurrence's tensor-core kernel
// (linrec_tc.cuh): tensor maps, the split of few long chains into segments and the kernel that
// chains the segments' states.
#include <cudaTypedefs.h>

#include "linrec_tc.cuh"

namespace dr {

PFN_cuTensorMapEncodeTiled_v12000 tc_tensor_map_encoder();

namespace {

using linrec::TcArgs;

constexpr int kSms = 152;

// [rows, H, d] bf16; boxes of 64 channels x 1 x 64 rows, 128-byte swizzle.  Rows behind the last
// read as zeros.
bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t H, int64_t d) {
    auto enc = tc_tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)(H * d) * 2};
    cuuint32_t box[3] = {64, 1, 64}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The segments' start states from their sums: per chain, in the order of the pass, start(0) = init,
// start(next) = 2^decay start + sum, over the sums (init may be the final state's buffer, which
// another block than the first segment's writes).  One thread per four state entries, the
// sums kAhead segments ahead of their use; a sequence of one segment is left alone.
__global__ void __launch_bounds__(256)
linrec_chain_kernel(const LinrecSeqs seqs, int H, int quads, bool rev, int64_t seg, bool by_rows,
                    const float *__restrict__ init, float *__restrict__ state, const float *__restrict__ decay) {
    const int64_t chain = blockIdx.x, n = chain / H;
    const int h = (int)(chain % H), e = blockIdx.y * 256 + threadIdx.x;
    int64_t lo, hi;
    seq_range(seqs, n, lo, hi);
    const int64_t segs = hi > lo ? (hi - lo + seg - 1) / seg : 1;
    const int base = linrec::state_slot(by_rows, (int)(lo / seg + n), lo, seg, n);
    if (segs < 2 || e >= quads) return;
    float4 s = init ? reinterpret_cast<const float4 *>(init)[chain * quads + e] : make_float4(0.f, 0.f, 0.f, 0.f);
    auto at = [&](int64_t i) { return (base + (rev ? segs - 1 - i : i)) * H + h; };
    float4 *st = reinterpret_cast<float4 *>(state);
    constexpr int kAhead = 8;
    for (int64_t i0 = 0; i0 < segs; i0 += kAhead) {
        float4 x[kAhead];
        float g[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {   // (the last segment has no sum)
            const bool has = i0 + k + 1 < segs;
            x[k] = has ? st[at(i0 + k) * quads + e] : make_float4(0.f, 0.f, 0.f, 0.f);
            g[k] = has ? decay[at(i0 + k)] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (i0 + k >= segs) break;
            st[at(i0 + k) * quads + e] = s;
            const float f = linrec::ex2(g[k]);
            s.x = fmaf(f, s.x, x[k].x); s.y = fmaf(f, s.y, x[k].y);
            s.z = fmaf(f, s.z, x[k].z); s.w = fmaf(f, s.w, x[k].w);
        }
    }
}

int dispatch(const CUtensorMap *m, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s) {
    if (a.p.dk == 128)
        return a.p.dv == 128 ? linrec::launch_128_128(m, a, dot, grid, s) : linrec::launch_128_64(m, a, dot, grid, s);
    return a.p.dv == 128 ? linrec::launch_64_128(m, a, dot, grid, s) : linrec::launch_64_64(m, a, dot, grid, s);
}

// Tokens of a segment; at least seqs.total when the chains are not cut.
//
// Sequences of one length: the number of segments with the least work on the busiest SM, in
// chunks of the output launch; the launch that sums the states reads half as much and skips each
// chain's last segment, and the cut costs about eight chunks' time in launches.
// Packed sequences: their lengths are on the device.  Segments of half an SM's share of
// all rows, 512 tokens at least, keep one long sequence from holding up the rest; shorter
// sequences stay whole.  Forward / backward of 20011 rows x 8 heads of 64 in 23 sequences (longest 4608)
// and of 16384 x 4 of 128 in 3 (11512), us on the GPU, by the least segment: 256 tokens 69 / 244 and
// 56 / 254, 512 69 / 244 and 40 / 179, 1024 76 / 263 and 57 / 247, 2048 107 / 363 and 96 / 401.
int64_t segment_tokens(const LinrecSeqs &s, int64_t H) {
    const int64_t whole = (s.total / kAnchor + 1) * kAnchor, per = kAnchor / linrec::kChunk;
    if (s.cu) {
        const int64_t share = (s.total * H / (2 * kSms) + kAnchor - 1) / kAnchor * kAnchor, seg = share < 2 * kAnchor ? 2 * kAnchor : share;
        return seg < whole ? seg : whole;
    }
    const int64_t chains = s.N * H, nc = (s.T + linrec::kChunk - 1) / linrec::kChunk;
    double best = (double)((chains + kSms - 1) / kSms) * nc;
    int64_t seg = whole;
    const int64_t most = 2 + 4 * kSms / chains;   // further cuts add launches' work and no blocks side by side
    for (int64_t cut = 2; cut <= most && cut * per <= nc; ++cut) {
        const int64_t len = ((nc + cut - 1) / cut + per - 1) / per * per, segs = (nc + len - 1) / len;
        const double cost = (double)((chains * segs + kSms - 1) / kSms) * len +
                            0.5 * (double)((chains * (segs - 1) + kSms - 1) / kSms) * len + 8;
        if (cost < best) {
            best = cost;
            seg = len * linrec::kChunk;
        }
    }
    return seg;
}

int64_t segment_slots(const LinrecSeqs &s, int64_t seg) { return s.total / seg + s.N; }   // blocks a head
// Of the segments' states: whole sequences have none, so many of them take no room.
bool slots_by_rows(const LinrecSeqs &s, int64_t seg) { return s.total / seg + 1 < s.N; }
int64_t state_slots(const LinrecSeqs &s, int64_t seg) {
    return slots_by_rows(s, seg) ? 2 * (s.total / seg) + 1 : segment_slots(s, seg);
}

}  // namespace

bool linrec_tc_supported(const LinrecSeqs &s, int64_t H, bool in_bf16, bool out_bf16) {
    // Up to 16 tokens the token recurrence is faster (forward / backward, us on the GPU: T 16, one chain of
    // 64 x 64 4.8 / 16.9 against 6.5 / 22.8; 1024 chains of 128 x 128 51.8 / 164 against 54.4 / 186), from 32
    // on the chunks are, but for many short chains of 64 x 64 (T 32, one chain 8.0 / 27.0 against 6.7 /
    // 23.5; 1024 chains of 128 x 128 92.9 / 305 against 55.1 / 190, of 64 x 64 27.3 / 96.0 against 47.1 / 161).
    // Packed sequences go by all their rows, which may be one sequence's.
    return in_bf16 && out_bf16 && (s.cu ? s.total : s.T) > 16 && s.total < ((int64_t)1 << 31) - 64 &&
           segment_slots(s, segment_tokens(s, H)) * H < ((int64_t)1 << 31);
}

size_t linrec_tc_workspace_bytes(const LinrecSeqs &s, int64_t H, int dk, int dv) {
    const int64_t seg = segment_tokens(s, H);
    if (seg >= s.total) return 0;
    return sizeof(float) * (size_t)(state_slots(s, seg) * H) * ((size_t)dk * dv + 4);
}

int launch_linrec_tc(const LinrecPass &p, void *workspace, int *status, cudaStream_t stream) {
    const LinrecSeqs &s = p.seqs;
    CUtensorMap m[5];
    if (!make_map(&m[0], p.q, s.total, p.H, p.dk) || !make_map(&m[1], p.k, s.total, p.H, p.dk) ||
        !make_map(&m[2], p.v, s.total, p.H, p.dv) || !make_map(&m[3], p.dot ? p.y : p.v, s.total, p.H, p.dv) ||
        !make_map(&m[4], p.out, s.total, p.H, p.dv))
        return kErrCuda;
    TcArgs a{};
    a.p = p;
    a.status = status;
    a.seg = segment_tokens(s, p.H);
    const unsigned grid = (unsigned)(segment_slots(s, a.seg) * p.H);
    if (a.seg < s.total) {
        a.by_rows = slots_by_rows(s, a.seg);
        a.seg_state = (float *)workspace;
        a.seg_decay = a.seg_state + (size_t)state_slots(s, a.seg) * p.H * p.dk * p.dv;
        if (!p.chained) {
            a.sums = true;
            int rc = dispatch(m, a, false, grid, stream);
            if (rc != kOk) return rc;
            const int quads = p.dk * p.dv / 4;
            linrec_chain_kernel<<<dim3((unsigned)(s.N * p.H), (unsigned)(quads / 256)), 256, 0, stream>>>(
                s, p.H, quads, p.rev, a.seg, a.by_rows, p.init, a.seg_state, a.seg_decay);
            if (cudaGetLastError() != cudaSuccess) return kErrCuda;
            a.sums = false;
        }
    }
    return dispatch(m, a, p.dot != nullptr, grid, stream);
}

}  // namespace dr
