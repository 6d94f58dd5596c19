// linrec_tc.cuh -- the additive gated linear recurrence on the 5th-generation tensor cores
// (tcgen05, TMEM, TMA) for bf16 rows, in chunks of 64 tokens.  The passes and their use for
// the gradients: linrec.h.
//
// Inside a chunk started from the state S, with c_r the log2 decay of the chunk's tokens up to
// and including r, e the chunk's last token, and (forwards) s <= r:
//     P_rs = 2^(c_r - c_s) q_r.k_s          out = diag(2^c) Q S + P V
//     S   <- 2^c_e S + (diag(2^(c_e - c)) K)^T V = 2^c_e S + Kt^T V.
// A backwards pass runs the chunks and the masks the other way, with c_r the decay of the
// tokens behind the chunk's first up to r and c_e including the first token behind the chunk:
//     P_rs = 2^(c_s - c_r) q_r.k_s (s >= r),  out = diag(2^(c_e - c)) Q S + P V,
//     S   <- 2^c_e S + (diag(2^c) K)^T V.
//
// Everything is kept transposed, so that the value channels are the tensor core's 128 rows:
//     X    = Q K^T           [64 x 64]     (rows 64..127 of the instruction's M are not used)
//     R^T  = S^T Q^T         [dv x 64]     S^T from tensor memory
//     O^T  = V^T P^T         [dv x 64]     V as loaded, an MN-major operand
//     D^T  = V^T Kt          [dv x dk]
// The state itself stays in the registers of eight warps in fp32 (S = 2^c_e S + D by fused
// multiply-add, so no truncation of the tensor core's accumulator builds up over a long
// sequence); each chunk it is written to tensor memory as R's bf16 operand.
//
// Precision.  Products of loaded rows are exact in fp32.  Kt = diag(..) K is split into three
// bf16 terms (24 bits, D is three products), so the state is an fp32 result.  P and the
// state operand of R enter as one bf16 each: for the bf16 output they are rounded once
// more than it is, each by at most half a step.  The log-decay gradient needs more (mode
// kDot): R takes the state in three bf16 terms, and the intra-chunk part of out.y is
// summed from the fp32 products X and X2 = Y V^T directly,
//     out_r.y_r (without the row's own term) = 2^c_r R_r.y_r + sum_{s != r} P_rs (y_r.v_s).
// log2 decays are summed in fp64 and split into a multiple of 2^-10 and a remainder, so
// that differences of prefix sums are exact whatever lies between (log alpha is taken as at least
// -120: exp(-120) is 0 in fp32, which makes -inf a full reset).
//
// Work split: one CTA per (sequence, head, segment) walks its chunks.  Warps 0..7 hold the state,
// warps 8..15 build P and Kt and write the outputs, warp 16 issues the TMA loads and scans the
// gates, one thread of warp 17 issues the MMAs.  Few long chains are cut into segments: a
// first launch sums each segment's state from zero (keys and values only), a small kernel
// chains them (the transition is the scalar 2^(sum c)), a second launch runs all segments
// from their true start states.
//
// A sequence's last chunk may hold rows of the next sequence or none: value rows behind the
// end are zeroed in shared memory, Kt and P are built as zero there, and the outputs leave by
// plain stores of the valid rows.  Every wait is bounded: on expiry the kernel records
// DR_ERR_TIMEOUT, runs its remaining steps without waiting, drains its copies and MMAs,
// frees its tensor memory and returns.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "linrec.h"
#include "tc_common.cuh"
#include "umma.cuh"

namespace dr {
namespace linrec {

using namespace umma;
using tc::pack_bf16;
using tc::wait_cycles;

constexpr int kChunk = 64;
constexpr int kStateWarps = 8, kEdgeWarps = 8, kLoadWarp = 16, kMmaWarp = 17, kThreads = 18 * 32;

struct TcArgs {
    LinrecPass p;
    int *status;
    int64_t seg;          // tokens of a segment, a multiple of kAnchor
    bool sums;            // first launch over segments: states from zero, no outputs
    float *seg_state;     // [slot][h][dk dv] in the caller's orientation: the segments' sums, then start states
    float *seg_decay;     // [slot][h] log2 decay over a segment
};

// Sequence n's segment j is slot lo / seg + n + j (every sequence has at least one); finds
// (n, j) of a slot, or false.
__device__ __forceinline__ bool find_segment(const LinrecSeqs &s, int64_t seg, int64_t slot, int64_t &n, int64_t &j) {
    int64_t a = 0, b = s.N - 1;   // the last n whose first slot is at most `slot`
    while (a < b) {
        const int64_t m = (a + b + 1) >> 1;
        int64_t lo, hi;
        seq_range(s, m, lo, hi);
        if (lo / seg + m <= slot) a = m;
        else b = m - 1;
    }
    int64_t lo, hi;
    seq_range(s, a, lo, hi);
    n = a;
    j = slot - (lo / seg + a);
    const int64_t runs = hi > lo ? (hi - lo + seg - 1) / seg : 1;
    return j >= 0 && j < runs;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(smem_u32(dst)), "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void tma_store_3d(const void *tmap, const void *src, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(tmap), "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ float ex2(float x) {   // 2^x, two ulp; 0 below the normal range
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
// The upper halves of two fp32 values: their leading 8 bits, truncated, as a bf16 pair; and the
// exact rest.  Three of these hold all 24 bits of a value.
__device__ __forceinline__ uint32_t take_bf16(float2 &x) {
    const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
    const float2 top = make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u));
    x = fma2(top, make_float2(-1.f, -1.f), x);
    return __byte_perm(a, b, 0x7632);
}
__device__ __forceinline__ uint32_t last_bf16(float2 x) {
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
// Largest log2 decay over a chunk for which P's factor 2^(c_r - c_s) is formed as a product of
// two powers around the chunk's middle, 2^(c_r - c_31) 2^(c_31 - c_s).
constexpr float kFactorSpan = 60.f;

// Shared memory.  A stage holds [Y? V | ...panels] and [Q K | ...panels], panels of 64 channels
// x 64 tokens (8 KB, 128-byte swizzle): every panel used as the first half of a 128-row
// operand has a loaded panel behind it, and so has V's when dv = 64.
template <int DK, int DV, bool DOT>
struct Layout {
    static constexpr int PK = DK / 64, PV = DV / 64;
    static constexpr int STAGES = DOT ? 2 : 3, NP = DOT ? 2 : 1;   // loaded chunks; buffers of P
    static constexpr uint32_t V_STEP = DOT ? 16384 : 8192, Y0 = 0, V0 = DOT ? 8192 : 0;
    static constexpr uint32_t Q0 = PV * V_STEP, K0 = Q0 + 8192, QK_STEP = 16384;
    static constexpr uint32_t STAGE = Q0 + PK * QK_STEP;
    static constexpr uint32_t KT = STAGES * STAGE;           // Kt: three terms of PK panels
    static constexpr uint32_t P = KT + 3 * PK * 8192;
    static constexpr uint32_t OUT = P + NP * 8192;           // output staging, PV panels
    static constexpr uint32_t SMALL = OUT + PV * 8192;
    // per stage: c [66] as (multiple of 2^-10, remainder), the last pair's first word for whether
    // P's factors are products; 2^.. factors of R, Kt, P's rows and P's columns [64] each
    static constexpr uint32_t GATE = 66 * 8 + 64 * 4 * 4;
    static constexpr uint32_t DOTS = SMALL + STAGES * GATE;  // (kDot) [3][2][64] of X X2, [4][64] of R, [8] of the state
    static constexpr uint32_t DOT_R = 3 * 2 * 64, DOT_S = DOT_R + 4 * 64;
    static constexpr uint32_t BARS = DOTS + (DOT ? (DOT_S + 8) * 4 : 0);
    static constexpr uint32_t TOTAL = BARS + 32 * 8;
    static_assert(TOTAL + 1024 <= 227 * 1024 && KT % 1024 == 0 && SMALL % 16 == 0 && BARS % 8 == 0, "layout");
    // tensor memory: U (X, then O^T) of two chunks, X2 (kDot) or a second R, R, D, the state operand
    static constexpr uint32_t TM_U = 0, TM_X2 = 128, TM_R = 192, TM_D = 256;
    static constexpr int ND = DOT && DK == 128 ? 2 : 1;      // D comes in this many parts, one at a time
    static constexpr int DW = DK / ND;
    static constexpr uint32_t TM_S = DOT ? 320 : 384;        // terms of DK / 2 columns
    static_assert(TM_D + DW <= TM_S && TM_S + (DOT ? 3 : 1) * DK / 2 <= 512, "tensor memory");
};

template <int DK, int DV, bool DOT>
__global__ void __launch_bounds__(kThreads, 1)
linrec_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap ty,
                    const __grid_constant__ CUtensorMap to, const TcArgs a) {
    using L = Layout<DK, DV, DOT>;
    constexpr int PK = L::PK, PV = L::PV, NS = DOT ? 3 : 1, NR = DOT ? 1 : 2, ND = L::ND;
    constexpr int kStages = L::STAGES;
    const LinrecPass &p = a.p;
    const int H = p.H, h = (int)(blockIdx.x % H);
    const int64_t slot = blockIdx.x / H;
    int64_t n, j, lo, hi;
    if (!find_segment(p.seqs, a.seg, slot, n, j)) return;
    seq_range(p.seqs, n, lo, hi);
    const bool rev = p.rev, outputs = !a.sums;
    const int64_t segs = hi > lo ? (hi - lo + a.seg - 1) / a.seg : 1;
    const bool last_run = rev ? j == 0 : j == segs - 1, first_run = rev ? j == segs - 1 : j == 0;
    if (a.sums && last_run) return;            // nobody needs its sum
    const int64_t s_lo = lo + j * a.seg, s_hi = min(hi, s_lo + a.seg);
    const int chunks = (int)((s_hi - s_lo + kChunk - 1) / kChunk);
    if (chunks == 0 && (!p.fin || !outputs)) return;

    extern __shared__ unsigned char dsm_raw[];
    unsigned char *sm = align1024(dsm_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_load = bars, *b_gate = bars + 3, *b_free = bars + 6;   // [kStages]
    uint64_t *b_x = bars + 9;          // X (and X2) of a chunk is there
    uint64_t *b_built = bars + 10;     // P, Kt are built, X and X2 read
    uint64_t *b_d = bars + 11;         // [ND] D is there
    uint64_t *b_dread = bars + 13;     // [ND] D is read
    uint64_t *b_s = bars + 15;         // the state operand is there
    uint64_t *b_r = bars + 16;         // R is there: the state operand may be replaced
    uint64_t *b_o = bars + 17;         // R and O are there
    uint64_t *b_oread = bars + 18;     // R and O are read
    uint64_t *b_end = bars + 19;       // every MMA is done
    __shared__ uint32_t tmem_s;
    __shared__ int abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(b_load + i, 1);
            mbar_init(b_gate + i, 1);
            mbar_init(b_free + i, 1 + kEdgeWarps + kStateWarps);
        }
        mbar_init(b_x, 1);
        mbar_init(b_built, kEdgeWarps);
        for (int i = 0; i < ND; ++i) {
            mbar_init(b_d + i, 1);
            mbar_init(b_dread + i, kStateWarps / ND);
        }
        mbar_init(b_s, kStateWarps);
        mbar_init(b_r, 1);
        mbar_init(b_o, 1);
        mbar_init(b_oread, kEdgeWarps);
        mbar_init(b_end, 1);
        abort_s = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_s, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_s;
    volatile int *aborted = &abort_s;
    // `k`-th completion of a barrier (k = 0, 1, ..); after an expiry nobody waits any more
    auto wait = [&](uint64_t *bar, int k) {
        if (!mbar_try_wait(bar, k & 1) && !*aborted && !wait_cycles(bar, k & 1)) {
            *aborted = 1;
            atomicExch(a.status, kErrTimeout);
        }
        tc_fence_after();
    };
    auto stage = [&](int it) { return sm + (it % kStages) * L::STAGE; };
    auto gate_c = [&](int it) { return reinterpret_cast<float2 *>(sm + L::SMALL + (it % kStages) * L::GATE); };
    auto gate_f = [&](int it) { return reinterpret_cast<float *>(gate_c(it) + 66); };   // [4][64] factors
    auto chunk_of = [&](int it) { return rev ? chunks - 1 - it : it; };
    auto row_of = [&](int it) { return s_lo + (int64_t)chunk_of(it) * kChunk; };
    auto count_of = [&](int it) { return (int)min((int64_t)kChunk, s_hi - row_of(it)); };

    if (warp == kLoadWarp) {
        // ---------------------------------------------------------------- loads and gates
        const uint32_t bytes = 8192u * (outputs ? 2 * PK + PV + (DOT ? PV : 0) : PK + PV);
        double total = 0.0;
        float x[2];
        int issued = 0;   // (lane 0) chunks whose loads were issued; none after an expiry
        auto load_gates = [&](int it) {   // two tokens a lane; backwards the tokens one further on
            const int64_t t = row_of(it) + 2 * lane + (rev ? 1 : 0), end = rev ? hi : row_of(it) + count_of(it);
#pragma unroll
            for (int e = 0; e < 2; ++e) x[e] = p.la && t + e < end ? p.la[(t + e) * H + h] : 0.f;
        };
        if (chunks > 0) load_gates(0);
        for (int it = 0; it < chunks; ++it) {
            const int s = it % kStages;
            if (it >= kStages) wait(b_free + s, it / kStages - 1);
            __syncwarp();
            if (lane == 0 && !*aborted) {
                unsigned char *st = stage(it);
                issued = it + 1;
                const int row = (int)row_of(it);
                mbar_arrive_expect_tx(b_load + s, bytes);
                for (int b = 0; b < PK; ++b) {
                    if (outputs) tma_load_3d(st + L::Q0 + b * L::QK_STEP, &tq, b_load + s, 64 * b, h, row);
                    tma_load_3d(st + L::K0 + b * L::QK_STEP, &tk, b_load + s, 64 * b, h, row);
                }
                for (int b = 0; b < PV; ++b) {
                    if (DOT && outputs) tma_load_3d(st + L::Y0 + b * L::V_STEP, &ty, b_load + s, 64 * b, h, row);
                    tma_load_3d(st + L::V0 + b * L::V_STEP, &tv, b_load + s, 64 * b, h, row);
                }
            }
            constexpr double kLog2e = 1.4426950408889634074;
            const double y0 = kLog2e * fmaxf(x[0], -120.f), y1 = kLog2e * fmaxf(x[1], -120.f);
            if (it + 1 < chunks) load_gates(it + 1);
            double c = y0 + y1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double z = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += z;
            }
            const double ce = __shfl_sync(0xffffffffu, c, 31), c0 = c - y1;   // c0, c: up to its first, its second token
            total += ce;
            float2 *g = gate_c(it);
            float *gr = gate_f(it);
            auto split = [](double v) {
                const float big = (float)(rint(v * 1024.0) * (1.0 / 1024.0));
                return make_float2(big, (float)(v - (double)big));
            };
            if (rev) {
                g[2 * lane + 1] = split(c0);
                g[2 * lane + 2] = split(c);
                if (lane == 0) g[0] = make_float2(0.f, 0.f);
                const double cb = c0 - y0;   // c of token 2 lane
                gr[2 * lane] = ex2((float)(ce - cb));
                gr[2 * lane + 1] = ex2((float)(ce - c0));
                gr[64 + 2 * lane] = ex2((float)cb);
                gr[64 + 2 * lane + 1] = ex2((float)c0);
                const double mid = __shfl_sync(0xffffffffu, c0, 15);   // c of token 31
                gr[128 + 2 * lane] = ex2((float)(mid - cb));
                gr[128 + 2 * lane + 1] = ex2((float)(mid - c0));
                gr[192 + 2 * lane] = ex2((float)(cb - mid));
                gr[192 + 2 * lane + 1] = ex2((float)(c0 - mid));
            } else {
                g[2 * lane] = split(c0);
                g[2 * lane + 1] = split(c);
                if (lane == 31) g[64] = split(c);
                gr[2 * lane] = ex2((float)c0);
                gr[2 * lane + 1] = ex2((float)c);
                gr[64 + 2 * lane] = ex2((float)(ce - c0));
                gr[64 + 2 * lane + 1] = ex2((float)(ce - c));
                const double mid = __shfl_sync(0xffffffffu, c, 15);
                gr[128 + 2 * lane] = ex2((float)(c0 - mid));
                gr[128 + 2 * lane + 1] = ex2((float)(c - mid));
                gr[192 + 2 * lane] = ex2((float)(mid - c0));
                gr[192 + 2 * lane + 1] = ex2((float)(mid - c));
            }
            if (lane == 0) g[65].x = -ce < (double)kFactorSpan ? 1.f : 0.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_gate + s);
        }
        if (a.sums && lane == 0) a.seg_decay[slot * H + h] = (float)total;
        // the loads have landed before the block ends, also after an expiry
        if (lane == 0)
            for (int it = max(0, issued - kStages); it < issued; ++it) wait_cycles(b_load + it % kStages, (it / kStages) & 1);
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------- MMA issue
        if (lane == 0 && chunks > 0) {
            constexpr uint32_t ID_KK = idesc_bf16(128, 64, false, false), ID_MK = idesc_bf16(128, 64, true, false),
                               ID_MM = idesc_bf16(128, L::DW, true, true);
            const uint64_t dK = smem_desc_sw128(smem_u32(sm), 16, 1024);              // K-major
            const uint64_t dV = smem_desc_sw128(smem_u32(sm), PV == 2 ? L::V_STEP : 8192, 1024);   // MN-major, V panels
            const uint64_t dT = smem_desc_sw128(smem_u32(sm), 8192, 1024);            // MN-major, Kt panels
            auto off = [&](const unsigned char *x) { return (uint32_t)(x - sm); };
            auto scores = [&](int it) {
                const uint32_t st = off(stage(it));
                for (int ks = 0; ks < 4 * PK; ++ks) {
                    const uint32_t o = st + (ks >> 2) * L::QK_STEP + (ks & 3) * 32;
                    mma_bf16(tm + L::TM_U + 64 * (it & 1), desc_add(dK, o + L::Q0), desc_add(dK, o + L::K0), ID_KK, ks > 0);
                }
                if (DOT)
                    for (int ks = 0; ks < 4 * PV; ++ks) {
                        const uint32_t o = st + (ks >> 2) * L::V_STEP + (ks & 3) * 32;
                        mma_bf16(tm + L::TM_X2, desc_add(dK, o + L::Y0), desc_add(dK, o + L::V0), ID_KK, ks > 0);
                    }
                mma_commit(b_x);
            };
            if (outputs) {
                wait(b_load, 0);
                scores(0);
            }
            for (int it = 0; it < chunks; ++it) {
                const uint32_t st = off(stage(it));
                wait(b_built, it);   // (X2 is read then, too)
                if (!outputs) wait(b_load + it % kStages, it / kStages);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    if (ND == 2) {
                        if (d == 1 || it > 0) wait(b_dread + (d ^ 1), d == 1 ? it : it - 1);   // one half at a time
                    } else if (it > 0) {
                        wait(b_dread, it - 1);
                    }
                    for (int t = 0; t < 3; ++t)
                        for (int ks = 0; ks < 4; ++ks)
                            mma_bf16(tm + L::TM_D, desc_add(dV, st + L::V0 + ks * 2048),
                                     desc_add(dT, L::KT + (t * PK + d) * 8192 + ks * 2048),
                                     ID_MM, t + ks > 0);
                    mma_commit(b_d + d);
                }
                if (outputs) {
                    // the next chunk's X, first if its rows are there already
                    bool next = it + 1 < chunks;
                    auto next_scores = [&]() {
                        wait(b_load + (it + 1) % kStages, (it + 1) / kStages);
                        if (it >= 1) wait(b_oread, it - 1);      // O of the chunk before is read
                        scores(it + 1);
                        next = false;
                    };
                    if (next && mbar_test(b_load + (it + 1) % kStages, ((it + 1) / kStages) & 1)) next_scores();
                    wait(b_s, it);
                    if (NR == 1 && it >= 1) wait(b_oread, it - 1);
                    const uint32_t r = tm + (NR == 2 && (it & 1) ? L::TM_X2 : L::TM_R);
                    for (int t = 0; t < NS; ++t)
                        for (int ks = 0; ks < 4 * PK; ++ks)
                            mma_bf16_ts(r, tm + L::TM_S + t * (DK / 2) + 8 * ks,
                                        desc_add(dK, st + L::Q0 + (ks >> 2) * L::QK_STEP + (ks & 3) * 32), ID_KK, t + ks > 0);
                    mma_commit(b_r);
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16(tm + L::TM_U + 64 * (it & 1), desc_add(dV, st + L::V0 + ks * 2048),
                                 desc_add(dK, L::P + (it % L::NP) * 8192 + ks * 32), ID_MK, ks > 0);
                    mma_commit(b_o);
                    mma_commit(b_free + it % kStages);
                    if (next) next_scores();
                } else {
                    mma_commit(b_free + it % kStages);
                }
            }
            mma_commit(b_end);
            wait_cycles(b_end, 0);
        }
        __syncwarp();
    } else if (warp < kStateWarps) {
        // ---------------------------------------------------------------- state
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, i0 = half * (DK / 2);
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        const bool mine = 32 * quarter < DV;       // value channel `row` exists
        constexpr int NV = DK / 2;
        auto at = [&](int i) { return p.state_t ? (size_t)row * DK + i0 + i : (size_t)(i0 + i) * DV + row; };
        float2 S[NV / 2];
        const float *init = a.sums ? nullptr
                            : first_run ? (p.init ? p.init + (size_t)(n * H + h) * (DK * DV) : nullptr)
                                        : a.seg_state + (size_t)(slot * H + h) * (DK * DV);
#pragma unroll
        for (int i = 0; i < NV / 2; ++i)
            S[i] = init && mine ? make_float2(init[at(2 * i)], init[at(2 * i + 1)]) : make_float2(0.f, 0.f);
        auto put_operand = [&]() {   // S^T as NS bf16 terms
            if (mine) {
#pragma unroll
                for (int b = 0; b < NV / 8; ++b) {
                    uint32_t w[NS][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 x = S[4 * b + i];
                        if (NS == 1) {
                            w[0][i] = pack_bf16(x.x, x.y);   // to the nearest
                        } else {
                            w[0][i] = take_bf16(x);
                            w[NS > 1 ? 1 : 0][i] = take_bf16(x);
                            w[NS - 1][i] = last_bf16(x);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NS; ++t) tmem_st4u(tl + L::TM_S + t * (DK / 2) + (i0 + 8 * b) / 2, w[t]);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_s);
        };
        // this thread's entries of a stored state
        auto anchor_ptr = [&](int it) {
            const int64_t run = (row_of(it) - lo + kChunk - 1) / kAnchor;
            return p.anchor + (size_t)(linrec_slot(lo, n, run) * H + h) * (DK * DV) + half * DV + row;
        };
        auto at_anchor = [&](int it) {   // the chunk ends a run of kAnchor tokens or the sequence
            const int64_t end = row_of(it) + count_of(it);
            return DOT && p.dot && outputs && (end == hi || (end - lo) % kAnchor == 0);
        };
        if (outputs && chunks > 0) put_operand();
        for (int it = 0; it < chunks; ++it) {
            wait(b_gate + it % kStages, it / kStages);
            const float2 ce = gate_c(it)[64], cl = gate_c(it)[63];
            const float decay = ex2(ce.x + ce.y);
            if (rev && at_anchor(it)) {
                float x = 0.f;
                if (mine) {
                    const float *d = anchor_ptr(it);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        x = fmaf(__ldcs(d + (size_t)i * 2 * DV), i & 1 ? S[i / 2].y : S[i / 2].x, x);
                        if (i % 8 == 7) asm volatile("" ::: "memory");   // eight loads at a time: registers
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                float *red = reinterpret_cast<float *>(sm + L::DOTS) + L::DOT_S;
                if (lane == 0) red[warp] = x;
                named_sync(2, 32 * kStateWarps);
                if (tid == 0) {
                    const int64_t run = (row_of(it) - lo + kChunk - 1) / kAnchor;
                    p.inner[linrec_slot(lo, n, run) * H + h] =
                        ex2((ce.x - cl.x) + (ce.y - cl.y)) *
                        (((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7])));
                }
                named_sync(2, 32 * kStateWarps);
            }
            const int d = ND == 2 ? half : 0;
            wait(b_d + d, it);
            if (mine) {
#pragma unroll
                for (int b = 0; b < NV / 16; ++b) {
                    float v[16];
                    tmem_ld16(tl + L::TM_D + (ND == 2 ? 0 : i0) + 16 * b, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        S[8 * b + i] = fma2(make_float2(decay, decay), S[8 * b + i], make_float2(v[2 * i], v[2 * i + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b_dread + d);
                mbar_arrive(b_free + it % kStages);
            }
            if (!rev && at_anchor(it) && mine) {
                float *dst = anchor_ptr(it);
#pragma unroll
                for (int i = 0; i < NV; ++i) __stcs(dst + (size_t)i * 2 * DV, i & 1 ? S[i / 2].y : S[i / 2].x);
            }
            if (outputs && it + 1 < chunks) {
                wait(b_r, it);
                put_operand();
            }
        }
        float *fin = a.sums ? a.seg_state + (size_t)(slot * H + h) * (DK * DV)
                     : last_run && p.fin ? p.fin + (size_t)(n * H + h) * (DK * DV) : nullptr;
        if (fin && mine) {
            // backwards, the state in front of the sequence is decayed by its first token
            const float f = rev && !a.sums && hi > lo && p.la ? expf(p.la[lo * H + h]) : 1.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) fin[at(i)] = f * (i & 1 ? S[i / 2].y : S[i / 2].x);
        }
    } else {
        // ---------------------------------------------------------------- operands and outputs
        const int ew = warp - kStateWarps, quarter = ew & 3, half = ew >> 2, row = 32 * quarter + lane;
        const int et = tid - 32 * kStateWarps;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        const uint32_t smb = smem_u32(sm);
        float *dots = reinterpret_cast<float *>(sm + L::DOTS);

        // Kt and P of chunk `it`.  The four warps whose lanes hold X's rows build P and a quarter
        // of Kt, the other four the rest.
        const int first_piece = (outputs ? (quarter < 2 ? half * 2 + quarter : 4 + 3 * (half * 2 + quarter - 2)) : 2 * ew) * PK;
        const int pieces = (outputs ? (quarter < 2 ? 1 : 3) : 2) * PK;
        auto build = [&](int it) {
            const int s = it % kStages, cnt = count_of(it);
            wait(b_gate + s, it / kStages);
            wait(b_load + s, it / kStages);
            // the last chunk's D has read Kt (and b_built is in this chunk's phase for every warp)
            if (it > 0) wait(b_d + ND - 1, it - 1);
            {
                const unsigned char *k = stage(it) + L::K0;
                const float *f = gate_f(it) + 64;
#pragma unroll
                for (int i = 0; i < 3 * PK; ++i) {
                    if (i >= pieces) break;
                    const uint32_t o = 512 * (first_piece + i) + 16 * lane, b = o >> 13;   // 16 bytes, at the place they have in K's panels
                    const int r = (o >> 7) & 63;
                    const uint4 u = *reinterpret_cast<const uint4 *>(k + b * (L::QK_STEP - 8192) + o);
                    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                    uint32_t w[3][4];
                    const float x = f[r];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 y = mul2(make_float2(lo_bf16(in[e]), hi_bf16(in[e])), make_float2(x, x));
                        if (r >= cnt) y = make_float2(0.f, 0.f);
                        w[0][e] = take_bf16(y);
                        w[1][e] = take_bf16(y);
                        w[2][e] = last_bf16(y);
                    }
#pragma unroll
                    for (int c = 0; c < 3; ++c) sts128(smb + L::KT + c * PK * 8192 + o, w[c][0], w[c][1], w[c][2], w[c][3]);
                }
                if (cnt < kChunk) {   // rows of no token are zero values
                    const int per = 8 * (kChunk - cnt);
                    for (int i = et; i < PV * per; i += 32 * kEdgeWarps)
                        sts128(smem_u32(stage(it)) + L::V0 + (i / per) * L::V_STEP + cnt * 128 + (i % per) * 16, 0, 0, 0, 0);
                }
            }
            if (outputs && quarter < 2) {
                // P: row `row`, columns 32 half ..
                const uint32_t dst = smb + L::P + (it % L::NP) * 8192 + row * 128;
                wait(b_x, it);
                if (L::NP == 1 && it > 0) wait(b_o, it - 1);   // the last chunk's O has read P
                float m = 0.f;
                if (rev ? quarter <= half : quarter >= half) {
                    const bool diagonal = quarter == half || cnt < kChunk;
                    const float2 *c = gate_c(it);
                    const bool product = c[65].x != 0.f;
                    const float2 cr = c[row];
                    const float *fs = gate_f(it) + 192 + 32 * half;
                    const float fr = gate_f(it)[128 + row];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float x[16], x2[16];
                        tmem_ld16(tl + L::TM_U + 64 * (it & 1) + 32 * half + 16 * b, x);
                        if (DOT) tmem_ld16(tl + L::TM_X2 + 32 * half + 16 * b, x2);
                        tmem_wait_ld();
                        if (product) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                const float4 f4 = *reinterpret_cast<const float4 *>(fs + 16 * b + i);
                                x[i] *= f4.x * fr;
                                x[i + 1] *= f4.y * fr;
                                x[i + 2] *= f4.z * fr;
                                x[i + 3] *= f4.w * fr;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 cs = c[32 * half + 16 * b + i];
                                const float d = (cr.x - cs.x) + (cr.y - cs.y);
                                x[i] *= ex2(rev ? -d : d);
                            }
                        }
                        if (diagonal) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int col = 32 * half + 16 * b + i;
                                const bool in = rev ? col >= row && col < cnt : col <= row;
                                x[i] = in ? x[i] : 0.f;
                                if (DOT) x2[i] = in && col != row ? x2[i] : 0.f;
                            }
                        }
                        if (DOT) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) m = fmaf(x[i], x2[i], m);
                        }
#pragma unroll
                        for (int g = 0; g < 2; ++g)
                            sts128(dst + ((((4 * half + 2 * b + g) ^ row) & 7) << 4), pack_bf16(x[8 * g], x[8 * g + 1]),
                                   pack_bf16(x[8 * g + 2], x[8 * g + 3]), pack_bf16(x[8 * g + 4], x[8 * g + 5]),
                                   pack_bf16(x[8 * g + 6], x[8 * g + 7]));
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 4; ++g) sts128(dst + ((((4 * half + g) ^ row) & 7) << 4), 0, 0, 0, 0);
                }
                if (DOT) dots[((it % 3) * 2 + half) * 64 + row] = m;
            }
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_built);
        };

        if (chunks > 0) build(0);
        for (int it = 0; it < chunks; ++it) {
            if (it + 1 < chunks) build(it + 1);
            if (!outputs) {
                __syncwarp();
                if (lane == 0) mbar_arrive(b_free + it % kStages);
                continue;
            }
            const int cnt = count_of(it);
            if (et == 0) bulk_wait_read_all();   // the staging has left
            named_sync(1, 32 * kEdgeWarps);
            wait(b_o, it);
            if (32 * quarter < DV) {
                // 32 channels x 32 tokens, transposed on the way: accumulator fragments, stored and
                // (Y) loaded as transposed 8 x 8 matrices
                float2 f[4], z[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    f[b] = *reinterpret_cast<const float2 *>(gate_f(it) + 32 * half + 8 * b + 2 * (lane & 3));
                    z[b] = make_float2(0.f, 0.f);
                }
                // this thread's matrix row: token 8 (matrix / 2) + lane % 8 of 16, channels + 8 (matrix % 2)
                const int tok = 32 * half + 8 * (lane >> 4) + (lane & 7);
#pragma unroll
                for (int g = 0; g < 2; ++g) {   // 16 channels
                    const uint32_t lanes = (uint32_t)(16 * g) << 16;
                    const int ch = 32 * quarter + 16 * g + 8 * ((lane >> 3) & 1);
                    const uint32_t mat = (ch >> 6) * 8192 + tok * 128 + ((((ch >> 3) ^ tok) & 7) << 4);
                    float r[16], o[16];
                    tmem_ld_frag32(tl + lanes + (NR == 2 && (it & 1) ? L::TM_X2 : L::TM_R) + 32 * half, r);
                    tmem_ld_frag32(tl + lanes + L::TM_U + 64 * (it & 1) + 32 * half, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {   // 16 tokens: matrices (b, channels), b = 2 e, 2 e + 1
                        uint32_t w[4], y[4];
                        if (DOT)
                            ldsm_x4_trans(smem_u32(stage(it)) + L::Y0 + mat + (ch >> 6) * (L::V_STEP - 8192) + e * 2048, y);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {   // block b, channels + 8 (i % 2)
                            const int b = 2 * e + (i >> 1), v = 4 * b + 2 * (i & 1);
                            const float2 x = mul2(f[b], make_float2(r[v], r[v + 1]));
                            if (DOT) z[b] = fma2(x, make_float2(lo_bf16(y[i]), hi_bf16(y[i])), z[b]);
                            w[i] = pack_bf16(x.x + o[v], x.y + o[v + 1]);
                        }
                        stsm_x4_trans(smb + L::OUT + mat + e * 2048, w[0], w[1], w[2], w[3]);
                    }
                }
                if (DOT) {   // over the 8 lanes of a token pair
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) {
                            z[b].x += __shfl_xor_sync(0xffffffffu, z[b].x, w);
                            z[b].y += __shfl_xor_sync(0xffffffffu, z[b].y, w);
                        }
                        if (lane < 4)
                            *reinterpret_cast<float2 *>(dots + L::DOT_R + quarter * 64 + 32 * half + 8 * b + 2 * lane) = z[b];
                    }
                }
            }
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b_oread);
                mbar_arrive(b_free + it % kStages);
            }
            named_sync(1, 32 * kEdgeWarps);
            const int64_t base = row_of(it);
            if (cnt == kChunk) {
                if (et == 0) {
                    for (int b = 0; b < PV; ++b) tma_store_3d(&to, sm + L::OUT + b * 8192, 64 * b, h, (int)base);
                    bulk_commit();
                }
            } else {
                for (int i = et; i < cnt * PV * 8; i += 32 * kEdgeWarps) {
                    const int r = i / (PV * 8), b = (i / 8) % PV, c = i % 8;
                    const uint4 u = *reinterpret_cast<const uint4 *>(sm + L::OUT + b * 8192 + r * 128 + (((c ^ r) & 7) << 4));
                    reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + ((size_t)(base + r) * H + h) * DV)[b * 8 + c] = u;
                }
            }
            if (DOT && p.dot && et < cnt) {
                const float *d = dots + (it % 3) * 2 * 64 + et, *e = dots + L::DOT_R + et;
                float x = d[0] + d[64] + e[0] + e[64];
                if (DV == 128) x += e[128] + e[192];
                p.dot[(size_t)h * p.seqs.total + base + et] = x;
            }
        }
        if (et == 0) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

template <int DK, int DV, bool DOT>
int launch(const CUtensorMap *maps, const TcArgs &a, unsigned grid, cudaStream_t stream) {
    const int smem = (int)Layout<DK, DV, DOT>::TOTAL + 1024;
    if (cudaFuncSetAttribute(linrec_chunk_kernel<DK, DV, DOT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return kErrCuda;
    linrec_chunk_kernel<DK, DV, DOT><<<grid, kThreads, smem, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[4], a);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

// one translation unit each (they compile side by side)
int launch_128_128(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s);
int launch_128_64(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s);
int launch_64_128(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s);
int launch_64_64(const CUtensorMap *maps, const TcArgs &a, bool dot, unsigned grid, cudaStream_t s);

}  // namespace linrec
}  // namespace dr
