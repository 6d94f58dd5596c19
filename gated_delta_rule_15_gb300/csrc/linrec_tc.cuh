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
//     X   = Q K^T           [64 x 64]     (rows 64..127 of the instruction's M are not used)
//     R^T = S^T Q^T         [dv x 64]     S^T from tensor memory
//     O^T = V^T P^T         [dv x 64]     V as loaded, an MN-major operand
//     D^T = Vt^T K = V^T Kt [dv x dk]     Vt = diag(w) V, Kt = diag(w) K, w the factors above
// The state itself stays in the registers of eight warps in fp32 (S = 2^c_e S + D by fused
// multiply-add, so no truncation of the tensor core's accumulator builds up over a long
// sequence); each chunk it is written to tensor memory as R's bf16 operand.
//
// Two forms.  Without Y (the forward, the dv pass) the factors w go to the values: Vt^T is made
// from transposed 8 x 8 fragments of V (ldmatrix) straight into tensor memory, K is used as
// loaded, and with P divided by its row's factor f_r of R, O is accumulated onto R and
//     out_r = f_r (R_r + O_r)                  (f_r = 2^max(., -60): below, R_r does not matter)
// With Y (the dq and dk passes of a gated backward) R is needed apart from O, tensor memory is full,
// and Kt is made in shared memory, its first term in K's place.
//
// Precision.  Products of loaded rows are exact in fp32.  Vt, Kt enter as three bf16 terms (all
// 24 bits, D is three products), so the state is an fp32 result.  P and, without Y, the state operand
// of R enter as two bf16 terms each (2^-17 of a value at most is lost), so that the bf16 results are off by
// their own rounding: 1.66e-3 of the 2-norm, as rounding the exact result is.  (One term each: 2.35e-3,
// and 105 instead of 121 us for the forward of B8 T4096 H16 d128, 273 instead of 289 for the backward at
// T2048.)  The log-decay gradient is an fp32 result: with Y, R takes the state in three terms, the third
// over the place of X2 once that is read, and the intra-chunk part of out.y is summed from the fp32
// products X and X2 = Y V^T directly,
//     out_r.y_r (without the row's own term) = f_r R_r.y_r + sum_{s != r} P_rs (y_r.v_s);
// it is 0.5e-6 to 0.9e-6 off in the 2-norm (two terms: 5e-6 to 6e-6, backward 289 instead of 304 us).  Terms are
// accumulated from the small one to the large one, since what the tensor core cuts off a sum goes by
// the sum's size (the other way round 0.8e-6 to 1.4e-6, and states 5e-7 instead of 3e-7).
// log2 decays are held as a multiple of 2^-10, whose sums over a chunk are exact in fp32, and
// a remainder, so that a difference of prefix sums is as exact as a single decay whatever
// lies between (log alpha is taken as at least -120: exp(-120) is 0 in fp32, which makes -inf a full
// reset).
//
// Work split: one CTA per (sequence, head, segment) walks its chunks.  Warps 0..7 hold the state;
// warps 8..15 make Vt, or Kt and P; warps 16..23 write the outputs and, without Y, build P; warp
// 24 issues the TMA loads, warp 27 scans the gates; one thread each of warps 25 and 26 issues the
// MMAs of X, and of D, R and O (D first: the next chunk's Vt waits for it).  Few long chains are cut
// into segments: a first launch sums each segment's state from zero (keys and values only), a
// small kernel chains them (the transition is the scalar 2^(sum c)), a second launch runs all
// segments from their true start states.
//
// What bounds it (B8 T4096 H16 d128, 128 CTAs of 64 chunks, 121 us, 67 % of the copy bandwidth's
// floor): the per-chunk work of 28 warps on an SM, about 8,500 warp instructions in 3,700 cycles,
// 74 % issue on the SMs in use.  What it took to get there, each step as measured (with one term of P
// and of the state): 182 us with eight warps for everything behind the state; 160 with MMAs issued by
// three threads instead of one that waits for them in turn; 141 with less code in the loop (the SM's
// instruction cache missed 16 % and the GPC's, which all its SMs share, ran at 76 % of its rate: rolled
// loops, fp32 gate scan); 131 with building and output on warps of their own; 117 with Vt in tensor memory
// (with Kt in shared memory the chunk moves 336 KB through it, 2,690 cycles at 128 bytes); 112
// with shorter waits; 105 with MMAs issued by an elected lane.  The form with Y runs 14,200 instructions
// in 6,600 cycles a chunk, 67 % issue: a stage's tiles take 4,400 cycles from their request to their
// arrival, shared memory holds two stages, and its loop is larger (the SM's instruction cache misses
// 15 %, the GPC's runs at 84 % of its rate).
//
// A sequence's last chunk may hold rows of the next sequence or none: rows behind the end are
// zeroed in shared memory, Vt, Kt and P are built as zero there, and the outputs leave by
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
constexpr int kStateWarps = 8, kBuildWarps = 8, kOutWarps = 8, kBuild0 = kStateWarps, kOut0 = kBuild0 + kBuildWarps,
              kLoadWarp = kOut0 + kOutWarps, kScoreWarp = kLoadWarp + 1, kUpdateWarp = kLoadWarp + 2, kGateWarp = kLoadWarp + 3,
              kThreads = (kLoadWarp + 4) * 32;
// Registers a thread: launched with kRegs; the state warps take what the others give back.
constexpr int kRegs = 72, kStateRegs = 104, kEdgeRegs = 64, kIssueRegs = 40;
static_assert(kStateWarps * kStateRegs + (kBuildWarps + kOutWarps) * kEdgeRegs + 4 * kIssueRegs <= kThreads / 32 * kRegs,
              "register split");

struct TcArgs {
    LinrecPass p;
    int *status;
    int64_t seg;          // tokens of a segment, a multiple of kAnchor
    bool sums;            // first launch over segments: states from zero, no outputs
    bool by_rows;         // how the states are numbered (state_slot)
    float *seg_state;     // [state slot][h][dk dv] in the caller's orientation: the segments' sums, then start states
    float *seg_decay;     // [state slot][h] log2 decay over a segment
};

// Slot of the state of segment j of a cut sequence, one of more than seg rows from row lo on.  Two
// numberings, the host takes the one with fewer slots: that of the blocks (find_segment), total / seg + N
// of them, or, by rows, 2 (lo / seg) + j: of two cut sequences in a row the second's
// lo / seg is greater by the whole segments d >= 1 of the first, which has at most d + 1 <= 2 d segments.
// lo / seg + j <= total / seg, so 2 (total / seg) + 1 slots do for any number of sequences.  From the
// block's slot of the segment; rows, and slots times heads, fit in 31 bits.
__device__ __forceinline__ int state_slot(bool by_rows, int slot, int64_t lo, int64_t seg, int64_t n) {
    return by_rows ? slot + (int)((uint32_t)lo / (uint32_t)seg) - (int)n : slot;
}

// Sequence n's segment j is slot lo / seg + n + j (every sequence has at least one); finds
// (n, j) of a slot, or false.  By whole warps: 32 sequences are asked at a time, since each
// round of the search is a load's latency at the start of every block (23 sequences by
// bisection: forward of 20011 rows x 8 heads of 64 87 us, this one 78).  Rows fit in 31 bits here.
__device__ __forceinline__ bool find_segment(const LinrecSeqs &s, int64_t seg, int64_t slot, int64_t &n, int64_t &j) {
    int64_t a = 0, b = s.N - 1;   // the last n whose first slot is at most `slot`
    while (a < b) {
        const int64_t step = (b - a + 31) >> 5, m = a + 1 + (threadIdx.x & 31) * step;
        bool in = false;
        if (m <= b) {
            int64_t lo, hi;
            seq_range(s, m, lo, hi);
            in = (uint32_t)lo / (uint32_t)seg + m <= slot;
        }
        const int k = __popc(__ballot_sync(0xffffffffu, in));
        b = min(b, a + k * step);
        if (k > 0) a += 1 + (k - 1) * step;
    }
    int64_t lo, hi;
    seq_range(s, a, lo, hi);
    n = a;
    j = slot - ((uint32_t)lo / (uint32_t)seg + a);
    const int64_t runs = hi > lo ? ((uint32_t)(hi - lo) + (uint32_t)seg - 1) / (uint32_t)seg : 1;
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
// Two fp32 values as two bf16 pairs, each rounded to the nearest: 2^-17 of a value at most is lost.
__device__ __forceinline__ void two_bf16(float2 x, uint32_t &w0, uint32_t &w1) {
    w0 = pack_bf16(x.x, x.y);
    x = fma2(make_float2(lo_bf16(w0), hi_bf16(w0)), make_float2(-1.f, -1.f), x);
    w1 = pack_bf16(x.x, x.y);
}
// Largest log2 decay over a chunk for which P's factor 2^(c_r - c_s) is formed as a product of
// two powers around the chunk's middle, 2^(c_r - c_31) 2^(c_31 - c_s).
constexpr float kFactorSpan = 60.f;

// Shared memory.  A stage holds the panels [V ..] and [Q K | ..], 64 channels x 64 tokens each (8 KB,
// 128-byte swizzle): every panel used as the first half of a 128-row operand has another
// one behind it, and so has V's when dv = 64.  Y, which the outputs read last, has stages of its own.
template <int DK, int DV, bool DOT>
struct Layout {
    static constexpr int PK = DK / 64, PV = DV / 64;
    static constexpr int STAGES = DOT ? 2 : 3, GATES = 4;    // chunks whose rows, whose gates are there
    static constexpr uint32_t V0 = 0, V_STEP = 8192, Q0 = PV * V_STEP, K0 = Q0 + 8192, QK_STEP = 16384;
    static constexpr uint32_t STAGE = Q0 + PK * QK_STEP;
    static constexpr int YS = DOT ? 3 : 0;
    static constexpr uint32_t Y = STAGES * STAGE, Y_STAGE = PV * 8192;
    static constexpr uint32_t KT = Y + YS * Y_STAGE;           // (kDot) Kt's second and third term (the first replaces K)
    static constexpr uint32_t P = KT + (DOT ? 2 * PK * 8192 : 0);   // two chunks' P, its first term
    static constexpr int PLS = DOT ? 1 : 2;                  // stages of P's second term
    static constexpr uint32_t PL = P + 2 * 8192, OUT = PL + PLS * 8192;   // output staging, PV panels
    static constexpr uint32_t SMALL = OUT + PV * 8192;
    // per chunk: c [66] as (multiple of 2^-10, remainder), the last pair's first word for whether
    // P's factors are products; 2^.. factors of R, Kt, P's rows and P's columns [64] each
    static constexpr uint32_t GATE = 66 * 8 + 64 * 4 * 4;
    static constexpr uint32_t DOTS = SMALL + GATES * GATE;   // (kDot) [3][2][64] of X X2, [4][64] of R, [8] of the state
    static constexpr uint32_t DOT_R = 3 * 2 * 64, DOT_S = DOT_R + 4 * 64;
    static constexpr uint32_t BARS = DOTS + (DOT ? (DOT_S + 8) * 4 : 0);
    static constexpr uint32_t TOTAL = BARS + 42 * 8;
    static_assert(TOTAL + 1024 <= 227 * 1024 && KT % 1024 == 0 && SMALL % 16 == 0 && BARS % 8 == 0, "layout");
    // tensor memory.  kDot: U (X, then O^T) of two chunks, X2 (then the state operand's third term), R, D,
    // the other two terms of the state operand.
    // Otherwise: X, R + O, D, two terms of the state operand, three of Vt.
    static constexpr int NU = DOT ? 2 : 1;
    static constexpr uint32_t TM_X2 = 128, TM_R = DOT ? 192 : 64, TM_D = DOT ? 256 : 128;
    static constexpr int HALVES = DOT ? 1 : 2;               // Kt (Vt) is handed over in this many parts
    static constexpr uint32_t TM_S = DOT ? 384 : 256, TM_V = 384;   // terms of DK / 2, of 32 columns
    static_assert(TM_D + DK <= TM_S && TM_S + DK <= (DOT ? 512 : TM_V), "tensor memory");
};

// One lane of a whole warp.  The compiler knows that this is one, and takes the operands of the MMAs
// and copies behind it as they are; behind `lane == 0` it wraps each in a search for equal lanes
// (forward of B8 T4096 H16 d128 144 us instead of 121).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}
// The rest of a wait that was not over at once: at most *polls more polls (each of 60 cycles at
// least: a thirtieth of a second in all); then *polls becomes 0 and nobody waits any more.  Few
// instructions, for the many places that wait, and no call: the register split rules calls out.
constexpr int kPolls = 1 << 20;
__device__ __forceinline__ void wait_longer(uint64_t *bar, uint32_t parity, volatile int *polls) {
    int i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        if (++i > *polls) {
            *polls = 0;
            break;
        }
    }
}

template <int N>
__device__ __forceinline__ void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int DK, int DV, bool DOT>
__global__ void __launch_bounds__(kThreads, 1)
linrec_chunk_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap ty,
                    const __grid_constant__ CUtensorMap to, const TcArgs a) {
    using L = Layout<DK, DV, DOT>;
    constexpr int PK = L::PK, PV = L::PV, NS = DOT ? 3 : 2, NU = L::NU;
    constexpr int kStages = L::STAGES;
    const LinrecPass &p = a.p;
    const int H = p.H, h = (int)(blockIdx.x % H);
    int slot = blockIdx.x / H;   // (64 bits: backward of B8 T2048 H16 d128 2 % slower)
    int64_t n, j, lo, hi;
    if (!find_segment(p.seqs, a.seg, slot, n, j)) return;
    seq_range(p.seqs, n, lo, hi);
    slot = state_slot(a.by_rows, slot, lo, a.seg, n);
    const bool rev = p.rev, outputs = !a.sums;
    const int64_t segs = hi > lo ? ((uint32_t)(hi - lo) + (uint32_t)a.seg - 1) / (uint32_t)a.seg : 1;
    const bool last_run = rev ? j == 0 : j == segs - 1;
    if (a.sums && last_run) return;            // nobody needs its sum
    const int64_t s_lo = lo + j * a.seg, s_hi = min(hi, s_lo + a.seg);
    const int rows = (int)(s_hi - s_lo), chunks = (rows + kChunk - 1) / kChunk;
    if (chunks == 0 && (!p.fin || !outputs)) return;

    extern __shared__ unsigned char dsm_raw[];
    unsigned char *sm = align1024(dsm_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_load = bars, *b_free = bars + 3;   // [kStages] rows are there, are done with
    uint64_t *b_gate = bars + 6, *b_gfree = bars + 10;   // [GATES] the same of the gates
    uint64_t *b_x = bars + 14;         // [NU] X of a chunk is there
    uint64_t *b_x2 = bars + 16;        // X2 is there
    uint64_t *b_kt = bars + 17;        // [HALVES] Kt (rows 0..31, 32..63) is built
    uint64_t *b_p = bars + 19;         // [2] P is built, X and X2 are read
    uint64_t *b_d = bars + 21;         // D is there
    uint64_t *b_d1 = bars + 23;        // D has taken Kt's first half
    uint64_t *b_dread = bars + 24;     // D is read
    uint64_t *b_s = bars + 26;         // the state operand is there
    uint64_t *b_r = bars + 27;         // R is there: the state operand (and its third term by X2) may be replaced
    uint64_t *b_o = bars + 28;         // [2] R and O are there
    uint64_t *b_oread = bars + 30;     // [4] R and O are read
    uint64_t *b_end = bars + 34;       // every MMA is done
    uint64_t *b_y = bars + 35, *b_yfree = bars + 38;   // [YS] Y is there, is done with
    // A parity wait tells a phase from its neighbours only: no barrier completes a second
    // time before everyone who waits for it has seen the first.  Where a warp may run ahead of
    // another (X of later chunks, outputs), consecutive chunks take different barriers.
    __shared__ uint32_t tmem_s;
    __shared__ int polls_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(b_load + i, 1);
            mbar_init(b_free + i, 1);
        }
        for (int i = 0; i < L::YS; ++i) {
            mbar_init(b_y + i, 1);
            mbar_init(b_yfree + i, 1 + kOutWarps);   // X2, the outputs
        }
        for (int i = 0; i < L::GATES; ++i) {
            mbar_init(b_gate + i, 1);
            mbar_init(b_gfree + i, kStateWarps + kBuildWarps + (outputs ? kOutWarps : 0));
        }
        for (int i = 0; i < NU; ++i) mbar_init(b_x + i, 1);
        mbar_init(b_x2, 1);
        for (int i = 0; i < L::HALVES; ++i) mbar_init(b_kt + i, kBuildWarps);
        mbar_init(b_d1, 1);
        for (int i = 0; i < 2; ++i) mbar_init(b_p + i, 4);
        mbar_init(b_d, 1);
        mbar_init(b_dread, kStateWarps);
        mbar_init(b_s, kStateWarps);
        mbar_init(b_r, 1);
        for (int i = 0; i < 2; ++i) mbar_init(b_o + i, 1);
        for (int i = 0; i < 4; ++i) mbar_init(b_oread + i, kOutWarps);
        mbar_init(b_end, outputs ? 2 : 1);
        polls_s = kPolls;
        fence_mbar_init();
    }
    if (warp == kUpdateWarp) {
        tmem_alloc(&tmem_s, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_s;
    volatile int *polls = &polls_s;
    // `k`-th completion of a barrier (k = 0, 1, ..); after an expiry nobody waits any more
    auto wait = [&](uint64_t *bar, int k) {
        if (!mbar_try_wait(bar, k & 1)) wait_longer(bar, k & 1, polls);
        tc_fence_after();
    };
    auto stage = [&](int it) { return sm + (it % kStages) * L::STAGE; };
    auto gate_c = [&](int it) { return reinterpret_cast<float2 *>(sm + L::SMALL + (it % L::GATES) * L::GATE); };
    auto gate_f = [&](int it) { return reinterpret_cast<float *>(gate_c(it) + 66); };   // [4][64] factors
    auto chunk_of = [&](int it) { return rev ? chunks - 1 - it : it; };
    auto row_of = [&](int it) { return s_lo + chunk_of(it) * kChunk; };
    auto count_of = [&](int it) { return min(kChunk, rows - chunk_of(it) * kChunk); };

    // P of chunk `nx`, by the warps whose lanes hold X's rows (quarters 0 and 1), 32 columns each: on
    // the diagonal (masked), full or empty.
    auto kind_of = [&](int quarter, int half) { return quarter == half ? 0 : (quarter == 1) != rev ? 1 : 2; };
    auto build_p = [&](int nx, int quarter, int half) {
        const int cnt = count_of(nx), kind = kind_of(quarter, half), row = 32 * quarter + lane;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16), smb = smem_u32(sm);
        wait(b_gate + nx % L::GATES, nx / L::GATES);
        wait(b_x + nx % NU, nx / NU);
        if (DOT) wait(b_x2, nx);
        const uint32_t dst = smb + L::P + (nx & 1) * 8192 + row * 128, low = smb + L::PL + (nx % L::PLS) * 8192 + row * 128;
        const uint32_t xs = tl + 64 * ((uint32_t)nx % NU);
        const float2 ce = gate_c(nx)[64];
        float m = 0.f;
        if (kind < 2) {
            const bool masked = kind == 0 || cnt < kChunk;
            const float2 *c = gate_c(nx);
            const bool product = c[65].x != 0.f;
            const float2 cr = c[row];
            const float *fs = gate_f(nx) + (DOT ? 192 : 128) + 32 * half;
            const float fr = gate_f(nx)[128 + row];
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                float x[16], x2[16];
                tmem_ld16(xs + 32 * half + 16 * b, x);
                if (DOT) tmem_ld16(tl + L::TM_X2 + 32 * half + 16 * b, x2);
                tmem_wait_ld();
                if (product) {
                    const float2 f2 = make_float2(fr, fr);
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 f4 = *reinterpret_cast<const float4 *>(fs + 16 * b + i);
                        float2 fu = make_float2(f4.x, f4.y), fv = make_float2(f4.z, f4.w);
                        if (DOT) {
                            fu = mul2(fu, f2);
                            fv = mul2(fv, f2);
                        }
                        const float2 u = mul2(make_float2(x[i], x[i + 1]), fu), v = mul2(make_float2(x[i + 2], x[i + 3]), fv);
                        x[i] = u.x;
                        x[i + 1] = u.y;
                        x[i + 2] = v.x;
                        x[i + 3] = v.y;
                    }
                } else {
                    const float lr = DOT ? 0.f : fmaxf(rev ? (ce.x - cr.x) + (ce.y - cr.y) : cr.x + cr.y, -kFactorSpan);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 cs = c[32 * half + 16 * b + i];
                        const float d = (cr.x - cs.x) + (cr.y - cs.y);
                        x[i] *= ex2((rev ? -d : d) - lr);
                    }
                }
                if (masked) {
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
                for (int g = 0; g < 2; ++g) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) two_bf16(make_float2(x[8 * g + 2 * i], x[8 * g + 2 * i + 1]), w[0][i], w[1][i]);
                    const uint32_t at = (((4 * half + 2 * b + g) ^ row) & 7) << 4;
                    sts128(dst + at, w[0][0], w[0][1], w[0][2], w[0][3]);
                    sts128(low + at, w[1][0], w[1][1], w[1][2], w[1][3]);
                }
            }
        } else {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const uint32_t at = (((4 * half + g) ^ row) & 7) << 4;
                sts128(dst + at, 0, 0, 0, 0);
                sts128(low + at, 0, 0, 0, 0);
            }
        }
        if (DOT) reinterpret_cast<float *>(sm + L::DOTS)[((nx % 3) * 2 + half) * 64 + row] = m;
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p + (nx & 1));
    };

    if (warp < kStateWarps) {
        more_regs<kStateRegs>();
        // ---------------------------------------------------------------- state
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, i0 = half * (DK / 2);
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        const bool mine = 32 * quarter < DV;       // value channel `row` exists
        constexpr int NV = DK / 2;
        auto at = [&](int i) { return p.state_t ? (size_t)row * DK + i0 + i : (size_t)(i0 + i) * DV + row; };
        float2 S[NV / 2];
        const float *init = a.sums ? nullptr
                            : segs == 1 ? (p.init ? p.init + (size_t)(n * H + h) * (DK * DV) : nullptr)
                                        : a.seg_state + (size_t)(slot * H + h) * (DK * DV);
#pragma unroll
        for (int i = 0; i < NV / 2; ++i)
            S[i] = init && mine ? make_float2(init[at(2 * i)], init[at(2 * i + 1)]) : make_float2(0.f, 0.f);
        auto put_operand = [&](int it) {   // S^T as two bf16 terms, with Y as three
            if (mine) {
#pragma unroll
                for (int b = 0; b < NV / 8; ++b) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 x = S[4 * b + i];
                        // (opaque, so that no term is computed ahead and kept: 550 bytes of spills)
                        asm volatile("" : "+f"(x.x), "+f"(x.y));
                        if (DOT) {   // truncated: with the third all 24 bits
                            w[0][i] = take_bf16(x);
                            w[1][i] = last_bf16(x);
                        } else {
                            two_bf16(x, w[0][i], w[1][i]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) tmem_st4u(tl + L::TM_S + t * (DK / 2) + (i0 + 8 * b) / 2, w[t]);
                }
            }
            if (DOT) {   // the third term goes over X2, which P's warps have read
                wait(b_p + (it & 1), it >> 1);
                if (mine) {
#pragma unroll
                    for (int b = 0; b < NV / 8; ++b) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float2 x = S[4 * b + i];
                            asm volatile("" : "+f"(x.x), "+f"(x.y));
                            take_bf16(x);
                            take_bf16(x);
                            w[i] = last_bf16(x);
                        }
                        tmem_st4u(tl + L::TM_X2 + (i0 + 8 * b) / 2, w);
                    }
                }
            }
            if (mine) tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_s);
        };
        // this thread's entries of a stored state
        auto anchor_ptr = [&](int it) {
            const int64_t run = (row_of(it) - lo + kChunk - 1) / kAnchor;
            return p.anchor + (size_t)(linrec_slot(kAnchor, lo, n, run) * H + h) * (DK * DV) + half * DV + row;
        };
        auto at_anchor = [&](int it) {   // the chunk ends a run of kAnchor tokens or the sequence
            const int64_t end = row_of(it) + count_of(it);
            return DOT && p.dot && outputs && (end == hi || (end - lo) % kAnchor == 0);
        };
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            if (outputs) {
                if (it > 0) wait(b_r, it - 1);
                put_operand(it);
            }
            wait(b_gate + it % L::GATES, it / L::GATES);
            const float2 ce = gate_c(it)[64], cl = gate_c(it)[63];
            const float decay = ex2(ce.x + ce.y);
            if (DOT && rev && it + 1 < chunks && at_anchor(it + 1) && mine) {   // the next one's stored state into L2
                const float *d = anchor_ptr(it + 1) - lane;
#pragma unroll
                for (int i = 0; i < NV; i += 32)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(d + (size_t)(i + lane) * 2 * DV));
            }
            if (rev && at_anchor(it)) {
                float x = 0.f;
                if (mine) {
                    const float *d = anchor_ptr(it);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        x = fmaf(__ldcs(d + (size_t)i * 2 * DV), i & 1 ? S[i / 2].y : S[i / 2].x, x);
                        if (i % 16 == 15) asm volatile("" ::: "memory");   // sixteen loads at a time: registers
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                float *red = reinterpret_cast<float *>(sm + L::DOTS) + L::DOT_S;
                if (lane == 0) red[warp] = x;
                named_sync(2, 32 * kStateWarps);
                if (tid == 0) {
                    const int64_t run = (row_of(it) - lo + kChunk - 1) / kAnchor;
                    p.inner[linrec_slot(kAnchor, lo, n, run) * H + h] =
                        ex2((ce.x - cl.x) + (ce.y - cl.y)) *
                        (((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7])));
                }
                named_sync(2, 32 * kStateWarps);
            }
            wait(b_d, it);
            if (mine) {
#pragma unroll
                for (int b = 0; b < NV / 16; ++b) {
                    float v[16];
                    tmem_ld16(tl + L::TM_D + i0 + 16 * b, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        S[8 * b + i] = fma2(make_float2(decay, decay), S[8 * b + i], make_float2(v[2 * i], v[2 * i + 1]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b_dread);
                mbar_arrive(b_gfree + it % L::GATES);
            }
            if (!rev && at_anchor(it) && mine) {
                float *dst = anchor_ptr(it);
#pragma unroll
                for (int i = 0; i < NV; ++i) __stcs(dst + (size_t)i * 2 * DV, i & 1 ? S[i / 2].y : S[i / 2].x);
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
    } else if (warp < kOut0) {
        fewer_regs<kEdgeRegs>();
        // ---------------------------------------------------------------- Kt
        const int bw = warp - kBuild0;
        const uint32_t smb = smem_u32(sm);
        // Without Y (P belongs to the output warps) Vt, in two halves of the rows, so that the
        // second is made while D takes the first.  With Y, Kt in pieces of 32 x 16 bytes (four
        // rows of a panel), and P: by instructions its diagonal blocks cost three pieces, its full
        // one two, so their warps take fewer pieces (of 32; of 16).
        const int quarter = bw & 3, half = bw >> 2, kind = quarter < 2 ? kind_of(quarter, half) : 3;
        const int none = PK == 2 ? 5 : 3, diag = PK == 2 ? 2 : 0, full = PK == 2 ? 3 : 1;
        const int pieces = kind == 0 ? diag : kind == 1 ? full : none;
        const int first_piece = kind == 3 ? (half * 2 + quarter - 2) * none : 4 * none + (kind == 0 ? half * diag : 2 * diag + (kind == 1 ? 0 : full));
#pragma unroll 1
        for (int it = 0; it < chunks; ++it) {
            const int s = it % kStages, cnt = count_of(it);
            wait(b_gate + it % L::GATES, it / L::GATES);
            wait(b_load + s, it / kStages);
            if (DOT) wait(b_x + it % NU, it / NU);      // K's place may be written
            if (it > 0) wait(L::HALVES == 2 ? b_d1 : b_d, it - 1);   // Kt's other terms, Vt's first half are read
            if (cnt < kChunk) {   // rows of no token are zero values (and keys, where they are not scaled)
                const int per = 8 * (kChunk - cnt);
                for (int i = 32 * bw + lane; i < PV * per; i += 32 * kBuildWarps)
                    sts128(smem_u32(stage(it)) + L::V0 + (i / per) * L::V_STEP + cnt * 128 + (i % per) * 16, 0, 0, 0, 0);
                if (!DOT) {
                    for (int i = 32 * bw + lane; i < PK * per; i += 32 * kBuildWarps)
                        sts128(smem_u32(stage(it)) + L::K0 + (i / per) * L::QK_STEP + cnt * 128 + (i % per) * 16, 0, 0, 0, 0);
                    named_sync(3, 32 * kBuildWarps);   // the warps read one another's rows
                }
            }
            if constexpr (!DOT) {
                // Vt: 16 channels by each warp, 16 tokens at a time: transposed fragments of V, scaled by
                // the tokens' factors, as three bf16 terms in tensor memory
                const int ch = 32 * quarter + 16 * half + 8 * ((lane >> 3) & 1), tok = 8 * (lane >> 4) + (lane & 7);
                const uint32_t src = smem_u32(stage(it)) + L::V0 + (ch >> 6) * L::V_STEP + tok * 128 + ((((ch >> 3) ^ tok) & 7) << 4);
                const uint32_t dst = tm + ((uint32_t)(32 * quarter + 16 * half) << 16) + L::TM_V;
                const float *f = gate_f(it) + 64 + 2 * (lane & 3);
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    if (b == 2) {   // the first half is done
                        tmem_wait_st();
                        fence_proxy_async();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_kt);
                        if (it > 0) wait(b_d, it - 1);
                    }
                    if (32 * quarter < DV) {
                        uint32_t u[4], w[3][4];
                        ldsm_x4_trans(src + b * 2048, u);
                        const float2 f0 = *reinterpret_cast<const float2 *>(f + 16 * b), f1 = *reinterpret_cast<const float2 *>(f + 16 * b + 8);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {   // tokens + 8 (e / 2), channels + 8 (e % 2)
                            float2 y = mul2(make_float2(lo_bf16(u[e]), hi_bf16(u[e])), e < 2 ? f0 : f1);
                            w[0][e] = take_bf16(y);
                            w[1][e] = take_bf16(y);
                            w[2][e] = last_bf16(y);
                        }
#pragma unroll
                        for (int t = 0; t < 3; ++t) tmem_st_frag8(dst + t * 32 + 8 * b, w[t]);
                    }
                }
                tmem_wait_st();
            } else {
                unsigned char *k = stage(it) + L::K0 + 16 * lane;
                const uint32_t k_at = smem_u32(k), kt_at = smb + L::KT + 16 * lane;
                const float *f = gate_f(it) + 64 + (lane >> 3);
                auto piece = [&](int i) { return (uint32_t)((i & 15) * 512 + (i >> 4) * L::QK_STEP); };   // its place in K's panels
                uint4 next = *reinterpret_cast<const uint4 *>(k + piece(first_piece));
#pragma unroll 1
                for (int i = first_piece; i < first_piece + pieces; ++i) {
                    const uint32_t o = piece(i);
                    uint4 u = next;
                    if (i + 1 < first_piece + pieces) next = *reinterpret_cast<const uint4 *>(k + piece(i + 1));
                    const float x = f[4 * (i & 15)];
                    if (4 * (i & 15) + (lane >> 3) >= cnt) u = make_uint4(0u, 0u, 0u, 0u);   // no token's row
                    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                    uint32_t w[3][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 y = mul2(make_float2(lo_bf16(in[e]), hi_bf16(in[e])), make_float2(x, x));
                        w[0][e] = take_bf16(y);
                        w[1][e] = take_bf16(y);
                        w[2][e] = last_bf16(y);
                    }
                    sts128(k_at + o, w[0][0], w[0][1], w[0][2], w[0][3]);
                    sts128(kt_at + 512 * i, w[1][0], w[1][1], w[1][2], w[1][3]);
                    sts128(kt_at + 512 * i + PK * 8192, w[2][0], w[2][1], w[2][2], w[2][3]);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_kt + L::HALVES - 1);
            if (DOT && quarter < 2) {
                if (it > 0) wait(b_o + ((it - 1) & 1), (it - 1) >> 1);   // P of the chunk before is read
                build_p(it, quarter, half);
            }
            if (lane == 0) mbar_arrive(b_gfree + it % L::GATES);
        }
    } else if (warp < kLoadWarp) {
        fewer_regs<kEdgeRegs>();
        // ---------------------------------------------------------------- outputs
        const int ow = warp - kOut0, quarter = ow & 3, half = ow >> 2, et = tid - 32 * kOut0;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16), smb = smem_u32(sm);
        float *dots = reinterpret_cast<float *>(sm + L::DOTS);
#pragma unroll 1
        for (int it = DOT ? 0 : -1; outputs && it < chunks; ++it) {
            if (!DOT && quarter < 2 && it + 1 < chunks) build_p(it + 1, quarter, half);
            if (it < 0) continue;   // (both terms of P of two chunks before are read: its output was waited for)
            const int cnt = count_of(it);
            if (et == 0) bulk_wait_read_all();   // the staging has left
            named_sync(1, 32 * kOutWarps);
            wait(b_gate + it % L::GATES, it / L::GATES);
            if (DOT) {   // Y and P's sums
                wait(b_y + it % 3, it / 3);
                wait(b_p + (it & 1), it >> 1);
            }
            wait(b_o + (it & 1), it >> 1);
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
#pragma unroll 1
                for (int g = 0; g < 2; ++g) {   // 16 channels
                    const uint32_t lanes = (uint32_t)(16 * g) << 16;
                    const int ch = 32 * quarter + 16 * g + 8 * ((lane >> 3) & 1);
                    const uint32_t mat = (ch >> 6) * 8192 + tok * 128 + ((((ch >> 3) ^ tok) & 7) << 4);
                    float r[16], o[16];
                    tmem_ld_frag32(tl + lanes + L::TM_R + 32 * half, r);
                    if (DOT) tmem_ld_frag32(tl + lanes + 64 * ((uint32_t)it % NU) + 32 * half, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {   // 16 tokens: matrices (b, channels), b = 2 e, 2 e + 1
                        uint32_t w[4], y[4];
                        if (DOT)
                            ldsm_x4_trans(smb + L::Y + (uint32_t)(it % 3) * L::Y_STAGE + mat + e * 2048, y);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {   // block b, channels + 8 (i % 2)
                            const int b = 2 * e + (i >> 1), v = 4 * b + 2 * (i & 1);
                            const float2 r2 = make_float2(r[v], r[v + 1]);
                            const float2 x = DOT ? fma2(f[b], r2, make_float2(o[v], o[v + 1])) : mul2(f[b], r2);
                            if (DOT) z[b] = fma2(mul2(f[b], r2), make_float2(lo_bf16(y[i]), hi_bf16(y[i])), z[b]);
                            w[i] = pack_bf16(x.x, x.y);
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
                mbar_arrive(b_oread + (it & 3));
                mbar_arrive(b_gfree + it % L::GATES);
                if (DOT) mbar_arrive(b_yfree + it % 3);
            }
            named_sync(1, 32 * kOutWarps);
            const int64_t base = row_of(it);
            if (cnt == kChunk) {
                if (et == 0) {
                    for (int b = 0; b < PV; ++b) tma_store_3d(&to, sm + L::OUT + b * 8192, 64 * b, h, (int)base);
                    bulk_commit();
                }
            } else {
                for (int i = et; i < cnt * PV * 8; i += 32 * kOutWarps) {
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
    } else {
        fewer_regs<kIssueRegs>();
        if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- loads
            if (elect_one()) {
                const uint32_t bytes = 8192u * (outputs ? 2 * PK + PV : PK + PV);
                int issued = 0;   // chunks whose loads were issued; none after an expiry
#pragma unroll 1
                for (int it = 0; it < chunks; ++it) {
                    const int s = it % kStages;
                    if (it >= kStages) wait(b_free + s, it / kStages - 1);
                    if (*polls == 0) break;
                    unsigned char *st = stage(it);
                    issued = it + 1;
                    const int row = (int)row_of(it);
                    mbar_arrive_expect_tx(b_load + s, bytes);
#pragma unroll 1
                    for (int b = 0; b < PK; ++b) {
                        if (outputs) tma_load_3d(st + L::Q0 + b * L::QK_STEP, &tq, b_load + s, 64 * b, h, row);
                        tma_load_3d(st + L::K0 + b * L::QK_STEP, &tk, b_load + s, 64 * b, h, row);
                    }
#pragma unroll 1
                    for (int b = 0; b < PV; ++b) tma_load_3d(st + L::V0 + b * L::V_STEP, &tv, b_load + s, 64 * b, h, row);
                    if (DOT) {
                        const int y = it % 3;
                        if (it >= 3) wait(b_yfree + y, it / 3 - 1);
                        mbar_arrive_expect_tx(b_y + y, L::Y_STAGE);
#pragma unroll 1
                        for (int b = 0; b < PV; ++b)
                            tma_load_3d(sm + L::Y + y * L::Y_STAGE + b * 8192, &ty, b_y + y, 64 * b, h, row);
                    }
                }
                // the loads have landed before the block ends, also after an expiry
                for (int it = max(0, issued - kStages); it < issued; ++it) wait_cycles(b_load + it % kStages, (it / kStages) & 1);
                for (int it = max(0, issued - 3); DOT && it < issued; ++it) wait_cycles(b_y + it % 3, (it / 3) & 1);
            }
            __syncwarp();
        } else if (warp == kGateWarp) {
            // ---------------------------------------------------------------- gates
            float total = 0.f;
            float x[2];
            auto load_gates = [&](int it) {   // two tokens a lane; backwards the tokens one further on
                const int64_t t = row_of(it) + 2 * lane + (rev ? 1 : 0), end = rev ? hi : row_of(it) + count_of(it);
#pragma unroll
                for (int e = 0; e < 2; ++e) x[e] = p.la && t + e < end ? p.la[(t + e) * H + h] : 0.f;
            };
            if (chunks > 0) load_gates(0);
#pragma unroll 1
            for (int it = 0; it < chunks; ++it) {
                if (it >= L::GATES) wait(b_gfree + it % L::GATES, it / L::GATES - 1);
                // log2 decays as (multiple of 2^-10, remainder): x log2(e) to twice fp32's precision (a
                // NaN stays one, and with it all that the token's decay reaches)
                float2 y[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float v = x[e] < -120.f ? -120.f : x[e], kLog2e = 1.44269504f, kRest = 1.92596299e-8f;
                    const float m = v * kLog2e, r = fmaf(v, kLog2e, -m) + v * kRest, q = rintf(m * 1024.f) * (1.f / 1024.f);
                    y[e] = make_float2(q, (m - q) + r);
                }
                if (it + 1 < chunks) load_gates(it + 1);
                auto add = [](float2 u, float2 v) { return make_float2(u.x + v.x, u.y + v.y); };
                auto sub = [](float2 u, float2 v) { return make_float2(u.x - v.x, u.y - v.y); };
                auto from = [](float2 u, int l) {
                    return make_float2(__shfl_sync(0xffffffffu, u.x, l), __shfl_sync(0xffffffffu, u.y, l));
                };
                float2 c = add(y[0], y[1]);   // inclusive sum over the lanes
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float2 z = make_float2(__shfl_up_sync(0xffffffffu, c.x, o), __shfl_up_sync(0xffffffffu, c.y, o));
                    if (lane >= o) c = add(c, z);
                }
                const float2 ce = from(c, 31);
                total += ce.x + ce.y;
                // c of this lane's two tokens: forwards with, backwards without what was loaded for it
                float2 u[2] = {sub(c, y[1]), c};
                if (rev) {
                    u[1] = u[0];
                    u[0] = sub(u[0], y[0]);
                }
                const float2 mid = from(u[1], 15);
                float2 *g = gate_c(it);
                float *gr = gate_f(it);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = 2 * lane + e;
                    const float2 w = sub(ce, u[e]);
                    const float lh = u[e].x + u[e].y, lt = w.x + w.y;
                    g[t] = u[e];
                    gr[64 + t] = ex2(rev ? lh : lt);
                    if (DOT) {
                        const float2 m = sub(u[e], mid);
                        const float d = rev ? -m.x - m.y : m.x + m.y;
                        gr[t] = ex2(rev ? lt : lh);
                        gr[128 + t] = ex2(d);
                        gr[192 + t] = ex2(-d);
                    } else {
                        const float lr = fmaxf(rev ? lt : lh, -kFactorSpan);
                        gr[t] = ex2(lr);
                        gr[128 + t] = ex2(-lr);
                    }
                }
                if (lane == 0) {
                    g[64] = ce;
                    g[65].x = -ce.x < kFactorSpan ? 1.f : 0.f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(b_gate + it % L::GATES);
            }
            if (a.sums && lane == 0) a.seg_decay[slot * H + h] = total;
        } else {
            // ---------------------------------------------------------------- MMA issue
            const int role = __shfl_sync(0xffffffffu, warp, 0);
            if (chunks > 0 && ((outputs && role == kScoreWarp) || role == kUpdateWarp) && elect_one()) {
                constexpr uint32_t ID_KK = idesc_bf16(128, 64, false, false), ID_MK = idesc_bf16(128, 64, true, false),
                                   ID_MM = idesc_bf16(128, DK, DOT, true);
                const uint64_t dK = smem_desc_sw128(smem_u32(sm), 16, 1024);              // K-major
                const uint64_t dV = smem_desc_sw128(smem_u32(sm), L::V_STEP, 1024);   // MN-major, V panels
                const uint64_t dT0 = smem_desc_sw128(smem_u32(sm), L::QK_STEP, 1024);      // MN-major, Kt's first term
                const uint64_t dT = smem_desc_sw128(smem_u32(sm), 8192, 1024);            // and its others
                auto at_stage = [&](int it) { return (uint32_t)(it % kStages) * L::STAGE; };
                auto u_of = [&](int it) { return tm + 64 * ((uint32_t)it % NU); };
                // K = 16 steps k0 .. k0 + kn - 1 through one panel (K-major: 32 bytes a step; MN-major: 2048)
                auto steps = [&](int k0, int kn, uint32_t d, uint64_t da, uint32_t astep, uint64_t db, uint32_t bstep, uint32_t id,
                                 bool more) {
#pragma unroll
                    for (int ks = 0; ks < kn; ++ks)
                        mma_bf16(d, desc_add(da, (k0 + ks) * astep), desc_add(db, (k0 + ks) * bstep), id, more || ks > 0);
                };
                auto four = [&](uint32_t d, uint64_t da, uint32_t astep, uint64_t db, uint32_t bstep, uint32_t id, bool more) {
                    steps(0, 4, d, da, astep, db, bstep, id, more);
                };
                auto scores = [&](int it) {
                    const uint32_t st = at_stage(it);
#pragma unroll 1
                    for (int b = 0; b < PK; ++b) {
                        const uint32_t o = st + b * L::QK_STEP;
                        four(u_of(it), desc_add(dK, o + L::Q0), 32, desc_add(dK, o + L::K0), 32, ID_KK, b > 0);
                    }
                    mma_commit(b_x + it % NU);
                };
                auto scores2 = [&](int it) {
                    const uint32_t st = at_stage(it);
#pragma unroll 1
                    for (int b = 0; b < PV; ++b) {
                        four(tm + L::TM_X2, desc_add(dK, L::Y + (uint32_t)(it % 3) * L::Y_STAGE + b * 8192), 32,
                             desc_add(dK, st + L::V0 + b * L::V_STEP), 32, ID_KK, b > 0);
                    }
                    mma_commit(b_x2);
                    mma_commit(b_yfree + it % 3);
                };
                auto update = [&](int it, int part) {   // part: of Kt's rows
                    const uint32_t st = at_stage(it);
                    constexpr int KN = 4 / L::HALVES;
#pragma unroll 1
                    for (int t = 2; t >= 0; --t) {
                        if (!DOT) {   // Vt from tensor memory, K as loaded
                            const uint64_t dk = desc_add(dT0, st + L::K0 + part * KN * 2048);
#pragma unroll
                            for (int ks = 0; ks < KN; ++ks)
                                mma_bf16_ts(tm + L::TM_D, tm + L::TM_V + 32 * t + 8 * (part * KN + ks), desc_add(dk, ks * 2048), ID_MM,
                                            part > 0 || t < 2 || ks > 0);
                            continue;
                        }
                        steps(part * KN, KN, tm + L::TM_D, desc_add(dV, st + L::V0), 2048,
                              t == 0 ? desc_add(dT0, st + L::K0) : desc_add(dT, L::KT + (t - 1) * PK * 8192),
                              2048, ID_MM, part > 0 || t < 2);
                    }
                    mma_commit(part + 1 < L::HALVES ? b_d1 : b_d);
                };
                auto read_state = [&](int it) {
                    const uint32_t st = at_stage(it);
                    // small terms first: what the tensor core cuts off a sum goes by the sum's size
#pragma unroll 1
                    for (int b = NS * PK - 1; b >= 0; --b) {
                        const uint64_t dq = desc_add(dK, st + L::Q0 + (PK == 2 ? (b & 1) * L::QK_STEP : 0));
                        const uint32_t s = tm + 32 * b + (DOT && b >= 2 * PK ? L::TM_X2 - 64 * PK : L::TM_S);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_bf16_ts(tm + L::TM_R, s + 8 * ks, desc_add(dq, ks * 32), ID_KK, b < NS * PK - 1 || ks > 0);
                    }
                    mma_commit(b_r);
                };
                auto read_scores = [&](int it) {   // without Y, onto R
#pragma unroll 1
                    for (int t = 1; t >= 0; --t)
                        four(DOT ? u_of(it) : tm + L::TM_R, desc_add(dV, at_stage(it) + L::V0), 2048,
                             desc_add(dK, t == 0 ? L::P + (it & 1) * 8192 : L::PL + (it % L::PLS) * 8192), 32, ID_MK, !DOT || t == 0);
                };
                auto read = [&](int it) {   // R and O of the chunk are read
                    if (it >= 0) wait(b_oread + (it & 3), it >> 2);
                };
                if (role == kScoreWarp) {
                    for (int it = 0; it < chunks; ++it) {
                        if (DOT) read(it - NU);
                        if (!DOT && it > 0) wait(b_p + ((it - 1) & 1), (it - 1) >> 1);   // X is read
                        wait(b_load + it % kStages, it / kStages);
                        scores(it);
                        if (DOT) {
                            // X2, and what R took over its place, are read
                            if (it > 0) wait(b_p + ((it - 1) & 1), (it - 1) >> 1);
                            if (it > 0) wait(b_r, it - 1);
                            wait(b_y + it % 3, it / 3);
                            scores2(it);
                        }
                    }
                } else {
                    // D first: the next chunk's Kt waits for it
#pragma unroll 1
                    for (int it = 0; it < chunks; ++it) {
                        wait(b_load + it % kStages, it / kStages);
                        wait(b_kt, it);
                        if (it > 0) wait(b_dread, it - 1);
                        update(it, 0);
                        if (L::HALVES == 2) {
                            wait(b_kt + 1, it);
                            update(it, 1);
                        }
                        if (outputs) {
                            read(it - 1);
                            wait(b_s, it);   // (with Y behind P)
                            read_state(it);
                            wait(b_p + (it & 1), it >> 1);
                            read_scores(it);
                            mma_commit(b_o + (it & 1));
                        }
                        mma_commit(b_free + it % kStages);
                    }
                }
                mma_commit(b_end);
                wait_cycles(b_end, 0);   // (after an expiry, too)
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && polls_s == 0) atomicExch(a.status, kErrTimeout);
    if (warp == kUpdateWarp) tmem_dealloc(tm, 512);
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
