// attn_tc_fwd.cu -- forward of the window attention on the 5th-generation tensor cores (tcgen05,
// TMEM, TMA) for bf16 rows.  The mathematics: attn.h.
//
// A block takes two tiles of 128 query rows (stages 0 and 1) that share their key tiles; it runs
// through items of that kind (a run of tokens, a key head, up to four of its query heads side by side).
//     S = Q K^T        [128 x 128]   both from shared memory, S in tensor memory
//     O += P V         [128 x d]     P (bf16) from tensor memory, over S's place (d = 64: apart, so that the next S
//                                    does not wait for the product); V as loaded (MN-major)
// The running softmax: with f = scale log2 e and m the row's reference, p = 2^(f s - f m), and
// O and l hold the sums for that m.  m follows the row's maximum only when that is more than 2^kAbove above it
// (P is a floating-point operand: its precision does not depend on m), so O in tensor memory is rescaled
// a few times a row at most.  A row's decisions depend on the row alone.
//
// Warps 0..7 and 8..15 are the stages' softmax and write their outputs, two for each 32 rows with 64 keys a
// thread, which ask one another only whether a maximum rose; warp 16 issues the copies, warps 17 and 18 the
// stages' MMAs: O += P V, then S of the next tile, so that one stage's softmax runs while the tensor cores work for the other.  (One thread for both stages is late: a tile's sixteen products take it 900 cycles to
// issue and their waits 400, which the tensor cores need 1024 for.)
//
// What bounds it (bf16, d = 128): the tensor cores need 2,048 cycles for a key tile of both stages (64 for 16 of a product's depth).  By
// the cycles of a launch and its tiles it takes 3,200 in long items (B1 T65536 H16/4 w4096: 1,540 us, 1.38 PFLOP/s), 3,590 where
// every query sees all before it (B2 T8192 H16: 430 us, 1.28 PFLOP/s), where items are of any length, and 4,110 with a window
// (B8 T4096 H16/4 w1024: 232 us, 1.04 PFLOP/s), where they are nine tiles long and each begins and ends with the tensor cores idle.  Between
// them stands the chain S, softmax, P, O += P V of a stage, which the other stage covers but for its ends: the
// softmax warps issue in about 60 % of the cycles.  Rows of 128 with a thread for half of one, so that a maximum or a sum is one
// exchange of two threads; with 16 lanes a row (fragments as mma.sync has them) fewer exponentials
// wait for tensor memory, but the reductions' shuffles cost more (1,825 against 1,730 us of B1 T65536 w4096 then).
//
// Rows of other sequences: their keys are masked; their values, which enter the product as 0 times
// whatever they hold, are overwritten with zeros in shared memory in a sequence's last tile.
// A parity wait tells a phase from its neighbours only: no barrier completes a second time before everyone who
// waits for it has seen the first.
// Every wait is bounded: on expiry the kernel records DR_ERR_TIMEOUT, runs its remaining steps
// without waiting, drains its copies and MMAs, frees its tensor memory and returns.
#include "attn_tc.cuh"

namespace dr {
namespace attn {
namespace {

constexpr int kStageWarps = 8, kLoadWarp = 2 * kStageWarps, kMmaWarp = kLoadWarp + 1, kThreads = 32 * (kLoadWarp + 4);   // (two MMA warps)
// Registers a thread: launched with 96; the softmax warps take what the others give back.
constexpr int kSoftRegs = 104, kIssueRegs = 56;
static_assert(2 * kStageWarps * kSoftRegs + 4 * kIssueRegs <= kThreads / 32 * 96, "register split");
constexpr float kAbove = 8.f;

struct FwdArgs {
    AttnProblem p;
    int *status;
    int polls;             // of a wait, at most
    int gs, runs;          // log2 of the query heads side by side; runs of them in a key head's group
    int tokens;            // of an item: 256 >> gs
    int64_t items;
    bool falling;          // later items are shorter
};

// What the load warp, which is ahead of them, tells the others of an item.
struct Item {
    int lo, len, q0, h0;   // first row of the sequence, its length (-1: no more items), first token, first query head
    KeyTiles kt;
    TileRanges tr[2];      // of the stages
    int last16, r0;        // rows of the last key tile: in the product, of the sequence
};

template <int D>
struct Layout {
    static constexpr int PANELS = D / 64, TILE = 128 * D * 2, NB = D == 128 ? 5 : 10;   // key and value buffers
    static constexpr uint32_t Q = 0, KV = 2 * TILE, ROWS = KV + NB * TILE, BARS = ROWS + 2 * 128 * 4;
    static constexpr uint32_t TOTAL = BARS + (2 * NB + 16) * 8 + 3 * sizeof(Item);
    // tensor memory: S of both stages, O of both, P of both where there is room for it apart from S
    static constexpr bool APART = D == 64;
    static constexpr uint32_t TM_O = 256, TM_P = 384;
    static_assert(TOTAL + 1024 <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                const FwdArgs a) {
    using L = Layout<D>;
    constexpr int NB = L::NB;
    extern __shared__ unsigned char dsm_raw[];
    unsigned char *sm = align1024(dsm_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_full = bars, *b_free = bars + NB;        // [NB] a key or value tile is there, is done with
    uint64_t *b_q = bars + 2 * NB, *b_qfree = b_q + 2;   // [2] the stage's queries (and the item)
    uint64_t *b_s = b_q + 4, *b_p = b_q + 6, *b_o = b_q + 8;   // [2] S is there; P is; O is complete
    uint64_t *b_sread = b_q + 10, *b_pv = b_q + 12;      // [2] (P apart) S is read; O += P V is done
    uint64_t *b_end = b_q + 14;
    Item *items = reinterpret_cast<Item *>(b_q + 16);    // [3]: a stage may be one behind the other
    __shared__ uint32_t tmem_s;
    __shared__ int polls_s;
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NB; ++i) {
            mbar_init(b_full + i, 1);
            mbar_init(b_free + i, 2);        // both stages
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_q + i, 1);
            mbar_init(b_qfree + i, 1 + kStageWarps);   // the MMAs, and every softmax warp has seen the item
            mbar_init(b_s + i, 1);
            mbar_init(b_p + i, kStageWarps);
            mbar_init(b_o + i, 1);
            mbar_init(b_sread + i, kStageWarps);
            mbar_init(b_pv + i, 1);
        }
        mbar_init(b_end, 2);
        polls_s = a.polls;
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
    volatile int *polls = &polls_s;
    // `k`-th completion of a barrier (k = 0, 1, ..); after an expiry nobody waits any more
    auto wait = [&](uint64_t *bar, int k) {
        if (!mbar_try_wait(bar, k & 1)) tc::wait_longer(bar, k & 1, polls);
        tc_fence_after();
    };
    auto wait_ring = [&](uint64_t *bar, int k) { wait(bar + k % NB, k / NB); };
    const int tt = a.tokens / 2;       // tokens of a stage

    if (warp < kLoadWarp) {
        tc::more_regs<kSoftRegs>();
        // ---------------------------------------------------------------- softmax
        // this thread: a row, half of the keys; the warp with the other half is the pair's other one
        const int st = warp / kStageWarps, quarter = warp & 3, half = warp >> 2 & 1, row = 32 * quarter + lane, col0 = 64 * half;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16), tS = tl + 128 * st, tO = tl + L::TM_O + D * st + half * (D / 2);
        const uint32_t tP = L::APART ? tl + L::TM_P + 64 * st + 32 * half : tS + col0, pair = 1 + 4 * st + quarter;
        float *rows = reinterpret_cast<float *>(sm + L::ROWS) + 128 * st + row;
        // the other thread's x, for both
        auto exchange = [&](float x, auto join) {
            if (half) *rows = x;
            named_sync(pair, 64);
            if (!half) *rows = x = join(x, *rows);
            named_sync(pair, 64);
            return half ? *rows : x;
        };
        const float f = p.scale * kLog2e;
        const float2 f2 = make_float2(f, f);
        int n_tile = 0, n_out = 0, ring = 0;   // tiles and results of this stage so far; copies
#pragma unroll 1
        for (int it = 0;; ++it) {
            wait(b_q + st, it);
            const Item &im = items[it % 3];
            if (im.len < 0 || *polls == 0) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_qfree + st);
            const KeyTiles &kt = im.kt;
            const TileRanges &tr = im.tr[st];
            const int ta = im.q0 + st * tt, i = ta + (row >> a.gs);
            float m = -INFINITY;
            float2 l = make_float2(0.f, 0.f);      // of this thread's keys
            bool first = true;
#pragma unroll 1
            for (int t = 0; t < kt.n; ++t) {
                if (!tr.meets(t)) continue;
                wait(b_s + st, n_tile);
                ++n_tile;
                float s[64];
                // (columns behind the last key hold anything and are masked)
                tmem_ld32(tS + col0, *reinterpret_cast<float(*)[32]>(s));
                tmem_ld32(tS + col0 + 32, *reinterpret_cast<float(*)[32]>(s + 32));
                tmem_wait_ld();
                bool stored = !L::APART || n_tile == 1;      // whether P's place (and O) is free
                if (L::APART) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_sread + st);
                }
                if (!tr.whole(t)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t bits = kt.bits(i, kKeys * t + col0 + 32 * c, p.window, p.sinks);
#pragma unroll
                        for (int x = 0; x < 32; ++x) s[32 * c + x] = bits >> x & 1 ? s[32 * c + x] : -INFINITY;
                    }
                }
                float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int x = 0; x < 64; x += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) t4[e] = max3(t4[e], s[x + 2 * e], s[x + 2 * e + 1]);
                float top = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]);
                // the row's reference follows its maximum
                if (any_of(pair, (top - m) * f > kAbove)) {
                    top = exchange(top, [](float x, float y) { return fmaxf(x, y); });
                    const bool up = (top - m) * f > kAbove;       // (also from -infinity; not where both are)
                    const float turn = up ? ex2((m - top) * f) : 1.f;
                    l = mul2(l, make_float2(turn, turn));
                    m = up ? top : m;
                    if (!first) {       // (P in S's place: S is there, so the products before it are done)
                        if (!stored) wait(b_pv + st, n_tile - 2);
                        stored = true;
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
                            uint32_t w[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * turn);
                            tmem_st16u(tO + 16 * c, w);
                        }
                    }
                }
                first = false;
                if (!stored) wait(b_pv + st, n_tile - 2);
                const float base = m == -INFINITY ? 0.f : -m * f;
                const float2 b2 = make_float2(base, base);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        float2 y = fma2(make_float2(s[32 * c + 2 * x], s[32 * c + 2 * x + 1]), f2, b2);
                        y.x = ex2(y.x);
                        y.y = ex2(y.y);
                        l = add2(l, y);
                        w[x] = pack_bf16(y.x, y.y);
                    }
                    tmem_st16u(tP + 16 * c, w);
                }
                // values of rows behind the sequence's end that the product takes in are zeros
                if (t == kt.n - 1 && im.last16 > im.r0) {
                    const int r0 = im.r0, last16 = im.last16;
                    const int v = ring + 2 * t + 1;
                    wait_ring(b_full, v);
                    const uint32_t V = smem_u32(sm) + L::KV + (v % NB) * L::TILE;
                    const int n = (last16 - r0) * 8;
                    for (int x = tid & 255; x < L::PANELS * n; x += 256) {
                        const int r = r0 + x % n / 8;
                        sts128(V + (x / n) * 16384 + r * 128 + (x % 8) * 16, 0, 0, 0, 0);
                    }
                    fence_proxy_async();
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_p + st);
            }
            ring += 2 * kt.n;
            if (ta < im.len) {
                const float sum = exchange(l.x + l.y, [](float x, float y) { return x + y; }), inv = 1.f / sum;
                if (half == 0 && i < im.len) p.lse[(int64_t)(im.lo + i) * p.Hq + im.h0 + (row & ((1 << a.gs) - 1))] = (m * f + log2f(sum)) * kLn2;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + ((int64_t)(im.lo + ta) * p.Hq + im.h0) * D + half * (D / 2);
                wait(b_o + st, n_out++);
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    float o[32];
                    uint4 u[4];
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                    to_pieces(o, inv, u);
                    put_rows<4>(u, lane, [&](int r) {
                        const int rr = 32 * quarter + r, x = rr >> a.gs;
                        return ta + x < im.len ? out + ((int64_t)x * p.Hq + (rr & ((1 << a.gs) - 1))) * D + 32 * c : nullptr;
                    });
                }
            }
            tc_fence_before();     // (the next item's first P follows)
        }
    } else {
        tc::fewer_regs<kIssueRegs>();
        if (warp == kLoadWarp) {
            // ---------------------------------------------------------------- copies
            int it = 0, ring = 0;
            auto load = [&](int k, const CUtensorMap *map, int hk, int lo, const KeyTiles &kt, int t) {   // by one lane
                const int b = k % NB;
                if (k >= NB) wait(b_free + b, k / NB - 1);
                const int boxes = (kt.count(t) + kBox - 1) / kBox;
                unsigned char *dst = sm + L::KV + b * L::TILE;
                mbar_arrive_expect_tx(b_full + b, boxes * kBox * 128 * L::PANELS);
                for (int e = 0; e < L::PANELS; ++e)
                    for (int x = 0; x < boxes; ++x)
                        tc::tma_load_3d(dst + e * 16384 + x * kBox * 128, map, b_full + b, 64 * e, hk, lo + kt.key(t * kKeys + x * kBox));
            };
#pragma unroll 1
            for (int64_t round = 0; round * gridDim.x < a.items && *polls != 0; ++round) {
                const int64_t k = dealt(round, a.falling);
                if (k >= a.items) continue;
                // long rows of keys first: the last tokens of all sequences, then the ones before them
                const int nh = p.Hk * a.runs;
                const int hr = (int)(k % nh);
                int64_t n, lo;
                int j, len;
                if (p.seqs.cu) {
                    if (!find_tile(p.seqs, a.tokens, (int)(k / nh), n, j, lo, len)) continue;
                } else {
                    const int per = (int)((p.seqs.T + a.tokens - 1) / a.tokens);
                    j = per - 1 - (int)(k / nh / p.seqs.N);
                    n = k / nh % p.seqs.N;
                    lo = n * p.seqs.T;
                    len = (int)p.seqs.T;
                }
                const int hk = hr / a.runs, q0 = j * a.tokens;
                Item im;
                im.lo = (int)lo;
                im.len = len;
                im.q0 = q0;
                im.h0 = hk * (p.Hq / p.Hk) + (hr % a.runs << a.gs);
                const KeyTiles kt(q0, a.tokens, len, p.window, p.sinks);
                im.kt = kt;
                for (int st = 0; st < 2; ++st) im.tr[st] = TileRanges(kt, q0 + st * tt, min(len, q0 + (st + 1) * tt), p.window, p.sinks);
                im.last16 = (kt.count(kt.n - 1) + 15) & ~15;
                im.r0 = kt.behind(kt.n - 1, len);
                if (elect_one()) {
                    for (int st = 0; st < 2; ++st) {
                        if (it > 0) wait(b_qfree + st, it - 1);
                        if (st == 0) items[it % 3] = im;
                        mbar_arrive_expect_tx(b_q + st, L::TILE);
                        for (int e = 0; e < L::PANELS; ++e)
                            tc::tma_load_3d(sm + L::Q + st * L::TILE + e * 16384, &tq, b_q + st, 64 * e, im.h0, im.lo + q0 + st * tt);
                        if (st == 0) load(ring, &tk, hk, im.lo, kt, 0);
                    }
                    for (int t = 0; t < kt.n; ++t) {
                        if (t > 0) load(ring + 2 * t, &tk, hk, im.lo, kt, t);
                        load(ring + 2 * t + 1, &tv, hk, im.lo, kt, t);
                    }
                }
                __syncwarp();
                ring += 2 * kt.n;
                ++it;
            }
            if (elect_one()) {
                // the loads have landed before the block ends, also after an expiry
                for (int k = max(0, ring - NB); k < ring; ++k) tc::wait_cycles(b_full + k % NB, (k / NB) & 1);
                for (int st = 0; st < 2; ++st) {
                    if (it > 0) {
                        wait(b_qfree + st, it - 1);
                        tc::wait_cycles(b_q + st, (it - 1) & 1);
                    }
                    if (st == 0) items[it % 3].len = -1;
                    mbar_arrive(b_q + st);
                }
            }
            __syncwarp();
        } else if (warp < kMmaWarp + 2) {
            // ---------------------------------------------------------------- MMAs of a stage
            const int st = warp - kMmaWarp;
            if (elect_one()) {
                const uint64_t dQ = smem_desc_sw128(smem_u32(sm) + L::Q + st * L::TILE, 16, 1024);   // K-major
                const uint64_t dK = smem_desc_sw128(smem_u32(sm) + L::KV, 16, 1024);
                const uint64_t dV = smem_desc_sw128(smem_u32(sm) + L::KV, 16384, 1024);     // MN-major, panels of 64 channels
                constexpr uint32_t ID_PV = idesc_bf16(128, D, false, true);
                const uint32_t tS = tm + 128 * st, tO = tm + L::TM_O + D * st, tP = L::APART ? tm + L::TM_P + 64 * st : tS;
                int ring = 0, n_p = 0, n_s = 0;
#pragma unroll 1
                for (int it = 0;; ++it) {
                    wait(b_q + st, it);
                    const Item &im = items[it % 3];
                    if (im.len < 0 || *polls == 0) break;
                    const KeyTiles &kt = im.kt;
                    const TileRanges tr = im.tr[st];
                    const int ta = im.q0 + st * tt;
                    int pend = -1;         // the tile whose S went last, if it was the one before
                    bool more = false;
                    auto flush = [&](int t) {     // O += P V of tile t - 1
                        const int v = ring + 2 * t - 1, b = v % NB;
                        wait(b_full + b, v / NB);
                        if (pend >= 0) {
                            const int ks = (kt.count(pend) + 15) / 16;
                            const uint64_t dv = desc_add(dV, b * L::TILE);
                            wait(b_p + st, n_p++);
                            if (ks == 8) {      // (a rolled loop issues a product in 85 cycles, which the tensor core takes in 64)
#pragma unroll
                                for (int k = 0; k < 8; ++k) mma_bf16_ts(tO, tP + 8 * k + (!L::APART && k >= 4 ? 32 : 0), desc_add(dv, k * 2048), ID_PV, more || k > 0);
                            } else {
#pragma unroll 1
                                for (int k = 0; k < ks; ++k) mma_bf16_ts(tO, tP + 8 * k + (!L::APART && k >= 4 ? 32 : 0), desc_add(dv, k * 2048), ID_PV, more || k > 0);
                            }
                            more = true;
                            if (L::APART) mma_commit(b_pv + st);
                        }
                        mma_commit(b_free + b);
                    };
#pragma unroll 1
                    for (int t = 0; t < kt.n; ++t) {
                        const int k = ring + 2 * t, b = k % NB, n16 = (kt.count(t) + 15) & ~15;
                        wait(b_full + b, k / NB);
                        if (!L::APART && t > 0) flush(t);
                        const bool met = tr.meets(t);
                        if (met) {
                            if (L::APART && n_s > 0) wait(b_sread + st, n_s - 1);
                            ++n_s;
                            const uint64_t dk = desc_add(dK, b * L::TILE);
                            const uint32_t id = idesc_bf16(128, 16, false, false) + ((uint32_t)(n16 - 16) << 14);
#pragma unroll
                            for (int e = 0; e < D / 16; ++e)
                                mma_bf16(tS, desc_add(dQ, (e >> 2) * 16384 + (e & 3) * 32), desc_add(dk, (e >> 2) * 16384 + (e & 3) * 32), id, e > 0);
                            mma_commit(b_s + st);
                        }
                        mma_commit(b_free + b);
                        if (L::APART && t > 0) flush(t);
                        pend = met ? t : -1;
                    }
                    mma_commit(b_qfree + st);
                    flush(kt.n);
                    if (ta < im.len) mma_commit(b_o + st);
                    ring += 2 * kt.n;
                }
                mma_commit(b_end);
                tc::wait_cycles(b_end, 0);      // every MMA is done
                if (*polls == 0) atomicExch(a.status, kErrTimeout);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

template <int D>
int launch(const CUtensorMap *m, const FwdArgs &a, cudaStream_t s) {
    constexpr int smem = Layout<D>::TOTAL + 1024;
    if (cudaFuncSetAttribute(attn_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return kErrCuda;
    attn_fwd_kernel<D><<<(unsigned)(a.items < kSms ? a.items : kSms), kThreads, smem, s>>>(m[0], m[1], m[2], a);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace
}  // namespace attn

int launch_attn_tc_fwd(const AttnProblem &p, int *status, cudaStream_t stream) {
    using namespace attn;
    FwdArgs a{};
    a.p = p;
    a.status = status;
    a.gs = heads_in_tile(p.Hq / p.Hk);
    a.runs = p.Hq / p.Hk >> a.gs;
    a.tokens = 256 >> a.gs;
    a.polls = item_polls(p, a.tokens);
    a.items = attn_tile_slots(p.seqs, a.tokens) * p.Hk * a.runs;
    a.falling = !p.seqs.cu && p.window > p.seqs.T / 2;
    CUtensorMap m[3];
    if (!make_map(&m[0], p.q, p.seqs.total, p.Hq, p.d, p.qs, 1 << a.gs, 128 >> a.gs) ||
        !make_map(&m[1], p.k, p.seqs.total, p.Hk, p.d, p.ks, 1, kBox) || !make_map(&m[2], p.v, p.seqs.total, p.Hk, p.d, p.vs, 1, kBox))
        return kErrCuda;
    return p.d == 64 ? launch<64>(m, a, stream) : launch<128>(m, a, stream);
}

}  // namespace dr
