// attn_tc_bwd.cu -- gradients of the window attention on the 5th-generation tensor cores (tcgen05,
// TMEM, TMA) for bf16 rows.  The mathematics: attn.h.
//
// Two kernels, so that no sum depends on the order of blocks (one kernel would add dq up in memory from
// many blocks); scores and do.v are formed in both, seven products a tile instead of five.
//
// dq: an item is 128 query rows (as in the forward); of each of its key tiles
//     S = Q K^T,  dP = dO V^T     [128 x 128]
//     dQ += dS K                  dS (bf16) from tensor memory, over dP's place; K as loaded (MN-major)
// with two places for dP; the next tile's S follows as soon as the softmax warps have S in registers.  Sixteen
// warps form dS, a thread of them 32 keys of a row.  Four more form delta = do.o an item ahead and leave it,
// with lse in log2, in the order of tiles for the second kernel.
//
// dk, dv: a block takes 128 keys of a head and runs over the tiles of 128 query rows that see one of them, all
// heads of the group one after another:
//     S^T = K Q^T,  dP^T = V dO^T
//     dV += P^T dO,  dK += dS^T Q       P^T, dS^T (bf16) from tensor memory over S's, dP's place; dO, Q as loaded
// While the softmax warps form P^T of a tile the tensor cores work at the tile before (dK) and the
// products of V, and the other way round.
// Which keys and queries a block takes, and how tiles that hold sinks are cut: attn_sinks.cuh.
//
// What bounds them (B8 T2048 H16/4 d128 w1024: dq 162 us, dk and dv 171): by the cycles of a launch and its tiles, items' begin and end
// among them, a tile of dq takes 3,420 cycles where the tensor cores need 1,536 and shared memory 1,790 (operands of three
// products, the last one's A from tensor memory, and two copies); a tile of dk, dv 3,410 where both need 2,048.  The rest is the chain from S and dP to dS, half covered by the
// products of the neighbouring tiles, and the items' begin and end.
//
// Rows of other sequences are masked; where they enter a product as 0 times whatever they hold they are
// overwritten with zeros in shared memory.  Waits are bounded as in the forward.
#include "attn_sinks.cuh"
#include "attn_tc.cuh"

namespace dr {
namespace attn {
namespace {

constexpr int kSoftWarps = 16, kLoadWarp = kSoftWarps, kMmaWarp = kLoadWarp + 1, kStatWarp = kLoadWarp + 3;   // (two MMA warps)
constexpr int kStatWarps = 4, kDqThreads = 32 * (kSoftWarps + 8), kDkvThreads = 32 * (kSoftWarps + 4);
// Registers a thread: launched with 80 and 96; the softmax warps take what the others give back.
constexpr int kDqSoftRegs = 96, kDqOtherRegs = 48, kDkvSoftRegs = 104, kDkvOtherRegs = 56;
static_assert(16 * kDqSoftRegs + 8 * kDqOtherRegs <= 24 * 80 && 16 * kDkvSoftRegs + 4 * kDkvOtherRegs <= 20 * 96, "register split");

struct BwdArgs {
    AttnProblem p;
    int *status;
    int polls;                 // of a wait, at most
    int gs, runs, tokens;      // log2 of the query heads side by side, runs of them, tokens of 128 rows
    int64_t items;             // of dq
    bool falling;              // later items are shorter
    float2 *stats;             // [key head and run][row][head of the run] (lse log2 e, delta)
    SinkPlan sinks;
};

struct Item {
    int lo, len, q0, h0, hr;   // first row of the sequence, its length (-1: no more items), first token, first query head, run
    KeyTiles kt;
    TileRanges tr;
    int last16, r0;            // rows of the last key tile: in the product, of the sequence
};

// The k-th item of dq; long rows of keys first.  By whole warps; false for none.
__device__ __forceinline__ bool item_of(const BwdArgs &a, int64_t k, Item &im) {
    const AttnProblem &p = a.p;
    const int nh = p.Hk * a.runs;
    int64_t n, lo;
    int j, len;
    im.hr = (int)(k % nh);
    if (p.seqs.cu) {
        if (!find_tile(p.seqs, a.tokens, (int)(k / nh), n, j, lo, len)) return false;
    } else {
        const int per = (int)((p.seqs.T + a.tokens - 1) / a.tokens);
        j = per - 1 - (int)(k / nh / p.seqs.N);
        n = k / nh % p.seqs.N;
        lo = n * p.seqs.T;
        len = (int)p.seqs.T;
    }
    im.lo = (int)lo;
    im.len = len;
    im.q0 = j * a.tokens;
    im.h0 = im.hr / a.runs * (p.Hq / p.Hk) + (im.hr % a.runs << a.gs);
    return true;
}

// Zeros into the rows r0 .. r1 - 1 of a tile of 128-byte rows in panels of 16 KB, by the softmax warps.
template <int PANELS>
__device__ __forceinline__ void zero_rows(uint32_t tile, int r0, int r1, int t) {
    const int n = (r1 - r0) * 8;
    for (int x = t; x < PANELS * n; x += 32 * kSoftWarps) sts128(tile + (x / n) * 16384 + (r0 + x % n / 8) * 128 + (x % 8) * 16, 0, 0, 0, 0);
    fence_proxy_async();
}

// ------------------------------------------------------------------ dq
template <int D>
struct DqLayout {
    static constexpr int PANELS = D / 64, TILE = 128 * D * 2, NB = D == 128 ? 5 : 10;
    static constexpr uint32_t Q = 0, O = TILE, KV = 2 * TILE, BARS = KV + NB * TILE;
    static constexpr uint32_t TOTAL = BARS + (2 * NB + 14) * 8 + 2 * sizeof(Item);
    static_assert(TOTAL + 1024 <= 227 * 1024, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(kDqThreads, 1)
attn_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const BwdArgs a) {
    using L = DqLayout<D>;
    constexpr int NB = L::NB;
    extern __shared__ unsigned char dsm_raw[];
    unsigned char *sm = align1024(dsm_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_full = bars, *b_free = bars + NB;      // [NB] a key or value tile is there, is done with
    uint64_t *b_q = bars + 2 * NB, *b_qfree = b_q + 1; // the item and its rows are there, are done with
    uint64_t *b_s = b_q + 2, *b_sread = b_q + 3, *b_dp = b_q + 4, *b_ds = b_q + 6, *b_dq = b_q + 8;   // S; S is read; [2] dP; [2] dS; dQ is complete
    uint64_t *b_stat = b_q + 9, *b_sfree = b_q + 11;   // [2] the rows' statistics are there, are read
    uint64_t *b_end = b_q + 13;
    Item *items = reinterpret_cast<Item *>(b_q + 14);  // [2]
    __shared__ uint32_t tmem_s;
    __shared__ int polls_s;
    const AttnProblem &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NB; ++i) {
            mbar_init(b_full + i, 1);
            mbar_init(b_free + i, 2);        // both MMA warps
        }
        mbar_init(b_q, 1);
        mbar_init(b_qfree, 2 + kSoftWarps);       // the MMAs, and every softmax warp has seen the item
        for (int i = 0; i < 2; ++i) {
            mbar_init(b_dp + i, 1);
            mbar_init(b_ds + i, kSoftWarps);     // (a warp may be a tile ahead of another one)
            mbar_init(b_stat + i, kStatWarps);
            mbar_init(b_sfree + i, kSoftWarps);
        }
        mbar_init(b_s, 1);
        mbar_init(b_sread, kSoftWarps);
        mbar_init(b_dq, 1);
        mbar_init(b_end, 2);
        polls_s = a.polls;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_s, 512);
        tmem_relinquish();
    }
    let_next_start();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_s;
    constexpr uint32_t TM_DP = 128, TM_DQ = 384;      // S at 0
    // places of an item's tiles in the ring: K0, V0, V1, K1, V2, K2, .., so that V is a tile ahead
    auto k_at = [](int t) { return t == 0 ? 0 : 2 * t + 1; };
    auto v_at = [](int t) { return t == 0 ? 1 : 2 * t; };
    volatile int *polls = &polls_s;
    auto wait = [&](uint64_t *bar, int k) {
        if (!mbar_try_wait(bar, k & 1)) tc::wait_longer(bar, k & 1, polls);
        tc_fence_after();
    };
    auto wait_ring = [&](uint64_t *bar, int k) { wait(bar + k % NB, k / NB); };

    if (warp < kSoftWarps) {
        tc::more_regs<kDqSoftRegs>();
        // ---------------------------------------------------------------- dS
        const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane, col0 = 32 * group;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        const float f = p.scale * kLog2e;
        int n_tile = 0, ring = 0;
#pragma unroll 1
        for (int it = 0;; ++it) {
            wait(b_q, it);
            const Item &im = items[it & 1];
            if (im.len < 0 || *polls == 0) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(b_qfree);
            const KeyTiles &kt = im.kt;
            const TileRanges &tr = im.tr;
            const int i = im.q0 + (row >> a.gs);
            wait(b_stat + (it & 1), it >> 1);
            const float2 stat = i < im.len ? a.stats[(((int64_t)im.hr * p.seqs.total + im.lo + i) << a.gs) + (row & ((1 << a.gs) - 1))] : make_float2(0.f, 0.f);
            __syncwarp();
            if (lane == 0) mbar_arrive(b_sfree + (it & 1));
            const float2 f2 = make_float2(f, f), l2 = make_float2(-stat.x, -stat.x), d2 = make_float2(-stat.y, -stat.y);
#pragma unroll 1
            for (int t = 0; t < kt.n; ++t, ++n_tile) {
                const bool whole = tr.whole(t);
                const uint32_t tD = tl + TM_DP + 128 * (n_tile & 1) + col0;
                float s[32];
                wait(b_s, n_tile);
                tmem_ld32(tl + col0, s);      // (columns behind the last key hold anything and are masked)
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_sread);
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 y = fma2(make_float2(s[x], s[x + 1]), f2, l2);
                    s[x] = ex2(y.x);
                    s[x + 1] = ex2(y.y);
                }
                if (t == kt.n - 1 && im.last16 > im.r0) zero_rows<L::PANELS>(smem_u32(sm) + L::KV + (ring + k_at(t)) % NB * L::TILE, im.r0, im.last16, tid);
                wait(b_dp + (n_tile & 1), n_tile >> 1);
                float dp[32];
                tmem_ld32(tD, dp);
                tmem_wait_ld();
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 y = mul2(make_float2(s[x], s[x + 1]), add2(make_float2(dp[x], dp[x + 1]), d2));
                    s[x] = y.x;
                    s[x + 1] = y.y;
                }
                if (!whole) {      // (0 times the product of rows of others may be anything)
                    const uint32_t bits = kt.bits(i, kKeys * t + col0, p.window, p.sinks);
#pragma unroll
                    for (int x = 0; x < 32; ++x) s[x] = bits >> x & 1 ? s[x] : 0.f;
                }
#pragma unroll
                for (int x = 0; x < 32; x += 2) w[x / 2] = pack_bf16(s[x], s[x + 1]);
                tmem_st16u(tD, w);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(b_ds + (n_tile & 1));
            }
            ring += 2 * kt.n;
            wait(b_dq, it);
            constexpr int C = D / 4;
            float o[C];
            uint4 u[C / 8];
            tmem_ld_cols(tl + TM_DQ + C * group, o);
            tmem_wait_ld();
            to_pieces(o, p.scale, u);
            put_rows<C / 8>(u, lane, [&](int r) {
                const int rr = 32 * quarter + r, ii = im.q0 + (rr >> a.gs);
                return ii < im.len ? static_cast<__nv_bfloat16 *>(p.dq) + (int64_t)(im.lo + ii) * p.dqs + (im.h0 + (rr & ((1 << a.gs) - 1))) * D + C * group : nullptr;
            });
            tc_fence_before();
        }
    } else if (warp == kLoadWarp) {
        tc::fewer_regs<kDqOtherRegs>();
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
            Item im;
            if (dealt(round, a.falling) >= a.items || !item_of(a, dealt(round, a.falling), im)) continue;
            const int hk = im.hr / a.runs;
            const KeyTiles kt(im.q0, a.tokens, im.len, p.window, p.sinks);
            im.kt = kt;
            im.tr = TileRanges(kt, im.q0, kt.end, p.window, p.sinks);
            im.last16 = (kt.count(kt.n - 1) + 15) & ~15;
            im.r0 = kt.behind(kt.n - 1, im.len);
            if (elect_one()) {
                if (it > 0) wait(b_qfree, it - 1);
                items[it & 1] = im;
                mbar_arrive_expect_tx(b_q, 2 * L::TILE);
                for (int e = 0; e < L::PANELS; ++e) {
                    tc::tma_load_3d(sm + L::Q + e * 16384, &tq, b_q, 64 * e, im.h0, im.lo + im.q0);
                    tc::tma_load_3d(sm + L::O + e * 16384, &to, b_q, 64 * e, im.h0, im.lo + im.q0);
                }
                auto tile = [&](bool key, int t) {
                    load(ring + (key ? k_at(t) : v_at(t)), key ? &tk : &tv, hk, im.lo, kt, t);
                };
                tile(true, 0);
                tile(false, 0);
                for (int t = 1; t < kt.n; ++t) {
                    tile(false, t);
                    tile(true, t);
                }
            }
            __syncwarp();
            ring += 2 * kt.n;
            ++it;
        }
        if (elect_one()) {
            // the loads have landed before the block ends, also after an expiry
            for (int k = max(0, ring - NB); k < ring; ++k) tc::wait_cycles(b_full + k % NB, (k / NB) & 1);
            if (it > 0) {
                wait(b_qfree, it - 1);
                tc::wait_cycles(b_q, (it - 1) & 1);
            }
            items[it & 1].len = -1;
            mbar_arrive(b_q);
        }
        __syncwarp();
    } else if (warp < kMmaWarp + 2) {
        tc::fewer_regs<kDqOtherRegs>();
        // ---------------------------------------------------------------- MMAs: S; dP and dQ
        const bool first = warp == kMmaWarp;
        if (elect_one()) {
            const uint64_t dA = smem_desc_sw128(smem_u32(sm) + (first ? L::Q : L::O), 16, 1024);        // K-major
            const uint64_t dK = smem_desc_sw128(smem_u32(sm) + L::KV, 16, 1024);
            const uint64_t dM = smem_desc_sw128(smem_u32(sm) + L::KV, 16384, 1024);     // MN-major, panels of 64 channels
            constexpr uint32_t ID_DQ = idesc_bf16(128, D, false, true);
            int ring = 0, n_tile = 0;
#pragma unroll 1
            for (int it = 0;; ++it) {
                wait(b_q, it);
                const Item &im = items[it & 1];
                if (im.len < 0 || *polls == 0) break;
                const KeyTiles &kt = im.kt;
                auto n16 = [&](int t) { return (kt.count(t) + 15) & ~15; };
                auto rows_by_rows = [&](uint32_t d, int b, int t) {
                    const uint64_t db = desc_add(dK, b * L::TILE);
                    const uint32_t id = idesc_bf16(128, 16, false, false) + ((uint32_t)(n16(t) - 16) << 14);
#pragma unroll
                    for (int e = 0; e < D / 16; ++e)
                        mma_bf16(d, desc_add(dA, (e >> 2) * 16384 + (e & 3) * 32), desc_add(db, (e >> 2) * 16384 + (e & 3) * 32), id, e > 0);
                };
                if (first) {
#pragma unroll 1
                    for (int t = 0; t < kt.n; ++t) {
                        const int k = ring + k_at(t), b = k % NB;
                        wait(b_full + b, k / NB);
                        if (n_tile + t > 0) wait(b_sread, n_tile + t - 1);
                        rows_by_rows(tm, b, t);
                        mma_commit(b_s);
                        mma_commit(b_free + b);
                    }
                    mma_commit(b_qfree);
                } else {
                    auto dps = [&](int t) {
                        const int g = n_tile + t, v = ring + v_at(t), b = v % NB;
                        wait(b_full + b, v / NB);
                        rows_by_rows(tm + TM_DP + 128 * (g & 1), b, t);
                        mma_commit(b_dp + (g & 1));
                        mma_commit(b_free + b);
                        mma_commit(b_free + b);      // (the other warp does not read it)
                        if (t + 1 == kt.n) mma_commit(b_qfree);
                    };
                    dps(0);
                    if (kt.n > 1) dps(1);
#pragma unroll 1
                    for (int t = 0; t < kt.n; ++t) {
                        const int k = ring + k_at(t), b = k % NB, ks = n16(t) / 16;
                        const uint64_t db = desc_add(dM, b * L::TILE);
                        const uint32_t src = tm + TM_DP + 128 * ((n_tile + t) & 1);
                        wait(b_full + b, k / NB);
                        wait(b_ds + ((n_tile + t) & 1), (n_tile + t) >> 1);
                        if (ks == 8) {      // (a rolled loop issues a product in 85 cycles, which the tensor core takes in 64)
#pragma unroll
                            for (int e = 0; e < 8; ++e) mma_bf16_ts(tm + TM_DQ, src + 32 * (e >> 1) + 8 * (e & 1), desc_add(db, e * 2048), ID_DQ, t > 0 || e > 0);
                        } else {
#pragma unroll 1
                            for (int e = 0; e < ks; ++e)
                                mma_bf16_ts(tm + TM_DQ, src + 32 * (e >> 1) + 8 * (e & 1), desc_add(db, e * 2048), ID_DQ, t > 0 || e > 0);
                        }
                        mma_commit(b_free + b);
                        if (t + 2 < kt.n) dps(t + 2);
                    }
                    mma_commit(b_dq);
                }
                ring += 2 * kt.n;
                n_tile += kt.n;
            }
            mma_commit(b_end);
            tc::wait_cycles(b_end, 0);      // every MMA is done
            if (*polls == 0) atomicExch(a.status, kErrTimeout);
        }
        __syncwarp();
    } else if (warp >= kStatWarp + kStatWarps) {
        tc::fewer_regs<kDqOtherRegs>();
    } else {
        tc::fewer_regs<kDqOtherRegs>();
        // ---------------------------------------------------------------- lse and delta of the rows
        constexpr int LPR = D / 8, RPW = 32 / LPR, U = 4, ROWS = 128 / kStatWarps;      // lanes a row, rows a warp's access, rows a warp
        const int l = lane % LPR;
        int it = 0;
#pragma unroll 1
        for (int64_t round = 0; round * gridDim.x < a.items && *polls != 0; ++round) {
            Item im;
            if (dealt(round, a.falling) >= a.items || !item_of(a, dealt(round, a.falling), im)) continue;
            if (it > 1) wait(b_sfree + (it & 1), (it >> 1) - 1);
#pragma unroll 1
            for (int r0 = ROWS * (warp - kStatWarp); r0 < ROWS * (warp - kStatWarp + 1); r0 += U * RPW) {
                uint4 o[U], d[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * RPW + lane / LPR, i = im.q0 + (r >> a.gs);
                    o[u] = d[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (i < im.len) {
                        const int64_t at = ((int64_t)(im.lo + i) * p.Hq + im.h0 + (r & ((1 << a.gs) - 1))) * D + 8 * l;
                        o[u] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.out) + at);
                        d[u] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.d_out) + at);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * RPW + lane / LPR, i = im.q0 + (r >> a.gs);
                    const uint32_t x[4] = {o[u].x, o[u].y, o[u].z, o[u].w}, y[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum = fmaf(__uint_as_float(x[e] << 16), __uint_as_float(y[e] << 16), sum);
                        sum = fmaf(__uint_as_float(x[e] & 0xffff0000u), __uint_as_float(y[e] & 0xffff0000u), sum);
                    }
#pragma unroll
                    for (int w = 1; w < LPR; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
                    if (l == 0 && i < im.len)
                        a.stats[(((int64_t)im.hr * p.seqs.total + im.lo + i) << a.gs) + (r & ((1 << a.gs) - 1))] =
                            make_float2(p.lse[(int64_t)(im.lo + i) * p.Hq + im.h0 + (r & ((1 << a.gs) - 1))] * kLog2e, sum);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_stat + (it & 1));
            ++it;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

// ------------------------------------------------------------------ dk, dv
template <int D>
struct DkvLayout {
    // query-side tiles (two in use, two on their way, one to spare), statistics
    static constexpr int PANELS = D / 64, TILE = 128 * D * 2, NB = D == 128 ? 5 : 10, NS = 2;
    static constexpr uint32_t K = 0, V = TILE, QO = 2 * TILE, STATS = QO + NB * TILE, BARS = STATS + NS * 128 * 8;
    static constexpr uint32_t TOTAL = BARS + (2 * NB + 2 * NS + 6) * 8 + 8;
    static_assert(TOTAL <= 227 * 1024, "shared memory");       // (no room for aligning: the array is declared aligned)
};

template <int D>
__global__ void __launch_bounds__(kDkvThreads, 1)
attn_dkv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap to, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const BwdArgs a) {
    using L = DkvLayout<D>;
    constexpr int NB = L::NB, NS = L::NS;
    const AttnProblem &p = a.p;
    KeyBlock kb;
    if (!kb.find(p, a.sinks, blockIdx.x)) {
        wait_for_last();
        return;
    }
    const int64_t lo = kb.lo;
    const int len = kb.len, hk = kb.hk, k0 = kb.k0, qa = kb.qa, qb = kb.qb;
    const int nt = (qb - qa + a.tokens - 1) / a.tokens, tiles = nt * a.runs;

    extern __shared__ __align__(1024) unsigned char sm[];
    if (smem_u32(sm) & 1023u) {      // (never seen: nothing static lies in front of it)
        if (threadIdx.x == 0) atomicExch(a.status, kErrCuda);
        return;
    }
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS);
    uint64_t *b_full = bars, *b_free = bars + NB;      // [NB] a query or d_out tile is there, is done with
    uint64_t *b_stat = bars + 2 * NB, *b_sfree = b_stat + NS;   // [NS] the tile's statistics
    uint64_t *b_kv = b_sfree + NS, *b_s = b_kv + 1, *b_p = b_kv + 2, *b_dp = b_kv + 3, *b_ds = b_kv + 4, *b_end = b_kv + 5;
    float *stats = reinterpret_cast<float *>(sm + L::STATS);   // [NS][-lse log2 e, -delta][128]
    uint32_t &tmem_s = *reinterpret_cast<uint32_t *>(b_end + 1);
    int &polls_s = *reinterpret_cast<int *>(&tmem_s + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NB; ++i) {
            mbar_init(b_full + i, 1);
            mbar_init(b_free + i, 2);        // both MMA warps
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(b_stat + i, 1);
            mbar_init(b_sfree + i, kSoftWarps);
        }
        mbar_init(b_kv, 1);
        mbar_init(b_s, 1);
        mbar_init(b_p, kSoftWarps);
        mbar_init(b_dp, 1);
        mbar_init(b_ds, kSoftWarps);
        mbar_init(b_end, 2);
        polls_s = a.polls;
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_s, 512);
        tmem_relinquish();
    }
    let_next_start();
    wait_for_last();       // its statistics, and the workspace of a call before it
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_s;
    constexpr uint32_t TM_DP = 128, TM_DV = 256, TM_DK = 384;
    volatile int *polls = &polls_s;
    auto wait = [&](uint64_t *bar, int k) {
        if (!mbar_try_wait(bar, k & 1)) tc::wait_longer(bar, k & 1, polls);
        tc_fence_after();
    };
    auto wait_ring = [&](uint64_t *bar, int k) { wait(bar + k % NB, k / NB); };

    if (warp < kSoftWarps) {
        tc::more_regs<kDkvSoftRegs>();
        // ---------------------------------------------------------------- P^T, dS^T
        const int quarter = warp & 3, group = warp >> 2, j = k0 + 32 * quarter + lane, col0 = 32 * group;
        const uint32_t tl = tm + ((uint32_t)(32 * quarter) << 16);
        const float f = p.scale * kLog2e;
        const float2 f2 = make_float2(f, f);
        const int see = min(qb, j < p.sinks ? len : min(j, kNoWindow - 1) + p.window);    // behind the last query that sees this key
        int q0 = qa;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const bool whole = q0 >= k0 + kKeys - 1 && q0 + a.tokens <= qb && (q0 + a.tokens - 1 - k0 < p.window || k0 + kKeys <= p.sinks);
            const float4 *st = reinterpret_cast<const float4 *>(stats + (t % NS) * 256 + col0);
            float s[32];
            uint32_t w[16], bits = 0xffffffffu;
            if (!whole) bits = low_bits(min(see - q0, 128) * (1 << a.gs) - col0) & ~low_bits((min(max(j - q0, 0), 128) << a.gs) - col0);
            wait(b_stat + t % NS, t / NS);
            wait(b_s, t);
            tmem_ld32(tl + col0, s);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                const float4 l = st[x / 4];
                const float2 y = fma2(make_float2(s[x], s[x + 1]), f2, make_float2(l.x, l.y)), z = fma2(make_float2(s[x + 2], s[x + 3]), f2, make_float2(l.z, l.w));
                s[x] = ex2(y.x);
                s[x + 1] = ex2(y.y);
                s[x + 2] = ex2(z.x);
                s[x + 3] = ex2(z.y);
            }
            if (!whole) {
#pragma unroll
                for (int x = 0; x < 32; ++x) s[x] = bits >> x & 1 ? s[x] : 0.f;
            }
#pragma unroll
            for (int x = 0; x < 32; x += 2) w[x / 2] = pack_bf16(s[x], s[x + 1]);
            tmem_st16u(tl + col0, w);
            if (q0 + a.tokens > len) {     // rows of no query of this sequence are zeros
                wait_ring(b_full, 2 * t + 1);
                for (int e = 0; e < 2; ++e)
                    zero_rows<L::PANELS>(smem_u32(sm) + L::QO + ((2 * t + e) % NB) * L::TILE, (len - q0) << a.gs, 128, tid);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(b_p);
            wait(b_dp, t);
            float dp[32];
            tmem_ld32(tl + TM_DP + col0, dp);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                const float4 d = st[32 + x / 4];
                float2 y = mul2(make_float2(s[x], s[x + 1]), add2(make_float2(dp[x], dp[x + 1]), make_float2(d.x, d.y)));
                float2 z = mul2(make_float2(s[x + 2], s[x + 3]), add2(make_float2(dp[x + 2], dp[x + 3]), make_float2(d.z, d.w)));
                if (!whole) {      // (0 times the product of rows of others may be anything)
                    y.x = bits >> x & 1 ? y.x : 0.f;
                    y.y = bits >> x & 2 ? y.y : 0.f;
                    z.x = bits >> x & 4 ? z.x : 0.f;
                    z.y = bits >> x & 8 ? z.y : 0.f;
                }
                w[x / 2] = pack_bf16(y.x, y.y);
                w[x / 2 + 1] = pack_bf16(z.x, z.y);
            }
            tmem_st16u(tl + TM_DP + col0, w);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(b_ds);
                mbar_arrive(b_sfree + t % NS);
            }
            q0 += a.tokens;
            if (q0 >= qb) q0 = qa;         // the next heads
        }
        wait(b_end, 0);
        // out: a sink's row is a part of a sum where its queries are cut
        constexpr int C = D / 4;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {      // dk, dv
            const float scale = e == 0 ? p.scale : 1.f;
            float o[C];
            tmem_ld_cols(tl + (e == 0 ? TM_DK : TM_DV) + C * group, o);
            tmem_wait_ld();
            if (kb.cut && j < min(p.sinks, len)) {
                float *sum = kb.sum(p, a.sinks, j) + e * D + C * group;
#pragma unroll
                for (int x = 0; x < C; x += 4) store4(sum + x, make_float4(o[x] * scale, o[x + 1] * scale, o[x + 2] * scale, o[x + 3] * scale));
            }
            if (kb.chunk >= 0) continue;
            uint4 u[C / 8];
            to_pieces(o, scale, u);
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(e == 0 ? p.dk : p.dv) + hk * D + C * group;
            const int64_t stride = e == 0 ? p.dks : p.dvs;
            put_rows<C / 8>(u, lane, [&](int r) {
                const int jj = k0 + 32 * quarter + r;
                return jj < len && !(kb.cut && jj < p.sinks) ? out + (lo + jj) * stride : nullptr;
            });
        }
    } else if (warp == kLoadWarp) {
        tc::fewer_regs<kDkvOtherRegs>();
        // ---------------------------------------------------------------- copies
        if (elect_one()) {
            mbar_arrive_expect_tx(b_kv, 2 * L::TILE);
            for (int e = 0; e < L::PANELS; ++e)
                for (int x = 0; x < kKeys / kBox; ++x) {
                    tc::tma_load_3d(sm + L::K + e * 16384 + x * kBox * 128, &tk, b_kv, 64 * e, hk, (int)lo + k0 + x * kBox);
                    tc::tma_load_3d(sm + L::V + e * 16384 + x * kBox * 128, &tv, b_kv, 64 * e, hk, (int)lo + k0 + x * kBox);
                }
            int issued = 0, q0 = qa, h0 = hk * (p.Hq / p.Hk);
#pragma unroll 1
            for (; issued < 2 * tiles; ++issued) {
                const int b = issued % NB;
                if (issued >= NB) wait(b_free + b, issued / NB - 1);
                if (*polls == 0) break;
                mbar_arrive_expect_tx(b_full + b, L::TILE);
                for (int e = 0; e < L::PANELS; ++e)
                    tc::tma_load_3d(sm + L::QO + b * L::TILE + e * 16384, issued & 1 ? &to : &tq, b_full + b, 64 * e, h0, (int)lo + q0);
                if (issued & 1) {
                    q0 += a.tokens;
                    if (q0 >= qb) {
                        q0 = qa;
                        h0 += 1 << a.gs;
                    }
                }
            }
            // the loads have landed before the block ends, also after an expiry
            tc::wait_cycles(b_kv, 0);
            for (int k = max(0, issued - NB); k < issued; ++k) tc::wait_cycles(b_full + k % NB, (k / NB) & 1);
        }
        __syncwarp();
    } else if (warp < kMmaWarp + 2) {
        tc::fewer_regs<kDkvOtherRegs>();
        // ---------------------------------------------------------------- MMAs: S and dV; dP and dK
        const int second = warp - kMmaWarp;      // S^T = K Q^T, dV += P^T dO; dP^T = V dO^T, dK += dS^T Q
        if (elect_one()) {
            const uint64_t dA = smem_desc_sw128(smem_u32(sm) + (second ? L::V : L::K), 16, 1024);        // K-major
            const uint64_t dB = smem_desc_sw128(smem_u32(sm) + L::QO, 16, 1024);
            const uint64_t dM = smem_desc_sw128(smem_u32(sm) + L::QO, 16384, 1024);     // MN-major, panels of 64 channels
            constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false), ID_D = idesc_bf16(128, D, false, true);
            const uint32_t x = tm + (second ? TM_DP : 0), sum = tm + (second ? TM_DK : TM_DV);
            uint64_t *b_made = second ? b_dp : b_s, *b_read = second ? b_ds : b_p;
            auto product = [&](int k) {
                const int b = k % NB;
                const uint64_t db = desc_add(dB, b * L::TILE);
                wait(b_full + b, k / NB);
#pragma unroll
                for (int e = 0; e < D / 16; ++e)
                    mma_bf16(x, desc_add(dA, (e >> 2) * 16384 + (e & 3) * 32), desc_add(db, (e >> 2) * 16384 + (e & 3) * 32), ID_S, e > 0);
                mma_commit(b_made);
                mma_commit(b_free + b);
            };
            wait(b_kv, 0);
            product(second);
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
                const int k = 2 * t + 1 - second, b = k % NB;
                const uint64_t db = desc_add(dM, b * L::TILE);
                wait(b_full + b, k / NB);
                wait(b_read, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) mma_bf16_ts(sum, x + 32 * (e >> 1) + 8 * (e & 1), desc_add(db, e * 2048), ID_D, t > 0 || e > 0);
                mma_commit(b_free + b);
                if (t + 1 < tiles) product(2 * t + 2 + second);
            }
            mma_commit(b_end);
            tc::wait_cycles(b_end, 0);      // every MMA is done
            if (*polls == 0) atomicExch(a.status, kErrTimeout);
        }
        __syncwarp();
    } else if (warp == kStatWarp) {
        tc::fewer_regs<kDkvOtherRegs>();
        // ---------------------------------------------------------------- statistics of the queries
        int q0 = qa;
        const float2 *src = a.stats + (((int64_t)hk * a.runs * p.seqs.total + lo) << a.gs);
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int rows = min(len - q0, a.tokens) << a.gs;
            float2 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = lane + 32 * e < rows ? src[((int64_t)q0 << a.gs) + lane + 32 * e] : make_float2(0.f, 0.f);
            if (t >= NS) wait(b_sfree + t % NS, t / NS - 1);
            float *dst = stats + (t % NS) * 256 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dst[32 * e] = -x[e].x;
                dst[128 + 32 * e] = -x[e].y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(b_stat + t % NS);
            q0 += a.tokens;
            if (q0 >= qb) {
                q0 = qa;
                src += p.seqs.total << a.gs;
            }
        }
    } else {
        tc::fewer_regs<kDkvOtherRegs>();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tm, 512);
}

// Where the workspace's parts lie.
size_t plan(const AttnProblem &p, BwdArgs &a, char *ws) {
    a.p = p;
    a.gs = heads_in_tile(p.Hq / p.Hk);
    a.runs = p.Hq / p.Hk >> a.gs;
    a.tokens = 128 >> a.gs;
    a.polls = item_polls(p, a.tokens);
    a.stats = (float2 *)ws;
    const size_t stats = round256(sizeof(float2) * (size_t)(p.seqs.total * p.Hq));
    return stats + plan_sinks(p, kKeys, 1024, ws + stats, a.sinks);
}

template <int D>
int launch(const AttnProblem &p, BwdArgs a, cudaStream_t s) {
    CUtensorMap m[4];
    if (!make_map(&m[0], p.q, p.seqs.total, p.Hq, p.d, p.qs, 1 << a.gs, 128 >> a.gs) ||
        !make_map(&m[1], p.d_out, p.seqs.total, p.Hq, p.d, (int64_t)p.Hq * p.d, 1 << a.gs, 128 >> a.gs) ||
        !make_map(&m[2], p.k, p.seqs.total, p.Hk, p.d, p.ks, 1, kBox) || !make_map(&m[3], p.v, p.seqs.total, p.Hk, p.d, p.vs, 1, kBox))
        return kErrCuda;
    constexpr int smem_q = DqLayout<D>::TOTAL + 1024, smem_kv = DkvLayout<D>::TOTAL;
    if (cudaFuncSetAttribute(attn_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_q) != cudaSuccess ||
        cudaFuncSetAttribute(attn_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_kv) != cudaSuccess)
        return kErrCuda;
    a.items = attn_tile_slots(p.seqs, a.tokens) * p.Hk * a.runs;
    a.falling = !p.seqs.cu && p.window > p.seqs.T / 2;
    attn_dq_kernel<D><<<(unsigned)(a.items < kSms ? a.items : kSms), kDqThreads, smem_q, s>>>(m[0], m[1], m[2], m[3], a);
    if (cudaGetLastError() != cudaSuccess) return kErrCuda;
    const int64_t blocks = key_blocks(p, a.sinks);
    const int rc = launch_after(attn_dkv_kernel<D>, (unsigned)blocks, kDkvThreads, smem_kv, s, m[0], m[1], m[2], m[3], a);
    return rc != kOk ? rc : launch_sink_sum<D, __nv_bfloat16>(p, a.sinks, s);
}

}  // namespace
}  // namespace attn

size_t attn_tc_bwd_workspace_bytes(const AttnProblem &p) {
    attn::BwdArgs a{};
    return attn::plan(p, a, nullptr);
}

int launch_attn_tc_bwd(const AttnProblem &p, void *workspace, int *status, cudaStream_t stream) {
    attn::BwdArgs a{};
    attn::plan(p, a, (char *)workspace);
    a.status = status;
    return p.d == 64 ? attn::launch<64>(p, a, stream) : attn::launch<128>(p, a, stream);
}

}  // namespace dr
