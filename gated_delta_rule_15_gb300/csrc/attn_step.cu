// attn_step.cu -- window attention of one new token for each sequence over a paged cache.  The
// mathematics: attn.h (the query is the sequence's last token).
//
// Every visible key and value is read once: HBM bandwidth bounds it.  The visible tokens of a unit (a
// sequence, a key head and up to 16 of the query heads that share it) are cut into groups of 16 (fp32: 8), which never
// cross a page: first the groups that hold sinks, then those of the window.  The units' groups, one
// after another, are dealt out evenly: block c takes the groups c * per .. (c + 1) * per - 1, whatever
// units they belong to, so that one long context fills the GPU as a batch does.  A unit that ends up
// in several blocks leaves a partial result (maximum, sum, sum of values) in each, which a second kernel joins
// in a fixed order.
//
// Inside a block the warps take every eighth group, each with copies of its own: a tensor-map box of
// a group's keys, one of its values, into a ring of kStages stages, so 192 KB are under way on an SM, and no
// warp waits for another one but at a unit's end, where their states are added up.
//   bf16: S = Q K^T and O += P V as 16 x 8 x 16 tensor-core products of one warp (the query heads are the
//   16 rows); P enters as two bf16 terms (2^-17 of a value is lost), which costs a memory-bound kernel
//   nothing.
//   fp32: dot products by lane = token, sums by lane = channel, in fp32.
// A table entry outside 0 .. n_pages - 1 makes its page's tokens invisible; their boxes are read
// from behind the tensor's end, where the copy fills in zeros.  Values of tokens that are not
// visible are taken as zero in a group that has some, so what an unused slot of a page holds never matters.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "../../include/dr.h"
#include "attn.h"
#include "common.cuh"
#include "tc_common.cuh"
#include "tc_issue.cuh"

namespace dr {

PFN_cuTensorMapEncodeTiled_v12000 tc_tensor_map_encoder();

namespace {

using namespace umma;

constexpr int kWarps = 8, kStages = 3, kThreads = 32 * kWarps, kHeads = 16, kBlocks = 152;
template <bool BF> constexpr int group_tokens() { return BF ? 16 : 8; }   // 8 KB of keys and values at d = 128
constexpr int kLeast = kWarps;       // groups of a block, at least: one a warp

// What a block leaves for the joining kernel: per row the maximum (log2) and the sum, then the values' sums.
constexpr int kPartialFloats = kHeads * (128 + 2);
struct Tail {                        // the unit that a block began and did not end
    int64_t b;                       // -1: none
    int hu, last;                    // unit of the sequence, last block that has a part of it
};

struct StepArgs {
    AttnStep p;
    int hus, per_h;                  // units a sequence, units a key head
    float *partial;                  // [block][head or tail part]
    Tail *tail;                      // [block]
    int *status;
};

// Visible groups of a sequence of `len` tokens: those of the sinks, `skip` others, those of the window.
template <int G>
struct Seen {
    int len, end, near0, sinks, ns, near_g, n;   // tokens; those of the table; the window's first; groups
    __device__ __forceinline__ Seen(const AttnStep &p, int64_t l) {
        const int64_t room = (int64_t)p.max_pages * p.page;
        const int64_t most = (int64_t)kNoWindow;
        len = (int)(l < 0 ? 0 : l < most ? l : most);
        end = (int)(len < room ? len : room);
        near0 = max(0, len - p.window);
        sinks = min(p.sinks, near0);
        ns = (min(sinks, end) + G - 1) / G;
        near_g = max(near0 / G, ns);
        n = ns + max(0, (end + G - 1) / G - near_g);
    }
    __device__ __forceinline__ int group(int g) const { return g < ns ? g : near_g + (g - ns); }
    __device__ __forceinline__ bool sees(int j) const { return j < end && (j >= near0 || j < sinks); }
    __device__ __forceinline__ bool whole(int j0) const {   // all 16 tokens from j0 on
        return j0 + G <= end && (j0 >= near0 || j0 + G <= sinks);
    }
};

// A place in the row of all units' groups.
template <int G>
struct Cursor {
    int64_t b, first;                // sequence; where its current unit begins
    int hu, n;                       // unit of the sequence; groups of the unit
    __device__ __forceinline__ void seek(const StepArgs &a, int64_t at) {   // forwards, to the unit that holds group `at`
        while (at >= first + n) {
            first += n;
            if (++hu == a.hus) {
                hu = 0;
                ++b;
                n = b < a.p.B ? Seen<G>(a.p, a.p.lens[b]).n : 0x7fffffff;
            }
        }
    }
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// One warp's running result for its unit: 16 rows (query heads).
template <int D, bool BF>
struct State;

// bf16: accumulator fragments; this lane has rows lane / 4 and + 8, columns 8 i + 2 (lane % 4), + 1
template <int D>
struct State<D, true> {
    static constexpr int KSTEPS = D / 16;
    uint32_t q[KSTEPS][4];
    float o[D / 8][4], m[2], l[2];
    __device__ __forceinline__ void begin(const StepArgs &a, const Cursor<16> &u, int lane) {
        const int g = a.p.Hq / a.p.Hk, hk = u.hu / a.per_h, h0 = (u.hu % a.per_h) * kHeads;
        const __nv_bfloat16 *src = (const __nv_bfloat16 *)a.p.q + (u.b * a.p.Hq + hk * g + h0) * D + 2 * (lane & 3);
        const int r = lane >> 2;
#pragma unroll
        for (int s = 0; s < KSTEPS; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = r + 8 * (e & 1);
                q[s][e] = h0 + row < g ? *reinterpret_cast<const uint32_t *>(src + row * D + 16 * s + 8 * (e >> 1)) : 0u;
            }
        reset();
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void group(const StepArgs &a, const Seen<16> &seen, int j0, const unsigned char *stage, int lane, const float *) {
        const uint32_t K = smem_u32(stage), V = K + D * 32;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int mat = lane >> 3, row = lane & 7;
        {   // matrices: tokens 8 (mat / 2), channels + 8 (mat % 2)
            const uint32_t at = K + (8 * (mat >> 1) + row) * 128;
#pragma unroll
            for (int ks = 0; ks < KSTEPS; ++ks) {
                uint32_t b[4];
                ldsm_x4(at + (ks >> 2) * 2048 + ((((2 * ks + (mat & 1)) ^ row) & 7) << 4), b);
                tc::mma_bf16_16x8x16(s[0], q[ks], b[0], b[1]);
                tc::mma_bf16_16x8x16(s[1], q[ks], b[2], b[3]);
            }
        }
        const float f = a.p.scale * kLog2e;
        const int t0 = j0 + 2 * (lane & 3);
        const bool whole = seen.whole(j0);
        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};   // of the value pairs of tokens t0, + 8
        if (!whole) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                keep[t] = 0u;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool in = seen.sees(t0 + 8 * t + e);
                    if (in) keep[t] |= e ? 0xffff0000u : 0xffffu;
                    else s[t][e] = s[t][2 + e] = -INFINITY;
                }
            }
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])) * f;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            top = fmaxf(top, m[r]);
            const float base = top == -INFINITY ? 0.f : top;
            if (__any_sync(0xffffffffu, top > m[r])) {   // somebody's maximum rose
                const float turn = tc::ex2(m[r] - base);
                l[r] *= turn;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][2 * r] *= turn;
                    o[i][2 * r + 1] *= turn;
                }
                m[r] = top;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float x = tc::ex2(fmaf(s[t][2 * r], f, -base)), y = tc::ex2(fmaf(s[t][2 * r + 1], f, -base));
                l[r] += x + y;
                tc::pack_hi_lo(x, y, hi[2 * t + r], lo[2 * t + r]);
            }
        }
        // matrices: tokens 8 (mat % 2), channels + 8 (mat / 2)
        const uint32_t at = V + (8 * (mat & 1) + row) * 128;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            uint32_t b[4];
            ldsm_x4_trans(at + (i >> 2) * 2048 + ((((2 * i + (mat >> 1)) ^ row) & 7) << 4), b);
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] &= keep[e & 1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                tc::mma_bf16_16x8x16(o[2 * i + e], lo, b[2 * e], b[2 * e + 1]);
                tc::mma_bf16_16x8x16(o[2 * i + e], hi, b[2 * e], b[2 * e + 1]);
            }
        }
    }
    __device__ __forceinline__ void end() {   // the rows' sums over the lanes that share them
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
    }
    // [16][D] sums, then [16] maxima and sums
    __device__ __forceinline__ void put(float *dst, int lane) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(dst + row * D + 8 * i + 2 * (lane & 3)) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
            if ((lane & 3) == 0) *reinterpret_cast<float2 *>(dst + kHeads * D + 2 * row) = make_float2(m[r], l[r]);
        }
    }
    __device__ __forceinline__ void add(const float *src, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
            const float2 ml = *reinterpret_cast<const float2 *>(src + kHeads * D + 2 * row);
            const float top = fmaxf(m[r], ml.x), base = top == -INFINITY ? 0.f : top;
            const float f = tc::ex2(m[r] - base), e = tc::ex2(ml.x - base);
            m[r] = top;
            l[r] = l[r] * f + ml.y * e;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float2 x = *reinterpret_cast<const float2 *>(src + row * D + 8 * i + 2 * (lane & 3));
                o[i][2 * r] = o[i][2 * r] * f + x.x * e;
                o[i][2 * r + 1] = o[i][2 * r + 1] * f + x.y * e;
            }
        }
    }
};

// fp32: scores by lane = token (lane % 8, a quarter of the channels each), sums by lane = channels
// (D / 32) lane ..; every lane has all rows' maxima and its own tokens' sums.
template <int D>
struct State<D, false> {
    static constexpr int C = D / 32;
    float o[kHeads][C], m[kHeads], l[kHeads];
    int rows;
    __device__ __forceinline__ void begin(const StepArgs &a, const Cursor<8> &u, int) {
        const int g = a.p.Hq / a.p.Hk;
        rows = min(kHeads, g - (u.hu % a.per_h) * kHeads);
        reset();
    }
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) o[h][c] = 0.f;
        }
    }
    __device__ __forceinline__ void group(const StepArgs &a, const Seen<8> &seen, int j0, const unsigned char *stage, int lane, const float *q_s) {
        const uint32_t K = smem_u32(stage), V = K + D * 32, Q = smem_u32(q_s);
        const int t = lane & 7, part = lane >> 3;
        const bool in = seen.sees(j0 + t), whole = seen.whole(j0);
        float s[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) s[h] = 0.f;
#pragma unroll 2
        for (int i = 0; i < D / 16; ++i) {
            const int c = part * (D / 16) + i;      // 16 bytes of the token's row
            const float4 k = lds128f(K + (c >> 3) * 1024 + t * 128 + (((c ^ t) & 7) << 4));
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= rows) break;
                const float4 q = lds128f(Q + (h * D + 4 * c) * 4);
                s[h] = fmaf(k.x, q.x, s[h]);
                s[h] = fmaf(k.y, q.y, s[h]);
                s[h] = fmaf(k.z, q.z, s[h]);
                s[h] = fmaf(k.w, q.w, s[h]);
            }
        }
        const float f = a.p.scale * kLog2e;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= rows) break;
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 8);
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 16);
            s[h] = in ? s[h] * f : -INFINITY;
            float top = s[h];
#pragma unroll
            for (int w = 4; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            top = fmaxf(top, m[h]);
            const float base = top == -INFINITY ? 0.f : top;
            if (top > m[h]) {   // (the same in every lane)
                const float turn = exp2f(m[h] - base);
                l[h] *= turn;
#pragma unroll
                for (int c = 0; c < C; ++c) o[h][c] *= turn;
                m[h] = top;
            }
            s[h] = exp2f(s[h] - base);
            l[h] += part == 0 ? s[h] : 0.f;
        }
        const int ch = C * lane;
#pragma unroll 2
        for (int t2 = 0; t2 < 8; ++t2) {
            const uint32_t at = V + (ch >> 5) * 1024 + t2 * 128 + ((((ch >> 2) ^ t2) & 7) << 4) + (ch & 3) * 4;
            float v[C];
            if (C == 4) {
                const float4 x = lds128f(at);
                v[0] = x.x; v[1] = x.y; v[C - 2] = x.z; v[C - 1] = x.w;
            } else {
                const float2 x = lds64f(at);
                v[0] = x.x; v[1] = x.y;
            }
            if (!whole && !seen.sees(j0 + t2)) continue;   // (its values may be anything)
#pragma unroll
            for (int h = 0; h < kHeads; ++h) {
                if (h >= rows) break;
                const float p = __shfl_sync(0xffffffffu, s[h], t2);
#pragma unroll
                for (int c = 0; c < C; ++c) o[h][c] = fmaf(p, v[c], o[h][c]);
            }
        }
    }
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
    }
    __device__ __forceinline__ void put(float *dst, int lane) const {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
#pragma unroll
            for (int c = 0; c < C; ++c) dst[h * D + C * lane + c] = o[h][c];
            if (lane == 0) *reinterpret_cast<float2 *>(dst + kHeads * D + 2 * h) = make_float2(m[h], l[h]);
        }
    }
    __device__ __forceinline__ void add(const float *src, int lane) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            const float2 ml = *reinterpret_cast<const float2 *>(src + kHeads * D + 2 * h);
            const float top = fmaxf(m[h], ml.x), base = top == -INFINITY ? 0.f : top;
            const float f = exp2f(m[h] - base), e = exp2f(ml.x - base);
            m[h] = top;
            l[h] = l[h] * f + ml.y * e;
#pragma unroll
            for (int c = 0; c < C; ++c) o[h][c] = o[h][c] * f + src[h * D + C * lane + c] * e;
        }
    }
};

template <int D, bool BF>
struct Layout {
    static constexpr int E = BF ? 2 : 4, TILE = group_tokens<BF>() * D * E, STAGE = 2 * TILE;   // keys, values of a group
    static constexpr int STAGES = kStages * 128 / D;                   // a warp's
    static constexpr int RING = kWarps * STAGES * STAGE;
    static constexpr int PART = kHeads * (D + 2) * 4;                                 // a warp's state
    static constexpr int PARTS = RING, Q = PARTS, BARS = PARTS + kWarps / 2 * PART;   // (fp32 queries in the states' place)
    static constexpr int TOTAL = BARS + kWarps * STAGES * 8;
    static_assert(TOTAL + 1024 <= 227 * 1024, "shared memory");
};

template <typename T>
__device__ __forceinline__ void put_out(T *dst, float x) { *dst = from_f32<T>(x); }

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1)
attn_step_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const StepArgs a) {
    using L = Layout<D, BF>;
    using T = typename std::conditional<BF, __nv_bfloat16, float>::type;
    extern __shared__ unsigned char dsm_raw[];
    __shared__ int polls_s;
    unsigned char *sm = align1024(dsm_raw);
    constexpr int G = group_tokens<BF>();
    const float *q_s = reinterpret_cast<const float *>(sm + L::Q);
    int64_t *sums = reinterpret_cast<int64_t *>(sm + L::PARTS);   // (until the first unit's end)
    static_assert(8 * kThreads <= L::PART, "shared memory");
    const AttnStep &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS) + warp * L::STAGES;
    if (lane == 0)
        for (int i = 0; i < L::STAGES; ++i) mbar_init(bars + i, 1);
    if (tid == 0) polls_s = tc::kPolls;
    fence_mbar_init();

    // the units' groups up to each of 256 runs of sequences
    const int64_t run = (p.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int64_t b = tid * run; b < min(p.B, (tid + 1) * run); ++b) mine += Seen<G>(p, p.lens[b]).n;
    mine *= a.hus;
    int64_t upto = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, w);
        if (lane >= w) upto += x;
    }
    __shared__ int64_t warps_s[kWarps];
    if (lane == 31) warps_s[warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warps_s[w];
        total += warps_s[w];
    }
    sums[tid] = before + upto - mine;
    __syncthreads();
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    per = per < kLeast ? kLeast : per;
    const int64_t begin = blockIdx.x * per, end = min(total, begin + per);

    // sequences without a visible token
    for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (Seen<G>(p, p.lens[b]).n > 0) continue;
        for (int i = tid; i < p.Hq * D; i += kThreads) put_out((T *)p.out + b * p.Hq * D + i, 0.f);
        for (int i = tid; p.lse && i < p.Hq; i += kThreads) p.lse[b * p.Hq + i] = -INFINITY;
    }
    if (tid == 0) a.tail[blockIdx.x].b = -1;
    if (begin >= end) return;

    Cursor<G> load, cur;
    {   // the last run that begins at or before `begin` and is not empty there
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sums[mid] <= begin) lo = mid;
            else hi = mid - 1;
        }
        cur.b = lo * run;
        cur.first = sums[lo];
        cur.hu = 0;
        cur.n = cur.b < p.B ? Seen<G>(p, p.lens[cur.b]).n : 0x7fffffff;
    }
    __syncthreads();
    cur.seek(a, begin);
    load = cur;

    unsigned char *ring = sm + warp * L::STAGES * L::STAGE;
    const int rows_all = (int)(p.n_pages * p.Hk * p.page);   // behind the cache's end: zeros
    int64_t next = begin + warp;          // group to load
    int issued = 0;
    auto issue = [&]() {
        if (next >= end) return;
        load.seek(a, next);
        if (lane == 0) {
            const Seen<G> seen(p, p.lens[load.b]);
            const int j0 = seen.group((int)(next - load.first)) * G;
            const int page = p.pages[load.b * p.max_pages + j0 / p.page];
            const int hk = load.hu / a.per_h;
            const int row = page >= 0 && page < p.n_pages ? (int)(((int64_t)page * p.Hk + hk) * p.page + j0 % p.page) : rows_all;
            const int s = issued % L::STAGES;
            mbar_arrive_expect_tx(bars + s, L::STAGE);
            tc::tma_load_3d(ring + s * L::STAGE, &tk, bars + s, 0, row, 0);
            tc::tma_load_3d(ring + s * L::STAGE + L::TILE, &tv, bars + s, 0, row, 0);
        }
        ++issued;
        next += kWarps;
    };
#pragma unroll 1
    for (int i = 0; i < L::STAGES; ++i) issue();

    State<D, BF> st;
    float *parts = reinterpret_cast<float *>(sm + L::PARTS);
    int64_t at = begin + warp;
    int done = 0;
#pragma unroll 1
    for (int64_t unit0 = begin; unit0 < end;) {
        cur.seek(a, unit0);
        const int64_t unit1 = min(end, cur.first + cur.n);
        const Seen<G> seen(p, p.lens[cur.b]);
        const int g = p.Hq / p.Hk, hk = cur.hu / a.per_h, h0 = (cur.hu % a.per_h) * kHeads, rows = min(kHeads, g - h0);
        const int64_t head = cur.b * p.Hq + hk * g + h0;
        if (!BF) {
            float *Q = reinterpret_cast<float *>(sm + L::Q);
            for (int i = tid; i < rows * D; i += kThreads) Q[i] = ((const float *)p.q)[head * D + i];
            __syncthreads();
        }
        st.begin(a, cur, lane);
#pragma unroll 1
        for (; at < unit1; at += kWarps) {
            const int s = done % L::STAGES;
            const int j0 = seen.group((int)(at - cur.first)) * G;
            // (a page that is not there is not visible)
            const int page = p.pages[cur.b * p.max_pages + j0 / p.page];
            if (!mbar_try_wait(bars + s, (done / L::STAGES) & 1)) tc::wait_longer(bars + s, (done / L::STAGES) & 1, &polls_s);
            if (page >= 0 && page < p.n_pages) st.group(a, seen, j0, ring + s * L::STAGE, lane, q_s);
            __syncwarp();
            ++done;
            issue();
        }
        st.end();
        if (!BF) __syncthreads();   // the queries are read
        // the warps' states, the upper half's into the lower half's
#pragma unroll 1
        for (int w = kWarps / 2; w > 0; w >>= 1) {
            if (warp >= w && warp < 2 * w) st.put(parts + (warp - w) * (L::PART / 4), lane);
            __syncthreads();
            if (warp < w) st.add(parts + warp * (L::PART / 4), lane);
            __syncthreads();
        }
        const bool starts = unit0 == cur.first, ends = unit1 == cur.first + cur.n;
        if (warp == 0) st.put(starts && ends ? parts : a.partial + ((int64_t)blockIdx.x * 2 + (starts ? 1 : 0)) * kPartialFloats, lane);
        if (starts && ends) {
            __syncthreads();
            for (int i = tid; i < rows * D; i += kThreads) {
                const float sum = parts[kHeads * D + 2 * (i / D) + 1];
                put_out((T *)p.out + head * D + i, sum > 0.f ? parts[i] / sum : 0.f);
            }
            if (p.lse && tid < rows) {
                const float2 ml = *reinterpret_cast<const float2 *>(parts + kHeads * D + 2 * tid);
                p.lse[head + tid] = ml.y > 0.f ? (ml.x + log2f(ml.y)) * kLn2 : -INFINITY;
            }
            __syncthreads();
        } else if (starts && tid == 0) {
            a.tail[blockIdx.x] = Tail{cur.b, cur.hu, (int)((cur.first + cur.n - 1) / per)};
        }
        unit0 = unit1;
    }
    // (after an expiry) the copies have landed before the block ends
    for (int i = max(0, issued - L::STAGES); i < issued; ++i) tc::wait_cycles(bars + i % L::STAGES, (i / L::STAGES) & 1);
    if (tid == 0 && polls_s == 0) atomicExch(a.status, kErrTimeout);
}

// Joins the parts of the unit that block blockIdx.x began and other blocks went on with.
template <int D, bool BF>
__global__ void __launch_bounds__(512) attn_join_kernel(const StepArgs a) {
    using T = typename std::conditional<BF, __nv_bfloat16, float>::type;
    const Tail tail = a.tail[blockIdx.x];
    if (tail.b < 0) return;
    __shared__ float weight[kBlocks][kHeads];
    __shared__ float4 sum_s[512];
    const AttnStep &p = a.p;
    const int g = p.Hq / p.Hk, hk = tail.hu / a.per_h, h0 = (tail.hu % a.per_h) * kHeads, rows = min(kHeads, g - h0);
    const int64_t head = tail.b * p.Hq + hk * g + h0;
    const int first = blockIdx.x, n = tail.last - first + 1, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto part = [&](int c) { return a.partial + ((int64_t)(first + c) * 2 + (c == 0 ? 1 : 0)) * kPartialFloats; };
    // a warp a row: the parts' weights
    if (warp < rows) {
        float top = -INFINITY;
        for (int c = lane; c < n; c += 32) top = fmaxf(top, part(c)[kHeads * D + 2 * warp]);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        const float base = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        for (int c = lane; c < n; c += 32) {
            const float e = exp2f(part(c)[kHeads * D + 2 * warp] - base);
            weight[c][warp] = e;
            sum = fmaf(part(c)[kHeads * D + 2 * warp + 1], e, sum);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        __syncwarp();
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        for (int c = lane; c < n; c += 32) weight[c][warp] *= inv;
        if (p.lse && lane == 0) p.lse[head + warp] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    }
    __syncthreads();
    // four channels of a row a thread, the parts dealt out to the threads that are left
    const int quads = rows * (D / 4), ways = 512 / quads, way = tid / quads, i = tid % quads, row = i / (D / 4);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (way < ways)
#pragma unroll 4
        for (int c = way; c < n; c += ways) {
            const float4 y = reinterpret_cast<const float4 *>(part(c))[i];
            const float w = weight[c][row];
            x.x = fmaf(w, y.x, x.x); x.y = fmaf(w, y.y, x.y); x.z = fmaf(w, y.z, x.z); x.w = fmaf(w, y.w, x.w);
        }
    sum_s[tid] = x;
    __syncthreads();
    if (tid < quads) {
        for (int c = 1; c < ways; ++c) {
            const float4 y = sum_s[c * quads + tid];
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        store4((T *)p.out + head * D + 4 * i, x);
    }
}

// The cache as [rows = pages x heads x slots][d]: boxes of 16 rows in columns of 128 bytes, 128-byte swizzle.
bool make_map(CUtensorMap *m, const void *base, const AttnStep &p) {
    auto enc = tc_tensor_map_encoder();
    if (!enc) return false;
    const int e = p.bf16 ? 2 : 4, w = 128 / e;
    cuuint64_t dims[3] = {(cuuint64_t)w, (cuuint64_t)(p.n_pages * p.Hk * p.page), (cuuint64_t)(p.d / w)};
    cuuint64_t strides[2] = {(cuuint64_t)(p.d * e), 128};
    cuuint32_t box[3] = {(cuuint32_t)w, (cuuint32_t)(p.bf16 ? 16 : 8), (cuuint32_t)(p.d / w)}, es[3] = {1, 1, 1};
    return enc(m, p.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base), dims,
               strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks: as many as the most groups that the sequences can have give work to.
int blocks_of(const AttnStep &p) {
    const int64_t G = p.bf16 ? 16 : 8;
    const int64_t units = p.B * p.Hk * ((p.Hq / p.Hk + kHeads - 1) / kHeads);
    const int64_t room = ((int64_t)p.max_pages * p.page + G - 1) / G;
    int64_t groups = room;
    if (p.window < kNoWindow) {
        const int64_t seen = (p.window + G - 1) / G + 1 + (p.sinks + G - 1) / G;
        groups = seen < room ? seen : room;
    }
    if (groups > kBlocks * kLeast || units > kBlocks * kLeast) return kBlocks;
    const int64_t n = (units * groups + kLeast - 1) / kLeast;
    return (int)(n < 1 ? 1 : n < kBlocks ? n : kBlocks);
}

template <int D, bool BF>
int launch(const CUtensorMap *m, const StepArgs &a, int blocks, cudaStream_t s) {
    constexpr int smem = Layout<D, BF>::TOTAL + 1024;
    if (cudaFuncSetAttribute(attn_step_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return kErrCuda;
    attn_step_kernel<D, BF><<<blocks, kThreads, smem, s>>>(m[0], m[1], a);
    if (cudaGetLastError() != cudaSuccess) return kErrCuda;
    if (blocks == 1) return kOk;
    attn_join_kernel<D, BF><<<blocks - 1, 512, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? kOk : kErrCuda;
}

}  // namespace

size_t attn_step_workspace_bytes(const AttnStep &p) {
    const int64_t n = blocks_of(p);
    return (size_t)n * (2 * sizeof(float) * kPartialFloats + sizeof(Tail));
}

int launch_attn_step(const AttnStep &p, void *workspace, int *status, cudaStream_t stream) {
    CUtensorMap m[2];
    if (!make_map(&m[0], p.kc, p) || !make_map(&m[1], p.vc, p)) return kErrCuda;
    const int blocks = blocks_of(p);
    StepArgs a{};
    a.p = p;
    a.per_h = (p.Hq / p.Hk + kHeads - 1) / kHeads;
    a.hus = p.Hk * a.per_h;
    a.partial = (float *)workspace;
    a.tail = (Tail *)((char *)workspace + (size_t)blocks * 2 * sizeof(float) * kPartialFloats);
    a.status = status;
    if (p.bf16) return p.d == 64 ? launch<64, true>(m, a, blocks, stream) : launch<128, true>(m, a, blocks, stream);
    return p.d == 64 ? launch<64, false>(m, a, blocks, stream) : launch<128, false>(m, a, blocks, stream);
}

}  // namespace dr
