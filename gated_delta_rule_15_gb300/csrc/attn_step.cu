// attn_step.cu -- window attention of one new token for each sequence over a paged cache.  The
// mathematics: attn.h (the query is the sequence's last token).
//
// Every visible key and value is read once: HBM bandwidth bounds it (256 sequences of 16 to 16384 tokens, H32/8 d128 w4096,
// 1.48 GB: 247 us, 6.0 TB/s; one of 131072 tokens, H16/4: 59 us, 48 of them in the first kernel, 5.6 TB/s).  The visible tokens of a unit (a
// sequence, a key head and up to 16 of the query heads that share it) are cut into groups of 16 (fp32: 8), which never
// cross a page: first the groups that hold sinks, then those of the window.  The units, one behind another,
// are dealt out evenly to all warps of the GPU, a unit counting as its groups and one more for what it costs to
// begin and end: a warp takes a run of groups, whatever units they belong to, so that one long context fills the
// GPU as a batch of any lengths does.  A unit that ends up in several warps leaves a partial result (maximum, sum,
// sum of values) for each, or for a block whose warps all work at it one, and a second kernel joins them in a fixed
// order.  (Blocks as the takers, all their warps at one unit and their states added up at its end, took 2126 us
// for 256 sequences of 16 to 16384 tokens: a block with the short ones spent 7 us on each.)
//
// A warp copies its groups by a tensor-map box of the group's keys and one of its values into a ring of
// kStages stages of its own, so 192 KB are under way on an SM, and no warp waits for another one.
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
#include "launch_chain.cuh"
#include "tc_common.cuh"
#include "tc_issue.cuh"

namespace dr {

PFN_cuTensorMapEncodeTiled_v12000 tc_tensor_map_encoder();

namespace {

using namespace umma;

constexpr int kWarps = 8, kStages = 3, kThreads = 32 * kWarps, kHeads = 16, kBlocks = 152;
template <bool BF> constexpr int group_tokens() { return BF ? 16 : 8; }   // 8 KB of keys and values at d = 128
constexpr int kLeast = 2;            // groups of a warp, at least
constexpr int kUnitCost = 1;         // what a unit's begin and end count as, in groups

struct Tail {                        // the unit that a warp (or a block, by its first warp) began and did not end
    int64_t b;                       // -1: none
    int64_t first, end, per, total;  // its place in the row of all units; what a warp takes; the row's length
    int hu;                          // unit of the sequence
};

struct StepArgs {
    AttnStep p;
    int hus, per_h;                  // units a sequence, units a key head
    float *partial;                  // [warp][head or tail part] of part_floats: [rows][d] sums, [rows] (maximum, sum)
    int part_floats;
    Tail *tail;                      // [warp]
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

// Walks the units of a warp's run [begin, end) of the row of all units.
template <int G>
struct Walk {
    int64_t b, first;                // sequence; where its current unit begins
    int hu;                          // unit of the sequence
    int lo, hi;                      // the unit's groups that are in the run
    Seen<G> seen;
    __device__ __forceinline__ Walk(const StepArgs &a, int64_t b0, int64_t first0, int64_t begin, int64_t end)
        : b(b0), first(first0), hu(0), lo(0), hi(0), seen(a.p, b0 < a.p.B ? a.p.lens[b0] : 0) {
        while (b < a.p.B && first + length(a) <= begin) {   // whole sequences in front of it
            first += length(a);
            ++b;
            seen = Seen<G>(a.p, b < a.p.B ? a.p.lens[b] : 0);
        }
        if (seen.n > 0) {
            hu = (int)((begin - first) / (seen.n + kUnitCost));
            first += (int64_t)hu * (seen.n + kUnitCost);
        }
        cut(begin, end);
    }
    // of the sequence in the row of all units (units of 2^30 tokens and some tens of heads pass 31 bits)
    __device__ __forceinline__ int64_t length(const StepArgs &a) const { return seen.n > 0 ? (int64_t)a.hus * (seen.n + kUnitCost) : 0; }
    __device__ __forceinline__ void cut(int64_t begin, int64_t end) {
        const int64_t l = begin - first - kUnitCost, h = end - first - kUnitCost;
        lo = (int)max((int64_t)0, l);
        hi = (int)min((int64_t)seen.n, h);
    }
    // On to the next unit; false behind the run.
    __device__ __forceinline__ bool next(const StepArgs &a, int64_t begin, int64_t end) {
        first += seen.n + kUnitCost;
        if (first >= end) return false;
        if (++hu == a.hus) {
            hu = 0;
            do {
                ++b;
                seen = Seen<G>(a.p, a.p.lens[b]);
            } while (seen.n == 0);
        }
        cut(begin, end);
        return true;
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
    __device__ __forceinline__ void begin(const StepArgs &a, const Walk<16> &u, int lane) {
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
    __device__ __forceinline__ void group(const StepArgs &a, const Seen<16> &seen, int j0, const unsigned char *stage, int lane, int64_t) {
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
    // [rows][D] sums, then [rows] maxima and sums
    __device__ __forceinline__ void put(float *dst, int rows, int lane) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
            if (row >= rows) continue;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(dst + row * D + 8 * i + 2 * (lane & 3)) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
            if ((lane & 3) == 0) *reinterpret_cast<float2 *>(dst + rows * D + 2 * row) = make_float2(m[r], l[r]);
        }
    }
    __device__ __forceinline__ void out(const AttnStep &p, int64_t head, int rows, int lane) const {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
            if (row >= rows) continue;
            const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
            __nv_bfloat16 *dst = (__nv_bfloat16 *)p.out + (head + row) * D + 2 * (lane & 3);
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<uint32_t *>(dst + 8 * i) = tc::pack_bf16(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
            if (p.lse && (lane & 3) == 0) p.lse[head + row] = l[r] > 0.f ? (m[r] + log2f(l[r])) * kLn2 : -INFINITY;
        }
    }
    __device__ __forceinline__ void add(const float *src, int rows, int lane) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = (lane >> 2) + 8 * r;
            if (row >= rows) continue;
            const float2 ml = *reinterpret_cast<const float2 *>(src + rows * D + 2 * row);
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
    int rows;                        // query heads of the unit
    __device__ __forceinline__ void begin(const StepArgs &a, const Walk<8> &u, int) {
        rows = min(kHeads, a.p.Hq / a.p.Hk - (u.hu % a.per_h) * kHeads);
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
    __device__ __forceinline__ void group(const StepArgs &a, const Seen<8> &seen, int j0, const unsigned char *stage, int lane, int64_t head) {
        const uint32_t K = smem_u32(stage), V = K + D * 32;
        const float4 *Q = reinterpret_cast<const float4 *>(a.p.q) + head * (D / 4);   // (stays in L1)
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
                const float4 q = __ldg(Q + h * (D / 4) + c);
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
    __device__ __forceinline__ void put(float *dst, int n, int lane) const {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= n) break;
#pragma unroll
            for (int c = 0; c < C; ++c) dst[h * D + C * lane + c] = o[h][c];
            if (lane == 0) *reinterpret_cast<float2 *>(dst + n * D + 2 * h) = make_float2(m[h], l[h]);
        }
    }
    __device__ __forceinline__ void out(const AttnStep &p, int64_t head, int n, int lane) const {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= n) break;
            const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) ((float *)p.out)[(head + h) * D + C * lane + c] = o[h][c] * inv;
            if (p.lse && lane == 0) p.lse[head + h] = l[h] > 0.f ? (m[h] + log2f(l[h])) * kLn2 : -INFINITY;
        }
    }
    __device__ __forceinline__ void add(const float *src, int n, int lane) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            if (h >= n) break;
            const float2 ml = *reinterpret_cast<const float2 *>(src + n * D + 2 * h);
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
    static constexpr int PARTS = RING, BARS = PARTS + kWarps / 2 * PART;
    static constexpr int TOTAL = BARS + kWarps * STAGES * 8;
    static_assert(TOTAL + 1024 <= 227 * 1024, "shared memory");
};

template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1)
attn_step_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const StepArgs a) {
    using L = Layout<D, BF>;
    using T = typename std::conditional<BF, __nv_bfloat16, float>::type;
    constexpr int G = group_tokens<BF>();
    extern __shared__ unsigned char dsm_raw[];
    __shared__ int polls_s;
    unsigned char *sm = align1024(dsm_raw);
    const AttnStep &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *parts = reinterpret_cast<float *>(sm + L::PARTS);
    int64_t *sums = reinterpret_cast<int64_t *>(sm + L::PARTS);   // [kThreads], [kWarps] (until the runs are known)
    static_assert(8 * (kThreads + kWarps) <= kWarps / 2 * L::PART, "shared memory");
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::BARS) + warp * L::STAGES;
    if (lane == 0)
        for (int i = 0; i < L::STAGES; ++i) mbar_init(bars + i, 1);
    if (tid == 0) polls_s = tc::kPolls;
    fence_mbar_init();
    let_next_start();

    // what the units in front of each of 256 runs of sequences cost
    const int64_t run = (p.B + kThreads - 1) / kThreads;
    int64_t mine = 0;
    for (int64_t b = tid * run; b < min(p.B, (tid + 1) * run); ++b) {
        const int n = Seen<G>(p, p.lens[b]).n;
        mine += n > 0 ? n + kUnitCost : 0;
    }
    mine *= a.hus;
    int64_t upto = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, w);
        if (lane >= w) upto += x;
    }
    if (lane == 31) sums[kThreads + warp] = upto;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[kThreads + w];
        total += sums[kThreads + w];
    }
    sums[tid] = before + upto - mine;
    __syncthreads();
    int64_t per = (total + gridDim.x * kWarps - 1) / (gridDim.x * kWarps);
    per = per < kLeast ? kLeast : per;
    const int wid = blockIdx.x * kWarps + warp;
    const int64_t block0 = min(total, (int64_t)blockIdx.x * kWarps * per), block1 = min(total, block0 + kWarps * per);
    const int64_t begin = min(total, wid * per), end = min(total, begin + per);

    // sequences without a visible token
    for (int64_t b = wid; b < p.B; b += gridDim.x * kWarps) {
        if (Seen<G>(p, p.lens[b]).n > 0) continue;
        for (int i = lane; i < p.Hq * D; i += 32) ((T *)p.out)[b * p.Hq * D + i] = from_f32<T>(0.f);
        for (int i = lane; p.lse && i < p.Hq; i += 32) p.lse[b * p.Hq + i] = -INFINITY;
    }
    if (lane == 0) a.tail[wid].b = -1;
    if (block0 >= block1) return;

    // the last run of sequences that begins at or before `at`
    auto run_of = [&](int64_t at) {
        int lo = 0, hi = kThreads - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (sums[mid] <= at) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    // (a warp without a run of its own stands where the block begins)
    const int r = run_of(begin < end ? begin : block0);
    Walk<G> u(a, r * run, sums[r], begin < end ? begin : block0, end);
    // whether all warps work at one unit
    const bool joint = block1 - block0 > per && u.first <= block0 && block1 <= u.first + u.seen.n + kUnitCost;
    const bool all_joint = __syncthreads_and(joint);

    unsigned char *ring = sm + warp * L::STAGES * L::STAGE;
    const int rows_all = (int)(p.n_pages * p.Hk * p.page);   // behind the cache's end: zeros
    Walk<G> load = u;
    bool loading = begin < end;
    int issued = 0;
    uint32_t there = 0;                   // of the stages: the group's page is there
    auto issue = [&]() {
        while (loading && load.lo >= load.hi) loading = load.next(a, begin, end);
        if (!loading) return;
        const int j0 = load.seen.group(load.lo++) * G, s = issued % L::STAGES;
        const int page = p.pages[load.b * p.max_pages + j0 / p.page];
        const bool is = page >= 0 && page < p.n_pages;
        there = (there & ~(1u << s)) | (uint32_t)is << s;
        if (lane == 0) {
            const int row = is ? (int)(((int64_t)page * p.Hk + load.hu / a.per_h) * p.page + j0 % p.page) : rows_all;
            mbar_arrive_expect_tx(bars + s, L::STAGE);
            tc::tma_load_3d(ring + s * L::STAGE, &tk, bars + s, 0, row, 0);
            tc::tma_load_3d(ring + s * L::STAGE + L::TILE, &tv, bars + s, 0, row, 0);
        }
        ++issued;
    };
#pragma unroll 1
    for (int i = 0; i < L::STAGES; ++i) issue();

    State<D, BF> st;
    int done = 0;
#pragma unroll 1
    for (bool more = begin < end; more || all_joint;) {
        const int h0 = (u.hu % a.per_h) * kHeads, g = p.Hq / p.Hk, rows = min(kHeads, g - h0);
        const int64_t head = u.b * p.Hq + u.hu / a.per_h * g + h0;
        st.begin(a, u, lane);
        const int lo = u.lo;
        if (more) {
#pragma unroll 1
            for (; u.lo < u.hi; ++u.lo) {
                const int s = done % L::STAGES, j0 = u.seen.group(u.lo) * G;
                if (!mbar_try_wait(bars + s, (done / L::STAGES) & 1)) tc::wait_longer(bars + s, (done / L::STAGES) & 1, &polls_s);
                if (there >> s & 1) st.group(a, u.seen, j0, ring + s * L::STAGE, lane, head);
                __syncwarp();
                ++done;
                issue();
            }
        }
        st.end();
        bool begins = lo == 0, ends = u.hi == u.seen.n;
        if (all_joint) {      // the warps' states, the upper half's into the lower half's
            begins = block0 <= u.first + kUnitCost;
            ends = block1 == u.first + u.seen.n + kUnitCost;
#pragma unroll 1
            for (int w = kWarps / 2; w > 0; w >>= 1) {
                if (warp >= w && warp < 2 * w) st.put(parts + (warp - w) * (L::PART / 4), rows, lane);
                __syncthreads();
                if (warp < w) st.add(parts + warp * (L::PART / 4), rows, lane);
                __syncthreads();
            }
        }
        if ((all_joint && warp == 0) || (!all_joint && lo < u.hi)) {
            if (begins && ends) {
                st.out(p, head, rows, lane);
            } else {
                st.put(a.partial + ((int64_t)wid * 2 + (begins ? 1 : 0)) * a.part_floats, rows, lane);
                if (begins && lane == 0) a.tail[wid] = Tail{u.b, u.first, u.first + u.seen.n + kUnitCost, per, total, u.hu};
            }
        }
        if (all_joint) break;
        more = u.next(a, begin, end);
    }
    // (after an expiry) the copies have landed before the block ends
    for (int i = max(0, issued - L::STAGES); i < issued; ++i) tc::wait_cycles(bars + i % L::STAGES, (i / L::STAGES) & 1);
    if (lane == 0 && polls_s == 0) atomicExch(a.status, kErrTimeout);
}

// Whether the warps of block c work at one unit, and left one part of it.
__device__ __forceinline__ bool joint_block(const Tail &t, int64_t c) {
    const int64_t x0 = c * t.per * kWarps, x1 = min(t.total, x0 + t.per * kWarps);
    return x1 - x0 > t.per && t.first <= x0 && x1 <= t.end;
}

// Joins the parts of the units that the warps of block blockIdx.x began and others went on with.  Units in few warps (those
// of short contexts, several a block): a warp each, a part a lane.  Units in more: the whole block, one after another.
template <int D, bool BF>
__global__ void __launch_bounds__(512) attn_join_kernel(const StepArgs a) {
    using T = typename std::conditional<BF, __nv_bfloat16, float>::type;
    constexpr int kMost = kBlocks + 2 * kWarps;      // parts: a block's one, but for the first and last block's warps
    __shared__ Tail tails[kWarps];
    __shared__ int slot_s[kMost], n_s;
    __shared__ float weight[kMost][kHeads];
    __shared__ float4 sum_s[512];
    const AttnStep &p = a.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = p.Hq / p.Hk;
    wait_for_last();
    if (tid < kWarps) tails[tid] = a.tail[blockIdx.x * kWarps + tid];
    __syncthreads();
    auto first_warp = [&](const Tail &t) { return (t.first + kUnitCost) / t.per; };
    auto warps_of = [&](const Tail &t) { return (t.end - 1) / t.per - first_warp(t) + 1; };
    if (tails[warp % kWarps].b >= 0 && warps_of(tails[warp % kWarps]) <= 32) {      // (two warps, every other row)
        const Tail &t = tails[warp % kWarps];
        const int h0 = (t.hu % a.per_h) * kHeads, rows = min(kHeads, g - h0), n = (int)warps_of(t);
        const int64_t head = t.b * p.Hq + t.hu / a.per_h * g + h0, w = first_warp(t) + lane;
        const bool is = lane < n && (!joint_block(t, w / kWarps) || w % kWarps == 0);
        const float *mine = a.partial + (w * 2 + (lane == 0 ? 1 : 0)) * a.part_floats;
        const uint32_t all = __ballot_sync(0xffffffffu, is);
        constexpr int C = D / 32;
#pragma unroll 2
        for (int row = warp / kWarps; row < rows; row += 2) {
            const float2 ml = is ? *reinterpret_cast<const float2 *>(mine + rows * D + 2 * row) : make_float2(-INFINITY, 0.f);
            float top = ml.x;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float base = top == -INFINITY ? 0.f : top, e = exp2f(ml.x - base);
            float sum = ml.y * e;
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            const float f = sum > 0.f ? e / sum : 0.f;
            float o[C];
#pragma unroll
            for (int c = 0; c < C; ++c) o[c] = 0.f;
            for (uint32_t left = all; left; left &= left - 1) {
                const int l = __ffs(left) - 1;
                const float *src = a.partial + ((first_warp(t) + l) * 2 + (l == 0 ? 1 : 0)) * a.part_floats + row * D + C * lane;
                const float x = __shfl_sync(0xffffffffu, f, l);
#pragma unroll
                for (int c = 0; c < C; ++c) o[c] = fmaf(x, src[c], o[c]);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) ((T *)p.out)[(head + row) * D + C * lane + c] = from_f32<T>(o[c]);
            if (p.lse && lane == 0) p.lse[head + row] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        }
    }
#pragma unroll 1
    for (int own = 0; own < kWarps; ++own) {
        const Tail &t = tails[own];
        if (t.b < 0 || warps_of(t) <= 32) continue;
        __syncthreads();
        const int h0 = (t.hu % a.per_h) * kHeads, rows = min(kHeads, g - h0);
        const int64_t head = t.b * p.Hq + t.hu / a.per_h * g + h0;
        // the parts' slots, in order
        if (warp == 0) {
            const int64_t group0 = t.first + kUnitCost, per = t.per;
            const int block_a = (int)(group0 / (per * kWarps)), block_b = (int)((t.end - 1) / (per * kWarps));
            int n = 0;
#pragma unroll 1
            for (int c0 = block_a; c0 <= block_b; c0 += 32) {
                const int c = c0 + lane;
                int first = 0, count = 0;      // warps of the block that have a part
                if (c <= block_b) {
                    const int64_t x0 = c * per * kWarps;
                    const bool joint = joint_block(t, c);
                    first = joint ? 0 : (int)max((int64_t)0, (group0 - x0) / per);
                    count = joint ? 1 : (int)min((int64_t)kWarps, (t.end - x0 + per - 1) / per) - first;
                }
                int at = count;
#pragma unroll
                for (int w = 1; w < 32; w <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, at, w);
                    if (lane >= w) at += x;
                }
                const int all = __shfl_sync(0xffffffffu, at, 31);
                at += n - count;
                for (int e = 0; e < count; ++e) slot_s[at + e] = c * kWarps + first + e;
                n += all;
            }
            if (lane == 0) n_s = n;
        }
        __syncthreads();
        const int n = n_s;
        auto part = [&](int c) { return a.partial + ((int64_t)slot_s[c] * 2 + (c == 0 ? 1 : 0)) * a.part_floats; };
        // a warp a row: the parts' weights
        if (warp < rows) {
            constexpr int E = (kMost + 31) / 32;
            float2 ml[E];
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                ml[e] = lane + 32 * e < n ? *reinterpret_cast<const float2 *>(part(lane + 32 * e) + rows * D + 2 * warp) : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) top = fmaxf(top, ml[e].x);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
            const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                ml[e].x = exp2f(ml[e].x - base);
                sum = fmaf(ml[e].y, ml[e].x, sum);
            }
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (lane + 32 * e < n) weight[lane + 32 * e][warp] = ml[e].x * inv;
            if (p.lse && lane == 0) p.lse[head + warp] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        }
        __syncthreads();
        // four channels of a row a thread, the parts dealt out to the threads that are left
        const int quads = rows * (D / 4), ways = 512 / quads, way = tid / quads, i = tid % quads, row = i / (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (way < ways)
#pragma unroll 10
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
    const int64_t G = p.bf16 ? 16 : 8, least = kWarps * kLeast;
    const int64_t units = p.B * p.Hk * ((p.Hq / p.Hk + kHeads - 1) / kHeads);
    const int64_t room = ((int64_t)p.max_pages * p.page + G - 1) / G;
    int64_t groups = room;
    if (p.window < kNoWindow) {
        const int64_t seen = (p.window + G - 1) / G + 1 + (p.sinks + G - 1) / G;
        groups = seen < room ? seen : room;
    }
    if (groups > kBlocks * least || units > kBlocks * least) return kBlocks;
    const int64_t n = (units * (groups + kUnitCost) + least - 1) / least;
    return (int)(n < kBlocks ? n : kBlocks);
}
int part_rows(const AttnStep &p) { return p.Hq / p.Hk < kHeads ? p.Hq / p.Hk : kHeads; }
int part_floats(const AttnStep &p) { return (part_rows(p) * (p.d + 2) + 3) / 4 * 4; }

template <int D, bool BF>
int launch(const CUtensorMap *m, const StepArgs &a, int blocks, cudaStream_t s) {
    constexpr int smem = Layout<D, BF>::TOTAL + 1024;
    if (cudaFuncSetAttribute(attn_step_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return kErrCuda;
    attn_step_kernel<D, BF><<<blocks, kThreads, smem, s>>>(m[0], m[1], a);
    if (cudaGetLastError() != cudaSuccess) return kErrCuda;
    return launch_after(attn_join_kernel<D, BF>, (unsigned)blocks, 512, 0, s, a);
}

}  // namespace

size_t attn_step_workspace_bytes(const AttnStep &p) {
    return (size_t)blocks_of(p) * kWarps * (2 * sizeof(float) * part_floats(p) + sizeof(Tail));
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
    a.part_floats = part_floats(p);
    a.tail = (Tail *)((char *)workspace + (size_t)blocks * kWarps * 2 * sizeof(float) * a.part_floats);
    a.status = status;
    if (p.bf16) return p.d == 64 ? launch<64, true>(m, a, blocks, stream) : launch<128, true>(m, a, blocks, stream);
    return p.d == 64 ? launch<64, false>(m, a, blocks, stream) : launch<128, false>(m, a, blocks, stream);
}

}  // namespace dr
