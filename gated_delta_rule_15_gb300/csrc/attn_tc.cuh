// attn_tc.cuh -- what the tensor-core kernels of the window attention share: tensor maps, bounded waits,
// masks and the key tiles of a run of queries.  The mathematics: attn.h.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn.h"
#include "common.cuh"
#include "tc_common.cuh"
#include "tc_issue.cuh"

namespace dr {

PFN_cuTensorMapEncodeTiled_v12000 tc_tensor_map_encoder();

namespace attn {

using namespace umma;
using tc::elect_one;
using tc::ex2;
using tc::pack_bf16;

constexpr int kSms = 152, kKeys = 128, kBox = 32;   // key tile; rows of a copy

// [rows, heads, d] bf16, rows `stride` elements apart; boxes of 64 channels x `heads_box` x `rows_box`, 128-byte
// swizzle.  Rows behind the last read as zeros.
inline bool make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t heads, int64_t d, int64_t stride, int heads_box, int rows_box) {
    auto enc = tc_tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)heads_box, (cuuint32_t)rows_box}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query heads (of those that share a key head) whose rows lie side by side in a tile of 128 rows, a
// power of two (its log2): tiles then span fewer tokens, and less of what they compute is masked.
inline int heads_in_tile(int group) { return group % 4 == 0 ? 2 : group % 2 == 0 ? 1 : 0; }

__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }
// Which of the keys j0 .. j0 + 31 the query i sees, of those before `end`.
__device__ __forceinline__ uint32_t seen_bits(int i, int j0, int end, int window, int sinks) {
    return low_bits(min(i + 1, end) - j0) & (~low_bits(i - window + 1 - j0) | low_bits(sinks - j0));
}

// The keys of the queries q0 .. q0 + count - 1 of a sequence, one behind another: the sinks in front of the first
// one's window, filled up to a multiple of 32 (the rest is masked), then the keys from there to the last one; in tiles of 128.
// (Tiles of sinks apart cost an item a tile's time for four keys.)
struct KeyTiles {
    int sinks, s32, near0, end, total, n;
    KeyTiles() = default;
    __device__ __forceinline__ KeyTiles(int q0, int count, int len, int window, int all_sinks) {
        near0 = max(0, q0 - window + 1);
        sinks = min(all_sinks, near0);
        s32 = (sinks + 31) & ~31;          // (at most q0: those rows are the sequence's)
        end = min(len, q0 + count);
        total = s32 + end - near0;
        n = (total + kKeys - 1) / kKeys;
    }
    __device__ __forceinline__ int count(int t) const { return min(kKeys, total - t * kKeys); }
    __device__ __forceinline__ int key(int at) const { return at < s32 ? at : near0 + at - s32; }
    // the keys of `at` .. + 31 (a multiple of 32) that query i sees
    __device__ __forceinline__ uint32_t bits(int i, int at, int window, int all_sinks) const {
        return seen_bits(i, key(at), at < s32 ? sinks : end, window, all_sinks);
    }
    // tile t's first row that is behind the sequence
    __device__ __forceinline__ int behind(int t, int len) const { return s32 + len - near0 - t * kKeys; }
};

// Of the tiles, those of which one of the queries a .. b - 1 sees a key, and those of which every one sees all keys.
struct TileRanges {
    int s_any, n_any0, n_any1, s_all, n_all0, n_all1;      // t < s or n0 <= t < n1
    TileRanges() = default;
    __device__ __forceinline__ TileRanges(const KeyTiles &kt, int a, int b, int window, int all_sinks) {
        // tile t of the window starts at key k0 + 128 t
        const int k0 = kt.near0 - kt.s32, some = (kt.s32 + kKeys - 1) / kKeys;
        s_any = a < b ? some : 0;
        n_any0 = a < b ? max(some, k0 < all_sinks && kt.near0 < all_sinks ? 0 : (max(0, a - window + 1 - kKeys - k0) + kKeys - 1) / kKeys) : kt.n;
        n_any1 = a < b ? min(kt.n, (max(0, b - k0) + kKeys - 1) / kKeys) : 0;
        s_all = kt.sinks / kKeys;
        n_all0 = max(some, (max(0, b - window - k0) + kKeys - 1) / kKeys);
        n_all1 = min(kt.total / kKeys, a + 1 - k0 >= 0 ? (a + 1 - k0) / kKeys : 0);
    }
    __device__ __forceinline__ bool meets(int t) const { return t < s_any || (t >= n_any0 && t < n_any1); }
    __device__ __forceinline__ bool whole(int t) const { return t < s_all || (t >= n_all0 && t < n_all1); }
};

// This block's item of a round.  Items of falling length (every query sees all before it) are dealt every other round
// backwards, so that blocks get equal shares of long ones and short ones: forward of B2 T8192 H16 d128 469 -> 427 us; equal
// ones are dealt straight on (dq of B8 T2048 H16/4 w1024 160 us, every other round backwards 180).
__device__ __forceinline__ int64_t dealt(int64_t round, bool falling) {
    return round * gridDim.x + (falling && round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// Polls of a wait (tc::wait_longer).  Most waits last a tile, but some an item: those of dq's statistics warps, which are
// items ahead, and those of a forward's second stage whose rows lie behind the sequence's end while the first runs through
// all key tiles.  So the bound follows the longest item: a tile takes some 60 polls of 60 cycles.
inline int item_polls(const AttnProblem &p, int tokens) {
    const int64_t longest = p.seqs.cu ? p.seqs.total : p.seqs.T, reach = (int64_t)p.window + p.sinks + tokens + 32;
    const int64_t tiles = (longest < reach ? longest : reach) / kKeys + 2;
    return tc::kPolls + (int)((tiles < 1 << 20 ? tiles : 1 << 20) << 10);
}

// Whether x holds in any thread of the two warps that share the named barrier `id`.
__device__ __forceinline__ bool any_of(uint32_t id, bool x) {
    uint32_t y;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbarrier.cta.red.or.pred q, %2, 64, p;\nselp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(y) : "r"((uint32_t)x), "r"(id) : "memory");
    return y != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}


// 8 N bf16 values of one row a lane (32 rows a warp) to global memory: the lanes exchange 16-byte pieces within
// groups of N, so that a group writes 16 N bytes of one row at a time.  `at(r)`: where this lane's columns' first
// one of the warp's row r lies, or NULL.
template <int N, class At>
__device__ __forceinline__ void put_rows(uint4 (&u)[N], int lane, At at) {
#pragma unroll
    for (int b = 1; b < N; b <<= 1)
#pragma unroll
        for (int s = 0; s < N; ++s) {
            if (s & b) continue;
            const bool up = lane & b;
            uint4 x = up ? u[s] : u[s | b];
            x.x = __shfl_xor_sync(0xffffffffu, x.x, b);
            x.y = __shfl_xor_sync(0xffffffffu, x.y, b);
            x.z = __shfl_xor_sync(0xffffffffu, x.z, b);
            x.w = __shfl_xor_sync(0xffffffffu, x.w, b);
            if (up) u[s] = x;
            else u[s | b] = x;
        }
#pragma unroll
    for (int r = 0; r < N; ++r) {
        __nv_bfloat16 *dst = at((lane & ~(N - 1)) + r);
        if (dst) reinterpret_cast<uint4 *>(dst)[lane & (N - 1)] = u[r];
    }
}
// C accumulator columns times f as bf16 pieces
template <int C>
__device__ __forceinline__ void to_pieces(const float (&o)[C], float f, uint4 (&u)[C / 8]) {
#pragma unroll
    for (int x = 0; x < C / 8; ++x)
        u[x] = make_uint4(pack_bf16(o[8 * x] * f, o[8 * x + 1] * f), pack_bf16(o[8 * x + 2] * f, o[8 * x + 3] * f),
                          pack_bf16(o[8 * x + 4] * f, o[8 * x + 5] * f), pack_bf16(o[8 * x + 6] * f, o[8 * x + 7] * f));
}
template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[C]) {
    if constexpr (C == 32) tmem_ld32(taddr, v);
    else tmem_ld16(taddr, v);
}

}  // namespace attn

// Tensor cores: bf16 rows.  `status`: the library's device status word.
int launch_attn_tc_fwd(const AttnProblem &p, int *status, cudaStream_t stream);
size_t attn_tc_bwd_workspace_bytes(const AttnProblem &p);   // (by seqs.cu being NULL or not, not what it holds)
int launch_attn_tc_bwd(const AttnProblem &p, void *workspace, int *status, cudaStream_t stream);

}  // namespace dr
