// attn_sinks.cuh -- the blocks of the window attention's dk and dv: which keys and queries a block takes.
//
// A block takes a tile of keys of a head and the queries whose window reaches it.  Sinks are seen by every later
// query: a tile that holds some would take as long as the sequence is.  Where few tiles do, the queries
// behind the tile's window are cut into chunks with blocks of their own, which leave fp32 sums of the sinks' rows, and so does
// the tile's own block; attn_sink_sum_kernel adds them up in order.
#pragma once

#include "attn.h"
#include "common.cuh"
#include "launch_chain.cuh"

namespace dr {
namespace attn {

// Key tiles with sinks that are cut: up to 1024 sinks of bf16 rows, 512 of fp32 rows, 128 where those go in tiles of 16.  With more, every
// block that holds some runs through all later queries (backward of T1037 H6/3 d64 w200, fp32: 99 us with 2 sinks, 219 with 200).
constexpr int kMaxSplitTiles = 8;

// Cut sequences, those of more than window + tile - 1 rows, have a place each for the sums of their tiles' own blocks, and one
// for each chunk.  Where there are more packed sequences than can be cut, a cut one's place is its first row / (window + tile - 1), which
// tells it from the other cut ones (they begin further apart than that): the workspace follows the rows, not the number of
// sequences (1000 sequences in 65536 rows, H8 d128 w1024, 1024 sinks: 1.4 GB; a place for each 16).
struct SinkPlan {
    int tile;                  // keys of a block
    int tiles, rows, chunk;    // tiles that are cut (0: none), rows of their sums, tokens of a chunk
    int apart;                 // a place for every so many rows (0: for every sequence)
    int64_t places, slots;     // for the tiles' own blocks; chunks of all sequences
    float *base, *parts;       // [place | chunk slot][Hk][tile][row][dk, dv][d]
};

inline size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// How the sinks' queries are cut, and the bytes of workspace (at ws) that this takes: at most four times the
// gradients in fp32 (else, as many sinks and a short window would need, they are not cut).
inline size_t plan_sinks(const AttnProblem &p, int tile, int least, char *ws, SinkPlan &s) {
    s = SinkPlan{};
    s.tile = tile;
    s.chunk = 1 << 30;
    const int64_t longest = p.seqs.cu ? p.seqs.total : p.seqs.T, sinks = p.sinks < longest ? p.sinks : longest;
    const int64_t tiles = (sinks + tile - 1) / tile, apart = (int64_t)p.window + tile - 1;
    // (nobody is behind the window of the first tile of the longest sequence: nothing to cut)
    if (p.window >= kNoWindow || sinks == 0 || tiles > kMaxSplitTiles || longest <= apart) return 0;
    const int64_t own = p.window + tile;       // about as long as a block without sinks
    const int64_t chunk = ((own < least ? least : own) + 127) / 128 * 128, rows = sinks < tile ? sinks : tile;
    const bool by_rows = p.seqs.cu && p.seqs.total / apart < p.seqs.N;
    const int64_t places = by_rows ? p.seqs.total / apart : p.seqs.N;
    const int64_t slots = p.seqs.cu ? p.seqs.total / chunk + places : p.seqs.N * ((p.seqs.T + chunk - 1) / chunk);
    const size_t one = sizeof(float) * (size_t)p.Hk * tiles * rows * 2 * p.d, base = round256(one * places);
    if (one * (places + slots) > 4 * sizeof(float) * (size_t)p.seqs.total * (p.Hq + 2 * (size_t)p.Hk) * p.d) return 0;
    s.tiles = (int)tiles;
    s.rows = (int)rows;
    s.chunk = (int)chunk;
    s.apart = by_rows ? (int)apart : 0;
    s.places = places;
    s.slots = slots;
    s.base = (float *)ws;
    s.parts = (float *)(ws + base);
    return base + round256(one * slots);
}

#ifdef __CUDACC__
// A cut sequence's place; its chunks' slots begin at its first row / chunk + that.
__device__ __forceinline__ int64_t place_of(const SinkPlan &s, int64_t n, int64_t lo) { return s.apart ? (uint32_t)lo / (uint32_t)s.apart : n; }
// The sequence of a place or, `chunks`, of a chunk's slot; false for none.  (Behind a cut sequence the next one's place is higher by one
// at least, its first row / chunk no lower than this one's last chunk's: the last sequence that begins at or before a slot of
// a cut one is that one.  Others may be found for slots that nobody has.)  By whole warps.
__device__ __forceinline__ bool find_place(const AttnProblem &p, const SinkPlan &s, int slot, bool chunks, int64_t &n, int &j, int64_t &lo, int &len) {
    if (!p.seqs.cu) {
        const int per = chunks ? (int)((p.seqs.T + s.chunk - 1) / s.chunk) : 1;
        n = slot / per;
        j = slot - (int)n * per;
        lo = n * p.seqs.T;
        len = (int)p.seqs.T;
        return true;
    }
    if (!chunks && !s.apart) {
        int64_t hi;
        n = slot;
        j = 0;
        seq_range(p.seqs, n, lo, hi);
        len = (int)(hi - lo);
        return true;
    }
    auto key = [&](int64_t m, int64_t at) { return (chunks ? (uint32_t)at / (uint32_t)s.chunk : 0u) + place_of(s, m, at); };
    n = last_sequence(p.seqs, slot, key, lo, len);
    j = slot - (int)key(n, lo);
    return j >= 0 && (chunks ? (int64_t)j * s.chunk < len : j == 0);
}
// Chunks come first, short blocks last (dk, dv of B8 T2048 H16/4 w1024 170 us; chunks last 194).
inline int64_t key_blocks(const AttnProblem &p, const SinkPlan &s) {
    return (attn_tile_slots(p.seqs, s.tile) + s.slots * s.tiles) * p.Hk;
}

struct KeyBlock {
    int64_t n, lo, slot;       // sequence, its first row; its place, or the chunk's slot
    int len, hk, jt, k0;       // its length; head, tile, first key
    int chunk;                 // -1: the tile's own block
    int qa, qb;                // queries
    bool cut;                  // the sinks' rows are parts of sums
    // What the block does, false for nothing.  By whole warps.
    __device__ __forceinline__ bool find(const AttnProblem &p, const SinkPlan &s, int64_t block) {
        const int64_t chunks = s.slots * p.Hk * s.tiles;
        chunk = -1;
        if (block >= chunks) {
            int64_t k = block - chunks;
            hk = (int)(k % p.Hk);
            k /= p.Hk;
            if (p.seqs.cu) {
                if (!find_tile(p.seqs, s.tile, (int)k, n, jt, lo, len)) return false;
            } else {       // early keys, which most queries see, first
                n = k % p.seqs.N;
                jt = (int)(k / p.seqs.N);
                lo = n * p.seqs.T;
                len = (int)p.seqs.T;
            }
            slot = place_of(s, n, lo);
        } else {
            int64_t k = block;
            hk = (int)(k % p.Hk);
            k /= p.Hk;
            jt = (int)(k % s.tiles);
            slot = k / s.tiles;
            if (!find_place(p, s, (int)slot, true, n, chunk, lo, len)) return false;
        }
        k0 = jt * s.tile;
        if (k0 >= len) return false;
        const int behind = min(len, min(k0 + s.tile - 1, kNoWindow - 1) + p.window);     // behind the last query whose window reaches the tile
        const bool sink = k0 < p.sinks;
        cut = sink && jt < s.tiles && behind < len;
        qa = k0;
        qb = sink && !cut ? len : behind;
        if (chunk >= 0) {
            qa = max(behind, chunk * s.chunk);
            qb = min(len, (chunk + 1) * s.chunk);
            return cut && qa < qb;
        }
        return true;
    }
    // The sum of key j's row, a sink (dk, then dv).
    __device__ __forceinline__ float *sum(const AttnProblem &p, const SinkPlan &s, int j) const {
        return (chunk >= 0 ? s.parts : s.base) + (((slot * p.Hk + hk) * s.tiles + jt) * s.rows + (j - k0)) * 2 * p.d;
    }
};

// The sinks' rows: what their window gave and the chunks, in order.  A block a key tile of a place and head.
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_sink_sum_kernel(const AttnProblem p, const SinkPlan s) {
    wait_for_last();       // (blocks without a row too: what follows in the stream waits for this kernel alone)
    int64_t k = blockIdx.x, n, lo;
    int first, len;
    const int jt = (int)(k % s.tiles);
    k /= s.tiles;
    const int hk = (int)(k % p.Hk);
    const int64_t place = k / p.Hk;
    if (!find_place(p, s, (int)place, false, n, first, lo, len)) return;
    const int k0 = jt * s.tile, rows = min(s.rows, min(p.sinks, len) - k0);
    const int behind = min(len, min(k0 + s.tile - 1, kNoWindow - 1) + p.window);
    if (rows <= 0 || behind >= len) return;
    const int64_t slot0 = p.seqs.cu ? lo / s.chunk + place : n * ((p.seqs.T + s.chunk - 1) / s.chunk);
    const int c0 = behind / s.chunk, c1 = (len + s.chunk - 1) / s.chunk;
    const int64_t tile = ((int64_t)hk * s.tiles + jt) * s.rows * 2 * D, step = (int64_t)p.Hk * s.tiles * s.rows * 2 * D;
    for (int x = threadIdx.x; x < rows * 2 * D / 4; x += 256) {
        float4 sum = load4(s.base + place * step + tile + 4 * x);
#pragma unroll 4
        for (int c = c0; c < c1; ++c) {
            const float4 y = load4(s.parts + (slot0 + c) * step + tile + 4 * x);
            sum.x += y.x; sum.y += y.y; sum.z += y.z; sum.w += y.w;
        }
        const int row = 4 * x / (2 * D), at = 4 * x % (2 * D);
        const int64_t r = lo + k0 + row;
        store4(at < D ? static_cast<T *>(p.dk) + r * p.dks + hk * D + at : static_cast<T *>(p.dv) + r * p.dvs + hk * D + at - D, sum);
    }
}
template <int D, typename T>
int launch_sink_sum(const AttnProblem &p, const SinkPlan &s, cudaStream_t stream) {
    if (s.tiles == 0) return kOk;
    return launch_after(attn_sink_sum_kernel<D, T>, (unsigned)(s.places * p.Hk * s.tiles), 256, 0, stream, p, s);
}
#endif

}  // namespace attn
}  // namespace dr
