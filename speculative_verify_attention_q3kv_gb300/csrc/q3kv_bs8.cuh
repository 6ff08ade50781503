// Verify attention over the block-scaled 8-bit cache: what both legs and the merge share.
//
// Work is cut into tiles of 128 positions of one (slot, row chunk, kv head) pair.  All tiles of a call,
// pair after pair, are shared out evenly: of G = min(CTAs, tiles), CTA i takes tiles [i n / G, (i + 1) n / G), one at least.  A pair inside one
// CTA's share goes straight to the output; of a pair that is cut, each CTA writes a partial (unnormalised
// output, maximum, sum), of which it has at most two: the pair its share begins inside, and the pair it ends
// inside.  So the workspace depends on the GPU alone, a ragged batch keeps every SM busy to the last tile, and
// the merge finds a pair's partials from the same arithmetic.
#pragma once

#include "q3kv_internal.h"

namespace q3kv {

constexpr int kBs8Tile = 128;
constexpr int kBs8Rows = 64;                 // query rows per chunk at most: 8 tokens of 8 heads
constexpr size_t kBs8PartFloats = (size_t)kBs8Rows * (kHeadDim + 2);     // per partial: outputs, then (maximum, sum) per row

struct Bs8Args {
    const uint8_t* pool;
    const int32_t* page_table;
    int32_t max_pages_per_slot;
    const int32_t* ctx_len;
    const int32_t* n_q;
    const int32_t* q_offsets;
    int32_t num_slots;
    int64_t max_ctx_len;
    int32_t max_n_q;
    int32_t num_layers;
    int32_t num_kv_heads;
    int32_t num_pages;
    int32_t layer;
    const void* q;
    void* out;
    int32_t dtype;               // of q and out
    int32_t rows;                // query rows per chunk
    int32_t ctas;                // G at most
    int32_t narrow;              // tiles x CTAs of the whole call fit 32 bits
    float* partials;             // [G][2][kBs8PartFloats]
    int32_t* status;
};

cudaError_t launch_bs8_fma(const Bs8Args& a, cudaStream_t stream);
cudaError_t launch_bs8_mma(const Bs8Args& a, cudaStream_t stream);
int bs8_mma_rows(int dtype, int max_n_q);                 // the tensor-core leg's chunk

// Lengths of one slot; tiles and chunks are 0 for a slot with nothing to do or with lengths the call does not allow.
struct Bs8Slot {
    int L, T, q0, tiles, chunks;             // q0: row of its first query token
    __device__ __forceinline__ int pairs(int heads) const { return chunks * heads; }
};

__device__ __forceinline__ Bs8Slot bs8_slot(const Bs8Args& a, int b, bool* bad) {
    Bs8Slot s{a.ctx_len[b], a.n_q[b], a.q_offsets[b], 0, 0};      // three loads at once
    const bool ok = (s.T > 0) & (s.T <= a.max_n_q) & (s.T <= s.L) & (s.L <= a.max_ctx_len) & (s.q0 >= 0) &
                    (s.L <= (int64_t)a.max_pages_per_slot * kPageSize);
    if (ok) {
        s.tiles = (s.L + kBs8Tile - 1) / kBs8Tile;
        s.chunks = (kGroup * s.T + a.rows - 1) / a.rows;
    } else if (bad && s.T != 0) {
        *bad = true;
    }
    return s;
}

// All of a call's tiles are counted in type N: 32 bits where the host has seen that tiles x CTAs fit (a fifth of the
// 64-bit steps' time), 64 otherwise.
__device__ __forceinline__ uint32_t bs8_warp_sum(uint32_t v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t bs8_warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <typename N>
__device__ __forceinline__ N bs8_total(const Bs8Slot& s, int heads) { return (N)s.tiles * (N)(s.chunks * heads); }

// Tiles of slots [0, b) by a warp; every lane gets it.
template <typename N>
__device__ __forceinline__ N bs8_tiles_before(const Bs8Args& a, int b, bool* bad) {
    N n = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) n += bs8_total<N>(bs8_slot(a, i, bad), a.num_kv_heads);
    return bs8_warp_sum(n);
}

// CTAs that have a share of n tiles; first tile of CTA i's share, and the CTA that owns tile t.
template <typename N>
__device__ __forceinline__ N bs8_ctas(const Bs8Args& a, N n) { return min((N)a.ctas, n); }
template <typename N>
__device__ __forceinline__ N bs8_begin(N i, N n, N G) { return i * n / G; }
template <typename N>
__device__ __forceinline__ int bs8_cta_of(N t, N n, N G) { return (int)(((t + 1) * G - 1) / n); }

// One CTA's share as a sequence of segments, each within one pair.
struct Bs8Share {
    int64_t left;                // tiles of the share behind the current segment
    Bs8Slot s;
    int slot, pair;              // pair = chunk * kv heads + head
    int tile, tiles;             // first tile of the segment and how many
    __device__ __forceinline__ int chunk(int heads) const { return pair / heads; }
    __device__ __forceinline__ int head(int heads) const { return pair % heads; }
    __device__ __forceinline__ bool whole() const { return tile == 0 && tiles == s.tiles; }
    // partial of a cut pair: 0 if the share begins inside the pair, 1 if at its beginning
    __device__ __forceinline__ int part() const { return tile == 0 ? 1 : 0; }
    // to the next segment; false at the end of the share
    __device__ __forceinline__ bool next(const Bs8Args& a) {
        if (left <= 0) return false;
        if (++pair >= s.pairs(a.num_kv_heads)) {
            pair = 0;
            do {
                s = bs8_slot(a, ++slot, nullptr);
            } while (s.tiles == 0);
        }
        tile = 0;
        tiles = (int)min((int64_t)s.tiles, left);
        left -= tiles;
        return true;
    }
};

// By one warp: the first segment of CTA i; tiles = 0 if its share is empty.
template <typename N>
__device__ __forceinline__ Bs8Share bs8_share_in(const Bs8Args& a, int i, bool* bad) {
    Bs8Share w{};
    const int lane = threadIdx.x & 31, heads = a.num_kv_heads;
    Bs8Slot s = lane < a.num_slots ? bs8_slot(a, lane, bad) : Bs8Slot{0, 0, 0, 0, 0};
    N n = bs8_total<N>(s, heads);
    for (int b = lane + 32; b < a.num_slots; b += 32) n += bs8_total<N>(bs8_slot(a, b, bad), heads);
    n = bs8_warp_sum(n);
    const N G = bs8_ctas(a, n);
    if ((N)i >= G) return w;
    const N begin = bs8_begin<N>(i, n, G), end = bs8_begin<N>(i + 1, n, G);
    N before = 0;
    for (int b0 = 0;; b0 += 32) {                                // ends: begin < n
        if (b0 > 0) s = b0 + lane < a.num_slots ? bs8_slot(a, b0 + lane, nullptr) : Bs8Slot{0, 0, 0, 0, 0};
        N upto = bs8_total<N>(s, heads);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const N v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + upto > begin);
        if (past) {
            const int l = __ffs(past) - 1;
            w.slot = b0 + l;
            w.s.L = __shfl_sync(0xffffffffu, s.L, l);
            w.s.T = __shfl_sync(0xffffffffu, s.T, l);
            w.s.q0 = __shfl_sync(0xffffffffu, s.q0, l);
            w.s.tiles = __shfl_sync(0xffffffffu, s.tiles, l);
            w.s.chunks = __shfl_sync(0xffffffffu, s.chunks, l);
            const N in = begin - (before + __shfl_sync(0xffffffffu, upto, l) - bs8_total<N>(w.s, heads));
            w.pair = (int)(in / (N)w.s.tiles);
            w.tile = (int)(in - (N)w.pair * (N)w.s.tiles);
            w.tiles = (int)min((N)(w.s.tiles - w.tile), end - begin);
            w.left = (int64_t)(end - begin) - w.tiles;
            return w;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
}
__device__ __forceinline__ Bs8Share bs8_share(const Bs8Args& a, int i, bool* bad) {
    return a.narrow ? bs8_share_in<uint32_t>(a, i, bad) : bs8_share_in<uint64_t>(a, i, bad);
}

}  // namespace q3kv
