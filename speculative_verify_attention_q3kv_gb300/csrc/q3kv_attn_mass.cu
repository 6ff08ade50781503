// Attention mass: the weight every cached position received from the step's
// queries, accumulated per kv head.
//
//   mass[j] = decay old[j] + sum over visible rows r of e^(q_r . k_hat_j / 16 - lse_r)
//
// With the rows' softmax statistic given, every position is independent of the
// others: one pass over the K records, no maxima, nothing to merge, and the bits of a
// position do not depend on how the work is cut.
//
// Precision.  A weight has the absolute error of its score as a relative one, so the
// scores are as good as float32's: queries as fp16 hi + lo pairs after a power of two for the (slot, kv
// head) pair (22 bits of every value, or 2^-27 of the pair's largest: see load_queries), keys exact.
// The 3-bit codec's value (c - 3.5) s needs 14 bits; instead of splitting it too,
// the tensor cores contract the codes, c - 3.5 exact in fp16, and each 32-dim
// block's sum goes to its own accumulator, which the epilogue multiplies by the
// block's scale in float32: two products per contraction instead of the four a
// split K_hat would need, and no bound on the scales.  E4M3 values are exact
// in fp16 (one accumulator per 64 dims, scale 1); turbo5k centroids are fp16 hi + lo
// pairs (four products, scales per 128 dims).
//
// Contraction (tcgen05, M = 128 positions, N = query rows padded to 16, at most
// 64 at a time): D_b[p][r] = sum over dims d of block b of code[p][d] (q_hi + q_lo)[r][d];
// A = codes in TMEM (lane = position), B = queries in shared memory (K-major).  A
// tile's 256 dims are four parts of 64 dims; a part's accumulators (128 columns for
// the 3-bit cache at 64 rows) form one slot of a ring, so the epilogue of a part overlaps
// the products of the next ones.
//
// Warp roles (24 warps; registers are moved between the roles with setmaxnreg):
//   E   warps 0-7    epilogue: thread = position (lane quarter warp & 3), all rows of the
//                    pass; the two warps of a lane quarter take every other tile.  Score
//                    sums start at -lse in log2 units, weights 2^s, rows summed in the
//                    thread.  Before a segment they rotate and split its queries.
//   D   warps 8-15   thread = position: its staged record converted into TMEM, one warp of
//                    a lane quarter for the even parts and one for the odd ones
//   M   warps 16-19  one thread each issues the products of one part: an issuing thread
//                    starts a K = 16 MMA about every 45 cycles, so four issue
//   P   warps 20-23  copy the records of the tiles ahead into shared memory, one stage per
//                    tile (one bulk copy; 16-byte cp.async where the stage is padded)
// TMEM (512 columns): one or two operand buffers (128 columns each, turbo5k 256) | ring of
// accumulator slots (see `double_buffered` and `acc_slots`).
//
// Work: the tiles of all (slot, kv head) pairs in one sequence, a share of about equal
// size per CTA (one per SM), whatever the slots' lengths, within one pair where the CTAs
// reach (see whole_shares); a CTA rotates and splits the queries of a pair itself when it
// enters it.
//
// Bound: not memory.  655,360 positions x 8 tokens x 2 kv heads take 100 us, 1,570 GB/s of K
// records and masses (the bytes alone: 23 us; the tensor pipe is 32 % active, the schedulers 69 %,
// a third of that in waits).  A tile of 64 rows takes about 2,800 cycles a CTA: its epilogue
// multiplies 128 x 64 x 8 accumulators by their scales and takes 8,192 exponentials in sixteen round
// trips to TMEM, with which two warps a lane quarter were busy 5,300 of 5,800 cycles each in a build of
// 104.5 us, and the ring holds three parts.  The time of this form moves by 5 % and more with the
// compiler's spills (4 bytes in this build, 20 to 36 in builds of 104 to 110 us) and with code that
// it does not run.  Up to 48 rows a group's accumulators come in one trip (6 tokens 92 us), up to
// 32 a part's (4 tokens 74 us, 1 token 65 us, where the conversion of the records decides, about
// 2,000 cycles a tile).  More warps, one event per accumulator, 64 columns a trip or passes of 32 rows were
// slower (114 to 160 us).  Short calls (32,768 positions x 6 tokens 12.3 us) wait 4,300 cycles for
// their share and 3,000 to 6,000 for the queries before the first tile.
//
// Every mbarrier wait is bounded; on a timeout the CTA sets Q3KV_STATUS_TIMEOUT, stops
// issuing, waits (bounded) for its MMAs in flight, frees its TMEM and returns.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "q3kv_common.cuh"
#include "q3kv_internal.h"
#include "q3kv_tcgen05.cuh"

namespace q3kv {
namespace {

constexpr int kWarps = 24;
constexpr int kWarpD = 8, kWarpM = 16, kWarpP = 20;     // first warps of the roles
constexpr int kIssuers = kWarpP - kWarpM;
constexpr int kCopyThreads = 32 * (kWarps - kWarpP);
constexpr int kQueryThreads = 32 * (kWarpD + kIssuers);  // that meet when a segment's queries are in place
// registers: launched with 80 a thread, 61,440 in all; the split gives E more out of the others' share
constexpr int kRegsE = 144, kRegsD = 56, kRegsMP = 40;
static_assert(256 * (kRegsE + kRegsD + kRegsMP) <= kWarps * 32 * 80, "register split");
constexpr int kTurns = 2;                   // E warps of a lane quarter
constexpr int kThreads = kWarps * 32;
constexpr int kTileP = 128;                 // positions per tile
constexpr int kChunkRows = 64;              // query rows per pass over a tile
constexpr int kMaxChunks = kMaxRows / kChunkRows;
constexpr int kParts = 4;                   // parts of 64 dims
constexpr int kFreeBars = 48;               // consumption events: a multiple of kParts and of every slot count
constexpr int kDoneBars = 4;                // generations of a part's completion barrier

template <int FMT>
struct Mf {                                 // 3-bit cache
    static constexpr int kGroups = 2;       // accumulators (scale groups) of a part
    static constexpr int kOps = 1;          // fp16 operands per value
    static constexpr int kRecB = kRecordBytes;
    static constexpr int kStride = kRecordBytes;   // of a staged record in shared memory
    static constexpr int kStages = 5;              // staged tiles (with scales: more than the E warps' turns)
    static constexpr bool kPadded = false;         // staged record by record
    static constexpr bool kScales = true;
    static constexpr bool kRot = true;
};
template <>
struct Mf<kFmtFp8> {
    static constexpr int kGroups = 1;
    static constexpr int kOps = 1;
    static constexpr int kRecB = kFp8RecordBytes;
    static constexpr int kStride = kFp8RecordBytes + 16;   // 16-byte loads of 8 lanes hit 8 bank groups
    static constexpr int kStages = 2;
    static constexpr bool kPadded = true;
    static constexpr bool kScales = false;
    static constexpr bool kRot = false;
};
template <>
struct Mf<kFmtT5k> {
    static constexpr int kGroups = 1;
    static constexpr int kOps = 2;
    static constexpr int kRecB = kT5kKRecordBytes;
    static constexpr int kStride = kT5kKRecordBytes;
    static constexpr int kStages = 3;
    static constexpr bool kPadded = false;
    static constexpr bool kScales = true;
    static constexpr bool kRot = true;
};
// Query operand: core matrices (8 rows x 8 dims, 128 bytes) 144 bytes apart along K, so that the
// 16-byte stores of a warp that holds one row meet all banks (at 128 bytes they meet four)
constexpr uint32_t kLbo = 144, kSbo = 32 * kLbo;
constexpr uint32_t kPartCols = 32;          // TMEM columns of a part's operand (64 fp16 values)
constexpr uint32_t kTmemCols = 512;

constexpr int kMaxStages = 5;
constexpr int kAhead = 2;                   // tiles whose old masses are loaded ahead
constexpr uint32_t kQueryLimit = 0x6D800000u;   // 2^92: the rotation and the products with the scales stay in float32

// An epilogue group that skips tiles, and an issuer that is up to a tile ahead,
// must not mistake an older phase for the one they wait for (only its parity is
// tested): hence several generations of done and acc_free.
struct Bars {
    unsigned long long a_full[kParts];             // one operand buffer: a part is in TMEM (4 D warps)
    unsigned long long done[kParts][kDoneBars];    // products of a part in pass ph (1 commit), by ph % 4
    unsigned long long a_free[kParts];             // every chunk's products of a part (1 commit): operand read
    unsigned long long b_full[2][2];               // two buffers: [buffer] the even / odd parts are in TMEM (4 D warps)
    unsigned long long b_free[2][2];               // and their products are done (2 commits)
    unsigned long long acc_free[kFreeBars];        // accumulators of event c read (4 E warps), by c % 48
    unsigned long long drain[kIssuers];            // everything an issuer started is done (1 commit)
    unsigned long long r_full[kMaxStages];         // a tile's records landed (copy bytes, or every P thread)
    unsigned long long r_free[kMaxStages];         // and were read (8 D warps; with scales, 4 E warps)
};

// One segment: tiles [t0, t0 + n) of a (slot, kv head) pair; n = 0: no more work.
struct Segment {
    int slot, g, t0, n;
    int T, L, chunks, q_row;                 // q_row: the slot's first query row
    int buffers;                             // operand buffers in TMEM
    int tiles_done;                          // tiles of earlier segments (phases of the stages)
    int tiles_single, tiles_double;          // of those with one operand buffer (a_full, a_free) and with two
    int phases;                              // (tile, chunk) passes of earlier segments (phases of done)
};

// A CTA's way through its share [w, w1) of the tile sequence; base: where the slot's tiles begin.
struct Walk {
    long long w, w1, base;
    int slot, tiles_done, tiles_single, tiles_double, phases;
};

template <int FMT>
struct __align__(16) MassSmem {
    uint8_t q[kMaxChunks][2][kChunkRows / 8 * kSbo];   // [chunk][hi | lo], B operand
    uint8_t rec[Mf<FMT>::kStages][kTileP * Mf<FMT>::kStride];   // staged records
    float nlse[kMaxRows];                             // -lse in log2 units; -inf leaves a row out
    uint32_t q_most[kWarpD];                          // largest |q| of a warp's rows, as float bits (query_scale)
    float unscale;                                    // 2^-e of the queries' 2^e
    int2 q_flags[2];                                  // [segment % 2] a value is too large for the usual scale; one is large enough
    Bars bar;
    uint32_t tmem_base;
    int abort;
    Walk walk;
    Segment seg[2];
};

// Tiles of a slot's kv head; 0 for a slot with nothing to do.
__device__ __forceinline__ int tiles_of(const MassArgs& a, int T, int L, bool* bad) {
    if (T <= 0) return 0;
    if (T > a.max_n_q || T > L || L > a.max_ctx_len || L > (int64_t)a.max_pages_per_slot * kPageSize) {
        *bad = true;
        return 0;
    }
    return (L + kTileP - 1) / kTileP;
}
__device__ __forceinline__ int slot_tiles(const MassArgs& a, int b, bool* bad) { return tiles_of(a, a.n_q[b], a.ctx_len[b], bad); }

__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float two_to(int e) { return __int_as_float((127 + e) << 23); }
// two float32 fused multiply-adds in one instruction
__device__ __forceinline__ unsigned long long fma2(unsigned long long x, unsigned long long y, unsigned long long z) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

__device__ __forceinline__ unsigned long long add2(unsigned long long x, unsigned long long y) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

// With at most 32 query rows the accumulators leave TMEM for a second operand buffer, so
// the conversion of a tile overlaps the products of the one before it (655,360 positions, 2 kv
// heads: 74 -> 69 us with 1 token, 79 -> 76 us with 4; more rows need the columns for a
// deeper ring).  A turbo5k operand has two fp16 parts and no room for that.
template <int FMT>
__host__ __device__ constexpr bool double_buffered(int tokens) {
    return Mf<FMT>::kOps == 1 && kGroup * tokens <= 32;
}
// First accumulator column and slots of the ring.
template <int FMT>
__host__ __device__ constexpr uint32_t acc_col(int buffers) { return kParts * kPartCols * Mf<FMT>::kOps * buffers; }
template <int FMT>
__host__ __device__ constexpr int acc_slots(int buffers, int cols) {
    return buffers == 2 ? 256 / (Mf<FMT>::kGroups * cols) : 192 / cols;
}

// Shares that stay within one (slot, kv head) pair: the smallest d for which giving every
// pair ceil(tiles / d) CTAs takes no more than the grid.  A pair change drains the pipeline and
// prepares other queries, about two tiles' time, so they are taken if d is at most that much above an
// even share, once per pair that an even share meets (8 ragged slots x 2 heads x 1 token, 9
// tiles a CTA: 13.5 us, with even shares 16.0; 8 slots of 40,000 positions x 4 heads, 79 tiles for
// 66: 74.5 us, with even shares 66.4).  One warp, a lane per slot; false if even shares are better,
// with more than 32 slots, or with more pairs than CTAs.
template <int FMT>
__device__ inline bool whole_shares(const MassArgs& a, Segment& seg, bool* bad) {
    if (a.num_slots > 32) return false;
    const int lane = threadIdx.x & 31, G = gridDim.x, H = a.num_kv_heads;
    const bool slot = lane < a.num_slots;
    const int q_row = slot ? a.q_offsets[lane] : 0, T = slot ? a.n_q[lane] : 0, L = slot ? a.ctx_len[lane] : 0;
    const int tiles = tiles_of(a, T, L, bad);
    const int slots = __popc(__ballot_sync(0xffffffffu, tiles > 0)), per = G / H;   // CTAs per kv head
    if (slots > per || slots == 0) return slots == 0;
    // d = ceil(total / (per - slots)) fits, as ceil(x / d) <= x / d + 1; d below total / per does not
    const int total = __reduce_add_sync(0xffffffffu, tiles);
    int lo = (total + per - 1) / per - 1;                  // does not fit
    int hi = slots < per ? (total + (per - slots) - 1) / (per - slots) : __reduce_max_sync(0xffffffffu, tiles);
    if (hi > lo + 1 && __reduce_add_sync(0xffffffffu, (tiles + lo) / (lo + 1)) <= per) hi = lo + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__reduce_add_sync(0xffffffffu, (tiles + mid - 1) / mid) <= per) hi = mid;
        else lo = mid;
    }
    if (hi > (total + per - 1) / per + 2 + 2 * slots / per) return false;
    const int ctas = (tiles + hi - 1) / hi;                // per pair of this lane's slot
    int incl = ctas * H;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, incl > (int)blockIdx.x);
    if (hit && lane == __ffs(hit) - 1) {                   // the lane of this CTA's slot
        const int r = (int)blockIdx.x - (incl - ctas * H), g = r / ctas, i = r - g * ctas;
        const int t0 = (int)((long long)tiles * i / ctas), t1 = (int)((long long)tiles * (i + 1) / ctas);
        seg = Segment{lane, g, t0, t1 - t0, T, L, (kGroup * T + kChunkRows - 1) / kChunkRows, q_row,
                      double_buffered<FMT>(T) ? 2 : 1, 0, 0, 0, 0};
    }
    return true;                                           // (no tiles are left for the CTAs behind the last)
}

// The segment at the walk's position, for every role to read (one thread calls).
template <int FMT>
__device__ void next_segment(const MassArgs& a, MassSmem<FMT>& sm, int k) {
    Segment& s = sm.seg[k & 1];
    s.n = 0;
    Walk& wk = sm.walk;
    if (wk.w >= wk.w1) return;
    bool ignore = false;
    int tiles = slot_tiles(a, wk.slot, &ignore);
    while (tiles == 0 || wk.w >= wk.base + (long long)tiles * a.num_kv_heads) {   // the next slot with tiles
        wk.base += (long long)tiles * a.num_kv_heads;
        tiles = slot_tiles(a, ++wk.slot, &ignore);
    }
    const long long off = wk.w - wk.base;
    s.slot = wk.slot;
    s.g = off <= UINT32_MAX ? (int)((uint32_t)off / (uint32_t)tiles) : (int)(off / tiles);
    s.t0 = (int)(off - (long long)s.g * tiles);
    s.n = (int)min((long long)(tiles - s.t0), wk.w1 - wk.w);
    s.T = a.n_q[wk.slot];
    s.L = a.ctx_len[wk.slot];
    s.q_row = a.q_offsets[wk.slot];
    s.chunks = (kGroup * s.T + kChunkRows - 1) / kChunkRows;
    s.buffers = double_buffered<FMT>(s.T) ? 2 : 1;
    s.tiles_done = wk.tiles_done;
    s.tiles_single = wk.tiles_single;
    s.tiles_double = wk.tiles_double;
    s.phases = wk.phases;
    wk.w += s.n;
    wk.tiles_done += s.n;
    (s.buffers == 2 ? wk.tiles_double : wk.tiles_single) += s.n;
    wk.phases += s.n * s.chunks;
}

// Accumulator columns of a group: the query rows of a pass, rounded up.
__device__ __forceinline__ int acc_cols(const Segment& s) {
    const int rows = kGroup * s.T;
    return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 48 ? 48 : kChunkRows));
}
// Query rows of pass j as the products read them.
__device__ __forceinline__ int mma_rows(const Segment& s, int j) {
    const int cols = acc_cols(s), rows = min(kChunkRows, kGroup * s.T - kChunkRows * j);
    return cols < kChunkRows ? cols : (rows + 31) & ~31;
}

// This CTA's share of the sequence of tiles, and its first segment.  One warp.
template <int FMT>
__device__ void share_of(const MassArgs& a, MassSmem<FMT>& sm) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (lane == 0) {
        sm.seg[0].n = 0;
        sm.walk = Walk{0, 0, 0, 0, 0, 0, 0, 0};
    }
    __syncwarp();
    if (!whole_shares<FMT>(a, sm.seg[0], &bad)) {
        // even shares [w0, w1), whatever the slots' lengths
        long long w0, w1, base = 0, total = 0;
        for (int b0 = 0; b0 < a.num_slots; b0 += 32)
            total += __reduce_add_sync(0xffffffffu, b0 + lane < a.num_slots ? slot_tiles(a, b0 + lane, &bad) : 0);
        total *= a.num_kv_heads;
        w0 = total * blockIdx.x / gridDim.x;
        w1 = total * (blockIdx.x + 1) / gridDim.x;
        int slot = a.num_slots;
        bool ignore = false;
        for (int b0 = 0; b0 < a.num_slots && w0 < w1; b0 += 32) {
            const long long mine = b0 + lane < a.num_slots ? (long long)slot_tiles(a, b0 + lane, &ignore) * a.num_kv_heads : 0;
            long long incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + incl > w0);
            if (hit) {
                const int l = __ffs(hit) - 1;
                slot = b0 + l;
                base += __shfl_sync(0xffffffffu, incl - mine, l);
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            sm.walk = Walk{w0, w1, base, slot, 0, 0, 0, 0};
            next_segment<FMT>(a, sm, 0);
        }
    }
    if (blockIdx.x == 0 && bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
}

// The 8 or 4 values of a 16-byte word.
__device__ __forceinline__ void unpack(const uint4& u, float* y, const __nv_bfloat16*) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(w[i] << 16);
        y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& u, float* y, const float*) {
    y[0] = __uint_as_float(u.x); y[1] = __uint_as_float(u.y); y[2] = __uint_as_float(u.z); y[3] = __uint_as_float(u.w);
}

// H y (unnormalised) of four rows of a warp, eight lanes a row.  Lane l begins with dims
// 32 (l % 8) .. of its row: dim bits 0 to 4 are register bits.  Bits 5, 6 and 7 are exchanged into
// register bits 3, 4 and 3, half of the registers by shuffle each (a butterfly across lanes needs all
// of them), so that y[8 c + i] comes out as dim 8 (l % 8 + 8 (c / 2) + 16 (c % 2)) + i.
__device__ __forceinline__ void rotate_four_rows(float (&y)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if ((i & h) == 0) {
                const float u = y[i], v = y[i + h];
                y[i] = u + v;
                y[i + h] = u - v;
            }
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        const int h = step == 1 ? 16 : 8, m = 1 << step;
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if ((i & h) == 0) {
                const float got = __shfl_xor_sync(0xffffffffu, upper ? y[i] : y[i + h], m);
                const float u = upper ? got : y[i], v = upper ? y[i + h] : got;
                y[i] = u + v;
                y[i + h] = u - v;
            }
    }
}

// Where a lane's dims 8 c .. 8 c + 7 (as rotate_four_rows leaves them) of row rr of a pass lie in the operand.
template <int FMT>
__device__ __forceinline__ uint32_t query_offset(int rr, int c) {
    const int l = threadIdx.x & 7;
    const uint32_t core = Mf<FMT>::kRot ? l + 8 * (c >> 1) + 16 * (c & 1) : 4 * l + c;
    return (uint32_t)(rr >> 3) * kSbo + core * kLbo + (uint32_t)(rr & 7) * 16u;
}

// Queries of the segment's pair: H, then 1/16 (H) 1/16 (softmax) log2(e) and 2^e, split
// into fp16 hi / lo, and -lse in log2 units; padding rows are zeros.  The E warps take four rows
// each, the next ones' loads in flight, while the D warps convert the first records.  (A row per
// warp and step took 40 shuffles a row, 8,000 cycles for 64 rows.)
//
// The power of two 2^e: hi + lo hold 22 bits of a value, but lo no finer than 2^-25.  The usual e = 8 serves a
// pair whose largest scaled value lies in [4, 2^15): rotated queries (with the rotation's 1/16) of 0.17 to
// 1,419 at most, for which 2^-25 is 2^-27 of the largest or less.  For others the E warps prepare the pair
// again with an e of its own (query_scale), 1 us of a call with one token and 4 with 8.  The epilogue takes
// 2^e out again with the position's scales; a power per row would cost it a multiply-add per row and
// position, and to look at all rows before the first split took 0.9 us of every call.
constexpr int kUsualExp = 8;
template <typename TIn, int FMT>
__device__ __forceinline__ void load_queries(const MassArgs& a, const Segment& s, MassSmem<FMT>& sm, int exp2q, bool again, int2& flags) {
    constexpr int kVecs = 2 * (int)sizeof(TIn);              // 16-byte loads of a lane's 32 dims
    constexpr int kPer = 32 / kVecs;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = kGroup * s.T, rows = s.chunks * kChunkRows;
    const int64_t Hq = a.num_kv_heads * kGroup;
    auto row_of = [&](int r) { return ((int64_t)s.q_row + r / kGroup) * Hq + s.g * kGroup + r % kGroup; };
    auto load = [&](uint4 (&raw)[kVecs], int r) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const TIn*>(a.q) + row_of(r) * kHeadDim + 32 * (lane & 7));
#pragma unroll
        for (int v = 0; v < kVecs; ++v) raw[v] = r < R ? p[v] : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 next[kVecs];
    load(next, 4 * warp + (lane >> 3));
    bool out = false;                                        // a statistic that is not finite
    if ((int)threadIdx.x < rows && !again) {
        const int r = threadIdx.x;
        const float l = r < R ? a.lse[row_of(r)] : CUDART_INF_F;
        const bool finite = fabsf(l) < CUDART_INF_F;
        out = r < R && !finite;
        sm.nlse[r] = finite ? -1.4426950408889634f * l : -CUDART_INF_F;
    }
    __syncwarp();
    const float scale = (Mf<FMT>::kRot ? 1.4426950408889634f / 256.0f : 1.4426950408889634f / 16.0f) * two_to(exp2q);
    __half2 most = __half2half2(__ushort_as_half((unsigned short)0));
#pragma unroll 1
    for (int r0 = 4 * warp; r0 < rows; r0 += 4 * kWarpD) {
        const int r = r0 + (lane >> 3), chunk = r0 / kChunkRows, rr = r % kChunkRows;
        float y[32];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) unpack(next[v], y + kPer * v, static_cast<const TIn*>(nullptr));
        load(next, r + 4 * kWarpD);
        if (r0 % kChunkRows >= mma_rows(s, chunk)) continue;
        if (Mf<FMT>::kRot) rotate_four_rows(y);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t hw[4], lw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x0 = y[8 * c + 2 * i] * scale, x1 = y[8 * c + 2 * i + 1] * scale;
                const __half2 h2 = __floats2half2_rn(x0, x1);
                const float2 hf = __half22float2(h2);
                most = __hmax2_nan(most, __habs2(h2));
                hw[i] = as_u32(h2);
                lw[i] = as_u32(__floats2half2_rn(x0 - hf.x, x1 - hf.y));
            }
            const uint32_t off = query_offset<FMT>(rr, c);
            *reinterpret_cast<uint4*>(&sm.q[chunk][0][off]) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
            *reinterpret_cast<uint4*>(&sm.q[chunk][1][off]) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
    }
    const uint32_t m = as_u32(most), top = max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
    if ((top >= 0x7800u || out) && !again) flags.x = 1;      // 2^15, and whatever is not finite
    if (top >= 0x4400u && !again) flags.y = 1;               // 4
    fence_proxy_async();
}

// Largest magnitude of 16 bytes, as float bits.
__device__ __forceinline__ uint32_t largest(const uint4& u, const __nv_bfloat16*) {
    const uint32_t lo = max(max(u.x << 16 & 0x7FFFFFFFu, u.y << 16 & 0x7FFFFFFFu), max(u.z << 16 & 0x7FFFFFFFu, u.w << 16 & 0x7FFFFFFFu));
    return max(lo, max(max(u.x & 0x7FFF0000u, u.y & 0x7FFF0000u), max(u.z & 0x7FFF0000u, u.w & 0x7FFF0000u)));
}
__device__ __forceinline__ uint32_t largest(const uint4& u, const float*) {
    return max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu));
}

// Which rows of the pair take part in its second preparation, and the e with which their rotated and scaled
// queries stay below 2^15.  A row whose statistic is not finite, or with a query from 2^92 on (an infinity or
// a NaN among them), is left out: its start becomes -inf, and clear_rows makes its operand zeros, as a NaN
// there would reach the sum of every position.  The e comes from the largest |q|, of rows without a
// finite statistic too: the rotation makes a value at most 256 times larger, and leaves the row's largest no
// smaller.  Where the usual e is known to serve by that, it is taken: the other rows' bits are those of a call
// without the ones left out.  The E warps, a row per warp and step.
template <typename TIn, int FMT>
__device__ __forceinline__ int query_scale(const MassArgs& a, const Segment& s, MassSmem<FMT>& sm) {
    constexpr int kVecs = (int)sizeof(TIn) / 2;              // 16-byte loads of a lane's part of a row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t Hq = a.num_kv_heads * kGroup;
    uint32_t most = 0u;
#pragma unroll 1
    for (int r = warp; r < kGroup * s.T; r += kWarpD) {
        const int64_t row = ((int64_t)s.q_row + r / kGroup) * Hq + s.g * kGroup + r % kGroup;
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const TIn*>(a.q) + row * kHeadDim) + lane;
        uint32_t m = 0u;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) m = max(m, largest(p[32 * v], static_cast<const TIn*>(nullptr)));
        m = __reduce_max_sync(0xffffffffu, m);
        if (m < kQueryLimit) most = max(most, m);
        if ((m >= kQueryLimit || !(fabsf(a.lse[row]) < CUDART_INF_F)) && lane == 0) {
            sm.nlse[r] = -CUDART_INF_F;
            if (a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
        }
    }
    if (lane == 0) sm.q_most[warp] = most;
    named_sync(2, 32 * kWarpD);
#pragma unroll
    for (int w = 0; w < kWarpD; ++w) most = max(most, sm.q_most[w]);
    const float bound = __uint_as_float(most) * (Mf<FMT>::kRot ? 1.4426950408889634f : 1.4426950408889634f / 16.0f);
    const float least = Mf<FMT>::kRot ? bound / 256.0f : bound;
    if (most == 0u || (bound * two_to(kUsualExp) < 32768.0f && least * two_to(kUsualExp) >= 4.0f)) return kUsualExp;
    return min(100, 14 - ((int)(__float_as_uint(bound) >> 23) - 127));    // the block scales times 2^-100 are normal
}

// Zeros in the operand for the rows that query_scale left out, by the lanes that wrote them in load_queries.
template <int FMT>
__device__ __forceinline__ void clear_rows(const Segment& s, MassSmem<FMT>& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int r = 4 * warp + (lane >> 3); r < kGroup * s.T; r += 4 * kWarpD) {
        if (sm.nlse[r] > -CUDART_INF_F) continue;
#pragma unroll 1
        for (int c = 0; c < 8; ++c)
            *reinterpret_cast<uint4*>(&sm.q[r / kChunkRows][c >> 2][query_offset<FMT>(r % kChunkRows, c & 3)]) = make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
    fence_proxy_async();
}

__device__ __forceinline__ int32_t page_of(const MassArgs& a, const Segment& s, int pos0) {
    const int32_t page = a.page_table[(int64_t)s.slot * a.max_pages_per_slot + pos0 / kPageSize];
    return (page >= 0 && page < a.num_pages) ? page : -1;
}

template <int FMT>
__device__ __forceinline__ const uint8_t* k_record(const MassArgs& a, const Segment& s, int32_t page, int pos) {
    return a.pool + (FMT == kFmtT5k ? t5k_offset(a.num_layers, a.num_kv_heads, page, a.layer, s.g, 0, pos % kPageSize)
                                    : record_offset(a.num_layers, a.num_kv_heads, page, a.layer, s.g, 0, pos % kPageSize,
                                                    Mf<FMT>::kRecB));
}

// Words of a part (64 dims) of a record.
template <int FMT>
struct Words {
    static constexpr int kN = FMT == kFmtFp8 ? 16 : (FMT == kFmtT5k ? 10 : 6);
};

// Part q of a staged record.
template <int FMT>
__device__ __forceinline__ void read_part(const uint8_t* rec, int q, uint32_t (&w)[Words<FMT>::kN]) {
    if constexpr (FMT == kFmtFp8) {
        const uint4* p = reinterpret_cast<const uint4*>(rec) + 4 * q;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint4 u = p[m];
            w[4 * m] = u.x; w[4 * m + 1] = u.y; w[4 * m + 2] = u.z; w[4 * m + 3] = u.w;
        }
    } else if constexpr (FMT == kFmtT5k) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(rec);
#pragma unroll
        for (int m = 0; m < 8; ++m) w[m] = p[8 * q + m];
#pragma unroll
        for (int m = 0; m < 2; ++m) w[8 + m] = p[32 + 2 * q + m];
    } else {
        const uint2* p = reinterpret_cast<const uint2*>(rec) + 3 * q;      // 24 bytes
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            const uint2 u = p[m];
            w[2 * m] = u.x; w[2 * m + 1] = u.y;
        }
    }
}

// Copies the records of tile i of the segment into its stage.  A tile's 128 records
// are contiguous: one bulk copy by one thread; a padded stage takes 16 bytes a
// thread and step (all P warps).  A page out of range completes the phase without
// data: its scores are unused.
template <int FMT>
__device__ __forceinline__ void stage_tile(const MassArgs& a, const Segment& s, MassSmem<FMT>& sm, int i, int counter) {
    const int t = threadIdx.x - 32 * kWarpP;
    const int st = counter % Mf<FMT>::kStages;
    const int pos0 = (s.t0 + i) * kTileP;
    const int32_t page = page_of(a, s, pos0);
    if (page < 0 && t == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
    if (Mf<FMT>::kPadded) {
        if (page >= 0) {
            const uint8_t* src = k_record<FMT>(a, s, page, pos0);
            constexpr int kVecs = Mf<FMT>::kRecB / 16;
#pragma unroll 4
            for (int k = 0; k < kTileP * kVecs / kCopyThreads; ++k) {
                const int v = kCopyThreads * k + t;
                cp_async16(sm.rec[st] + (v / kVecs) * Mf<FMT>::kStride + (v % kVecs) * 16, src + (size_t)v * 16);
            }
        }
        cp_async_mbar_arrive(&sm.bar.r_full[st]);
    } else if (t == 0) {
        if (page >= 0) {
            fence_proxy_async();
            mbar_arrive_expect_tx(&sm.bar.r_full[st], (uint32_t)(kTileP * Mf<FMT>::kRecB));
            bulk_g2s(sm.rec[st], k_record<FMT>(a, s, page, pos0), (uint32_t)(kTileP * Mf<FMT>::kRecB), &sm.bar.r_full[st]);
        } else {
            mbar_arrive(&sm.bar.r_full[st]);
        }
    }
}

// Half a part (32 dims) of this thread's position as fp16 pairs in K order, to the
// TMEM columns at col (turbo5k: hi there, lo one operand further).
template <int FMT>
__device__ __forceinline__ void store_half(const uint32_t (&w)[Words<FMT>::kN], int b, float cent, uint32_t col) {
    uint32_t h[16];
    if constexpr (FMT == kFmtFp8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) e4m3x4_to_f16(w[8 * b + k], h[2 * k], h[2 * k + 1]);
        tmem_st16(col, h);
    } else if constexpr (FMT == kFmtT5k) {
        // lane l holds centroid l: a code's value by shuffle, split into fp16 hi / lo
        uint32_t lo[16];
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            const uint32_t nw = w[4 * b + m / 4], top = w[8 + b];
            const uint32_t c0 = ((nw >> (8 * (m % 4))) & 0xFu) | (((top >> (2 * m)) & 1u) << 4);
            const uint32_t c1 = ((nw >> (8 * (m % 4) + 4)) & 0xFu) | (((top >> (2 * m + 1)) & 1u) << 4);
            const float v0 = __shfl_sync(0xffffffffu, cent, (int)c0);
            const float v1 = __shfl_sync(0xffffffffu, cent, (int)c1);
            const __half2 h2 = __floats2half2_rn(v0, v1);
            const float2 hf = __half22float2(h2);
            h[m] = as_u32(h2);
            lo[m] = as_u32(__floats2half2_rn(v0 - hf.x, v1 - hf.y));
        }
        tmem_st16(col, h);
        tmem_st16(col + kParts * kPartCols, lo);
    } else {
        // A code pair at bits (o, o + 16) of a word, under the exponent of 2^(10 - o), is
        // 2^(10 - o) + c: for o = 3 and 6 an and-or and one exact subtraction give c - 3.5.
        // The fields at 0, 9 and 12 come to 3, 3 and 6 with one shift for the first and one
        // for the other two.
        const __half2 m3 = __half2half2(__ushort_as_half((unsigned short)0xD81Cu));   // -131.5
        const __half2 m6 = __half2half2(__ushort_as_half((unsigned short)0xCCE0u));   // -19.5
        const __half2 m12 = __half2half2(__ushort_as_half((unsigned short)0xCA00u));  // -12
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const uint32_t u = w[3 * b + k], l = u << 3, r = u >> 6;
            h[5 * k] = as_u32(__hadd2(as_h2((l & 0x00380038u) | 0x58005800u), m3));
            h[5 * k + 1] = as_u32(__hadd2(as_h2((u & 0x00380038u) | 0x58005800u), m3));
            h[5 * k + 2] = as_u32(__hadd2(as_h2((u & 0x01C001C0u) | 0x4C004C00u), m6));
            h[5 * k + 3] = as_u32(__hadd2(as_h2((r & 0x00380038u) | 0x58005800u), m3));
            h[5 * k + 4] = as_u32(__hadd2(as_h2((r & 0x01C001C0u) | 0x4C004C00u), m6));
        }
        // (8.5 + c) - 12, exact
        h[15] = as_u32(__hadd2(as_h2(code_pair_last(w[3 * b], w[3 * b + 1], w[3 * b + 2])), m12));
        tmem_st16(col, h);
    }
}

// What the epilogue of a segment needs besides the segment.
struct EpiState {
    uint32_t tmem_acc;           // first accumulator column, this warp's lanes
    volatile int* abort;
};

// Scale of group gi of a part, from the position's scale words.
template <int FMT>
__device__ __forceinline__ float part_scale(const uint4& sc, int part, int gi) {
    if (FMT == kFmtQ3) {
        const uint32_t word = part == 0 ? sc.x : (part == 1 ? sc.y : (part == 2 ? sc.z : sc.w));
        return __half2float(__ushort_as_half((unsigned short)(gi ? word >> 16 : word & 0xFFFFu)));
    }
    if (FMT == kFmtT5k) return __half2float(__ushort_as_half((unsigned short)(part >= 2 ? sc.x >> 16 : sc.x & 0xFFFFu)));
    return 1.0f;
}

// Epilogue of this warp's tiles of a segment; COLS accumulator columns per group
// (16, 32, 48 or 64 query rows of a pass).
template <int FMT, int COLS, int BUFFERS>
__device__ __forceinline__ bool epilogue(const MassArgs& a, const Segment& s, MassSmem<FMT>& sm, const EpiState& e, bool ok) {
    constexpr int G = Mf<FMT>::kGroups, ST = Mf<FMT>::kStages, SLOTS = acc_slots<FMT>(BUFFERS, COLS);
    constexpr int LD = COLS < 32 ? 16 : 32;                  // columns of one TMEM load
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int turn = warp >> 2;
    const int p = 32 * (warp & 3) + lane;
    const int Nctx = s.L - s.T, R = kGroup * s.T;
    Bars& bar = sm.bar;
    float* mass = a.mass + ((int64_t)s.slot * a.num_kv_heads + s.g) * a.mass_stride;
    // old masses and page checks of the next tiles, ahead of their use
    auto old_of = [&](int i) {
        const int pos = (s.t0 + i) * kTileP + p;
        return (i < s.n && a.decay > 0.0f && pos < Nctx) ? mass[pos] : 0.0f;
    };
    float old_q[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) old_q[k] = old_of(turn + k * kTurns);
    int32_t page_next = turn < s.n ? page_of(a, s, (s.t0 + turn) * kTileP) : -1;
#pragma unroll 1
    for (int i = turn; i < s.n; i += kTurns) {
        const float old = old_q[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) old_q[k] = old_q[k + 1];
        old_q[kAhead - 1] = old_of(i + kAhead * kTurns);
        const int pos0 = (s.t0 + i) * kTileP;
        const int pos = pos0 + p;
        const bool page_ok = page_next >= 0;
        if (i + kTurns < s.n) page_next = page_of(a, s, pos0 + kTurns * kTileP);
        uint4 sc = make_uint4(0u, 0u, 0u, 0u);
        if (Mf<FMT>::kScales) {
            // this position's scales from the staged record
            const int rc = s.tiles_done + i;
            ok = ok && mbar_wait_fast(&bar.r_full[rc % ST], (uint32_t)((rc / ST) & 1), e.abort);
            const uint8_t* rec = sm.rec[rc % ST] + p * Mf<FMT>::kStride;
            if (FMT == kFmtQ3) sc = *reinterpret_cast<const uint4*>(rec + 96);
            if (FMT == kFmtT5k) sc.x = *reinterpret_cast<const uint32_t*>(rec + 160);
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.r_free[rc % ST]);
        }
        unsigned long long sum0 = 0ull, sum1 = 0ull;         // pairs of zeros
        // 2^-e, read for every tile and through a warp's maximum, after which the compiler knows that it is uniform: held
        // in a register of the thread it made the 64-row form spill (8 tokens 110 us, so 100)
        const float unscale = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(sm.unscale)));
#pragma unroll 1
        for (int j = 0; j < s.chunks; ++j) {
            const int ph = s.phases + i * s.chunks + j;
            const int halves = COLS == 64 && R - kChunkRows * j <= 32 ? 1 : COLS / LD;   // loads of a group
            unsigned long long acc[COLS / 2];
#pragma unroll
            for (int k = 0; k < COLS / 4; ++k) {
                const float4 u = *reinterpret_cast<const float4*>(&sm.nlse[kChunkRows * j + 4 * k]);
                acc[2 * k] = pack2(u.x, u.y);
                acc[2 * k + 1] = pack2(u.z, u.w);
            }
#pragma unroll
            for (int part = 0; part < kParts; ++part) {
                const int c = kParts * ph + part;
                ok = ok && mbar_wait_fast(&bar.done[part][ph % kDoneBars], (uint32_t)((ph / kDoneBars) & 1), e.abort);
                __syncwarp();
                tc_fence_after();
                const uint32_t col = e.tmem_acc + (uint32_t)((c % SLOTS) * G * COLS);
                if (COLS <= 32) {
                    // the whole part in one round trip
                    float x[G][LD];
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        if (LD == 16) tmem_ld16(col + COLS * gi, x[gi]);
                        else tmem_ld32(col + COLS * gi, x[gi]);
                    }
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.acc_free[c % kFreeBars]);
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        const float scale = part_scale<FMT>(sc, part, gi) * unscale;
                        const unsigned long long s2 = pack2(scale, scale);
#pragma unroll
                        for (int k = 0; k < LD / 2; ++k) acc[k] = fma2(pack2(x[gi][2 * k], x[gi][2 * k + 1]), s2, acc[k]);
                    }
                } else if (COLS == 48) {
                    // a group in one round trip (655,360 positions x 6 tokens: 92 us, in the form for 64 rows 105)
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        const float scale = part_scale<FMT>(sc, part, gi) * unscale;
                        float x[32], z[16];
                        tmem_ld32(col + COLS * gi, x);
                        tmem_ld16(col + COLS * gi + 32, z);
                        tmem_ld_wait();
                        if (gi == G - 1) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&bar.acc_free[c % kFreeBars]);
                        }
#pragma unroll
                        for (int k = 0; k < COLS / 2; ++k) {
                            float a0, a1;
                            unpack2(acc[k], a0, a1);
                            const float x0 = k < 16 ? x[2 * k % 32] : z[(2 * k) % 16], x1 = k < 16 ? x[(2 * k + 1) % 32] : z[(2 * k + 1) % 16];
                            acc[k] = pack2(fmaf(x0, scale, a0), fmaf(x1, scale, a1));
                        }
                    }
                } else {
#pragma unroll
                    for (int gi = 0; gi < G; ++gi) {
                        const float scale = part_scale<FMT>(sc, part, gi) * unscale;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h < halves) {
                                float x[LD];
                                tmem_ld32(col + COLS * gi + 32 * h, x);
                                tmem_ld_wait();
                                if (gi == G - 1 && h == halves - 1) {
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) mbar_arrive(&bar.acc_free[c % kFreeBars]);
                                }
#pragma unroll
                                for (int k = 0; k < LD / 2; ++k) {
                                    // single multiply-adds here: 512 a tile spread over both FMA pipes, where
                                    // the paired form goes to one of them (8 tokens: 110 -> 106 us)
                                    float a0, a1;
                                    unpack2(acc[16 * h + k], a0, a1);
                                    acc[16 * h + k] = pack2(fmaf(x[2 * k], scale, a0), fmaf(x[2 * k + 1], scale, a1));
                                }
                            }
                    }
                }
            }
            // weights; padding rows start at -inf and weigh nothing.  Row r (token r / 8) sees
            // positions <= Nctx + r / 8.
            const int r_min = pos0 + kTileP - 1 > Nctx ? kGroup * (pos - Nctx) - kChunkRows * j : 0;
            if (pos0 + kTileP - 1 > Nctx) {
#pragma unroll
                for (int k = 0; k < COLS / 2; ++k) {
                    float x0, x1;
                    unpack2(acc[k], x0, x1);
                    if (2 * k < r_min) x0 = -CUDART_INF_F;
                    if (2 * k + 1 < r_min) x1 = -CUDART_INF_F;
                    acc[k] = pack2(x0, x1);
                }
            }
#pragma unroll
            for (int k = 0; k < COLS / 2; ++k) {
                float x0, x1;
                unpack2(acc[k], x0, x1);
                const unsigned long long w2 = pack2(fast_exp2(x0), fast_exp2(x1));
                if (k & 1) sum1 = add2(sum1, w2);
                else sum0 = add2(sum0, w2);
            }
        }
        float a0, a1;
        unpack2(add2(sum0, sum1), a0, a1);
        if (pos < s.L) mass[pos] = fmaf(a.decay, old, page_ok ? a0 + a1 : 0.0f);
    }
    return ok;
}

template <typename TIn, int FMT>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassArgs a) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    MassSmem<FMT>& sm = *reinterpret_cast<MassSmem<FMT>*>(smem_raw);
    Bars& bar = sm.bar;
    constexpr int ST = Mf<FMT>::kStages;
    volatile int* abort = &sm.abort;
    constexpr int G = Mf<FMT>::kGroups, OPS = Mf<FMT>::kOps;
    static_assert(acc_col<FMT>(1) + 192 * G <= kTmemCols && acc_col<kFmtQ3>(2) + 256 <= kTmemCols, "TMEM");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Before the first segment: a P warp finds this CTA's share, another sets the barriers up, an M
    // warp gets the TMEM, and the E warps run the query preparation on no rows, which warms its code.
    auto prepared = [&] {
        tc_fence_before();
        named_sync(0, kThreads);
        tc_fence_after();
        return sm.tmem_base;
    };

    // Every role runs through the CTA's segments; E and M meet when a segment's queries are in
    // place, the block when it is done, by when the next one is known.
    bool ok = true;
    if (warp < kWarpD) {
        // ================================================================ E: epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsE));
        uint32_t tmem = 0;
#pragma unroll 1
        for (int k = -1; k < 0 || sm.seg[k & 1].n > 0; ++k) {
            const Segment s = k < 0 ? Segment{0, 0, 0, 0, 0, 0, 1, 0, 1, 0, 0, 0, 0} : sm.seg[k & 1];
            int exp2q = kUsualExp;
            int2& flags = sm.q_flags[k & 1];
            bool again = false;
#pragma unroll 1
            do {
                if (again) exp2q = query_scale<TIn, FMT>(a, s, sm);
                load_queries<TIn, FMT>(a, s, sm, exp2q, again, flags);
                if (k < 0) break;
                if (again) clear_rows<FMT>(s, sm);
                if (tid == 0) {
                    sm.unscale = two_to(-exp2q);
                    sm.q_flags[(k + 1) & 1] = make_int2(0, 0);
                }
                named_sync(1, kQueryThreads);
                again = !again && (flags.x != 0 || flags.y == 0);        // M decides the same
            } while (again);
            if (k < 0) {
                tmem = prepared();
                continue;
            }
            const EpiState e{tmem + ((uint32_t)(32 * (warp & 3)) << 16) + acc_col<FMT>(s.buffers), abort};
            constexpr int B = double_buffered<FMT>(1) ? 2 : 1;
            const int rows = kGroup * s.T;
            if (rows > 48) ok = epilogue<FMT, 64, 1>(a, s, sm, e, ok);
            else if (rows > 32) ok = epilogue<FMT, 48, 1>(a, s, sm, e, ok);
            else if (rows > 16) ok = epilogue<FMT, 32, B>(a, s, sm, e, ok);
            else ok = epilogue<FMT, 16, B>(a, s, sm, e, ok);
            named_sync(0, kThreads);
            if (*abort) break;
        }
    } else if (warp < kWarpM) {
        // ================================================================ D: keys -> TMEM
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsD));
        const float cent = FMT == kFmtT5k ? a.t5k.c[lane] : 0.0f;
        const int odd = (warp - kWarpD) >> 2;                // this warp's parts: odd and odd + 2
        const int p = 32 * (warp & 3) + lane;
        const uint32_t tmem = prepared();
        const uint32_t col0 = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
        for (int k = 0; sm.seg[k & 1].n > 0; ++k) {
            const Segment s = sm.seg[k & 1];
            const int n = s.n;
            int rs = s.tiles_done % ST;                     // stage and its phase
            uint32_t rp = (uint32_t)(s.tiles_done / ST) & 1u;
            if (s.buffers == 2) {
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int use = (s.tiles_double + i) >> 1, buf = (s.tiles_double + i) & 1;
                    const uint8_t* rec = sm.rec[rs] + p * Mf<FMT>::kStride;
                    // the records are there, and the products of this buffer's last tile have read it
                    ok = ok && (use > 0 ? mbar_wait_two(&bar.r_full[rs], rp, &bar.b_free[buf][odd], (uint32_t)((use - 1) & 1), abort)
                                        : mbar_wait_all(&bar.r_full[rs], rp, abort));
                    __syncwarp();
                    tc_fence_after();
                    const uint32_t col = col0 + kPartCols * (kParts * buf + odd);
                    // rolled: 655,360 positions x 8 tokens, which do not take this path, 106 -> 100 us, fp8 49.0 -> 47.7,
                    // 6 tokens 90.6 -> 92.1, 1 token the same.  The code is smaller and lies elsewhere; which of the two
                    // counts was not looked into
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        uint32_t wc[Words<FMT>::kN];
                        read_part<FMT>(rec, odd + 2 * h, wc);
                        store_half<FMT>(wc, 0, cent, col + 2 * kPartCols * h);
                        store_half<FMT>(wc, 1, cent, col + 2 * kPartCols * h + 16);
                    }
                    if (lane == 0) mbar_arrive(&bar.r_free[rs]);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.b_full[buf][odd]);
                    if (++rs == ST) {
                        rs = 0;
                        rp ^= 1u;
                    }
                }
            }
#pragma unroll 1
            for (int i = 0; s.buffers == 1 && i < n; ++i) {
                ok = ok && mbar_wait_fast(&bar.r_full[rs], rp, abort);
                const uint8_t* rec = sm.rec[rs] + p * Mf<FMT>::kStride;
#pragma unroll 1
                for (int part = odd; part < kParts; part += 2) {
                    uint32_t wc[Words<FMT>::kN];
                    read_part<FMT>(rec, part, wc);
                    // the previous tile's products have read the operand
                    if (i > 0) ok = ok && mbar_wait_fast(&bar.a_free[part], (uint32_t)((s.tiles_single + i - 1) & 1), abort);
                    __syncwarp();
                    tc_fence_after();
                    store_half<FMT>(wc, 0, cent, col0 + kPartCols * part);
                    store_half<FMT>(wc, 1, cent, col0 + kPartCols * part + 16);
                    if (part >= kParts - 2 && lane == 0) mbar_arrive(&bar.r_free[rs]);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.a_full[part]);
                }
                if (++rs == ST) {
                    rs = 0;
                    rp ^= 1u;
                }
            }
            named_sync(0, kThreads);
            if (*abort) break;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsMP));
        if (warp < kWarpP) {
        // ================================================================ M: products of one part
        if (warp == kWarpM) tmem_alloc(&sm.tmem_base, kTmemCols);
        const uint32_t tmem = prepared();
        const int first_part = warp - kWarpM;                // this issuer's parts: every kIssuers-th
#pragma unroll 1
        for (int k = 0; sm.seg[k & 1].n > 0; ++k) {
            const Segment s = sm.seg[k & 1];
            named_sync(1, kQueryThreads);
            const int2 flags = sm.q_flags[k & 1];
            if (flags.x != 0 || flags.y == 0) named_sync(1, kQueryThreads);      // E prepares them again
            const int n = s.n;
            const int cols = acc_cols(s);
            const int slots = acc_slots<FMT>(s.buffers, cols);
            const int c_first = kParts * s.phases;
#pragma unroll 1
            for (int i = 0; ok && i < n; ++i) {
#pragma unroll 1
                for (int j = 0; ok && j < s.chunks; ++j) {
                    const uint32_t idesc = make_idesc(mma_rows(s, j), false, false);
                    const int ph = s.phases + i * s.chunks + j;
#pragma unroll 1
                    for (int part = first_part; ok && part < kParts; part += kIssuers) {
                        const int c = kParts * ph + part;
                        const int td = s.tiles_double + i, buf = s.buffers == 2 ? td & 1 : 0;
                        if (j == 0)
                            ok = s.buffers == 2 ? mbar_wait_all(&bar.b_full[buf][part & 1], (uint32_t)((td >> 1) & 1), abort)
                                                : mbar_wait_all(&bar.a_full[part], (uint32_t)((s.tiles_single + i) & 1), abort);
                        // the slot's last accumulators (event c - slots) are read; earlier segments' all are
                        if (ok && c - slots >= c_first)
                            ok = mbar_wait_all(&bar.acc_free[(c - slots) % kFreeBars], (uint32_t)(((c - slots) / kFreeBars) & 1), abort);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem + acc_col<FMT>(s.buffers) + (uint32_t)((c % slots) * G * cols);
                        const uint32_t aop = tmem + kPartCols * (kParts * buf + part);
                        // dims 64 part ..: two 8-dim cores per K step, start address in 16-byte units
                        const uint64_t bh = make_desc(smem_u32(sm.q[j][0]) + part * 8 * kLbo, kLbo, kSbo);
                        const uint64_t bl = make_desc(smem_u32(sm.q[j][1]) + part * 8 * kLbo, kLbo, kSbo);
                        constexpr uint64_t kStep = 2 * kLbo / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t dg = d + (G == 2 ? (uint32_t)(cols * (k / 2)) : 0u);
                                const uint32_t first = (G == 2 ? (k & 1) : k) == 0 ? 0u : 1u;
                                mma_ts(dg, aop + 8 * k, bh + kStep * k, idesc, first);
                                mma_ts(dg, aop + 8 * k, bl + kStep * k, idesc, 1u);
                                if (OPS == 2) {
                                    mma_ts(dg, aop + kParts * kPartCols + 8 * k, bh + kStep * k, idesc, 1u);
                                    mma_ts(dg, aop + kParts * kPartCols + 8 * k, bl + kStep * k, idesc, 1u);
                                }
                            }
                            mma_commit(&bar.done[part][ph % kDoneBars]);
                            if (j == s.chunks - 1) mma_commit(s.buffers == 2 ? &bar.b_free[buf][part & 1] : &bar.a_free[part]);
                        }
                        __syncwarp();
                    }
                }
            }
            named_sync(0, kThreads);
            if (*abort) break;
        }
        if (elect_one()) mma_commit(&bar.drain[first_part]);
        __syncwarp();
        mbar_drain(&bar.drain[first_part], 0);
        } else {
        // ================================================================ P: records -> shared memory
        if (warp == kWarpP + 1) {                             // a lane per barrier
            if (lane < kParts) {
                mbar_init(&bar.a_full[lane], 4);
                mbar_init(&bar.a_free[lane], 1);
                mbar_init(&bar.b_full[lane >> 1][lane & 1], 4);
                mbar_init(&bar.b_free[lane >> 1][lane & 1], 2);
            }
            for (int e = lane; e < kParts * kDoneBars; e += 32) mbar_init(&bar.done[e / kDoneBars][e % kDoneBars], 1);
            for (int e = lane; e < kFreeBars; e += 32) mbar_init(&bar.acc_free[e], 4);
            if (lane < kIssuers) mbar_init(&bar.drain[lane], 1);
            if (lane < ST) {
                mbar_init(&bar.r_full[lane], Mf<FMT>::kPadded ? kCopyThreads : 1);
                mbar_init(&bar.r_free[lane], Mf<FMT>::kScales ? 12 : 8);
            }
            if (lane == 0) sm.abort = 0;
            if (lane < 2) sm.q_flags[lane] = make_int2(0, 0);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        if (warp == kWarpP) share_of<FMT>(a, sm);
        prepared();
#pragma unroll 1
        for (int k = 0; sm.seg[k & 1].n > 0; ++k) {
            const Segment s = sm.seg[k & 1];
            const int n = s.n;
            if (tid == 32 * kWarpP + 32) next_segment<FMT>(a, sm, k + 1);
            int staged = s.tiles_done;                      // next tile to copy
            if (Mf<FMT>::kPadded || warp == kWarpP) {
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int rc = s.tiles_done + i;
                    // every stage is free when a segment begins
                    if (i >= ST) ok = ok && mbar_wait_all(&bar.r_free[rc % ST], (uint32_t)((rc / ST - 1) & 1), abort);
                    if (!ok) break;
                    stage_tile<FMT>(a, s, sm, i, rc);
                    staged = rc + 1;
                }
            }
            named_sync(0, kThreads);
            if (*abort) {
                // copies in flight land before the CTA leaves
                if (Mf<FMT>::kPadded) asm volatile("cp.async.wait_all;" ::: "memory");
                else if (warp == kWarpP)
                    for (int k = max(s.tiles_done, staged - ST); k < staged; ++k) mbar_drain(&bar.r_full[k % ST], (uint32_t)((k / ST) & 1));
                break;
            }
        }
        }
    }
    tc_fence_before();
    named_sync(0, kThreads);
    if (warp == kWarpM) tmem_dealloc(sm.tmem_base, kTmemCols);
    if (*abort && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_TIMEOUT);
}

template <typename TIn, int FMT>
cudaError_t launch_mass(const MassArgs& a, int sms, cudaStream_t stream) {
    // the shared-memory opt-in is a per-device function attribute
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const int smem = (int)sizeof(MassSmem<FMT>);
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute(mass_kernel<TIn, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    const int64_t most = (int64_t)a.num_slots * a.num_kv_heads * ((a.max_ctx_len + kTileP - 1) / kTileP);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(sms, most));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mass_kernel<TIn, FMT>, a);
}

int mass_impl(int fmt, void* stream, const q3kv_cache_desc* desc, const void* d_pool, const int32_t* d_page_table,
              int32_t max_pages_per_slot, const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
              int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer, const void* q, int32_t dtype,
              const float* lse, float decay, float* d_mass, int64_t mass_stride, int32_t* d_status) {
    const int e = check_desc(desc);
    if (e != Q3KV_OK) return e;
    if (num_slots < 0 || max_pages_per_slot <= 0 || layer < 0 || layer >= desc->num_layers || max_n_q < 0 ||
        max_ctx_len < 0 || mass_stride < max_ctx_len)
        return Q3KV_ERR_INVALID_ARG;
    if (max_ctx_len > (int64_t)INT32_MAX - kPageSize) return Q3KV_ERR_INVALID_ARG;
    if (!(decay >= 0.0f && decay <= 1.0f)) return Q3KV_ERR_INVALID_ARG;
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (max_n_q > kMaxNq || num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (num_slots == 0 || max_n_q == 0 || max_ctx_len == 0) return Q3KV_OK;
    if (!d_pool || !d_page_table || !d_ctx_len || !d_n_q || !d_q_offsets || !q || !lse || !d_mass)
        return Q3KV_ERR_INVALID_ARG;
    if (!aligned16(d_pool) || !aligned16(q)) return Q3KV_ERR_INVALID_ARG;
    MassArgs a{};
    a.pool = static_cast<const uint8_t*>(d_pool);
    a.page_table = d_page_table;
    a.max_pages_per_slot = max_pages_per_slot;
    a.ctx_len = d_ctx_len;
    a.n_q = d_n_q;
    a.q_offsets = d_q_offsets;
    a.num_slots = num_slots;
    a.max_ctx_len = max_ctx_len;
    a.max_n_q = max_n_q;
    a.num_layers = desc->num_layers;
    a.num_kv_heads = desc->num_kv_heads;
    a.num_pages = desc->num_pages;
    a.layer = layer;
    a.q = q;
    a.dtype = dtype;
    a.lse = lse;
    a.decay = decay;
    a.mass = d_mass;
    a.mass_stride = mass_stride;
    a.status = d_status;
    a.fmt = fmt;
    if (fmt == kFmtT5k) a.t5k = t5k_table();
    int sms = 0;
    const int es = device_sm_count(&sms);
    if (es != Q3KV_OK) return es;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f32 = dtype == Q3KV_F32;
    if (fmt == kFmtFp8) return cuda_status(f32 ? launch_mass<float, kFmtFp8>(a, sms, st) : launch_mass<__nv_bfloat16, kFmtFp8>(a, sms, st));
    if (fmt == kFmtT5k) return cuda_status(f32 ? launch_mass<float, kFmtT5k>(a, sms, st) : launch_mass<__nv_bfloat16, kFmtT5k>(a, sms, st));
    return cuda_status(f32 ? launch_mass<float, kFmtQ3>(a, sms, st) : launch_mass<__nv_bfloat16, kFmtQ3>(a, sms, st));
}

}  // namespace
}  // namespace q3kv

using namespace q3kv;

extern "C" {

#define Q3KV_MASS_ENTRY(NAME, FMT)                                                                                  \
    int NAME(void* stream, const q3kv_cache_desc* desc, const void* d_pool, const int32_t* d_page_table,            \
             int32_t max_pages_per_slot, const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets, \
             int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer, const void* q, int32_t dtype,   \
             const float* lse, float decay, float* d_mass, int64_t mass_stride, int32_t* d_status) {                 \
        return mass_impl(FMT, stream, desc, d_pool, d_page_table, max_pages_per_slot, d_ctx_len, d_n_q, d_q_offsets, \
                         num_slots, max_ctx_len, max_n_q, layer, q, dtype, lse, decay, d_mass, mass_stride, d_status); \
    }

Q3KV_MASS_ENTRY(q3kv_attn_mass, kFmtQ3)
Q3KV_MASS_ENTRY(q3kv_fp8_attn_mass, kFmtFp8)
Q3KV_MASS_ENTRY(q3kv_t5k_attn_mass, kFmtT5k)

}  // extern "C"
