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
// scores are float32-exact: queries as fp16 hi + lo pairs (22 bits), keys exact.
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
// the 3-bit cache: two blocks of 64 rows) form one slot of a ring of three, so the
// epilogue of a part overlaps the products of the next ones.
//
// Warp roles (16 warps, 128 registers each):
//   E   warps 0-7    epilogue: thread = position (lane quarter warp & 3), rows 0-31 or
//                    32-63 of the chunk (warp >> 2); score sums start at -lse in log2
//                    units, weights 2^s, rows summed in the thread
//   D   warps 8-11   thread = position: its record in registers a tile (or a part)
//                    ahead, converted part by part into TMEM
//   M   warps 12-15  one thread each issues the products of one part: an issuing
//                    thread starts a K = 16 MMA about every 54 cycles, so four issue
// TMEM (512 columns): operand (128, turbo5k 256) | ring of three slots (3 x 128, or x 64).
//
// Work: the tiles of all (slot, kv head) pairs in one sequence, an equal share per
// CTA (one per SM), whatever the slots' lengths; a CTA rotates and splits the
// queries of a pair itself when it enters it.
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

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kTileP = 128;                 // positions per tile
constexpr int kChunkRows = 64;              // query rows per pass over a tile
constexpr int kMaxChunks = kMaxRows / kChunkRows;
constexpr int kParts = 4;                   // parts of 64 dims
constexpr int kSlots = 3;                   // accumulator slots
constexpr int kFreeBars = 12;               // consumption events: a multiple of kParts and kSlots

template <int FMT>
struct Mf {                                 // 3-bit cache
    static constexpr int kGroups = 2;       // accumulators (scale groups) of a part
    static constexpr int kOps = 1;          // fp16 operands per value
    static constexpr int kRecB = kRecordBytes;
    static constexpr bool kRot = true;
};
template <>
struct Mf<kFmtFp8> {
    static constexpr int kGroups = 1;
    static constexpr int kOps = 1;
    static constexpr int kRecB = kFp8RecordBytes;
    static constexpr bool kRot = false;
};
template <>
struct Mf<kFmtT5k> {
    static constexpr int kGroups = 1;
    static constexpr int kOps = 2;
    static constexpr int kRecB = kT5kKRecordBytes;
    static constexpr bool kRot = true;
};
constexpr uint32_t kPartCols = 32;          // TMEM columns of a part's operand (64 fp16 values)
constexpr uint32_t kTmemCols = 512;

struct Bars {
    unsigned long long a_full[kParts];      // operand part in TMEM (4 D warps)
    unsigned long long done[kParts];        // products of a part and chunk (1 commit): accumulators ready
    unsigned long long a_free[kParts];      // every chunk's products of a part (1 commit): operand read
    unsigned long long acc_free[kFreeBars]; // accumulators of the event read (8 E warps)
    unsigned long long drain[kParts];       // everything an issuer started is done (1 commit)
};

struct __align__(16) MassSmem {
    __half q[kMaxChunks][2][kChunkRows * kHeadDim];   // [chunk][hi | lo], B operand
    float nlse[kMaxRows];                             // -lse in log2 units; -inf leaves a row out
    float part[2][kTileP];                            // sums of rows 32..63, double-buffered by tile
    Bars bar;
    uint32_t tmem_base;
    int abort;
    int first_slot;
    long long first_base, w0, w1;
};

// Tiles of a slot's kv head; 0 for a slot with nothing to do.
__device__ __forceinline__ int slot_tiles(const MassArgs& a, int b, bool* bad) {
    const int T = a.n_q[b], L = a.ctx_len[b];
    if (T <= 0) return 0;
    if (T > a.max_n_q || T > L || L > a.max_ctx_len || L > (int64_t)a.max_pages_per_slot * kPageSize) {
        *bad = true;
        return 0;
    }
    return (L + kTileP - 1) / kTileP;
}

__device__ __forceinline__ unsigned long long pack2(float lo, float hi) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
// two float32 fused multiply-adds in one instruction
__device__ __forceinline__ unsigned long long fma2(unsigned long long x, unsigned long long y, unsigned long long z) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}

// One segment: tiles [t0, t1) of a (slot, kv head) pair.
struct Segment {
    int slot, g, t0, t1;
    int T, L, chunks;
    const int32_t* pt;
};

// Queries of the segment's pair: H, then 1/16 (H) 1/16 (softmax) log2(e), split
// into fp16 hi / lo, and -lse in log2 units; padding rows are zeros.  One row per warp.
template <typename TIn, int FMT>
__device__ void load_queries(const MassArgs& a, const Segment& s, MassSmem& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int R = kGroup * s.T;
    const int Hq = a.num_kv_heads * kGroup;
    const int64_t q_base = a.q_offsets[s.slot];
    for (int r = warp; r < s.chunks * kChunkRows; r += kWarps) {
        const int chunk = r / kChunkRows, rr = r % kChunkRows;
        const int64_t row = (q_base + r / kGroup) * Hq + s.g * kGroup + r % kGroup;
        float y[8];
        if (r < R) {
            load8(static_cast<const TIn*>(a.q) + row * kHeadDim + 8 * lane, y);
            if (Mf<FMT>::kRot) rotate_row_regs(y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        }
        constexpr float kScale = Mf<FMT>::kRot ? 1.4426950408889634f / 256.0f : 1.4426950408889634f / 16.0f;
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x0 = y[2 * i] * kScale, x1 = y[2 * i + 1] * kScale;
            const __half2 h2 = __floats2half2_rn(x0, x1);
            const float2 hf = __half22float2(h2);
            hw[i] = as_u32(h2);
            lw[i] = as_u32(__floats2half2_rn(x0 - hf.x, x1 - hf.y));
        }
        *reinterpret_cast<uint4*>(&sm.q[chunk][0][q_off(rr, 8 * lane)]) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(&sm.q[chunk][1][q_off(rr, 8 * lane)]) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        if (lane == 0) {
            float v = -CUDART_INF_F;
            if (r < R) {
                const float l = a.lse[row];
                if (l > -CUDART_INF_F && l < CUDART_INF_F) v = -1.4426950408889634f * l;
                else if (a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
            }
            sm.nlse[r] = v;
        }
    }
    fence_proxy_async();
}

__device__ __forceinline__ int32_t page_of(const MassArgs& a, const int32_t* pt, int pos0) {
    const int32_t page = pt[pos0 / kPageSize];
    return (page >= 0 && page < a.num_pages) ? page : -1;
}

template <int FMT>
__device__ __forceinline__ const uint8_t* k_record(const MassArgs& a, const Segment& s, int32_t page, int pos) {
    return a.pool + (FMT == kFmtT5k ? t5k_offset(a.num_layers, a.num_kv_heads, page, a.layer, s.g, 0, pos % kPageSize)
                                    : record_offset(a.num_layers, a.num_kv_heads, page, a.layer, s.g, 0, pos % kPageSize,
                                                    Mf<FMT>::kRecB));
}

// Words of a part of a record that a D thread holds ahead.
template <int FMT>
struct Words {
    static constexpr int kN = FMT == kFmtFp8 ? 16 : (FMT == kFmtT5k ? 10 : 6);
};

template <int FMT>
__device__ __forceinline__ void fetch_part(const uint8_t* rec, int q, uint32_t (&w)[Words<FMT>::kN]) {
    if constexpr (FMT == kFmtFp8) {
        const uint4* p = reinterpret_cast<const uint4*>(rec) + 4 * q;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const uint4 u = rec ? __ldg(p + m) : make_uint4(0u, 0u, 0u, 0u);
            w[4 * m] = u.x; w[4 * m + 1] = u.y; w[4 * m + 2] = u.z; w[4 * m + 3] = u.w;
        }
    } else if constexpr (FMT == kFmtT5k) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(rec);
#pragma unroll
        for (int m = 0; m < 8; ++m) w[m] = rec ? __ldg(p + 8 * q + m) : 0u;
#pragma unroll
        for (int m = 0; m < 2; ++m) w[8 + m] = rec ? __ldg(p + 32 + 2 * q + m) : 0u;
    } else {
        const uint2* p = reinterpret_cast<const uint2*>(rec) + 3 * q;      // 24 bytes
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            const uint2 u = rec ? __ldg(p + m) : make_uint2(0u, 0u);
            w[2 * m] = u.x; w[2 * m + 1] = u.y;
        }
    }
}

// 64 dims of this thread's position into the TMEM columns at col.
template <int FMT>
__device__ __forceinline__ void store_part(const uint32_t (&w)[Words<FMT>::kN], float cent, uint32_t col) {
    if constexpr (FMT == kFmtFp8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t h8[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) e4m3x4_to_f16(w[4 * c + k], h8[2 * k], h8[2 * k + 1]);
            tmem_st8(col + 8 * c, h8);
        }
    } else if constexpr (FMT == kFmtT5k) {
        // lane l holds centroid l: a code's value by shuffle, split into fp16 hi / lo
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int mm = 0; mm < 8; ++mm) {
                const int m = 8 * c + mm;                      // pair of the part
                const uint32_t nw = w[m / 4], top = w[8 + m / 16];
                const uint32_t c0 = ((nw >> (8 * (m % 4))) & 0xFu) | (((top >> (2 * (m % 16))) & 1u) << 4);
                const uint32_t c1 = ((nw >> (8 * (m % 4) + 4)) & 0xFu) | (((top >> (2 * (m % 16) + 1)) & 1u) << 4);
                const float v0 = __shfl_sync(0xffffffffu, cent, (int)c0);
                const float v1 = __shfl_sync(0xffffffffu, cent, (int)c1);
                const __half2 h2 = __floats2half2_rn(v0, v1);
                const float2 hf = __half22float2(h2);
                hi[mm] = as_u32(h2);
                lo[mm] = as_u32(__floats2half2_rn(v0 - hf.x, v1 - hf.y));
            }
            tmem_st8(col + 8 * c, hi);
            tmem_st8(col + kParts * kPartCols + 8 * c, lo);
        }
    } else {
        const __half2 m12 = __half2half2(__ushort_as_half((unsigned short)0xCA00u));   // -12
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t h16[16];
#pragma unroll
            for (int m = 0; m < 16; ++m) {
                const uint32_t x = m < 15 ? code_pair_word(w[3 * b + m / 5], 3 * (m % 5))
                                          : code_pair_last(w[3 * b], w[3 * b + 1], w[3 * b + 2]);
                h16[m] = as_u32(__hadd2(as_h2(x), m12));       // (8.5 + c) - 12, exact
            }
            tmem_st16(col + 16 * b, h16);
        }
    }
}

template <typename TIn, int FMT>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassArgs a) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    MassSmem& sm = *reinterpret_cast<MassSmem*>(smem_raw);
    Bars& bar = sm.bar;
    volatile int* abort = &sm.abort;
    constexpr int G = Mf<FMT>::kGroups, OPS = Mf<FMT>::kOps;
    constexpr uint32_t kColAcc = kParts * kPartCols * OPS;
    constexpr uint32_t kSlotCols = G * kChunkRows;
    static_assert(kColAcc + kSlots * kSlotCols <= kTmemCols, "TMEM");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (tid == 0) {
        for (int q = 0; q < kParts; ++q) {
            mbar_init(&bar.a_full[q], 4);
            mbar_init(&bar.done[q], 1);
            mbar_init(&bar.a_free[q], 1);
            mbar_init(&bar.drain[q], 1);
        }
        for (int e = 0; e < kFreeBars; ++e) mbar_init(&bar.acc_free[e], 8);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) tmem_alloc(&sm.tmem_base, kTmemCols);
    if (warp == 0) {
        // this CTA's share [w0, w1) of the sequence, and the slot it starts in
        bool bad = false;
        long long total = 0;
        for (int b0 = 0; b0 < a.num_slots; b0 += 32)
            total += warp_sum_i(b0 + lane < a.num_slots ? slot_tiles(a, b0 + lane, &bad) : 0);
        if (blockIdx.x == 0 && bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        total *= a.num_kv_heads;
        const long long w0 = total * blockIdx.x / gridDim.x, w1 = total * (blockIdx.x + 1) / gridDim.x;
        long long base = 0;
        int slot = a.num_slots;
        for (int b0 = 0; b0 < a.num_slots && w0 < w1; b0 += 32) {
            const long long mine = b0 + lane < a.num_slots ? (long long)slot_tiles(a, b0 + lane, &bad) * a.num_kv_heads : 0;
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
            sm.first_slot = slot;
            sm.first_base = base;
            sm.w0 = w0;
            sm.w1 = w1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    const long long w1 = sm.w1;
    long long w = sm.w0, base = sm.first_base;
    int slot = sm.first_slot;
    int tiles_done = 0;                      // tiles of earlier segments (a_full and a_free phases)
    int phases = 0;                          // (tile, chunk) passes of earlier segments (done phases)
    bool ok = true;
    const float cent = FMT == kFmtT5k ? a.t5k.c[lane] : 0.0f;

    while (w < w1) {
        Segment s;
        bool ignore = false;
        const int tiles = slot_tiles(a, slot, &ignore);
        const long long off = w - base;
        s.slot = slot;
        s.g = (int)(off / tiles);
        s.t0 = (int)(off - (long long)s.g * tiles);
        s.t1 = (int)min((long long)tiles, s.t0 + (w1 - w));
        s.T = a.n_q[slot];
        s.L = a.ctx_len[slot];
        s.chunks = (kGroup * s.T + kChunkRows - 1) / kChunkRows;
        s.pt = a.page_table + (int64_t)slot * a.max_pages_per_slot;
        load_queries<TIn, FMT>(a, s, sm);
        __syncthreads();
        const int n = s.t1 - s.t0;
        const int Nctx = s.L - s.T;

        if (warp < 8) {
            // ============================================================ E: epilogue
            const int q4 = warp & 3, rh = warp >> 2, r0 = 32 * rh;
            const int p = 32 * q4 + lane;
            const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
            float* mass = a.mass + ((int64_t)s.slot * a.num_kv_heads + s.g) * a.mass_stride;
            // this thread's scales of a tile, a tile ahead
            auto fetch_scales = [&](int i, uint4& sc) {
                const int pos0 = (s.t0 + i) * kTileP;
                const int32_t page = i < n ? page_of(a, s.pt, pos0) : -1;
                sc = make_uint4(0u, 0u, 0u, 0u);
                if (page >= 0 && pos0 + p < s.L) {
                    const uint8_t* rec = k_record<FMT>(a, s, page, pos0 + p);
                    if (FMT == kFmtQ3) sc = __ldg(reinterpret_cast<const uint4*>(rec + 96));
                    if (FMT == kFmtT5k) sc.x = __ldg(reinterpret_cast<const uint32_t*>(rec + 160));
                }
            };
            uint4 next;
            fetch_scales(0, next);
            for (int i = 0; i < n; ++i) {
                const uint4 sc = next;
                fetch_scales(i + 1, next);
                const int pos0 = (s.t0 + i) * kTileP;
                const int pos = pos0 + p;
                const bool page_ok = page_of(a, s.pt, pos0) >= 0;
                if (!page_ok && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
                float old = 0.0f;
                if (rh == 0 && a.decay > 0.0f && pos < Nctx) old = mass[pos];
                const bool interior = pos0 + kTileP - 1 <= Nctx;
                float sum = 0.0f;
                for (int j = 0; j < s.chunks; ++j) {
                    const int rows = min(kChunkRows, kGroup * s.T - kChunkRows * j);
                    const int N = (rows + 15) & ~15;
                    const int ph = phases + i * s.chunks + j;
                    unsigned long long acc[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 u = *reinterpret_cast<const float4*>(&sm.nlse[kChunkRows * j + r0 + 4 * k]);
                        acc[2 * k] = pack2(u.x, u.y);
                        acc[2 * k + 1] = pack2(u.z, u.w);
                    }
#pragma unroll
                    for (int part = 0; part < kParts; ++part) {
                        const int c = kParts * ph + part;
                        ok = ok && warp_wait(&bar.done[part], (uint32_t)(ph & 1), abort);
                        tc_fence_after();
                        const uint32_t col = tmem + lane_base + kColAcc + (uint32_t)(c % kSlots) * kSlotCols + r0;
#pragma unroll
                        for (int gi = 0; gi < G; ++gi) {
                            float scale = 1.0f;
                            if (FMT == kFmtQ3) {
                                const uint32_t word = part == 0 ? sc.x : (part == 1 ? sc.y : (part == 2 ? sc.z : sc.w));
                                scale = __half2float(__ushort_as_half((unsigned short)(gi ? word >> 16 : word & 0xFFFFu)));
                            } else if (FMT == kFmtT5k) {
                                scale = __half2float(__ushort_as_half((unsigned short)(part >= 2 ? sc.x >> 16 : sc.x & 0xFFFFu)));
                            }
                            const unsigned long long s2 = pack2(scale, scale);
                            float x[32];
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (r0 + 16 * h < N) tmem_ld16(col + kChunkRows * gi + 16 * h, &x[16 * h]);
                            tmem_ld_wait();
                            if (gi == G - 1) {
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) mbar_arrive(&bar.acc_free[c % kFreeBars]);
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (r0 + 16 * h < N)
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        acc[8 * h + k] = fma2(pack2(x[16 * h + 2 * k], x[16 * h + 2 * k + 1]), s2, acc[8 * h + k]);
                        }
                    }
                    // weights; row r (token r / 8) sees positions <= Nctx + r / 8
                    const int r_min = interior ? 0 : kGroup * (pos - Nctx) - kChunkRows * j - r0;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (r0 + 16 * h < N)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float x0, x1;
                                unpack2(acc[8 * h + k], x0, x1);
                                const int r = 16 * h + 2 * k;
                                sum += r >= r_min ? fast_exp2(x0) : 0.0f;
                                sum += r + 1 >= r_min ? fast_exp2(x1) : 0.0f;
                            }
                }
                if (rh == 1) sm.part[i & 1][p] = sum;
                named_sync(1 + q4, 64);
                if (rh == 0 && pos < s.L) {
                    const float t = page_ok ? sum + sm.part[i & 1][p] : 0.0f;
                    mass[pos] = fmaf(a.decay, old, t);
                }
            }
        } else if (warp < 12) {
            // ============================================================ D: keys -> TMEM
            const int p = 32 * (warp & 3) + lane;
            const uint32_t col0 = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            auto record = [&](int i) -> const uint8_t* {
                const int pos0 = (s.t0 + i) * kTileP;
                const int32_t page = i < n ? page_of(a, s.pt, pos0) : -1;
                return (page >= 0 && pos0 + p < s.L) ? k_record<FMT>(a, s, page, pos0 + p) : nullptr;
            };
            const uint8_t* rec = record(0);
            uint32_t wn[kParts][Words<FMT>::kN];
#pragma unroll
            for (int part = 0; part < kParts; ++part) fetch_part<FMT>(rec, part, wn[part]);
            for (int i = 0; i < n; ++i) {
                rec = record(i + 1);
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    uint32_t wc[Words<FMT>::kN];
#pragma unroll
                    for (int m = 0; m < Words<FMT>::kN; ++m) wc[m] = wn[part][m];
                    fetch_part<FMT>(rec, part, wn[part]);
                    // the previous tile's products have read the operand
                    if (i > 0) ok = ok && warp_wait(&bar.a_free[part], (uint32_t)((tiles_done + i - 1) & 1), abort);
                    tc_fence_after();
                    store_part<FMT>(wc, cent, col0 + kPartCols * part);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.a_full[part]);
                }
            }
        } else {
            // ============================================================ M: products of one part
            const int part = warp - 12;
            const uint32_t aop = tmem + kPartCols * part;
            for (int i = 0; ok && i < n; ++i) {
                ok = warp_wait(&bar.a_full[part], (uint32_t)((tiles_done + i) & 1), abort);
                for (int j = 0; ok && j < s.chunks; ++j) {
                    const int rows = min(kChunkRows, kGroup * s.T - kChunkRows * j);
                    const uint32_t idesc = make_idesc((rows + 15) & ~15, false, false);
                    const int c = kParts * (phases + i * s.chunks + j) + part;
                    // the slot's last accumulators (event c - 3) are read
                    if (c >= kSlots)
                        ok = warp_wait(&bar.acc_free[(c - kSlots) % kFreeBars], (uint32_t)(((c - kSlots) / kFreeBars) & 1), abort);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + kColAcc + (uint32_t)(c % kSlots) * kSlotCols;
                    // dims 64 part ..: two 8-dim cores (256 bytes) per K step, start address in 16-byte units
                    const uint64_t bh = make_desc(smem_u32(sm.q[j][0]) + part * 1024, kQLbo, kQSbo);
                    const uint64_t bl = make_desc(smem_u32(sm.q[j][1]) + part * 1024, kQLbo, kQSbo);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t dg = d + (G == 2 ? kChunkRows * (k / 2) : 0);
                            const uint32_t first = (G == 2 ? (k & 1) : k) == 0 ? 0u : 1u;
                            mma_ts(dg, aop + 8 * k, bh + 16 * k, idesc, first);
                            mma_ts(dg, aop + 8 * k, bl + 16 * k, idesc, 1u);
                            if (OPS == 2) {
                                mma_ts(dg, aop + kParts * kPartCols + 8 * k, bh + 16 * k, idesc, 1u);
                                mma_ts(dg, aop + kParts * kPartCols + 8 * k, bl + 16 * k, idesc, 1u);
                            }
                        }
                        mma_commit(&bar.done[part]);
                        if (j == s.chunks - 1) mma_commit(&bar.a_free[part]);
                    }
                    __syncwarp();
                }
            }
        }
        tiles_done += n;
        phases += n * s.chunks;
        __syncthreads();                     // queries and barriers are free for the next segment
        if (*abort) break;
        w += n;
        if (w >= base + (long long)tiles * a.num_kv_heads && w < w1) {
            base += (long long)tiles * a.num_kv_heads;
            do ++slot;
            while (slot_tiles(a, slot, &ignore) == 0);
        }
    }
    if (warp >= 12) {
        if (elect_one()) mma_commit(&bar.drain[warp - 12]);
        __syncwarp();
        mbar_drain(&bar.drain[warp - 12], 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) tmem_dealloc(tmem, kTmemCols);
    if (*abort && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_TIMEOUT);
}

template <typename TIn, int FMT>
cudaError_t launch_mass(const MassArgs& a, int sms, cudaStream_t stream) {
    // the shared-memory opt-in is a per-device function attribute
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    const int smem = (int)sizeof(MassSmem);
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
