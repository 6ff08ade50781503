// Verify attention over the block-scaled 8-bit cache, tensor-core leg (bf16 or float32 queries and outputs).
//
// The cache's codes are the MMAs' operands as they lie in memory: a page stores them in the 8 x 16-byte cores that
// tcgen05.mma reads, so a tile of 128 positions is one bulk copy of 32 KiB for K and one for V, and nothing is
// decoded.  What the other operands lose in 8 bits is carried by more than one code per value:
//   q  = 2^-k (q1 + q2)      two E4M3 codes, k per row, the second times 2^5: a bf16 value has 8 significant bits, and two
//                            codes hold them all from 2^-14 of the row's largest value on; below, the half step is 2^-22 of it at most
//   p' = p1 + p2 + p3        three E5M2 codes (3 significant bits each, every one rounded to nearest, so that signs add a
//                            bit to the second and third) hold the weight as fp16 exactly from 2^-10 on: 11 bits, at most
//                            2^-11 off; E5M2 for its range (2^-16 .. 2^15), and the last code times 2^7: a long context's
//                            many small weights are not lost next to a large one, and where they are equal, and so is
//                            what they lose, their sum is right
// Float32 queries take six codes of each, in two groups.
// Contractions (M = 128, float32 accumulation in TMEM):
//   S^T[p][r | R + r] = K[p][:] . q1[r][:] | q2[r][:]   A = K codes (K-major), N = 2 R columns, K = 256 dims
//   O^T[d][r] += V[:][d] . p_i'[:][r], i = 1..3          A = V codes (MN-major), two halves of 128 dims, K = 128 positions,
//                                                        two or three codes side by side in the columns, summed at the end
// with R = 16, 32, 48 or 64 query rows (8 heads x tokens, padded).  A position is a TMEM lane, so its block's scales are two
// numbers of one thread: the score is (S1 + 2^-5 S2) 2^(eK - k) log2(e) / 16, and V's scale goes into the weight's
// exponent, p' = 2^(score + eV - m), while the row sum takes p' 2^-eV.  m is raised only when a score passes it by more
// than 2^7 of headroom (a vote per tile), so most tiles need no maximum and no rescaling.
//
// Bound: the codes' bytes.  At 8 tokens a tile's 64 KiB take about 2,900 cycles of an SM's share of HBM (655,360 positions
// of 2 heads: 112 us, 6,000 GB/s; 1 token 103 us, 6,500 GB/s); its 24 MMAs and its softmax, which overlap, less.  9 to 16
// tokens are two chunks of rows: the second reads its tiles from L2, and the chain from scores to codes bounds both (12 tokens 166 us,
// 16 212 us).  One CTA per SM; warp 0 copies, warps 1-3 issue the MMAs, the others are the softmax: groups of
// four warps with a thread per position and 8 or 16 rows.
#include <math_constants.h>

#include <type_traits>

#include "q3kv_bs8.cuh"
#include "q3kv_tcgen05.cuh"

namespace q3kv {
namespace {

constexpr uint32_t kTileBytes = kBs8Tile * kHeadDim;
constexpr float kAbove = 8.0f;                 // m is set this far below the largest score: p' <= 2^8 then,
constexpr float kRaise = 15.0f;                // and at most 2^15 until it is raised
constexpr float kQLast = 32.0f;               // before a bf16 query's second code: what one leaves of 2^8 is 2^3 at most
constexpr float kQStep = 4096.0f;             // between the two groups of a float32 query's codes
constexpr float kPStep = 2048.0f;             // and of a float32 weight's: what three codes leave of 2^15 is 2^4 at most
constexpr float kPLast = 128.0f;              // before a bf16 weight's last code: what two leave of 2^15 is 2^8 at most
constexpr int kMeta = 8;                       // tiles whose scales are kept

template <int R, bool F32>
struct Cfg {
    // Rows per softmax thread; a warpgroup has all positions.  More warps hide more of each other's latency (32,768 positions,
    // 16 -> 8 rows: 4 tokens 16.2 -> 15.1 us, 6 tokens 17.2 -> 16.6); 8 rows of 64 would be more threads than a CTA has,
    // and 4 rows of 16 gain nothing (14.0, 14.3).
    static constexpr int kH = R > 48 ? 16 : 8, kWgs = R / kH;
    static constexpr int kSoftmax = 128 * kWgs, kThreads = 128 + kSoftmax;
    static constexpr int kQ = F32 ? 6 : 2, kP = F32 ? 6 : 3;            // codes per query value and per weight
    // Weight codes side by side in the columns of a PV MMA, as many as TMEM has room for: an MMA of few columns takes as
    // long as one of 64 (32,768 x 1: 14.4 -> 13.9 us; float32 5 slots x 16: 26.8 -> 25.4).
    static constexpr int kBeside = F32 ? (R == 16 ? 6 : 2) : R > 48 ? 2 : 3;
    static constexpr int kParts = (kP + kBeside - 1) / kBeside;        // MMAs that share their columns
    // Code n of a weight is code `column` of part `part`.  Codes that are scaled up (float32's second three, bf16's last)
    // have columns of their own: of two columns the second.
    __host__ __device__ static constexpr int part(int n) { return F32 ? n % kParts : kBeside == 2 && n == 1 ? 1 : 0; }
    __host__ __device__ static constexpr int column(int n) { return F32 ? n / kParts : kBeside == 2 ? n / 2 : n; }
    __host__ __device__ static constexpr int wide(int part) { return F32 || (part + 1) * kBeside <= kP ? kBeside : kP - part * kBeside; }
    // Weight buffers: PV of a tile runs during the next tile's softmax (655,360 x 8: 117 -> 111 us).  Float32 waits for each
    // tile's outputs anyway.
    static constexpr int kPBufs = F32 ? 1 : 2;
    // tiles in shared memory, as many as the queries and weights leave room for; V waits for the softmax
    static constexpr int kK = R > 16 || F32 ? 2 : 3, kV = R > 48 || (F32 && R == 32) ? 2 : 3;
    static constexpr uint32_t kS = kQ * R, kO = 2 * kS;                // TMEM columns: two S buffers, then O halves of kBeside R
    static constexpr uint32_t kUsed = kO + 2 * kBeside * R, kTmem = kUsed > 256 ? 512 : kUsed > 128 ? 256 : 128;
    static_assert(kUsed <= 512 && kS <= 256, "TMEM and the MMA's N");
};

template <int R, bool F32>
struct Smem {
    alignas(128) uint8_t k[Cfg<R, F32>::kK][kTileBytes];
    alignas(128) uint8_t v[Cfg<R, F32>::kV][kTileBytes];
    alignas(128) uint8_t q[Cfg<R, F32>::kQ * R * kHeadDim];
    alignas(128) uint8_t p[Cfg<R, F32>::kPBufs][Cfg<R, F32>::kP * R * kBs8Tile];
    alignas(16) float meta[kMeta][16];         // K scales of a tile's 8 blocks, then V scales
    alignas(16) float rs[R], m[R], dm[R];      // of each row: 2^-k, the maximum negated, its last change
    float red[Cfg<R, F32>::kWgs][4][Cfg<R, F32>::kH];
    Bs8Share first;
    int bad_page[kMeta];
    uint32_t tmem;
    volatile int abort;
    unsigned long long k_full[Cfg<R, F32>::kK], k_free[Cfg<R, F32>::kK], v_full[Cfg<R, F32>::kV], v_free[Cfg<R, F32>::kV], s_full[2], s_free[2], p_full[2], p_free[2], q_full, drained, meta_full[kMeta];
};

// Instruction descriptor, kind::f8f6f4: E4M3 A, E4M3 or E5M2 B, fp32 D, M = 128.
__host__ __device__ constexpr uint32_t idesc8(int n, bool mn_major, bool b_e5m2) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((mn_major ? 1u : 0u) << 15) | ((mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, float* v) {
    if constexpr (N == 8) {
        float t[8];
        tmem_ld8(at, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = t[i];
    } else if constexpr (N == 16) {
        tmem_ld16(at, v);
    } else {
        tmem_ld32(at, v);
    }
}
template <int N>
__device__ __forceinline__ void tmem_store(uint32_t at, const float* v) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[i + j]);
        tmem_st8(at + i, r);
    }
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t last2(uint32_t a) { return as_u32(__hmul2(as_h2(a), __float2half2_rn(kPLast))); }
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) { return as_u32(__hsub2(as_h2(a), as_h2(b))); }

// ---------------------------------------------------------------- roles
// A barrier is waited for by parity, so whoever waits for one has to see each of its phases: K and V have rings of their own.
//
// Bulk copies of a segment's tiles in the order of their use: K0 K1 V0 K2 V1 ... V(n-2) V(n-1).
template <int R, bool F32>
__device__ void produce(const Bs8Args& a, Smem<R, F32>& sm, Bs8Share w) {
    using C = Cfg<R, F32>;
    const int lane = threadIdx.x & 31, heads = a.num_kv_heads;
    uint32_t it = 0, ks = 0, vs = 0;       // tiles before the segment; copies of K and of V so far
    bool ok = true;
    do {
        const int32_t* table = a.page_table + (int64_t)w.slot * a.max_pages_per_slot;
        const int last_page = (w.tile + w.tiles - 1) >> 1;
        int window = (w.tile >> 1) - 32, ids = 0;
        const uint8_t* prev = nullptr;
        for (int i = 0; i <= w.tiles && ok; ++i) {
            const int tile = w.tile + i, half = tile & 1;
            const uint8_t* unit = nullptr;
            if (i < w.tiles) {
                const int pg = tile >> 1;
                if (pg >= window + 32) {
                    window = pg;
                    ids = window + lane <= last_page ? table[window + lane] : 0;
                }
                int id = __shfl_sync(0xffffffffu, ids, pg - window);
                const bool bad = id < 0 || id >= a.num_pages;      // the tile counts as hidden; page 0 stands in for its bytes
                if (bad) id = 0;
                unit = a.pool + bs8_offset(a.num_layers, heads, id, a.layer, w.head(heads), 0);
                if (lane == 0) {
                    const uint32_t t = it + i, st = t % C::kK, slot = t % kMeta;
                    ok = t < C::kK || mbar_wait(&sm.k_free[st], (t / C::kK + 1) & 1, &sm.abort);
                    if (ok) {
                        if (bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
                        sm.bad_page[slot] = bad;
                        mbar_arrive_expect_tx(&sm.meta_full[slot], 64);
                        bulk_g2s(&sm.meta[slot][0], unit + kBs8CodeBytes + half * 32, 32, &sm.meta_full[slot]);
                        bulk_g2s(&sm.meta[slot][8], unit + kBs8UnitBytes + kBs8CodeBytes + half * 32, 32, &sm.meta_full[slot]);
                        mbar_arrive_expect_tx(&sm.k_full[st], kTileBytes);
                        bulk_g2s(sm.k[st], unit + half * kTileBytes, kTileBytes, &sm.k_full[st]);
                        ks = t + 1;
                    }
                }
                unit += kBs8UnitBytes + half * kTileBytes;         // V of the same tile
            }
            if (i > 0 && lane == 0 && ok) {
                const uint32_t t = it + i - 1, st = t % C::kV;
                ok = t < C::kV || mbar_wait(&sm.v_free[st], (t / C::kV + 1) & 1, &sm.abort);
                if (ok) {
                    mbar_arrive_expect_tx(&sm.v_full[st], kTileBytes);
                    bulk_g2s(sm.v[st], prev, kTileBytes, &sm.v_full[st]);
                    vs = t + 1;
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            prev = unit;
        }
        it += w.tiles;
    } while (ok && w.next(a));
    // no copy may land after the CTA is gone, whatever stopped the others
    if (lane == 0) {
        for (uint32_t t = ks > C::kK ? ks - C::kK : 0; t < ks; ++t) mbar_drain(&sm.k_full[t % C::kK], (t / C::kK) & 1);
        for (uint32_t t = vs > C::kV ? vs - C::kV : 0; t < vs; ++t) mbar_drain(&sm.v_full[t % C::kV], (t / C::kV) & 1);
        for (uint32_t t = ks > kMeta ? ks - kMeta : 0; t < ks; ++t) mbar_drain(&sm.meta_full[t % kMeta], (t / kMeta) & 1);
    }
    __syncwarp();
}

// MMAs, by one thread of each of three warps: QK, and PV into the two halves of O.  A thread needs about 100 cycles to
// form the descriptors of an MMA and issue it, twice what the tensor pipe takes for one, so one thread would bound a tile
// (24 MMAs at 8 tokens).  Each waits for its own operands only: QK of later tiles runs while the softmax works on this one.
template <int R, bool F32>
__device__ void issue_qk(const Bs8Args& a, Smem<R, F32>& sm, Bs8Share w, uint32_t tmem) {
    using C = Cfg<R, F32>;
    const uint64_t kdesc = make_desc(smem_u32(sm.k[0]), 128, 2048), qdesc = make_desc(smem_u32(sm.q), 128, 2048);
    uint32_t it = 0, seg = 0;
    bool ok = true;
    do {
        ok = mbar_wait(&sm.q_full, seg & 1, &sm.abort);
        for (int i = 0; i < w.tiles && ok; ++i) {
            const uint32_t t = it + i, b = t & 1, st = t % C::kK;
            ok = mbar_wait(&sm.k_full[st], (t / C::kK) & 1, &sm.abort);
            if (t >= 2) ok = ok && mbar_wait(&sm.s_free[b], ((t >> 1) + 1) & 1, &sm.abort);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = kdesc + st * (kTileBytes / 16);
#pragma unroll
            for (int k = 0; k < kHeadDim / 32; ++k) mma8(tmem + b * C::kS, ad + k * 16, qdesc + k * 16, idesc8(C::kS, false, false), k > 0);
            mma_commit(&sm.k_free[st]);
            mma_commit(&sm.s_full[b]);
        }
        it += w.tiles;
        ++seg;
    } while (ok && w.next(a));
    mma_commit(&sm.drained);
}

template <int R, bool F32>
__device__ void issue_pv(const Bs8Args& a, Smem<R, F32>& sm, Bs8Share w, uint32_t tmem, int half) {
    using C = Cfg<R, F32>;
    const uint64_t vdesc = make_desc(smem_u32(sm.v[0]) + half * 1024, 2048, 128), pdesc = make_desc(smem_u32(sm.p[0]), C::kBeside * R / 16 * 128, 128);
    const uint64_t pdesc1 = make_desc(smem_u32(sm.p[0]), R / 16 * 128, 128);         // of a last code alone
    const uint32_t o = tmem + C::kO + half * C::kBeside * R;
    uint32_t it = 0;
    bool ok = true;
    do {
        for (int i = 0; i < w.tiles && ok; ++i) {
            const uint32_t t = it + i, st = t % C::kV, pb = t % C::kPBufs;
            ok = mbar_wait(&sm.v_full[st], (t / C::kV) & 1, &sm.abort) && mbar_wait(&sm.p_full[pb], (t / C::kPBufs) & 1, &sm.abort);
            if (!ok) break;
            tc_fence_after();
            const uint64_t ad = vdesc + st * (kTileBytes / 16);
#pragma unroll
            for (int part = 0; part < C::kParts; ++part) {
                const int wide = C::wide(part);
#pragma unroll
                for (int k = 0; k < kBs8Tile / 32; ++k)
                    mma8(o, ad + k * (8192 / 16),
                         (wide == 1 ? pdesc1 : pdesc) + (pb * C::kP + part * C::kBeside) * (R * kBs8Tile / 16) + k * (4 * (wide * R / 16) * 128 / 16),
                         idesc8(wide * R, true, true), (!F32 && i > 0) || part > 0 || k > 0);
            }
            mma_commit(&sm.v_free[st]);
            mma_commit(&sm.p_free[pb]);
        }
        it += w.tiles;
    } while (ok && w.next(a));
    mma_commit(&sm.drained);
}

// The queries of a segment as codes; a row that is not finite gets a NaN scale and comes out as NaN.
template <int R, bool F32>
__device__ void prepare_q(const Bs8Args& a, Smem<R, F32>& sm, const Bs8Share& w, int warp) {
    using C = Cfg<R, F32>;
    using T = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr int kWarps = C::kSoftmax / 32, kEach = R / kWarps, kVecs = F32 ? 2 : 1;
    const int lane = threadIdx.x & 31, heads = a.num_kv_heads;
    const int T0 = w.chunk(heads) * (a.rows / kGroup), nrows = min(R, kGroup * (w.s.T - T0));
    const T* q = static_cast<const T*>(a.q) + (((int64_t)w.s.q0 + T0) * heads * kGroup + w.head(heads) * kGroup) * kHeadDim + 8 * lane;
    auto load = [&](int n, uint4 (&to)[kVecs]) {       // padding rows load the last row
        const int r = min(warp + n * kWarps, nrows - 1);
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            to[v] = reinterpret_cast<const uint4*>(q + ((int64_t)(r >> 3) * heads * kGroup + (r & 7)) * kHeadDim)[v];
    };
    uint4 in[kVecs], next[kVecs], third[kVecs];
    load(0, in);
    load(1, next);
    // rolled, two rows ahead: code that runs once costs its fetch
#pragma unroll 1
    for (int n = 0; n < kEach; ++n) {
        const int r = warp + n * kWarps;
        load(n + 2, third);
        uint32_t x[8];                           // float32 bits
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                const uint4 u = in[F32 ? i >> 1 : 0];
                x[2 * i] = (i & 1) ? u.z : u.x;
                x[2 * i + 1] = (i & 1) ? u.w : u.y;
            } else {
                const uint32_t u = i == 0 ? in[0].x : i == 1 ? in[0].y : i == 2 ? in[0].z : in[0].w;
                x[2 * i] = u << 16;
                x[2 * i + 1] = u & 0xffff0000u;
            }
        }
        // magnitudes are ordered as integers, and what is not finite comes last
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, x[i] & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        const bool finite = top < 0x7f800000u, zero = top == 0 || r >= nrows;
        // largest value to 128 .. 256
        const int k = zero || !finite ? 0 : min(100, 7 - ((int)(top >> 23) - 127));
        const float up = zero ? 0.0f : __uint_as_float((uint32_t)(k + 127) << 23);
        uint8_t* to = sm.q + ((r >> 3) * 16 + (lane >> 1)) * 128 + (r & 7) * 16 + (lane & 1) * 8;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(x[i]) * up;
#pragma unroll
        for (int c = 0; c < C::kQ; ++c) {
            uint32_t code[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                code[i] = e4m3_pair(y[4 * i], y[4 * i + 1]) | (e4m3_pair(y[4 * i + 2], y[4 * i + 3]) << 16);
                if (c + 1 == C::kQ) continue;
                uint32_t h01, h23;
                e4m3x4_to_f16(code[i], h01, h23);
                const float2 f0 = __half22float2(as_h2(h01)), f1 = __half22float2(as_h2(h23));
                const float rest = !F32 ? kQLast : c == 2 ? kQStep : 1.0f;      // float32: the second three codes carry 12 bits less
                y[4 * i] = (y[4 * i] - f0.x) * rest;
                y[4 * i + 1] = (y[4 * i + 1] - f0.y) * rest;
                y[4 * i + 2] = (y[4 * i + 2] - f1.x) * rest;
                y[4 * i + 3] = (y[4 * i + 3] - f1.y) * rest;
            }
            *reinterpret_cast<uint2*>(to + c * R * kHeadDim) = make_uint2(code[0], code[1]);
        }
        if (lane == 0) sm.rs[r] = finite || r >= nrows ? __uint_as_float((uint32_t)(127 - k) << 23) : __int_as_float(0x7fc00000);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            in[v] = next[v];
            next[v] = third[v];
        }
    }
}

// Each of H values reduced over the warp, value (lane / (32 / H)) for each lane: halves are exchanged until one is left.
template <int H, typename Op>
__device__ __forceinline__ float reduce_rows(const float (&in)[H], Op op) {
    const int lane = threadIdx.x & 31;
    float v[H];
#pragma unroll
    for (int c = 0; c < H; ++c) v[c] = in[c];
    int mask = 16;
#pragma unroll
    for (int n = H / 2; n > 0; n >>= 1, mask >>= 1) {
        const bool upper = lane & mask;
#pragma unroll
        for (int c = 0; c < n; ++c) {
            const float other = __shfl_xor_sync(0xffffffffu, upper ? v[c] : v[c + n], mask);
            v[c] = op(upper ? v[c + n] : v[c], other);
        }
    }
#pragma unroll
    for (; mask > 0; mask >>= 1) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], mask));
    return v[0];
}

// One arrival per warp.
__device__ __forceinline__ void warp_arrive(unsigned long long* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Pairs of float32 in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
          "l"(reinterpret_cast<unsigned long long&>(c)));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two floats -> two E5M2 bytes (lo in the low byte); and minus the values of two such bytes.
__device__ __forceinline__ uint32_t e5m2_pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e5m2_negative(uint32_t two) {
    return __half22float2(as_h2(__byte_perm(two, 0, 0x1404) ^ 0x80008000u));
}

// A thread's rows of one half of O: the sums of the codes beside each other, smallest first.
template <int R, bool F32>
__device__ __forceinline__ void outputs(uint32_t lanes, int r0, int half, float* o) {
    using C = Cfg<R, F32>;
    float part[C::kBeside][C::kH];
#pragma unroll
    for (int n = 0; n < C::kBeside; ++n) tmem_load<C::kH>(lanes + C::kO + (half * C::kBeside + n) * R + r0, part[n]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < C::kH; ++c) {
        constexpr int kScaled = F32 ? C::kBeside / 2 : 1;        // columns
        o[c] = part[C::kBeside - 1][c];
#pragma unroll
        for (int n = C::kBeside - 2; n >= 0; --n)
            o[c] = n == C::kBeside - kScaled - 1 ? fmaf(o[c], 1.0f / (F32 ? kPStep : kPLast), part[n][c]) : o[c] + part[n][c];
    }
}

// Float32 outputs leave TMEM after every tile: its accumulators need not round to nearest, and a long context's many
// additions would show that.
template <int R, bool F32>
__device__ __forceinline__ void drain(uint32_t lanes, int r0, float* acc) {
    using C = Cfg<R, F32>;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float o[C::kH];
        outputs<R, F32>(lanes, r0, h, o);
#pragma unroll
        for (int c = 0; c < C::kH; ++c) acc[h * C::kH + c] += o[c];
    }
}

template <int R, bool F32>
__device__ void softmax(const Bs8Args& a, Smem<R, F32>& sm, Bs8Share w, uint32_t tmem) {
    using C = Cfg<R, F32>;
    constexpr int H = C::kH, kAll = 1 + C::kWgs;                     // kAll: barrier of all softmax warps
    const int tid = threadIdx.x - 128, lane = threadIdx.x & 31, warp = tid >> 5, heads = a.num_kv_heads;
    const int wg = warp >> 2, quarter = (threadIdx.x >> 5) & 3;      // rows wg H .., positions 32 quarter ..: a warp reads its own TMEM lanes
    const int p = quarter * 32 + lane, r0 = wg * H, bar = 1 + wg;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t it = 0;
    bool ok = true;
    const auto wait_pv = [&](uint32_t t) { return mbar_wait_fast(&sm.p_free[t % C::kPBufs], (t / C::kPBufs) & 1, &sm.abort); };
    do {
        prepare_q<R, F32>(a, sm, w, warp);
        if (tid < R) sm.m[tid] = 0.0f;
        fence_proxy_async();
        warp_arrive(&sm.q_full);
        named_sync(kAll, C::kSoftmax);     // rs and m are there
        float2 l[H / 2];
#pragma unroll
        for (int c = 0; c < H / 2; ++c) l[c] = both(0.0f);
        float acc[F32 ? 2 * H : 1];        // float32: outputs so far
        if constexpr (F32) {
#pragma unroll
            for (int c = 0; c < 2 * H; ++c) acc[c] = 0.0f;
        }
        const int seen = w.s.L - w.s.T + w.chunk(heads) * (a.rows / kGroup);      // last position that the chunk's first token sees
        bool fresh = true;                 // no tile of the segment has shown a position yet: pages out of range hide theirs
        for (int i = 0; i < w.tiles; ++i, ++it) {
            const uint32_t b = it & 1, slot = it % kMeta;
            const int p0 = (w.tile + i) * kBs8Tile;
            ok = ok && mbar_wait_fast(&sm.meta_full[slot], (it / kMeta) & 1, &sm.abort);
            const float ks = sm.meta[slot][p >> 4] * (1.44269504f / 16.0f);
            // a block behind the context may hold anything
            const int ev = min(kBs8MaxExp, max(-kBs8MaxExp, (int)((__float_as_uint(sm.meta[slot][8 + (p >> 4)]) >> 23) & 0xff) - 127));
            const bool hidden = sm.bad_page[slot] != 0;
            ok = ok && mbar_wait_fast(&sm.s_full[b], (it >> 1) & 1, &sm.abort);
            __syncwarp();
            tc_fence_after();
            float d[H];
            float2* d2 = reinterpret_cast<float2*>(d);
            {
                // the codes' scores, smallest first
                float s2[H];
                tmem_load<H>(lanes + b * C::kS + (C::kQ - 1) * R + r0, d);
#pragma unroll
                for (int q = C::kQ - 2; q >= 0; --q) {
                    tmem_load<H>(lanes + b * C::kS + q * R + r0, s2);
                    tmem_ld_wait();
#pragma unroll
                    for (int c = 0; c < H / 2; ++c)
                        d2[c] = !F32 || q == 2 ? fma2(d2[c], both(1.0f / (F32 ? kQStep : kQLast)), reinterpret_cast<float2*>(s2)[c])
                                               : add2(d2[c], reinterpret_cast<float2*>(s2)[c]);
                }
            }
            tc_fence_before();
            warp_arrive(&sm.s_free[b]);
#pragma unroll
            for (int c = 0; c < H; c += 4) {
                const float4 rs = *reinterpret_cast<const float4*>(&sm.rs[r0 + c]), m = *reinterpret_cast<const float4*>(&sm.m[r0 + c]);
                d2[c / 2] = fma2(mul2(d2[c / 2], make_float2(rs.x, rs.y)), both(ks), add2(both((float)ev), make_float2(m.x, m.y)));
                d2[c / 2 + 1] = fma2(mul2(d2[c / 2 + 1], make_float2(rs.z, rs.w)), both(ks), add2(both((float)ev), make_float2(m.z, m.w)));
            }
            if (hidden || p0 + kBs8Tile > seen + 1) {
                // row r sees positions up to L - T + its token
                const int ahead = hidden ? (1 << 20) : p0 + p - seen;
#pragma unroll
                for (int c = 0; c < H; ++c)
                    if (ahead > ((r0 + c) >> 3) || p0 + p >= w.s.L) d[c] = -CUDART_INF_F;
            }
            float top = d[0];
#pragma unroll
            for (int c = 1; c < H; ++c) top = fmaxf(top, d[c]);
            const bool raise = named_or(bar, 128, fresh || top > kRaise || !ok);
            if (raise) {
                if (named_or(bar, 128, !ok)) {
                    ok = false;
                    break;
                }
                // new maxima of the rows over the tile's positions
                {
                    float t[H];
#pragma unroll
                    for (int c = 0; c < H; ++c) t[c] = d[c] - sm.m[r0 + c];
                    const float x = reduce_rows<H>(t, [](float u, float v) { return fmaxf(u, v); });
                    if (lane % (32 / H) == 0) sm.red[wg][quarter][lane / (32 / H)] = x;
                }
                named_sync(bar, 128);
                if (p < H) {
                    const float x = fmaxf(fmaxf(sm.red[wg][0][p], sm.red[wg][1][p]), fmaxf(sm.red[wg][2][p], sm.red[wg][3][p]));
                    const float m = -sm.m[r0 + p];
                    // the first visible tile sets m; a row that sees nothing of it sees nothing of the segment's later tiles
                    const float now = !fresh ? fmaxf(m, x - kAbove) : x > -CUDART_INF_F ? x - kAbove : 0.0f;
                    sm.m[r0 + p] = -now;
                    sm.dm[r0 + p] = m - now;
                }
                named_sync(bar, 128);
#pragma unroll
                for (int c = 0; c < H / 2; ++c) {
                    const float2 dm = *reinterpret_cast<const float2*>(&sm.dm[r0 + 2 * c]);
                    d2[c] = add2(d2[c], dm);
                    if (!fresh) l[c] = mul2(l[c], make_float2(fast_exp2(dm.x), fast_exp2(dm.y)));
                }
                if (!F32 && !fresh) {
                    ok = wait_pv(it - 1);      // PV of the tile before, and all earlier ones
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int g = 0; g < 2 * C::kBeside * H; g += 8) {
                        const uint32_t at = lanes + C::kO + (g / H) * R + r0 + g % H;
                        float o[8];
                        tmem_load<8>(at, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int c = 0; c < 8; ++c) o[c] *= fast_exp2(sm.dm[r0 + g % H + c]);
                        tmem_store<8>(at, o);
                    }
                    tmem_st_wait();
                }
            }
            const float2 iv = both(__uint_as_float((uint32_t)(127 - ev) << 23));       // 2^-eV
            uint32_t code[C::kP][H / 4];
#pragma unroll
            for (int c = 0; c < H / 4; ++c) {
                float2 x = make_float2(fast_exp2(d[4 * c]), fast_exp2(d[4 * c + 1]));
                float2 y = make_float2(fast_exp2(d[4 * c + 2]), fast_exp2(d[4 * c + 3]));
                l[2 * c] = fma2(x, iv, l[2 * c]);
                l[2 * c + 1] = fma2(y, iv, l[2 * c + 1]);
                if constexpr (F32) {
#pragma unroll
                    for (int n = 0; n < C::kP; ++n) {
                        code[n][c] = e5m2_pair(x.x, x.y) | (e5m2_pair(y.x, y.y) << 16);
                        if (n + 1 == C::kP) break;
                        x = add2(x, e5m2_negative(code[n][c]));
                        y = add2(y, e5m2_negative(code[n][c] >> 16));
                        if (n == 2) {                // exact; without it a weight below 2^-25 of the largest would be gone
                            x = mul2(x, both(kPStep));
                            y = mul2(y, both(kPStep));
                        }
                    }
                } else {
                    // E5M2 is the upper byte of fp16, and half a step of it is 0x80, whatever the sign.  (A NaN's codes become
                    // zeros: the row sum keeps it.)
                    constexpr uint32_t kHalf = 0x00800080u, kByte = 0xff00ff00u;
                    const uint32_t lo = f16_pair(x.x, x.y), hi = f16_pair(y.x, y.y), a0 = lo + kHalf, b0 = hi + kHalf;
                    const uint32_t ar = sub2(lo, a0 & kByte), br = sub2(hi, b0 & kByte), a1 = ar + kHalf, b1 = br + kHalf;
                    const uint32_t a2 = last2(sub2(ar, a1 & kByte)) + kHalf, b2 = last2(sub2(br, b1 & kByte)) + kHalf;
                    code[0][c] = __byte_perm(a0, b0, 0x7531);
                    code[1][c] = __byte_perm(a1, b1, 0x7531);
                    code[2][c] = __byte_perm(a2, b2, 0x7531);
                }
            }
            if (it >= C::kPBufs) ok = ok && wait_pv(it - C::kPBufs);
            if constexpr (F32) {
                __syncwarp();
                tc_fence_after();
                if (i > 0) drain<R, F32>(lanes, r0, acc);
                if (raise && !fresh) {           // before, there is nothing to scale, and the factor may be infinite
#pragma unroll
                    for (int c = 0; c < 2 * H; ++c) acc[c] *= fast_exp2(sm.dm[r0 + c % H]);
                }
            }
            uint8_t* pb = sm.p[it % C::kPBufs] + (r0 / 16) * 128 + (p & 7) * 16 + (r0 & 15);
#pragma unroll
            for (int n = 0; n < C::kP; ++n) {
                const int part = C::part(n);
                uint8_t* to = pb + part * C::kBeside * R * kBs8Tile + C::column(n) * (R / 16 * 128) + (p >> 3) * (C::wide(part) * R / 16 * 128);
                if constexpr (H == 8) *reinterpret_cast<uint2*>(to) = make_uint2(code[n][0], code[n][1]);
                else *reinterpret_cast<uint4*>(to) = make_uint4(code[n][0], code[n][1], code[n][2], code[n][3]);
            }
            const int valid = hidden ? 0 : w.s.L - p0;
            if (valid < kBs8Tile) {
                // rows behind the context may hold anything, and 0 x NaN is NaN: they become zeros before PV reads them
                const uint32_t st = it % C::kV;
                ok = ok && mbar_wait_fast(&sm.v_full[st], (it / C::kV) & 1, &sm.abort);      // PV of the tile kV before is done
                if (p >= valid) {
                    for (int c = wg; c < kHeadDim / 16; c += C::kWgs)
                        *reinterpret_cast<uint4*>(sm.v[st] + ((p >> 3) * 16 + c) * 128 + (p & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async();
            tc_fence_before();
            warp_arrive(&sm.p_full[it % C::kPBufs]);
            fresh = fresh && hidden;
        }
        ok = ok && wait_pv(it - 1);
        if (named_or(kAll, C::kSoftmax, !ok)) {      // all softmax warps leave together
            ok = false;
            break;
        }
        tc_fence_after();
        if constexpr (F32) drain<R, F32>(lanes, r0, acc);
        // row sums over the positions
        {
            const float x = reduce_rows<H>(reinterpret_cast<float (&)[H]>(l), [](float u, float v) { return u + v; });
            if (lane % (32 / H) == 0) sm.red[wg][quarter][lane / (32 / H)] = x;
        }
        named_sync(bar, 128);
        const int T0 = w.chunk(heads) * (a.rows / kGroup), nrows = min(R, kGroup * (w.s.T - T0));
        const bool whole = w.whole();
        float* part = a.partials + ((size_t)blockIdx.x * 2 + w.part()) * kBs8PartFloats;
        using T = std::conditional_t<F32, float, __nv_bfloat16>;
        T* out = static_cast<T*>(a.out) + (((int64_t)w.s.q0 + T0) * heads * kGroup + w.head(heads) * kGroup) * kHeadDim;
        if (p < H) {                       // one thread per row; then all read their rows' factors
            const float mine = (sm.red[wg][0][p] + sm.red[wg][1][p]) + (sm.red[wg][2][p] + sm.red[wg][3][p]);
            if (!whole && r0 + p < nrows)
                *reinterpret_cast<float2*>(part + kBs8Rows * kHeadDim + 2 * (r0 + p)) =
                    make_float2(mine != 0.0f ? -sm.m[r0 + p] : -CUDART_INF_F, mine);      // an empty partial weighs nothing
            sm.dm[r0 + p] = mine != 0.0f ? __fdividef(1.0f, mine) : 0.0f;
        }
        named_sync(bar, 128);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float o[H];
            if constexpr (F32) {
#pragma unroll
                for (int c = 0; c < H; ++c) o[c] = acc[h * H + c];
            } else {
                outputs<R, F32>(lanes, r0, h, o);
            }
            if (whole) {
                T* to = out + ((int64_t)(r0 >> 3) * heads * kGroup) * kHeadDim + h * 128 + p;
#pragma unroll
                for (int c = 0; c < H; ++c)
                    if (r0 + c < nrows) to[((int64_t)(c >> 3) * heads * kGroup + (c & 7)) * kHeadDim] = (T)(o[c] * sm.dm[r0 + c]);
            } else {
                float* to = part + r0 * kHeadDim + h * 128 + p;
                if (r0 + H <= nrows) {
#pragma unroll
                    for (int c = 0; c < H; ++c) to[c * kHeadDim] = o[c];
                } else {
#pragma unroll
                    for (int c = 0; c < H; ++c)
                        if (r0 + c < nrows) to[c * kHeadDim] = o[c];
                }
            }
        }
        tc_fence_before();
        named_sync(kAll, C::kSoftmax);     // all groups are done with rs, m and red before the next segment's queries
    } while (w.next(a));
    if (!ok && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_TIMEOUT);
}

template <int R, bool F32>
__global__ void __launch_bounds__(Cfg<R, F32>::kThreads, 1) verify_bs8_mma_kernel(Bs8Args a) {
    using C = Cfg<R, F32>;
    extern __shared__ uint8_t raw[];
    Smem<R, F32>& sm = *reinterpret_cast<Smem<R, F32>*>((reinterpret_cast<uintptr_t>(raw) + 127) & ~(uintptr_t)127);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 32) {
        for (int i = 0; i < C::kK; ++i) {
            mbar_init(&sm.k_full[i], 1);
            mbar_init(&sm.k_free[i], 1);
        }
        for (int i = 0; i < C::kV; ++i) {
            mbar_init(&sm.v_full[i], 1);
            mbar_init(&sm.v_free[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], C::kSoftmax / 32);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.p_full[i], C::kSoftmax / 32);
            mbar_init(&sm.p_free[i], 2);
        }
        mbar_init(&sm.q_full, C::kSoftmax / 32);
        mbar_init(&sm.drained, 3);
        for (int i = 0; i < kMeta; ++i) mbar_init(&sm.meta_full[i], 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(&sm.tmem, C::kTmem);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // only now: the merge reads the lengths before its own wait, and whoever writes them is done here
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (warp == 0) {
        bool bad = false;
        const Bs8Share w = bs8_share(a, blockIdx.x, &bad);
        if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        if (threadIdx.x == 0) sm.first = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const Bs8Share w = sm.first;
    const uint32_t tmem = sm.tmem;
    if (w.tiles > 0) {
        if (warp == 0) {
            produce<R, F32>(a, sm, w);
        } else if (warp < 4) {
            if ((threadIdx.x & 31) == 0) {
                if (warp == 1) issue_qk<R, F32>(a, sm, w, tmem);
                else issue_pv<R, F32>(a, sm, w, tmem, warp - 2);
                mbar_drain(&sm.drained, 0);        // TMEM and the operands stay until the last MMA is done
            }
            __syncwarp();
        } else {
            softmax<R, F32>(a, sm, w, tmem);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::kTmem);
}

template <int R, bool F32>
cudaError_t launch_r(const Bs8Args& a, cudaStream_t st) {
    constexpr size_t smem = sizeof(Smem<R, F32>) + 128;
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    static std::atomic<bool> allowed[kMaxDevices];
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(verify_bs8_mma_kernel<R, F32>), smem, allowed);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.ctas);
    cfg.blockDim = dim3(Cfg<R, F32>::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_bs8_mma_kernel<R, F32>, a);
}

}  // namespace

// More than 64 rows are two chunks alike, so that 9 to 12 tokens take 48 rows each instead of 64 and a rest.
int bs8_mma_rows(int dtype, int max_n_q) {
    if (dtype == Q3KV_F32) return 32;
    return kGroup * max_n_q > kBs8Rows && kGroup * max_n_q <= 96 ? 48 : kBs8Rows;
}

cudaError_t launch_bs8_mma(const Bs8Args& a, cudaStream_t st) {
    const int rows = kGroup * a.max_n_q;
    if (a.dtype == Q3KV_F32) return rows <= 16 ? launch_r<16, true>(a, st) : launch_r<32, true>(a, st);
    if (rows <= 32) return rows <= 16 ? launch_r<16, false>(a, st) : launch_r<32, false>(a, st);
    return rows <= 48 || a.rows == 48 ? launch_r<48, false>(a, st) : launch_r<64, false>(a, st);
}

}  // namespace q3kv
