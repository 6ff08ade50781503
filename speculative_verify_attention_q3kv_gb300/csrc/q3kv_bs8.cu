// The block-scaled 8-bit cache: append, the CUDA-core leg of its verify attention, the merge and the entry points.
//
// Format.  A block is 16 consecutive positions of one kv head, K or V.  Its scale is 2^e with the smallest e in
// [-64, 64] for which no |x| of the block is above 448 2^e; the codes are E4M3 of x 2^-e.  A code that is itself a
// floating-point number gains nothing from a scale's fraction, and a power of two makes a rescaling exact but
// for codes that fall under E4M3's smallest normal value: so a block can grow by appends.  When the rows appended
// to a block that holds earlier rows need a larger e, the earlier codes are rewritten for it; e never falls within a
// block (a rejected draft may leave it larger than the rows that stay need).
//
// A NaN in V would reach rows that do not see its position (0 x NaN is NaN in the product with the weights), one in K
// only rows that do.  So a V NaN is stored as a zero there and a NaN in K's code of the same position and dim.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "q3kv_bs8.cuh"

namespace q3kv {
namespace {

// ---------------------------------------------------------------- append
// One CTA per (block, slot, kv head), a thread per row and 16 dims of K and V: it reads 32 or 64 neighbouring bytes of
// each, and a warp writes four whole cores (512 bytes).  Bound: latency and issue slots together (8 prompts of up to 4,096,
// bf16: 14.9 us, 4,200 GB/s; 1 of 30,000 18.7 us, 4,900 GB/s; float32 8 x 4,096 30, 5,600).  A row's 32 bytes come in one load, also
// because lanes that lie 32 bytes apart fetch each sector twice with 16-byte loads (16.1 us; float32 34).
constexpr int kAppendThreads = 256;

// Sixteen values as they lie in memory: fewer registers than float32 (bf16) while they wait for the block's maximum.
template <typename T>
struct Raw16 {
    static constexpr int kWords = (int)sizeof(T) * 4;
    uint32_t w[kWords];
    // wide: src is on 32 bytes
    __device__ __forceinline__ void load(const T* src, bool wide) {
        if (wide) {
#pragma unroll
            for (int i = 0; i < kWords; i += 8)
                asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                             : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]), "=r"(w[i + 6]), "=r"(w[i + 7])
                             : "l"(reinterpret_cast<const uint32_t*>(src) + i));
            return;
        }
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(src) + i);
            w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    // NaNs become zeros here and NaNs in k
    __device__ __forceinline__ void nan_to(Raw16& k) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float v = at(i);
            if (v == v) continue;
            if constexpr (sizeof(T) == 4) {
                k.w[i] = 0x7fc00000u;
                w[i] = 0u;
            } else {
                const uint32_t half = (i & 1) ? 0xffff0000u : 0x0000ffffu;
                k.w[i >> 1] = (k.w[i >> 1] & ~half) | (0x7fc07fc0u & half);
                w[i >> 1] &= ~half;
            }
        }
    }
    // largest finite magnitude, as float32 bits (which are in the magnitudes' order)
    __device__ __forceinline__ uint32_t top(bool* finite) const {
        uint32_t m = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);       // two values at a time
            m = max(m & 0xffff0000u, m << 16);
        }
        if (m >= 0x7f800000u) {
            *finite = false;
            m = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t u = __float_as_uint(at(i)) & 0x7fffffffu;
                m = max(m, u < 0x7f800000u ? u : 0u);
            }
        }
        return m;
    }
};

// Two floats -> two E4M3 bytes (lo in the low byte), to nearest even, magnitudes above 448 to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float2 times(float a, float b, float f) {       // both products in one instruction
    float2 x = make_float2(a, b), y = make_float2(f, f), r;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<unsigned long long&>(r))
        : "l"(reinterpret_cast<unsigned long long&>(x)), "l"(reinterpret_cast<unsigned long long&>(y)));
    return r;
}
template <typename At>
__device__ __forceinline__ uint4 encode16(At x, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = times(x(4 * i), x(4 * i + 1), inv), hi = times(x(4 * i + 2), x(4 * i + 3), inv);
        w[i] = __byte_perm(e4m3x2(lo.x, lo.y), e4m3x2(hi.x, hi.y), 0x5410);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int scale_exp(float s) {       // of a stored scale, whatever its bytes hold
    return min(kBs8MaxExp, max(-kBs8MaxExp, (int)((__float_as_uint(s) >> 23) & 0xff) - 127));
}

template <typename T>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 2 ? 6 : 4) append_bs8_kernel(AppendArgs a) {
    __shared__ __align__(16) uint32_t s_max[2][kAppendThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int slot = blockIdx.y, head = blockIdx.z;
    const int n_new = a.n_new[slot], len = a.slot_len[slot], first_row = a.row_offsets[slot];
    if (n_new == 0) return;
    const bool report = blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0 && a.status;
    if (n_new < 0 || n_new > a.max_n_new || len < 0 || first_row < 0) {
        if (report) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        return;
    }
    // positions as unsigned 32-bit numbers; those behind the table are skipped
    const uint32_t room = (uint32_t)min((int64_t)a.max_pages_per_slot * kPageSize, (int64_t)INT32_MAX + 1), want = (uint32_t)len + (uint32_t)n_new;
    if (want > room && report) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
    const uint32_t end = min(want, room), p0 = ((uint32_t)len / kBs8Block + blockIdx.x) * kBs8Block;
    if (p0 >= end) return;
    const int32_t page = a.page_table[(int64_t)slot * a.max_pages_per_slot + p0 / kPageSize];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t row = (warp & 1) * 8 + (lane & 7), chunk = (warp >> 1) * 4 + (lane >> 3);
    const uint32_t pos = p0 + row;
    const bool kept = pos < (uint32_t)len, fresh = !kept && pos < end;
    Raw16<T> x[2];
    if (fresh) {
        const int64_t at = ((int64_t)(first_row + (int)(pos - (uint32_t)len)) * a.num_kv_heads + head) * kHeadDim + chunk * 16;
        const bool wide = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 31) == 0;
        x[0].load(static_cast<const T*>(a.k) + at, wide);
        x[1].load(static_cast<const T*>(a.v) + at, wide);
    }
    if (page < 0 || page >= a.num_pages) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
        return;
    }
    uint8_t* unit = a.pool + bs8_offset(a.num_layers, a.num_kv_heads, page, a.layer, head, 0);
    const uint32_t in_page = p0 % kPageSize;
    uint8_t* code = unit + ((in_page + row) / 8 * 16 + chunk) * 128 + (row % 8) * 16;
    uint8_t* scale = unit + kBs8CodeBytes + 4 * (in_page / kBs8Block);
    int old[2] = {-kBs8MaxExp, -kBs8MaxExp};
    uint4 was[2];
    if (p0 < (uint32_t)len) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            old[kv] = scale_exp(*reinterpret_cast<const float*>(scale + kv * kBs8UnitBytes));
            if (kept) was[kv] = *reinterpret_cast<const uint4*>(code + kv * kBs8UnitBytes);
        }
    }
    bool finite = true;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, fresh ? x[kv].top(&finite) : 0u);
        if (lane == 0) s_max[kv][warp] = top;
    }
    if (!finite) x[1].nan_to(x[0]);
    if (!__all_sync(0xffffffffu, finite) && lane == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
    __syncthreads();
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const uint4 lo = reinterpret_cast<const uint4*>(s_max[kv])[0], hi = reinterpret_cast<const uint4*>(s_max[kv])[1];
        const uint32_t u = max(max(max(lo.x, lo.y), max(lo.z, lo.w)), max(max(hi.x, hi.y), max(hi.z, hi.w)));
        // top = m 2^k with 1 <= m < 2 and 448 = 1.75 2^8; zero and subnormal values give the smallest e
        const int need = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
        if (need > kBs8MaxExp && threadIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_SCALE_OVERFLOW);
        const int e = min(kBs8MaxExp, max(old[kv], need));
        if (fresh) {
            *reinterpret_cast<uint4*>(code + kv * kBs8UnitBytes) = encode16([&](int i) { return x[kv].at(i); }, pow2(-e));
        } else if (kept && e != old[kv]) {
            const uint32_t w[4] = {was[kv].x, was[kv].y, was[kv].z, was[kv].w};
            *reinterpret_cast<uint4*>(code + kv * kBs8UnitBytes) = encode16([&](int i) {
                const float2 f = e4m3x2_to_f32((w[i >> 2] >> (16 * ((i >> 1) & 1))) & 0xffffu);
                return (i & 1) ? f.y : f.x;
            }, pow2(max(old[kv] - e, -126)));
        }
        if (threadIdx.x == 0) *reinterpret_cast<float*>(scale + kv * kBs8UnitBytes) = pow2(e);
    }
}

// ---------------------------------------------------------------- verify attention on CUDA cores
// The reference leg: float32 arithmetic throughout.  One CTA per share; sub-tiles of 64 positions are decoded to
// shared memory.  Bound: the FMAs of 64 rows x 64 positions x 256 dims, twice; each thread holds 4 x 4 scores and
// 8 x 8 outputs, so that two shared 16-byte loads feed 8 (scores) or 16 (outputs) FMAs each.
constexpr int kFmaThreads = 256;
constexpr int kSub = 64;                  // positions per sub-tile
constexpr int kLd = kHeadDim + 4;         // floats per row in shared memory: neighbouring rows start 4 banks apart
constexpr int kLdP = kBs8Rows + 4;
// A row's maximum before its first position: finite, and times log2(e) too, so that a row that sees nothing takes no difference
// of infinities and a row of NaNs is no empty partial.
constexpr float kLowest = -2.35e38f;
struct FmaSmem {
    float q[kBs8Rows * kLd];
    float kv[kSub * kLd];
    float p[kSub * kLdP];                 // [position][row]
    float m[kBs8Rows], l[kBs8Rows], f[kBs8Rows];
    Bs8Share first;
};

__device__ __forceinline__ float ld_any(const void* p, int64_t i, int dtype) {
    return dtype == Q3KV_F32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void st4(void* p, int64_t i, int dtype, float4 v) {
    if (dtype == Q3KV_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
    } else {
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p) + i) = *reinterpret_cast<uint2*>(h);
    }
}

// 64 positions from p0 of a unit into shared memory as float32; positions from `valid` on become zero.
__device__ __forceinline__ void decode_sub(const uint8_t* unit, int in_page, int valid, float* dst) {
    const float* scales = reinterpret_cast<const float*>(unit + kBs8CodeBytes);
    for (int i = threadIdx.x; i < kSub * 16; i += kFmaThreads) {
        const int row = (i >> 7) * 8 + (i & 7), chunk = (i >> 3) & 15;         // memory order
        float* to = dst + row * kLd + chunk * 16;
        float4 o[4];
        if (unit && row < valid) {
            const uint4 c = *reinterpret_cast<const uint4*>(unit + (((in_page + row) >> 3) * 16 + chunk) * 128 + (row & 7) * 16);
            const float s = scales[(in_page + row) / kBs8Block];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 lo = e4m3x2_to_f32(w[j] & 0xffffu), hi = e4m3x2_to_f32(w[j] >> 16);
                o[j] = make_float4(lo.x * s, lo.y * s, hi.x * s, hi.y * s);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) reinterpret_cast<float4*>(to)[j] = o[j];
    }
}

__global__ void __launch_bounds__(kFmaThreads) verify_bs8_fma_kernel(Bs8Args a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    FmaSmem& sm = *reinterpret_cast<FmaSmem*>(smem_raw);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");      // after the wait: the merge reads the lengths before its own
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 0) {
        bool bad = false;
        const Bs8Share w = bs8_share(a, blockIdx.x, &bad);
        if (bad && blockIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        if (lane == 0) sm.first = w;
    }
    __syncthreads();
    Bs8Share w = sm.first;
    if (w.tiles == 0) return;
    const int heads = a.num_kv_heads, qheads = heads * kGroup;
    const int ry = tid >> 4, px = tid & 15;               // scores: rows 4 ry.., positions px + 16 j
    const int rows8 = (tid >> 5) * 8;                     // outputs: 8 rows, dims 4 lane.. and 128 + 4 lane..
    do {
        const int T0 = w.chunk(heads) * (kBs8Rows / kGroup), head = w.head(heads);
        const int nrows = min(kBs8Rows, kGroup * (w.s.T - T0));
        const int64_t q0 = (int64_t)w.s.q0 + T0;
        __syncthreads();                                  // the last segment's outputs are read
        for (int i = tid; i < kBs8Rows * kHeadDim; i += kFmaThreads) {
            const int r = i >> 8, d = i & 255;
            const float x = r < nrows ? ld_any(a.q, ((q0 + (r >> 3)) * qheads + head * kGroup + (r & 7)) * kHeadDim + d, a.dtype) : 0.0f;
            // an infinity as a NaN: against keys of one sign it would hide every position (all scores -inf)
            sm.q[r * kLd + d] = isinf(x) ? CUDART_NAN_F : x * 0.0625f;
        }
        if (tid < kBs8Rows) {
            sm.m[tid] = kLowest;
            sm.l[tid] = 0.0f;
        }
        float o[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) o[i][j] = 0.0f;
        const int pos_end = min(w.s.L, (w.tile + w.tiles) * kBs8Tile);
        for (int p0 = w.tile * kBs8Tile; p0 < pos_end; p0 += kSub) {
            const int valid = min(kSub, w.s.L - p0);
            const int32_t page = a.page_table[(int64_t)w.slot * a.max_pages_per_slot + p0 / kPageSize];
            const bool good = page >= 0 && page < a.num_pages;
            if (!good && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
            const uint8_t* unit = good ? a.pool + bs8_offset(a.num_layers, heads, page, a.layer, head, 0) : nullptr;
            __syncthreads();                              // q is there; the last sub-tile is read
            decode_sub(unit, p0 % kPageSize, valid, sm.kv);
            __syncthreads();
            float s[4][4] = {};
            for (int d = 0; d < kHeadDim; d += 4) {
                float4 qv[4], kv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qv[i] = *reinterpret_cast<const float4*>(sm.q + (4 * ry + i) * kLd + d);
                    kv[i] = *reinterpret_cast<const float4*>(sm.kv + (px + 16 * i) * kLd + d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
                        s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
                        s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
                        s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
                    }
            }
            // row 4 ry + i: its 64 scores are held by the 16 threads of half a warp
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * ry + i;
                const int last = good ? w.s.L - w.s.T + T0 + (r >> 3) - p0 : -1;        // last visible position of the sub-tile
                float top = -CUDART_INF_F;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = px + 16 * j;
                    if (p > last || p >= valid) s[i][j] = -CUDART_INF_F;
                    top = fmaxf(top, s[i][j]);
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float m0 = sm.m[r], m1 = fmaxf(m0, top);
                float sum = 0.0f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = expf(s[i][j] - m1);
                    sum += p;
                    sm.p[(px + 16 * j) * kLdP + r] = p;
                }
#pragma unroll
                for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                __syncwarp();
                if (px == 0) {
                    const float f = expf(m0 - m1);
                    sm.f[r] = f;
                    sm.m[r] = m1;
                    sm.l[r] = fmaf(sm.l[r], f, sum);
                }
            }
            __syncthreads();
            decode_sub(good ? unit + kBs8UnitBytes : nullptr, p0 % kPageSize, valid, sm.kv);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = sm.f[rows8 + i];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[i][j] *= f;
            }
#pragma unroll 4
            for (int p = 0; p < kSub; ++p) {
                const float4 p0v = *reinterpret_cast<const float4*>(sm.p + p * kLdP + rows8);
                const float4 p1v = *reinterpret_cast<const float4*>(sm.p + p * kLdP + rows8 + 4);
                const float4 v0 = *reinterpret_cast<const float4*>(sm.kv + p * kLd + 4 * lane);
                const float4 v1 = *reinterpret_cast<const float4*>(sm.kv + p * kLd + 128 + 4 * lane);
                const float pr[8] = {p0v.x, p0v.y, p0v.z, p0v.w, p1v.x, p1v.y, p1v.z, p1v.w};
                const float vr[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[i][j] = fmaf(pr[i], vr[j], o[i][j]);
            }
        }
        __syncthreads();
        const bool whole = w.whole();
        float* part = a.partials + ((size_t)blockIdx.x * 2 + w.part()) * kBs8PartFloats;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = rows8 + i;
            if (r >= nrows) break;
            const float l = sm.l[r], n = whole ? (l != 0.0f ? 1.0f / l : 0.0f) : 1.0f;
            const float4 lo = make_float4(o[i][0] * n, o[i][1] * n, o[i][2] * n, o[i][3] * n);
            const float4 hi = make_float4(o[i][4] * n, o[i][5] * n, o[i][6] * n, o[i][7] * n);
            if (whole) {
                const int64_t at = ((q0 + (r >> 3)) * qheads + head * kGroup + (r & 7)) * kHeadDim + 4 * lane;
                st4(a.out, at, a.dtype, lo);
                st4(a.out, at + 128, a.dtype, hi);
            } else {
                *reinterpret_cast<float4*>(part + r * kHeadDim + 4 * lane) = lo;
                *reinterpret_cast<float4*>(part + r * kHeadDim + 128 + 4 * lane) = hi;
                if (lane == 0) *reinterpret_cast<float2*>(part + kBs8Rows * kHeadDim + 2 * r) = make_float2(l != 0.0f ? sm.m[r] * 1.44269504f : -CUDART_INF_F, l);
            }
        }
    } while (w.next(a));
}

// ---------------------------------------------------------------- merge
// out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the partials of a cut pair.  A group of 64 threads loads its
// partials of a row together with their maxima, ten at a time, and groups that share a row agree on M at the end.
// Bound: latency.  Few rows (one slot): eight groups per row and one row per CTA, so that 80 partials of a row are under
// way at once; many rows, which then have few partials each: a group per row, four rows per CTA, so that few CTAs come and
// go (1,280 rows of 5 slots: 19 us with a CTA each, 7 so; 128 rows of 76 partials: 6 us with a CTA each).
constexpr int kMergeBatch = 10;

template <int GROUPS, int ROWS>          // groups per row, rows per CTA
__global__ void __launch_bounds__(64 * GROUPS * ROWS) merge_bs8_kernel(Bs8Args a) {
    __shared__ float4 s_o[GROUPS][64];
    __shared__ float2 s_ml[GROUPS];
    __shared__ uint64_t s_at[2];                 // tiles before the slot, and of all slots
    // The lengths were complete before the verify kernel let this one start; its partials are after the wait.  Every CTA
    // waits, also one without work: whoever follows this kernel goes by its end.
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, heads = a.num_kv_heads;
    const int col = tid & 63, group = (tid >> 6) % GROUPS;
    const int slot = blockIdx.z, pair = blockIdx.y, r = blockIdx.x * ROWS + (tid >> 6) / GROUPS;
    const Bs8Slot s = bs8_slot(a, slot, nullptr);
    const int T0 = pair / heads * (a.rows / kGroup), head = pair % heads;
    if (warp < 2) {
        const int upto = warp == 0 ? slot : a.num_slots;
        const uint64_t n = a.narrow ? bs8_tiles_before<uint32_t>(a, upto, nullptr) : bs8_tiles_before<uint64_t>(a, upto, nullptr);
        if (lane == 0) s_at[warp] = n;
    }
    __syncthreads();
    int c0 = 0, c1 = 0;
    if (pair < s.pairs(heads)) {
        const uint64_t total = s_at[1], begin = s_at[0] + (uint64_t)pair * s.tiles, last = begin + s.tiles - 1;
        if (a.narrow) {
            const uint32_t n = (uint32_t)total, G = bs8_ctas(a, n);
            c0 = bs8_cta_of((uint32_t)begin, n, G);
            c1 = bs8_cta_of((uint32_t)last, n, G);
        } else {
            const uint64_t G = bs8_ctas(a, total);
            c0 = bs8_cta_of(begin, total, G);
            c1 = bs8_cta_of(last, total, G);
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (c0 == c1) return;                        // nothing here, or the pair was not cut
    if (r >= min(a.rows, kGroup * (s.T - T0))) return;       // a CTA of several rows has no barrier from here on
    const int n = c1 - c0 + 1;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float m = -CUDART_INF_F, l = 0.0f;
    for (int i0 = group; i0 < n; i0 += GROUPS * kMergeBatch) {
        float4 v[kMergeBatch];
        float2 ml[kMergeBatch];
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const int i = i0 + k * GROUPS;
            if (i < n) {                         // the pair's first CTA ends inside it, the others begin inside it
                const float* p = a.partials + ((size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) * kBs8PartFloats;
                ml[k] = *reinterpret_cast<const float2*>(p + kBs8Rows * kHeadDim + 2 * r);
                v[k] = *reinterpret_cast<const float4*>(p + r * kHeadDim + 4 * col);
            } else {
                ml[k] = make_float2(-CUDART_INF_F, 0.0f);
                v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) top = fmaxf(top, ml[k].x);
        if (top == -CUDART_INF_F) continue;      // empty partials
        const float f0 = exp2f(m - top);
        m = top;
        l *= f0;
        o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
#pragma unroll
        for (int k = 0; k < kMergeBatch; ++k) {
            const float f = exp2f(ml[k].x - top);
            l = fmaf(f, ml[k].y, l);
            o.x = fmaf(f, v[k].x, o.x);
            o.y = fmaf(f, v[k].y, o.y);
            o.z = fmaf(f, v[k].z, o.z);
            o.w = fmaf(f, v[k].w, o.w);
        }
    }
    if constexpr (GROUPS > 1) {
        s_o[group][col] = o;
        if (col == 0) s_ml[group] = make_float2(m, l);
        __syncthreads();
        if (tid >= 64) return;
        float top = -CUDART_INF_F;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) top = fmaxf(top, s_ml[g].x);
        if (top == -CUDART_INF_F) top = 0.0f;    // the row saw nothing
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        l = 0.0f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const float f = exp2f(s_ml[g].x - top);
            const float4 v = s_o[g][col];
            l = fmaf(f, s_ml[g].y, l);
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
    }
    const float inv = l != 0.0f ? 1.0f / l : 0.0f;
    const int64_t at = (((int64_t)s.q0 + T0 + (r >> 3)) * heads * kGroup + head * kGroup + (r & 7)) * kHeadDim + 4 * col;
    st4(a.out, at, a.dtype, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
}

template <typename K, typename A>
cudaError_t launch(K kernel, const A& a, dim3 grid, int threads, size_t smem, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// The merge's grid covers every pair that may be cut.
cudaError_t launch_merge_bs8(const Bs8Args& a, cudaStream_t st) {
    const int chunks = (kGroup * a.max_n_q + a.rows - 1) / a.rows, pairs = chunks * a.num_kv_heads;
    const int rows = chunks > 1 ? a.rows : kGroup * a.max_n_q;
    if ((int64_t)rows * pairs * a.num_slots > 2 * a.ctas)
        return launch(merge_bs8_kernel<1, 4>, a, dim3((unsigned)((rows + 3) / 4), (unsigned)pairs, (unsigned)a.num_slots), 256, 0, st);
    return launch(merge_bs8_kernel<8, 1>, a, dim3((unsigned)rows, (unsigned)pairs, (unsigned)a.num_slots), 512, 0, st);
}

int bs8_check(const q3kv_cache_desc* d, int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t impl) {
    const int e = check_desc(d);
    if (e != Q3KV_OK) return e;
    if (num_slots < 0 || max_ctx_len < 0 || max_n_q < 0) return Q3KV_ERR_INVALID_ARG;
    if (max_ctx_len > (int64_t)INT32_MAX - kPageSize) return Q3KV_ERR_INVALID_ARG;
    if (impl < Q3KV_IMPL_AUTO || impl > Q3KV_IMPL_MMA) return Q3KV_ERR_INVALID_ARG;
    if (num_slots > 65535 || max_n_q > kMaxNq) return Q3KV_ERR_UNSUPPORTED;
    return Q3KV_OK;
}

// A buffer that a call writes shares a byte with its page table, its lists or its status.
bool over_lists(const void* buffer, int64_t bytes, const int32_t* table, int32_t pages_per_slot, const int32_t* lengths, const int32_t* counts,
                const int32_t* offsets, int32_t num_slots, const int32_t* status) {
    const int64_t list = 4 * (int64_t)num_slots;
    return overlap(buffer, bytes, table, list * pages_per_slot) || overlap(buffer, bytes, lengths, list) || overlap(buffer, bytes, counts, list) ||
           overlap(buffer, bytes, offsets, list) || (status && overlap(buffer, bytes, status, 4));
}

size_t bs8_pool_size(const q3kv_cache_desc* d) { return (size_t)d->num_pages * d->num_layers * d->num_kv_heads * 2 * kBs8UnitBytes; }

size_t bs8_partials(int ctas) { return (size_t)ctas * 2 * kBs8PartFloats * sizeof(float); }

}  // namespace

cudaError_t launch_bs8_fma(const Bs8Args& a, cudaStream_t st) {
    static std::atomic<bool> allowed[kMaxDevices];
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(verify_bs8_fma_kernel), sizeof(FmaSmem), allowed);
    if (e != cudaSuccess) return e;
    return launch(verify_bs8_fma_kernel, a, dim3((unsigned)a.ctas), kFmaThreads, sizeof(FmaSmem), st);
}

}  // namespace q3kv

extern "C" {

int q3kv_bs8_pool_bytes(const q3kv_cache_desc* desc, size_t* bytes) {
    int e = q3kv::check_desc(desc);
    if (e != Q3KV_OK) return e;
    if (!bytes) return Q3KV_ERR_INVALID_ARG;
    *bytes = q3kv::bs8_pool_size(desc);
    return Q3KV_OK;
}

int q3kv_bs8_append(void* stream, const q3kv_cache_desc* desc, void* d_pool, const int32_t* d_page_table, int32_t max_pages_per_slot,
                    const int32_t* d_slot_len, const int32_t* d_n_new, const int32_t* d_row_offsets, int32_t num_slots,
                    int32_t max_n_new, int32_t layer, const void* k, const void* v, int32_t dtype, int32_t* d_status) {
    using namespace q3kv;
    int e = check_desc(desc);
    if (e != Q3KV_OK) return e;
    if (num_slots < 0 || max_n_new < 0 || max_pages_per_slot <= 0) return Q3KV_ERR_INVALID_ARG;
    if (num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (layer < 0 || layer >= desc->num_layers) return Q3KV_ERR_INVALID_ARG;
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (num_slots == 0 || max_n_new == 0) return Q3KV_OK;
    if (!d_pool || !d_page_table || !d_slot_len || !d_n_new || !d_row_offsets || !k || !v) return Q3KV_ERR_INVALID_ARG;
    if (!aligned16(d_pool) || !aligned16(k) || !aligned16(v)) return Q3KV_ERR_INVALID_ARG;
    const int64_t pool_bytes = (int64_t)bs8_pool_size(desc);          // of k and v the call knows where they begin
    if (over_lists(d_pool, pool_bytes, d_page_table, max_pages_per_slot, d_slot_len, d_n_new, d_row_offsets, num_slots, d_status) ||
        overlap(d_pool, pool_bytes, k, 16) || overlap(d_pool, pool_bytes, v, 16))
        return Q3KV_ERR_INVALID_ARG;
    AppendArgs a{};
    a.pool = static_cast<uint8_t*>(d_pool);
    a.page_table = d_page_table;
    a.max_pages_per_slot = max_pages_per_slot;
    a.slot_len = d_slot_len;
    a.n_new = d_n_new;
    a.row_offsets = d_row_offsets;
    a.num_slots = num_slots;
    a.max_n_new = max_n_new;
    a.num_layers = desc->num_layers;
    a.num_kv_heads = desc->num_kv_heads;
    a.num_pages = desc->num_pages;
    a.layer = layer;
    a.k = k;
    a.v = v;
    a.dtype = dtype;
    a.status = d_status;
    a.fmt = kFmtBs8;
    // n rows from any place of a block touch at most (n - 1) / 16 + 2 blocks
    const dim3 grid((unsigned)((max_n_new - 1) / kBs8Block + 2), (unsigned)num_slots, (unsigned)desc->num_kv_heads);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(dtype == Q3KV_F32 ? launch(append_bs8_kernel<float>, a, grid, kAppendThreads, 0, st)
                                         : launch(append_bs8_kernel<__nv_bfloat16>, a, grid, kAppendThreads, 0, st));
}

int q3kv_bs8_workspace_bytes(const q3kv_cache_desc* desc, int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t impl,
                             size_t* bytes) {
    if (!bytes) return Q3KV_ERR_INVALID_ARG;
    int ctas = 0, e = q3kv::bs8_check(desc, num_slots, max_ctx_len, max_n_q, impl);
    if (e == Q3KV_OK) e = q3kv::device_sm_count(&ctas);
    if (e == Q3KV_OK) *bytes = q3kv::bs8_partials(ctas);
    return e;
}

int q3kv_bs8_verify_attn(void* stream, const q3kv_cache_desc* desc, const void* d_pool, const int32_t* d_page_table,
                         int32_t max_pages_per_slot, const int32_t* d_ctx_len, const int32_t* d_n_q, const int32_t* d_q_offsets,
                         int32_t num_slots, int64_t max_ctx_len, int32_t max_n_q, int32_t layer, const void* q, int32_t dtype,
                         void* out, int32_t impl, void* d_workspace, size_t workspace_bytes, int32_t* d_status) {
    using namespace q3kv;
    if (max_pages_per_slot <= 0) return Q3KV_ERR_INVALID_ARG;
    if (desc && (layer < 0 || layer >= desc->num_layers)) return Q3KV_ERR_INVALID_ARG;
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    int e = bs8_check(desc, num_slots, max_ctx_len, max_n_q, impl);
    if (e != Q3KV_OK) return e;
    if (num_slots == 0 || max_n_q == 0 || max_ctx_len == 0) return Q3KV_OK;
    if (!d_pool || !d_page_table || !d_ctx_len || !d_n_q || !d_q_offsets || !q || !out) return Q3KV_ERR_INVALID_ARG;
    if (!aligned16(d_pool) || !aligned16(q) || !aligned16(out) || !aligned16(d_workspace)) return Q3KV_ERR_INVALID_ARG;
    if (!d_workspace) return Q3KV_ERR_WORKSPACE_TOO_SMALL;
    const int64_t pool_bytes = (int64_t)bs8_pool_size(desc);          // of q and out the call knows where they begin
    if (over_lists(out, 16, d_page_table, max_pages_per_slot, d_ctx_len, d_n_q, d_q_offsets, num_slots, d_status) || overlap(out, 16, d_pool, pool_bytes))
        return Q3KV_ERR_INVALID_ARG;
    int ctas = 0;
    e = device_sm_count(&ctas);
    if (e != Q3KV_OK) return e;
    if (workspace_bytes < bs8_partials(ctas)) return Q3KV_ERR_WORKSPACE_TOO_SMALL;
    const int64_t ws_bytes = (int64_t)bs8_partials(ctas);             // other operands may lie behind what the call uses
    if (over_lists(d_workspace, ws_bytes, d_page_table, max_pages_per_slot, d_ctx_len, d_n_q, d_q_offsets, num_slots, d_status) ||
        overlap(d_workspace, ws_bytes, d_pool, pool_bytes) || overlap(d_workspace, ws_bytes, q, 16) || overlap(d_workspace, ws_bytes, out, 16))
        return Q3KV_ERR_INVALID_ARG;
    Bs8Args a{};
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
    a.out = out;
    a.dtype = dtype;
    a.ctas = ctas;
    a.partials = static_cast<float*>(d_workspace);
    const bool mma = impl != Q3KV_IMPL_FMA;
    a.rows = mma ? bs8_mma_rows(dtype, max_n_q) : kBs8Rows;
    const double most = (double)num_slots * ((max_ctx_len + kBs8Tile - 1) / kBs8Tile) * desc->num_kv_heads *
                        ((kGroup * max_n_q + a.rows - 1) / a.rows) * ctas;
    a.narrow = most < 4.0e9;
    a.status = d_status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t ce = mma ? launch_bs8_mma(a, st) : launch_bs8_fma(a, st);
    if (ce == cudaSuccess) ce = launch_merge_bs8(a, st);
    return cuda_status(ce);
}

}  // extern "C"
