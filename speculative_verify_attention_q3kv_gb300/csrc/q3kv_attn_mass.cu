// Attention mass: the weight every cached position received from the step's
// queries, accumulated per kv head.
//
//   mass[j] = decay old[j] + sum over visible rows r of e^(q_r . k_hat_j / 16 - lse_r)
//
// With the rows' softmax statistic given, every position is independent of the
// others: one pass over the K records, no maxima, nothing to merge.
//
// One CTA = (slot, kv head, 64 positions): dequantise 32 positions at a time
// into shared memory, a warp per query row and a lane per position, float32
// multiply-adds; the rows of a warp are added in the lane, the warps in order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "q3kv_common.cuh"
#include "q3kv_internal.h"

namespace q3kv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 32;
constexpr int kTilesPerCta = 4;
constexpr int kKStride = 260;

struct MassSmem {
    float q[kMaxRows][kHeadDim];
    float k[kTile][kKStride];
    float lse[kMaxRows];
    float part[kWarps][kTile];
};

template <int FMT>
__device__ __forceinline__ void decode32(const MassArgs& a, const uint8_t* rec, int b, float (&x)[32]) {
    if (FMT == kFmtFp8) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(rec + 32 * b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = w[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                __nv_fp8_e4m3 v;
                v.__x = (unsigned char)(u >> (8 * e));
                x[4 * j + e] = (float)v;
            }
        }
    } else if (FMT == kFmtT5k) {
        const uint32_t* nib = reinterpret_cast<const uint32_t*>(rec) + 4 * b;
        const uint32_t top = reinterpret_cast<const uint32_t*>(rec + 128)[b];
        const float s = __half2float(reinterpret_cast<const __half*>(rec + 160)[b >> 2]);
#pragma unroll
        for (int d = 0; d < 32; ++d) {
            const uint32_t c = ((nib[d / 8] >> (4 * (d % 8))) & 0xFu) | (((top >> d) & 1u) << 4);
            x[d] = a.t5k.c[c] * s;
        }
    } else {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(rec) + 3 * b;
        const float s = __half2float(reinterpret_cast<const __half*>(rec + 96)[b]);
#pragma unroll
        for (int m = 0; m < 15; ++m) {
            const uint32_t u = w[m / 5] >> (3 * (m % 5));
            x[2 * m] = ((float)(u & 7u) - 3.5f) * s;
            x[2 * m + 1] = ((float)((u >> 16) & 7u) - 3.5f) * s;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bit = 15 + 16 * h;
            const uint32_t c = ((w[0] >> bit) & 1u) | (((w[1] >> bit) & 1u) << 1) | (((w[2] >> bit) & 1u) << 2);
            x[30 + h] = ((float)c - 3.5f) * s;
        }
    }
}

template <typename TIn, int FMT>
__global__ void __launch_bounds__(kThreads, 1) mass_kernel(const __grid_constant__ MassArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    MassSmem& sm = *reinterpret_cast<MassSmem*>(smem_raw);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.y % a.num_kv_heads;
    const int slot = blockIdx.y / a.num_kv_heads;
    const int T = a.n_q[slot], L = a.ctx_len[slot];
    if (T <= 0) return;
    if (T > a.max_n_q || T > L || L > a.max_ctx_len || L > (int64_t)a.max_pages_per_slot * kPageSize) {
        if (tid == 0 && blockIdx.x == 0 && g == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        return;
    }
    const int p_first = blockIdx.x * kTile * kTilesPerCta;
    if (p_first >= L) return;
    const int R = kGroup * T;
    const int Hq = a.num_kv_heads * kGroup;
    const int64_t q_base = a.q_offsets[slot];
    const TIn* qin = static_cast<const TIn*>(a.q);
    for (int idx = tid; idx < R * kHeadDim; idx += kThreads) {
        const int r = idx / kHeadDim, d = idx % kHeadDim;
        sm.q[r][d] = load_in(qin + ((q_base + r / kGroup) * Hq + g * kGroup + r % kGroup) * kHeadDim + d);
    }
    for (int r = tid; r < R; r += kThreads) {
        const float v = a.lse[(q_base + r / kGroup) * Hq + g * kGroup + r % kGroup];
        const bool finite = v > -CUDART_INF_F && v < CUDART_INF_F;
        if (!finite && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
        sm.lse[r] = finite ? v : CUDART_INF_F;             // e^(s - inf) = 0
    }
    __syncthreads();
    if (FMT != kFmtFp8) rotate_rows(&sm.q[0][0], R);
    const float scale = FMT == kFmtFp8 ? 1.0f / 16.0f : 1.0f / 256.0f;   // softmax 1/16, H 1/16
    const int32_t* pt = a.page_table + (int64_t)slot * a.max_pages_per_slot;
    float* mass = a.mass + ((int64_t)slot * a.num_kv_heads + g) * a.mass_stride;
    const int N = L - T;
    for (int p0 = p_first; p0 < min(L, p_first + kTile * kTilesPerCta); p0 += kTile) {
        const int32_t page = pt[p0 / kPageSize];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok && tid == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
        __syncthreads();
        {
            const int i = tid >> 3, b = tid & 7;
            float x[32];
            if (ok && p0 + i < L) {
                const uint8_t* rec = a.pool + (FMT == kFmtT5k ? t5k_offset(a.num_layers, a.num_kv_heads, page, a.layer, g, 0, (p0 + i) % kPageSize)
                                                              : record_offset(a.num_layers, a.num_kv_heads, page, a.layer, g, 0, (p0 + i) % kPageSize,
                                                                              FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes));
                decode32<FMT>(a, rec, b, x);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 4)
                *reinterpret_cast<float4*>(&sm.k[i][32 * b + e]) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        }
        __syncthreads();
        const int pos = p0 + lane;
        float sum = 0.0f;
        for (int r = warp; r < R; r += kWarps) {
            float s0 = 0.0f, s1 = 0.0f;
            for (int d = 0; d < kHeadDim; d += 8) {
                const float4 k0 = *reinterpret_cast<const float4*>(&sm.k[lane][d]);
                const float4 k1 = *reinterpret_cast<const float4*>(&sm.k[lane][d + 4]);
                const float4 q0 = *reinterpret_cast<const float4*>(&sm.q[r][d]);
                const float4 q1 = *reinterpret_cast<const float4*>(&sm.q[r][d + 4]);
                s0 = fmaf(q0.x, k0.x, fmaf(q0.y, k0.y, fmaf(q0.z, k0.z, fmaf(q0.w, k0.w, s0))));
                s1 = fmaf(q1.x, k1.x, fmaf(q1.y, k1.y, fmaf(q1.z, k1.z, fmaf(q1.w, k1.w, s1))));
            }
            if (pos <= N + r / kGroup) sum += expf((s0 + s1) * scale - sm.lse[r]);
        }
        sm.part[warp][lane] = ok ? sum : 0.0f;
        __syncthreads();
        if (warp == 0 && pos < L) {
            float t = sm.part[0][lane];
            for (int w = 1; w < kWarps; ++w) t += sm.part[w][lane];
            const float old = (a.decay > 0.0f && pos < N) ? a.decay * mass[pos] : 0.0f;
            mass[pos] = old + t;
        }
    }
}

template <typename TIn, int FMT>
cudaError_t launch_mass(const MassArgs& a, cudaStream_t stream) {
    const int smem = (int)sizeof(MassSmem);
    const cudaError_t e = cudaFuncSetAttribute(mass_kernel<TIn, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int per = kTile * kTilesPerCta;
    cfg.gridDim = dim3((unsigned)((a.max_ctx_len + per - 1) / per), (unsigned)(a.num_slots * a.num_kv_heads));
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
    if (max_n_q > kMaxNq || num_slots > 65535 || (int64_t)num_slots * desc->num_kv_heads > 65535)
        return Q3KV_ERR_UNSUPPORTED;
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool f32 = dtype == Q3KV_F32;
    if (fmt == kFmtFp8) return cuda_status(f32 ? launch_mass<float, kFmtFp8>(a, st) : launch_mass<__nv_bfloat16, kFmtFp8>(a, st));
    if (fmt == kFmtT5k) return cuda_status(f32 ? launch_mass<float, kFmtT5k>(a, st) : launch_mass<__nv_bfloat16, kFmtT5k>(a, st));
    return cuda_status(f32 ? launch_mass<float, kFmtQ3>(a, st) : launch_mass<__nv_bfloat16, kFmtQ3>(a, st));
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
