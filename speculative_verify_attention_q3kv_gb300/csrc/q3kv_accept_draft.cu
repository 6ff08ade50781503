// Acceptance of sampled drafts: the rejection rule with the drafter's own
// probabilities, and the residual sample.
//
// Source: "Quasar" (q27) wiki, "Model tool protocol" bullet (sampled speculative
// decode: Gumbel-max sampling and rejection-sampled acceptance, seeded), for a
// drafter that draws from q_j instead of naming one token.
//
//   accept d_{j+1} iff u_j q_j(d) < p_j(d),   p_j = softmax(logits_j / tau)
//   first rejected row a: argmax of r(x) / E(x), r = max(p_a - q_a, 0), E = -log U
//   (r / E is e^(log r + Gumbel): one logarithm instead of two); bonus: p / E.
//
// Bound: memory and latency.  Every target row is read once for its (max, sum of
// exp); the residual needs one target row (now in L2) and one draft row per slot.
// Two launches: stats_kernel, grid (vocabulary chunks, rows); residual_kernel,
// grid (chunks, slots), in which every CTA merges its slot's row statistics and
// runs the acceptance chain itself (a few hundred loads that hit L2), then races
// its chunk of row a.  The race's winner is a 64-bit atomic maximum of (key,
// ~index) per slot, whatever the order; the slot's last CTA stores the results.
//
// 8 slots x 1 to 8 tokens, vocab 248,320, bf16: 17.1 us, of which the bytes alone are 3.2;
// 1 slot x 6 tokens 10.8 us: two launches and about eight dependent trips to L2 or HBM.
//
// Issue slots decide beside that: the statistics take six instructions an entry
// (bad logits show in the sum, not per entry), and the race computes a clock only
// where it can win (see race).
//
// Exponents: e^((l - max) / tau) with l - max taken on the raw logits (exact for
// the ones that count); a tested probability has log2(e) / tau split in two floats,
// so it is within a few float32 roundings of its definition.
#include <cuda_bf16.h>
#include <float.h>
#include <math.h>
#include <math_constants.h>

#include <algorithm>

#include "q3kv_internal.h"
#include "q3kv_sampling.cuh"

namespace q3kv {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct DraftArgs {
    const void* logits;          // [num_rows, vocab]
    const void* draft;           // [num_rows, vocab]
    int32_t vocab;
    int32_t vec_logits;          // rows of logits / draft are 16-byte aligned
    int32_t vec_draft;
    int32_t chunk1, num_chunks1; // entries (a multiple of 8) and chunks per row of the statistics
    int32_t chunk2, num_chunks2; // the same of the race
    const int32_t* q_offsets;
    const int32_t* n_q;
    const int32_t* tokens;
    int32_t num_slots;
    int32_t num_rows;
    int32_t max_n_q;
    const int32_t* ctx_len;
    float c_hi, c_lo;            // log2(e) / tau
    float d_min;                 // d c_hi = -160, below every exponent that counts; -inf where no float32 d is so low
    const float* uniforms;
    uint64_t seed;
    int32_t* n_accepted;
    int32_t* next_token;
    int32_t* committed_len;
    float* accept_prob;
    float2* stats;               // [num_rows, num_chunks1] (max of raw logits, sum of exp)
    unsigned long long* best;    // [num_slots, 2] race winners: residual, target
    unsigned int* arrived;       // [num_slots] CTAs of the race that are done
    int32_t* status;
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// e^((l - m) / tau); l <= m, m finite (l = -inf gives 0).  Below d_min the result is 0 whatever the
// exponent's second part: a finite mask at a low temperature overflows that too, to either sign.
__device__ __forceinline__ float weight(const DraftArgs& a, float l, float m) {
    const float d = l - m;
    return exp2_approx(d > a.d_min ? fmaf(d, a.c_hi, d * a.c_lo) : -CUDART_INF_F);
}

// the same for a term of the sum, with log2(e) / tau in one float: 2^-25 of an exponent that
// counts (below 20) is lost
__device__ __forceinline__ float term(const DraftArgs& a, float l, float m) { return exp2_approx((l - m) * a.c_hi); }

// (max, sum) of two parts of a row
__device__ __forceinline__ float2 merge(const DraftArgs& a, float2 x, float2 y) {
    const float m = fmaxf(x.x, y.x);
    if (m == -CUDART_INF_F) return make_float2(m, 0.0f);
    return make_float2(m, x.y * weight(a, x.x, m) + y.y * weight(a, y.x, m));
}

__device__ __forceinline__ float2 warp_merge(const DraftArgs& a, float2 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = merge(a, v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
    return v;
}

// 8 entries from k on (entries at or past c1 are `pad`); k and c1 as in the
// chunks, whose bounds are multiples of 8.
template <typename T>
__device__ __forceinline__ void load8(const T* row, bool vec, int k, int c1, float pad, float (&x)[8]) {
    if (vec && k + 8 <= c1) {
        if (sizeof(T) == 2) {
            const uint4 u = *reinterpret_cast<const uint4*>(row + k);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        } else {
            const float4 u = reinterpret_cast<const float4*>(row + k)[0];
            const float4 w = reinterpret_cast<const float4*>(row + k)[1];
            x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
            x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < c1 ? to_f(row[k + i]) : pad;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) stats_kernel(const DraftArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float2 red[kWarps];
    const int row = blockIdx.y, chunk = blockIdx.x;
    const int64_t linear = (int64_t)row * gridDim.x + chunk;
    // clears the slots' race state for the next kernel
    for (int64_t b = linear * kThreads + threadIdx.x; b < a.num_slots; b += (int64_t)gridDim.x * gridDim.y * kThreads) {
        a.best[2 * b] = 0ull;
        a.best[2 * b + 1] = 0ull;
        a.arrived[b] = 0u;
    }
    const int c0 = chunk * a.chunk1;
    const int c1 = min(a.vocab, c0 + a.chunk1);
    const T* lg = static_cast<const T*>(a.logits) + (int64_t)row * a.vocab;
    float m = -CUDART_INF_F, s = 0.0f;
    constexpr int kU = 4;                                  // 32 entries of a thread in flight
    for (int k0 = c0 + 8 * threadIdx.x; k0 < c1; k0 += 8 * kU * kThreads) {
        float x[kU][8];
#pragma unroll
        for (int r = 0; r < kU; ++r) load8(lg, a.vec_logits, k0 + 8 * r * kThreads, c1, -CUDART_INF_F, x[r]);
        float bm = x[0][0];
#pragma unroll
        for (int r = 0; r < kU; ++r)
#pragma unroll
            for (int i = 0; i < 8; ++i) bm = fmaxf(bm, x[r][i]);
        if (bm > m) {
            s = m == -CUDART_INF_F ? 0.0f : s * weight(a, m, bm);
            m = bm;
        }
        // a row of -inf so far: 0 in place of the maximum keeps the terms at 0, and NaN at NaN
        const float mm = m == -CUDART_INF_F ? 0.0f : m;
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int r = 0; r < kU; ++r)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                t0 += term(a, x[r][i], mm);
                t1 += term(a, x[r][i + 1], mm);
            }
        s += t0 + t1;
    }
    // a NaN logit makes its sum NaN, and so does +inf (inf - inf)
    if (__any_sync(0xffffffffu, s != s) && (threadIdx.x & 31) == 0 && a.status)
        atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
    float2 v = warp_merge(a, make_float2(m, s));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kWarps; ++w) v = merge(a, v, red[w]);
        a.stats[(int64_t)row * a.num_chunks1 + chunk] = v;
    }
}

// (key, ~index) of a candidate: larger keys first, then lower indexes.  Keys are
// non-negative floats, whose bit patterns are ordered as they are.
__device__ __forceinline__ unsigned long long candidate(float key, int x) {
    return ((unsigned long long)__float_as_uint(key) << 32) | (uint32_t)~x;
}
__device__ __forceinline__ unsigned long long warp_max(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The race w / E of 8 entries of every lane, from index k on, w >= 0.  With U = (n + 1/2) / 2^23,
// E = -log U >= 1 - U = (2^23 - n - 1/2) / 2^23, so w / (1 - U), a little generous, bounds a key
// without a logarithm.  Every lane computes the key of the entry with its largest bound, and
// after that only those whose bound reaches the warp's best key: about one logarithm a lane and step
// where eight tests against the keys of earlier steps took most of the eight (8 slots 19.1 -> 17.1 us).
__device__ __forceinline__ void race(const float (&w)[8], const float (&n)[8], int k, unsigned long long& best, float& top) {
    auto enter = [&](float wi, float ni, int x) {
        const float e = -logf((ni + 0.5f) * (1.0f / 8388608.0f));
        best = max(best, candidate(wi / e, x));
    };
    float bound[8];
    float b = 0.0f, bw = 0.0f, bn = 0.0f;
    int bi = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bound[i] = __fdividef(w[i], (8388607.5f - n[i]) * (0.9999f / 8388608.0f));
        if (bound[i] > b) {
            b = bound[i];
            bw = w[i];
            bn = n[i];
            bi = i;
        }
    }
    if (!__any_sync(0xffffffffu, b >= top && b > 0.0f)) return;
    if (b >= top && b > 0.0f) enter(bw, bn, k + bi);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32)));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (bound[i] >= top && bound[i] > 0.0f && i != bi) enter(w[i], n[i], k + i);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32)));
}

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads, 2) residual_kernel(const DraftArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ float2 st[kMaxNq];
    __shared__ int s_acc;
    __shared__ unsigned long long red[2][kWarps];
    const int b = blockIdx.y, chunk = blockIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = a.n_q[b];
    const int32_t L = a.ctx_len[b];
    const int r0 = a.q_offsets[b];
    const bool skip = n <= 0 || n > a.max_n_q || n > L || r0 < 0 || r0 > a.num_rows - n;
    int acc = 0;
    if (!skip) {
        // lane j of warp 0 tests the draft that follows query token j; its values are on the way
        // while the rows' statistics are merged
        const bool drafted = warp == 0 && lane < n - 1;
        const int d = drafted ? a.tokens[r0 + lane + 1] : -1;
        const bool known = drafted && d >= 0 && d < a.vocab;
        float ld = 0.0f, q = 0.0f, u = 1.0f;
        if (known) {
            const int64_t at = (int64_t)(r0 + lane) * a.vocab + d;
            ld = to_f(static_cast<const T*>(a.logits)[at]);
            q = to_f(static_cast<const Q*>(a.draft)[at]);
            u = a.uniforms[r0 + lane];
        }
        // the rows' statistics: one warp per row, its lanes over the chunks
        for (int j = warp; j < n; j += kWarps) {
            const float2* p = a.stats + (int64_t)(r0 + j) * a.num_chunks1;
            float2 v = make_float2(-CUDART_INF_F, 0.0f);
            for (int k = lane; k < a.num_chunks1; k += 32) v = merge(a, v, p[k]);
            v = warp_merge(a, v);
            if (lane == 0) st[j] = v;
        }
        __syncthreads();
        if (warp == 0) {
            const float2 v = st[drafted ? lane : 0];
            const float p = known && v.y > 0.0f ? weight(a, ld, v.x) / v.y : 0.0f;
            const bool pass = drafted && u * q < p;
            const unsigned miss = __ballot_sync(0xffffffffu, drafted && !pass);
            const int first = miss ? __ffs(miss) - 1 : n - 1;
            if (lane == 0) s_acc = first;
            if (chunk == 0 && drafted) {
                if (!(q >= 0.0f && q < CUDART_INF_F) && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
                if (a.accept_prob) a.accept_prob[r0 + lane] = q > 0.0f ? fminf(1.0f, p / q) : (p > 0.0f ? 1.0f : 0.0f);
            }
        }
        __syncthreads();
        acc = s_acc;
        // the race over this chunk of row acc
        const int64_t row = r0 + acc;
        const float2 v = st[acc];
        const bool bonus = acc == n - 1;
        const T* lg = static_cast<const T*>(a.logits) + row * a.vocab;
        const Q* dr = static_cast<const Q*>(a.draft) + row * a.vocab;
        const float inv = v.y > 0.0f ? 1.0f / v.y : 0.0f;
        const int c0 = chunk * a.chunk2;
        const int c1 = min(a.vocab, c0 + a.chunk2);
        unsigned long long best_r = 0ull, best_p = 0ull;
        // the warp's best keys so far: a candidate has to reach them
        float top_r = 0.0f, top_p = 0.0f;
        bool bad = false;
        if (v.x > -CUDART_INF_F) {
            for (int k0 = c0 + 8 * (threadIdx.x & ~31); k0 < c1; k0 += 8 * kThreads) {   // warp-uniform
                const int k = k0 + 8 * lane;
                float p[8], r[8], n[8];
                load8(lg, a.vec_logits, k, c1, -CUDART_INF_F, p);
                if (!bonus) load8(dr, a.vec_draft, k, c1, 0.0f, r);
                const uint64_t z = noise_state(a.seed, (uint32_t)row, (uint32_t)k);
                float most = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // NaN and -inf: probability 0, or NaN (where d_min is -inf), which no key is made of
                    const float d = fmaxf(p[i] - v.x, a.d_min);
                    p[i] = exp2_approx(fmaf(d, a.c_hi, d * a.c_lo)) * inv;
                    if (bonus) {
                        r[i] = p[i];
                    } else {
                        bad |= !(r[i] >= 0.0f && r[i] < CUDART_INF_F);
                        r[i] = fmaxf(p[i] - r[i], 0.0f);                     // NaN counts as nothing
                    }
                    most = fmaxf(most, r[i]);
                    n[i] = noise_level(z + (uint64_t)i * kNoiseStep);
                }
                if (top_r > 0.0f || __any_sync(0xffffffffu, most > 0.0f)) race(r, n, k, best_r, top_r);
                else race(p, n, k, best_p, top_p);                           // wanted if no residual is positive at all
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
        best_r = warp_max(best_r);
        best_p = warp_max(best_p);
        if (lane == 0) {
            red[0][warp] = best_r;
            red[1][warp] = best_p;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        if (!skip) {
            unsigned long long r = red[0][0], p = red[1][0];
            for (int w = 1; w < kWarps; ++w) {
                r = max(r, red[0][w]);
                p = max(p, red[1][w]);
            }
            if (r) atomicMax(&a.best[2 * b], r);
            if (p) atomicMax(&a.best[2 * b + 1], p);
        }
        __threadfence();
        // the last CTA of the slot stores (every CTA has read ctx_len by then, so
        // committed_len may be the same array)
        if (atomicAdd(&a.arrived[b], 1u) == gridDim.x - 1) {
            __threadfence();
            if (skip) {
                if (n != 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
                a.n_accepted[b] = 0;
                a.next_token[b] = -1;
                a.committed_len[b] = L;
            } else {
                const unsigned long long r = __ldcg(&a.best[2 * b]), p = __ldcg(&a.best[2 * b + 1]);
                const unsigned long long w = r ? r : p;
                a.n_accepted[b] = acc;
                a.next_token[b] = w ? (int32_t)~(uint32_t)w : -1;
                a.committed_len[b] = L - (n - 1 - acc);
            }
        }
    }
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, const DraftArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Chunks of one vocabulary row: over `units` rows at most the two CTAs per SM that run at
// once (a few more make a second wave: 8 slots 22.8 us, in one wave 19.1), at least 2,048
// entries each (4,096: one slot 10.8 -> 12.3 us), a multiple of 8.
int chunk_plan(int64_t units, int32_t vocab, int32_t* chunk, int32_t* num) {
    int sms = 0;
    const int e = device_sm_count(&sms);
    if (e != Q3KV_OK) return e;
    units = std::max<int64_t>(units, 1);
    const int64_t target = std::max<int64_t>(1, 2 * (int64_t)sms / units);
    const int64_t n = std::min<int64_t>(target, ((int64_t)vocab + 2047) / 2048);
    const int64_t c = (((int64_t)vocab + n - 1) / n + 7) / 8 * 8;
    *chunk = (int32_t)c;
    *num = (int32_t)(((int64_t)vocab + c - 1) / c);
    return Q3KV_OK;
}

constexpr int32_t kMaxVocab = 1 << 28;   // chunk arithmetic stays within 32 bits

struct DraftPlan {
    int32_t chunk1, num1, chunk2, num2;
    size_t stats_bytes, slot_bytes;
    size_t total() const { return stats_bytes + slot_bytes; }
};

int draft_plan(int32_t num_slots, int32_t num_rows, int32_t vocab, DraftPlan* p) {
    if (num_slots < 0 || num_rows < 0 || vocab <= 0) return Q3KV_ERR_INVALID_ARG;
    if (num_rows > 65535 || num_slots > 65535 || vocab > kMaxVocab) return Q3KV_ERR_UNSUPPORTED;
    int e = chunk_plan(num_rows, vocab, &p->chunk1, &p->num1);
    if (e != Q3KV_OK) return e;
    e = chunk_plan(num_slots, vocab, &p->chunk2, &p->num2);
    if (e != Q3KV_OK) return e;
    p->stats_bytes = (((size_t)num_rows * p->num1 * sizeof(float2)) + 15) / 16 * 16;
    p->slot_bytes = (size_t)num_slots * 2 * 8 + ((size_t)num_slots * 4 + 15) / 16 * 16;
    return Q3KV_OK;
}

}  // namespace
}  // namespace q3kv

using namespace q3kv;

extern "C" {

int q3kv_accept_draft_workspace_bytes(int32_t num_slots, int32_t num_rows, int32_t vocab, size_t* bytes) {
    if (!bytes) return Q3KV_ERR_INVALID_ARG;
    DraftPlan p;
    const int e = draft_plan(num_slots, num_rows, vocab, &p);
    if (e != Q3KV_OK) return e;
    *bytes = p.total();
    return Q3KV_OK;
}

int q3kv_accept_draft(void* stream, const void* logits, int32_t dtype, int32_t vocab, const void* draft_probs,
                      int32_t draft_dtype, const int32_t* d_q_offsets, const int32_t* d_n_q, const int32_t* d_tokens,
                      int32_t num_slots, int32_t num_rows, int32_t max_n_q, const int32_t* d_ctx_len,
                      float temperature, const float* d_uniforms, uint64_t seed, int32_t* d_n_accepted,
                      int32_t* d_next_token, int32_t* d_committed_len, float* d_accept_prob, void* d_workspace,
                      size_t workspace_bytes, int32_t* d_status) {
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (draft_dtype != Q3KV_F32 && draft_dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (max_n_q < 0) return Q3KV_ERR_INVALID_ARG;
    if (!(temperature > 0.0f) || !(temperature < 3.0e38f)) return Q3KV_ERR_INVALID_ARG;
    const double c = 1.4426950408889634074 / (double)temperature;
    if (c > (double)FLT_MAX) return Q3KV_ERR_INVALID_ARG;
    const float c_hi = (float)c;
    // accept_prob is written while other CTAs still read the uniforms
    if (d_accept_prob && num_rows > 0 && d_accept_prob < d_uniforms + num_rows && d_uniforms < d_accept_prob + num_rows)
        return Q3KV_ERR_INVALID_ARG;
    if (max_n_q > kMaxNq) return Q3KV_ERR_UNSUPPORTED;
    DraftPlan p;
    int e = draft_plan(num_slots, num_rows, vocab, &p);
    if (e != Q3KV_OK) return e;
    if (num_slots == 0) return Q3KV_OK;
    if (!d_q_offsets || !d_n_q || !d_ctx_len || !d_n_accepted || !d_next_token || !d_committed_len) return Q3KV_ERR_INVALID_ARG;
    if (num_rows > 0 && (!logits || !draft_probs || !d_tokens || !d_uniforms)) return Q3KV_ERR_INVALID_ARG;
    if (workspace_bytes < p.total() || !d_workspace) return Q3KV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned16(d_workspace)) return Q3KV_ERR_INVALID_ARG;
    DraftArgs a{};
    a.logits = logits;
    a.draft = draft_probs;
    a.vocab = vocab;
    a.vec_logits = aligned16(logits) && ((size_t)vocab * (dtype == Q3KV_F32 ? 4 : 2)) % 16 == 0;
    a.vec_draft = aligned16(draft_probs) && ((size_t)vocab * (draft_dtype == Q3KV_F32 ? 4 : 2)) % 16 == 0;
    a.chunk1 = p.chunk1;
    a.num_chunks1 = p.num1;
    a.chunk2 = p.chunk2;
    a.num_chunks2 = p.num2;
    a.q_offsets = d_q_offsets;
    a.n_q = d_n_q;
    a.tokens = d_tokens;
    a.num_slots = num_slots;
    a.num_rows = num_rows;
    a.max_n_q = max_n_q;
    a.ctx_len = d_ctx_len;
    a.c_hi = c_hi;
    a.c_lo = (float)(c - (double)c_hi);
    a.d_min = 160.0 / c > (double)FLT_MAX ? -INFINITY : (float)(-160.0 / c);
    a.uniforms = d_uniforms;
    a.seed = seed;
    a.n_accepted = d_n_accepted;
    a.next_token = d_next_token;
    a.committed_len = d_committed_len;
    a.accept_prob = d_accept_prob;
    uint8_t* ws = static_cast<uint8_t*>(d_workspace);
    a.stats = reinterpret_cast<float2*>(ws);
    a.best = reinterpret_cast<unsigned long long*>(ws + p.stats_bytes);
    a.arrived = reinterpret_cast<unsigned int*>(ws + p.stats_bytes + (size_t)num_slots * 16);
    a.status = d_status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 g1((unsigned)p.num1, (unsigned)num_rows), g2((unsigned)p.num2, (unsigned)num_slots);
    if (num_rows == 0) {
        // no statistics: every slot is idle or out of range
        cudaError_t ce = cudaMemsetAsync(a.best, 0, p.slot_bytes, st);
        if (ce != cudaSuccess) return cuda_status(ce);
    } else {
        const cudaError_t ce = dtype == Q3KV_F32 ? launch_pdl(stats_kernel<float>, g1, a, st)
                                                 : launch_pdl(stats_kernel<__nv_bfloat16>, g1, a, st);
        if (ce != cudaSuccess) return cuda_status(ce);
    }
    if (dtype == Q3KV_F32)
        return cuda_status(draft_dtype == Q3KV_F32 ? launch_pdl(residual_kernel<float, float>, g2, a, st)
                                                   : launch_pdl(residual_kernel<float, __nv_bfloat16>, g2, a, st));
    return cuda_status(draft_dtype == Q3KV_F32 ? launch_pdl(residual_kernel<__nv_bfloat16, float>, g2, a, st)
                                               : launch_pdl(residual_kernel<__nv_bfloat16, __nv_bfloat16>, g2, a, st));
}

}  // extern "C"
