// Token counts of the slots, and the logits of a verify step with penalties for repeated tokens,
// biases and grammar masks: what runs between the model's logits and the acceptance.
//
// A slot's state is one int16 per vocabulary entry: bits 0..14 how often the token was generated
// (saturating), bit 15 whether the prompt holds it.  Row j of a slot comes after the step's own
// tokens t_0..t_j, which the counts do not hold yet, so for it c(x) = count(x) + #{i <= j : t_i = x}:
//   y = l                                                     the row's logit
//   y = y > 0 ? y / theta : y * theta     if c > 0 or the prompt holds x    (repetition)
//   y = y - alpha c - beta [c > 0]                            (frequency, presence)
//   y = y + bias(x);  y = -inf where the row's mask has a 0 bit
// in float32, rounded once to the logits' type.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "q3kv_internal.h"

namespace q3kv {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                       // entries per thread
constexpr int kChunk = kThreads * kPer;       // vocabulary entries per CTA

struct LogitArgs {
    const void* logits;
    void* out;
    int32_t vocab;
    const int32_t* q_offsets;
    const int32_t* n_q;
    const int32_t* tokens;
    int32_t num_rows;
    int32_t max_n_q;
    const int16_t* counts;       // [slots, counts_stride] or null
    int64_t counts_stride;
    const float* repetition;     // [slots] each, or null
    const float* frequency;
    const float* presence;
    const int32_t* bias_offsets; // [slots + 1] or null
    const int32_t* bias_tokens;
    const float* bias_values;
    int32_t num_biases;
    const int32_t* mask;         // [rows, ceil(vocab / 32)] or null
    int32_t* status;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
struct alignas(16) Row8 {
    T x[kPer];
};

// A CTA takes 2,048 entries of up to kBatch rows of one slot: their logits, masks and counts are all loaded before the
// first barrier.  Bound: bytes (logits in and out); small calls: the chain of loads lengths -> tokens -> biases.
constexpr int kBatch = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) process_logits_kernel(LogitArgs a) {
    __shared__ float s_bias[kChunk];
    __shared__ int s_tok[kMaxNq];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, slot = blockIdx.y, j0 = blockIdx.z * kBatch;
    const int base = blockIdx.x * kChunk;
    const int w = a.n_q[slot], r0 = a.q_offsets[slot];
    int b0 = 0, b1 = 0;
    if (a.bias_offsets) {
        b0 = a.bias_offsets[slot];
        b1 = a.bias_offsets[slot + 1];
    }
    const float theta = a.repetition ? a.repetition[slot] : 1.0f;
    const float alpha = a.frequency ? a.frequency[slot] : 0.0f, beta = a.presence ? a.presence[slot] : 0.0f;
    // this thread's entries: 8 neighbours, or every 256th where rows are not 16-byte aligned
    const int first = VEC ? base + tid * kPer : base + tid;
    constexpr int kStep = VEC ? 1 : kThreads;
    union {
        Row8<int16_t> v;
        int16_t x[kPer];
    } count;
    if (a.counts && first < a.vocab) {
        const int16_t* c = a.counts + (int64_t)slot * a.counts_stride;
        if (VEC) {
            count.v = *reinterpret_cast<const Row8<int16_t>*>(c + first);   // the stride covers whole vectors
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e) count.x[e] = first + e * kStep < a.vocab ? c[first + e * kStep] : (int16_t)0;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e) count.x[e] = 0;
    }
    const bool report = blockIdx.x == 0 && blockIdx.z == 0 && a.status;
    if (w == 0) return;
    if (w < 0 || w > a.max_n_q || r0 < 0 || r0 > a.num_rows - w) {
        if (report && tid == 0) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        return;
    }
    if (j0 >= w) return;
    if (tid < w) {
        const int t = a.tokens[r0 + tid];
        s_tok[tid] = t;
        if (report && (t < 0 || t >= a.vocab)) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
    }
    const int64_t mask_words = (a.vocab + 31) / 32;
    const T* in = static_cast<const T*>(a.logits) + (int64_t)(r0 + j0) * a.vocab + first;
    const int rows = min(kBatch, w - j0);
    Row8<T> x[kBatch];
    uint32_t allowed[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (k >= rows) break;
        const T* p = in + (int64_t)k * a.vocab;
        if (VEC) {
            if (first < a.vocab) x[k] = *reinterpret_cast<const Row8<T>*>(p);
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (first + e * kStep < a.vocab) x[k].x[e] = p[e * kStep];
        }
        allowed[k] = ~0u;
        if (a.mask) {
            const uint32_t* m = reinterpret_cast<const uint32_t*>(a.mask) + (r0 + j0 + k) * mask_words;
            if (VEC) {
                if (first < a.vocab) allowed[k] = reinterpret_cast<const uint8_t*>(m)[first >> 3];
            } else {
                // a warp's entries of one step share a word: lane e holds step e's
                const int word = (first - lane + lane * kStep) >> 5;
                allowed[k] = lane < kPer && word < mask_words ? m[word] : 0;
            }
        }
    }
    if (b0 < 0 || b1 < b0 || b1 > a.num_biases) {
        if (report && tid == 0) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        b0 = b1 = 0;
    }
    if (b1 > b0) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_bias[tid + i * kThreads] = 0.0f;
        __syncthreads();
        for (int i = b0 + tid; i < b1; i += kThreads) {
            const int t = a.bias_tokens[i];
            // ascending ids: no id twice, so the sum does not depend on an order
            if (t < 0 || t >= a.vocab || (i > b0 && a.bias_tokens[i - 1] >= t)) {
                if (report) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
            } else if (t >= base && t < base + kChunk) {
                s_bias[t - base] = a.bias_values[i];
            }
        }
    }
    __syncthreads();
    if (VEC && first >= a.vocab) return;

    uint32_t step[kPer];         // bit i: t_i is this entry
    bool stepping = false;
#pragma unroll
    for (int e = 0; e < kPer; ++e) step[e] = 0;
    for (int i = 0; i < min(w, j0 + kBatch); ++i) {
        const int d = s_tok[i] - first;
        if (VEC ? (unsigned)d < (unsigned)kPer : d >= 0 && d < kChunk && d % kThreads == 0) {
            stepping = true;
#pragma unroll
            for (int e = 0; e < kPer; ++e) step[e] |= (d == e * kStep ? 1u : 0u) << i;
        }
    }
    const bool in_place = a.logits == a.out;
    T* out = static_cast<T*>(a.out) + (int64_t)(r0 + j0) * a.vocab + first;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        if (k >= rows) break;
        T* p = out + (int64_t)k * a.vocab;
        Row8<T> o;
        bool changed = !in_place;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            int c = count.x[e];
            const bool prompt = c < 0;
            c &= 0x7fff;
            if (stepping) c += __popc(step[e] & ((2u << (j0 + k)) - 1u));
            float y = to_f32(x[k].x[e]);
            if (c > 0 || prompt) {
                y = y > 0.0f ? __fdiv_rn(y, theta) : y * theta;
                if (c > 0) y = (y - alpha * (float)c) - beta;
            }
            if (b1 > b0) y += s_bias[first - base + e * kStep];
            const bool allow = VEC || !a.mask ? (allowed[k] >> e) & 1u : (__shfl_sync(0xffffffffu, allowed[k], e) >> lane) & 1u;
            if (!allow) y = -CUDART_INF_F;
            o.x[e] = from_f32<T>(y);
            // NaN differs from itself and is stored again
            if (in_place) changed |= !(to_f32(o.x[e]) == to_f32(x[k].x[e]));
        }
        if (VEC) {
            if (changed) *reinterpret_cast<Row8<T>*>(p) = o;
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (first + e * kStep < a.vocab) p[e * kStep] = o.x[e];
        }
    }
}

// ---------------------------------------------------------------- counts
struct CountArgs {
    int16_t* counts;
    int64_t stride;
    int32_t vocab;
    const int32_t* tokens;
    int64_t num_tokens;
    const int32_t* offsets;
    const int32_t* n;
    int32_t max_n;
    int32_t* status;
};

constexpr int kCountCap = 0x7fff;

__device__ __forceinline__ uint32_t* count_word(int16_t* at) {
    return reinterpret_cast<uint32_t*>(reinterpret_cast<uintptr_t>(at) & ~(uintptr_t)3);
}
// word with add added to the 16-bit half at `shift`, saturating in its low 15 bits
__device__ __forceinline__ uint32_t add_to(uint32_t word, int shift, int add) {
    const uint32_t now = (uint32_t)min((int)((word >> shift) & kCountCap) + add, kCountCap);
    return (word & ~((uint32_t)kCountCap << shift)) | (now << shift);
}
// the order of additions does not matter
__device__ __forceinline__ void add_count(int16_t* at, int add) {
    uint32_t* word = count_word(at);
    const int shift = (reinterpret_cast<uintptr_t>(at) & 2) ? 16 : 0;
    uint32_t old = *reinterpret_cast<volatile uint32_t*>(word), seen;
    do {
        seen = old;
        const uint32_t now = add_to(seen, shift, add);
        if (now == seen) return;
        old = atomicCAS(word, seen, now);
    } while (old != seen);
}

__device__ __forceinline__ bool slot_range(const CountArgs& a, int slot, int64_t* begin, int* n) {
    *n = a.n[slot];
    *begin = a.offsets[slot];
    if (*n >= 0 && *n <= a.max_n && *begin >= 0 && *begin + *n <= a.num_tokens) return true;
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
    return false;
}

// Few tokens per slot, or marks of a prompt (a mark that is there already costs no atomic): a thread per
// token; equal tokens of a warp are added once.
template <bool PROMPT>
__global__ void __launch_bounds__(kThreads) count_kernel(CountArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int slot = blockIdx.y;
    int64_t begin;
    int n;
    if (!slot_range(a, slot, &begin, &n)) return;
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if ((int)(blockIdx.x * kThreads + (threadIdx.x & ~31)) >= n) return;      // whole warps leave
    int t = i < n ? a.tokens[begin + i] : -1;
    if (i < n && (t < 0 || t >= a.vocab)) {
        if (a.status) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
        t = -1;
    }
    int16_t* at = a.counts + (int64_t)slot * a.stride + max(t, 0);
    if (PROMPT) {
        if (t >= 0 && *reinterpret_cast<volatile int16_t*>(at) >= 0) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(at);
            atomicOr(reinterpret_cast<uint32_t*>(p & ~(uintptr_t)3), (p & 2) ? 0x80000000u : 0x8000u);
        }
        return;
    }
    const uint32_t same = __match_any_sync(0xffffffffu, t);
    if (t >= 0 && (threadIdx.x & 31) == __ffs(same) - 1) add_count(at, __popc(same));
}

// Long histories: frequent tokens would meet in the same words, so a CTA first adds up its 4,096 tokens in
// a shared hash table (half full at most) and then adds each different token once.  Every phase is a few
// independent accesses per thread: 4 tokens, 8 places of the table.
constexpr int kHistory = 4096, kTable = 8192, kHistoryThreads = 1024;

__global__ void __launch_bounds__(kHistoryThreads) count_history_kernel(CountArgs a) {
    extern __shared__ int s_table[];              // [kTable] keys, then [kTable] counts
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int* keys = s_table;
    int* sums = s_table + kTable;
#pragma unroll
    for (int i = 0; i < kTable / kHistoryThreads; ++i) {
        keys[i * kHistoryThreads + threadIdx.x] = -1;
        sums[i * kHistoryThreads + threadIdx.x] = 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int slot = blockIdx.y;
    int64_t begin;
    int n;
    if (!slot_range(a, slot, &begin, &n)) return;
    const int64_t from = (int64_t)blockIdx.x * kHistory;
    if (from >= n) return;
    int t[kHistory / kHistoryThreads];
#pragma unroll
    for (int k = 0; k < kHistory / kHistoryThreads; ++k) {
        const int64_t i = from + k * kHistoryThreads + threadIdx.x;
        t[k] = i < n ? a.tokens[begin + i] : -1;
        if (i < n && (t[k] < 0 || t[k] >= a.vocab)) {
            if (a.status) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
            t[k] = -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kHistory / kHistoryThreads; ++k) {
        if (t[k] < 0) continue;
        // open addressing ends: at most kHistory of kTable places are taken
        uint32_t h = ((uint32_t)t[k] * 2654435761u) >> 19;
        for (int key = atomicCAS(&keys[h], -1, t[k]); key != -1 && key != t[k]; key = atomicCAS(&keys[h], -1, t[k])) h = (h + 1) & (kTable - 1);
        atomicAdd(&sums[h], 1);
    }
    __syncthreads();
    int16_t* counts = a.counts + (int64_t)slot * a.stride;
    constexpr int kPlaces = kTable / kHistoryThreads;
    int key[kPlaces];
    uint32_t seen[kPlaces];
#pragma unroll
    for (int k = 0; k < kPlaces; ++k) {
        key[k] = keys[k * kHistoryThreads + threadIdx.x];
        if (key[k] >= 0) seen[k] = *reinterpret_cast<volatile uint32_t*>(count_word(counts + key[k]));
    }
    uint32_t open = 0;                            // places whose addition has not gone through
#pragma unroll
    for (int k = 0; k < kPlaces; ++k)
        if (key[k] >= 0) {
            const int shift = (key[k] & 1) * 16;  // rows begin on whole words
            const uint32_t now = add_to(seen[k], shift, sums[k * kHistoryThreads + threadIdx.x]);
            if (now != seen[k] && atomicCAS(count_word(counts + key[k]), seen[k], now) != seen[k]) open |= 1u << k;
        }
    while (open) {
        const int k = __ffs(open) - 1;
        open &= open - 1;
        const int place = k * kHistoryThreads + threadIdx.x;
        add_count(counts + keys[place], sums[place]);
    }
}

template <typename K, typename A>
cudaError_t launch(K kernel, const A& a, dim3 grid, size_t smem, cudaStream_t st, int threads = kThreads) {
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

}  // namespace
}  // namespace q3kv

extern "C" {

int q3kv_count_tokens(void* stream, int16_t* d_counts, int64_t counts_stride, int32_t vocab, const int32_t* d_tokens,
                      int64_t num_tokens, const int32_t* d_offsets, const int32_t* d_n, int32_t num_slots, int32_t max_n,
                      int32_t prompt, int32_t* d_status) {
    using namespace q3kv;
    if (vocab <= 0 || num_tokens < 0 || num_slots < 0 || max_n < 0 || (prompt != 0 && prompt != 1)) return Q3KV_ERR_INVALID_ARG;
    if (counts_stride < vocab || counts_stride % 8 != 0) return Q3KV_ERR_INVALID_ARG;
    if (num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (num_slots == 0 || max_n == 0 || num_tokens == 0) return Q3KV_OK;
    if (!d_counts || !d_tokens || !d_offsets || !d_n || !aligned16(d_counts)) return Q3KV_ERR_INVALID_ARG;
    const int64_t bytes = (int64_t)num_slots * counts_stride * 2;
    if (overlap(d_counts, bytes, d_tokens, num_tokens * 4) || overlap(d_counts, bytes, d_offsets, (int64_t)num_slots * 4) ||
        overlap(d_counts, bytes, d_n, (int64_t)num_slots * 4) || (d_status && overlap(d_counts, bytes, d_status, 4)))
        return Q3KV_ERR_INVALID_ARG;
    CountArgs a{d_counts, counts_stride, vocab, d_tokens, num_tokens, d_offsets, d_n, max_n, d_status};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!prompt && max_n > kThreads) {
        constexpr size_t smem = 2 * kTable * sizeof(int);
        cudaError_t ce = cudaFuncSetAttribute(count_history_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (ce != cudaSuccess) return cuda_status(ce);
        return cuda_status(launch(count_history_kernel, a, dim3((unsigned)(((int64_t)max_n + kHistory - 1) / kHistory), num_slots), smem, st,
                                  kHistoryThreads));
    }
    const dim3 grid((unsigned)(((int64_t)max_n + kThreads - 1) / kThreads), (unsigned)num_slots);
    return cuda_status(prompt ? launch(count_kernel<true>, a, grid, 0, st) : launch(count_kernel<false>, a, grid, 0, st));
}

int q3kv_process_logits(void* stream, const void* logits, void* out, int32_t dtype, int32_t vocab, const int32_t* d_q_offsets,
                        const int32_t* d_n_q, const int32_t* d_tokens, int32_t num_slots, int32_t num_rows, int32_t max_n_q,
                        const int16_t* d_counts, int64_t counts_stride, const float* d_repetition, const float* d_frequency,
                        const float* d_presence, const int32_t* d_bias_offsets, const int32_t* d_bias_tokens,
                        const float* d_bias_values, int32_t num_biases, const int32_t* d_mask, int32_t* d_status) {
    using namespace q3kv;
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (vocab <= 0 || num_slots < 0 || num_rows < 0 || max_n_q < 0 || num_biases < 0) return Q3KV_ERR_INVALID_ARG;
    if (max_n_q > kMaxNq || num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (d_counts && (counts_stride < vocab || counts_stride % 8 != 0)) return Q3KV_ERR_INVALID_ARG;
    if (num_slots == 0 || num_rows == 0 || max_n_q == 0) return Q3KV_OK;
    if (!logits || !out || !d_q_offsets || !d_n_q || !d_tokens) return Q3KV_ERR_INVALID_ARG;
    if (!aligned16(logits) || !aligned16(out) || (d_counts && !aligned16(d_counts))) return Q3KV_ERR_INVALID_ARG;
    if (d_bias_offsets && num_biases > 0 && (!d_bias_tokens || !d_bias_values)) return Q3KV_ERR_INVALID_ARG;
    const int64_t size = dtype == Q3KV_F32 ? 4 : 2, bytes = (int64_t)num_rows * vocab * size, slots4 = 4 * (int64_t)num_slots;
    if (logits != out && overlap(out, bytes, logits, bytes)) return Q3KV_ERR_INVALID_ARG;
    if (overlap(out, bytes, d_q_offsets, slots4) || overlap(out, bytes, d_n_q, slots4) || overlap(out, bytes, d_tokens, 4 * (int64_t)num_rows) ||
        (d_counts && overlap(out, bytes, d_counts, 2 * num_slots * counts_stride)) || (d_repetition && overlap(out, bytes, d_repetition, slots4)) ||
        (d_frequency && overlap(out, bytes, d_frequency, slots4)) || (d_presence && overlap(out, bytes, d_presence, slots4)) ||
        (d_bias_offsets && (overlap(out, bytes, d_bias_offsets, slots4 + 4) || overlap(out, bytes, d_bias_tokens, 4 * (int64_t)num_biases) ||
                            overlap(out, bytes, d_bias_values, 4 * (int64_t)num_biases))) ||
        (d_mask && overlap(out, bytes, d_mask, 4 * (int64_t)num_rows * ((vocab + 31) / 32))) || (d_status && overlap(out, bytes, d_status, 4)))
        return Q3KV_ERR_INVALID_ARG;
    LogitArgs a{};
    a.logits = logits;
    a.out = out;
    a.vocab = vocab;
    a.q_offsets = d_q_offsets;
    a.n_q = d_n_q;
    a.tokens = d_tokens;
    a.num_rows = num_rows;
    a.max_n_q = max_n_q;
    a.counts = d_counts;
    a.counts_stride = counts_stride;
    a.repetition = d_repetition;
    a.frequency = d_frequency;
    a.presence = d_presence;
    a.bias_offsets = d_bias_offsets;
    a.bias_tokens = d_bias_tokens;
    a.bias_values = d_bias_values;
    a.num_biases = num_biases;
    a.mask = d_mask;
    a.status = d_status;
    const dim3 grid((unsigned)(((int64_t)vocab + kChunk - 1) / kChunk), (unsigned)num_slots, (unsigned)((max_n_q + kBatch - 1) / kBatch));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // rows start on 16 bytes and end with a whole group of 8 entries
    const bool vec = vocab % 8 == 0;
    if (dtype == Q3KV_F32)
        return cuda_status(vec ? launch(process_logits_kernel<float, true>, a, grid, 0, st) : launch(process_logits_kernel<float, false>, a, grid, 0, st));
    return cuda_status(vec ? launch(process_logits_kernel<__nv_bfloat16, true>, a, grid, 0, st)
                           : launch(process_logits_kernel<__nv_bfloat16, false>, a, grid, 0, st));
}

}  // extern "C"
