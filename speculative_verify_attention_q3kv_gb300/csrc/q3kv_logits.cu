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
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "q3kv_internal.h"

namespace q3kv {
namespace {

constexpr int kMaxVocab = 1 << 28;            // entries' indexes, and those of the vectors behind the last, fit 32 bits
constexpr int kThreads = 256;
constexpr int kPer = 8;                       // entries per thread
constexpr int kChunk = kThreads * kPer;       // vocabulary entries per CTA
constexpr int kBiasAhead = 2;

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

// A CTA takes 2,048 entries of a slot's rows, or of a part of them where the CTAs would be few, one row after the other.
// Bound: bytes (logits in and out) and, close behind, issue slots.  So the rows come by asynchronous 16-byte copies into a
// ring of two, whole vectors also where a row does not start on one, and no registers hold them (longer rings and rows in
// groups cost more in CTAs per SM than they hide: 8 slots x 16 float32 17.0 us, three rows 17.5, two groups of two 18.6; with
// four CTAs per SM instead of five 18.7); an entry's penalty
// alpha c + beta [c > 0] - bias is worked out once for all rows but where the step's own tokens count; and a warp
// looks only at those of its eight steps in which some lane's entry changes (most entries are not seen, away from the
// frequent tokens): the others only take the mask.
constexpr int kRing = 2;                      // rows
template <typename T>
constexpr int kRowBytes = kChunk * (int)sizeof(T) + 16;

// 16 bytes to shared memory, of which the first `bytes` are read and the rest becomes zero.
__device__ __forceinline__ void copy16(void* dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(bytes) : "memory");
}

// 8 entries with the ones whose bit is 0 set to -inf
__device__ __forceinline__ void apply_mask(Row8<float>& o, uint32_t allowed) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        if (!((allowed >> e) & 1u)) o.x[e] = -CUDART_INF_F;
}
// Each byte of the result: the sign of one of x's bytes, in all its bits.
template <uint32_t SELECT>
__device__ __forceinline__ uint32_t spread(uint32_t x) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(x), "n"(SELECT));
    return r;
}
__device__ __forceinline__ void apply_mask(Row8<__nv_bfloat16>& o, uint32_t allowed) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
    for (int e = 0; e < kPer; e += 4) {
        // bits e .. e + 3 to the sign bits of four bytes, which the permutations then repeat over two bytes each
        const uint32_t signs = (((allowed >> e) & 15u) * 0x00204081u & 0x01010101u) << 7;
        const uint32_t low = spread<0x9988>(signs), high = spread<0xbbaa>(signs);
        w[e / 2] = (w[e / 2] & low) | (0xff80ff80u & ~low);
        w[e / 2 + 1] = (w[e / 2 + 1] & high) | (0xff80ff80u & ~high);
    }
}
__device__ __forceinline__ bool same_bits(uint4 a, uint4 b) { return ((a.x ^ b.x) | (a.y ^ b.y) | (a.z ^ b.z) | (a.w ^ b.w)) == 0; }

// Where the ids do not ascend throughout, one may be left twice (5, 3, 5): by one warp and in order, so that the last entry stays.
// A call of its own: inlined, it costs rows of an odd vocabulary 5 % whether they have biases or not.
__device__ __noinline__ void biases_in_order(const int32_t* tokens, const float* values, int b0, int b1, int base, int limit, float* s_bias) {
    const int lane = threadIdx.x & 31;
    for (int i0 = b0; i0 < b1; i0 += 32) {
        const int i = i0 + lane;
        const int t = i < b1 ? tokens[i] : -1, before = i > b0 && i < b1 ? tokens[i - 1] : -1;
        const bool mine = t >= base && t < limit && before < t;
        const uint32_t same = __match_any_sync(0xffffffffu, mine ? t : -1);
        if (mine && lane == 31 - __clz(same)) s_bias[t - base] = values[i];
        __syncwarp();
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 5) process_logits_kernel(LogitArgs a, int per) {
    extern __shared__ __align__(16) uint8_t s_rows[];       // [kRing][kRowBytes]
    __shared__ float s_bias[kChunk];
    __shared__ int s_tok[kMaxNq];
    __shared__ int s_unsorted;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, slot = blockIdx.y;
    const int base = blockIdx.x * kChunk;
    const int w = a.n_q[slot], r0 = a.q_offsets[slot];
    int b0 = 0, b1 = 0;
    if (a.bias_offsets) {
        b0 = a.bias_offsets[slot];
        b1 = a.bias_offsets[slot + 1];
    }
    const float theta = a.repetition ? a.repetition[slot] : 1.0f;
    const float alpha = a.frequency ? a.frequency[slot] : 0.0f, beta = a.presence ? a.presence[slot] : 0.0f;
    // this thread's entries: vectors of 16 bytes, neighbours in neighbouring threads, or single ones where rows are not aligned
    constexpr int kVec = VEC ? 16 / (int)sizeof(T) : 1, kVecs = kPer / kVec, kNext = kThreads * kVec;
    const int first = base + tid * kVec;
    const auto off = [](int e) { return e / kVec * kNext + e % kVec; };
    Row8<int16_t> count;
    {
        const int16_t* c = a.counts + (int64_t)slot * a.counts_stride + first;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {                      // the stride covers whole vectors
            using V = std::conditional_t<kVec == 8, uint4, std::conditional_t<kVec == 4, uint2, int16_t>>;
            reinterpret_cast<V*>(&count)[v] = a.counts && first + v * kNext < a.vocab ? *reinterpret_cast<const V*>(c + v * kNext) : V{};
        }
    }
    const bool report = blockIdx.x == 0 && blockIdx.z == 0 && a.status;
    if (w == 0) return;
    if (w < 0 || w > a.max_n_q || r0 < 0 || r0 > a.num_rows - w) {
        if (report && tid == 0) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        return;
    }
    const int j0 = blockIdx.z * per, j1 = min(w, j0 + per);      // rows of this CTA
    if (j0 >= j1) return;
    const int64_t begin = ((int64_t)(r0 + j0) * a.vocab + base) * (int)sizeof(T);      // byte of the first row's first entry
    const int64_t row_bytes = (int64_t)a.vocab * (int)sizeof(T);
    const int bytes = min(kChunk, a.vocab - base) * (int)sizeof(T);
    const uint8_t* in = static_cast<const uint8_t*>(a.logits) + begin;      // the next row to be copied
    int ahead = j0;
    auto copy_row = [&]() {                                        // empty behind the last row
        if (ahead < j1) {
            uint8_t* to = s_rows + (ahead - j0) % kRing * kRowBytes<T>;
            if (VEC) {                                             // each thread its own entries
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
                    if (first + v * kNext < a.vocab) copy16(to + (v * kThreads + tid) * 16, in + (v * kThreads + tid) * 16, 16);
            } else {
                const int shift = (int)(reinterpret_cast<uintptr_t>(in) & 15);       // the buffer begins on 16 bytes
                for (int at = tid * 16; at < bytes + shift; at += kThreads * 16) copy16(to + at, in - shift + at, min(16, bytes + shift - at));
            }
            in += row_bytes;
            ++ahead;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    copy_row();
    // masks: this thread's bits, or, as a warp's entries of one step share a word where rows are not aligned, step `lane`'s word
    const int64_t mask_bytes = (a.vocab + 31) / 32 * 4;
    const int word = (first - lane + lane * kNext) >> 5;
    const bool own = a.mask && (VEC ? first < a.vocab : lane < kPer && word * 4 < mask_bytes);
    const uint8_t* mask = reinterpret_cast<const uint8_t*>(a.mask) + (r0 + j0) * mask_bytes;
    auto load_mask = [&](int j) -> uint32_t {
        if (!own || j >= j1) return VEC ? 0xffu : 0u;
        if (!VEC) return reinterpret_cast<const uint32_t*>(mask)[word];
        uint32_t bits = mask[first >> 3];
        if (kVecs == 2) {                                          // a half of each of two bytes
            const uint32_t more = first + kNext < a.vocab ? mask[(first + kNext) >> 3] : 0u;
            bits = (bits >> (first & 4) & 15u) | (more >> (first & 4) & 15u) << 4;
        }
        return bits;
    };
    uint32_t allowed = load_mask(j0);
    bool near = false;                   // a token of the step is in the chunk
    if (tid < w) {
        const int t = a.tokens[r0 + tid];
        s_tok[tid] = t;
        if (report && (t < 0 || t >= a.vocab)) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
        near = t >= base && t < min(base + kChunk, a.vocab) && tid < j1;
    }
    if (b0 < 0 || b1 < b0 || b1 > a.num_biases) {
        if (report && tid == 0) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        b0 = b1 = 0;
    }
    bool biased = false;                 // a bias is
    if (b1 > b0) {
        if (tid == 0) s_unsorted = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s_bias[tid + i * kThreads] = 0.0f;
        __syncthreads();
        for (int i0 = b0 + tid; i0 < b1; i0 += kBiasAhead * kThreads) {
            int t[kBiasAhead], before[kBiasAhead];
            float value[kBiasAhead];
#pragma unroll
            for (int k = 0; k < kBiasAhead; ++k) {             // all loads at once, also of values that are not needed
                const int i = i0 + k * kThreads;
                t[k] = i < b1 ? a.bias_tokens[i] : 0;
                before[k] = i < b1 && i > b0 ? a.bias_tokens[i - 1] : -1;
                value[k] = i < b1 ? a.bias_values[i] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kBiasAhead; ++k) {
                if (i0 + k * kThreads >= b1) break;
                // ascending ids: no id twice, so no order of the stores
                if (t[k] < 0 || t[k] >= a.vocab || before[k] >= t[k]) {
                    s_unsorted = 1;
                    if (report) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
                } else if (t[k] >= base && t[k] < base + kChunk) {
                    s_bias[t[k] - base] = value[k];
                    biased = true;
                }
            }
        }
        biased = __syncthreads_or(biased);
        if (s_unsorted && biased && tid < 32) biases_in_order(a.bias_tokens, a.bias_values, b0, b1, base, min(base + kChunk, a.vocab), s_bias);
    }
    near = __syncthreads_or(near);

    // what this thread's entries lose in every row, and where the step's tokens add to it
    const uint32_t* words = reinterpret_cast<const uint32_t*>(&count);
    uint32_t seen = 0, marks = 0;        // bit e: entry e is seen in every row; it changes in some
    if (words[0] | words[1] | words[2] | words[3])
#pragma unroll
        for (int e = 0; e < kPer; ++e) seen |= (count.x[e] != 0 ? 1u : 0u) << e;
    marks = seen;
    if (biased)
#pragma unroll
        for (int e = 0; e < kPer; ++e) marks |= (s_bias[first - base + off(e)] != 0.0f ? 1u : 0u) << e;
    uint32_t step[kPer / 2] = {0, 0, 0, 0};                 // 16 bits per entry, bit i set where t_i is the entry
    if (near)
        for (int i = 0; i < j1; ++i) {
            const int d = s_tok[i] - first;
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (d == off(e)) {
                    step[e / 2] |= 1u << (i + 16 * (e & 1));
                    marks |= 1u << e;
                }
        }
    const uint32_t changing = __reduce_or_sync(0xffffffffu, marks);     // the warp skips the other entries
    float less[kPer];
    float inverse = 1.0f;
    if (changing) {
        inverse = __fdiv_rn(1.0f, theta);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int c = count.x[e] & 0x7fff;
            less[e] = c > 0 ? fmaf(alpha, (float)c, beta) : 0.0f;
            if (biased) less[e] -= s_bias[first - base + off(e)];
        }
    }
    const bool in_place = a.logits == a.out;
    const int valid = (a.vocab - first + kNext - 1) / kNext;      // this thread's vectors that exist
    uint8_t* out = static_cast<uint8_t*>(a.out) + begin;
#pragma unroll 1
    for (int j = j0; j < j1; ++j, out += row_bytes) {
        if (!VEC) __syncthreads();       // all are done with the row before, whose place the next one takes
        copy_row();
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (!VEC) __syncthreads();       // others' copies have landed too
        mask += mask_bytes;
        const uint32_t next = load_mask(j + 1);
        const uint8_t* row = s_rows + (j - j0) % kRing * kRowBytes<T>;
        Row8<T> x, o;
        if (VEC) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) reinterpret_cast<uint4*>(&x)[v] = reinterpret_cast<const uint4*>(row)[v * kThreads + tid];
        } else {
            const T* p = reinterpret_cast<const T*>(row + (reinterpret_cast<uintptr_t>(out) & 15)) + tid;      // in and out are aligned alike
#pragma unroll
            for (int e = 0; e < kPer; ++e) x.x[e] = p[e * kThreads];     // anything behind the end
        }
        o = x;
        if (changing) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (!((changing >> e) & 1u)) continue;
                float y = to_f32(x.x[e]), s = less[e];
                bool known = (seen >> e) & 1u;
                if (near) {
                    const int more = __popc(step[e / 2] & (((2u << j) - 1u) << (16 * (e & 1))));
                    if (more) {
                        s += (count.x[e] & 0x7fff) > 0 ? alpha * (float)more : fmaf(alpha, (float)more, beta);
                        known = true;
                    }
                }
                y = known ? y * (y > 0.0f ? inverse : theta) : y;
                o.x[e] = from_f32<T>(y - s);
            }
        }
        if (a.mask) {
            if (VEC) {
                apply_mask(o, allowed);
            } else {
                const uint32_t bit = 1u << lane;
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (!(__shfl_sync(0xffffffffu, allowed, e) & bit)) o.x[e] = from_f32<T>(-CUDART_INF_F);
            }
        }
        allowed = next;
        if (VEC) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const uint4 to = reinterpret_cast<const uint4*>(&o)[v];
                if (v < valid && (!in_place || !same_bits(to, reinterpret_cast<const uint4*>(&x)[v])))
                    reinterpret_cast<uint4*>(out)[v * kThreads + tid] = to;
            }
        } else {
            T* p = reinterpret_cast<T*>(out) + tid;
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (e < valid) p[e * kThreads] = o.x[e];
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
    const uint32_t now = min(((word >> shift) & kCountCap) + (uint32_t)add, (uint32_t)kCountCap);
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

constexpr int kFew = 64;      // tokens per slot up to which every token has a thread of its own

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
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i - (threadIdx.x & 31) >= n) return;      // whole warps leave
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

// Long histories: frequent tokens of many threads would meet in the same words.  So a CTA owns 16,384 vocabulary entries
// of a slot, reads all of the slot's tokens (they come from L2 for all but the first CTA), counts its own in shared
// memory and adds each entry once: no atomics in global memory, no order.  Where slots are few, a cluster of up to four
// CTAs shares a range's tokens, and each adds up its part of the entries from the shared memory of all (1 x 524,288: 13.5 us
// with four CTAs, 15.8 with eight, whose cluster takes 5 us more to start).
// Bound: the rounds' latency and issue slots; a token costs each range's CTA about seven instructions (8 x 65,536 of 248,320
// entries: 8.2 us, 11.7 with a check of the end at every token).
constexpr int kRange = 16384, kHistoryThreads = 1024;
constexpr unsigned kMaxParts = 4;

template <int kAhead, bool CLUSTER>      // loads under way per thread
__global__ void __launch_bounds__(kHistoryThreads) count_history_kernel(CountArgs a) {
    extern __shared__ __align__(16) int s_count[];              // [kRange]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int i = threadIdx.x; i < kRange / 4; i += kHistoryThreads) reinterpret_cast<int4*>(s_count)[i] = make_int4(0, 0, 0, 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int slot = blockIdx.y, base = blockIdx.x * kRange;
    int64_t begin;
    int n;
    if (!slot_range(a, slot, &begin, &n) || n == 0) return;
    __syncthreads();
    // this CTA's part of the tokens: whole rounds of kAhead loads per thread, then single ones
    const int64_t part = ((int64_t)n + gridDim.z - 1) / gridDim.z, first = min((int64_t)n, blockIdx.z * part);
    const int mine = (int)min(n - first, part);
    const int32_t* tokens = a.tokens + begin + first + threadIdx.x;
    const uint32_t entries = min(kRange, a.vocab - base);
    uint32_t largest = 0;                        // a negative token is a large number
    const auto add_one = [&](uint32_t t) {
        largest = max(largest, t);
        const uint32_t at = t - base;
        if (at < entries) atomicAdd(&s_count[at], 1);
    };
    int left = mine;
    for (; left >= kAhead * kHistoryThreads; left -= kAhead * kHistoryThreads, tokens += kAhead * kHistoryThreads) {
        uint32_t t[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) t[k] = tokens[k * kHistoryThreads];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) add_one(t[k]);
    }
    left -= threadIdx.x;
    uint32_t t[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (k * kHistoryThreads < left) t[k] = tokens[k * kHistoryThreads];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (k * kHistoryThreads < left) add_one(t[k]);
    if (largest >= (uint32_t)a.vocab && blockIdx.x == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_TOKEN);
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();      // the CTAs along z
    if (CLUSTER) cluster.sync();
    else __syncthreads();
    // two entries per word; the stride is even, so a word belongs to one slot and range
    uint32_t* words = reinterpret_cast<uint32_t*>(a.counts + (int64_t)slot * a.stride + base);
    const int share = CLUSTER ? kRange / 2 / gridDim.z : kRange / 2, from = CLUSTER ? blockIdx.z * share : 0;
    constexpr int kWords = kRange / 2 / kHistoryThreads;
    uint32_t was[kWords];
    int2 add[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int i = k * kHistoryThreads + threadIdx.x;
        add[k] = make_int2(0, 0);
        if (!CLUSTER) {
            add[k] = reinterpret_cast<const int2*>(s_count)[i];
        } else if (i < share) {
            int2 c[kMaxParts];
#pragma unroll
            for (unsigned r = 0; r < kMaxParts; ++r)
                c[r] = r < gridDim.z ? reinterpret_cast<const int2*>(cluster.map_shared_rank(s_count, r))[from + i] : make_int2(0, 0);
#pragma unroll
            for (unsigned r = 0; r < kMaxParts; ++r) {
                add[k].x += c[r].x;
                add[k].y += c[r].y;
            }
        }
        if (add[k].x | add[k].y) was[k] = words[from + i];
    }
#pragma unroll
    for (int k = 0; k < kWords; ++k)
        if (add[k].x | add[k].y) words[from + k * kHistoryThreads + threadIdx.x] = add_to(add_to(was[k], 0, add[k].x), 16, add[k].y);
    if (CLUSTER) cluster.sync();         // the others are done with this CTA's counts
}

template <typename K, typename A, typename... More>
cudaError_t launch(K kernel, const A& a, dim3 grid, size_t smem, cudaStream_t st, int threads = kThreads, More... more) {
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
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
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
    if (num_slots > 65535 || vocab > kMaxVocab) return Q3KV_ERR_UNSUPPORTED;
    if (num_slots == 0 || max_n == 0 || num_tokens == 0) return Q3KV_OK;
    if (!d_counts || !d_tokens || !d_offsets || !d_n || !aligned16(d_counts)) return Q3KV_ERR_INVALID_ARG;
    const int64_t bytes = (int64_t)num_slots * counts_stride * 2;
    if (overlap(d_counts, bytes, d_tokens, num_tokens * 4) || overlap(d_counts, bytes, d_offsets, (int64_t)num_slots * 4) ||
        overlap(d_counts, bytes, d_n, (int64_t)num_slots * 4) || (d_status && overlap(d_counts, bytes, d_status, 4)))
        return Q3KV_ERR_INVALID_ARG;
    CountArgs a{d_counts, counts_stride, vocab, d_tokens, num_tokens, d_offsets, d_n, max_n, d_status};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!prompt && max_n > kFew) {
        constexpr size_t smem = kRange * sizeof(int);
        int sms = 0;
        const int e = device_sm_count(&sms);
        if (e != Q3KV_OK) return e;
        const int64_t ranges = ((int64_t)vocab + kRange - 1) / kRange;
        // clusters while each CTA has an SM and 16,384 tokens at least (1 x 65,536: 8.0 us with one CTA per range, 7.4 with two,
        // 6.2 with four; 1 x 32,768: 5.9 with one, 6.2 with two)
        unsigned parts = 1;
        while (parts < kMaxParts && 2 * parts * ranges * num_slots <= sms && max_n / (2 * (int)parts) >= 16384) parts *= 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ranges, (unsigned)num_slots, parts);
        cfg.blockDim = dim3(kHistoryThreads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = parts;
        cfg.attrs = attr;
        cfg.numAttrs = parts > 1 ? 2 : 1;
        // 16 loads a thread let one CTA onto an SM, 8 two of them (8 x 65,536: 8.2 us with 16, 10.9 with 8; 32 x 4,096: 12.3 with
        // 16, 7.7 with 8)
        const int kind = parts > 1 ? 2 : ranges * num_slots > sms ? 1 : 0;
        static constexpr void (*kernels[3])(CountArgs) = {count_history_kernel<16, false>, count_history_kernel<8, false>,
                                                          count_history_kernel<16, true>};
        static std::atomic<bool> allowed[3][kMaxDevices];
        const cudaError_t ce = allow_smem(reinterpret_cast<const void*>(kernels[kind]), smem, allowed[kind]);
        return cuda_status(ce != cudaSuccess ? ce : cudaLaunchKernelEx(&cfg, kernels[kind], a));
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
    if (max_n_q > kMaxNq || num_slots > 65535 || vocab > kMaxVocab) return Q3KV_ERR_UNSUPPORTED;
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
    int sms = 0;
    const int e = device_sm_count(&sms);
    if (e != Q3KV_OK) return e;
    // a slot's rows go to one CTA per chunk where that gives every SM eight CTAs, else to several (8 slots x 16 float32:
    // 20.0 us with five per SM, 17.0 with eight, 19.0 with ten)
    const int64_t chunks = ((int64_t)vocab + kChunk - 1) / kChunk, few = chunks * num_slots;
    const int parts = (int)std::min<int64_t>(max_n_q, std::max<int64_t>(1, (8 * (int64_t)sms + few / 2) / few)), per = (max_n_q + parts - 1) / parts;
    const dim3 grid((unsigned)chunks, (unsigned)num_slots, (unsigned)((max_n_q + per - 1) / per));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // rows start on 16 bytes and end with a whole group of 8 entries
    const bool vec = vocab % 8 == 0;
    if (dtype == Q3KV_F32)
        return cuda_status(launch(vec ? process_logits_kernel<float, true> : process_logits_kernel<float, false>, a, grid,
                                  kRing * kRowBytes<float>, st, kThreads, per));
    return cuda_status(launch(vec ? process_logits_kernel<__nv_bfloat16, true> : process_logits_kernel<__nv_bfloat16, false>, a, grid,
                              kRing * kRowBytes<__nv_bfloat16>, st, kThreads, per));
}

}  // extern "C"
