// Rotary positions with several axes, for the query and key rows of a step.
//
// Pair i of a row turns by a_i = position[axis_i] * f_i:
//   (x, y) -> (x cos a - y sin a, x sin a + y cos a),
// float32, rounded once to the output type.  The angle is kept in turns as a
// 64-bit fixed-point fraction: position * turns_i modulo 2^64 drops whole turns
// exactly, so its error is that of the frequency times the position.  The frequency
// carries a few roundings of a double below 0.16 (pow, 2 pi, the division): at most 2^-53
// of a turn a position (2^-55 was the largest found against 300-bit arithmetic), 2^-33 at
// 10^6 positions; a caller who needs more fills in turns[].  The top 32 bits, read
// as a signed number of turns in [-1/2, 1/2), go to sincospi.  The product is
// integer work; no float64 is needed.
//
// Bound: memory (a row is read and written once): 4,096 rows of 18 bf16 heads take 14.8 us,
// 5,100 GB/s; 8,191 float32 rows 50.4 us, 6,000 GB/s; 6 rows 2.4 us, one launch.  One CTA takes kRowsPerCta
// rows: its threads first fill the rows' (cos, sin) table in shared memory, once
// per row for all its heads, with the first 32 bytes of their data already
// in flight, then rotate.  A work item is two 16-byte vectors of one head: the
// two partners of a half-split pair, or two neighbours otherwise (the copied
// tail among them), so every load and store is 16 bytes wide.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "q3kv_internal.h"

namespace q3kv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kMaxRowsPerCta = 2;

struct RopeArgs {
    q3kv_rope_plan plan;
    const int32_t* positions;
    int32_t num_rows;
    int32_t rows_per_cta;
    int32_t heads[2];            // q, k
    const void* in[2];
    void* out[2];
    int64_t in_stride[2];
    int64_t out_stride[2];
};

__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8], const __nv_bfloat16*) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4], const float*) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8], const __nv_bfloat16*) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4], const float*) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}

// One work item: two vectors, at elements e0 and e1 of head h (q heads first)
// of row r of the CTA; pair0 is the pair of its first rotated element, or -1
// in the tail that is copied.
struct Item {
    const uint4* src0;
    const uint4* src1;
    uint4* dst0;
    uint4* dst1;
    int row;
    int pair0;
};

template <typename T, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int V = 16 / sizeof(T);                    // elements per 16-byte vector
    constexpr int kSlots = kHeadDim / V / 2;             // work items per head
    __shared__ __align__(16) float2 cs[kMaxRowsPerCta][kMaxPairs];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row0 = blockIdx.x * a.rows_per_cta;
    const int rows = min(a.rows_per_cta, a.num_rows - row0);
    const int half = a.plan.rotary_dim / 2;
    const int heads = a.heads[0] + a.heads[1];
    const int per_row = heads * kSlots;
    const int total = rows * per_row;

    auto item_of = [&](int idx) {
        Item it;
        const int r = idx / per_row, rest = idx - r * per_row;
        const int hh = rest / kSlots, s = rest % kSlots;
        const int which = hh >= a.heads[0] ? 1 : 0;
        const int h = which ? hh - a.heads[0] : hh;
        const int rot_slots = half / V;                  // rotary_dim is a multiple of 16, so of 2 V
        const bool rot = s < rot_slots;
        int e0, e1;
        if (ADJ || !rot) {
            e0 = 2 * V * s;
            e1 = e0 + V;
            it.pair0 = rot ? e0 / 2 : -1;
        } else {
            e0 = V * s;
            e1 = e0 + half;
            it.pair0 = e0;
        }
        const int64_t row = row0 + r;
        const T* in = static_cast<const T*>(a.in[which]) + row * a.in_stride[which] + h * kHeadDim;
        T* out = static_cast<T*>(a.out[which]) + row * a.out_stride[which] + h * kHeadDim;
        it.src0 = reinterpret_cast<const uint4*>(in + e0);
        it.src1 = reinterpret_cast<const uint4*>(in + e1);
        it.dst0 = reinterpret_cast<uint4*>(out + e0);
        it.dst1 = reinterpret_cast<uint4*>(out + e1);
        it.row = r;
        return it;
    };

    // the first item's data is in flight while the table is made
    Item it;
    uint4 u0, u1;
    int idx = threadIdx.x;
    if (idx < total) {
        it = item_of(idx);
        u0 = *it.src0;
        u1 = *it.src1;
    }
    for (int k = threadIdx.x; k < rows * half; k += kRopeThreads) {
        const int r = k / half, i = k - r * half;
        const int32_t pos = a.positions[(int64_t)(row0 + r) * a.plan.num_axes + a.plan.axis[i]];
        const uint64_t t = (uint64_t)(int64_t)pos * a.plan.turns[i];       // turns mod 1, exact
        const int32_t top = (int32_t)(uint32_t)((t + 0x80000000ull) >> 32);
        float s, c;
        sincospif((float)top * (1.0f / 2147483648.0f), &s, &c);            // pi * 2 * (top / 2^32)
        cs[r][i] = make_float2(c, s);
    }
    __syncthreads();

    while (idx < total) {
        const Item cur = it;
        const uint4 v0 = u0, v1 = u1;
        idx += kRopeThreads;
        if (idx < total) {                                                 // the next item's data
            it = item_of(idx);
            u0 = *it.src0;
            u1 = *it.src1;
        }
        if (cur.pair0 < 0) {
            *cur.dst0 = v0;
            *cur.dst1 = v1;
            continue;
        }
        float x[V], y[V];
        unpack(v0, x, static_cast<const T*>(nullptr));
        unpack(v1, y, static_cast<const T*>(nullptr));
        const float2* t = &cs[cur.row][cur.pair0];
        if (ADJ) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 p = t[i], q = t[i + V / 2];
                const float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
                x[2 * i] = x0 * p.x - x1 * p.y;
                x[2 * i + 1] = x0 * p.y + x1 * p.x;
                y[2 * i] = y0 * q.x - y1 * q.y;
                y[2 * i + 1] = y0 * q.y + y1 * q.x;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const float4 p = *reinterpret_cast<const float4*>(t + i);
                const float x0 = x[i], y0 = y[i], x1 = x[i + 1], y1 = y[i + 1];
                x[i] = x0 * p.x - y0 * p.y;
                y[i] = x0 * p.y + y0 * p.x;
                x[i + 1] = x1 * p.z - y1 * p.w;
                y[i + 1] = x1 * p.w + y1 * p.z;
            }
        }
        *cur.dst0 = pack(x, static_cast<const T*>(nullptr));
        *cur.dst1 = pack(y, static_cast<const T*>(nullptr));
    }
}

template <typename T, bool ADJ>
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.num_rows + a.rows_per_cta - 1) / a.rows_per_cta));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<T, ADJ>, a);
}

// A frequency's fraction of a turn per position as a 64-bit fixed-point number.
// f < 1 rad, so f / 2 pi < 0.16 and f / 2 pi * 2^64 fits; the double's 53 bits
// are kept whole by scaling with a power of two (the bits below them are zeros).
uint64_t turns_of(double f) {
    const double two_pi = 6.283185307179586476925286766559;
    const double x = f / two_pi * 18446744073709551616.0;
    return (uint64_t)(x + 0.5);
}

bool rows_ok(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int32_t heads, size_t esize) {
    if (heads == 0) return true;
    if (!in || !out || !aligned16(in) || !aligned16(out)) return false;
    const int64_t least = (int64_t)heads * kHeadDim;
    const int64_t step = (int64_t)(16 / esize);
    return in_stride >= least && out_stride >= least && in_stride % step == 0 && out_stride % step == 0;
}

// Rows [p + i step, + width) in bytes, i < n; step >= width where n > 1.
struct Rows {
    const void* p;
    int64_t step, width, n;
};

// Two sets of rows share a byte.  Rows may interleave (query and key rows of one projection): equal steps are
// one division, others a division a row of a, taken only where the extents meet.
bool rows_meet(const Rows& a, const Rows& b) {
    if (!overlap(a.p, (a.n - 1) * a.step + a.width, b.p, (b.n - 1) * b.step + b.width)) return false;
    const int64_t delta = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    auto floor_div = [](int64_t x, int64_t y) { return x >= 0 ? x / y : -((-x + y - 1) / y); };
    if (a.step == b.step) {
        // row j of b against row i of a, d = j - i: the last one that begins before a's end
        const int64_t d = std::min(floor_div(a.width - 1 - delta, b.step), b.n - 1);
        return d >= 1 - a.n && delta + d * b.step > -b.width;
    }
    for (int64_t i = 0; i < a.n; ++i) {
        const int64_t from = delta - i * a.step;             // b's first row from row i of a
        const int64_t j = std::min(floor_div(a.width - 1 - from, b.step), b.n - 1);
        if (j >= 0 && from + j * b.step > -b.width) return true;
    }
    return false;
}

}  // namespace
}  // namespace q3kv

using namespace q3kv;

extern "C" {

int q3kv_rope_plan_init(const q3kv_rope_config* c, q3kv_rope_plan* plan) {
    if (!c || !plan) return Q3KV_ERR_INVALID_ARG;
    if (!(c->theta > 1.0) || !(c->theta < 1.0e300)) return Q3KV_ERR_INVALID_ARG;
    if (c->rotary_dim < 16 || c->rotary_dim > kHeadDim || c->rotary_dim % 16 != 0) return Q3KV_ERR_INVALID_ARG;
    if (c->num_axes < 1 || c->num_axes > Q3KV_ROPE_MAX_AXES) return Q3KV_ERR_INVALID_ARG;
    if (c->flags & ~(Q3KV_ROPE_ADJACENT | Q3KV_ROPE_DEAL_AXES | Q3KV_ROPE_AXIS_FREQS)) return Q3KV_ERR_INVALID_ARG;
    if (c->reserved != 0) return Q3KV_ERR_INVALID_ARG;
    const int half = c->rotary_dim / 2;
    int64_t sum = 0;
    for (int a = 0; a < c->num_axes; ++a) {
        if (c->sections[a] < 0) return Q3KV_ERR_INVALID_ARG;
        sum += c->sections[a];
    }
    if (sum != half) return Q3KV_ERR_INVALID_ARG;
    q3kv_rope_plan p = {};
    p.rotary_dim = c->rotary_dim;
    p.num_axes = c->num_axes;
    p.flags = c->flags;
    int seen[Q3KV_ROPE_MAX_AXES] = {0, 0, 0, 0};
    int axis = 0;
    for (int i = 0; i < half; ++i) {
        // the axis of pair i: the next one with pairs left, moving on after every
        // pair (dealt) or only when it has all of its own (runs)
        while (seen[axis] == c->sections[axis]) axis = (axis + 1) % c->num_axes;
        const double e = (c->flags & Q3KV_ROPE_AXIS_FREQS) ? (double)seen[axis] / c->sections[axis] : (double)i / half;
        p.turns[i] = turns_of(pow(c->theta, -e));
        p.axis[i] = (uint8_t)axis;
        ++seen[axis];
        if (c->flags & Q3KV_ROPE_DEAL_AXES) axis = (axis + 1) % c->num_axes;
    }
    *plan = p;
    return Q3KV_OK;
}

int q3kv_rope(void* stream, const q3kv_rope_plan* plan, const int32_t* d_positions, int32_t num_rows,
              const void* q_in, int64_t q_in_stride, void* q_out, int64_t q_out_stride, int32_t num_q_heads,
              const void* k_in, int64_t k_in_stride, void* k_out, int64_t k_out_stride, int32_t num_kv_heads,
              int32_t dtype) {
    if (!plan || num_rows < 0 || num_q_heads < 0 || num_kv_heads < 0) return Q3KV_ERR_INVALID_ARG;
    if (num_q_heads > 4096 || num_kv_heads > 4096) return Q3KV_ERR_UNSUPPORTED;
    if (dtype != Q3KV_F32 && dtype != Q3KV_BF16) return Q3KV_ERR_INVALID_ARG;
    if (plan->rotary_dim < 16 || plan->rotary_dim > kHeadDim || plan->rotary_dim % 16 != 0 || plan->num_axes < 1 ||
        plan->num_axes > Q3KV_ROPE_MAX_AXES)
        return Q3KV_ERR_INVALID_ARG;
    for (int i = 0; i < plan->rotary_dim / 2; ++i)
        if (plan->axis[i] >= plan->num_axes) return Q3KV_ERR_INVALID_ARG;
    if (num_rows == 0 || num_q_heads + num_kv_heads == 0) return Q3KV_OK;
    const size_t esize = dtype == Q3KV_F32 ? 4 : 2;
    if (!d_positions || !rows_ok(q_in, q_in_stride, q_out, q_out_stride, num_q_heads, esize) ||
        !rows_ok(k_in, k_in_stride, k_out, k_out_stride, num_kv_heads, esize))
        return Q3KV_ERR_INVALID_ARG;
    // an output may lie on its own input's rows and on no other operand's
    const int64_t es = (int64_t)esize, wq = num_q_heads * (int64_t)kHeadDim * es, wk = num_kv_heads * (int64_t)kHeadDim * es;
    const Rows qi{q_in, q_in_stride * es, wq, num_rows}, qo{q_out, q_out_stride * es, wq, num_rows};
    const Rows ki{k_in, k_in_stride * es, wk, num_rows}, ko{k_out, k_out_stride * es, wk, num_rows};
    const Rows pos{d_positions, 4ll * plan->num_axes, 4ll * plan->num_axes, num_rows};
    const bool q = num_q_heads > 0, k = num_kv_heads > 0;
    auto same = [](const Rows& x, const Rows& y) { return x.p == y.p && (x.step == y.step || x.n == 1); };
    if ((q && !same(qi, qo) && rows_meet(qi, qo)) || (k && !same(ki, ko) && rows_meet(ki, ko)) ||
        (q && k && (rows_meet(qo, ki) || rows_meet(ko, qi) || rows_meet(qo, ko))) || (q && rows_meet(pos, qo)) || (k && rows_meet(pos, ko)))
        return Q3KV_ERR_INVALID_ARG;
    RopeArgs a{};
    a.plan = *plan;
    a.positions = d_positions;
    a.num_rows = num_rows;
    // two rows per CTA where rows are many: the second row's loads overlap the first one's table and
    // rotation (4,096 rows of 18 bf16 heads 17.8 -> 15.1 us, four rows 16.2); few rows want their own
    // CTAs (6 rows: 2.4 us against 2.8)
    a.rows_per_cta = num_rows >= 1024 ? 2 : 1;
    a.heads[0] = num_q_heads;
    a.heads[1] = num_kv_heads;
    a.in[0] = q_in;
    a.in[1] = k_in;
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.in_stride[0] = q_in_stride;
    a.in_stride[1] = k_in_stride;
    a.out_stride[0] = q_out_stride;
    a.out_stride[1] = k_out_stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool adj = (plan->flags & Q3KV_ROPE_ADJACENT) != 0;
    if (dtype == Q3KV_F32)
        return cuda_status(adj ? launch_rope<float, true>(a, st) : launch_rope<float, false>(a, st));
    return cuda_status(adj ? launch_rope<__nv_bfloat16, true>(a, st) : launch_rope<__nv_bfloat16, false>(a, st));
}

}  // extern "C"
