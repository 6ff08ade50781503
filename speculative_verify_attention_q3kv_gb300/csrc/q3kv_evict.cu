// Eviction by attention mass: choose the positions to keep, compact their records.
//
// select_kernel, one thread-block cluster per (layer, slot, kv head) row: a radix
// select over the masses' order keys finds the k-th largest (k = budget minus the
// protected positions) exactly, 11 + 11 + 10 bits.  Every CTA of the cluster counts
// its own contiguous segment in shared memory; the cluster adds the histograms
// through distributed shared memory and every CTA walks the totals itself.  Then
// each CTA takes its segment in order (ballots within a warp, a scan over the warps)
// and writes positions and masses at their final ranks: the CTAs before it hold
// known counts above and at the threshold, and of the positions at the threshold
// the lowest ones are taken.  No float is added, so nothing depends on an order.
// A segment of at most 4,096 positions stays in registers over the five passes;
// longer ones are read again, from L2, with eight loads of a thread in flight.  512
// threads of at most 64 registers let two CTAs share an SM, so that the clusters of
// 38 rows run at once (one CTA of 1,024 threads per SM left room for a dozen).
//
// gather_kernel: a CTA moves up to 256 kept records, one destination page, of K and V:
// their source offsets go to shared memory first, so all 16-byte loads (4-byte ones
// for the 164-byte K records) of a thread are independent, and the stores, to
// consecutive records, coalesce.
//
// Bound: memory (masses read once from HBM and again from L2, kept records read
// and written once; a 112-byte record scattered over 64-byte DRAM bursts costs about
// half as much again to read).
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>

#include "q3kv_internal.h"

namespace cg = cooperative_groups;

namespace q3kv {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPerLane = 8;                               // elements of a lane per ordered tile
constexpr int kTileElems = kSelThreads * kPerLane;
constexpr int kBins = 2048;
constexpr int kLevels = 3;
constexpr int kMaxCluster = 8;

struct EvictArgs {
    uint8_t* pool;
    const int32_t* page_table;
    int32_t max_pages_per_slot;
    const int32_t* ctx_len;
    int32_t num_slots;
    int64_t max_ctx_len;
    const int32_t* budget;
    int32_t max_budget;
    int32_t n_sink, n_recent;
    int32_t layer, num_call_layers;
    const float* mass;
    int64_t mass_stride;
    const int32_t* dst_table;
    int32_t dst_max_pages;
    int32_t* kept;
    float* mass_out;
    int32_t* new_len;
    int32_t* status;
    int32_t num_layers, num_kv_heads, num_pages;
};

// What a slot keeps: n positions of L, `recent` last ones and `sink` first ones
// protected; n = 0 leaves the slot out.
struct SlotPlan {
    int L, n, sink, recent;
    bool bad;
};

__device__ __forceinline__ SlotPlan slot_plan(const EvictArgs& a, int slot) {
    SlotPlan s;
    s.L = a.ctx_len[slot];
    const int budget = a.budget[slot];
    s.bad = budget > 0 && (budget > a.max_budget || s.L < 0 || s.L > a.max_ctx_len ||
                           s.L > (int64_t)a.max_pages_per_slot * kPageSize ||
                           min(s.L, budget) > (int64_t)a.dst_max_pages * kPageSize);
    s.n = (budget <= 0 || s.bad) ? 0 : min(s.L, budget);
    s.recent = min(a.n_recent, s.n);
    s.sink = min(a.n_sink, s.n - s.recent);
    return s;
}

// Order key of a mass: larger masses have larger keys, -0 equals +0, NaN is below all.
__device__ __forceinline__ uint32_t mass_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);          // -0 + 0 = +0
    const uint32_t key = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return x == x ? key : 0u;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ int warp_scan(int v) {   // inclusive
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

struct __align__(16) SelectSmem {
    int hist[kLevels][kBins];   // this CTA's counts
    int coarse[kLevels][64];    // and of 32 bins each
    int warp_a[kSelWarps];
    int warp_b[kSelWarps];
    int found_bin;
    int found_above;            // entries in bins above it
    int local[2];               // this CTA's entries above the threshold, and at it
};

__global__ void __launch_bounds__(kSelThreads, 2) select_kernel(const EvictArgs a) {
    __shared__ SelectSmem sm;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / C;                    // (layer, slot, kv head)
    const int slot = (int)(row / a.num_kv_heads) % a.num_slots;
    const SlotPlan s = slot_plan(a, slot);
    if (rank == 0 && tid == 0 && row % a.num_kv_heads == 0 && row / a.num_kv_heads < a.num_slots) {   // one per slot
        if (s.bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        // where new_len is the array ctx_len, length_kernel writes it when every kernel has read it
        if (a.new_len != a.ctx_len) a.new_len[slot] = s.n > 0 ? s.n : s.L;
    }
    if (s.n == 0) return;                                  // the whole cluster agrees

    const float* m = a.mass + row * a.mass_stride;
    int32_t* kept = a.kept + row * a.max_budget;
    float* mass_out = a.mass_out ? a.mass_out + row * a.max_budget : nullptr;
    const int lo = s.sink, hi = s.L - s.recent;            // free positions [lo, hi)
    const int k = s.n - s.sink - s.recent;                 // of which k are kept
    // protected positions keep their order at both ends
    for (int i = rank * kSelThreads + tid; i < s.sink + s.recent; i += C * kSelThreads) {
        const int pos = i < s.sink ? i : s.L - s.recent + (i - s.sink);
        const int dst = i < s.sink ? i : s.n - s.recent + (i - s.sink);
        kept[dst] = pos;
        if (mass_out) mass_out[dst] = m[pos];
    }
    const int count = hi - lo;
    const int seg = ((count + C - 1) / C + 31) / 32 * 32;
    const int begin = min(hi, lo + rank * seg), end = min(hi, begin + seg);

    if (tid < 2) sm.local[tid] = 0;
    for (int i = tid; i < kLevels * kBins / 4; i += kSelThreads) reinterpret_cast<int4*>(&sm.hist[0][0])[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    uint32_t prefix = 0u;                                  // key bits found so far
    int want = k;                                          // entries still to take at or below the prefix's range
    bool nan = false;
    // tile t0 of the segment: a warp has 32 * kPerLane consecutive positions, 32 at a time
    float x[kPerLane];
    auto load_tile = [&](int t0) {
        const int i0 = t0 + warp * 32 * kPerLane + lane;
        if (t0 + kTileElems <= end) {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) x[j] = __ldg(m + i0 + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) x[j] = i0 + 32 * j < end ? __ldg(m + i0 + 32 * j) : 0.0f;
        }
    };
    // one pass of a radix level over the tile in x: counts the keys that begin with the prefix
    auto count_tile = [&](int t0, int level) {
        const int i0 = t0 + warp * 32 * kPerLane + lane;
        const int left = end - i0;                         // entry j exists if 32 j < left
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            const uint32_t key = mass_key(x[j]);
            const bool in = level == 0 || (level == 1 ? key >> 21 : key >> 10) == prefix;
            const uint32_t bin = level == 0 ? key >> 21 : (level == 1 ? (key >> 10) & 2047u : key & 1023u);
            if (in && 32 * j < left) atomicAdd(&sm.hist[level][bin], 1);
            if (level == 0) nan |= x[j] != x[j];
        }
    };
    const bool resident = end - begin <= kTileElems;       // one tile: loaded once
    if (resident) load_tile(begin);
    if (k > 0 && k < count) {
#pragma unroll
        for (int level = 0; level < kLevels; ++level) {
#pragma unroll 1
            for (int t0 = begin; t0 < end; t0 += kTileElems) {
                if (!resident) load_tile(t0);
                count_tile(t0, level);
            }
            __syncthreads();
            {   // thread t adds bins 4 t .. 4 t + 3, eight threads a coarse bin
                const int4 u = reinterpret_cast<const int4*>(&sm.hist[level][0])[tid];
                int t = (u.x + u.y) + (u.z + u.w);
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if ((tid & 7) == 0) sm.coarse[level][tid >> 3] = t;
            }
            if (C > 1) cluster.sync();
            else __syncthreads();
            if (warp == 0) {
                // from the top: the coarse bin that holds the want-th entry of the cluster, then the bin
                int hi_t = 0, lo_t = 0;
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < C) {
                        const int* p = cluster.map_shared_rank(&sm.coarse[level][0], c);
                        hi_t += p[63 - 2 * lane];
                        lo_t += p[62 - 2 * lane];
                    }
                int incl = warp_scan(hi_t + lo_t);
                int before = incl - hi_t - lo_t;
                int hit = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
                const bool second = before + hi_t < want;            // of the hitting lane's two
                const int cb = __shfl_sync(0xffffffffu, 63 - 2 * lane - (second ? 1 : 0), hit);
                const int above_c = __shfl_sync(0xffffffffu, before + (second ? hi_t : 0), hit);
                int t = 0;
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < C) t += cluster.map_shared_rank(&sm.hist[level][0], c)[32 * cb + 31 - lane];
                incl = above_c + warp_scan(t);
                hit = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
                if (lane == hit) {
                    sm.found_bin = 32 * cb + 31 - lane;
                    sm.found_above = incl - t;
                }
            }
            __syncthreads();
            const int found = sm.found_bin;
            want -= sm.found_above;
            // this CTA's entries above the bin
            int above = 0;
            if (tid < 64) above = tid > (found >> 5) ? sm.coarse[level][tid] : 0;
            else if (tid < 96) above = (tid & 31) > (found & 31) ? sm.hist[level][(found & ~31) + (tid & 31)] : 0;
            if (warp < 3) {
                above = warp_sum(above);
                if (lane == 0 && above) atomicAdd(&sm.local[0], above);
            }
            if (level == kLevels - 1 && tid == 0) sm.local[1] = sm.hist[level][found];
            prefix = (prefix << (level == 2 ? 10 : 11)) | (uint32_t)found;
            __syncthreads();
        }
    } else {
        // everything or nothing between the protected ends
        if (k > 0)
            for (int i = begin + tid; i < end; i += kSelThreads) {
                const float v = __ldg(m + i);
                nan |= v != v;
            }
        if (tid == 0) sm.local[0] = k > 0 ? end - begin : 0;
        __syncthreads();
    }
    if (__any_sync(0xffffffffu, nan) && lane == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
    const bool all = k == count;
    if (C > 1) cluster.sync();                             // local counts are complete everywhere
    int above_before = 0, ties_before = 0;
    for (int c = 0; c < rank; ++c) {
        const int* l = cluster.map_shared_rank(&sm.local[0], c);
        above_before += l[0];
        ties_before += l[1];
    }
    if (k > 0) {
        // ordered pass
#pragma unroll 1
        for (int t0 = begin; t0 < end; t0 += kTileElems) {
            const int w0 = t0 + warp * 32 * kPerLane;
            uint32_t gt[kPerLane], eq[kPerLane];
            int ngt = 0, neq = 0;
            if (!resident) load_tile(t0);
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                const int i = w0 + 32 * j + lane;
                const uint32_t key = mass_key(x[j]);
                gt[j] = __ballot_sync(0xffffffffu, i < end && (all || key > prefix));
                eq[j] = __ballot_sync(0xffffffffu, i < end && !all && key == prefix);
                ngt += __popc(gt[j]);
                neq += __popc(eq[j]);
            }
            __syncthreads();                               // the previous tile's totals are read
            if (lane == 0) {
                sm.warp_a[warp] = ngt;
                sm.warp_b[warp] = neq;
            }
            __syncthreads();
            const int ca = lane < kSelWarps ? sm.warp_a[lane] : 0, cb = lane < kSelWarps ? sm.warp_b[lane] : 0;
            int g = above_before + warp_sum(lane < warp ? ca : 0);
            int e = ties_before + warp_sum(lane < warp ? cb : 0);
            above_before += warp_sum(ca);
            ties_before += warp_sum(cb);
            const uint32_t below = (1u << lane) - 1u;
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                const int my_e = e + __popc(eq[j] & below);
                const bool is_gt = (gt[j] >> lane) & 1u;
                const bool is_eq = ((eq[j] >> lane) & 1u) && my_e < want;
                if (is_gt || is_eq) {
                    const int dst = s.sink + g + __popc(gt[j] & below) + min(my_e, want);
                    kept[dst] = w0 + 32 * j + lane;
                    if (mass_out) mass_out[dst] = x[j];
                }
                g += __popc(gt[j]);
                e += __popc(eq[j]);
            }
        }
    }
    if (C > 1) cluster.sync();                             // no CTA leaves while its counts are read
}

// Units of U bytes of the kept K (kv = 0) or V (kv = 1) records.
template <int FMT>
__device__ __forceinline__ size_t rec_at(const EvictArgs& a, int64_t page, int layer, int head, int kv, int row) {
    if (FMT == kFmtT5k) return t5k_offset(a.num_layers, a.num_kv_heads, page, layer, head, kv, row);
    return record_offset(a.num_layers, a.num_kv_heads, page, layer, head, kv, row,
                         FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes);
}

constexpr int kGatherThreads = 256;

// Copies n records of UNITS units each from the offsets off[] to consecutive records at dst.
template <typename U, int UNITS>
__device__ __forceinline__ void move_records(uint8_t* pool, const size_t* off, int n, uint8_t* dst) {
    constexpr int kU = sizeof(U) == 16 ? 7 : 8;              // loads of a thread in flight
    const int total = n * UNITS;
#pragma unroll 1
    for (int u0 = threadIdx.x; u0 < total; u0 += kGatherThreads * kU) {
        U v[kU];
        bool ok[kU];
#pragma unroll
        for (int r = 0; r < kU; ++r) {
            const int u = u0 + r * kGatherThreads;
            ok[r] = u < total;
            if (!ok[r]) continue;
            const int i = u / UNITS, part = u - i * UNITS;
            const size_t o = off[i];
            ok[r] = o != ~(size_t)0;
            if (ok[r]) v[r] = *reinterpret_cast<const U*>(pool + o + part * sizeof(U));
        }
#pragma unroll
        for (int r = 0; r < kU; ++r)
            if (ok[r]) *reinterpret_cast<U*>(dst + (size_t)(u0 + r * kGatherThreads) * sizeof(U)) = v[r];
    }
}

// CTA: kept records [256 x, 256 x + 256) of one (layer, slot, kv head) row: one destination page.
template <int FMT>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const EvictArgs a) {
    __shared__ size_t off[2][kPageSize];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t row = blockIdx.y + (int64_t)gridDim.y * blockIdx.z;
    if (row >= (int64_t)a.num_call_layers * a.num_slots * a.num_kv_heads) return;
    const int head = (int)(row % a.num_kv_heads);
    const int slot = (int)(row / a.num_kv_heads) % a.num_slots;
    const int layer = a.layer + (int)(row / a.num_kv_heads / a.num_slots);
    const SlotPlan s = slot_plan(a, slot);
    const int first = blockIdx.x * kPageSize;
    const int n = min(kPageSize, s.n - first);
    if (n <= 0) return;
    const int32_t dp = a.dst_table[(int64_t)slot * a.dst_max_pages + blockIdx.x];
    const bool dst_ok = dp >= 0 && dp < a.num_pages;
    bool bad = !dst_ok;
    if (threadIdx.x < n) {
        const int pos = a.kept[row * a.max_budget + first + threadIdx.x];
        const int32_t sp = a.page_table[(int64_t)slot * a.max_pages_per_slot + pos / kPageSize];
        const bool ok = sp >= 0 && sp < a.num_pages;
        bad |= !ok;
        off[0][threadIdx.x] = ok ? rec_at<FMT>(a, sp, layer, head, 0, pos % kPageSize) : ~(size_t)0;
        off[1][threadIdx.x] = ok ? rec_at<FMT>(a, sp, layer, head, 1, pos % kPageSize) : ~(size_t)0;
    }
    if (bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
    __syncthreads();
    if (!dst_ok) return;
    uint8_t* dk = a.pool + rec_at<FMT>(a, dp, layer, head, 0, 0);
    uint8_t* dv = a.pool + rec_at<FMT>(a, dp, layer, head, 1, 0);
    if (FMT == kFmtT5k) move_records<uint32_t, kT5kKRecordBytes / 4>(a.pool, off[0], n, dk);
    else move_records<uint4, (FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes) / 16>(a.pool, off[0], n, dk);
    move_records<uint4, (FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes) / 16>(a.pool, off[1], n, dv);
}

// New lengths, after every other kernel of the call has read ctx_len (which may
// be the same array).
__global__ void __launch_bounds__(256) length_kernel(const EvictArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int b = blockIdx.x * 256 + threadIdx.x; b < a.num_slots; b += gridDim.x * 256) {
        const SlotPlan s = slot_plan(a, b);
        a.new_len[b] = s.n > 0 ? s.n : s.L;
    }
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, int cluster, const EvictArgs& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int FMT>
cudaError_t launch_gather(const EvictArgs& a, cudaStream_t stream) {
    const int64_t rows = (int64_t)a.num_call_layers * a.num_slots * a.num_kv_heads;
    const int64_t most = std::min<int64_t>(a.max_budget, a.max_ctx_len);
    const int64_t gy = std::min<int64_t>(rows, 32768), gz = (rows + gy - 1) / gy;
    return launch_pdl(gather_kernel<FMT>, dim3((unsigned)((most + kPageSize - 1) / kPageSize), (unsigned)gy, (unsigned)gz),
                      kGatherThreads, 0, a, stream);
}

int evict_impl(int fmt, void* stream, const q3kv_cache_desc* desc, void* d_pool, const int32_t* d_page_table,
               int32_t max_pages_per_slot, const int32_t* d_ctx_len, int32_t num_slots, int64_t max_ctx_len,
               const int32_t* d_budget, int32_t max_budget, int32_t n_sink, int32_t n_recent, int32_t layer,
               int32_t num_call_layers, const float* d_mass, int64_t mass_stride, const int32_t* d_dst_page_table,
               int32_t dst_max_pages, int32_t* d_kept, float* d_mass_out, int32_t* d_new_len, int32_t* d_status) {
    int e = check_desc(desc);
    if (e != Q3KV_OK) return e;
    if (num_slots < 0 || max_pages_per_slot <= 0 || dst_max_pages <= 0 || max_ctx_len < 0 || max_budget < 0 ||
        n_sink < 0 || n_recent < 0 || layer < 0 || num_call_layers < 0 || mass_stride < max_ctx_len)
        return Q3KV_ERR_INVALID_ARG;
    if (layer > desc->num_layers || num_call_layers > desc->num_layers - layer) return Q3KV_ERR_INVALID_ARG;
    if (max_ctx_len > (int64_t)INT32_MAX - kPageSize) return Q3KV_ERR_INVALID_ARG;
    if (num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (num_slots == 0) return Q3KV_OK;
    if (!d_ctx_len || !d_budget || !d_new_len) return Q3KV_ERR_INVALID_ARG;
    const bool work = num_call_layers > 0 && max_budget > 0 && max_ctx_len > 0;
    if (work && (!d_pool || !d_page_table || !d_dst_page_table || !d_mass || !d_kept || !aligned16(d_pool)))
        return Q3KV_ERR_INVALID_ARG;
    int sms = 0;
    e = device_sm_count(&sms);
    if (e != Q3KV_OK) return e;
    EvictArgs a{};
    a.pool = static_cast<uint8_t*>(d_pool);
    a.page_table = d_page_table;
    a.max_pages_per_slot = max_pages_per_slot;
    a.ctx_len = d_ctx_len;
    a.num_slots = num_slots;
    a.max_ctx_len = max_ctx_len;
    a.budget = d_budget;
    a.max_budget = max_budget;
    a.n_sink = n_sink;
    a.n_recent = n_recent;
    a.layer = layer;
    a.num_call_layers = num_call_layers;
    a.mass = d_mass;
    a.mass_stride = mass_stride;
    a.dst_table = d_dst_page_table;
    a.dst_max_pages = dst_max_pages;
    a.kept = d_kept;
    a.mass_out = d_mass_out;
    a.new_len = d_new_len;
    a.status = d_status;
    a.num_layers = desc->num_layers;
    a.num_kv_heads = desc->num_kv_heads;
    a.num_pages = desc->num_pages;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t rows = (int64_t)num_call_layers * num_slots * desc->num_kv_heads;
    if (rows * kMaxCluster > INT32_MAX) return Q3KV_ERR_UNSUPPORTED;
    if (work) {
        // cluster size: segments of one tile (registers) where eight CTAs reach that, and no
        // more CTAs than run at once (two per SM)
        int c = kMaxCluster;
        while (c > 1 && (rows * c > 2 * (int64_t)sms || (int64_t)(c / 2) * kTileElems >= max_ctx_len)) c >>= 1;
        cudaError_t ce = launch_pdl(select_kernel, dim3((unsigned)(rows * c)), kSelThreads, c, a, st);
        if (ce != cudaSuccess) return cuda_status(ce);
        ce = fmt == kFmtFp8 ? launch_gather<kFmtFp8>(a, st)
                            : (fmt == kFmtT5k ? launch_gather<kFmtT5k>(a, st) : launch_gather<kFmtQ3>(a, st));
        if (ce != cudaSuccess) return cuda_status(ce);
    }
    if (work && d_new_len != d_ctx_len) return Q3KV_OK;      // the select kernel wrote the lengths
    return cuda_status(launch_pdl(length_kernel, dim3((unsigned)std::min(64, (num_slots + 255) / 256)), 256, 0, a, st));
}

}  // namespace
}  // namespace q3kv

using namespace q3kv;

extern "C" {

#define Q3KV_EVICT_ENTRY(NAME, FMT)                                                                                  \
    int NAME(void* stream, const q3kv_cache_desc* desc, void* d_pool, const int32_t* d_page_table,                   \
             int32_t max_pages_per_slot, const int32_t* d_ctx_len, int32_t num_slots, int64_t max_ctx_len,            \
             const int32_t* d_budget, int32_t max_budget, int32_t n_sink, int32_t n_recent, int32_t layer,            \
             int32_t num_call_layers, const float* d_mass, int64_t mass_stride, const int32_t* d_dst_page_table,      \
             int32_t dst_max_pages_per_slot, int32_t* d_kept, float* d_mass_out, int32_t* d_new_len,                  \
             int32_t* d_status) {                                                                                     \
        return evict_impl(FMT, stream, desc, d_pool, d_page_table, max_pages_per_slot, d_ctx_len, num_slots,          \
                          max_ctx_len, d_budget, max_budget, n_sink, n_recent, layer, num_call_layers, d_mass,        \
                          mass_stride, d_dst_page_table, dst_max_pages_per_slot, d_kept, d_mass_out, d_new_len,       \
                          d_status);                                                                                  \
    }

Q3KV_EVICT_ENTRY(q3kv_evict, kFmtQ3)
Q3KV_EVICT_ENTRY(q3kv_fp8_evict, kFmtFp8)
Q3KV_EVICT_ENTRY(q3kv_t5k_evict, kFmtT5k)

}  // extern "C"
