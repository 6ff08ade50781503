// Eviction by attention mass: choose the positions to keep, compact their records.
//
// select_kernel, one thread-block cluster per (layer, slot, kv head) row: a radix
// select over the masses' order keys finds the k-th largest (k = budget minus the
// protected positions) exactly, 11 + 11 + 10 bits.  A warp has a consecutive share of
// the row: the first pass (HBM) counts the leading 11 bits in shared memory; the second
// (L2) counts what lies above the found bin and puts the bin's own masses, compared as
// floats, into the warp's list, from which the other two levels count; the last (L2)
// writes positions and masses at their final ranks, with no barrier inside, as the
// warps before it have known counts above the threshold and at it, of which the lowest
// positions are taken.  A list that overflows (more than 512 masses of a warp in one bin)
// is replaced by reading the share again.  A share of at most 256 masses stays in
// registers.  No float is added, so nothing depends on an order.
//
// A level's bin: 64 coarse counts go to every CTA of the cluster (distributed shared
// memory), then one warp finds the coarse bin that holds the k-th and reads its 32 bins
// from every CTA; reading all bins of all CTAs took longer than counting.
//
// 1,024 threads of an SM, in two CTAs or one, with at most 64 registers each.  The lists are
// short because the L1 lines that loads in flight need come out of the same 256 KB: with
// lists of 1,024 masses 32 rows of 655,360 took 60 us more.
//
// gather_kernel: a CTA moves up to 256 kept records, one destination page, of K and V:
// their source offsets go to shared memory first, so all 16-byte loads (4-byte ones
// for the 164-byte K records) of a thread are independent, and the stores, to
// consecutive records, coalesce.
//
// Bound: memory.  32 rows of 655,360 masses, 65,536 kept, take 239 us: select 63 us (84 MB
// from HBM once and from L2 twice; about a third each for the first pass, the second with
// the levels, and the last), gather 176 us (470 MB of records read and written; a
// scattered 112-byte record touches 64-byte DRAM bursts worth half as much again, with
// which the traffic alone takes 173 us).  2 rows of 5,000: 12.9 us, where each of the three
// levels costs a cluster barrier and a trip to the other CTAs, 1.5 us.
#include <cooperative_groups.h>
#include <math_constants.h>

#include <algorithm>
#include <atomic>

#include "q3kv_internal.h"

namespace cg = cooperative_groups;

namespace q3kv {
namespace {

constexpr int kPerLane = 8;                               // masses of a lane per tile
constexpr int kTile = 32 * kPerLane;                      // a warp's
constexpr int kBins = 2048;
constexpr int kCoarse = kBins / 32;
constexpr int kLevels = 3;
constexpr int kMaxCluster = 16;
constexpr int kListCap = 512;
constexpr uint32_t kKeyInf = 0xff800000u, kKeyMinusInf = 0x007fffffu;   // order keys of the infinities
static_assert(kBins == 4 * 512 && kMaxCluster <= 32, "find_bin");

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
    int32_t late_len;            // new_len is ctx_len or budget: length_kernel writes it
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

// The float with an order key (of a number that is not NaN).
__device__ __forceinline__ float key_float(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
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

template <int kWarps>
struct __align__(16) SelectSmem {
    int hist[kLevels][kBins];                  // this CTA's counts
    int coarse[2][kMaxCluster][kCoarse];       // every CTA's counts of 32 bins each, by level % 2
    int2 total[kMaxCluster];                   // every CTA's entries above the threshold, and at it
    int2 warp[kWarps];                      // the same of this CTA's warps
    int found_bin;
    int found_above;                           // entries in bins above it
    float list[kWarps][kListCap];           // a warp's masses in the first level's bin
};

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads) select_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kSelWarps = kSelThreads / 32;
    SelectSmem<kSelWarps>& sm = *reinterpret_cast<SelectSmem<kSelWarps>*>(smem_raw);
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks();
    const int rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t below = (1u << lane) - 1u;
    const int64_t row = blockIdx.x / C;                    // (layer, slot, kv head)
    const int slot = (int)(row / a.num_kv_heads) % a.num_slots;
    const SlotPlan s = slot_plan(a, slot);
    if (rank == 0 && tid == 0 && row % a.num_kv_heads == 0 && row / a.num_kv_heads < a.num_slots) {   // one per slot
        if (s.bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        // where new_len is an array the plans read, length_kernel writes it when every kernel has read it
        if (!a.late_len) a.new_len[slot] = s.n > 0 ? s.n : s.L;
    }
    if (s.n == 0) return;                                  // the whole cluster agrees

    const float* m = a.mass + row * a.mass_stride;
    int32_t* kept = a.kept + row * a.max_budget;
    float* mass_out = a.mass_out ? a.mass_out + row * a.max_budget : nullptr;
    const int lo = s.sink, hi = s.L - s.recent;            // free positions [lo, hi)
    const int k = s.n - s.sink - s.recent;                 // of which k are kept
    bool nan = false;                                      // anywhere in the row
    // protected positions keep their order at both ends
    for (int i = rank * kSelThreads + tid; i < s.sink + s.recent; i += C * kSelThreads) {
        const int pos = i < s.sink ? i : s.L - s.recent + (i - s.sink);
        const int dst = i < s.sink ? i : s.n - s.recent + (i - s.sink);
        const float v = m[pos];
        nan |= v != v;
        kept[dst] = pos;
        if (mass_out) mass_out[dst] = v;
    }
    if (k == 0) {                                          // nothing to choose
        for (int i = lo + rank * kSelThreads + tid; i < hi; i += C * kSelThreads) nan |= m[i] != m[i];
        if (__any_sync(0xffffffffu, nan) && lane == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
        return;
    }
    if (C > 1) cluster.barrier_arrive();                   // waited for before the first access to another CTA
    // a warp's share of the free positions, consecutive in the order (CTA, warp)
    const int count = hi - lo;
    const int parts = C * kSelWarps;
    const int seg = ((count + parts - 1) / parts + 31) / 32 * 32;
    const int begin = min(hi, lo + (rank * kSelWarps + warp) * seg), end = min(hi, begin + seg);
    const bool resident = seg <= kTile;                    // one tile: loaded once
    const float kNan = __int_as_float(0x7fffffff);

    // A tile: kTile consecutive positions of a warp, 32 at a time; NaN behind the end.
    auto load = [&](float (&x)[kPerLane], int t0) {
        const float* p = m + t0 + lane;
        if (t0 + kTile <= end) {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) x[j] = p[32 * j];
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) x[j] = t0 + 32 * j + lane < end ? p[32 * j] : kNan;
        }
    };
    float x[kPerLane];
    // f(first position) over the warp's tiles in x, the next tile's loads in flight
    auto tiles = [&](auto&& f) {
        if (resident) {
            if (begin < end) f(begin);
            return;
        }
        float y[kPerLane];
        if (begin < end) load(x, begin);
#pragma unroll 1
        for (int t0 = begin; t0 < end; t0 += kTile) {
            if (t0 + kTile < end) load(y, t0 + kTile);
            f(t0);
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) x[j] = y[j];
        }
    };
    if (resident) load(x, begin);

    int want = k;                                          // entries still to take at or below the prefix's range
    uint32_t prefix = 0u;                                  // key bits found so far
    // Finds the bin of hist[level] that holds the cluster's want-th entry from the top.
    auto find_bin = [&](int level) {
        __syncthreads();
        if (tid < kBins / 4) {   // thread t adds bins 4 t .. 4 t + 3, eight threads a coarse bin, given to every CTA
            const int4 u = reinterpret_cast<const int4*>(&sm.hist[level][0])[tid];
            int t = (u.x + u.y) + (u.z + u.w);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (C == 1) sm.coarse[level & 1][0][tid >> 3] = t;
            else
                for (int c = tid & 7; c < C; c += 8) *cluster.map_shared_rank(&sm.coarse[level & 1][rank][tid >> 3], c) = t;
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        if (warp == 0) {
            // the coarse bin that holds the want-th entry, then the bin
            int2 t2 = make_int2(0, 0);                     // bins 62 - 2 lane, 63 - 2 lane
            for (int c = 0; c < C; ++c) {
                const int2 u = *reinterpret_cast<const int2*>(&sm.coarse[level & 1][c][62 - 2 * lane]);
                t2.x += u.x;
                t2.y += u.y;
            }
            int incl = warp_scan(t2.x + t2.y);
            const int before = incl - t2.x - t2.y;
            int hit = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
            const bool second = before + t2.y < want;      // of the hitting lane's two
            const int cb = __shfl_sync(0xffffffffu, 63 - 2 * lane - (second ? 1 : 0), hit);
            const int above_c = __shfl_sync(0xffffffffu, before + (second ? t2.y : 0), hit);
            int t = C == 1 ? sm.hist[level][32 * cb + 31 - lane] : 0;
#pragma unroll 1
            for (int c0 = 0; C > 1 && c0 < C; c0 += 8)     // eight remote loads in flight
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (c0 + c < C) t += cluster.map_shared_rank(&sm.hist[level][0], c0 + c)[32 * cb + 31 - lane];
            incl = above_c + warp_scan(t);
            hit = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
            if (lane == hit) {
                sm.found_bin = 32 * cb + 31 - lane;
                sm.found_above = incl - t;
            }
        }
        __syncthreads();
        want -= sm.found_above;
        return (uint32_t)sm.found_bin;
    };

    const bool all = k == count;                           // everything between the protected ends
    bool nan_thr = false;                                  // the k-th is a NaN
    float thr = 0.0f;
    int n_gt = 0, n_eq = 0;                                // the warp's entries above the threshold, and at it
    if (all) {
        tiles([&](int t0) {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) nan |= x[j] != x[j] && t0 + 32 * j + lane < end;
        });
        n_gt = end - begin;
        if (C > 1) cluster.barrier_wait();
    } else {
        for (int i = tid; i < kLevels * kBins / 4; i += kSelThreads)
            reinterpret_cast<int4*>(&sm.hist[0][0])[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
        tiles([&](int t0) {
            if (t0 + kTile <= end) {
#pragma unroll
                for (int j = 0; j < kPerLane; ++j) {
                    nan |= x[j] != x[j];
                    atomicAdd(&sm.hist[0][mass_key(x[j]) >> 21], 1);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPerLane; ++j)
                    if (t0 + 32 * j + lane < end) {
                        nan |= x[j] != x[j];
                        atomicAdd(&sm.hist[0][mass_key(x[j]) >> 21], 1);
                    }
            }
        });
        if (C > 1) cluster.barrier_wait();
        prefix = find_bin(0);
        nan_thr = prefix == 0u;                            // NaN is alone in bin 0: every number is taken
        if (!nan_thr) {
            // the bin's numbers are those of [f_lo, f_hi]; -0 belongs to +0's
            const float f_lo = key_float(max(prefix << 21, kKeyMinusInf));
            uint32_t key_hi = min(prefix << 21 | 0x1fffffu, kKeyInf);
            key_hi -= key_hi == 0x7fffffffu;
            const float f_hi = key_float(key_hi);
            int n = 0, above = 0;
            if (!resident) {
                float* list = sm.list[warp];
                tiles([&](int) {
#pragma unroll
                    for (int j = 0; j < kPerLane; ++j) {
                        above += x[j] > f_hi;
                        const bool in = x[j] >= f_lo && x[j] <= f_hi;
                        const uint32_t who = __ballot_sync(0xffffffffu, in);
                        const int at = n + __popc(who & below);
                        if (in && at < kListCap) list[at] = x[j];
                        n += __popc(who);
                    }
                });
                __syncwarp();
            }
            const bool listed = !resident && n <= kListCap;
#pragma unroll 1
            for (int level = 1; level < kLevels; ++level) {
                const int shift = level == 1 ? 10 : 0, bits = level == 1 ? 11 : 10;
                auto count_key = [&](float v) {
                    const uint32_t key = mass_key(v);
                    if (key >> shift >> bits == prefix) atomicAdd(&sm.hist[level][key >> shift & ((1u << bits) - 1u)], 1);
                };
                if (listed) {
                    for (int i = lane; i < n; i += 32) count_key(sm.list[warp][i]);
                } else {
                    tiles([&](int) {                       // NaN (behind the end too) is in no bin but 0
#pragma unroll
                        for (int j = 0; j < kPerLane; ++j) count_key(x[j]);
                    });
                }
                prefix = prefix << bits | find_bin(level);
            }
            thr = key_float(prefix);
            if (listed) {
                for (int i = lane; i < n; i += 32) {
                    const float v = sm.list[warp][i];
                    above += v > thr;
                    n_eq += v == thr;
                }
                n_gt = warp_sum(above);
                n_eq = warp_sum(n_eq);
            }
            if (!listed) {
                above = 0;
                tiles([&](int) {
#pragma unroll
                    for (int j = 0; j < kPerLane; ++j) {
                        above += x[j] > thr;
                        n_eq += x[j] == thr;
                    }
                });
                n_gt = warp_sum(above);
                n_eq = warp_sum(n_eq);
            }
        } else {
            tiles([&](int) {
#pragma unroll
                for (int j = 0; j < kPerLane; ++j) n_gt += x[j] == x[j];
            });
            n_gt = warp_sum(n_gt);
            n_eq = end - begin - n_gt;
        }
    }
    if (__any_sync(0xffffffffu, nan) && lane == 0 && a.status) atomicOr(a.status, Q3KV_STATUS_NONFINITE_INPUT);
    // the entries taken before this warp's
    if (lane == 0) sm.warp[warp] = make_int2(n_gt, n_eq);
    __syncthreads();
    if (warp == 0) {
        const int2 u = lane < kSelWarps ? sm.warp[lane] : make_int2(0, 0);
        const int2 t = make_int2(warp_sum(u.x), warp_sum(u.y));
        if (C == 1) sm.total[0] = t;
        else if (lane < C) *cluster.map_shared_rank(&sm.total[rank], lane) = t;
    }
    if (C > 1) cluster.sync();                             // the last remote access is done: a CTA may leave
    else __syncthreads();
    int2 u = lane < warp ? sm.warp[lane] : make_int2(0, 0);
    if (lane < rank) {
        u.x += sm.total[lane].x;
        u.y += sm.total[lane].y;
    }
    int ties = warp_sum(u.y);
    int at = s.sink + warp_sum(u.x) + min(ties, want);     // where the next taken entry goes
    tiles([&](int t0) {
        bool tie = false;
        uint32_t take[kPerLane];
        if (all || nan_thr) {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                const bool in = t0 + 32 * j + lane < end;
                take[j] = __ballot_sync(0xffffffffu, all ? in : x[j] == x[j]);
                tie |= nan_thr && in && x[j] != x[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                take[j] = __ballot_sync(0xffffffffu, x[j] > thr);
                tie |= x[j] == thr;
            }
        }
        if (__any_sync(0xffffffffu, tie)) {                // the first ones at the threshold
#pragma unroll
            for (int j = 0; j < kPerLane; ++j) {
                const bool eq = nan_thr ? x[j] != x[j] && t0 + 32 * j + lane < end : x[j] == thr;
                const uint32_t who = __ballot_sync(0xffffffffu, eq);
                take[j] |= __ballot_sync(0xffffffffu, eq && ties + __popc(who & below) < want);
                ties += __popc(who);
            }
        }
#pragma unroll
        for (int j = 0; j < kPerLane; ++j) {
            if (take[j] >> lane & 1u) {
                const int dst = at + __popc(take[j] & below);
                kept[dst] = t0 + 32 * j + lane;
                if (mass_out) mass_out[dst] = x[j];
            }
            at += __popc(take[j]);
        }
    });
}

// Units of U bytes of the kept K (kv = 0) or V (kv = 1) records.
template <int FMT>
__device__ __forceinline__ size_t rec_at(const EvictArgs& a, int64_t page, int layer, int head, int kv, int row) {
    if (FMT == kFmtT5k) return t5k_offset(a.num_layers, a.num_kv_heads, page, layer, head, kv, row);
    return record_offset(a.num_layers, a.num_kv_heads, page, layer, head, kv, row,
                         FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes);
}

constexpr int kGatherThreads = 256;

// A load for which L2 fetches 64 bytes from memory; a plain one fetches the 128-byte line, of
// which a scattered record leaves half (16 layers x 655,360: gather 198 -> 176 us).
__device__ __forceinline__ void load_64b(const void* p, uint4& v) {
    asm volatile("ld.global.L2::64B.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
}
__device__ __forceinline__ void load_64b(const void* p, uint32_t& v) {
    asm volatile("ld.global.L2::64B.u32 %0, [%1];" : "=r"(v) : "l"(p));
}

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
            if (ok[r]) load_64b(pool + o + part * sizeof(U), v[r]);
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

// New lengths, after every other kernel of the call has read ctx_len and budget (which may
// be the same array).
__global__ void __launch_bounds__(256) length_kernel(const EvictArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int b = blockIdx.x * 256 + threadIdx.x; b < a.num_slots; b += gridDim.x * 256) {
        const SlotPlan s = slot_plan(a, b);
        a.new_len[b] = s.n > 0 ? s.n : s.L;
        if (s.bad && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);   // also of a call without rows
    }
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, int cluster, const EvictArgs& a, cudaStream_t stream, size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = smem;
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

template <int kSelThreads>
cudaError_t launch_select(const EvictArgs& a, unsigned rows, int cluster, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> attr_set[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    constexpr size_t smem = sizeof(SelectSmem<kSelThreads / 32>);
    if (!attr_set[dev].load(std::memory_order_acquire)) {
        cudaError_t e = cudaFuncSetAttribute(select_kernel<kSelThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(select_kernel<kSelThreads>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        attr_set[dev].store(true, std::memory_order_release);
    }
    return launch_pdl(select_kernel<kSelThreads>, dim3(rows * (unsigned)cluster), kSelThreads, cluster, a, stream, smem);
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
    if (max_ctx_len > (int64_t)INT32_MAX - 65536) return Q3KV_ERR_INVALID_ARG;   // positions behind a tile's end are ints
    if (num_slots > 65535) return Q3KV_ERR_UNSUPPORTED;
    if (num_slots == 0) return Q3KV_OK;
    if (!d_ctx_len || !d_budget || !d_new_len) return Q3KV_ERR_INVALID_ARG;
    const bool work = num_call_layers > 0 && max_budget > 0 && max_ctx_len > 0;
    if (work && (!d_pool || !d_page_table || !d_dst_page_table || !d_mass || !d_kept || !aligned16(d_pool)))
        return Q3KV_ERR_INVALID_ARG;
    // a row's CTAs write kept and mass_out while others read its masses; the plans are read until the end
    const int64_t pairs = (int64_t)num_slots * desc->num_kv_heads;
    if (num_call_layers > 0 && pairs > INT32_MAX / kMaxCluster / num_call_layers) return Q3KV_ERR_UNSUPPORTED;
    const int64_t rows = num_call_layers * pairs;
    const int64_t read = rows * std::min<int64_t>(mass_stride, (int64_t)1 << 33) * 4, written = rows * max_budget * 4, lens = (int64_t)num_slots * 4;
    if (work && (overlap(d_kept, written, d_mass, read) || overlap(d_mass_out, d_mass_out ? written : 0, d_mass, read) ||
                 overlap(d_mass_out, d_mass_out ? written : 0, d_kept, written)))
        return Q3KV_ERR_INVALID_ARG;
    if ((d_new_len != d_ctx_len && overlap(d_new_len, lens, d_ctx_len, lens)) || (d_new_len != d_budget && overlap(d_new_len, lens, d_budget, lens)))
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
    a.late_len = d_new_len == d_ctx_len || d_new_len == d_budget;
    a.status = d_status;
    a.num_layers = desc->num_layers;
    a.num_kv_heads = desc->num_kv_heads;
    a.num_pages = desc->num_pages;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (work) {
        // cluster size: up to 16 CTAs a row while each has an SM of its own (2 rows of 655,360: 71 -> 50 us a call,
        // 8 rows 109 -> 94), else up to 8 of two per SM (16 rows: 165 us, with 16 CTAs 172); half while half keeps a
        // row in registers
        int c = kMaxCluster;
        while (c > 1 && (rows * c > (c > 8 ? 1 : 2) * (int64_t)sms || (int64_t)(c / 2) * 512 * kPerLane >= max_ctx_len)) c >>= 1;
        // where two would share an SM, one of 1,024 threads: a barrier and a remote trip have half the partners (32
        // rows of 32,768: 44.3 -> 41.4 us a call, of 655,360 266 -> 261; 2 rows of 5,000, which one CTA
        // then holds, 13.4 -> 12.9; with an SM each, 16 x 1,024 threads a row are
        // slower than 16 x 512: 8 rows 109 us for 91)
        cudaError_t ce = c > 1 && (rows * c > sms || max_ctx_len <= 1024 * kPerLane) ? launch_select<1024>(a, (unsigned)rows, c / 2, st)
                                                 : launch_select<512>(a, (unsigned)rows, c, st);
        if (ce != cudaSuccess) return cuda_status(ce);
        ce = fmt == kFmtFp8 ? launch_gather<kFmtFp8>(a, st)
                            : (fmt == kFmtT5k ? launch_gather<kFmtT5k>(a, st) : launch_gather<kFmtQ3>(a, st));
        if (ce != cudaSuccess) return cuda_status(ce);
    }
    if (work && !a.late_len) return Q3KV_OK;      // the select kernel wrote the lengths
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
