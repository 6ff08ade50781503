// Copies of whole pages or of their first positions, in all layers: what the first write of a
// forked slot and a compaction of the pool ask for.
//
// A page's bytes are contiguous (pages are the outermost dimension of every pool), so a whole page
// is a straight copy; the first r positions are, per (layer, kv head, K|V) unit, the first bytes of
// its records (3-bit, fp8, turbo5k) or, in the block-scaled cache, the rows below r of its
// 8-row x 16-byte cores and the scales of the blocks that begin below r.
//
// Bound: the copied bytes, once read and once written.  One CTA moves 32 KiB of one page with eight
// 16-byte loads in flight per thread; it reads the list of pairs while its loads are under way to
// see that no other pair reads or writes its destination, so neither an extra launch nor a workspace
// is needed for that check.
#include "q3kv_internal.h"

namespace q3kv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;                                        // 16-byte loads in flight per thread
constexpr uint32_t kCopyBytes = kCopyThreads * kCopyVecs * 16;      // of one page, per CTA
constexpr int kMaxPairs = 4096;                                     // every CTA reads the list

struct CopyArgs {
    const uint8_t* src_pool;
    uint8_t* dst_pool;
    int32_t same_pool;
    int32_t src_pages, dst_pages;
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;         // positions of each page to copy, or null: all
    int32_t n;
    uint32_t page_bytes;
    int32_t* status;
};

// Bytes of the 16 at offset `off` of a page that belong to its first `rows` positions (a multiple of 4).
template <int FMT>
__device__ __forceinline__ int kept_bytes(uint32_t off, int rows) {
    if (FMT == kFmtBs8) {
        const uint32_t o = off % kBs8UnitBytes;
        if (o < kBs8CodeBytes) return (int)(o >> 11) * 8 + (int)((o >> 4) & 7) < rows ? 16 : 0;
        return min(16, max(0, 4 * ((rows + kBs8Block - 1) / kBs8Block) - (int)(o - kBs8CodeBytes)));
    }
    if (FMT == kFmtT5k) {
        const uint32_t o = off % (uint32_t)kT5kChunkBytes;
        constexpr uint32_t k = kPageSize * kT5kKRecordBytes;
        return o < k ? min(16, max(0, rows * kT5kKRecordBytes - (int)o)) : min(16, max(0, rows * kRecordBytes - (int)(o - k)));
    }
    constexpr int rec = FMT == kFmtFp8 ? kFp8RecordBytes : kRecordBytes;
    return min(16, max(0, rows * rec - (int)(off % (uint32_t)(kPageSize * rec))));
}

template <int FMT, bool PART>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(CopyArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int i = blockIdx.y;
    const int src = a.src[i], dst = a.dst[i];
    const bool first = blockIdx.x == 0 && threadIdx.x == 0;
    if (src < 0 || src >= a.src_pages || dst < 0 || dst >= a.dst_pages) {
        if (first && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
        return;
    }
    const int rows = PART ? a.rows[i] : kPageSize;
    if (PART && (rows < 0 || rows > kPageSize)) {
        if (first && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_LENGTH);
        return;
    }
    if (a.same_pool && src == dst) return;          // nothing moves
    const uint32_t base = blockIdx.x * kCopyBytes + threadIdx.x * 16;
    const uint8_t* from = a.src_pool + (size_t)src * a.page_bytes;
    uint8_t* to = a.dst_pool + (size_t)dst * a.page_bytes;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
        const uint32_t off = base + j * (kCopyThreads * 16);
        if (off < a.page_bytes && (!PART || kept_bytes<FMT>(off, rows) > 0)) v[j] = __ldcs(reinterpret_cast<const uint4*>(from + off));
    }
    // a destination that another pair reads or writes would make the result depend on the order
    bool clash = false;
    for (int j = threadIdx.x; j < a.n; j += kCopyThreads) clash |= j != i && (a.dst[j] == dst || (a.same_pool && a.src[j] == dst));
    if (__syncthreads_or(clash)) {
        if (first && a.status) atomicOr(a.status, Q3KV_STATUS_BAD_PAGE);
        return;
    }
#pragma unroll
    for (int j = 0; j < kCopyVecs; ++j) {
        const uint32_t off = base + j * (kCopyThreads * 16);
        if (off >= a.page_bytes) continue;
        const int bytes = PART ? kept_bytes<FMT>(off, rows) : 16;
        if (bytes == 16) {
            *reinterpret_cast<uint4*>(to + off) = v[j];
        } else if (PART && bytes > 0) {              // the last record of a unit may end inside the 16 bytes
            const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (4 * k < bytes) *reinterpret_cast<uint32_t*>(to + off + 4 * k) = w[k];
        }
    }
}

template <int FMT>
cudaError_t launch_copy(const CopyArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.page_bytes + kCopyBytes - 1) / kCopyBytes, (unsigned)a.n);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.rows ? cudaLaunchKernelEx(&cfg, copy_pages_kernel<FMT, true>, a) : cudaLaunchKernelEx(&cfg, copy_pages_kernel<FMT, false>, a);
}

int copy_impl(int fmt, void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool, int32_t dst_num_pages,
              const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows, int32_t n, int32_t* d_status) {
    int e = check_desc(desc);
    if (e != Q3KV_OK) return e;
    if (n < 0 || dst_num_pages <= 0) return Q3KV_ERR_INVALID_ARG;
    if (n > kMaxPairs) return Q3KV_ERR_UNSUPPORTED;
    const size_t unit = fmt == kFmtBs8 ? 2 * (size_t)kBs8UnitBytes : fmt == kFmtT5k ? kT5kChunkBytes
                        : 2 * (size_t)kPageSize * (fmt == kFmtFp8 ? kFp8RecordBytes : kRecordBytes);
    const size_t page = unit * desc->num_layers * desc->num_kv_heads;
    if (page > (size_t)INT32_MAX - kCopyBytes) return Q3KV_ERR_UNSUPPORTED;      // offsets within a page are 32 bits
    if (n == 0) return Q3KV_OK;
    if (!d_src_pool || !d_dst_pool || !d_src || !d_dst) return Q3KV_ERR_INVALID_ARG;
    if (!aligned16(d_src_pool) || !aligned16(d_dst_pool)) return Q3KV_ERR_INVALID_ARG;
    const int64_t src_bytes = (int64_t)(page * desc->num_pages), dst_bytes = (int64_t)(page * dst_num_pages);
    if (d_src_pool == d_dst_pool ? dst_num_pages != desc->num_pages : overlap(d_src_pool, src_bytes, d_dst_pool, dst_bytes))
        return Q3KV_ERR_INVALID_ARG;
    const int64_t list = 4 * (int64_t)n;
    if (overlap(d_dst_pool, dst_bytes, d_src, list) || overlap(d_dst_pool, dst_bytes, d_dst, list) ||
        (d_rows && overlap(d_dst_pool, dst_bytes, d_rows, list)) || (d_status && overlap(d_dst_pool, dst_bytes, d_status, 4)))
        return Q3KV_ERR_INVALID_ARG;
    CopyArgs a{};
    a.src_pool = static_cast<const uint8_t*>(d_src_pool);
    a.dst_pool = static_cast<uint8_t*>(d_dst_pool);
    a.same_pool = d_src_pool == d_dst_pool;
    a.src_pages = desc->num_pages;
    a.dst_pages = dst_num_pages;
    a.src = d_src;
    a.dst = d_dst;
    a.rows = d_rows;
    a.n = n;
    a.page_bytes = (uint32_t)page;
    a.status = d_status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (fmt) {
        case kFmtQ3: return cuda_status(launch_copy<kFmtQ3>(a, st));
        case kFmtFp8: return cuda_status(launch_copy<kFmtFp8>(a, st));
        case kFmtT5k: return cuda_status(launch_copy<kFmtT5k>(a, st));
        default: return cuda_status(launch_copy<kFmtBs8>(a, st));
    }
}

}  // namespace
}  // namespace q3kv

extern "C" {

int q3kv_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool, int32_t dst_num_pages,
                    const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows, int32_t n, int32_t* d_status) {
    return q3kv::copy_impl(q3kv::kFmtQ3, stream, desc, d_src_pool, d_dst_pool, dst_num_pages, d_src, d_dst, d_rows, n, d_status);
}
int q3kv_fp8_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool, int32_t dst_num_pages,
                        const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows, int32_t n, int32_t* d_status) {
    return q3kv::copy_impl(q3kv::kFmtFp8, stream, desc, d_src_pool, d_dst_pool, dst_num_pages, d_src, d_dst, d_rows, n, d_status);
}
int q3kv_t5k_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool, int32_t dst_num_pages,
                        const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows, int32_t n, int32_t* d_status) {
    return q3kv::copy_impl(q3kv::kFmtT5k, stream, desc, d_src_pool, d_dst_pool, dst_num_pages, d_src, d_dst, d_rows, n, d_status);
}
int q3kv_bs8_copy_pages(void* stream, const q3kv_cache_desc* desc, const void* d_src_pool, void* d_dst_pool, int32_t dst_num_pages,
                        const int32_t* d_src, const int32_t* d_dst, const int32_t* d_rows, int32_t n, int32_t* d_status) {
    return q3kv::copy_impl(q3kv::kFmtBs8, stream, desc, d_src_pool, d_dst_pool, dst_num_pages, d_src, d_dst, d_rows, n, d_status);
}

}  // extern "C"
