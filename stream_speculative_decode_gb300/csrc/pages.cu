// Copies between pages of paged pools: the first keys of page src[i] to page
// dst[i] in every pool (a layer's K or V) at once. A fork copies its parent's
// partly filled last page before it appends (copy-on-write); a compaction moves
// whole pages.
//
// The lists come from the host and travel as kernel arguments, so the call
// needs no device scratch, no copy and no wait, and a captured graph holds
// them. Source and destination pages are checked to be apart, so the copies
// are independent and their order does not matter.
//
// HBM bound: 1,024 bytes (8 heads x 128) a key, read and written. One CTA a
// (copy, pool); a whole page is one contiguous run, a part of it 8 runs of
// keys x 128 bytes. Measured: 1,000 whole 64-key pages in 8 pools 152 us (1.05
// GB, the measured copy rate); 64 forks of 16-key pages in 20 pools 5.2 us.
#include <algorithm>
#include <memory>
#include <vector>

#include "tf_internal.cuh"

namespace tf {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;         // 16-byte loads in flight a thread
constexpr int kPools = 64;         // pools a launch
constexpr int kRowVecs = TF_D * 2 / 16;

struct Copy {
    int32_t src, dst, keys;
};
// Up to kN copies a launch (kernel arguments hold 32,764 bytes).
template <int kN>
struct Batch {
    uint4* pools[kPools];
    Copy copies[kN];
};

template <int kN>
__global__ void __launch_bounds__(kThreads)
pages_copy_kernel(const __grid_constant__ Batch<kN> b, int page_keys) {
    const Copy c = b.copies[blockIdx.x];
    uint4* pool = b.pools[blockIdx.y];
    const size_t page_vecs = size_t(TF_NKV) * page_keys * kRowVecs;
    const uint4* src = pool + size_t(c.src) * page_vecs;
    uint4* dst = pool + size_t(c.dst) * page_vecs;
    const int run = c.keys * kRowVecs, gap = (page_keys - c.keys) * kRowVecs;   // vectors copied and skipped a head
    const int n = TF_NKV * run;
    pdl_wait();
    for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kUnroll) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            if (i < n) v[u] = __ldcs(src + i + (gap ? i / run * gap : 0));
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0 + u * kThreads;
            if (i < n) __stcs(dst + i + (gap ? i / run * gap : 0), v[u]);
        }
    }
    pdl_trigger();
}

template <int kN>
int launch_batches(void* const* pools, int n_pools, int page_keys, const int32_t* src, const int32_t* dst,
                   const int32_t* keys, int n, cudaStream_t stream) {
    auto b = std::make_unique<Batch<kN>>();
    for (int p0 = 0; p0 < n_pools; p0 += kPools) {
        const int np = std::min(kPools, n_pools - p0);
        for (int p = 0; p < np; ++p) b->pools[p] = static_cast<uint4*>(pools[p0 + p]);
        for (int c0 = 0; c0 < n; c0 += kN) {
            int nc = 0;
            for (int i = c0; i < std::min(n, c0 + kN); ++i)
                if (!keys || keys[i] > 0) b->copies[nc++] = {src[i], dst[i], keys ? keys[i] : page_keys};
            if (nc == 0) continue;
            const int rc = launch_pdl(pages_copy_kernel<kN>, dim3(nc, np), dim3(kThreads), 0, stream, *b, page_keys);
            if (rc != TF_OK) return rc;
        }
    }
    return TF_OK;
}

int copy_pages(void* const* pools, int n_pools, int page_keys, int n_pages, const int32_t* src, const int32_t* dst,
               const int32_t* keys, int n, cudaStream_t stream) {
    if (n_pools < 0 || n < 0 || n_pages < 1) return TF_EINVAL;
    if (page_keys < TF_MIN_PAGE_KEYS || page_keys > TF_MAX_PAGE_KEYS || (page_keys & (page_keys - 1))) return TF_EINVAL;
    if (n_pages > TF_MAX_PAGES || n_pools > 2 * 4096) return TF_ERANGE;
    if ((n_pools > 0 && !pools) || (n > 0 && (!src || !dst))) return TF_EINVAL;
    const size_t bytes = size_t(n_pages) * TF_NKV * page_keys * TF_D * 2;
    std::vector<uintptr_t> at;
    for (int p = 0; p < n_pools; ++p) {
        if (!pools[p] || !aligned16(pools[p])) return TF_EINVAL;
        at.push_back(reinterpret_cast<uintptr_t>(pools[p]));
    }
    std::sort(at.begin(), at.end());
    for (size_t p = 1; p < at.size(); ++p)
        if (at[p] - at[p - 1] < bytes) return TF_EINVAL;
    // ids in the pool; no page written twice, none both read and written
    for (int i = 0; i < n; ++i) {
        if (src[i] < 0 || src[i] >= n_pages || dst[i] < 0 || dst[i] >= n_pages) return TF_EINVAL;
        if (keys && (keys[i] < 0 || keys[i] > page_keys)) return TF_EINVAL;
    }
    if (n_pages <= int64_t(1024) * (n + 64)) {   // a bit a page, unless the pool is huge beside the lists
        std::vector<uint64_t> written(n_pages / 64 + 1);
        for (int i = 0; i < n; ++i) {
            const uint64_t bit = uint64_t(1) << (dst[i] & 63);
            if (written[dst[i] >> 6] & bit) return TF_EINVAL;
            written[dst[i] >> 6] |= bit;
        }
        for (int i = 0; i < n; ++i)
            if (written[src[i] >> 6] >> (src[i] & 63) & 1) return TF_EINVAL;
    } else {
        std::vector<int32_t> written(dst, dst + n);
        std::sort(written.begin(), written.end());
        if (std::adjacent_find(written.begin(), written.end()) != written.end()) return TF_EINVAL;
        for (int i = 0; i < n; ++i)
            if (std::binary_search(written.begin(), written.end(), src[i])) return TF_EINVAL;
    }
    if (n_pools == 0 || n == 0) return TF_OK;
    for (int p = 0; p < n_pools; ++p)
        if (!on_this_device(pools[p])) return TF_EINVAL;
    // few copies travel in a small argument block
    constexpr int kFew = 64, kMany = 2400;
    return n <= kFew ? launch_batches<kFew>(pools, n_pools, page_keys, src, dst, keys, n, stream)
                     : launch_batches<kMany>(pools, n_pools, page_keys, src, dst, keys, n, stream);
}

}  // namespace
}  // namespace tf

extern "C" int tf_pages_copy(void* const* pools, int n_pools, int32_t page_keys, int32_t n_pages, const int32_t* src,
                             const int32_t* dst, const int32_t* keys, int n_copies, tf_cuda_stream stream) {
    try {
        return tf::copy_pages(pools, n_pools, page_keys, n_pages, src, dst, keys, n_copies, stream);
    } catch (...) {
        return TF_ENOMEM;   // out of host memory
    }
}
