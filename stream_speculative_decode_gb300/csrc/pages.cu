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
// Scaled pools (tf_pages_copy_scaled) hold a byte a value, and the scale bytes
// of the 16-key blocks that the copied keys fall in go with them.
//
// HBM bound: 1,024 bytes (8 heads x 128) a key, read and written (scaled: 512.5).
// One CTA a (copy, pool); a whole page is one contiguous run, a part of it 8 runs
// of keys x 128 bytes. Measured: 1,000 whole 64-key pages in 8 pools 152 us (1.05
// GB, the measured copy rate); 64 forks of 16-key pages in 20 pools 5.2 us. Scaled,
// 1,000 whole 128-key pages in 8 pools 154 us; 64 forks of 64-key pages, partly
// filled, in 20 pools 9.6 us. Few copies of large pages take several CTAs each (3
// parts of 256-key pages in 8 pools 4.1 us, a CTA a copy 7.6).
#include <algorithm>
#include <memory>
#include <utility>
#include <vector>

#include "tf_internal.cuh"

namespace tf {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;         // 16-byte loads in flight a thread
constexpr int kPart = kThreads * kUnroll;   // vectors that a CTA has in flight
constexpr int kPools = 64;         // pools a launch

struct Copy {
    int32_t src, dst, keys;
};
// Up to kN copies a launch (kernel arguments hold 32,764 bytes).
template <int kN>
struct Batch {
    uint4* pools[kPools];
    uint8_t* scales[kPools];
    Copy copies[kN];
};

template <int kN, bool kScaled>
__global__ void __launch_bounds__(kThreads)
pages_copy_kernel(const __grid_constant__ Batch<kN> b, int page_keys) {
    constexpr int kRowVecs = TF_D * (kScaled ? 1 : 2) / 16;
    const Copy c = b.copies[blockIdx.x];
    uint4* pool = b.pools[blockIdx.y];
    const size_t page_vecs = size_t(TF_NKV) * page_keys * kRowVecs;
    const uint4* src = pool + size_t(c.src) * page_vecs;
    uint4* dst = pool + size_t(c.dst) * page_vecs;
    const int run = c.keys * kRowVecs, gap = (page_keys - c.keys) * kRowVecs;   // vectors copied and skipped a head
    const int n = TF_NKV * run;
    pdl_wait();
    if constexpr (kScaled) {
        uint8_t* scales = b.scales[blockIdx.y];
        const int per_head = page_keys / TF_SCALE_KEYS, used = (c.keys + TF_SCALE_KEYS - 1) / TF_SCALE_KEYS;
        const int i = threadIdx.x, at = i / per_head, block = i % per_head;   // at most 8 x 16 bytes a page
        if (at < TF_NKV && block < used && blockIdx.z == 0)
            scales[size_t(c.dst) * TF_NKV * per_head + i] = scales[size_t(c.src) * TF_NKV * per_head + i];
    }
    for (int i0 = blockIdx.z * kPart + threadIdx.x; i0 < n; i0 += gridDim.z * kPart) {
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

template <int kN, bool kScaled>
int launch_batches(void* const* pools, void* const* scales, int n_pools, int page_keys, const int32_t* src,
                   const int32_t* dst, const int32_t* keys, int n, cudaStream_t stream) {
    auto b = std::make_unique<Batch<kN>>();
    for (int p0 = 0; p0 < n_pools; p0 += kPools) {
        const int np = std::min(kPools, n_pools - p0);
        for (int p = 0; p < np; ++p) {
            b->pools[p] = static_cast<uint4*>(pools[p0 + p]);
            if (kScaled) b->scales[p] = static_cast<uint8_t*>(scales[p0 + p]);
        }
        for (int c0 = 0; c0 < n; c0 += kN) {
            int nc = 0;
            for (int i = c0; i < std::min(n, c0 + kN); ++i)
                if (!keys || keys[i] > 0) b->copies[nc++] = {src[i], dst[i], keys ? keys[i] : page_keys};
            if (nc == 0) continue;
            // few copies of large pages: several CTAs a copy, as long as SMs would stand idle
            const int parts = (TF_NKV * page_keys * TF_D * (kScaled ? 1 : 2) / 16 + kPart - 1) / kPart;
            const int64_t ctas = int64_t(nc) * np, idle = 2 * sm_count() / ctas;
            const int z = idle < 1 ? 1 : idle < parts ? int(idle) : parts;
            const int rc = launch_pdl(pages_copy_kernel<kN, kScaled>, dim3(nc, np, z), dim3(kThreads), 0, stream, *b,
                                      page_keys);
            if (rc != TF_OK) return rc;
        }
    }
    return TF_OK;
}

template <bool kScaled>
int copy_pages(void* const* pools, void* const* scales, int n_pools, int page_keys, int n_pages, const int32_t* src,
               const int32_t* dst, const int32_t* keys, int n, cudaStream_t stream) {
    if (n_pools < 0 || n < 0 || n_pages < 1) return TF_EINVAL;
    if (page_keys < TF_MIN_PAGE_KEYS || page_keys > TF_MAX_PAGE_KEYS || (page_keys & (page_keys - 1))) return TF_EINVAL;
    if (n_pages > TF_MAX_PAGES || n_pools > 2 * 4096) return TF_ERANGE;
    if ((n_pools > 0 && (!pools || (kScaled && !scales))) || (n > 0 && (!src || !dst))) return TF_EINVAL;
    const size_t slots = size_t(n_pages) * TF_NKV * page_keys, bytes = slots * TF_D * (kScaled ? 1 : 2);
    std::vector<std::pair<uintptr_t, uintptr_t>> at;   // where the pools lie: [first, last)
    for (int p = 0; p < n_pools; ++p) {
        if (!pools[p] || !aligned16(pools[p])) return TF_EINVAL;
        const uintptr_t a = reinterpret_cast<uintptr_t>(pools[p]);
        at.push_back({a, a + bytes});
        if constexpr (kScaled) {
            if (!scales[p]) return TF_EINVAL;
            const uintptr_t b = reinterpret_cast<uintptr_t>(scales[p]);
            at.push_back({b, b + slots / TF_SCALE_KEYS});
        }
    }
    std::sort(at.begin(), at.end());
    for (size_t p = 1; p < at.size(); ++p)
        if (at[p].first < at[p - 1].second) return TF_EINVAL;
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
        if (!on_this_device(pools[p]) || (kScaled && !on_this_device(scales[p]))) return TF_EINVAL;
    // few copies travel in a small argument block
    constexpr int kFew = 64, kMany = 2400;
    return n <= kFew ? launch_batches<kFew, kScaled>(pools, scales, n_pools, page_keys, src, dst, keys, n, stream)
                     : launch_batches<kMany, kScaled>(pools, scales, n_pools, page_keys, src, dst, keys, n, stream);
}

}  // namespace
}  // namespace tf

extern "C" int tf_pages_copy(void* const* pools, int n_pools, int32_t page_keys, int32_t n_pages, const int32_t* src,
                             const int32_t* dst, const int32_t* keys, int n_copies, tf_cuda_stream stream) {
    try {
        return tf::copy_pages<false>(pools, nullptr, n_pools, page_keys, n_pages, src, dst, keys, n_copies, stream);
    } catch (...) {
        return TF_ENOMEM;   // out of host memory
    }
}

extern "C" int tf_pages_copy_scaled(void* const* pools, void* const* scales, int n_pools, int32_t page_keys,
                                    int32_t n_pages, const int32_t* src, const int32_t* dst, const int32_t* keys,
                                    int n_copies, tf_cuda_stream stream) {
    try {
        return tf::copy_pages<true>(pools, scales, n_pools, page_keys, n_pages, src, dst, keys, n_copies, stream);
    } catch (...) {
        return TF_ENOMEM;   // out of host memory
    }
}
