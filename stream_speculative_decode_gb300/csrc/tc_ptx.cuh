// Inline-PTX building blocks of the tensor-core kernels on sm_103a: shared
// memory matrix descriptors, mbarriers with bounded waits, TMA tile loads and
// the tcgen05 MMA / commit / tensor-memory load and store forms they use.
//
// Every wait here is bounded by %globaltimer: mbar_wait gives up after the
// CTA's wait limit (tf_set_wait_limit_ns, passed in the table; raising the
// CTA's abort flag), mbar_drain after kDrainNs whatever that limit is, so
// that a CTA which gave up still lets its own copies and MMAs land.
#pragma once

#include "tf_internal.cuh"

namespace tf {
namespace {

constexpr unsigned long long kDrainNs = 200000000ull;

// What a CTA's bounded waits share, in shared memory: the abort flag a wait
// that runs out raises (the CTA's other waits then give up at once), and the
// wait limit in nanoseconds.
struct WaitCtl {
    uint32_t flag;
    uint32_t pad_;
    unsigned long long limit_ns;
};

// Shared-memory matrix descriptor: start address, leading / stride byte
// offsets (16-byte units), descriptor version 1, 128-byte swizzle (layout 2).
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = uint64_t((addr >> 4) & 0x3FFFu);
    d |= uint64_t((lbo >> 4) & 0x3FFFu) << 16;
    d |= uint64_t((sbo >> 4) & 0x3FFFu) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ unsigned long long gtime() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ void mbar_init(uint32_t a, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t a, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t a) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t a, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(a), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait; false on timeout (raises the abort flag) or when another
// thread raised it.
__device__ bool mbar_wait(uint32_t a, uint32_t parity, volatile WaitCtl* wc) {
    if (mbar_test(a, parity)) return true;
    const unsigned long long t0 = gtime(), limit = wc->limit_ns;
    for (;;) {
        if (mbar_test(a, parity)) return true;
        if (wc->flag) return false;
        if (gtime() - t0 > limit) {
            wc->flag = 1;
            return false;
        }
    }
}
// The same wait by a whole warp, with one outcome for all its lanes (a lane
// that ran out would otherwise leave the warp's collective operations short).
__device__ __forceinline__ bool mbar_wait_warp(uint32_t a, uint32_t parity, volatile WaitCtl* wc) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(a, parity, wc));
}
// Bounded wait that ignores the abort flag (draining after an abort).
__device__ void mbar_drain(uint32_t a, uint32_t parity) {
    const unsigned long long t0 = gtime();
    while (!mbar_test(a, parity) && gtime() - t0 < kDrainNs) {
    }
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// 64 consecutive columns of this thread's lane (one wait by the caller)
__device__ __forceinline__ void tc_ld64(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}
// N (2..64) consecutive 32-bit columns of this thread's lane; the caller waits
template <int N>
__device__ __forceinline__ void tc_ld_n(uint32_t taddr, uint32_t (&r)[N]) {
    if constexpr (N == 2) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
    } else if constexpr (N == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    } else if constexpr (N == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                       "=r"(r[7]) : "r"(taddr));
    } else if constexpr (N == 16) {
        tc_ld16(taddr, r);
    } else if constexpr (N == 64) {
        tc_ld64(taddr, r);
    } else {
        static_assert(N == 32, "2, 4, 8, 16, 32 or 64 columns");
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
              "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
              "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(taddr));
    }
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tc_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void tc_st_n(uint32_t taddr, const uint32_t (&r)[N]) {
    if constexpr (N == 4) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                     ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    } else if constexpr (N == 8) {
        tc_st8(taddr, r);
    } else if constexpr (N == 32) {
        tc_st32(taddr, r);
    } else {
        static_assert(N == 16, "4, 8, 16 or 32 columns");
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
            ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
              "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
    }
}
// The 16x32bx2 shape: threads 0-15 of the warp access lanes 0-15 of its
// quadrant at columns [c, c + N), threads 16-31 the same lanes at columns
// [c + OFF, c + OFF + N) -- two threads share a lane, each with its half of the
// columns.
template <int OFF>
__device__ __forceinline__ void tc_ld16x2_16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ void tc_ld16x2_32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr), "n"(OFF));
}
template <int OFF>
__device__ __forceinline__ void tc_st16x2_16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %1, {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17};"
        ::"r"(taddr), "n"(OFF), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4& v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
// The same load with an L2 cache policy (e.g. l2_evict_last()).
__device__ __forceinline__ void tma_load_2d_hint(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "l"(policy) : "memory");
}
// L2 policy: keep the lines (evicted after normal and evict-first lines).
__device__ __forceinline__ uint64_t l2_evict_last() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}
// Fetch a tile of a 3-D tensor map into L2 only (no shared memory, no barrier).
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const int sz = valid ? 16 : 0;   // 0: fill the 16 bytes with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(sz) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The same 3-D load with an L2 cache policy (e.g. l2_evict_first()).
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                                 uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy) : "memory");
}
// L2 policy: lines read once (evicted before normal lines).
__device__ __forceinline__ uint64_t l2_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void tc_alloc(uint32_t slot_smem, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot_smem), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t taddr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// ---- what the tensor-core attention kernels share ----------------------------
// (attn_tc.cu over bf16 caches and pools, attn_scaled_tc.cu over scaled pools):
// units of work and their tiles, the queue that hands a persistent CTA its units,
// the queries' tile, Blackwell's paired fp32 instructions. B: a kernel's barriers,
// with uq, uq_full, uq_empty and grp.

constexpr int kKT = 64;                     // keys per tile
constexpr int kQRows = 128;                 // MMA M
constexpr int kQB = kQRows * TF_D * 2;      // 16 KB
constexpr int kUQ = 4;                      // queue of the CTA's next units

// One unit of work: one key chunk of one stream (an attention item) for one
// KV head. A CTA takes the units blockIdx.x, blockIdx.x + gridDim.x, ... of the
// tensor-core items (largest first); every role walks the same list.
struct Unit {
    SegStream st;
    const CUtensorMap* kmap;
    const CUtensorMap* vmap;
    int stream, chunk, g, c0, T;
    int pages;   // paged: the list entry of the chunk's first key
};
template <bool kPaged>
__device__ __forceinline__ Unit unit_of(const SegTable& t, int layer, int u) {
    Unit U;
    const AttnItem it = t.items[t.n_items_mma + u / TF_NKV];   // tensor-core items follow the mma.sync ones
    U.g = u % TF_NKV;
    U.stream = it.stream;
    U.chunk = it.chunk;
    U.st = t.streams[it.stream];
    U.pages = it.pages;
    U.c0 = it.chunk * U.st.chunk_keys;
    U.T = (min(U.st.chunk_keys, U.st.keys - U.c0) + kKT - 1) / kKT;
    const size_t slot = kPaged ? size_t(layer) : size_t(layer) * t.S + it.stream;
    U.kmap = t.k_maps + slot;
    U.vmap = t.v_maps + slot;
    return U;
}

// The page ids of tile j of a unit (x only for pages of 64 keys or more, x and
// y for 32-key pages, all four for 16-key pages).
__device__ __forceinline__ int4 tile_pages(const SegTable& t, const Unit& U, int j) {
    const int32_t* ids = t.pages + U.pages + ((j * kKT) >> t.page_shift);   // c0 starts a page
    if (t.page_shift == 4) return __ldg(reinterpret_cast<const int4*>(ids));
    if (t.page_shift == 5) {
        const int2 p = __ldg(reinterpret_cast<const int2*>(ids));
        return make_int4(p.x, p.y, 0, 0);
    }
    return make_int4(__ldg(ids), 0, 0, 0);
}
// Tile j of a paged unit: f(offset in the tile, slot in the page, page) for each of its boxes.
template <typename F>
__device__ __forceinline__ void tile_boxes(const SegTable& t, const Unit& U, int j, int4 id, F&& f) {
    const int ps = t.page_shift;
    f(0u, ps >= 6 ? (U.c0 + j * kKT) & ((1 << ps) - 1) : 0, id.x);
    if (ps == 5) f(32u * 128u, 0, id.y);
    if (ps == 4) {
        f(16u * 128u, 0, id.y);
        f(32u * 128u, 0, id.z);
        f(48u * 128u, 0, id.w);
    }
}

// Blackwell's three-input max and paired fp32 FMA / add: each of these does
// the work of two instructions with the same per-element rounding.
__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2pack(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2unpack(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The m-th unit the producer handed this CTA after its first (blockIdx.x), or
// -1: no more (or the CTA gave up). Single-thread consumer (the MMA thread).
template <typename B>
__device__ __forceinline__ int next_unit_thread(B* bars, int m, volatile WaitCtl* abortp) {
    const int slot = m % kUQ;
    if (!mbar_wait(su32(&bars->uq_full[slot]), (m / kUQ) & 1, abortp)) return -1;
    const int u = reinterpret_cast<volatile int32_t*>(bars->uq)[slot];
    mbar_arrive(su32(&bars->uq_empty[slot]));
    return u;
}
// The same for a whole warp: every lane reads, then lane 0 releases the slot.
template <typename B>
__device__ __forceinline__ int next_unit_warp(B* bars, int m, volatile WaitCtl* abortp) {
    const int slot = m % kUQ;
    int u = -1;
    if (mbar_wait_warp(su32(&bars->uq_full[slot]), (m / kUQ) & 1, abortp))
        u = reinterpret_cast<volatile int32_t*>(bars->uq)[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(su32(&bars->uq_empty[slot]));
    return u;
}

// The four softmax warps (128 threads) meet; bounded like every wait here.
template <typename B>
__device__ __forceinline__ bool group_sync(B* bars, int& ph, volatile WaitCtl* abortp) {
    mbar_arrive(su32(&bars->grp));
    const bool ok = mbar_wait(su32(&bars->grp), ph & 1, abortp);
    ++ph;
    return ok;
}

// Query rows of a unit per TMEM lane quadrant: 16 for windows of at most 16
// rows (dual softmax: lanes L and L + 16 of a quadrant hold the same query),
// 32 for the prompt's wider windows. Quadrant w holds the unit's queries
// [per*w, per*w + per), i.e. window rows per/4*w .. +per/4 - 1 with their four
// heads of the KV head.
__device__ __forceinline__ int q_per(int rows) { return rows <= 16 ? 16 : 32; }

// The unit's queries into shared memory by TMA (one thread), K-major with the
// 128-byte swizzle, lane L of the Q tile holding query per*(L/32) + L%per
// (dual: lanes L%32 < 16 only): boxes of 16 query rows (4 window rows x 4
// heads), completing `bar` with 16 KB. Rows past the window belong to no query
// of the unit (other streams' rows, or zeros past the last row): their lanes
// are not valid rows and their results are never written.
__device__ __forceinline__ void issue_q(uint32_t sQ, const CUtensorMap* qmap, const Unit& U, uint32_t bar) {
    const bool dual = U.st.rows <= 16;
    mbar_expect_tx(bar, dual ? kQB / 2 : kQB);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int w = k >> 1, h = k & 1;
        // dual: lanes 0-15 of quadrant w hold window rows 4w..4w+3 (lanes 16-31
        // hold no query: their S rows are never read); else the halves hold
        // rows 8w..8w+3 and 8w+4..8w+7
        if (dual && h) continue;
        const int row = U.st.row_offset + (dual ? 4 * w : 8 * w + 4 * h);
        tma_load_3d(sQ + uint32_t(32 * w + 16 * h) * 128u, qmap, 0, 4 * U.g, row, bar);
    }
}

}  // namespace
}  // namespace tf
