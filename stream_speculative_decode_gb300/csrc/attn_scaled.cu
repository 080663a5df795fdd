// Attention (tf_attn_paged) over scaled pools: keys and values as e4m3 codes
// with a power-of-two scale for each 16 keys of a head. Items, partial records
// and merges are those of attn.cu, and so are the chunks; a window of more than 8 rows runs as
// several items over its chunk, next to each other in the grid.
//
// With c the codes, ek and ev a block's exponents and x the scores in log2 units:
//   x_t = (q . ck_t) * 2^ek * log2(e) / 8
//   o = sum 2^x_t 2^ev cv_t / sum 2^x_t
// HBM bound: 128 bytes of K and V (and 1/8 of scales) a key and KV head, half of
// the bf16 caches', so what a key costs in instructions counts twice as much:
//
// - The products run transposed on mma.sync m16n8k16: 16 keys (then 16 dimensions
//   of V) by 8 queries, so that a window of two rows fills a tile; 16 queries a
//   tile would double the MMAs and softmax work of narrow windows.
// - A lane's fragments of K are 16 consecutive codes of a key's row, those of V
//   8 consecutive dimensions of four keys: the order of the summed index is free
//   as long as both factors have it. Codes become fp16 in registers (exact).
// - K's scale is a factor of the block's scores. V's enters the weights that go
//   into P.V, w = 2^(x - m) * 2^(ev - E) with E the chunk's largest exponent, so
//   the accumulators hold o / 2^E; the sum l takes 2^(x - m) itself. The
//   reference m moves when a w passes 2^15 (fp16 holds 65,504), to put the
//   largest at 2^6: the small weights then keep fp16's 11 bits down to 2^-20 of
//   the largest and vanish below 2^-31. A V block 2^64 below the chunk's largest
//   counts as if it were 2^64 below (its codes are weighed by 2^-64).
// - Queries become fp16 under a power of two of their own that puts a head's
//   largest at 2^14: exact for bf16 values down to 2^-28 of it, off by at most
//   2^-39 of it below.
//
// Four warps share a chunk: warp w takes the stages (32 keys) w, w + 4, ... of
// it through a ring of its own (cp.async, no CTA barrier in the loop); their
// results are joined at the end. A stage's two blocks go through the products and
// the softmax together: a warp's instructions wait mostly for one another, with
// three or four warps a scheduler, and a test of the reference serves both.
//
// Measured: 4 windows of 6 rows at 65,536 to 130,816 keys 90.8 us (4.6 TB/s; a
// block at a time 97.1), of 2 rows 72.8 us (5.7 TB/s, 85 % of the measured copy
// rate); 16 single rows at 256 to 4,096 keys 9.4 us. What bounds it is latency: three
// warps a scheduler in chains of dependent instructions, some 245 a block of 24
// queries, which wait mostly for one another; half of the issue slots are used, and no
// pipe above 40 %. The queries of 3 or 4 tiles lie in shared memory, which leaves three
// CTAs an SM their registers; four CTAs a block at a time with 24 queries 97.7 us.
//
// What no row of the item may see is kept out: scores are masked, and in blocks
// that reach past the first row's keys a NaN code of V is taken out of the
// product and put back, as NaN, into the rows that see its key.
#include "attn_item.cuh"
#include "scaled.cuh"

namespace tf {
namespace {

using item::kThreads;
using item::kWarps;
using item::ex2;
using item::pack_h2;
using item::mma_f16;
using item::smem_u32;

constexpr int kKeys = TF_SCALE_KEYS;           // a block: the keys that share a scale
constexpr int kStageKeys = 2 * kKeys;
constexpr int kBlockB = kKeys * TF_D;          // 1 KB of codes
constexpr int kStageB = 4 * kBlockB;           // K of two blocks, then V of them
constexpr int kStages = 3;
constexpr int kRingB = kStages * kStageB;
constexpr int kOStride = TF_D + 4;             // floats a query row of the warps' joining
constexpr int kBlocks = 512 * TF_MAX_ROWS / kKeys;   // blocks of the longest chunk
constexpr float kLog2e8 = 0.18033688011112042f;      // log2(e) / sqrt(64)
constexpr float kNoRef = -3e38f;               // the reference of a query without a key so far
constexpr float kLargest = 32768.f;            // 2^15: a weight beyond it moves the row's reference
constexpr float kHeadroom = 6.f;               // log2 of the largest weight after that
constexpr int kMaxShift = 64;
static_assert(kStageKeys * kWarps <= 256, "chunks are whole rounds of the warps");
static_assert(kKeys == item::kBlockKeys && kBlocks * 4 == item::kBlocksB, "one block index for pools and scales");

// ring (joined through it at the end), block indices, scales (K's, and V's exponent), the warps' largest V
constexpr int smem_bytes(int NT) {
    return kWarps * kRingB + kBlocks * 4 + kBlocks * 8 + 16 + (NT >= 3 ? NT * 1024 : 0);
}
static_assert(kWarps * kRingB >= kWarps * 8 * 4 * (kOStride + 2) * 4, "the joining fits the rings");

__device__ __forceinline__ void movmatrix_t(uint32_t& d, uint32_t a) {
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// Pairs of fp32, an instruction for both.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 both(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Where the 16 bytes `c` (0..3) of key row r lie in a block's 1 KB of shared
// memory: two rows a 128-byte line, their order such that the lanes of a phase
// (K: rows i and 4 + i, all of c; V: four consecutive rows, two of c) fall on
// different banks.
__device__ __forceinline__ uint32_t k_at(int r, int c) { return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 4)) << 4); }
__device__ __forceinline__ uint32_t v_at(int r, int c) { return (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 2)) << 4); }

// MMA row i of a K tile is key perm(i) of its block: the keys 2 t4, 2 t4 + 1 (and
// + 8) that a lane weighs are then the four rows t4, 4 + t4, ... of V.
__device__ __forceinline__ int perm(int i) { return (i & 8) | ((i & 1) << 2) | ((i & 7) >> 1); }

// Bytes 0xFF where a code is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// One item: one key chunk of one stream, query rows [q0, q0 + 8 NT) of KV head
// g, by 128 threads.
template <int NT>
__global__ void __launch_bounds__(kThreads, NT <= 2 ? 4 : 3)
attn_scaled_kernel(SegTable t, int layer, const uint16_t* __restrict__ q, float* __restrict__ part_o,
                   float2* __restrict__ part_ml, uint16_t* __restrict__ out, int full) {
    extern __shared__ __align__(128) unsigned char smem[];
    uint32_t* const blocks = reinterpret_cast<uint32_t*>(smem + kWarps * kRingB);
    float2* const scales = reinterpret_cast<float2*>(blocks + kBlocks);   // K's scale, V's exponent
    uint32_t* const top = reinterpret_cast<uint32_t*>(scales + kBlocks);
    uint2* const sq = reinterpret_cast<uint2*>(top + kWarps) + (threadIdx.x & 31);   // [nt][ks][lane], kSharedQ
    constexpr bool kSharedQ = NT >= 3;   // query fragments in shared memory
    constexpr int B = kStageKeys / kKeys;   // blocks at a time (for every NT: a stream's bits are its own)
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int g = blockIdx.x % TF_NKV;
    const AttnItem it = t.items[blockIdx.x / TF_NKV];
    const SegStream st = t.streams[it.stream];
    const int q0 = it.q0;
    const int nq = min(8 * NT, st.rows * 4 - q0);
    const int c0 = it.chunk * st.chunk_keys;
    const int nkeys = min(st.chunk_keys, st.keys - c0);
    const int nblocks = (nkeys + kKeys - 1) / kKeys;
    item::load_blocks(t, it, nkeys, g, blocks, tid, kThreads);
    const size_t slot = size_t(layer) * t.S + it.stream;
    const uint8_t* const Kp = static_cast<const uint8_t*>(t.k_cache[slot]);
    const uint8_t* const Vp = static_cast<const uint8_t*>(t.v_cache[slot]);
    __syncthreads();
    pdl_wait();   // the table above; queries and caches below

    // ---- the ring
    const uint32_t ring = smem_u32(smem) + warp * kRingB;
    const int nst = (nkeys + kStageKeys - 1) / kStageKeys;
    const int mine = nst > warp ? (nst - warp + kWarps - 1) / kWarps : 0;
    // this lane's two 16-byte pieces of a block: rows lane / 4 and 8 + lane / 4
    const uint32_t kd = k_at(lane >> 2, lane & 3), vd = v_at(lane >> 2, lane & 3);
    auto issue = [&](int i) {
        const uint32_t buf = ring + (i % kStages) * kStageB;
        const uint2 b = *reinterpret_cast<const uint2*>(blocks + 2 * (warp + i * kWarps));
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // a second block past the chunk is block 0: read, never used
            const size_t off = size_t(k ? b.y : b.x) * kBlockB + lane * 16;
            copy16(buf + k * kBlockB + kd, Kp + off);
            copy16(buf + k * kBlockB + kd + kBlockB / 2, Kp + off + kBlockB / 2);
            copy16(buf + (2 + k) * kBlockB + vd, Vp + off);
            copy16(buf + (2 + k) * kBlockB + vd + kBlockB / 2, Vp + off + kBlockB / 2);
        }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < mine) issue(i);
        item::cp_async_commit();
    }

    // ---- the chunk's scales
    {
        const uint8_t *ks = t.k_scale[layer], *vs = t.v_scale[layer];
        uint32_t m = 0;
        for (int i = tid; i < nblocks; i += kThreads) {
            const uint32_t b = blocks[i], e = vs[b];
            scales[i] = make_float2(scale_value(ks[b]), float(e));
            m = max(m, e);
        }
        if (tid == 0 && (nblocks & 1)) scales[nblocks] = make_float2(1.f, 0.f);   // a last pair's missing block, masked
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (lane == 0) top[warp] = m;
    }

    // ---- queries: column n of a tile is query row q0 + 8 nt + n (window row / 4, head % 4)
    uint2 qf[kSharedQ ? 1 : NT][4];
    uint64_t cq[NT];   // factors of the columns 2 t4, 2 t4 + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int qi = nt * 8 + g8;
        uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (qi < nq) {
            const size_t row = st.row_offset + ((q0 + qi) >> 2);
            const uint16_t* src = q + (row * TF_NQ + 4 * g + (qi & 3)) * TF_D + 16 * t4;
            const uint4 a = *reinterpret_cast<const uint4*>(src), b = *reinterpret_cast<const uint4*>(src + 8);
            w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            most = max(most, max(finite_bits(__uint_as_float(w[i] << 16)),
                                 finite_bits(__uint_as_float(w[i] & 0xFFFF0000u))));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int up = min(141 - int(most >> 23), 100);   // the head's largest becomes 2^14..2^15
        const float mul = __uint_as_float(uint32_t(127 + up) << 23);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            auto half2 = [&](uint32_t v) {
                return pack_h2(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xFFFF0000u) * mul);
            };
            const uint2 f = make_uint2(half2(w[2 * ks]), half2(w[2 * ks + 1]));
            if constexpr (!kSharedQ)
                qf[nt][ks] = f;
            else if (warp == nt)
                sq[(nt * 4 + ks) * 32] = f;
        }
        const float back = __uint_as_float(uint32_t(127 - up) << 23) * kLog2e8;
        cq[nt] = pair(__shfl_sync(0xFFFFFFFFu, back, 8 * t4), __shfl_sync(0xFFFFFFFFu, back, 8 * t4 + 4));
    }
    __syncthreads();
    const int E = int(max(max(top[0], top[1]), max(top[2], top[3])));

    // keys that a column's window row sees, chunk-local (a tile's columns 2 t4 and 2 t4 + 1 are of one row)
    int lim[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int qi = nt * 8 + 2 * t4;
        const int vis = (full ? st.keys : st.keys - st.rows + ((q0 + qi) >> 2) + 1) - c0;
        lim[nt] = qi < nq ? max(0, min(vis, nkeys)) : 0;
    }
    const int lim_all = min((full ? st.keys : st.keys - st.rows + (q0 >> 2) + 1) - c0, nkeys);

    float o[NT][4][4];
    uint64_t nm[NT], l[NT];   // of both columns: minus the reference, this lane's sum of 2^(x - m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
        nm[nt] = pair(-kNoRef, -kNoRef);
        l[nt] = pair(0.f, 0.f);
    }
    // this lane's pieces in a block: K rows perm(g8) and 8 + perm(g8), V rows t4, 4 + t4, 8 + t4, 12 + t4
    const uint32_t ka = k_at(perm(g8), t4);
    const uint32_t va0 = v_at(t4, g8 >> 1) + (g8 & 1) * 8, va1 = v_at(4 + t4, g8 >> 1) + (g8 & 1) * 8;

    for (int i = 0; i < mine; ++i) {
        if (i + kStages - 1 < mine) issue(i + kStages - 1);
        item::cp_async_commit();
        item::cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t buf = ring + (i % kStages) * kStageB;
        const int bi = 2 * (warp + i * kWarps);
        const int key0 = bi * kKeys;
        const bool edge = key0 + B * kKeys > lim_all;
        const uint64_t tiny2 = pair(0x1p-149f, 0x1p-149f);   // keeps a factor above 0: a masked score is -inf
        float dv[B], kf[B];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float2 sc = scales[bi + b];
            kf[b] = sc.x;
            dv[b] = fmaxf(sc.y - float(E), float(-kMaxShift));
        }

        // scores
        float s[B][NT][4];
        {
            uint4 w[B][2];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                w[b][0] = lds16(buf + b * kBlockB + ka);
                w[b][1] = lds16(buf + b * kBlockB + ka + kBlockB / 2);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[b][nt][0] = s[b][nt][1] = s[b][nt][2] = s[b][nt][3] = 0.f;
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                uint2 qs[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) qs[nt] = kSharedQ ? sq[(nt * 4 + ks) * 32] : qf[kSharedQ ? 0 : nt][ks];
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const uint32_t r0 = (&w[b][0].x)[ks], r1 = (&w[b][1].x)[ks];
                    const uint32_t a[4] = {e4m3_low(r0), e4m3_low(r1), e4m3_high(r0), e4m3_high(r1)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(s[b][nt], a, qs[nt].x, qs[nt].y);
                }
            }
        }
        if (edge) {
#pragma unroll
            for (int b = 0; b < B; ++b)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int key = key0 + b * kKeys + perm(g8);
                    if (key >= lim[nt]) s[b][nt][0] = s[b][nt][1] = -INFINITY;
                    if (key + 8 >= lim[nt]) s[b][nt][2] = s[b][nt][3] = -INFINITY;
                }
        }
        // weights, in fp32 and (pw) as fp16 pairs; a weight is at most the sum of all
        uint32_t pw[B][NT][2];
        uint64_t ln[NT];   // l with these blocks'
        auto weigh = [&]() {
            uint64_t all = pair(0.f, 0.f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ln[nt] = l[nt];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                const float down = ex2(-dv[b]);
                const uint64_t kf2 = pair(kf[b], kf[b]), dv2 = pair(dv[b], dv[b]), down2 = pair(down, down);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint64_t f = fma2(cq[nt], kf2, tiny2), c = add2(nm[nt], dv2);
                    const float2 x = both(fma2(pair(s[b][nt][0], s[b][nt][1]), f, c));
                    const float2 y = both(fma2(pair(s[b][nt][2], s[b][nt][3]), f, c));
                    const float w0 = ex2(x.x), w1 = ex2(x.y), w2 = ex2(y.x), w3 = ex2(y.y);
                    const uint64_t ps = add2(pair(w0, w1), pair(w2, w3));
                    all = add2(all, ps);
                    ln[nt] = fma2(ps, down2, ln[nt]);
                    pw[b][nt][0] = pack_h2(w0, w1);
                    pw[b][nt][1] = pack_h2(w2, w3);
                }
            }
            const float2 a = both(all);
            return !(a.x + a.y <= kLargest);
        };
        if (__any_sync(0xFFFFFFFFu, weigh())) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float2 old = both(nm[nt]);
                float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int b = 0; b < B; ++b) {
                    const float2 f = both(fma2(cq[nt], pair(kf[b], kf[b]), tiny2));
                    y[0] = fmaxf(y[0], fmaxf(s[b][nt][0] * f.x, s[b][nt][2] * f.x) + dv[b]);
                    y[1] = fmaxf(y[1], fmaxf(s[b][nt][1] * f.y, s[b][nt][3] * f.y) + dv[b]);
                }
                float to[2] = {-old.x, -old.y}, alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int d = 4; d < 32; d *= 2) y[e] = fmaxf(y[e], __shfl_xor_sync(0xFFFFFFFFu, y[e], d));
                    y[e] -= kHeadroom;
                    alpha[e] = 1.f;
                    if (y[e] > to[e] + (15.f - kHeadroom)) {   // this row's own: others do not move it
                        alpha[e] = ex2(to[e] - y[e]);
                        to[e] = y[e];
                    }
                }
                nm[nt] = pair(-to[0], -to[1]);
                l[nt] = mul2(l[nt], pair(alpha[0], alpha[1]));
#pragma unroll
                for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][mt][e] *= alpha[e & 1];
            }
            weigh();
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt] = ln[nt];
#pragma unroll
            for (int b = 0; b < B; ++b) {
                movmatrix_t(pw[b][nt][0], pw[b][nt][0]);
                movmatrix_t(pw[b][nt][1], pw[b][nt][1]);
            }
        }
        // P.V: MMA row g8 of tile mt is dimension 8 g8 + 2 mt, row 8 + g8 the next one
        auto product = [&](const uint2 (&c)[4], const uint32_t (&p)[NT][2], float (&acc)[NT][4][4]) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;   // bytes 2 mt, 2 mt + 1 of both
                const uint32_t lo = __byte_perm(mt < 2 ? c[0].x : c[0].y, mt < 2 ? c[1].x : c[1].y, sel);
                const uint32_t hi = __byte_perm(mt < 2 ? c[2].x : c[2].y, mt < 2 ? c[3].x : c[3].y, sel);
                const uint32_t a[4] = {e4m3_low(lo), e4m3_high(lo), e4m3_low(hi), e4m3_high(hi)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(acc[nt][mt], a, p[nt][0], p[nt][1]);
            }
        };
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const uint32_t bv = buf + (2 + b) * kBlockB;
            uint2 v[4] = {lds8(bv + va0), lds8(bv + va1), lds8(bv + kBlockB / 2 + va0), lds8(bv + kBlockB / 2 + va1)};
            if (edge) {
                uint2 bad[4];
                uint32_t any = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    bad[j] = make_uint2(nan_bytes(v[j].x), nan_bytes(v[j].y));
                    any |= bad[j].x | bad[j].y;
                }
                if (__any_sync(0xFFFFFFFFu, any != 0)) {
                    const int key = key0 + b * kKeys + perm(g8);
                    uint32_t sees[NT][2];   // 1 where the column's row sees the key
                    float hits[NT][4][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t one = 0x3C003C00u;
                        movmatrix_t(sees[nt][0], key < lim[nt] ? one : 0u);
                        movmatrix_t(sees[nt][1], key + 8 < lim[nt] ? one : 0u);
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) hits[nt][mt][e] = 0.f;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j].x &= ~bad[j].x;
                        v[j].y &= ~bad[j].y;
                        bad[j].x &= 0x38383838u;   // 1 as a code
                        bad[j].y &= 0x38383838u;
                    }
                    product(bad, sees, hits);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (hits[nt][mt][e] > 0.f) o[nt][mt][e] = __uint_as_float(0x7FC00000u);
                }
            }
            product(v, pw[b], o);
        }
        __syncwarp();   // the stage is read: its buffer may be filled again
    }
    item::cp_async_wait<0>();
    __syncthreads();
    pdl_trigger();

    // ---- join the four warps (the ring's memory): the record, or the output
    float* const sO = reinterpret_cast<float*>(smem);   // [4][8 NT][kOStride]
    float* const sM = sO + kWarps * 8 * NT * kOStride;  // [4][8 NT]
    float* const sL = sM + kWarps * 8 * NT;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const float2 sums = both(l[nt]), refs = both(nm[nt]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float sum = e ? sums.y : sums.x;
#pragma unroll
            for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            const int col = warp * 8 * NT + nt * 8 + 2 * t4 + e;
            if (g8 == 0) {
                sM[col] = e ? -refs.y : -refs.x;
                sL[col] = sum;
            }
            float4* row = reinterpret_cast<float4*>(sO + col * kOStride + 8 * g8);
            row[0] = make_float4(o[nt][0][e], o[nt][0][2 + e], o[nt][1][e], o[nt][1][2 + e]);
            row[1] = make_float4(o[nt][2][e], o[nt][2][2 + e], o[nt][3][e], o[nt][3][2 + e]);
        }
    }
    __syncthreads();
    const int mode = out ? st.merge_mode : kMergeKernel;
    const int64_t rec0 = st.pbase + (int64_t(it.chunk) * TF_NKV + g) * (st.rows * 4) + q0;
    const int half = (E - kScaleBias) / 2;   // 2^E in two factors, both normal numbers
    const float up0 = __uint_as_float(uint32_t(127 + half) << 23);
    const float up1 = __uint_as_float(uint32_t(127 + E - kScaleBias - half) << 23);
    for (int idx = tid; idx < nq * (TF_D / 4); idx += kThreads) {
        const int qi = idx >> 4, d4 = (idx & 15) * 4;
        float M = kNoRef;   // (a weight NaN leaves o NaN as well)
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sM[w * 8 * NT + qi]);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            // 0 for a warp without a key of the row, whose sums are 0 or NaN
            const float f = ex2(sM[w * 8 * NT + qi] - M);
            const float4 v = *reinterpret_cast<const float4*>(sO + (w * 8 * NT + qi) * kOStride + d4);
            L += f * sL[w * 8 * NT + qi];
            acc.x += f * v.x;
            acc.y += f * v.y;
            acc.z += f * v.z;
            acc.w += f * v.w;
        }
        if (mode == kMergeDirect) {
            const float inv = 1.f / L;
            store_out4(out_row(out, st, g, q0 + qi) + d4,
                       make_float4(acc.x * inv * up0 * up1, acc.y * inv * up0 * up1, acc.z * inv * up0 * up1,
                                   acc.w * inv * up0 * up1));
        } else {
            *reinterpret_cast<float4*>(part_o + (rec0 + qi) * TF_D + d4) =
                make_float4(acc.x * up0 * up1, acc.y * up0 * up1, acc.z * up0 * up1, acc.w * up0 * up1);
            if (d4 == 0) {   // a row without a key; a sum that is no number, which a merge must not take for none
                const bool lost = !(L <= 3e38f);
                part_ml[rec0 + qi] = make_float2(M > kNoRef ? M : lost ? 0.f : -INFINITY, lost ? INFINITY : L);
            }
        }
    }
    if (mode == kMergeLastCta) {
        __shared__ int last_flag;
        finish_last_cta<8>(t, layer, it.stream, st, g, part_o, part_ml, out, &last_flag);
    }
}

template <int NT>
int prepare_one() {
    cudaError_t e = cudaFuncSetAttribute(attn_scaled_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_bytes(NT));
    return e == cudaSuccess ? TF_OK : cuda_fail(e);
}

template <int NT>
int launch_one(const SegTable& t, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
               uint16_t* out, int full) {
    return launch_pdl(attn_scaled_kernel<NT>, dim3(t.n_items_mma * TF_NKV), dim3(kThreads), smem_bytes(NT), stream, t,
                      layer, q, po, pml, out, full);
}

int launch_mma(const SegTable& t, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
               uint16_t* out, int full) {
    const int nt = (t.item_rows + 1) / 2;   // tiles of 8 query rows in the widest item
    return nt == 1 ? launch_one<1>(t, layer, q, po, pml, stream, out, full)
         : nt == 2 ? launch_one<2>(t, layer, q, po, pml, stream, out, full)
         : nt == 3 ? launch_one<3>(t, layer, q, po, pml, stream, out, full)
                   : launch_one<4>(t, layer, q, po, pml, stream, out, full);
}

}  // namespace

int attn_scaled_prepare() {
    int rc;
    if ((rc = prepare_one<1>()) != TF_OK || (rc = prepare_one<2>()) != TF_OK) return rc;
    if ((rc = prepare_one<3>()) != TF_OK || (rc = prepare_one<4>()) != TF_OK) return rc;
    return attn_scaled_tc_prepare();
}

int launch_attn_scaled(const SegTable& t, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
                       uint16_t* out, int full) {
    if (t.n_items_mma == t.n_items) return launch_mma(t, layer, q, po, pml, stream, out, full);
    if (t.n_items_mma > 0 && t.side) {   // both kinds of windows side by side, as over bf16 caches (attn.cu)
        cudaError_t e = cudaEventRecord(t.ev_fork, stream);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(t.side, t.ev_fork, 0);
        if (e != cudaSuccess) return cuda_fail(e);
        int rc = launch_attn_scaled_tc(t, layer, q, po, pml, stream, out, full, t.tc_grid_mixed);
        if (rc == TF_OK) rc = launch_mma(t, layer, q, po, pml, t.side, out, full);
        if (rc != TF_OK) return rc;
        e = cudaEventRecord(t.ev_join, t.side);
        if (e == cudaSuccess) e = cudaStreamWaitEvent(stream, t.ev_join, 0);
        return e == cudaSuccess ? TF_OK : cuda_fail(e);
    }
    if (t.n_items_mma > 0) {
        const int rc = launch_mma(t, layer, q, po, pml, stream, out, full);
        if (rc != TF_OK) return rc;
    }
    return launch_attn_scaled_tc(t, layer, q, po, pml, stream, out, full);
}

}  // namespace tf
