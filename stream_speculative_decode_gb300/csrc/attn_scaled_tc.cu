// Attention over scaled pools on the 5th-generation tensor cores: windows of 9 rows
// or more and prompt windows (attn_scaled.cu takes the narrower ones). Units,
// records and merges are those of attn_tc.cu, and so is the softmax with a thread a
// query row; what differs is what the codes ask for.
//
// With c the codes, ek and ev a block's exponents, E the chunk's largest ev and x the
// scores in log2 units:
//   x_t = (q . ck_t) * 2^ek * log2(e) / 8
//   o = 2^E * sum 2^(x_t - m + ev - E) cv_t / sum 2^(x_t - m)
// K's codes go into the MMA as they are (kind::f8f6f4): a query, under a power of two
// of its own that puts its largest at 2^7..2^8, is split into two e4m3 parts, its
// rounding and the rounding of the remainder. A bf16 value has 8 significant bits and
// the two parts 4 each, so together they are exact down to 2^-9 of the largest, and
// off by at most 2^-10 (2^-17 of the largest) below. K's scale is a factor of the
// softmax's 16 scores of a block, which costs it nothing but the factor. V's enters
// the weights that go into P.V, w = 2^(x - m + ev - E), as in attn_scaled.cu, and V's
// codes become fp16 tiles in shared memory as they are (exact): a key is rounded by what
// it adds to the output, and the sum l takes w * 2^(E - ev). (With the scales on V's
// tiles instead, a key of a small weight and a large scale would vanish from P.V.)
//
// Persistent, two CTAs an SM, 8 warps:
//   warp 7      TMA loads of the codes (64 keys: 4 KB of K, 64-byte swizzle, and 4 KB
//               of V) into a ring of 6 stages, each with its blocks' scales beside it;
//               at a unit's start its V scales, for E;
//   warps 5, 6  the conversion of the V tiles, half a tile each, ring of 3;
//   warp 4      both products' MMAs, and the queries' TMA loads;
//   warps 0-3   softmax and records; at a unit's start the queries' two parts, each
//               row by the thread that owns it.
// Tensor memory: S/P of tile j at columns 64 * (j % 2), O at 128, the queries' parts at
// 192. (An MMA of 64 keys that reads its 128 query rows from shared memory is bound by
// that: 4 KB of queries beside 2 KB of keys.)
//
// Measured: 64 windows of 16 rows at 16 to 32,768 keys 112 us (3.4 TB/s, 51 % of the
// measured copy rate); a 2,048-row prompt chunk at 8,179 keys 181 us (664 TFLOP/s). With
// V's scales on its tiles, which leaves out the keys named above, 110.5 and 176 us.
// What bounds it is the chain of a tile, no unit by itself: a 64-key tile is 8 KB
// from HBM, 350 cycles of an SM's share, and the tensor cores take some 270 (M = 128
// whatever the window's rows), but from weights to weights two tiles on it is P.V's
// issue (265), its completion (400), q.K's issue (240), the scores (250) and the
// softmax (750, with 32 query rows a warp 1,050), for each of two CTAs. A unit's
// beginning and end are 8,500 cycles, and the tail of some 900 units of up to 128 tiles
// on 304 CTAs is 15 % (chunks of half the keys: 125 against 123 us). Copies of the
// kernel without the exponentials: 104 and 137 us; without V's conversion 104 and 172.
//
// Tried and slower: K converted to fp16 as well, by the load warp (212 us for the 64
// windows); queries in shared memory with a third S buffer in their place (117 and
// 185); weights in columns of their own, so that q.K need not wait for P.V (120 and
// 196; with P.V in a warp of its own, which leaves 96 registers a thread, 144 and
// 211); a quarter of the exponentials as polynomials (125 and 213); the second half
// of a tile's scores loaded ahead (111 and 189 against 111 and 184).
//
// A weight w is at most 2^15 (fp16), the largest of a row at 2^6 when its reference
// moves: it is off by 2^-11 of itself, or by 2^-31 of the row's largest where that is
// more (those below vanish). A block of V whose scale is more than 2^64 below the
// chunk's largest counts as if it were 2^64 below.
//
// A NaN code of V must not reach the rows that do not see its key (0 * NaN): in tiles
// that reach past the first row's keys the converters write 0 for it and note, for
// each dimension, the first such key; a row that sees it gets the NaN when it is
// stored. Slots past the chunk's keys are zeroed.
//
// Waits are bounded as in attn_tc.cu.
#include "tc_ptx.cuh"
#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kStages = 6;
constexpr int kRawB = kKT * TF_D;           // 4 KB: the codes of a K or V tile
constexpr int kStageB = 2 * kRawB;          // K then V
constexpr int kTileB = kKT * TF_D * 2;      // 8 KB: a tile in fp16
constexpr int kBuf = 2;                     // S/P buffers: tile j uses buffer j % 2
constexpr int kVBuf = 3;                    // V buffers
constexpr int kDone = kVBuf + 1;            // the P.Vs' barriers: none comes round while its V buffer is waited for
constexpr int kThreads = 256;
constexpr uint32_t kCols = 256;
constexpr uint32_t kColS = 0;               // + 64 * (tile % 2)
constexpr uint32_t kColO = 128;             // 64 columns
constexpr uint32_t kColQ = 192;             // 32 columns: dimensions 0-31 (8 columns a part), then 32-63
constexpr float kLog2e8 = 0.18033688011112042f;
constexpr float kSumMax = 32768.f;          // a thread's weights of a tile adding up to more move the row's reference
constexpr float kHeadroom = 6.f;            // log2 of the largest weight after that
constexpr int kMaxShift = 64;
constexpr int kBlocks = 512 * TF_MAX_ROWS / TF_SCALE_KEYS;   // blocks of the longest chunk
constexpr int kScaleRing = 16;              // tiles whose scales are kept
constexpr int kUnits = 8;                   // units whose notes are kept (no role is that far ahead of another)
constexpr int kUQConsumers = 7;             // the MMA thread, 2 V converter warps, 4 softmax warps

struct Bars {
    uint64_t raw_full[kStages];
    uint64_t v_read[kStages];    // both V converters have read the stage
    uint64_t k_free[kStages];    // its q.K completed (softmax warp 0 has seen the scores)
    uint64_t v_ready[kVBuf];
    uint64_t s_full[kBuf];
    uint64_t p_full[kBuf];       // by tile % 2, though the weights have one place
    uint64_t o_done[kDone];      // P.V completed, by tile % kDone
    uint64_t q_full;             // the unit's queries landed (one phase a unit)
    uint64_t q_ready;            // and are in their two parts
    uint64_t uq_full[kUQ];
    uint64_t uq_empty[kUQ];
    int32_t uq[kUQ];
    Unit next[kUQ];              // the unit uq[], when there is one
    uint64_t grp;
    uint64_t drain;              // the MMAs in flight (drained at the end)
    uint32_t tmem_base;
    WaitCtl wc;
    int32_t last;
    int32_t top[kUnits];                     // a unit's E, as a scale byte
    int32_t any_nan[kUnits];
    int32_t nan_key[kUnits][TF_D];           // first key (of the chunk) with a NaN code taken out, by dimension
    float4 scale[kScaleRing][4];             // by running tile, a block each: K's scale, ev - E, 2^(E - ev)
    alignas(16) uint32_t block[kBlocks];     // warp 7: where the unit's blocks lie in the pools, and their scale bytes
    alignas(16) uint8_t k_byte[kBlocks];
    alignas(16) uint8_t v_byte[kBlocks];
};
constexpr int kVOff = kQB, kRawOff = kVOff + kVBuf * kTileB;
constexpr int kBarsOff = kRawOff + kStages * kStageB;
constexpr int kSmemBytes = 1024 + kBarsOff + int(sizeof(Bars));
static_assert(kSmemBytes <= 113 * 1024, "two CTAs an SM");

// Instruction descriptors (attn_tc.cu): fp32 sums, M = 128, N = 64; format 0 is e4m3 for
// kind::f8f6f4 (q.K) and fp16 for kind::f16 (P.V, V MN-major).
constexpr uint32_t kIdescQK = (1u << 4) | (uint32_t(64 >> 3) << 17) | (uint32_t(128 >> 4) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// sdesc's descriptor for K-major tiles of 64-byte rows under the 64-byte swizzle (layout
// 4): groups of 8 rows 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc64(uint32_t addr) {
    uint64_t d = uint64_t((addr >> 4) & 0x3FFFu);
    d |= uint64_t(1) << 16;
    d |= uint64_t(512 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(4) << 61;
    return d;
}
// Bounded waits by a whole warp, with one outcome for its lanes. The clock is looked at
// every kTests tests only: reading %globaltimer takes longer than most waits here, and a
// chain of waits is what a tile's time is.
constexpr int kTests = 32;
__device__ __noinline__ bool wait_long(uint32_t a, uint32_t parity, volatile WaitCtl* wc) {
    unsigned long long t0 = 0;
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < kTests; ++i)
            if (__all_sync(0xFFFFFFFFu, mbar_test(a, parity))) return true;
        if (__any_sync(0xFFFFFFFFu, wc->flag != 0)) return false;
        const unsigned long long now = gtime();
        if (t0 == 0) t0 = now;
        if (now - t0 > wc->limit_ns) wc->flag = 1;
    }
}
__device__ __forceinline__ bool wait_warp(uint32_t a, uint32_t parity, volatile WaitCtl* wc) {
    return __all_sync(0xFFFFFFFFu, mbar_test(a, parity)) || wait_long(a, parity, wc);
}
// Two barriers at once: every lane tests one of them.
__device__ __forceinline__ bool wait_both(uint32_t a, uint32_t pa, uint32_t b, uint32_t pb, volatile WaitCtl* wc) {
    const bool odd = threadIdx.x & 1;
    return wait_warp(odd ? b : a, odd ? pb : pa, wc);
}
// One lane of a converged warp, the same every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
// A place in a ring of N barriers and the parity of its current use. A wait for the
// use before it (parity ^ 1) passes at once in the first round.
template <int N>
struct Ring {
    int i = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            parity ^= 1u;
        }
    }
};
__device__ __forceinline__ void tc_mma_ts_f8(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}"
                 ::"r"(d), "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
// What a block's scales make of a row's scores and weights: x = score * f + d, 2^-d = u.
struct BlockScale {
    float f, d, u;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t scale, float cq) {
    const uint4 s = lds128(scale);   // f is never 0: masked scores are -inf
    return {fmaf(cq, __uint_as_float(s.x), 0x1p-149f), __uint_as_float(s.y), __uint_as_float(s.z)};
}

// Weights 2^(v * f + d - mu) of a thread's scores, 16 of a block, packed to fp16 pairs.
// Returns their sum, and adds theirs without V's scales to l. mu = 0 stands for a
// reference of -inf.
template <int NV>
__device__ __forceinline__ float weigh(const float (&v)[NV], uint32_t scale, float cq, float mref,
                                       uint32_t (&own)[NV / 2], float& l) {
    const float mu = (mref == -INFINITY) ? 0.f : mref;
    float all = 0.f;
#pragma unroll
    for (int b = 0; b < NV / 16; ++b) {
        const BlockScale s = block_scale(scale + 16 * b, cq);
        const float at = s.d - mu;
        const uint64_t f2 = f2pack(s.f, s.f), at2 = f2pack(at, at);
        uint64_t sum2[2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = 8 * b + i;
            float x0, x1;
            f2unpack(ffma2(f2pack(v[2 * c], v[2 * c + 1]), f2, at2), x0, x1);
            const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
            sum2[i & 1] = i < 2 ? f2pack(p0, p1) : fadd2(sum2[i & 1], f2pack(p0, p1));
            own[c] = pack_h2(p0, p1);
        }
        float s0, s1;
        f2unpack(fadd2(sum2[0], sum2[1]), s0, s1);
        all += s0 + s1;
        l = fmaf(s0 + s1, s.u, l);
    }
    return all;
}

// State of one softmax thread for one unit; rows and lanes as in attn_tc.cu (windows
// of at most 16 rows run dual: lanes L and L + 16 of a quadrant share a query, each
// with its half of a tile's keys).
struct SoftState {
    Bars* bars;
    volatile WaitCtl* abortp;
    uint32_t trow;
    int g0, T, lim, lim_all;
    bool wact;
    float cq;     // factor of the row's scores, but for K's scales
    float mref;
    float l;
};

template <bool DUAL>
__device__ __forceinline__ void softmax_tiles(SoftState& st) {
    const int lane = threadIdx.x & 31;
    const int half = DUAL ? (lane >> 4) : 0;
    constexpr int NB = DUAL ? 2 : 4;   // blocks, and halves of a tile, that a thread scores
    constexpr int NH = NB / 2;
    Bars* bars = st.bars;
    for (int j = 0; j < st.T; ++j) {
        const int gj = st.g0 + j;
        const int b = gj % kBuf;
        const uint32_t colS = kColS + 64 * b;
        if (!wait_warp(su32(&bars->s_full[b]), (gj / kBuf) & 1, st.abortp)) break;
        if (threadIdx.x == 0) mbar_arrive(su32(&bars->k_free[gj % kStages]));
        tc_fence_after();
        if (st.wact) {
            const uint32_t scale = su32(&bars->scale[gj % kScaleRing][half * NB]);
            const bool edge = j * kKT + kKT > st.lim_all;
            // 32 of the thread's scores, -inf past the row's last key
            auto load_scores = [&](int h, float (&v)[32]) {
                uint32_t r[32];
                if constexpr (DUAL)
                    tc_ld16x2_32<kKT / 2>(st.trow + colS, r);
                else
                    tc_ld_n<32>(st.trow + colS + 32 * h, r);
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
                if (edge) {
                    const int k0 = j * kKT + half * 32 + 32 * h;
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (k0 + c >= st.lim) v[c] = -INFINITY;
                }
            };
            // the tile's weights, kept in registers until all are there (P lies over S)
            uint32_t own[NH][16];
            float l;   // this tile's part of st.l
            auto weigh_tile = [&]() {
                float sum = 0.f;
                l = 0.f;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float v[32];
                    load_scores(h, v);
                    sum += weigh<32>(v, scale + 32 * h, st.cq, st.mref, own[h], l);
                }
                return sum;
            };
            const float psum = weigh_tile();
            // a weight is at most its tile's sum; a row that has no reference yet, or too
            // large a sum (or a NaN), takes the warp through the maxima, and moves its own
            // reference (which other rows have no say in)
            const bool slow = (st.mref == -INFINITY && st.lim > 0) || !(psum <= kSumMax);
            if (__any_sync(0xFFFFFFFFu, slow)) {
                float mx = -INFINITY;
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    float v[32];
                    load_scores(h, v);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float m2[2] = {v[16 * i], v[16 * i + 1]};
#pragma unroll
                        for (int c = 2; c < 14; c += 4) {
                            m2[0] = max3f(m2[0], v[16 * i + c], v[16 * i + c + 2]);
                            m2[1] = max3f(m2[1], v[16 * i + c + 1], v[16 * i + c + 3]);
                        }
                        m2[0] = fmaxf(m2[0], v[16 * i + 14]);
                        m2[1] = fmaxf(m2[1], v[16 * i + 15]);
                        const BlockScale s = block_scale(scale + 32 * h + 16 * i, st.cq);
                        mx = fmaxf(mx, fmaf(fmaxf(m2[0], m2[1]), s.f, s.d));
                    }
                }
                bool row_slow = slow;
                if (DUAL) {
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
                    row_slow |= __shfl_xor_sync(0xFFFFFFFFu, int(slow), 16) != 0;
                }
                const float to = mx - kHeadroom;
                const bool resc = row_slow && to > st.mref;
                if (__any_sync(0xFFFFFFFFu, resc)) {
                    if (j >= 1 && !wait_warp(su32(&bars->o_done[(gj - 1) % kDone]), ((gj - 1) / kDone) & 1, st.abortp))
                        break;
                    tc_fence_after();
                    const float alpha = resc ? ex2_approx(st.mref - to) : 1.f;
                    if (resc) {
                        st.mref = to;
                        st.l *= alpha;
                    }
                    if (j >= 1) {
#pragma unroll 1
                        for (int h = 0; h < (DUAL ? 2 : 4); ++h) {
                            uint32_t o16[16];
                            if constexpr (DUAL)
                                tc_ld16x2_16<32>(st.trow + kColO + 16 * h, o16);
                            else
                                tc_ld16(st.trow + kColO + 16 * h, o16);
                            tc_wait_ld();
#pragma unroll
                            for (int c = 0; c < 16; ++c) o16[c] = __float_as_uint(__uint_as_float(o16[c]) * alpha);
                            if constexpr (DUAL)
                                tc_st16x2_16<32>(st.trow + kColO + 16 * h, o16);
                            else
                                tc_st_n<16>(st.trow + kColO + 16 * h, o16);
                        }
                        tc_wait_st();
                    }
                }
                weigh_tile();
            }
            if constexpr (DUAL) {
                tc_st16x2_16<kKT / 4>(st.trow + colS, own[0]);
            } else {
                tc_st_n<16>(st.trow + colS, own[0]);
                tc_st_n<16>(st.trow + colS + 16, own[NH - 1]);
            }
            st.l += l;
            tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(su32(&bars->p_full[b]));
    }
}

// Two columns of the thread's lane; dual: threads 16-31 write those 16 columns on.
template <bool DUAL>
__device__ __forceinline__ void st_two(uint32_t taddr, uint32_t a, uint32_t b) {
    if constexpr (DUAL)
        asm volatile("tcgen05.st.sync.aligned.16x32bx2.x2.b32 [%0], 16, {%1,%2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(a), "r"(b) : "memory");
}
// The thread's query row (tensor memory lane 32 * warp + row of the tile) from bf16 to
// its two e4m3 parts in tensor memory, under the power of two that puts its largest at
// 2^7..2^8; returns the factor of its scores. Dual: two threads a row, 32 dimensions
// each. 8 columns hold 32 dimensions (an MMA's K) of a part.
// (Loops, here and where a unit ends, and not all of it straight code: what runs once a
// unit is fetched anew each time.)
template <bool DUAL>
__device__ __forceinline__ float convert_query(uint32_t sQ, uint32_t trow, int warp, int lane) {
    const int r = 32 * warp + (DUAL ? (lane & 15) : lane);
    constexpr int NP = DUAL ? 4 : 8;   // pieces of 8 dimensions
    const int p0 = DUAL ? (lane >> 4) * 4 : 0;
    uint32_t most = 0;
#pragma unroll 4
    for (int i = 0; i < NP; ++i) {
        const uint4 v = lds128(sQ + r * 128 + (((p0 + i) ^ (r & 7)) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            most = max(most, max(finite_bits(__uint_as_float(w[k] << 16)),
                                 finite_bits(__uint_as_float(w[k] & 0xFFFF0000u))));
    }
    if (DUAL) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 16));
    const int up = min(134 - int(most >> 23), 126);
    const float mul = __uint_as_float(uint32_t(127 + up) << 23);
#pragma unroll 4
    for (int i = 0; i < NP; ++i) {
        const uint4 v = lds128(sQ + r * 128 + (((p0 + i) ^ (r & 7)) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float y[4] = {__uint_as_float(w[2 * c] << 16) * mul, __uint_as_float(w[2 * c] & 0xFFFF0000u) * mul,
                                __uint_as_float(w[2 * c + 1] << 16) * mul,
                                __uint_as_float(w[2 * c + 1] & 0xFFFF0000u) * mul};
            hi[c] = e4m3_quad(y[0], y[1], y[2], y[3]);
            const float2 a = h2_to_f2(e4m3_low(hi[c])), b = h2_to_f2(e4m3_high(hi[c]));
            lo[c] = e4m3_quad(y[0] - a.x, y[1] - a.y, y[2] - b.x, y[3] - b.y);
        }
        // 32 dimensions: 8 columns of the first part, 8 of the second
        const uint32_t at = trow + kColQ + (i >> 2) * 16 + (i & 3) * 2;
        st_two<DUAL>(at, hi[0], hi[1]);
        st_two<DUAL>(at + 8, lo[0], lo[1]);
    }
    tc_wait_st();
    return __uint_as_float(uint32_t(127 - up) << 23) * kLog2e8;
}

// Where the 16 codes `p` (0..3) of key row r go in a fp16 tile (128-byte rows, 128-byte
// swizzle): two 16-byte pieces.
__device__ __forceinline__ void store_codes(uint32_t tile, int r, int p, const uint32_t (&h)[8]) {
    const uint32_t row = tile + r * 128;
    sts128(row + (((2 * p) ^ (r & 7)) << 4), make_uint4(h[0], h[1], h[2], h[3]));
    sts128(row + (((2 * p + 1) ^ (r & 7)) << 4), make_uint4(h[4], h[5], h[6], h[7]));
}

// The m-th unit that the load warp handed this CTA after its first (unit blockIdx.x); false
// where there is none, or the CTA gave up. Units travel through shared memory: looking one
// up in the table is two trips to L2, which every role would stand still for.
__device__ __forceinline__ bool next_unit(Bars* bars, int m, volatile WaitCtl* abortp, Unit& U) {
    const int slot = m % kUQ;
    const bool more = wait_warp(su32(&bars->uq_full[slot]), (m / kUQ) & 1, abortp) &&
                      reinterpret_cast<volatile int32_t*>(bars->uq)[slot] >= 0;
    if (more) U = bars->next[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(su32(&bars->uq_empty[slot]));
    return more;
}

__global__ void __launch_bounds__(kThreads, 2)
attn_scaled_tc_kernel(SegTable t, int layer, float* __restrict__ part_o, float2* __restrict__ part_ml,
                      uint16_t* __restrict__ out, int full, int n_units, const __grid_constant__ CUtensorMap qmap) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = su32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base, sV = base + kVOff, sRaw = base + kRawOff;
    Bars* bars = reinterpret_cast<Bars*>(gbase + kBarsOff);
    volatile WaitCtl* abortp = &bars->wc;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(su32(&bars->raw_full[s]), 1);
            mbar_init(su32(&bars->v_read[s]), 2);
            mbar_init(su32(&bars->k_free[s]), 1);
        }
        for (int b = 0; b < kBuf; ++b) {
            mbar_init(su32(&bars->s_full[b]), 1);
            mbar_init(su32(&bars->p_full[b]), 4);
        }
        for (int b = 0; b < kDone; ++b) mbar_init(su32(&bars->o_done[b]), 1);
        for (int b = 0; b < kVBuf; ++b) {
            mbar_init(su32(&bars->v_ready[b]), 2);
        }
        mbar_init(su32(&bars->q_full), 1);
        mbar_init(su32(&bars->q_ready), 4);
        for (int k = 0; k < kUQ; ++k) {
            mbar_init(su32(&bars->uq_full[k]), 1);
            mbar_init(su32(&bars->uq_empty[k]), kUQConsumers);
        }
        mbar_init(su32(&bars->grp), 128);
        mbar_init(su32(&bars->drain), 1);
        bars->wc.flag = t.wait_ns == 0;   // a limit of 0: what does not complete at once is given up
        bars->wc.limit_ns = t.wait_ns;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int i = tid; i < kUnits * TF_D; i += kThreads) (&bars->nan_key[0][0])[i] = INT32_MAX;
    if (tid < kUnits) bars->any_nan[tid] = 0;
    pdl_wait();   // the table above; queries and caches below
    if (warp == 4) tc_alloc(su32(&bars->tmem_base), kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;

    if (warp == 4) {
        // ------------------------------------------------------------ MMAs
        // P.V of tile j, then the q.K of tile j + 2, which takes over its S buffer. The whole
        // warp walks the loop and one lane of it issues: with the control flow the warp's,
        // addresses and descriptors stay in uniform registers (in a lone thread's code an
        // MMA took some 70 cycles to issue, and everything else stands behind it). Even so an MMA
        // or a commit is 45 to 50 cycles and a wait that is already over some 100, so a product
        // has one commit, and two barriers are waited for at once.
        Ring<kStages> kr;   // the stage of the next q.K
        Ring<kVBuf> vr;     // the V buffer of the next P.V
        uint32_t qs = 0, ps = 0;   // their S buffers' uses so far: buffer & 1, parity >> 1
        const uint64_t dk0 = sdesc64(sRaw), dv0 = sdesc(sV, kTileB, 1024);
        bool ok = true;
        Unit U = unit_of<true>(t, layer, blockIdx.x);
        if (elect_one()) issue_q(sQ, &qmap, U, su32(&bars->q_full));
        int q_issued = 1;
        bool more = true;
        for (int n = 0; more && ok; ++n) {
            const int T = U.T;
            auto qk = [&]() {
                const uint32_t b = qs & 1;
                const uint32_t raw = su32(&bars->raw_full[kr.i]), last = qs - kBuf;   // the S buffer's last tile
                if (!(qs < kBuf ? wait_warp(raw, kr.parity, abortp)
                                : wait_both(raw, kr.parity, su32(&bars->o_done[last % kDone]), last / kDone & 1,
                                            abortp)))
                    return false;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dk = dk0 + uint32_t(kr.i) * (kStageB >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)   // both parts, K = 64 in 2 steps of 32 bytes each
                        tc_mma_ts_f8(tmem + kColS + 64 * b, tmem + kColQ + 8 * k, dk + 2 * (k >> 1), kIdescQK,
                                     k > 0 ? 1u : 0u);
                    tc_commit(su32(&bars->s_full[b]));
                }
                __syncwarp();
                kr.next();
                ++qs;
                return true;
            };
            ok = wait_warp(su32(&bars->q_ready), n & 1, abortp);
            if (!ok) break;
            tc_fence_after();
            ok = qk() && (T < 2 || qk());
            bool entered = false;   // the next unit is known, its queries on their way
            auto enter_next = [&]() {
                entered = true;
                more = next_unit(bars, n, abortp, U);
                // the bf16 tile of the queries has been free since q_ready
                if (more && elect_one()) issue_q(sQ, &qmap, U, su32(&bars->q_full));
                __syncwarp();
                q_issued += more;
            };
            for (int j = 0; j < T && ok; ++j) {
                const uint32_t b = ps & 1;
                ok = wait_both(su32(&bars->p_full[b]), ps >> 1 & 1, su32(&bars->v_ready[vr.i]), vr.parity, abortp);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t dv = dv0 + uint32_t(vr.i) * (kTileB >> 4);
#pragma unroll
                    for (int k = 0; k < kKT / 16; ++k)
                        tc_mma_ts(tmem + kColO, tmem + kColS + 64 * b + 8 * k, dv + 128 * k, kIdescPV,
                                  (j > 0 || k > 0) ? 1u : 0u);
                    tc_commit(su32(&bars->o_done[ps % kDone]));
                }
                __syncwarp();
                vr.next();
                ++ps;
                if (j + 2 < T)
                    ok = qk();
                else if (!entered && __all_sync(0xFFFFFFFFu, mbar_test(su32(&bars->uq_full[n % kUQ]), n / kUQ & 1)))
                    enter_next();
            }
            if (ok && !entered) enter_next();
        }
        if (elect_one()) {
            tc_commit(su32(&bars->drain));
            mbar_drain(su32(&bars->drain), 0);
            mbar_drain(su32(&bars->q_full), (q_issued - 1) & 1);   // the last query load has landed
        }
        __syncwarp();
    } else if (warp == 7) {
        // ------------------------------------------------------------ loads, scales
        const uint64_t once = l2_evict_first();
        const uint8_t *const ks = t.k_scale[layer], *const vs = t.v_scale[layer];
        Ring<kStages> r;
        Ring<kUQ> ur;
        int gt = 0;
        bool ok = true;
        Unit U = unit_of<true>(t, layer, blockIdx.x);
        for (int u = blockIdx.x, m = 0; u >= 0 && ok; ++m) {
            const int nblocks = (min(U.st.chunk_keys, U.st.keys - U.c0) + TF_SCALE_KEYS - 1) / TF_SCALE_KEYS;
            const int bs = t.page_shift - 4;
            uint32_t top = 0;
            for (int i = lane; i < 4 * U.T; i += 32) {   // slots past the chunk: any K scale, no V
                const uint32_t at = ((uint32_t(__ldg(t.pages + U.pages + (i >> bs))) * TF_NKV + U.g) << bs) +
                                    (i & ((1 << bs) - 1));
                bars->block[i] = at;
                const uint32_t e = i < nblocks ? uint32_t(__ldg(vs + at)) : 0u;
                bars->k_byte[i] = __ldg(ks + at);
                bars->v_byte[i] = uint8_t(e);
                top = max(top, e);
            }
            top = __reduce_max_sync(0xFFFFFFFFu, top);
            if (lane == 0) bars->top[m % kUnits] = int32_t(top);
            __syncwarp();
            for (int j = 0; j < U.T; ++j, ++gt) {
                const int s = r.i;
                if (!wait_both(su32(&bars->v_read[s]), r.parity ^ 1u, su32(&bars->k_free[s]), r.parity ^ 1u,
                               abortp)) {
                    ok = false;
                    break;
                }
                r.next();
                if (lane < 4) {
                    const int down = min(int(top) - int(bars->v_byte[4 * j + lane]), kMaxShift);
                    bars->scale[gt % kScaleRing][lane] =
                        make_float4(scale_value(bars->k_byte[4 * j + lane]), float(-down),
                                    __uint_as_float(uint32_t(127 + down) << 23), 0.f);
                }
                __syncwarp();
                if (lane == 0) {
                    const uint32_t bar = su32(&bars->raw_full[s]);
                    mbar_expect_tx(bar, kStageB);
                    // a box is 64 keys of a head, or the whole of a smaller page
                    for (int i = 0; i < 4; i += bs >= 2 ? 4 : 1 << bs) {
                        const uint32_t at = bars->block[4 * j + i];
                        const int head = int(at >> bs), row = int(at & ((1u << bs) - 1u)) * TF_SCALE_KEYS;
                        const uint32_t dst = sRaw + s * kStageB + i * (TF_SCALE_KEYS * TF_D);
                        tma_load_3d_hint(dst, U.kmap, 0, row, head, bar, once);
                        tma_load_3d_hint(dst + kRawB, U.vmap, 0, row, head, bar, once);
                    }
                }
            }
            if (!ok) break;
            // the next unit of the launch, for this CTA's roles
            int un = 0;
            if (lane == 0) un = int(gridDim.x) + atomicAdd(&t.tc_work[2 * layer], 1);
            un = __shfl_sync(0xFFFFFFFFu, un, 0);
            if (un >= n_units) un = -1;
            if (un >= 0) U = unit_of<true>(t, layer, un);
            if (!wait_warp(su32(&bars->uq_empty[ur.i]), ur.parity ^ 1u, abortp)) break;
            if (lane == 0) {
                bars->uq[ur.i] = un;
                bars->next[ur.i] = U;
                mbar_arrive(su32(&bars->uq_full[ur.i]));
            }
            ur.next();
            __syncwarp();
            u = un;
        }
        if (abortp->flag && lane == 0)   // let the copies in flight land before the CTA exits
            for (int k = gt > kStages ? gt - kStages : 0; k < gt; ++k)
                mbar_drain(su32(&bars->raw_full[k % kStages]), (k / kStages) & 1);
        __syncwarp();
    } else if (warp == 5 || warp == 6) {
        // ------------------------------------------------------------ V tiles, rows 32 * (warp - 5) ..
        const int r0 = 32 * (warp - 5);
        Ring<kStages> r;
        Ring<kVBuf> vr;
        int gt = 0;
        bool ok = true, more = true;
        Unit U = unit_of<true>(t, layer, blockIdx.x);
        for (int m = 0; more && ok; ++m) {
            const int nkeys = min(U.st.chunk_keys, U.st.keys - U.c0);
            const int lim_all = min((full ? U.st.keys : U.st.keys - U.st.rows + 1) - U.c0, nkeys);
            for (int j = 0; j < U.T; ++j, ++gt) {
                const int s = r.i, b = vr.i;
                if (!wait_warp(su32(&bars->raw_full[s]), r.parity, abortp)) {
                    ok = false;
                    break;
                }
                r.next();
                const uint32_t src = sRaw + s * kStageB + kRawB + r0 * TF_D + uint32_t(lane) * 16u;
                uint4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = lds128(src + i * 512);
                __syncwarp();
                if (lane == 0) mbar_arrive(su32(&bars->v_read[s]));
                if (j * kKT + r0 + 32 > lim_all) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = j * kKT + r0 + 8 * i + (lane >> 2);
                        uint32_t* w = &v[i].x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (key >= nkeys) w[k] = 0u;
                            const uint32_t bad = __vcmpeq4(w[k] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                            if (bad) {
                                for (int c = 0; c < 4; ++c)
                                    if (bad >> (8 * c) & 1)
                                        atomicMin(&bars->nan_key[m % kUnits][16 * (lane & 3) + 4 * k + c], key);
                                bars->any_nan[m % kUnits] = 1;
                                w[k] &= ~bad;
                            }
                        }
                    }
                }
                const int last = gt - kVBuf;   // the V buffer's last tile
                if (last >= 0 && !wait_warp(su32(&bars->o_done[last % kDone]), (last / kDone) & 1, abortp)) {
                    ok = false;
                    break;
                }
                vr.next();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t o[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        o[2 * k] = e4m3_low(w[k]);
                        o[2 * k + 1] = e4m3_high(w[k]);
                    }
                    store_codes(sV + b * kTileB, r0 + 8 * i + (lane >> 2), lane & 3, o);
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(su32(&bars->v_ready[b]));
            }
            if (ok) more = next_unit(bars, m, abortp, U);
        }
    } else {
        // ------------------------------------------------------------ softmax + records
        int gt = 0, gph = 0;
        const uint32_t trow = tmem + (uint32_t(warp * 32) << 16);
        bool more = true;
        Unit U = unit_of<true>(t, layer, blockIdx.x);
        for (int m = 0; more; ++m) {
            const SegStream& st = U.st;
            const int nq = st.rows * 4, per = q_per(st.rows);
            const bool dual = per == 16;
            const int ql = dual ? (lane & 15) : lane;
            const int qi = per * warp + ql;
            const bool qvalid = qi < nq;
            const bool wact = per * warp < nq;
            const int mode = out ? st.merge_mode : kMergeKernel;
            SoftState ss;
            ss.bars = bars;
            ss.abortp = abortp;
            ss.trow = trow;
            ss.g0 = gt;
            ss.T = U.T;
            ss.lim = qvalid ? (full ? st.keys : st.keys - st.rows + (qi >> 2) + 1) - U.c0 : 0;
            ss.lim_all = (full ? st.keys : st.keys - st.rows + 1) - U.c0;
            ss.wact = wact;
            ss.cq = 0.f;
            ss.mref = -INFINITY;
            ss.l = 0.f;
            if (wait_warp(su32(&bars->q_full), m & 1, abortp))
                ss.cq = dual ? convert_query<true>(sQ, trow, warp, lane) : convert_query<false>(sQ, trow, warp, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(su32(&bars->q_ready));
            if (dual)
                softmax_tiles<true>(ss);
            else
                softmax_tiles<false>(ss);
            gt += U.T;
            if (!abortp->flag) wait_warp(su32(&bars->o_done[(gt - 1) % kDone]), ((gt - 1) / kDone) & 1, abortp);
            tc_fence_after();
            const bool aborted = abortp->flag != 0;
            const volatile int32_t* const nan_key = bars->nan_key[m % kUnits];
            const bool any_nan = reinterpret_cast<volatile int32_t*>(bars->any_nan)[m % kUnits] != 0;
            if (wact) {
                // (m, l, O) relative to the row's reference -> the chunk's record, O in units of 2^E
                const int e = reinterpret_cast<volatile int32_t*>(bars->top)[m % kUnits] - kScaleBias;
                const float up0 = __uint_as_float(uint32_t(127 + e / 2) << 23);
                const float up1 = __uint_as_float(uint32_t(127 + e - e / 2) << 23);
                float lsum = ss.l;
                if (dual) lsum += __shfl_xor_sync(0xFFFFFFFFu, lsum, 16);
                const int d0 = dual ? 32 * (lane >> 4) : 0, n16 = dual ? 2 : 4;
                const bool direct = mode == kMergeDirect, empty = ss.mref == -INFINITY && !(lsum != lsum);
                const int64_t rec = st.pbase + (int64_t(U.chunk) * TF_NKV + U.g) * nq + qi;
                float up = up0;   // of an output: / l
                if (direct) up *= 1.f / lsum;
                if (aborted) up = NAN;
                if (!direct && empty) up = 0.f;
#pragma unroll 1
                for (int i = 0; i < n16; ++i) {
                    uint32_t ro[16];
                    if (dual)
                        tc_ld16x2_16<32>(trow + kColO + 16 * i, ro);
                    else
                        tc_ld16(trow + kColO + 16 * i, ro);
                    tc_wait_ld();
                    const int d = d0 + 16 * i;
                    if (any_nan) {
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if (nan_key[d + c] < ss.lim) ro[c] = 0x7FC00000u;
                    }
                    if (qvalid) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float4 v = make_float4(
                                __uint_as_float(ro[4 * c]) * up * up1, __uint_as_float(ro[4 * c + 1]) * up * up1,
                                __uint_as_float(ro[4 * c + 2]) * up * up1, __uint_as_float(ro[4 * c + 3]) * up * up1);
                            if (direct)
                                store_out4(out_row(out, st, U.g, qi) + d + 4 * c, v);
                            else
                                *reinterpret_cast<float4*>(part_o + rec * TF_D + d + 4 * c) = v;
                        }
                    }
                    __syncwarp();
                }
                if (qvalid && !direct && d0 == 0) {   // a sum that is no number must not pass for none in a merge
                    const bool lost = aborted || !(lsum <= 3e38f);
                    const float m = ss.mref > -INFINITY ? ss.mref : lost ? 0.f : -INFINITY;
                    part_ml[rec] = make_float2(aborted ? NAN : m, lost ? INFINITY : empty ? 0.f : lsum);
                }
            }
            tc_fence_before();
            if (any_nan && group_sync(bars, gph, abortp)) {   // every warp has read the unit's notes
                if (warp == 0) {
                    bars->nan_key[m % kUnits][lane] = INT32_MAX;
                    bars->nan_key[m % kUnits][32 + lane] = INT32_MAX;
                    if (lane == 0) bars->any_nan[m % kUnits] = 0;
                }
            }
            if (mode == kMergeLastCta) {
                __threadfence();
                if (group_sync(bars, gph, abortp)) {
                    int* ctr = t.counters + (size_t(layer) * t.S + U.stream) * TF_NKV + U.g;
                    if (tid == 0) bars->last = atomicAdd(ctr, 1) == st.n_chunks - 1;
                    if (group_sync(bars, gph, abortp) && bars->last) {
                        __threadfence();
                        merge_stream_head<2, 4>(st, U.g, part_o, part_ml, out, tid, 128);
                        if (tid == 0) atomicExch(ctr, 0);
                    }
                }
            }
            more = next_unit(bars, m, abortp, U);
        }
    }
    tc_fence_before();
    __syncthreads();   // every role is done
    tc_fence_after();
    if (tid == 0) {
        if (abortp->flag) atomicOr(t.status, uint32_t(TF_STATUS_ATTN_TIMEOUT));
        __threadfence();
        if (atomicAdd(&t.tc_work[2 * layer + 1], 1) == int(gridDim.x) - 1) {   // the last CTA resets the work counters
            atomicExch(&t.tc_work[2 * layer], 0);
            atomicExch(&t.tc_work[2 * layer + 1], 0);
        }
    }
    pdl_trigger();
    if (warp == 4) {
        tc_fence_after();
        tc_dealloc(tmem, kCols);
    }
}

}  // namespace

int attn_scaled_tc_prepare() {
    const cudaError_t e =
        cudaFuncSetAttribute(attn_scaled_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return e == cudaSuccess ? TF_OK : cuda_fail(e);
}

int launch_attn_scaled_tc(const SegTable& t0, int layer, const uint16_t* q, float* po, float2* pml, cudaStream_t stream,
                          uint16_t* out, int full, int grid_cap) {
    if (!t0.k_maps || !t0.v_maps) return TF_EINVAL;
    SegTable t = t0;
    t.wait_ns = wait_limit_ns();
    const int n_units = (t.n_items - t.n_items_mma) * TF_NKV;
    const int slots = grid_cap > 0 ? grid_cap : 2 * sm_count();
    const int grid = n_units < slots ? n_units : slots;
    CUtensorMap qmap;
    if (!encode_q_map(&qmap, q, t.R)) return cuda_fail(cudaErrorInvalidValue);
    return launch_pdl(attn_scaled_tc_kernel, dim3(grid), dim3(kThreads), kSmemBytes, stream, t, layer, po, pml, out, full,
                      n_units, qmap);
}

}  // namespace tf
