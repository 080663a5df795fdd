// Rows times a matrix of 4-bit weights with a scale for each 32 inputs
// (tf_linear_rows): a round's projections and its logits.
//
//   y[r][n] = s[n] * sum_k x[r][k] * g[n][k / 32] * (c[n][k] - 8)
// c the 4-bit codes, g e4m3, s and the sum in fp32, y rounded once to bf16; x is
// bf16, or e4m3 codes under a power of two for each 32 inputs (what tf_norm_rows
// writes). A product (c - 8) * g has at most 8 significant bits and a code of x
// times its power of two at most 4: both are exact in bf16, so the products run
// on bf16 MMAs with fp32 sums and nothing is rounded before the store.
//
// For few rows 17/32 bytes a weight have to be read, whatever the rows' number.
// mma.sync m16n8k16 with 16 outputs by 8 rows a tile: the weights are the operand
// whose fragments come straight from memory, 32 codes of one row and scale (16
// bytes) a lane, four lanes a row's 128 inputs; the order of the inputs in an MMA is
// free as long as x has the same. A nibble becomes 128 + c in bf16 by masks
// (0x4300 | c), and one bf16 FMA (128 + c) * g - 136 * g gives the weight.
//
// x lies in shared memory in the order in which the fragments want it (a row's 8
// inputs 8 w .. 8 w + 7 of a group as 0 4 1 5 2 6 3 7, the groups of a 128-input
// chunk side by side), staged once a CTA where it fits. One CTA of 16 warps an
// SM with a run of 16-output tiles, whose inputs the warps share out evenly.
//
// Measured, 128,000 outputs by 2,048 inputs (139 MB): 1 row 27.3 us, 16 rows 34.1
// us (5.1 and 4.2 TB/s; the same loads alone 21.5 us). What bounds it is the pipe that
// takes the codes apart, at half rate 56 of a chunk's 144 instructions: the warps wait
// for it and for one another's turn (54 % of the issue slots used), not for memory. That
// is paid again for every 32 rows: 32 rows 52 us, 64 96, 1,024 1,700 (316 TFLOP/s; the
// products alone would take 283 at the cuBLAS rate), and 16,381 rows of 2,048 to 2,048
// outputs 461 (72): this is a kernel for few rows. Warps that share tiles and meet at
// each one's end (37.1 and 45.8), loads a chunk at a time into a ring in shared
// memory (47 and 80), into the registers just used (48.5 and 56) or with the scales'
// codes picked apart as they arrive (44 and 51) were slower.
#include <cuda_bf16.h>

#include <atomic>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 128;                 // inputs of a chunk: four groups, one a lane of a row
constexpr int kGroup = TF_SCALE_COLUMNS;
constexpr int kPair = 2;                    // chunks whose loads are in flight together (linear_rows_kernel)

struct Linear {
    const uint8_t* x;          // bf16 or codes
    const uint8_t* xs;         // scale bytes, or null: x is bf16
    const uint8_t* w;
    const uint8_t* g;
    const float* s;
    uint16_t* y;
    int64_t x_stride, y_stride;
    int R, K, N;
    int row_tiles;             // CTAs side by side that share the weights' tiles
    int slab;                  // chunks of x in shared memory at a time
    uint32_t nibbles;          // 0x000F000F: as a value that the compiler does not know it stays in a register, and
                               // masking and setting the exponent are one instruction (two constants make it two)
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t fma_bf2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ uint4 load_once(const uint8_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Bytes of a row of x in shared memory: 64 past a multiple of 128, so that two
// rows' pieces fall on different banks.
__host__ __device__ constexpr int row_bytes(int chunks) { return chunks * kChunk * 2 + 64; }

// 8 inputs as (0, 4), (1, 5), (2, 6), (3, 7): of codes with their scale, or of bf16.
__device__ __forceinline__ uint4 pairs_of(uint2 c, float e) {
    const float2 p = h2_to_f2(e4m3_low(c.x)), q = h2_to_f2(e4m3_high(c.x));
    const float2 s = h2_to_f2(e4m3_low(c.y)), t = h2_to_f2(e4m3_high(c.y));
    return make_uint4(pack_bf2(p.x * e, s.x * e), pack_bf2(p.y * e, s.y * e), pack_bf2(q.x * e, t.x * e),
                      pack_bf2(q.y * e, t.y * e));
}
__device__ __forceinline__ uint4 pairs_of(const uint4& c) {
    return make_uint4(__byte_perm(c.x, c.z, 0x5410), __byte_perm(c.x, c.z, 0x7632), __byte_perm(c.y, c.w, 0x5410),
                      __byte_perm(c.y, c.w, 0x7632));
}

// Rows [r0, r0 + 8 NT) and chunks [c0, c0 + n) of x into shared memory, in units of 8
// inputs, kFly of them a thread in flight together.
template <int NT, bool kCodes>
__device__ __forceinline__ void stage_as(const Linear& a, int r0, int c0, int n, unsigned char* sx, int rowb) {
    // (bf16 units one by one, which the compiler unrolls; a code's scale would be waited for before the next one's is
    // asked for: 16 rows of 2,048 to few outputs, 4.8 us, four together 5.2; codes 5.5, one by one 6.2)
    constexpr int kFly = kCodes ? 4 : 1;
    const int units = n * kChunk / 8, total = 8 * NT * units;
    // i / units as a product: (i / 16) / n, exact for i / 16 up to 32 n and n up to 180
    const uint32_t inverse = ((1u << 20) + n - 1) / n;
    for (int i0 = threadIdx.x; i0 < total; i0 += kFly * kThreads) {
        uint4 v[kFly];
        uint8_t e[kFly];
        int to[kFly];
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            const int i = i0 + j * kThreads, r = int((uint32_t(i >> 4) * inverse) >> 20), u = i - r * units;
            const int k = c0 * kChunk + u * 8;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            e[j] = 127;
            to[j] = r * rowb + (u >> 4) * 256 + (u & 3) * 64 + ((u >> 2) & 3) * 16;
            if (i < total && r0 + r < a.R && k < a.K) {
                const int64_t at = int64_t(r0 + r) * a.x_stride + k;
                if constexpr (kCodes) {
                    const uint2 c = *reinterpret_cast<const uint2*>(a.x + at);
                    v[j].x = c.x;
                    v[j].y = c.y;
                    e[j] = a.xs[int64_t(r0 + r) * (a.K / kGroup) + k / kGroup];
                } else {
                    v[j] = *reinterpret_cast<const uint4*>(a.x + 2 * at);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kFly; ++j) {
            if (i0 + j * kThreads >= total) break;
            uint4 o;
            if constexpr (kCodes)
                o = pairs_of(make_uint2(v[j].x, v[j].y), scale_value(e[j]));
            else
                o = pairs_of(v[j]);
            *reinterpret_cast<uint4*>(sx + to[j]) = o;
        }
    }
}
template <int NT>
__device__ __forceinline__ void stage(const Linear& a, int r0, int c0, int n, unsigned char* sx, int rowb) {
    if (a.xs)
        stage_as<NT, true>(a, r0, c0, n, sx, rowb);
    else
        stage_as<NT, false>(a, r0, c0, n, sx, rowb);
}

// A lane's weights of one chunk of its two outputs, and the scales (kWords: the
// chunk's four codes of an output as a word; otherwise the lane's own code).
struct Piece {
    uint4 w[2];
    uint32_t g[2];
};

// Where a warp's lanes read: the rows of its tile's outputs.
struct Rows2 {
    const uint8_t* w[2];   // + 64 bytes a chunk
    const uint8_t* g[2];   // + 4 codes a chunk
};
__device__ __forceinline__ Rows2 rows_of(const Linear& a, int tile, int g8, int t4) {
    Rows2 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // outputs past N read the last one's weights and are not stored
        const int64_t n = min(tile * 16 + 8 * i + g8, a.N - 1);
        r.w[i] = a.w + n * (a.K / 2) + t4 * 16;
        r.g[i] = a.g + n * (a.K / kGroup);
    }
    return r;
}
template <bool kWords>
__device__ __forceinline__ void load_piece(const Linear& a, const Rows2& r, int c, int chunk, int t4, Piece& p) {
    if (!kWords && chunk * 4 + t4 >= a.K / kGroup) {   // groups past the row's end: scale 0
        p.w[0] = p.w[1] = make_uint4(0u, 0u, 0u, 0u);
        p.g[0] = p.g[1] = 0u;
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        p.w[i] = load_once(r.w[i] + int64_t(c) * 64);
        // (volatile: the compiler would move a plain load to its use)
        if constexpr (kWords)
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(p.g[i]) : "l"(r.g[i] + c * 4));
        else
            asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(p.g[i]) : "l"(r.g[i] + c * 4 + t4));
    }
}

// One chunk's products: a lane's codes and scales of two outputs times x's fragments
// at xr (+ nt * 8 rows). Even and odd MMAs have accumulators of their own, so that
// they need not wait for one another.
template <int NT, bool kWords>
__device__ __forceinline__ void multiply(const Piece& p, const unsigned char* xr, int rowb, uint32_t sel,
                                         uint32_t nibbles, float (&acc)[NT][2][4]) {
    const float2 g = h2_to_f2(e4m3_low(__byte_perm(p.g[0], p.g[1], sel)));
    const uint32_t s0 = pack_bf2(g.x, g.x), s1 = pack_bf2(g.y, g.y);
    const uint32_t z0 = mul_bf2(s0, 0xC308C308u), z1 = mul_bf2(s1, 0xC308C308u);   // -136
    const uint32_t w0[4] = {p.w[0].x, p.w[0].y, p.w[0].z, p.w[0].w};
    const uint32_t w1[4] = {p.w[1].x, p.w[1].y, p.w[1].z, p.w[1].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint4 b[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) b[nt] = *reinterpret_cast<const uint4*>(xr + nt * 8 * rowb + k * 64);
        auto weights = [&](uint32_t w, int i, uint32_t s, uint32_t z) {
            return fma_bf2(((w >> (4 * i)) & nibbles) | 0x43004300u, s, z);
        };
        const uint32_t lo[4] = {weights(w0[k], 0, s0, z0), weights(w1[k], 0, s1, z1), weights(w0[k], 1, s0, z0),
                                weights(w1[k], 1, s1, z1)};
        const uint32_t hi[4] = {weights(w0[k], 2, s0, z0), weights(w1[k], 2, s1, z1), weights(w0[k], 3, s0, z0),
                                weights(w1[k], 3, s1, z1)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mma_bf16(acc[nt][0], lo, b[nt].x, b[nt].y);
            mma_bf16(acc[nt][1], hi, b[nt].z, b[nt].w);
        }
    }
}

// The S warps of a group (named barriers 1..) meet.
__device__ __forceinline__ void group_sync(int group, int S) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(S * 32) : "memory");
}

template <int NT>
__device__ __forceinline__ float4 tile_sum(const float (&acc)[NT][2][4], int nt) {
    const float (&v)[2][4] = acc[nt];
    return make_float4(v[0][0] + v[1][0], v[0][1] + v[1][1], v[0][2] + v[1][2], v[0][3] + v[1][3]);
}
__device__ __forceinline__ void add4(float4& v, const float4& u) {
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
}
// The scales of a lane's outputs n and n + 8.
__device__ __forceinline__ float2 load_scales(const Linear& a, int n) {
    return make_float2(__ldg(a.s + min(n, a.N - 1)), __ldg(a.s + min(n + 8, a.N - 1)));
}
// A lane's sums of rows r, r + 1 and outputs n, n + 8, scaled and stored.
__device__ __forceinline__ void store_sums(const Linear& a, int n, int r, const float2& sc, const float4& v) {
    const float d[4] = {v.x * sc.x, v.y * sc.x, v.z * sc.y, v.w * sc.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int nn = n + 8 * (e >> 1), rr = r + (e & 1);
        if (nn < a.N && rr < a.R) {
            const __nv_bfloat16 b = __float2bfloat16_rn(d[e]);
            a.y[int64_t(rr) * a.y_stride + nn] = *reinterpret_cast<const uint16_t*>(&b);
        }
    }
}

// A tile's end: the parts' sums added in order, scaled and stored.
template <int NT>
__device__ __forceinline__ void finish_tile(const Linear& a, int S, int tile, int tiles, int r0, int group, int part,
                                            const float (&acc)[NT][2][4], float4* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int n = tile * 16 + g8, r = r0 + 2 * t4;
    const float2 sc = load_scales(a, n);
    if (S == 1) {
        if (tile < tiles)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) store_sums(a, n, r + nt * 8, sc, tile_sum<NT>(acc, nt));
    } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            sums[(warp * NT + nt) * 32 + lane] = tile_sum<NT>(acc, nt);
        group_sync(group, S);
        if (tile < tiles)
            for (int nt = part; nt < NT; nt += S) {   // the parts' sums in order
                float4 v = sums[(group * S * NT + nt) * 32 + lane];
                for (int p = 1; p < S; ++p) add4(v, sums[((group * S + p) * NT + nt) * 32 + lane]);
                store_sums(a, n, r + nt * 8, sc, v);
            }
        group_sync(group, S);
    }
}

// The same with x in one slab, in steps of U chunks (the last one filled up with zeros). A CTA takes a run of
// tiles, its warps even parts of the run's steps, so that no warp waits for another
// before the end: a warp that begins inside a tile leaves its sums of it in shared
// memory, and the one that has the tile's beginning adds them in order. Two sets of
// registers take turns, one being multiplied while the other's loads are on their way.
template <int NT, int U, bool kWords>
__global__ void __launch_bounds__(kThreads, 1)
linear_steps_kernel(const __grid_constant__ Linear a, int) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int r0 = (blockIdx.x % a.row_tiles) * 8 * NT;
    const int cta = blockIdx.x / a.row_tiles, ctas = gridDim.x / a.row_tiles;
    const int tiles = (a.N + 15) / 16, chunks = a.slab, steps = chunks / U, rowb = row_bytes(chunks);
    const int tile0 = int(int64_t(tiles) * cta / ctas), run = (int(int64_t(tiles) * (cta + 1) / ctas) - tile0) * steps;
    auto begin = [&](int w) { return int(int64_t(run) * w / kWarps); };
    float4* const sums = reinterpret_cast<float4*>(smem + 8 * NT * rowb);   // [warp][NT][lane]
    const unsigned char* const x0 = smem + g8 * rowb + t4 * 16;
    const uint32_t sel = kWords ? uint32_t(t4 | (4 + t4) << 4) : 0x40u;   // the lane's scale codes of two outputs
    struct Set {
        Piece p[U];
    };
    int left = begin(warp + 1) - begin(warp), tile = tile0 + begin(warp) / steps, at = begin(warp) % steps;
    int l_left = left, l_tile = tile, l_at = at;   // what has not been asked for yet
    Rows2 rows = rows_of(a, min(tile, tiles - 1), g8, t4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        rows.w[i] += at * (U * 64);
        rows.g[i] += at * (U * 4);
    }
    auto load = [&](Set& set) {
        if (l_left == 0) return;
        --l_left;
#pragma unroll
        for (int j = 0; j < U; ++j) load_piece<kWords>(a, rows, j, l_at * U + j, t4, set.p[j]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rows.w[i] += U * 64;
            rows.g[i] += U * 4;
        }
        if (++l_at == steps) {
            l_at = 0;
            rows = rows_of(a, min(++l_tile, tiles - 1), g8, t4);
        }
    };
    pdl_wait();
    Set one, two;
    load(one);
    stage<NT>(a, r0, 0, chunks, smem, rowb);
    __syncthreads();
    bool joined = at != 0;   // the tile was begun by a warp before this one
    float2 sc = load_scales(a, tile * 16 + g8);   // (long before they are needed)
    float acc[NT][2][4] = {};
    auto leave = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sums[(warp * NT + nt) * 32 + lane] = tile_sum<NT>(acc, nt);
    };
    auto take = [&](const Set& set) {
#pragma unroll
        for (int j = 0; j < U; ++j) multiply<NT, kWords>(set.p[j], x0 + (at * U + j) * 256, rowb, sel, a.nibbles, acc);
        --left;
        if (++at == steps) {
            if (joined)
                leave();
            else
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    store_sums(a, tile * 16 + g8, r0 + nt * 8 + 2 * t4, sc, tile_sum<NT>(acc, nt));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[nt][e >> 2][e & 3] = 0.f;
            joined = false;
            at = 0;
            ++tile;
            sc = load_scales(a, tile * 16 + g8);
        }
    };
    while (left) {
        load(two);
        take(one);
        if (!left) break;
        load(one);
        take(two);
    }
    if (at != 0 && joined) leave();
    __syncthreads();
    if (at != 0 && !joined) {
        int need = steps - at;
        float4 v[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) v[nt] = tile_sum<NT>(acc, nt);
        for (int w = warp + 1; need > 0; ++w) {
            const int n = begin(w + 1) - begin(w);
            if (n == 0) continue;
            need -= n;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) add4(v[nt], sums[(w * NT + nt) * 32 + lane]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) store_sums(a, tile * 16 + g8, r0 + nt * 8 + 2 * t4, sc, v[nt]);
    }
    pdl_trigger();
}

// The same for more inputs than shared memory holds of 8 rows, which are staged a slab at
// a time: row tiles of 8 NT rows, S warps an output tile. Every warp goes through its
// tiles, the slabs of x and its part of a slab's chunks, two chunks at a time, with the
// next two's loads (those of its next tile among them) in flight.
template <int NT, bool kWords>
__global__ void __launch_bounds__(kThreads, 1)
linear_rows_kernel(const __grid_constant__ Linear a, int S) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int r0 = (blockIdx.x % a.row_tiles) * 8 * NT;
    const int per_cta = kWarps / S, group = warp / S, part = warp % S;
    const int first = (blockIdx.x / a.row_tiles) * per_cta, step = gridDim.x / a.row_tiles * per_cta;
    const int tiles = (a.N + 15) / 16, chunks = (a.K + kChunk - 1) / kChunk;
    const int rowb = row_bytes(min(a.slab, chunks));
    unsigned char* const sx = smem;
    float4* const sums = reinterpret_cast<float4*>(smem + 8 * NT * rowb);   // [warp][NT][lane], when S > 1
    const bool one_slab = a.slab >= chunks;

    // this warp's chunks [c, end) of the slab at c0
    struct Place {
        int tile, c0, c, end;
    };
    auto enter = [&](int tile, int c0) {
        const int n = min(a.slab, chunks - c0);
        return Place{tile, c0, c0 + n * part / S, c0 + n * (part + 1) / S};
    };
    // the next chunks after p that are this warp's, tile >= tiles at the end
    auto after = [&](Place p) {
        p.c += kPair;
        while (p.c >= p.end && p.tile < tiles) {
            const int c0 = p.c0 + a.slab;
            p = c0 < chunks ? enter(p.tile, c0) : enter(p.tile + step, 0);
        }
        return p;
    };
    pdl_wait();
    Place at = enter(first + group, 0);
    if (at.c >= at.end) at = after(at);
    Rows2 rows = rows_of(a, at.tile, g8, t4);
    Piece now[kPair], next[kPair];
    auto load = [&](const Place& p, Piece (&piece)[kPair]) {
        const int n = p.tile < tiles ? p.end - p.c : 0;
#pragma unroll
        for (int j = 0; j < kPair; ++j)
            if (j < n) load_piece<kWords>(a, rows, p.c + j, p.c + j, t4, piece[j]);
    };
    load(at, now);
    if (one_slab) {
        stage<NT>(a, r0, 0, chunks, sx, rowb);
        __syncthreads();
    }
    const uint32_t sel = kWords ? uint32_t(t4 | (4 + t4) << 4) : 0x40u;   // the lane's scale codes of two outputs
    for (int base = first; base < tiles; base += step) {
        const int tile = base + group;
        float acc[NT][2][4] = {};
        for (int c0 = 0; c0 < chunks; c0 += a.slab) {
            if (!one_slab) {
                __syncthreads();
                stage<NT>(a, r0, c0, min(a.slab, chunks - c0), sx, rowb);
                __syncthreads();
            }
            while (at.tile == tile && at.c0 == c0 && tile < tiles) {
                const Place then = after(at);
                if (then.tile != at.tile) rows = rows_of(a, then.tile, g8, t4);
                load(then, next);
                const int left = at.end - at.c;
                const unsigned char* const xq = sx + g8 * rowb + (at.c - c0) * 256 + t4 * 16;
#pragma unroll
                for (int j = 0; j < kPair; ++j) {
                    if (j < left) {
                        multiply<NT, kWords>(now[j], xq + j * 256, rowb, sel, a.nibbles, acc);
                    }
                }
#pragma unroll
                for (int j = 0; j < kPair; ++j) now[j] = next[j];
                at = then;
            }
        }
        finish_tile<NT>(a, S, tile, tiles, r0, group, part, acc, sums);
    }
    pdl_trigger();
}

// Warps that share a tile: the S with the shortest longest warp, counted in
// chunks with one more a round for the adding up.
int split_of(int tiles, int chunks, int ctas) {
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int S = 1; S <= kWarps; S *= 2) {
        const int per_round = ctas * (kWarps / S), rounds = (tiles + per_round - 1) / per_round;
        const int64_t c = int64_t(rounds) * ((chunks + S - 1) / S + (S > 1 ? 1 : 0));
        if (c < cost) {
            cost = c;
            best = S;
        }
    }
    return best;
}

constexpr int kMaxSmem = 227 << 10;
constexpr int sum_bytes(int NT, int S) { return S > 1 ? kWarps * NT * 512 : 0; }

// A launch of one of the kernels; `ready` remembers its shared memory's attribute by device.
int launch_one(void (*kernel)(Linear, int), std::atomic<bool> (&ready)[64], const Linear& a, int ctas, int S, int smem,
               cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return cuda_fail(e);
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    return launch_pdl(kernel, dim3(ctas * a.row_tiles), dim3(kThreads), smem, stream, a, S);
}

template <int NT>
int launch(Linear a, cudaStream_t stream) {
    constexpr int kSums = kWarps * NT * 512;
    static std::atomic<bool> ready[6][64] = {};
    const int chunks = (a.K + kChunk - 1) / kChunk, tiles = (a.N + 15) / 16, sms = sm_count();
    a.row_tiles = (a.R + 8 * NT - 1) / (8 * NT);
    int ctas = sms / a.row_tiles;
    if (ctas < 1) ctas = 1;
    a.nibbles = 0x000F000Fu;
    const bool whole_chunks = a.K % kChunk == 0;
    const bool words = whole_chunks && (reinterpret_cast<uintptr_t>(a.g) & 3u) == 0;
    // Steps of two chunks where every warp has several of them: with four in flight, or with more warps and fewer
    // registers, a lane's weights leave no room to work ahead (128,000 outputs, 1 and 16 rows: 27.7 and 34.9 us; four
    // chunks 31.6 and 42.7; 24 warps 32.8 and 45.9, one chunk 29.3 and 41.5). An odd number of chunks is filled up
    // where the last one ends inside a chunk: its scales are read a byte at a time, which knows the row's end. (The
    // step decides where warps divide a sum, so it goes by K and N and not by the scales' address.)
    const int tiles_cta = (tiles + ctas - 1) / ctas;
    const bool two = (!whole_chunks || chunks % 2 == 0) && tiles_cta * ((chunks + 1) / 2) >= 2 * kWarps;
    a.slab = two ? (chunks + 1) / 2 * 2 : chunks;
    const int whole = 8 * NT * row_bytes(a.slab) + kSums;
    if (whole <= kMaxSmem) {
        if (ctas > tiles) ctas = tiles;
        if (words)
            return two ? launch_one(linear_steps_kernel<NT, 2, true>, ready[0], a, ctas, 1, whole, stream)
                       : launch_one(linear_steps_kernel<NT, 1, true>, ready[1], a, ctas, 1, whole, stream);
        return two ? launch_one(linear_steps_kernel<NT, 2, false>, ready[2], a, ctas, 1, whole, stream)
                   : launch_one(linear_steps_kernel<NT, 1, false>, ready[3], a, ctas, 1, whole, stream);
    }
    const int S = split_of(tiles, chunks, ctas), need = (tiles + kWarps / S - 1) / (kWarps / S);
    if (ctas > need) ctas = need;
    a.slab = ((kMaxSmem - sum_bytes(NT, S)) / (8 * NT) - 64) / (kChunk * 2);
    if (a.slab > chunks) a.slab = chunks;
    const int smem = 8 * NT * row_bytes(a.slab) + sum_bytes(NT, S);
    return words ? launch_one(linear_rows_kernel<NT, true>, ready[4], a, ctas, S, smem, stream)
                 : launch_one(linear_rows_kernel<NT, false>, ready[5], a, ctas, S, smem, stream);
}

// Tiles of 8 rows that a CTA takes: as many as there are, up to four, if their inputs lie
// in shared memory as a whole; fewer (the weights then come from L2 more than once)
// before they are staged a slab at a time; and fewer while SMs would stand idle, since
// most of a small call's time is the staging. 16 rows of 8,192 inputs to 4,992 outputs
// 15.0 us in two tiles of 8 rows, 44.6 in slabs; 32 rows of 4,096 to 10,000 17 and
// 49.2; 32 rows of 2,048 to 512 outputs 4.1 us in four tiles on 128 SMs, 7.6 on 32.
int row_tiles_of(int R, int K, int N) {
    const int chunks = ((K + kChunk - 1) / kChunk + 1) / 2 * 2, most = R < 25 ? (R + 7) / 8 : 4;   // (filled up)
    int nt = most;
    while (nt > 0 && 8 * nt * row_bytes(chunks) + sum_bytes(nt, 2) > kMaxSmem) --nt;
    if (nt == 0) return most;
    const int groups = (R + 7) / 8;
    auto abreast = [&](int tiles) { return (groups + tiles - 1) / tiles; };   // CTAs that share outputs
    while (nt > 1 && int64_t((N + 15) / 16) * abreast(nt - 1) <= sm_count()) --nt;
    nt = (groups + abreast(nt) - 1) / abreast(nt);   // 32 rows as 16 and 16, not 24 and 8
    return nt;
}

bool overlap(const void* p, size_t np, const void* q, size_t nq) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + nq && b < a + np;
}

}  // namespace
}  // namespace tf

extern "C" int tf_linear_rows(const void* x, int64_t x_stride, const void* x_scales, int R, int K, const void* w,
                              const void* w_scales, const float* s, int N, void* y, int64_t y_stride,
                              tf_cuda_stream stream) {
    using namespace tf;
    if (R < 0 || K < 1 || K % kGroup || N < 1) return TF_EINVAL;
    if (R > TF_LINEAR_MAX_ROWS || K > TF_LINEAR_MAX_INPUTS || N > TF_LINEAR_MAX_OUTPUTS) return TF_ERANGE;
    if (R == 0) return TF_OK;
    if (!x || !w || !w_scales || !s || !y || !aligned16(x) || !aligned16(w)) return TF_EINVAL;
    if (reinterpret_cast<uintptr_t>(s) & 3u || reinterpret_cast<uintptr_t>(y) & 1u) return TF_EINVAL;
    if (x_stride < K || x_stride % (x_scales ? 16 : 8) || y_stride < N) return TF_EINVAL;
    constexpr int64_t kMaxStride = int64_t(1) << 32;
    if (x_stride > kMaxStride || y_stride > kMaxStride) return TF_ERANGE;
    const size_t xb = size_t((R - 1) * x_stride + K) * (x_scales ? 1 : 2), yb = size_t((R - 1) * y_stride + N) * 2;
    if (overlap(x, xb, y, yb) || overlap(w, size_t(N) * K / 2, y, yb) ||
        overlap(w_scales, size_t(N) * (K / kGroup), y, yb) || overlap(s, size_t(N) * 4, y, yb) ||
        (x_scales && overlap(x_scales, size_t(R) * (K / kGroup), y, yb)))
        return TF_EINVAL;
    for (const void* p : {x, x_scales, w, w_scales, static_cast<const void*>(s), static_cast<const void*>(y)})
        if (p && !on_this_device(p)) return TF_EINVAL;
    Linear a = {};
    a.x = static_cast<const uint8_t*>(x);
    a.xs = static_cast<const uint8_t*>(x_scales);
    a.w = static_cast<const uint8_t*>(w);
    a.g = static_cast<const uint8_t*>(w_scales);
    a.s = s;
    a.y = static_cast<uint16_t*>(y);
    a.x_stride = x_stride;
    a.y_stride = y_stride;
    a.R = R;
    a.K = K;
    a.N = N;
    switch (row_tiles_of(R, K, N)) {
        case 1: return launch<1>(a, stream);
        case 2: return launch<2>(a, stream);
        case 3: return launch<3>(a, stream);
        default: return launch<4>(a, stream);
    }
}
