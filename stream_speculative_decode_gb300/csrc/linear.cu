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
// HBM bound for few rows: 17/32 bytes a weight, whatever their number. mma.sync
// m16n8k16 with 16 outputs by 8 rows a tile: the weights are the operand whose
// fragments come straight from memory, 32 codes of one row and scale (16 bytes)
// a lane, four lanes a row's 128 inputs; the order of the inputs in an MMA is
// free as long as x has the same. A nibble becomes 128 + c in bf16 by masks
// (0x4300 | c), and one bf16 FMA (128 + c) * g - 136 * g gives the weight.
//
// x lies in shared memory in the order in which the fragments want it (a row's 8
// inputs 8 w .. 8 w + 7 of a group as 0 4 1 5 2 6 3 7, the groups of a 128-input
// chunk side by side), staged once a CTA where it fits. One CTA of 16 warps an
// SM. For few outputs, S warps share a 16-output tile, each with its part of the
// inputs, and their sums are added in order through shared memory.
#include <cuda_bf16.h>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 128;                 // inputs of a chunk: four groups, one a lane of a row
constexpr int kGroup = TF_SCALE_COLUMNS;
constexpr int kQuad = 4;                    // chunks whose loads are in flight together
constexpr int kMaxX = 160 << 10;            // shared memory for x

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
    int words;                 // the scales of a chunk are an aligned word
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

// Rows [r0, r0 + 8 NT) and chunks [c0, c0 + n) of x into shared memory.
template <int NT>
__device__ __forceinline__ void stage(const Linear& a, int r0, int c0, int n, unsigned char* sx, int rowb) {
    const int units = n * kChunk / 8;   // 8 inputs each
    for (int i = threadIdx.x; i < 8 * NT * units; i += kThreads) {
        const int r = i / units, u = i % units, k = (c0 * kChunk) + u * 8;
        uint32_t v[4] = {0u, 0u, 0u, 0u};   // inputs (0, 4), (1, 5), (2, 6), (3, 7)
        if (r0 + r < a.R && k < a.K) {
            const int64_t at = int64_t(r0 + r) * a.x_stride + k;
            if (a.xs) {
                const uint2 c = *reinterpret_cast<const uint2*>(a.x + at);
                const float e = scale_value(a.xs[int64_t(r0 + r) * (a.K / kGroup) + k / kGroup]);
                const float2 p = h2_to_f2(e4m3_low(c.x)), q = h2_to_f2(e4m3_high(c.x));
                const float2 s = h2_to_f2(e4m3_low(c.y)), t = h2_to_f2(e4m3_high(c.y));
                v[0] = pack_bf2(p.x * e, s.x * e);
                v[1] = pack_bf2(p.y * e, s.y * e);
                v[2] = pack_bf2(q.x * e, t.x * e);
                v[3] = pack_bf2(q.y * e, t.y * e);
            } else {
                const uint4 c = *reinterpret_cast<const uint4*>(a.x + 2 * at);
                v[0] = __byte_perm(c.x, c.z, 0x5410);
                v[1] = __byte_perm(c.x, c.z, 0x7632);
                v[2] = __byte_perm(c.y, c.w, 0x5410);
                v[3] = __byte_perm(c.y, c.w, 0x7632);
            }
        }
        const int chunk = u >> 4, lane = (u >> 2) & 3, w = u & 3;
        *reinterpret_cast<uint4*>(sx + r * rowb + chunk * 256 + w * 64 + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// A lane's weights of up to four chunks of its two outputs, and their scales' bytes.
struct Piece {
    uint4 w[kQuad][2];
    uint32_t g[kQuad];   // the code of output g8 in the low byte, of 8 + g8 in the next
};

__device__ __forceinline__ void load_piece(const Linear& a, int64_t n0, int64_t n1, int c, int end, int t4, Piece& p) {
    const int groups = a.K / kGroup;
#pragma unroll
    for (int j = 0; j < kQuad; ++j) {
        const int grp = (c + j) * 4 + t4;
        p.w[j][0] = p.w[j][1] = make_uint4(0u, 0u, 0u, 0u);
        p.g[j] = 0;   // scale 0: no weight
        if (c + j < end && grp < groups) {
            p.w[j][0] = load_once(a.w + n0 * (a.K / 2) + grp * 16);
            p.w[j][1] = load_once(a.w + n1 * (a.K / 2) + grp * 16);
            if (a.words) {
                const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(a.g + n0 * groups) + c + j);
                const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(a.g + n1 * groups) + c + j);
                p.g[j] = __byte_perm(u, v, uint32_t(t4 | (4 + t4) << 4));
            } else {
                p.g[j] = uint32_t(__ldg(a.g + n0 * groups + grp)) | uint32_t(__ldg(a.g + n1 * groups + grp)) << 8;
            }
        }
    }
}

// Row tiles of 8 NT rows; S warps share an output tile.
template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
linear_rows_kernel(const __grid_constant__ Linear a, int S) {
    extern __shared__ __align__(128) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int r0 = (blockIdx.x % a.row_tiles) * 8 * NT;
    const int cta = blockIdx.x / a.row_tiles, ctas = gridDim.x / a.row_tiles;
    const int chunks = (a.K + kChunk - 1) / kChunk, rowb = row_bytes(min(a.slab, chunks));
    unsigned char* const sx = smem;
    float4* const sums = reinterpret_cast<float4*>(smem + 8 * NT * rowb);   // [warp][NT][lane], when S > 1
    const int per_cta = kWarps / S, part = warp % S, tiles = (a.N + 15) / 16;
    const bool one_slab = a.slab >= chunks;
    pdl_wait();
    if (one_slab) {
        stage<NT>(a, r0, 0, chunks, sx, rowb);
        __syncthreads();
    }
    for (int first = cta * per_cta; first < tiles; first += ctas * per_cta) {
        const int tile = first + warp / S;
        // outputs past N read the last one's weights and are not stored
        const int64_t n0 = min(tile * 16 + g8, a.N - 1), n1 = min(tile * 16 + 8 + g8, a.N - 1);
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
        for (int c0 = 0; c0 < chunks; c0 += a.slab) {
            const int n = min(a.slab, chunks - c0);
            if (!one_slab) {
                __syncthreads();
                stage<NT>(a, r0, c0, n, sx, rowb);
                __syncthreads();
            }
            const int begin = c0 + n * part / S, end = c0 + n * (part + 1) / S;
            if (tile >= tiles) continue;
            Piece now, next;
            load_piece(a, n0, n1, begin, end, t4, now);
            for (int c = begin; c < end; c += kQuad) {
                load_piece(a, n0, n1, c + kQuad, end, t4, next);
#pragma unroll
                for (int j = 0; j < kQuad; ++j) {
                    if (c + j >= end) break;
                    const float2 g = h2_to_f2(e4m3_low(now.g[j]));
                    const uint32_t s0 = pack_bf2(g.x, g.x), s1 = pack_bf2(g.y, g.y);
                    const uint32_t z0 = pack_bf2(-136.f * g.x, -136.f * g.x), z1 = pack_bf2(-136.f * g.y, -136.f * g.y);
                    const uint32_t w0[4] = {now.w[j][0].x, now.w[j][0].y, now.w[j][0].z, now.w[j][0].w};
                    const uint32_t w1[4] = {now.w[j][1].x, now.w[j][1].y, now.w[j][1].z, now.w[j][1].w};
                    const unsigned char* xr = sx + g8 * rowb + (c + j - c0) * 256 + t4 * 16;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint4 b[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            b[nt] = *reinterpret_cast<const uint4*>(xr + nt * 8 * rowb + k * 64);
                        auto weights = [&](uint32_t w, int i, uint32_t s, uint32_t z) {
                            return fma_bf2(((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, s, z);
                        };
                        const uint32_t lo[4] = {weights(w0[k], 0, s0, z0), weights(w1[k], 0, s1, z1),
                                                weights(w0[k], 1, s0, z0), weights(w1[k], 1, s1, z1)};
                        const uint32_t hi[4] = {weights(w0[k], 2, s0, z0), weights(w1[k], 2, s1, z1),
                                                weights(w0[k], 3, s0, z0), weights(w1[k], 3, s1, z1)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_bf16(acc[nt], lo, b[nt].x, b[nt].y);
                            mma_bf16(acc[nt], hi, b[nt].z, b[nt].w);
                        }
                    }
                }
                now = next;
            }
        }
        auto store = [&](int tl, int nt, int ln, const float4& v) {
            const int n = tl * 16 + (ln >> 2), r = r0 + nt * 8 + 2 * (ln & 3);
            const float d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int nn = n + 8 * (e >> 1), rr = r + (e & 1);
                if (nn < a.N && rr < a.R) {
                    const __nv_bfloat16 b = __float2bfloat16_rn(d[e] * __ldg(a.s + nn));
                    a.y[int64_t(rr) * a.y_stride + nn] = *reinterpret_cast<const uint16_t*>(&b);
                }
            }
        };
        if (S == 1) {
            if (tile < tiles)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    store(tile, nt, lane, make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]));
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                sums[(warp * NT + nt) * 32 + lane] = make_float4(acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
            __syncthreads();
            for (int i = tid; i < per_cta * NT * 32; i += kThreads) {
                const int tl = i / (NT * 32), at = i % (NT * 32);
                if (first + tl >= tiles) continue;
                float4 v = sums[tl * S * NT * 32 + at];
                for (int p = 1; p < S; ++p) {
                    const float4 u = sums[(tl * S + p) * NT * 32 + at];
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
                store(first + tl, at / 32, at % 32, v);
            }
            __syncthreads();
        }
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

template <int NT>
int launch(Linear a, cudaStream_t stream) {
    const int chunks = (a.K + kChunk - 1) / kChunk, tiles = (a.N + 15) / 16, sms = sm_count();
    a.row_tiles = (a.R + 8 * NT - 1) / (8 * NT);
    a.slab = (kMaxX / (8 * NT) - 64) / (kChunk * 2);
    if (a.slab > chunks) a.slab = chunks;
    int ctas = sms / a.row_tiles;
    if (ctas < 1) ctas = 1;
    const int S = split_of(tiles, chunks, ctas), need = (tiles + kWarps / S - 1) / (kWarps / S);
    if (ctas > need) ctas = need;
    const int smem = 8 * NT * row_bytes(a.slab) + (S > 1 ? kWarps * NT * 32 * 16 : 0);
    static bool ready[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !ready[dev]) {
        const cudaError_t e = cudaFuncSetAttribute(linear_rows_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxX + kWarps * NT * 32 * 16);
        if (e != cudaSuccess) return cuda_fail(e);
        if (dev >= 0 && dev < 64) ready[dev] = true;
    }
    return launch_pdl(linear_rows_kernel<NT>, dim3(ctas * a.row_tiles), dim3(kThreads), smem, stream, a, S);
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
    if (overlap(x, xb, y, yb) || overlap(w, size_t(N) * K / 2, y, yb) || overlap(w_scales, size_t(N) * (K / kGroup), y, yb) ||
        overlap(s, size_t(N) * 4, y, yb) || (x_scales && overlap(x_scales, size_t(R) * (K / kGroup), y, yb)))
        return TF_EINVAL;
    if (!on_this_device(x) || !on_this_device(w) || !on_this_device(y)) return TF_EINVAL;
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
    a.words = K % kChunk == 0 && (reinterpret_cast<uintptr_t>(w_scales) & 3u) == 0;
    return R <= 8 ? launch<1>(a, stream) : R <= 16 ? launch<2>(a, stream) : launch<4>(a, stream);
}
