// Queries and keys of one attention layer made ready (tf_qk_rows) over a table
// of scaled pools: the RMS norm of each head, the half-split rotation by the
// row's position, and the append of the rows' K and V to their streams' caches,
// held as e4m3 codes with a scale for each 16 keys of a head.
//
// Norm and rotation are those of qk.cu (fp32; angles as 64-bit fractions of a
// turn). A block of 16 keys of a head takes the scale of the rows that it keeps
// (those before the window) and of the window's rows together (scaled.cuh): the
// kept rows are read back, and coded again when the scale's exponent moved. A
// code holds the same value under any scale while it is normal there, so a kept
// row changes only where it lies below 2^-14 of the block's largest; rows that a
// window rejected lose their say on the block's scale with the next append.
//
// One launch of two kinds of CTA, 4 warps each. Appending: the rows of the window
// that fall into one block take four CTAs, K or V and half of the heads each, a warp
// a head; a row is two lanes with 32 dimensions apiece (16 and their rotation
// partners), and K's CTAs work the block's sines and cosines out into shared memory.
// Queries: a warp a row (its 32 angles worked out once, a lane an angle, and spread
// by shuffles), 8 heads after another with the next one's loads in flight; for few
// rows a CTA a row, a warp 8 heads, as in qk.cu.
// HBM bound: 11,264 bytes a row read and written with a full block. A prompt of
// 16,381 rows in 32 sequences: 34.2 us, 5.4 TB/s, 81 % of the measured copy rate (one
// CTA of 512 threads a block, each thread working out its own angles from a table with
// no padding: 43.5 us); 16 streams of one row: 3.5 us (4.1 with the frequencies read as
// constants and every number tested for infinity).
#include <cuda_bf16.h>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kKeys = TF_SCALE_KEYS;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kBlockCtas = 2 * TF_NKV / kWarps;  // CTAs of a block: K, K, V, V
constexpr int kGroups = TF_NQ / 8;               // a warp takes 8 query heads at a time, 4 lanes a head
constexpr int kAngles = TF_D / 2 + 1;            // a row's angles in shared memory, padded: 16 rows are read at once
constexpr int kManyRows = 512;                   // qk.cu's
static_assert(kBlockCtas == 4 && kGroups == kWarps && TF_D == 64, "the CTAs' shapes");

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One head of K or V: the block's slots, two lanes a slot.
template <bool kV>
__device__ __forceinline__ void append_head(const SegTable& t, int layer, const AppendItem& it, const QkvRows& in,
                                            const uint16_t* k_norm, float eps, const float2 (*angle)[kAngles], int g,
                                            int lane) {
    const int ps = t.page_shift, in_page = it.key0 & ((1 << ps) - 1);
    const int64_t head = int64_t(t.pages[t.page_first[it.stream] + (it.key0 >> ps)]) * TF_NKV + g;
    const size_t slot = size_t(layer) * t.S + it.stream;
    const int r = lane >> 1, h = lane & 1;   // the slot; dimensions 16h.. and 32 + 16h..
    uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(kV ? t.v_cache[slot] : t.k_cache[slot])) +
                     ((head << ps) + in_page + r) * TF_D + 16 * h;
    uint8_t* scale = (kV ? t.v_scale : t.k_scale)[layer] + ((head << ps) + in_page) / kKeys;
    const bool fresh = r >= it.slot0 && r < it.slot0 + it.n_rows, kept = r < it.slot0;
    uint4 raw[4];
    int e_old = 0;
    if (fresh) {
        const int64_t row = it.row0 + r - it.slot0;
        const uint16_t* src = (kV ? in.v + row * in.v_stride : in.k + row * in.k_stride) + g * TF_D + 16 * h;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + (i >> 1) * (TF_D / 2) + (i & 1) * 8);
    } else if (kept) {
        e_old = int(*scale) - kScaleBias;
#pragma unroll
        for (int i = 0; i < 2; ++i) raw[i] = *reinterpret_cast<const uint4*>(codes + i * (TF_D / 2));
    }
    float x[32];
    if (!fresh) {
        const float s = kept ? scale_value(uint32_t(e_old + kScaleBias)) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 a = h2_to_f2(e4m3_low(kept ? w[j] : 0u)), b = h2_to_f2(e4m3_high(kept ? w[j] : 0u));
                x[16 * i + 4 * j] = a.x * s;
                x[16 * i + 4 * j + 1] = a.y * s;
                x[16 * i + 4 * j + 2] = b.x * s;
                x[16 * i + 4 * j + 3] = b.y * s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack8(raw[i], x + 8 * i);
    }
    if constexpr (!kV) {   // the kept rows are normed and rotated already
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) ss += x[i] * x[i];
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 1);
        if (fresh) {
            const float inv = rsqrtf(ss * (1.f / TF_D) + eps);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float wa[8], wb[8];
                unpack8(*reinterpret_cast<const uint4*>(k_norm + 16 * h + 8 * i), wa);
                unpack8(*reinterpret_cast<const uint4*>(k_norm + TF_D / 2 + 16 * h + 8 * i), wb);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int d = 8 * i + k;
                    const float u = x[d] * inv * wa[k], v = x[16 + d] * inv * wb[k];
                    const float2 a = angle[r][16 * h + d];
                    x[d] = u * a.x - v * a.y;
                    x[16 + d] = v * a.x + u * a.y;
                }
            }
        }
    }
    float top = 0.f;   // (a NaN is passed over)
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[i]));
    uint32_t most = __float_as_uint(top);
    if (most >= 0x7F800000u) {   // an infinity has no say, and becomes NaN
        most = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            most = max(most, finite_bits(x[i]));
            if (fabsf(x[i]) > 3.4e38f) x[i] = __uint_as_float(0x7FC00000u);
        }
    }
    __syncwarp();
    const int e = scale_exponent(__reduce_max_sync(0xFFFFFFFFu, most));
    if (fresh || (kept && e != e_old)) {
        const float inv = scale_inverse(e);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float* y = x + 16 * i + 4 * j;
                w[j] = e4m3_finite(y[0] * inv, y[1] * inv) | e4m3_finite(y[2] * inv, y[3] * inv) << 16;
            }
            *reinterpret_cast<uint4*>(codes + i * (TF_D / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    __syncwarp();   // the kept rows' lanes have read the old scale
    if (lane == 0) *scale = uint8_t(e + kScaleBias);
}

__device__ __forceinline__ float2 angle_of(int pos, uint64_t frequency) {   // (cos, sin)
    const uint64_t turn = uint64_t(uint32_t(pos)) * frequency;                 // positions below 2^22
    float sn, cs;
    sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cs);
    return make_float2(cs, sn);
}

// A lane's frequency, by a load: lanes that read different constants wait for one another.
__device__ __forceinline__ uint64_t frequency(const Turns& turns, int lane) {
    const uint64_t* f = turns.f;
    asm volatile("" : "+l"(f));
    return f[lane];
}

// 8 query heads of a row, 16 values a lane (d0.. and 32 + d0..), normed, rotated and stored.
__device__ __forceinline__ void finish_heads(uint4 a4, uint4 b4, uint4 wa4, uint4 wb4, const float (&c)[8],
                                             const float (&sine)[8], float eps, uint16_t* dst) {
    float a[8], b[8], wa[8], wb[8];
    unpack8(a4, a);
    unpack8(b4, b);
    unpack8(wa4, wa);
    unpack8(wb4, wb);
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) ss += a[k] * a[k] + b[k] * b[k];
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 1);
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 2);
    const float inv = rsqrtf(ss * (1.f / TF_D) + eps);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float u = a[k] * inv * wa[k], v = b[k] * inv * wb[k];
        a[k] = u * c[k] - v * sine[k];
        b[k] = v * c[k] + u * sine[k];
    }
    *reinterpret_cast<uint4*>(dst) = pack8(a);
    *reinterpret_cast<uint4*>(dst + TF_D / 2) = pack8(b);
}

// kMany: a warp a row of queries; otherwise a CTA a row.
template <bool kMany>
__global__ void __launch_bounds__(kThreads)
qk_scaled_kernel(SegTable t, int layer, QkvRows in, const uint16_t* __restrict__ q_norm,
                 const uint16_t* __restrict__ k_norm, float eps, const __grid_constant__ Turns turns, uint16_t* q_out) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int append_ctas = kBlockCtas * t.n_appends;
    if (int(blockIdx.x) < append_ctas) {
        __shared__ float2 angle[kKeys][kAngles];   // of slot, frequency
        const AppendItem it = t.appends[blockIdx.x / kBlockCtas];
        const int part = blockIdx.x % kBlockCtas, g = (part & 1) * kWarps + warp;
        if (part < 2) {
            const uint64_t f = frequency(turns, lane);
            for (int r = it.slot0 + warp; r < it.slot0 + it.n_rows; r += kWarps)
                angle[r][lane] = angle_of(it.key0 + r, f);
            __syncthreads();
        }
        pdl_wait();
        if (part < 2)
            append_head<false>(t, layer, it, in, k_norm, eps, angle, g, lane);
        else
            append_head<true>(t, layer, it, in, k_norm, eps, angle, g, lane);
    } else {
        const int i = int(blockIdx.x) - append_ctas, row = kMany ? i * kWarps + warp : i;
        if (row >= t.R) return;
        const int head = lane >> 2, d0 = (lane & 3) * 8;
        const uint16_t* src = in.q + int64_t(row) * in.q_stride + head * TF_D + d0;
        uint16_t* dst = q_out + (int64_t(row) * TF_NQ + head) * TF_D + d0;
        const SegStream& st = t.streams[t.row_stream[row]];
        const float2 z = angle_of(st.keys - st.rows + row - st.row_offset, frequency(turns, lane));
        float c[8], sine[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            c[k] = __shfl_sync(0xFFFFFFFFu, z.x, d0 + k);
            sine[k] = __shfl_sync(0xFFFFFFFFu, z.y, d0 + k);
        }
        pdl_wait();
        const uint4 wa4 = *reinterpret_cast<const uint4*>(q_norm + d0);
        const uint4 wb4 = *reinterpret_cast<const uint4*>(q_norm + TF_D / 2 + d0);
        constexpr int kN = kMany ? kGroups : 1;
        const int first = kMany ? 0 : warp;
        uint4 a4 = *reinterpret_cast<const uint4*>(src + first * 8 * TF_D);
        uint4 b4 = *reinterpret_cast<const uint4*>(src + first * 8 * TF_D + TF_D / 2);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            uint4 na4 = a4, nb4 = b4;
            if (j + 1 < kN) {
                na4 = *reinterpret_cast<const uint4*>(src + (first + j + 1) * 8 * TF_D);
                nb4 = *reinterpret_cast<const uint4*>(src + (first + j + 1) * 8 * TF_D + TF_D / 2);
            }
            finish_heads(a4, b4, wa4, wb4, c, sine, eps, dst + (first + j) * 8 * TF_D);
            a4 = na4;
            b4 = nb4;
        }
    }
    pdl_trigger();
}

}  // namespace

int launch_qk_scaled(const SegTable& t, int layer, const QkvRows& in, const uint16_t* q_norm, const uint16_t* k_norm,
                     float eps, const Turns& turns, uint16_t* q_out, cudaStream_t stream) {
    const int appends = kBlockCtas * t.n_appends;
    if (t.R >= kManyRows)
        return launch_pdl(qk_scaled_kernel<true>, dim3(appends + (t.R + kWarps - 1) / kWarps), dim3(kThreads), 0,
                          stream, t, layer, in, q_norm, k_norm, eps, turns, q_out);
    return launch_pdl(qk_scaled_kernel<false>, dim3(appends + t.R), dim3(kThreads), 0, stream, t, layer, in, q_norm,
                      k_norm, eps, turns, q_out);
}

}  // namespace tf
