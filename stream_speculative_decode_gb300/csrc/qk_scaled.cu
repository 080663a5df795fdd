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
// A CTA takes one block (16 keys, or the window's part of it): its 8 K heads and
// 8 V heads a warp each, a row being two lanes with 32 dimensions apiece (16 and
// their rotation partners), then the block's query heads, 4 lanes each. The
// rows' sines and cosines are worked out once, a thread an angle, into shared
// memory. HBM bound: 11,264 bytes a row read and written with a full block.
#include <cuda_bf16.h>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kKeys = TF_SCALE_KEYS;
constexpr int kThreads = 512;
constexpr int kQThreads = TF_NQ * 4;   // threads that share a row's queries: 4 a head
static_assert(kThreads / 32 == 2 * TF_NKV && kThreads == kKeys * TF_D / 2 && TF_D == 64, "the CTA's shape");

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

__global__ void __launch_bounds__(kThreads, 2)
qk_scaled_kernel(SegTable t, int layer, QkvRows in, const uint16_t* __restrict__ q_norm,
                 const uint16_t* __restrict__ k_norm, float eps, const __grid_constant__ Turns turns, uint16_t* q_out) {
    __shared__ float2 angle[kKeys][TF_D / 2];   // (cos, sin) of slot, frequency
    const AppendItem it = t.appends[blockIdx.x];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {
        const int pos = it.key0 + warp;   // a warp a slot: positions below 2^22
        const uint64_t turn = uint64_t(uint32_t(pos)) * turns.f[lane];
        float sn, cs;
        sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cs);
        angle[warp][lane] = make_float2(cs, sn);
    }
    const int ps = t.page_shift;
    const int64_t page = t.pages[t.page_first[it.stream] + (it.key0 >> ps)];
    const int in_page = it.key0 & ((1 << ps) - 1);
    __syncthreads();
    pdl_wait();

    {   // ---- one head of K or V
        const bool is_v = warp >= TF_NKV;
        const int g = warp & (TF_NKV - 1);
        const size_t slot = size_t(layer) * t.S + it.stream;
        const int64_t head = page * TF_NKV + g;
        uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(is_v ? t.v_cache[slot] : t.k_cache[slot]));
        uint8_t* scale = (is_v ? t.v_scale : t.k_scale)[layer] + ((head << ps) + in_page) / kKeys;
        const int r = lane >> 1, h = lane & 1;   // the block's slot; dimensions 16h.. and 32 + 16h..
        codes += ((head << ps) + in_page + r) * TF_D + 16 * h;
        const bool fresh = r >= it.slot0 && r < it.slot0 + it.n_rows, kept = r < it.slot0;
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
        int e_old = 0;
        if (fresh) {
            const int64_t row = it.row0 + r - it.slot0;
            const uint16_t* src = (is_v ? in.v + row * in.v_stride : in.k + row * in.k_stride) + g * TF_D + 16 * h;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                unpack8(*reinterpret_cast<const uint4*>(src + (i >> 1) * (TF_D / 2) + (i & 1) * 8), x + 8 * i);
        } else if (kept) {
            e_old = int(*scale) - kScaleBias;
            const float s = scale_value(uint32_t(e_old + kScaleBias));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 c = *reinterpret_cast<const uint4*>(codes + i * (TF_D / 2));
                const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 a = h2_to_f2(e4m3_low(w[j])), b = h2_to_f2(e4m3_high(w[j]));
                    x[16 * i + 4 * j] = a.x * s;
                    x[16 * i + 4 * j + 1] = a.y * s;
                    x[16 * i + 4 * j + 2] = b.x * s;
                    x[16 * i + 4 * j + 3] = b.y * s;
                }
            }
        }
        if (!is_v) {   // the kept rows are normed and rotated already
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) ss += x[i] * x[i];
            ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 1);
            if (fresh) {
                const float inv = rsqrtf(ss * (1.f / TF_D) + eps);
                float w[32];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    unpack8(*reinterpret_cast<const uint4*>(k_norm + 16 * h + (i >> 1) * (TF_D / 2) + (i & 1) * 8),
                            w + 8 * i);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float u = x[i] * inv * w[i], v = x[16 + i] * inv * w[16 + i];
                    const float2 a = angle[r][16 * h + i];
                    x[i] = u * a.x - v * a.y;
                    x[16 + i] = v * a.x + u * a.y;
                }
            }
        }
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) most = max(most, finite_bits(x[i]));
        const int e = scale_exponent(__reduce_max_sync(0xFFFFFFFFu, most));
        if (fresh || (kept && e != e_old)) {
            const float inv = scale_inverse(e);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float* y = x + 16 * i + 4 * j;
                    w[j] = e4m3_quad(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                }
                *reinterpret_cast<uint4*>(codes + i * (TF_D / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncwarp();   // the kept rows' lanes have read the old scale
        if (lane == 0) *scale = uint8_t(e + kScaleBias);
    }

    // ---- the block's queries
    const int head = (tid & (kQThreads - 1)) >> 2, d0 = (tid & 3) * 8;
    for (int i = tid / kQThreads; i < it.n_rows; i += kThreads / kQThreads) {
        const int64_t row = it.row0 + i;
        const uint16_t* src = in.q + row * in.q_stride + head * TF_D + d0;
        float a[8], b[8], wa[8], wb[8];
        unpack8(*reinterpret_cast<const uint4*>(src), a);
        unpack8(*reinterpret_cast<const uint4*>(src + TF_D / 2), b);
        unpack8(*reinterpret_cast<const uint4*>(q_norm + d0), wa);
        unpack8(*reinterpret_cast<const uint4*>(q_norm + TF_D / 2 + d0), wb);
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) ss += a[k] * a[k] + b[k] * b[k];
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 1);
        ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 2);
        const float inv = rsqrtf(ss * (1.f / TF_D) + eps);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float u = a[k] * inv * wa[k], v = b[k] * inv * wb[k];
            const float2 z = angle[it.slot0 + i][d0 + k];
            a[k] = u * z.x - v * z.y;
            b[k] = v * z.x + u * z.y;
        }
        uint16_t* dst = q_out + (row * TF_NQ + head) * TF_D + d0;
        *reinterpret_cast<uint4*>(dst) = pack8(a);
        *reinterpret_cast<uint4*>(dst + TF_D / 2) = pack8(b);
    }
    pdl_trigger();
}

}  // namespace

int launch_qk_scaled(const SegTable& t, int layer, const QkvRows& in, const uint16_t* q_norm, const uint16_t* k_norm,
                     float eps, const Turns& turns, uint16_t* q_out, cudaStream_t stream) {
    return launch_pdl(qk_scaled_kernel, dim3(t.n_appends), dim3(kThreads), 0, stream, t, layer, in, q_norm, k_norm, eps,
                      turns, q_out);
}

}  // namespace tf
