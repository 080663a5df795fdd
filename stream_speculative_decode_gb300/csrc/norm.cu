// The step between two projections of a residual stream: the residual's
// addition, the RMS norm and the coding of the normed rows into 8 bits, in one
// pass over the rows (tf_norm_rows).
//
//   h = bf16(x + res)          (h = x without a residual)
//   n_c = h_c * w_c / sqrt(mean(h^2) + eps)        fp32
//   codes and scale bytes of n for each 32 columns (scaled.cuh)
//
// The norm is taken of the h that is stored, so that it is the norm of the
// stream that the next addition reads. A row is read once and stays in registers
// between its sum of squares and its codes: 8 columns a thread (and pass of the
// width), 4 neighbouring lanes a scale. HBM bound with a residual, 7 bytes a value:
// 16,381 rows of 2,048 35.7 us, 6.6 TB/s, 98 % of the measured copy rate. Without
// one, 3 bytes a value, issue bounds it (23.3 us, 65 %), so pairs of numbers go
// through packed fp32 instructions, and what only an infinity needs is in a branch.
#include <cuda_bf16.h>

#include <cmath>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kVec = 8;   // columns a thread holds at a time
constexpr int kManyRows = 1024;

struct NormRows {
    const uint16_t* x;
    const uint16_t* res;
    const uint16_t* w;
    uint16_t* sum;
    uint8_t* codes;
    uint8_t* scales;
    int64_t x_stride, res_stride, sum_stride;
    float eps;
    int width, R;
};

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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t unpack2(uint32_t w) {
    return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t code2(uint64_t v) {
    const float2 f = both(v);
    return e4m3_finite(f.x, f.y);
}

// kRows rows a CTA, each by blockDim.x / kRows threads in kIter passes over the width.
template <int kIter, int kRows>
__global__ void __launch_bounds__(kMaxThreads)
norm_rows_kernel(const __grid_constant__ NormRows a) {
    __shared__ float part[kMaxThreads / 32];
    const int threads = blockDim.x / kRows, warps = threads / 32;   // of a row
    const int mine = kRows == 1 ? 0 : threadIdx.x / threads, tid = threadIdx.x - mine * threads;
    const int64_t row = int64_t(blockIdx.x) * kRows + mine;
    const int vecs = kRows == 1 || row < a.R ? a.width / kVec : 0;
    pdl_wait();
    uint4 xv[kIter], rv[kIter], wv[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int v = tid + i * threads;
        xv[i] = rv[i] = wv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (v < vecs) {
            xv[i] = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + v * kVec);
            if (a.res) rv[i] = *reinterpret_cast<const uint4*>(a.res + row * a.res_stride + v * kVec);
            wv[i] = *reinterpret_cast<const uint4*>(a.w + v * kVec);
        }
    }
    uint64_t squares = pair(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        uint32_t* const x = &xv[i].x;
        if (a.res) {
            const uint32_t* const r = &rv[i].x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 h = both(add2(unpack2(x[k]), unpack2(r[k])));
                const __nv_bfloat162 b = __floats2bfloat162_rn(h.x, h.y);
                x[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            const int v = tid + i * threads;
            if (v < vecs) *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + v * kVec) = xv[i];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) squares = fma2(unpack2(x[k]), unpack2(x[k]), squares);
    }
    const float2 two = both(squares);
    float ss = two.x + two.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
        __syncthreads();
        ss = 0.f;
        for (int k = 0; k < warps; ++k) ss += part[mine * warps + k];
    }
    const float inv = rsqrtf(ss / float(a.width) + a.eps);
    const uint64_t inv2 = pair(inv, inv);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int v = tid + i * threads;
        const uint32_t *const x = &xv[i].x, *const w = &wv[i].x;
        uint64_t n[4];
        float top = 0.f;   // of this thread's numbers (a NaN is passed over)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            n[k] = mul2(mul2(unpack2(x[k]), inv2), unpack2(w[k]));
            const float2 f = both(n[k]);
            top = fmaxf(fmaxf(top, fabsf(f.x)), fabsf(f.y));
        }
        uint32_t most = __float_as_uint(top);
        const bool infinite = most >= 0x7F800000u;
        if (infinite) {   // it has no say, and becomes NaN
            most = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 f = both(n[k]);
                most = max(most, max(finite_bits(f.x), finite_bits(f.y)));
                if (fabsf(f.x) > 3.4e38f) f.x = __uint_as_float(0x7FC00000u);
                if (fabsf(f.y) > 3.4e38f) f.y = __uint_as_float(0x7FC00000u);
                n[k] = pair(f.x, f.y);
            }
        }
        __syncwarp();
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int e = scale_exponent(most);
        const float up = scale_inverse(e);
        const uint64_t up2 = pair(up, up);
        if (v < vecs) {
            const uint2 c = make_uint2(code2(mul2(n[0], up2)) | code2(mul2(n[1], up2)) << 16,
                                       code2(mul2(n[2], up2)) | code2(mul2(n[3], up2)) << 16);
            *reinterpret_cast<uint2*>(a.codes + row * a.width + v * kVec) = c;
            if ((v & 3) == 0) a.scales[row * (a.width / TF_SCALE_COLUMNS) + (v >> 2)] = uint8_t(e + kScaleBias);
        }
    }
    pdl_trigger();
}

// Bytes that `rows` rows of `width` bytes at a stride take up.
struct Span {
    uintptr_t at;
    int64_t rows, stride, width;
    uintptr_t end() const { return at + uintptr_t((rows - 1) * stride + width); }
};
bool apart(const Span& a, const Span& b) {
    if (!a.at || !b.at || a.at >= b.end() || b.at >= a.end()) return true;
    if (a.stride != b.stride) return false;
    const int64_t d = int64_t((b.at > a.at ? b.at - a.at : a.at - b.at) % uintptr_t(a.stride));   // rows side by side
    return b.at > a.at ? d >= a.width && a.stride - d >= b.width : d >= b.width && a.stride - d >= a.width;
}

// At most `most` threads a row, a whole number of warps with the fewest idle.
template <int kRows>
int launch(const NormRows& a, int most, cudaStream_t stream) {
    const int vecs = a.width / kVec, iters = (vecs + most - 1) / most;
    const int threads = ((vecs + iters - 1) / iters + 31) / 32 * 32;
    const dim3 grid((a.R + kRows - 1) / kRows), block(threads * kRows);
    if (iters == 1) return launch_pdl(norm_rows_kernel<1, kRows>, grid, block, 0, stream, a);
    if (iters == 2) return launch_pdl(norm_rows_kernel<2, kRows>, grid, block, 0, stream, a);
    if (iters == 3) return launch_pdl(norm_rows_kernel<3, kRows>, grid, block, 0, stream, a);
    if (iters == 4) return launch_pdl(norm_rows_kernel<4, kRows>, grid, block, 0, stream, a);
    return launch_pdl(norm_rows_kernel<8, kRows>, grid, block, 0, stream, a);
}

}  // namespace
}  // namespace tf

extern "C" int tf_norm_rows(const void* x, int64_t x_stride, const void* res, int64_t res_stride, const void* w,
                            float eps, int R, int width, void* sum, int64_t sum_stride, void* codes, void* scales,
                            tf_cuda_stream stream) {
    using namespace tf;
    if (R < 0 || width < 1 || width % TF_SCALE_COLUMNS || !(eps > 0.f) || !std::isfinite(eps)) return TF_EINVAL;
    if (R > (1 << 24) || width > TF_NORM_MAX_WIDTH) return TF_ERANGE;
    if (R == 0) return TF_OK;
    if (!x || !w || !codes || !scales || (res != nullptr) != (sum != nullptr)) return TF_EINVAL;
    for (const void* p : {x, res, w, static_cast<const void*>(sum), static_cast<const void*>(codes)})
        if (p && !aligned16(p)) return TF_EINVAL;
    if (!res) res_stride = sum_stride = width;
    constexpr int64_t kMaxStride = int64_t(1) << 32;
    for (int64_t s : {x_stride, res_stride, sum_stride}) {
        if (s < width || s % kVec) return TF_EINVAL;
        if (s > kMaxStride) return TF_ERANGE;
    }
    const auto span = [&](const void* p, int64_t stride, int64_t rows, int64_t n) {
        return Span{reinterpret_cast<uintptr_t>(p), rows, stride, n};
    };
    const Span sx = span(x, 2 * x_stride, R, 2 * width), sr = span(res, 2 * res_stride, R, 2 * width),
               sw = span(w, 2 * width, 1, 2 * width), ss = span(sum, 2 * sum_stride, R, 2 * width),
               sc = span(codes, width, R, width),
               sb = span(scales, width / TF_SCALE_COLUMNS, R, width / TF_SCALE_COLUMNS);
    // the sum may lie where an addend lay: a value is read and written by one thread
    if ((sum != x || sum_stride != x_stride) && !apart(ss, sx)) return TF_EINVAL;
    if ((sum != res || sum_stride != res_stride) && !apart(ss, sr)) return TF_EINVAL;
    for (const Span& in : {sx, sr, sw, ss})
        if (!apart(in, sc) || !apart(in, sb)) return TF_EINVAL;
    if (!apart(ss, sw) || !apart(sc, sb)) return TF_EINVAL;
    for (const void* p : {x, res, w, static_cast<const void*>(sum), static_cast<const void*>(codes),
                          static_cast<const void*>(scales)})
        if (p && !on_this_device(p)) return TF_EINVAL;
    const NormRows a = {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(res),
                        static_cast<const uint16_t*>(w), static_cast<uint16_t*>(sum), static_cast<uint8_t*>(codes),
                        static_cast<uint8_t*>(scales), x_stride, res_stride, sum_stride, eps, width, R};
    // Many narrow rows: a warp a row, 8 rows a CTA, since CTAs start at no more than one a nanosecond (16,000 rows of
    // 96 5.5 us, a CTA a row 18.5; of 1,024 without a residual 13.0 and 18.5; of 1,024 with one 20.1 and 19.8).
    // Otherwise up to 128 threads a row, to four vectors a thread, then 256: the more rows an SM has under way, the
    // better its loads cover one another's latency (16,381 rows of 2,048 36.1 us, 256 threads 39.0, two rows a CTA
    // 37.5; 4,000 of 8,192 38.3 and, with 256 threads, 36.1).
    const int vecs = width / kVec;
    if (R >= kManyRows && vecs <= 4 * 32) return launch<8>(a, 32, stream);
    return launch<1>(a, vecs <= 4 * 128 ? 128 : kMaxThreads, stream);
}
