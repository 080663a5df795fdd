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
// between its sum of squares and its codes: a CTA a row, 8 columns a thread (and
// pass of the width), 4 neighbouring lanes a scale. HBM bound: 7 bytes a value
// with a residual (3 without). 16,381 rows of 2,048 with a residual: 36.8 us, 6.4
// TB/s, 96 % of the measured copy rate.
#include <cuda_bf16.h>

#include <cmath>

#include "scaled.cuh"

namespace tf {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kVec = 8;   // columns a thread holds at a time

struct NormRows {
    const uint16_t* x;
    const uint16_t* res;
    const uint16_t* w;
    uint16_t* sum;
    uint8_t* codes;
    uint8_t* scales;
    int64_t x_stride, res_stride, sum_stride;
    float eps;
    int width;
};

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// kIter passes of the CTA's threads over the width.
template <int kIter>
__global__ void __launch_bounds__(kMaxThreads)
norm_rows_kernel(NormRows a) {
    __shared__ float part[kMaxThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, vecs = a.width / kVec;
    const int64_t row = blockIdx.x;
    pdl_wait();
    uint4 xv[kIter], rv[kIter], wv[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int v = tid + i * blockDim.x;
        xv[i] = rv[i] = wv[i] = make_uint4(0u, 0u, 0u, 0u);
        if (v < vecs) {
            xv[i] = *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + v * kVec);
            if (a.res) rv[i] = *reinterpret_cast<const uint4*>(a.res + row * a.res_stride + v * kVec);
            wv[i] = *reinterpret_cast<const uint4*>(a.w + v * kVec);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        if (a.res) {
            float x[kVec], r[kVec];
            unpack8(xv[i], x);
            unpack8(rv[i], r);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k] + r[2 * k], x[2 * k + 1] + r[2 * k + 1]);
                h[k] = *reinterpret_cast<const uint32_t*>(&b);
            }
            xv[i] = make_uint4(h[0], h[1], h[2], h[3]);
            const int v = tid + i * blockDim.x;
            if (v < vecs) *reinterpret_cast<uint4*>(a.sum + row * a.sum_stride + v * kVec) = xv[i];
        }
        float h[kVec];
        unpack8(xv[i], h);
#pragma unroll
        for (int k = 0; k < kVec; ++k) ss += h[k] * h[k];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    if (blockDim.x > 32) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = 0.f;
        for (int k = 0; k < int(blockDim.x) / 32; ++k) ss += part[k];
    }
    const float inv = rsqrtf(ss / float(a.width) + a.eps);
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
        const int v = tid + i * blockDim.x;
        float n[kVec], w[kVec];
        unpack8(xv[i], n);
        unpack8(wv[i], w);
        uint32_t most = 0;
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            n[k] = n[k] * inv * w[k];
            most = max(most, finite_bits(n[k]));
        }
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int e = scale_exponent(most);
        const float up = scale_inverse(e);
        if (v < vecs) {
            const uint2 c = make_uint2(e4m3_quad(n[0] * up, n[1] * up, n[2] * up, n[3] * up),
                                       e4m3_quad(n[4] * up, n[5] * up, n[6] * up, n[7] * up));
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
    if (!on_this_device(x) || !on_this_device(codes)) return TF_EINVAL;
    const NormRows a = {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(res),
                        static_cast<const uint16_t*>(w), static_cast<uint16_t*>(sum), static_cast<uint8_t*>(codes),
                        static_cast<uint8_t*>(scales), x_stride, res_stride, sum_stride, eps, width};
    // Up to 128 threads a row: the more rows an SM has under way, the better its loads cover one another's latency
    // (16,381 rows of 2,048: 64 or 128 threads 36.8 us, 256 or 512 threads 44.0 us). More than four vectors a thread
    // would cost more in registers than that gains.
    const int vecs = width / kVec, most = vecs <= 4 * 128 ? 128 : kMaxThreads;
    const int threads = vecs < most ? (vecs + 31) / 32 * 32 : most;
    const int iters = (vecs + threads - 1) / threads;
    const dim3 grid(R), block(threads);
    if (iters == 1) return launch_pdl(norm_rows_kernel<1>, grid, block, 0, stream, a);
    if (iters == 2) return launch_pdl(norm_rows_kernel<2>, grid, block, 0, stream, a);
    if (iters <= 4) return launch_pdl(norm_rows_kernel<4>, grid, block, 0, stream, a);
    return launch_pdl(norm_rows_kernel<8>, grid, block, 0, stream, a);
}
