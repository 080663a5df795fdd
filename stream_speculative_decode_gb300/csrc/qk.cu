// Queries and keys of one attention layer made ready in one pass: the RMS norm
// of each head, the half-split rotation by the row's position, and the append
// of the rows' K and V to their streams' caches (dense or paged).
//
// With p the row's position (keys - rows + i for window row i, so that the
// window's rows end the stream's keys), x a head's 64 values and w its norm
// weight:
//   n_d = x_d * w_d / sqrt(mean(x^2) + eps)
//   y_j = n_j cos(p f_j) - n_{j+32} sin(p f_j),
//   y_{j+32} = n_{j+32} cos(p f_j) + n_j sin(p f_j),   f_j = theta^(-2j/64), j < 32
// in fp32, rounded once to bf16 at the store.
//
// Angles: positions reach 2^22, where an fp32 product p * f_j is off by a
// quarter of a radian. f_j / (2 pi) comes as a 64-bit fraction of a turn, and
// p * fraction modulo 2^64 is the angle's fraction of a turn with no range
// reduction to lose bits in (the fraction is good to 2^-55, so the angle of
// position 2^22 is good to 2^-33 of a turn); its top 32 bits go to sincospif.
//
// A warp works on a group of 8 heads (of a row's 4 groups of queries, 1 of K, 1 of
// V): one warp a group, a CTA a row, or for many rows a warp a row. A head is 4
// lanes, each holding dimensions 8l..8l+7 and 32+8l.. of it, so a rotation needs
// no exchange, and two shuffles sum the squares. Lane j computes the sine and
// cosine of f_j, read by shuffles.
// HBM bound: 6,144 bytes in and as many out a row.
#include <cmath>

#include "tf_internal.cuh"

namespace tf {
namespace {

constexpr int kWarps = (TF_NQ + 2 * TF_NKV) / 8;
constexpr int kThreads = kWarps * 32;
static_assert(TF_D == 64 && TF_NKV == 8, "a warp's 8 heads of 4 lanes");

struct Turns {
    uint64_t f[TF_D / 2];   // f_j as a fraction of a turn, 2^64 = one turn
};

struct Rows {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;
};

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The cosines and sines of dimensions d0..d0+7's angles, from the lanes that hold them.
__device__ __forceinline__ void spread(float cs, float sn, int d0, float (&c)[8], float (&sine)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = __shfl_sync(0xFFFFFFFFu, cs, d0 + i);
        sine[i] = __shfl_sync(0xFFFFFFFFu, sn, d0 + i);
    }
}

// A lane's 16 values of a head (d0.. and 32 + d0..), normed with the weights and rotated.
__device__ __forceinline__ void norm_rotate(uint4 (&x)[2], uint4 wa4, uint4 wb4, const float (&c)[8],
                                            const float (&sine)[8], float eps) {
    float a[8], b[8], wa[8], wb[8];
    unpack8(x[0], a);
    unpack8(x[1], b);
    unpack8(wa4, wa);
    unpack8(wb4, wb);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 1);
    ss += __shfl_xor_sync(0xFFFFFFFFu, ss, 2);
    const float inv = rsqrtf(ss * (1.f / TF_D) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = a[i] * inv * wa[i], v = b[i] * inv * wb[i];
        a[i] = u * c[i] - v * sine[i];
        b[i] = v * c[i] + u * sine[i];
    }
    x[0] = pack8(a);
    x[1] = pack8(b);
}

// First element of KV head g's slot for key `pos` of stream s in a cache or pool.
__device__ __forceinline__ size_t kv_slot(const SegTable& t, int s, const SegStream& st, int g, int pos) {
    if (t.page_shift == 0) return (size_t(g) * st.cap + pos) * TF_D;
    const int ps = t.page_shift;
    const int64_t page = t.pages[t.page_first[s] + (pos >> ps)];
    return ((size_t(page * TF_NKV + g) << ps) + (pos & ((1 << ps) - 1))) * TF_D;
}

__global__ void __launch_bounds__(kThreads)
qk_rows_kernel(SegTable t, int layer, Rows in, const uint16_t* __restrict__ q_norm,
               const uint16_t* __restrict__ k_norm, float eps, const __grid_constant__ Turns turns,
               uint16_t* q_out) {
    const int row = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = lane >> 2, d0 = (lane & 3) * 8;   // this lane's head of the group and first dimensions
    const int s = t.row_stream[row];
    const SegStream st = t.streams[s];
    const int pos = st.keys - st.rows + row - st.row_offset;
    const size_t layer_slot = size_t(layer) * t.S + s;

    const bool is_q = warp < TF_NQ / 8, is_v = warp == kWarps - 1;
    uint16_t* dst;
    const uint16_t* src;
    if (is_q) {
        src = in.q + row * in.q_stride + warp * 8 * TF_D;
        dst = q_out + (size_t(row) * TF_NQ + warp * 8 + head) * TF_D;
    } else {
        src = is_v ? in.v + row * in.v_stride : in.k + row * in.k_stride;
        void* cache = const_cast<void*>(is_v ? t.v_cache[layer_slot] : t.k_cache[layer_slot]);
        dst = static_cast<uint16_t*>(cache) + kv_slot(t, s, st, head, pos);
    }
    src += head * TF_D + d0;
    dst += d0;
    const uint64_t turn = uint64_t(uint32_t(pos)) * turns.f[lane];
    float sn, cs;
    sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cs);

    pdl_wait();
    const uint4 a4 = *reinterpret_cast<const uint4*>(src);
    const uint4 b4 = *reinterpret_cast<const uint4*>(src + TF_D / 2);
    if (is_v) {
        pdl_trigger();
        *reinterpret_cast<uint4*>(dst) = a4;
        *reinterpret_cast<uint4*>(dst + TF_D / 2) = b4;
        return;
    }
    const uint16_t* w = (is_q ? q_norm : k_norm) + d0;
    const uint4 wa4 = *reinterpret_cast<const uint4*>(w);
    const uint4 wb4 = *reinterpret_cast<const uint4*>(w + TF_D / 2);
    pdl_trigger();
    float c[8], sine[8];
    spread(cs, sn, d0, c, sine);
    uint4 y[2] = {a4, b4};
    norm_rotate(y, wa4, wb4, c, sine, eps);
    *reinterpret_cast<uint4*>(dst) = y[0];
    *reinterpret_cast<uint4*>(dst + TF_D / 2) = y[1];
}

// Many rows: a warp takes a whole row, so a row's 32 angles are worked out once
// instead of in five warps (the other kernel is bound by its instructions there,
// half of which are the angles and their spreading), one group of heads after
// another with the next group's loads in flight. 16,381 rows 33.6 us against
// 43.7 (6.0 TB/s, 88 % of the measured copy rate), 60,000 rows 114.8 us against
// 150.9 (95 %); two or three groups' loads in flight took registers and ran
// slower (34.2, 39.1 us). From 512 rows it is the faster one (512 rows 2.9 us
// against 3.0, 256 rows 2.8 against 2.4).
constexpr int kManyRows = 512;
constexpr int kRowWarps = 4;
__global__ void __launch_bounds__(kRowWarps * 32)
qk_rows_many_kernel(SegTable t, int layer, Rows in, const uint16_t* __restrict__ q_norm,
                    const uint16_t* __restrict__ k_norm, float eps, const __grid_constant__ Turns turns,
                    uint16_t* q_out) {
    const int row = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int head = lane >> 2, d0 = (lane & 3) * 8;
    pdl_wait();
    if (row >= t.R) return;
    auto load = [&](int g, uint4 (&x)[2]) {
        const uint16_t* src = g < TF_NQ / 8 ? in.q + row * in.q_stride + g * 8 * TF_D
                              : g == kWarps - 1 ? in.v + row * in.v_stride : in.k + row * in.k_stride;
        src += head * TF_D + d0;
        x[0] = *reinterpret_cast<const uint4*>(src);
        x[1] = *reinterpret_cast<const uint4*>(src + TF_D / 2);
    };
    uint4 x[2], next[2];
    load(0, x);
    const int s = t.row_stream[row];
    const SegStream st = t.streams[s];
    const int pos = st.keys - st.rows + row - st.row_offset;
    const size_t layer_slot = size_t(layer) * t.S + s, slot = kv_slot(t, s, st, head, pos) + d0;
    uint16_t* const kd = static_cast<uint16_t*>(const_cast<void*>(t.k_cache[layer_slot])) + slot;
    uint16_t* const vd = static_cast<uint16_t*>(const_cast<void*>(t.v_cache[layer_slot])) + slot;
    uint16_t* const qd = q_out + (size_t(row) * TF_NQ + head) * TF_D + d0;
    const uint64_t turn = uint64_t(uint32_t(pos)) * turns.f[lane];
    float sn, cs, c[8], sine[8];
    sincospif(float(int32_t(turn >> 32)) * 0x1p-31f, &sn, &cs);
    spread(cs, sn, d0, c, sine);
#pragma unroll
    for (int g = 0; g < kWarps; ++g) {
        if (g + 1 < kWarps) load(g + 1, next);
        if (g < kWarps - 1) {
            const uint16_t* w = (g < TF_NQ / 8 ? q_norm : k_norm) + d0;
            norm_rotate(x, *reinterpret_cast<const uint4*>(w), *reinterpret_cast<const uint4*>(w + TF_D / 2), c, sine, eps);
        }
        uint16_t* dst = g < TF_NQ / 8 ? qd + g * 8 * TF_D : g == kWarps - 1 ? vd : kd;
        *reinterpret_cast<uint4*>(dst) = x[0];
        *reinterpret_cast<uint4*>(dst + TF_D / 2) = x[1];
        x[0] = next[0];
        x[1] = next[1];
    }
    pdl_trigger();
}

// Whether `rows` rows of `width` bf16 at a stride and the dense output's rows overlap.
bool overlaps(const void* p, int64_t stride, int64_t rows, int64_t width, const void* out, int64_t out_rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(out);
    return a < b + uintptr_t(out_rows) * TF_NQ * TF_D * 2 && b < a + uintptr_t((rows - 1) * stride + width) * 2;
}

}  // namespace
}  // namespace tf

extern "C" int tf_qk_rows(const tf_segments* seg, int attn_layer, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const void* q_norm, const void* k_norm,
                          float eps, double theta, void* q_out, tf_cuda_stream stream) {
    using namespace tf;
    if (!seg) return TF_EINVAL;
    const SegTable& t = seg->dev;
    if (attn_layer < 0 || attn_layer >= t.n_attn) return TF_EINVAL;
    if (!(eps > 0.f) || !std::isfinite(eps) || !(theta >= 1.0) || !std::isfinite(theta)) return TF_EINVAL;
    if (t.R == 0) return TF_OK;
    if (!on_this_device(seg)) return TF_EINVAL;
    for (const void* p : {q, k, v, q_norm, k_norm, static_cast<const void*>(q_out)})
        if (!p || !aligned16(p)) return TF_EINVAL;
    constexpr int64_t kQ = TF_NQ * TF_D, kKV = TF_NKV * TF_D, kMaxStride = int64_t(1) << 32;
    if (q_stride < kQ || k_stride < kKV || v_stride < kKV || (q_stride | k_stride | v_stride) % 8) return TF_EINVAL;
    if (q_stride > kMaxStride || k_stride > kMaxStride || v_stride > kMaxStride) return TF_ERANGE;
    const bool in_place = q == q_out && q_stride == kQ;   // each head is read and written by its own lanes
    if ((!in_place && overlaps(q, q_stride, t.R, kQ, q_out, t.R)) || overlaps(k, k_stride, t.R, kKV, q_out, t.R) ||
        overlaps(v, v_stride, t.R, kKV, q_out, t.R))
        return TF_EINVAL;
    for (const void* w : {q_norm, k_norm})   // TF_D weights: rows would be normed with what others wrote
        if (overlaps(w, 0, 1, TF_D, q_out, t.R)) return TF_EINVAL;
    Turns turns;
    for (int j = 0; j < TF_D / 2; ++j)
        turns.f[j] = uint64_t(std::ldexp(std::pow(theta, -2.0 * j / TF_D) * 0.15915494309189533577, 64));   // 1 / (2 pi)
    const Rows in = {static_cast<const uint16_t*>(q), static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                     q_stride, k_stride, v_stride};
    const uint16_t *qw = static_cast<const uint16_t*>(q_norm), *kw = static_cast<const uint16_t*>(k_norm);
    uint16_t* out = static_cast<uint16_t*>(q_out);
    if (t.R >= kManyRows)
        return launch_pdl(qk_rows_many_kernel, dim3((t.R + kRowWarps - 1) / kRowWarps), dim3(kRowWarps * 32), 0, stream,
                          t, attn_layer, in, qw, kw, eps, turns, out);
    return launch_pdl(qk_rows_kernel, dim3(t.R), dim3(kThreads), 0, stream, t, attn_layer, in, qw, kw, eps, turns, out);
}
