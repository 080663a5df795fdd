// Sampling of each row of bf16 logits from a given uniform number, with
// temperature, top-k, top-p and min-p.
//
// Tokens in order of (logit descending, id ascending); w = exp((x - max) / T).
// Top-k keeps the first k tokens, their mass Z. Top-p keeps the shortest prefix
// of mass at least p Z, min-p the tokens of w >= min_p; what is kept is the
// shortest of the three prefixes, and the pick is the first token at which the
// cumulative mass exceeds u times the kept mass.
//
// A cumulative mass over 128,000 tokens in fp32 would move the pick of every
// few hundredth row, so masses are exact to 64 bits: bf16 logits take few
// distinct values, a value's mass is its count times one weight, the counts
// are integers (a histogram in shared memory, so the order of its atomics does
// not matter) and the weights are 64-bit fixed point. Masses of up to V tokens
// of weight 1 fit 64 bits at 63 - log2(V) fraction bits (46 at V = 128,000: a
// weight is off by at most 2^-47 of the largest).
//
// Values are handled as signed magnitudes (key = +-(bits & 0x7FFF), so -0 is
// +0 and keys rise with values), in windows of 4,096 keys from the largest key
// down; a window covers 32 powers of two, so N(0, 3) logits take two.
#include <cmath>

#include "tf_internal.cuh"

namespace tf {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 4096;                    // keys of a window
constexpr int kBins = kWindow / kThreads;        // keys of a window a thread scans
constexpr int kMaxWindows = 2 * 0x7F80 / kWindow + 2;
constexpr int kMinKey = -0x7F80;                 // the key of -infinity: a masked token
constexpr int kInfKey = 0x7F80;

using u64 = unsigned long long;

// 2^(-i/64) and 2^(-i/4096) in units of 2^-63, i < 64, by repeated products of
// the step's value (each product is off by less than 2^-63).
struct ExpTables {
    u64 coarse[64], fine[64];
};
constexpr u64 mul_hi(u64 a, u64 b) {
    const u64 a0 = a & 0xFFFFFFFFu, a1 = a >> 32, b0 = b & 0xFFFFFFFFu, b1 = b >> 32;
    const u64 m = a1 * b0 + (a0 * b0 >> 32), n = a0 * b1 + (m & 0xFFFFFFFFu);
    return a1 * b1 + (m >> 32) + (n >> 32);
}
constexpr u64 sqrt63(u64 x) {   // square root of x / 2^63, in the same units, by bisection
    u64 lo = 0, hi = u64(1) << 63;
    while (hi - lo > 1) {
        const u64 mid = lo + (hi - lo) / 2;
        (mul_hi(mid, mid) << 1 > x ? hi : lo) = mid;
    }
    return lo;
}
constexpr ExpTables make_tables() {
    ExpTables t{};
    u64 step = u64(1) << 62;                       // 2^-1
    for (int i = 0; i < 6; ++i) step = sqrt63(step);
    t.coarse[0] = t.fine[0] = u64(1) << 63;
    for (int i = 1; i < 64; ++i) t.coarse[i] = mul_hi(t.coarse[i - 1], step) << 1;
    for (int i = 0; i < 6; ++i) step = sqrt63(step);
    for (int i = 1; i < 64; ++i) t.fine[i] = mul_hi(t.fine[i - 1], step) << 1;
    return t;
}
__device__ const ExpTables kExpTables = make_tables();

// 2^-y in units of 2^-frac, y >= 0: the integer part shifts, the next two
// groups of six bits look up, and the rest, r < 2^-12, is 1 - a + a^2/2 - a^3/6
// with a = r ln 2 (the next term is below 2^-54).
__device__ __forceinline__ u64 weight(double y, int frac, const ExpTables& tab) {
    if (!(y < 62.0)) return 0;
    const u64 fx = __double2ull_rz(y * 0x1p52);
    const int n = int(fx >> 52);
    const u64 c = tab.coarse[(fx >> 46) & 63], f = tab.fine[(fx >> 40) & 63];
    const u64 a = __umul64hi(fx << 24, 0xB17217F7D1CF79ABull) >> 12;   // r ln 2 in units of 2^-64
    const u64 a2 = __umul64hi(a, a), a3 = __umul64hi(a2, a);
    const u64 poly = (u64(1) << 63) - (a >> 1) + (a2 >> 2) - a3 / 12;
    const u64 w = __umul64hi(__umul64hi(c, f) << 1, poly) << 1;        // 2^-(fraction of y), units of 2^-63
    const int shift = 63 - frac + n;
    return shift > 63 ? 0 : (w + (u64(1) << shift >> 1)) >> shift;
}

__device__ __forceinline__ int key_of(uint32_t bits) {
    const int mag = int(bits & 0x7FFFu);
    return bits & 0x8000u ? -mag : mag;
}
__device__ __forceinline__ double value_of(int key) {
    const float v = __uint_as_float(uint32_t(key < 0 ? -key : key) << 16);
    return key < 0 ? -double(v) : double(v);
}

struct Shared {
    ExpTables tab;
    uint32_t hist[kWindow];
    int32_t top[kMaxWindows];          // windows used, from the largest key down
    u64 mass_before[kMaxWindows];
    int32_t count_before[kMaxWindows];
    u64 warp_mass[kWarps];
    int32_t warp_int[kWarps];
    u64 mass[4];
    int32_t num[4];
};

__device__ __forceinline__ int block_max(int v, Shared& sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh.warp_int[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh.warp_int[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return __shfl_sync(0xFFFFFFFFu, v, 0);
}

// Sums over the threads before this one, and the block's totals.
struct Scan {
    int32_t count, total;
    u64 mass, total_mass;
};
__device__ __forceinline__ Scan block_scan(int32_t c, u64 m, Shared& sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t ci = c;
    u64 mi = m;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t c2 = __shfl_up_sync(0xFFFFFFFFu, ci, o);
        const u64 m2 = __shfl_up_sync(0xFFFFFFFFu, mi, o);
        if (lane >= o) {
            ci += c2;
            mi += m2;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sh.warp_int[warp] = ci;
        sh.warp_mass[warp] = mi;
    }
    __syncthreads();
    Scan s = {ci - c, 0, mi - m, 0};
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            s.count += sh.warp_int[w];
            s.mass += sh.warp_mass[w];
        }
        s.total += sh.warp_int[w];
        s.total_mass += sh.warp_mass[w];
    }
    return s;
}

struct Args {
    const uint16_t* logits;
    int64_t stride;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* pick;
    float* prob;
    uint8_t* flag;
    int32_t V;
    int32_t frac;
};

__global__ void __launch_bounds__(kThreads)
sample_rows_kernel(Args a) {
    __shared__ Shared sh;
    const int row = blockIdx.x, tid = threadIdx.x;
    const uint16_t* p = a.logits + size_t(row) * size_t(a.stride);
    if (tid < 64) {
        sh.tab.coarse[tid] = kExpTables.coarse[tid];
        sh.tab.fine[tid] = kExpTables.fine[tid];
    }
    pdl_wait();
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const float tp = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int32_t tk = a.top_k ? a.top_k[row] : 0;
    const int32_t K = tk > 0 && tk < a.V ? tk : a.V;
    const bool bad_setting = !(T >= 0.f && T < INFINITY) || isnan(tp) || isnan(mp) || !(mp <= 1.f) ||
                             !(u >= 0.f && u < 1.f);

    int hi = kMinKey;
    for (int i = tid; i < a.V; i += kThreads) {
        const int k = key_of(p[i]);
        hi = max(hi, k >= kInfKey || k < kMinKey ? 0x10000 : k);   // NaN or +infinity: beyond every key
    }
    hi = block_max(hi, sh);
    if (hi == 0x10000 || hi == kMinKey || bad_setting) {
        if (tid == 0) {
            a.pick[row] = -1;
            if (a.prob) a.prob[row] = 0.f;
            a.flag[row] = uint8_t((hi == 0x10000 || hi == kMinKey ? TF_SAMPLE_NO_LOGITS : 0) |
                                  (bad_setting ? TF_SAMPLE_BAD_SETTING : 0));
        }
        return;
    }
    const double vmax = value_of(hi), per = T > 0.f ? 1.4426950408889634074 / double(T) : 0.0;   // log2(e) / T
    // log2 of the smallest kept weight, negated
    const double y_min = mp > 0.f ? -log2(double(mp)) : 2e308;

    int32_t want = 0, pick_key = hi;   // the pick: the want-th token (by id) of value pick_key
    float prob = 1.f;
    if (T > 0.f) {
        // counts of window `top` into the histogram; the largest key below it
        auto count = [&](int top) {
            __syncthreads();
            for (int i = tid; i < kWindow; i += kThreads) sh.hist[i] = 0;
            __syncthreads();
            int below = kMinKey;
            for (int i = tid; i < a.V; i += kThreads) {
                const int k = key_of(p[i]);
                if (k > top || k == kMinKey) continue;
                if (top - k < kWindow) atomicAdd(&sh.hist[top - k], 1u);
                else below = max(below, k);
            }
            return block_max(below, sh);   // a barrier: the histogram is complete
        };
        // f(key, tokens kept by top-k, tokens before, mass before, weight) of this thread's values of
        // window w, in descending order; the masses of the whole window
        auto walk = [&](int w, auto&& f) {
            const int top = sh.top[w];
            int32_t c[kBins], cs = 0;
            u64 wt[kBins], ms = 0;
#pragma unroll
            for (int j = 0; j < kBins; ++j) {
                c[j] = int32_t(sh.hist[tid * kBins + j]);
                cs += c[j];
            }
            const Scan sc = block_scan(cs, 0, sh);
            int32_t before = sh.count_before[w] + sc.count;
            const int32_t before0 = before;
#pragma unroll
            for (int j = 0; j < kBins; ++j) {
                wt[j] = c[j] ? weight((vmax - value_of(top - tid * kBins - j)) * per, a.frac, sh.tab) : 0;
                const int32_t n = max(0, min(c[j], K - before));
                before += c[j];
                c[j] = n;
                ms += u64(n) * wt[j];
            }
            const Scan sm = block_scan(0, ms, sh);
            u64 mass = sh.mass_before[w] + sm.mass;
            before = min(before0, K);
#pragma unroll
            for (int j = 0; j < kBins; ++j) {
                if (c[j]) f(top - tid * kBins - j, c[j], before, mass, wt[j]);
                before += c[j];
                mass += u64(c[j]) * wt[j];
            }
            return Scan{0, sc.total, 0, sm.total_mass};
        };

        // windows down to the k-th token, and the mass Z of the first k
        int nw = 0;
        for (int top = hi, counted = 0;;) {
            const int below = count(top);
            __syncthreads();
            if (tid == 0) {
                sh.top[nw] = top;
                if (nw == 0) {
                    sh.count_before[0] = 0;
                    sh.mass_before[0] = 0;
                }
            }
            __syncthreads();
            const Scan s = walk(nw, [](int, int32_t, int32_t, u64, u64) {});
            counted += s.total;
            ++nw;
            if (tid == 0) {
                sh.count_before[nw] = counted;
                sh.mass_before[nw] = sh.mass_before[nw - 1] + s.total_mass;
            }
            if (below == kMinKey || counted >= K) break;
            top = below;
        }
        int held = nw - 1;   // the window whose counts the histogram holds
        __syncthreads();
        const u64 Z = sh.mass_before[nw];
        auto hold = [&](int w) {
            if (held != w) count(sh.top[w]);
            held = w;
        };

        // the kept mass: of the shortest prefix
        u64 kept = Z;
        if (tp < 1.f) {
            const double need = double(fmaxf(tp, 0.f)) * double(Z);
            const u64 least = max(u64(1), u64(ceil(need)));   // the first prefix of at least this mass
            int w = 0;
            while (sh.mass_before[w + 1] < least) ++w;
            hold(w);
            walk(w, [&](int, int32_t n, int32_t, u64 m, u64 wt) {
                if (m < least && least <= m + u64(n) * wt) sh.mass[0] = m + (least - m + wt - 1) / wt * wt;
            });
            __syncthreads();
            kept = min(kept, sh.mass[0]);
        }
        if (mp > 0.f) {
            // the last window whose largest value is kept holds the cut
            int w = 0;
            while (w + 1 < nw && (vmax - value_of(sh.top[w + 1])) * per <= y_min) ++w;
            hold(w);
            if (tid == 0) sh.mass[1] = 0;
            __syncthreads();
            walk(w, [&](int key, int32_t n, int32_t, u64 m, u64 wt) {
                if ((vmax - value_of(key)) * per <= y_min) atomicMax(&sh.mass[1], m + u64(n) * wt);
            });
            __syncthreads();
            kept = min(kept, sh.mass[1]);
        }
        const u64 target = min(u64(double(u) * double(kept)), kept - 1);
        {
            int w = 0;
            while (sh.mass_before[w + 1] <= target) ++w;
            hold(w);
            walk(w, [&](int key, int32_t n, int32_t, u64 m, u64 wt) {
                if (m <= target && target < m + u64(n) * wt) {
                    sh.num[0] = key;
                    sh.num[1] = int32_t((target - m) / wt);
                }
            });
            __syncthreads();
            pick_key = sh.num[0];
            want = sh.num[1];
            // the pick's weight again, to all 63 bits
            const u64 w63 = weight((vmax - value_of(pick_key)) * per, 63, sh.tab);
            prob = float(ldexp(double(w63), a.frac - 63) / double(kept));
        }
    }
    pdl_trigger();

    // the want-th token of value pick_key, in id order: contiguous ranges a thread
    const int per_thread = (a.V + kThreads - 1) / kThreads;
    const int i0 = min(a.V, tid * per_thread), i1 = min(a.V, i0 + per_thread);
    int32_t n = 0;
    for (int i = i0; i < i1; ++i) n += key_of(p[i]) == pick_key;
    const Scan s = block_scan(n, 0, sh);
    if (s.count <= want && want < s.count + n) {
        int32_t left = want - s.count;
        int i = i0;
        for (;; ++i)
            if (key_of(p[i]) == pick_key && left-- == 0) break;
        a.pick[row] = i;
        if (a.prob) a.prob[row] = prob;
        a.flag[row] = 0;
    }
}

}  // namespace
}  // namespace tf

extern "C" int tf_sample_rows(const void* logits, int R, int V, int64_t row_stride, const float* temperature,
                              const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                              int32_t* pick, float* prob, uint8_t* flag, tf_cuda_stream stream) {
    using namespace tf;
    if (R < 0) return TF_EINVAL;
    if (R == 0) return TF_OK;
    if (!logits || !u || !pick || !flag || V < 1 || row_stride < V) return TF_EINVAL;
    if (V > TF_SAMPLE_MAX_VOCAB || R > (1 << 24)) return TF_ERANGE;
    int bits = 0;
    while ((int64_t(1) << bits) < V) ++bits;
    const Args a = {static_cast<const uint16_t*>(logits), row_stride, temperature, top_k, top_p, min_p, u,
                    pick, prob, flag, V, 63 - bits};
    return launch_pdl(sample_rows_kernel, dim3(R), dim3(kThreads), 0, stream, a);
}
