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
// not matter) and the weights are 64-bit fixed point. A row has as many fraction
// bits as its whole mass M leaves room for, 63 - ceil(log2 M) or up to two fewer (M
// from 1, its largest value's weight, to V; a rough float sum over the counts says
// which). With bits for M = V a peak before a long flat tail would have its borders
// off by up to V^2 2^-64 (2^-26 at 2^19 tokens); with its own a weight is off by
// M 2^-61 at most and a border by V 2^-59 of the kept mass, the weights below 2^-62,
// which are 0, among it (9e-13 at 2^19 tokens).
//
// One pass over a row: its tokens are counted as they arrive, in a folded
// window of both signs' magnitudes (2^-33, 128) and zero, which needs no maximum
// first; the largest occupied value is the maximum. A row with any other finite
// value (one N(0, 3) row in 250,000) is counted again in windows of 10,240
// consecutive values from its largest down, unless what is outside has no weight
// (a mask by a large negative number). A second pass, from L2, finds the
// picked value's j-th token.
//
// A row is shared by a cluster of 1 to 8 CTAs. Each counts a part of the
// tokens, then sums one slice of the sorted values over the cluster
// (distributed shared memory), weighs it, and every CTA learns the slices'
// totals: all of them follow the same steps with the same numbers.
//
// Measured on a GB300 (1,024 rows of 128,000 N(0, 3) logits): 102 us, 2.6 TB/s,
// 38 % of the copy rate; with half of the tokens masked 100. A CTA's row takes
// 53,000 cycles, two CTAs an SM, of which the count is 24,000 (HBM and
// shared-memory atomics), the weights 9,000, the search 9,000, the rough mass some
// 1,200. 16 rows, 4 CTAs each: 15.2 us, 18.1 with top-k, top-p and min-p, a chain
// of latencies.
#include <cfloat>
#include <cmath>

#include <cooperative_groups.h>

#include "tf_internal.cuh"

namespace cg = cooperative_groups;

namespace tf {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;                       // 16-byte loads a thread asks for at a time
constexpr int kSide = 5120;                      // positions a side of the sorted window
constexpr int kTopMag = 0x42FF;                  // the folded window's largest magnitude, just below 128
constexpr int kLowMag = kTopMag - kSide + 2;     // and its smallest, just above 2^-33: kSide - 1 of them
constexpr int kValues = 2 * kSide;               // sorted positions of a window
constexpr int kGroup = 8;                        // of which a thread weighs so many at a time
constexpr int kMaxWindows = 2 * 0x7F80 / kValues + 2;
constexpr int kMinKey = -0x7F80;                 // the key of -infinity: a masked token
constexpr int kInfKey = 0x7F80;
constexpr int kBadKey = 0x10000;                 // stands for a NaN or +infinity
constexpr int kMaxCluster = 8;
static_assert((kLowMag - 1) % 128 == 0 && kSide % kGroup == 0 && kValues % (kGroup * kMaxCluster) == 0 && kSide <= 8192, "");

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

// 2^-y in units of 2^-frac for y in units of 2^-52: the integer part shifts, the
// next two groups of six bits look up, and the rest, r < 2^-12, is
// 1 - a + a^2/2 - a^3/6 with a = r ln 2 (the next term is below 2^-54).
constexpr u64 kYLimit = u64(62) << 52;   // beyond it a weight is 0
__device__ __forceinline__ u64 weight(u64 y, int frac, const ExpTables& tab) {
    if (y >= kYLimit) return 0;
    const u64 a = __umul64hi(y << 24, 0xB17217F7D1CF79ABull) >> 12;   // r ln 2 in units of 2^-64
    const uint32_t ah = uint32_t(a >> 20);                             // < 2^32, in units of 2^-44
    const uint32_t a2 = __umulhi(ah, ah);                              // a^2 in units of 2^-56
    const uint32_t a3 = __umulhi(a2, ah);                              // a^3 in units of 2^-68
    const u64 poly = (u64(1) << 63) - (a >> 1) + (u64(a2) << 6) - (a3 / 12 >> 4);
    const u64 c = tab.coarse[(y >> 46) & 63], f = tab.fine[(y >> 40) & 63];
    const u64 w = __umul64hi(__umul64hi(c, f) << 1, poly) << 1;        // 2^-(fraction of y), units of 2^-63
    const int shift = 63 - frac + int(y >> 52);
    return shift > 63 ? 0 : (w + (u64(1) << shift >> 1)) >> shift;
}

__device__ __forceinline__ float exp2_of(float x) {   // 2^x, good to 2^-22 of it, for the rough mass
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Values are handled as keys, signed magnitudes: -0 is +0 and keys rise with values.
__device__ __forceinline__ int key_of(uint32_t bits) {
    const int mag = int(bits & 0x7FFFu);
    return bits & 0x8000u ? -mag : mag;
}
__device__ __forceinline__ float float_of(int key) {
    const float v = __uint_as_float(uint32_t(key < 0 ? -key : key) << 16);
    return key < 0 ? -v : v;
}
__device__ __forceinline__ double value_of(int key) { return double(float_of(key)); }
// A folded window's value in units of 2^-40 (0, or 8 significant bits shifted by up to 39).
__device__ __forceinline__ long long fixed_of(int key) {
    const int mag = key < 0 ? -key : key;
    const long long x = mag ? (long long)((mag & 0x7F) | 0x80) << ((mag >> 7) - (kLowMag >> 7)) : 0;
    return key < 0 ? -x : x;
}

// Sorted positions, largest value first. Folded: the positive magnitudes, zero
// at kSide - 1, (kSide is empty,) the negative ones. Otherwise kValues
// consecutive keys from `top` down.
template <bool kFold>
__device__ __forceinline__ int key_at(int pos, int top) {
    if constexpr (!kFold) return top - pos;
    if (pos < kSide) return pos == kSide - 1 ? 0 : kTopMag - pos;
    return kSide + 1 - kLowMag - pos;
}
// The histogram's word of a position: downwards from word kSide - 1, then
// upwards from word 8,192, so that a folded token's byte offset is its
// magnitude above kLowMag - 1 times 4, its sign as bit 15, and zero's is 0. The
// gap between holds the rest of the shared memory's contents.
__device__ __forceinline__ int word_of(int pos) { return pos < kSide ? kSide - 1 - pos : 8192 - kSide + pos; }

// What a row's settings give: log2(e) / T, as a double and as a 64-bit fraction
// with its product's shifts, -log2(min_p) in units of 2^-52, and top_p and u in
// units of 2^-64 (cut there). Doubles run at a 64th of the fp32 rate and so do
// conversions to and from 64 bits, so one warp works these out while the others count.
struct Setting {
    double per;
    u64 mant, y_min, p, u;
    int shift;   // left, before the product (the low 8 bits), and right, after it
    float per_f;
};
__device__ __forceinline__ Setting setting_of(float T, float top_p, float min_p, float u) {
    Setting s = {0.0, 0, kYLimit, __float2ull_rz(fmaxf(top_p, 0.f) * 0x1p64f), __float2ull_rz(u * 0x1p64f), 15, 0.f};
    if (T > 0.f) {
        s.per = 1.4426950408889634074 / double(T);
        s.per_f = fminf(float(s.per), FLT_MAX);
        // y 2^52 = d 2^12 per = d mant 2^(e - 64), d the difference in units of 2^-40
        int e;
        s.mant = u64(frexp(s.per * 4096.0, &e) * 0x1p64);
        // d goes up by e + 5, so that the product's upper half holds all of y's 58 bits and 5 more
        // (15 for T above 5.8: any difference, 2^49 at most, fits)
        const int up = max(15, min(e + 5, 63));
        s.shift = up | max(0, up - e) << 8;
    }
    if (min_p > 0.f) {
        const double y = -log2(double(min_p));
        if (y < 62.0) s.y_min = __double2ull_rz(y * 0x1p52);
    }
    return s;
}

// y = (max - x) log2(e) / T of a key, in units of 2^-52.
struct Scale {
    double vmax, per;     // any value
    long long xmax;       // folded window: the difference is an integer
    u64 mant;
    int shift, top_key;
    __device__ __forceinline__ Scale any(const Setting& s) const {
        return {value_of(top_key), s.per, xmax, mant, shift, top_key};
    }
    __device__ __forceinline__ u64 y_of(u64 d) const {   // of a difference, cut to whole units
        const int up = shift & 255, right = shift >> 8;
        if (d >> (64 - up)) return kYLimit;
        const u64 p = __umul64hi(d << up, mant);
        return right > 63 ? 0 : p >> right;
    }
    template <bool kFold>
    __device__ __forceinline__ u64 y(int key) const {
        if constexpr (kFold) return y_of(u64(xmax - fixed_of(key)));
        const double v = (vmax - value_of(key)) * per;
        return v < 62.0 ? __double2ull_rz(v * 0x1p52) : kYLimit;
    }
};
__device__ __forceinline__ Scale scale_of(int top_key, bool fold, const Setting& s) {
    return {0.0, 0.0, fold ? fixed_of(top_key) : 0, s.mant, s.shift, top_key};   // any(): for the rows that need it
}

// The floor of a part of m, f in units of 2^-64, and the ceiling.
__device__ __forceinline__ u64 part_of(u64 f, u64 m) { return __umul64hi(f, m); }
__device__ __forceinline__ u64 part_up(u64 f, u64 m) { return __umul64hi(f, m) + (f * m != 0); }

// n / d for a quotient below 2^34: a float quotient, its remainder's, and a last step of one.
__device__ __forceinline__ u64 quotient(u64 n, u64 d) {
    const float inv = 1.f / __ull2float_rn(d);
    u64 q = __float2ull_rz(__ull2float_rn(n) * inv);
    q += (long long)(__ll2float_rn((long long)(n - q * d)) * inv);
    const long long rest = (long long)(n - q * d);
    return rest < 0 ? q - 1 : u64(rest) >= d ? q + 1 : q;
}

struct Shared {
    uint32_t above[4];        // the window's words for positive tokens outside
    ExpTables tab;
    Setting set;
    u64 ratio[kSide / 128];   // folded: the weight of one step of each power of two, in units of 2^-63
    u64 warp_mass[kWarps];
    int32_t warp_int[3][kWarps];
    // what the cluster's CTAs tell one another, by rank
    u64 mass[kMaxCluster];
    int32_t first[kMaxCluster], count[kMaxCluster], other[kMaxCluster], found[kMaxCluster];
    float part[kMaxCluster];   // of the row's rough mass
    u64 min_p_mass;         // mass kept by min-p
    // the token that find() found: its value, its number among the value's tokens and the mass up to its end
    int32_t hit_key, hit_rank;
    u64 hit_mass;
    // what one thread keeps for the end
    Scale scale;
    u64 kept;
    int32_t pick_key, fold, frac;
    u64 before[kValues / kGroup + 1];   // the mass before each group of the slice, and its whole
};
static_assert(kSide * 4 + sizeof(Shared) <= 32768, "the gap");
// Behind the histogram: its words for negative tokens outside, and the windows of
// a row outside the folded one.
struct Windows {
    uint32_t above[4];
    u64 mass_before[kMaxWindows + 1];
    int32_t top[kMaxWindows], count_before[kMaxWindows];
};
constexpr int kSmemBytes = 32768 + kSide * 4 + int(sizeof(Windows));

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
    int32_t chunk;       // tokens a CTA of the cluster counts, a multiple of 8
};

// f(16 bytes, 8 tokens) and f1(bits) for the rest of a row's [begin, end): the
// tokens before the first 16-byte boundary and after the last (`head` and 8 of
// them at most).
template <typename F, typename F1>
__device__ __forceinline__ void for_tokens(const uint16_t* p, int begin, int end, int head, F&& f, F1&& f1) {
    const int body = min(end, begin + head), nvec = (end - body) >> 3;
    const uint4* pv = reinterpret_cast<const uint4*>(p + body);
    // the next vectors are asked for before the ones at hand are used
    uint4 v[kUnroll], next[kUnroll];
    auto load = [&](uint4 (&x)[kUnroll], int i) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            if (i + u * kThreads < nvec) x[u] = __ldg(pv + i + u * kThreads);
    };
    load(v, threadIdx.x);
#pragma unroll 1
    for (int i = threadIdx.x; i < nvec; i += kUnroll * kThreads) {
        load(next, i + kUnroll * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (i + u * kThreads >= nvec) break;
            f(v[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) v[u] = next[u];
    }
    const int tail = body + nvec * 8, t = int(threadIdx.x);
    if (t < body - begin) f1(uint32_t(p[begin + t]));
    if (t < end - tail) f1(uint32_t(p[tail + t]));
}

// Counts into the folded window; `other` becomes the largest value outside it
// (NaN and +infinity as kBadKey), masked tokens aside.
__device__ __forceinline__ int count_one(uint32_t* hist, uint32_t b, int other) {
    const int d = int(b & 0x7FFFu) - kLowMag;
    if (uint32_t(d) < uint32_t(kSide - 1)) {
        atomicAdd(hist + (b & 0x8000u ? 8193 + d : 1 + d), 1u);
    } else if (b != 0xFF80u) {
        const int k = key_of(b);
        if (k == 0) atomicAdd(hist, 1u);
        else other = max(other, k >= kInfKey || k < kMinKey ? kBadKey : k);
    }
    return other;
}
// The magnitudes of a word's two tokens above kLowMag, modulo 2^16: kSide - 1 or
// more for a token outside the window.
__device__ __forceinline__ uint32_t above_low(uint32_t w) {
    return __vadd2(w & 0x7FFF7FFFu, uint32_t(0x10000 - kLowMag) * 0x10001u);
}
constexpr uint32_t kOutside = uint32_t(kSide - 1) * 0x10001u;
// Counts both, those outside in a word behind their side's positions, so that masked tokens cost no branch.
__device__ __forceinline__ void count_word(unsigned char* dyn, uint32_t w, uint32_t d) {
    const uint32_t e = (w & 0x80008000u) | __vminu2(d, kOutside) << 2;   // byte offsets less 4
    atomicAdd(reinterpret_cast<uint32_t*>(dyn + (e & 0xFFFFu) + 4), 1u);
    atomicAdd(reinterpret_cast<uint32_t*>(dyn + (e >> 16) + 4), 1u);
}
// Of a word with a token outside: finite ones from -128 down, and masked ones,
// are 0 to kMasked here, in order of their magnitudes, all others more.
constexpr uint32_t kMasked = 0xFF80 - 0xC300;
__device__ __forceinline__ uint32_t below_low(uint32_t w) { return __vadd2(w, (0x10000u - 0xC300u) * 0x10001u); }
// 8 tokens' part in `other`, and their zeros.
__device__ __noinline__ int count_odd(uint4 v, int other) {
    extern __shared__ __align__(128) unsigned char dyn[];
#pragma unroll 1
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = v.x & 0xFFFFu;
        if ((above_low(b) & 0xFFFFu) >= kSide - 1) other = count_one(reinterpret_cast<uint32_t*>(dyn), b, other);
        v.x = k & 1 ? v.y : v.x >> 16;
        if (k & 1) v.y = v.z, v.z = v.w;
    }
    return other;
}

// The tokens of [i, i + 8) that lie in [begin, end) one by one, `none` in the place of the others.
__device__ __noinline__ uint4 load_part(const uint16_t* p, int i, int begin, int end, uint32_t none) {
    uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        x[k / 2] |= ((i + k >= begin && i + k < end ? uint32_t(p[i + k]) : none) & 0xFFFFu) << 16 * (k & 1);
    return make_uint4(x[0], x[1], x[2], x[3]);
}

// One CTA's part in its row. Every step that ends in sync() is taken by all
// threads of all CTAs of the cluster, with the same numbers.
struct Row {
    const Args& a;
    unsigned char* dyn;
    Shared& sh;
    int ncl, rank;
    int begin, end;      // this CTA's tokens,
    int head;            // and those of them before a 16-byte boundary
    int s0, s1;          // and its slice of the sorted positions
    const uint16_t* p;
    float tp;
    int32_t K;
    int top_key;
    int frac;            // fraction bits of the row's weights

    __device__ __forceinline__ uint32_t* hist() const { return reinterpret_cast<uint32_t*>(dyn); }
    __device__ __forceinline__ u64* before() const { return sh.before; }
    __device__ __forceinline__ void sync() const {
        if (ncl > 1) cg::this_cluster().sync();
        else __syncthreads();
    }
    // the block's value v (the same in every thread) into every CTA's `mine`; called by all threads
    template <typename X>
    __device__ __forceinline__ void tell(X& mine, X v) const {
        if (int(threadIdx.x) < ncl) *cg::this_cluster().map_shared_rank(&mine, threadIdx.x) = v;
    }
    // one thread's value into every CTA's `mine`
    template <typename X>
    __device__ __forceinline__ void tell_alone(X& mine, X v) const {
#pragma unroll 1
        for (int r = 0; r < ncl; ++r) *cg::this_cluster().map_shared_rank(&mine, r) = v;
    }

    __device__ __forceinline__ void clear() const {
        uint4* h = reinterpret_cast<uint4*>(dyn);
#pragma unroll 1
        for (int i = threadIdx.x; i < kSide / 2; i += kThreads)
            h[i < kSide / 4 ? i : 2048 + i - kSide / 4] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    // The counts of group g of the slice, in sorted order; whether there are any.
    __device__ __forceinline__ bool load_group(int g, uint32_t (&n)[kGroup]) const {
        const int pos = s0 + kGroup * g;
        const bool down = pos < kSide;   // the group's words run down, or up
        uint32_t any = 0;
#pragma unroll
        for (int k = 0; k < kGroup / 4; ++k) {
            const uint4 c = *reinterpret_cast<const uint4*>(hist() + (down ? word_of(pos + 4 * k) - 3 : word_of(pos + 4 * k)));
            n[4 * k] = down ? c.w : c.x;
            n[4 * k + 1] = down ? c.z : c.y;
            n[4 * k + 2] = down ? c.y : c.z;
            n[4 * k + 3] = down ? c.x : c.w;
            any |= c.x | c.y | c.z | c.w;
        }
        return any != 0;
    }
    __device__ __forceinline__ int groups() const { return (s1 - s0) / kGroup; }

    // The weight of a value relative to that of one not below it.
    __device__ __forceinline__ float relative(float from, float to) const { return exp2_of((to - from) * sh.set.per_f); }
    // The mass of a folded group's n tokens (c, by position) relative to the weight of the value
    // `ref`, that of `first`, the first occupied position here or in an earlier group. Where the
    // group's weights are within a factor of 2, all get the largest; otherwise, as its values are
    // equal steps apart (zero aside), a polynomial in the step's weight, from the last position up.
    __device__ __forceinline__ float group_mass(int pos, int first, float ref, int n,
                                                const uint32_t (&c)[kGroup]) const {
        const int key = key_at<true>(pos, 0);
        const float from = fminf(ref, float_of(key));   // position max(pos, first)'s value
        const float step = __uint_as_float((uint32_t(abs(key)) >> 7) - 7 << 23) * sh.set.per_f;
        float m = float(n);
        if (7.f * step > 1.f || pos == kSide - kGroup) {
            const float w = exp2_of(-step);
            m = 0.f;
#pragma unroll
            for (int j = kGroup - 1; j >= 0; --j) {
                if (pos + j < first) continue;
                m *= w;
                if (pos + j != kSide - 1) m += float(c[j]);
            }
            if (pos == kSide - kGroup) m += float(c[kGroup - 1]) * relative(from, 0.f);
        }
        return m * relative(ref, from);
    }
    // The warp's sum of masses m, each relative to the weight of its lane's value v, relative to `top`'s.
    __device__ __forceinline__ uint32_t rough_sum(float m, float v, float top) const {
        return __reduce_add_sync(0xFFFFFFFFu, __float2uint_ru(m * relative(top, v)));
    }

    // After the count: sums the slice over the cluster and surveys it. The
    // window's first occupied position and tokens, the largest of every
    // thread's `other`, and (folded) the tokens' mass, of which the first position's
    // tokens have 1 each: too large by a factor of 2 1/4 at most, too small by 2^-14 of it.
    struct Survey {
        int first, count, other;
        float mass;
    };
    template <bool kFold>
    __device__ __forceinline__ Survey survey(int other) const {
        sync();
        if (ncl > 1) {
#pragma unroll 1
            for (int i = s0 / 4 + int(threadIdx.x); i < s1 / 4; i += kThreads) {
                const int w4 = min(word_of(4 * i), word_of(4 * i + 3)) / 4;   // 4 positions are 4 words
                uint4 c = reinterpret_cast<uint4*>(hist())[w4], o[kMaxCluster];
#pragma unroll
                for (int r = 1; r < kMaxCluster; ++r) {   // every peer's words asked for before any is used
                    const int peer = rank + r < ncl ? rank + r : rank + r - ncl;
                    o[r] = make_uint4(0, 0, 0, 0);
                    if (r < ncl) o[r] = reinterpret_cast<uint4*>(cg::this_cluster().map_shared_rank(hist(), peer))[w4];
                }
#pragma unroll
                for (int r = 1; r < kMaxCluster; ++r) {
                    c.x += o[r].x;
                    c.y += o[r].y;
                    c.z += o[r].z;
                    c.w += o[r].w;
                }
                reinterpret_cast<uint4*>(hist())[w4] = c;
            }
            __syncthreads();
        }
        int first = kValues, n = 0;
        float mass = 0.f, ref = -INFINITY;   // the thread's, relative to its first position's value
#pragma unroll 1
        for (int g = int(threadIdx.x); g < groups(); g += kThreads) {
            uint32_t c[kGroup];
            if (!load_group(g, c)) continue;
            int in_group = 0;
#pragma unroll
            for (int j = kGroup - 1; j >= 0; --j) {
                in_group += c[j];
                if (c[j]) first = min(first, s0 + kGroup * g + j);
            }
            n += in_group;
            if constexpr (kFold) {
                if (mass == 0.f) ref = float_of(key_at<true>(first, 0));
                mass += group_mass(s0 + kGroup * g, first, ref, in_group, c);
            }
        }
        first = __reduce_min_sync(0xFFFFFFFFu, first);
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        other = __reduce_max_sync(0xFFFFFFFFu, other);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float top = -INFINITY;
        uint32_t rough = 0;   // the sums in units of 2^-12, rounded up
        if constexpr (kFold) {
            if (first < kValues) top = float_of(key_at<true>(first, 0));
            rough = rough_sum(mass * 4096.f, ref, top);
        }
        if (lane == 0) {
            sh.warp_int[0][warp] = first;
            sh.warp_int[1][warp] = n;
            sh.warp_int[2][warp] = other;
            if constexpr (kFold) sh.warp_mass[warp] = u64(__float_as_uint(top)) << 32 | rough;
        }
        __syncthreads();
        Survey s;
        const int theirs = sh.warp_int[0][lane % kWarps];
        s.first = __reduce_min_sync(0xFFFFFFFFu, theirs);
        s.mass = 0.f;
        if constexpr (kFold) {
            const u64 x = sh.warp_mass[lane % kWarps];
            const float m = lane < kWarps ? float(uint32_t(x)) : 0.f, v = __uint_as_float(uint32_t(x >> 32));
            if (s.first < kValues) top = float_of(key_at<true>(s.first, 0));
            s.mass = float(rough_sum(m, v, top)) * 0x1p-12f;
        }
        s.count = __reduce_add_sync(0xFFFFFFFFu, lane < kWarps ? sh.warp_int[1][lane] : 0);
        s.other = __reduce_max_sync(0xFFFFFFFFu, sh.warp_int[2][lane % kWarps]);
        if (ncl == 1) {
            if (threadIdx.x == 0) sh.count[0] = s.count;
            __syncthreads();
            return s;
        }
        tell(sh.first[rank], s.first);
        tell(sh.count[rank], s.count);
        tell(sh.other[rank], s.other);
        if constexpr (kFold) tell(sh.part[rank], s.mass);
        sync();
        s = {kValues, 0, kMinKey, 0.f};
#pragma unroll 1
        for (int r = 0; r < ncl; ++r) {
            s.first = min(s.first, sh.first[r]);
            s.count += sh.count[r];
            s.other = max(s.other, sh.other[r]);
        }
        if constexpr (kFold) {
            const float top = float_of(key_at<true>(s.first, 0));
#pragma unroll 1
            for (int r = 0; r < ncl; ++r)
                if (sh.first[r] < kValues)
                    s.mass += sh.part[r] * relative(top, float_of(key_at<true>(sh.first[r], 0)));
        }
        return s;
    }

    // before()[g] of every group of the slice (written, with the threads synchronised, by any
    // thread) into the sum of the groups before g; before()[groups()] becomes the whole.
    __device__ __forceinline__ u64 prefix() const {
        const int G = groups(), per = (G + kThreads - 1) / kThreads;
        const int g0 = min(G, int(threadIdx.x) * per), g1 = min(G, g0 + per);
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        u64 sum = 0;
#pragma unroll 1
        for (int g = g0; g < g1; ++g) sum += before()[g];
        u64 incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 t = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) sh.warp_mass[warp] = incl;
        __syncthreads();
        u64 w = sh.warp_mass[lane % kWarps];
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const u64 t = __shfl_up_sync(0xFFFFFFFFu, w, o, kWarps);
            if (lane % kWarps >= o) w += t;
        }
        const u64 total = __shfl_sync(0xFFFFFFFFu, w, kWarps - 1), prev = __shfl_sync(0xFFFFFFFFu, w, warp ? warp - 1 : 0);
        u64 at = (warp ? prev : 0) + incl - sum;
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
            const u64 v = before()[g];
            before()[g] = at;
            at += v;
        }
        if (threadIdx.x == 0) before()[G] = total;
        __syncthreads();
        return total;
    }

    // Cuts the slice's counts to the first K tokens (`counted` come before the window) and
    // weighs it: before() holds the mass before each group, relative to the slice's. The
    // window's mass, and the mass of the slices before this one in `slice_at`.
    template <bool kFold>
    __device__ __forceinline__ u64 weigh(const Scale& scale, int top, int32_t counted, u64& slice_at) const {
        uint32_t keep = ~0u;   // this thread's groups that top-k leaves tokens in, a bit a round
        u64 mine;
        // counts first where top-k may cut them, then masses
#pragma unroll 1
        for (int masses = K < a.V ? 0 : 1;; masses = 1) {
            uint32_t left_in = keep;
#pragma unroll 1
            for (int g = int(threadIdx.x); g < groups(); g += kThreads, left_in >>= 1) {
                u64 m = 0;
                uint32_t n[kGroup];
                if ((left_in & 1u) && load_group(g, n)) {
                    u64 w[kGroup];
                    if (masses) {
                        group_weights<kFold>(g, scale, top, w);
                    } else {
#pragma unroll
                        for (int j = 0; j < kGroup; ++j) w[j] = 1;
                    }
#pragma unroll
                    for (int j = 0; j < kGroup; ++j) m += n[j] * w[j];
                }
                before()[g] = m;
            }
            __syncthreads();
            mine = prefix();
            if (masses) break;
#pragma unroll 1
            for (int r = 0; r < rank; ++r) counted += sh.count[r];
            keep = 0;
#pragma unroll 1
            for (int g = int(threadIdx.x), bit = 0; g < groups(); g += kThreads, ++bit) {
                int32_t left = K - counted - int32_t(before()[g]);
                if (left <= 0) break;
                keep |= 1u << bit;
                if (left >= int32_t(before()[g + 1] - before()[g])) continue;
#pragma unroll 1
                for (int pos = s0 + kGroup * g; pos < s0 + kGroup * (g + 1); ++pos) {   // the K-th token's group
                    const int32_t c = int32_t(hist()[word_of(pos)]);
                    if (c > left) hist()[word_of(pos)] = uint32_t(left);
                    left -= min(c, left);
                }
            }
            __syncthreads();
        }
        slice_at = 0;
        if (ncl == 1) return mine;
        tell(sh.mass[rank], mine);
        sync();
        u64 total = 0;
#pragma unroll 1
        for (int r = 0; r < ncl; ++r) {
            if (r < rank) slice_at += sh.mass[r];
            total += sh.mass[r];
        }
        return total;
    }

    // The weights of group g's positions. A group of a folded window lies in one power of two
    // (the zero's aside), so its values are equal steps apart and each weight is the one before
    // times the step's, ratio[exponent]. Positions above the largest value hold no tokens.
    struct Weights {
        u64 x, ratio;     // a position's weight and the step's, in units of 2^-63
        int key, round;
    };
    template <bool kFold>
    __device__ __forceinline__ Weights first_weight(int pos, const Scale& scale, int top) const {
        const int key = key_at<kFold>(pos, top);
        return {weight(scale.y<kFold>(min(key, top_key)), 63, sh.tab),
                kFold ? sh.ratio[(abs(key) >> 7) - (kLowMag >> 7)] : 0, key, 63 - frac};
    }
    // The position's weight, and on to the next position's.
    template <bool kFold>
    __device__ __forceinline__ u64 next_weight(Weights& w, int pos, const Scale& scale) const {
        const u64 x = (w.x + (u64(1) << w.round >> 1)) >> w.round;
        --w.key;
        if constexpr (kFold) {
            if (w.key < top_key) w.x = __umul64hi(w.x, w.ratio) << 1;
            return pos == kSide - 1 ? zero_weight(scale) : x;
        }
        w.x = weight(scale.y<false>(min(w.key, top_key)), 63, sh.tab);
        return x;
    }
    template <bool kFold>
    __device__ __forceinline__ void group_weights(int g, const Scale& scale, int top, u64 (&w)[kGroup]) const {
        const int pos = s0 + kGroup * g;
        Weights at = first_weight<kFold>(pos, scale, top);
        if constexpr (kFold) {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                w[j] = (at.x + (u64(1) << at.round >> 1)) >> at.round;
                if (--at.key < top_key) at.x = __umul64hi(at.x, at.ratio) << 1;
            }
            if (pos == kSide - kGroup) w[kGroup - 1] = zero_weight(scale);
        } else {
#pragma unroll
            for (int j = 0; j < kGroup; ++j) w[j] = 0;
#pragma unroll 1
            for (int j = 0; j < kGroup; ++j) {   // a register a turn
                const u64 x = next_weight<false>(at, pos + j, scale);
#pragma unroll
                for (int i = 0; i + 1 < kGroup; ++i) w[i] = w[i + 1];
                w[kGroup - 1] = x;
            }
        }
    }
    __device__ __forceinline__ u64 zero_weight(const Scale& scale) const {
        return weight(scale.y<true>(min(0, top_key)), frac, sh.tab);
    }

    // The token whose masses (before, after] hold m into every CTA's hit_*, by the one thread that
    // holds it; `at` precedes the slice. A sync() has to follow. (The division by all threads took
    // 4,500 cycles.)
    template <bool kFold>
    __device__ __forceinline__ void find(u64 m, u64 at, const Scale& scale, int top) const {
        if (m <= at || m > at + before()[groups()]) return;
#pragma unroll 1
        for (int g = int(threadIdx.x); g < groups(); g += kThreads) {
            if (!(at + before()[g] < m && m <= at + before()[g + 1])) continue;
            const int pos = s0 + kGroup * g;
            Weights next = first_weight<kFold>(pos, scale, top);
            u64 x = at + before()[g];
#pragma unroll 1
            for (int j = 0; j < kGroup; ++j) {
                const u64 w = next_weight<kFold>(next, pos + j, scale), x1 = x + hist()[word_of(pos + j)] * w;
                if (m <= x1) {
                    tell_alone(sh.hit_key, key_at<kFold>(pos + j, top));
                    const u64 n = quotient(m - 1 - x, w);
                    tell_alone(sh.hit_rank, int32_t(n));
                    tell_alone(sh.hit_mass, x + (n + 1) * w);
                    break;
                }
                x = x1;
            }
        }
    }
    // The mass that a top-p prefix has at least.
    __device__ __forceinline__ u64 least_of(u64 Z) const { return max(u64(1), part_up(sh.set.p, Z)); }
    // The mass of the window's values with y <= y_min, and what precedes it, into every
    // CTA's min_p_mass: the last such position is found by bisection (y rises with positions)
    // in the slice that holds it; `Z` is the mass up to the window's end.
    template <bool kFold>
    __device__ __forceinline__ void min_p_cut(u64 Z, u64 at, const Scale& scale, int top) const {
        if (threadIdx.x >= 32) return;
        const u64 y_min = sh.set.y_min;
        auto keeps = [&](int pos) {
            const int key = key_at<kFold>(pos, top);
            return key >= top_key || (key >= kMinKey && scale.y<kFold>(key) <= y_min);
        };
        int lo = 0;   // positions below lo are kept; 32 looked at a time, 320, 10 and 1 apart
#pragma unroll 1
        for (int step = kValues / 32; step; step = step == 1 ? 0 : step / 32 > 1 ? step / 32 : 1) {
            const int pos = lo + int(threadIdx.x) * step;
            const bool k = pos < kValues && keeps(pos);
            const uint32_t kept = __ballot_sync(0xFFFFFFFFu, k);
            if (step > 1) lo += kept ? (31 - __clz(kept)) * step : 0;   // the last kept one
            else lo += __popc(kept);
        }
        if (threadIdx.x != 0) return;
        if (lo == kValues) {   // all of it: the last CTA's to tell
            if (rank == ncl - 1) tell_alone(sh.min_p_mass, Z);
            return;
        }
        if (lo < s0 || lo >= s1) return;
        const int g = (lo - s0) / kGroup, pos = s0 + kGroup * g;
        Weights next = first_weight<kFold>(pos, scale, top);
        u64 x = at + before()[g];
#pragma unroll 1
        for (int j = 0; pos + j < lo; ++j) x += hist()[word_of(pos + j)] * next_weight<kFold>(next, pos + j, scale);
        tell_alone(sh.min_p_mass, min(x, at + before()[g + 1]));   // a group past the K-th token weighs nothing
    }

    // The counts of the window of kValues keys from `top` down, surveyed: `other` is the largest key below it.
    __device__ __forceinline__ Survey count_window(int top) const {
        sync();   // every CTA is done with the counts so far
        clear();
        int below = kMinKey;
        auto one = [&](uint32_t b) {
            const int k = key_of(b);
            if (k > top || k == kMinKey) return;
            if (top - k < kValues) atomicAdd(hist() + word_of(top - k), 1u);
            else below = max(below, k);
        };
        for_tokens(p, begin, end, head, [&](uint4 v) {
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                one(v.x & 0xFFFFu);
                one(v.x >> 16);
                v = make_uint4(v.y, v.z, v.w, 0);
            }
        }, one);
        return survey<false>(below);
    }

};

// The fraction bits of a row of rough mass m (1 or more): m 2^frac <= 2^63, so that half
// a unit more for each of its tokens passes no 2^64.
__device__ __forceinline__ int frac_of(float m) {
    return 63 + 126 - (__float_as_int(m * (1.f + 0x1p-8f)) >> 23);
}

// The mass of all of a row's tokens, any values; for all threads of the cluster.
__device__ __noinline__ float mass_of_all(const Row R) {
    Shared& sh = R.sh;
    // log2(e) / T may not be a float, nor the difference of two values: parts and halves of them
    const bool tiny = sh.set.per > 0x1p64;
    const float per = float(tiny ? sh.set.per * 0x1p-64 : sh.set.per), up = tiny ? 0x1p64f : 1.f;
    const float half = 0.5f * float_of(R.top_key);
    float m = 0.f;
    auto one = [&](uint32_t b) {
        if (b == 0xFF80u) return;
        const float d = half - 0.5f * float_of(key_of(b));
        m += d > 0.f ? exp2_of(-2.f * (d * up * per)) : 1.f;
    };
    for_tokens(R.p, R.begin, R.end, R.head, [&](uint4 v) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            one(v.x & 0xFFFFu);
            one(v.x >> 16);
            v = make_uint4(v.y, v.z, v.w, 0);
        }
    }, one);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o; o /= 2) m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
    if (lane == 0) sh.warp_mass[warp] = __float_as_uint(m);
    __syncthreads();
    m = __uint_as_float(uint32_t(sh.warp_mass[lane % kWarps]));
#pragma unroll
    for (int o = kWarps / 2; o; o /= 2) m += __shfl_xor_sync(0xFFFFFFFFu, m, o);
    if (R.ncl == 1) return m;
    R.sync();   // the parts of the survey are read
    R.tell(sh.part[R.rank], m);
    R.sync();
    m = 0.f;
#pragma unroll 1
    for (int r = 0; r < R.ncl; ++r) m += sh.part[r];
    return m;
}

// A row outside the folded window: windows of kValues keys from its largest
// down. The kept mass; hit_* describe the pick at u of it. (Out of line, with its
// own copy of the row's variables, and one site of each step in its loop: few
// rows come here, and the others' code has to stay in the instruction caches.)
__device__ __noinline__ u64 general(const Row R, Scale scale, float mp) {
    Shared& sh = R.sh;
    Windows& win = *reinterpret_cast<Windows*>(R.dyn + 32768 + kSide * 4);
    scale = scale.any(sh.set);
    u64 slice_at = 0, Z = 0, kept = 0;
    int nw = 0, held = 0;
    bool building = true;
    int step = 0;
#pragma unroll 1
    for (int top = R.top_key, counted = 0; step < 3;) {
        // windows down to the K-th token; afterwards the one that a step needs
        const auto s = R.count_window(top);
        if (building && threadIdx.x == 0) {
            win.top[nw] = top;
            win.count_before[nw] = counted;
            win.mass_before[nw] = Z;
        }
        const u64 m = R.weigh<false>(scale, top, building ? counted : win.count_before[held], slice_at);
        if (building) {
            Z += m;
            counted += s.count;
            ++nw;
            if (s.other != kMinKey && counted < R.K) {
                top = s.other;
                continue;
            }
            building = false;
            held = nw - 1;
            kept = Z;
            if (threadIdx.x == 0) win.mass_before[nw] = Z;
            __syncthreads();
        }
        // the top-p cut, the min-p cut and the pick, each in the window that holds it
#pragma unroll 1
        for (; step < 3; ++step) {
            if ((step == 0 && !(R.tp < 1.f)) || (step == 1 && !(mp > 0.f))) continue;
            const u64 to = step == 0 ? R.least_of(Z) : part_of(sh.set.u, kept) + 1;
            int w = 0;
            if (step == 1) {   // the last window whose largest value is kept
                while (w + 1 < nw && scale.y<false>(win.top[w + 1]) <= sh.set.y_min) ++w;
            } else {
                while (win.mass_before[w + 1] < to) ++w;
            }
            if (held != w) {
                held = w;
                top = win.top[w];
                break;
            }
            const u64 at = win.mass_before[w] + slice_at;
            if (step == 1) R.min_p_cut<false>(win.mass_before[w + 1], at, scale, win.top[w]);
            else R.find<false>(to, at, scale, win.top[w]);
            R.sync();
            if (step < 2) kept = min(kept, step == 0 ? sh.hit_mass : sh.min_p_mass);
            R.sync();   // hit_* are read before the next find
        }
    }
    return kept;
}

// The row's prob and flag.
__device__ __noinline__ void report(const Args& a, int row, const Shared& sh) {
    float prob = 1.f;
    if (sh.kept) {
        // the weight's first 64 bits over the mass's first 32 (2^-31 of it off at most),
        // the remainder as the quotient's last bit, so that the one rounding sees it
        const u64 y = sh.fold ? sh.scale.y<true>(sh.pick_key) : sh.scale.any(sh.set).y<false>(sh.pick_key);
        const u64 w = weight(y, 63, sh.tab);
        const int wu = __clzll((long long)w), ku = __clzll((long long)sh.kept);
        const u64 den = (sh.kept << ku) >> 32, q = quotient(w << wu, den);
        prob = ldexpf(float(q | u64(q * den != w << wu)), ku - wu + sh.frac - 63 - 32);
    }
    if (a.prob) a.prob[row] = prob;
    a.flag[row] = 0;
}

__global__ void __launch_bounds__(kThreads, 2)
sample_rows_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) unsigned char dyn[];
    Shared& sh = *reinterpret_cast<Shared*>(dyn + kSide * 4);
    const int row = blockIdx.y, tid = threadIdx.x;
    const int ncl = gridDim.x, rank = blockIdx.x;   // a cluster is one row's CTAs
    const int slice = kValues / ncl;
    const uint16_t* p = a.logits + size_t(row) * size_t(a.stride);
    // the row's tokens before a 16-byte boundary are the first CTA's, the parts begin at boundaries
    const int skew = int(-reinterpret_cast<uintptr_t>(p) & 15u) / 2;
    const int begin = rank ? min(a.V, skew + rank * a.chunk) : 0;
    const int end = rank == ncl - 1 ? a.V : min(a.V, skew + (rank + 1) * a.chunk);
    Row R{a, dyn, sh, ncl, rank, begin, end, rank ? 0 : skew, rank * slice, (rank + 1) * slice, p, 1.f, a.V,
          kMinKey, 0};
    uint32_t* const hist = R.hist();
    if (tid < 64) {
        sh.tab.coarse[tid] = kExpTables.coarse[tid];
        sh.tab.fine[tid] = kExpTables.fine[tid];
    }
    R.clear();
    pdl_wait();
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const float tp = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f, u = a.u[row];
    const int32_t tk = a.top_k ? a.top_k[row] : 0;
    R.K = tk > 0 && tk < a.V ? tk : a.V;
    R.tp = tp;
    const bool bad_setting = !(T >= 0.f && T < INFINITY) || isnan(tp) || isnan(mp) || !(mp <= 1.f) ||
                             !(u >= 0.f && u < 1.f);
    if (tid >= kThreads - 32) {   // one warp; read after the count's barriers
        const Setting set = setting_of(T, tp, mp, u);
        const Scale step = scale_of(0, true, set);
        if (tid == kThreads - 32) sh.set = set;
#pragma unroll 1
        for (int e = tid % 32; e < kSide / 128; e += 32) sh.ratio[e] = weight(step.y_of(u64(1) << e), 63, kExpTables);
    }

    // ---- the first pass: the folded window
    int other = kMinKey;   // the largest value outside it
    for_tokens(
        p, begin, end, R.head,
        [&](const uint4& v) {
            const uint32_t d[4] = {above_low(v.x), above_low(v.y), above_low(v.z), above_low(v.w)};
            count_word(dyn, v.x, d[0]);
            count_word(dyn, v.y, d[1]);
            count_word(dyn, v.z, d[2]);
            count_word(dyn, v.w, d[3]);
            const uint32_t most = __vmaxu2(__vmaxu2(d[0], d[1]), __vmaxu2(d[2], d[3]));
            if (max(most & 0xFFFFu, most >> 16) < kSide - 1) return;
            uint32_t x[4] = {v.x, v.y, v.z, v.w}, below = ~0u;
            uint32_t odd = 0;   // its largest value is that of tokens outside which are not below
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                asm volatile("" : "+r"(x[k]));   // d is not kept for this branch: the registers cost 3 us
                const uint32_t b = below_low(x[k]);
                below = __vminu2(below, b);
                odd = __vmaxu2(odd, __vminu2(above_low(x[k]), kOutside) + __vminu2(b, (kMasked + 1) * 0x10001u));
            }
            below = min(below & 0xFFFFu, below >> 16);
            if (below < kMasked) other = max(other, -int(below + 0x4300));
            if (max(odd & 0xFFFFu, odd >> 16) == kSide + kMasked) other = count_odd(v, other);
        },
        [&](uint32_t b) { other = count_one(hist, b, other); });

    const auto found = R.survey<true>(other);
    const int most = found.first < kValues ? key_at<true>(found.first, 0) : kMinKey, top_key = max(most, found.other);
    // what lies outside does not matter if it has no weight, as a large negative number has
    // none (y >= 62; a row close to that is right either way)
    const bool fold = found.other == kMinKey ||
                      (most > found.other && (float_of(most) - float_of(found.other)) * sh.set.per_f > 62.1f);
    R.top_key = top_key;
    if (top_key == kBadKey || top_key == kMinKey || bad_setting) {
        if (tid == 0 && rank == 0) {
            a.pick[row] = -1;
            if (a.prob) a.prob[row] = 0.f;
            a.flag[row] = uint8_t((top_key == kBadKey || top_key == kMinKey ? TF_SAMPLE_NO_LOGITS : 0) |
                                  (bad_setting ? TF_SAMPLE_BAD_SETTING : 0));
        }
        return;   // the cluster's last exchange was the survey's
    }

    const Scale scale = scale_of(top_key, fold, sh.set);
    u64 kept = 0;
    int pick_key = top_key, want = 0;   // the pick: the want-th token (by id) of value pick_key
    if (T > 0.f) {
        R.frac = frac_of(fold ? found.mass : mass_of_all(R));
        if (fold) {
            u64 at;
            const u64 Z = R.weigh<true>(scale, 0, 0, at);
            kept = Z;
            if (mp > 0.f) R.min_p_cut<true>(Z, at, scale, 0);
            // the top-p cut, if there is one, and the pick
#pragma unroll 1
            for (int pick = tp < 1.f ? 0 : 1; pick < 2; ++pick) {
                if (pick && mp > 0.f) {
                    if (!(tp < 1.f)) R.sync();
                    kept = min(kept, sh.min_p_mass);
                }
                const u64 to = pick ? part_of(sh.set.u, kept) + 1 : R.least_of(Z);
                R.find<true>(to, at, scale, 0);
                R.sync();
                if (pick) break;
                kept = min(kept, sh.hit_mass);
                R.sync();   // hit_* are read before the next find
            }
        } else {
            kept = general(R, scale, mp);
        }
        pick_key = sh.hit_key;
        want = sh.hit_rank;
    }
    pdl_trigger();

    const int lane = tid & 31, warp = tid >> 5;
    if (tid == kThreads - 1) {   // for report(), below
        sh.scale = scale;
        sh.fold = fold;
        sh.frac = R.frac;
        sh.kept = T > 0.f ? kept : 0;
        sh.pick_key = pick_key;
    }

    // ---- the second pass: the want-th token of value pick_key, over the CTA's
    // tokens in chunks, a step of each warp's in turn, the next chunk's loads in
    // flight. A CTA alone in its row stops at the chunk that holds the token, half way
    // through the row on average; in a cluster each counts all of its chunks, and the
    // one that holds the token reads its step again.
    constexpr int kStep = kUnroll * 32 * 8, kChunk = kStep * kWarps;
    static_assert((TF_SAMPLE_MAX_VOCAB / kChunk + 2) * kWarps <= kSide, "the counts go over the histogram");
    const uint32_t bits = uint32_t(pick_key < 0 ? -pick_key | 0x8000 : pick_key), both = bits * 0x10001u;
    const __nv_bfloat162 ref = *reinterpret_cast<const __nv_bfloat162*>(&both);
    auto load = [&](uint4 (&v)[kUnroll], int i0) {
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + 256 * k + 8 * lane;
            v[k] = make_uint4(~both, ~both, ~both, ~both);   // which no pick equals
            if (i >= begin && i + 8 <= end) v[k] = __ldg(reinterpret_cast<const uint4*>(p + i));
            else if (i < end) v[k] = load_part(p, i, begin, end, ~bits);
        }
    };
    // a lane's 8 tokens that are the pick's value, a bit each
    auto hits = [&](const uint4& v) {
        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
        uint32_t m[4], h = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = __heq2_mask(*reinterpret_cast<const __nv_bfloat162*>(&x[k]), ref);
        if (m[0] | m[1] | m[2] | m[3]) {   // rarely
#pragma unroll
            for (int k = 0; k < 4; ++k) h |= (m[k] & 0x10001u) << 2 * k;
            h = (h | h >> 15) & 0xFFu;   // the high tokens' bits between the low ones'
        }
        return h;
    };
    int32_t* const counts = reinterpret_cast<int32_t*>(hist);   // [chunk][warp]; the histogram is done with
    const int from = R.head ? R.head - 8 : begin;   // a 16-byte boundary at or before the first token
    const int chunks = (end - from + kChunk - 1) / kChunk;
    int32_t before = 0;    // tokens of the value in the chunks so far
    int32_t left = -1;     // the pick is the left-th of this warp's tokens of the value in chunk `mine`
    int mine = 0;
    uint4 v[kUnroll], next[kUnroll];
    load(v, from + warp * kStep);
#pragma unroll 1
    for (int j = 0; j < chunks; ++j) {
        load(next, from + (j + 1) * kChunk + warp * kStep);
        int32_t c = 0;
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (const uint32_t h = hits(v[k])) c += __popc(h);
        c = __reduce_add_sync(0xFFFFFFFFu, c);
        if (lane == 0) counts[j * kWarps + warp] = c;
        if (ncl == 1) {
            __syncthreads();
            const int32_t x = lane < kWarps ? counts[j * kWarps + lane] : 0;
            const int32_t all = __reduce_add_sync(0xFFFFFFFFu, x);
            if (want < before + all) {
                left = want - before - __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0);
                if (left >= c) left = -1;
                mine = j;
                break;
            }
            before += all;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) v[k] = next[k];
    }
    if (ncl > 1) {
        __syncthreads();
        // this CTA's count; then the counts of the CTAs before it
        int32_t n = 0;
#pragma unroll 1
        for (int i = lane; i < chunks * kWarps; i += 32) n += counts[i];
        n = __reduce_add_sync(0xFFFFFFFFu, n);
        R.tell(sh.found[rank], n);
        R.sync();   // the last use of another CTA's memory
#pragma unroll 1
        for (int r = 0; r < rank; ++r) before += sh.found[r];
#pragma unroll 1
        for (; mine < chunks && left < 0; ++mine) {   // the warp whose step it is
            const int32_t x = lane < kWarps ? counts[mine * kWarps + lane] : 0;
            const int32_t at = before + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? x : 0);
            before += __reduce_add_sync(0xFFFFFFFFu, x);
            if (at <= want && want < at + __shfl_sync(0xFFFFFFFFu, x, warp)) {
                left = want - at;
                break;
            }
        }
    }
    if (tid == kThreads - 1 && rank == 0) report(a, row, sh);   // now, as the search's steps wait for every warp
    if (left < 0) return;
    load(v, from + mine * kChunk + warp * kStep);
#pragma unroll 1
    for (int k = 0; k < kUnroll; ++k) {
        uint32_t h = hits(v[0]);
#pragma unroll
        for (int j = 0; j + 1 < kUnroll; ++j) v[j] = v[j + 1];
        const int32_t c = __popc(h);
        int32_t upto = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
            if (lane >= o) upto += t;
        }
        if (left >= upto - c && left < upto) {
            for (int q = upto - c; q < left; ++q) h &= h - 1;
            a.pick[row] = from + mine * kChunk + warp * kStep + 256 * k + 8 * lane + __ffs(h) - 1;
        }
        left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
        if (left < 0) break;
    }
}

int prepare() {
    const cudaError_t r = cudaFuncSetAttribute(sample_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    return r == cudaSuccess ? TF_OK : cuda_fail(r);
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
    if (reinterpret_cast<uintptr_t>(logits) & 1) return TF_EINVAL;
    for (const void* x : {static_cast<const void*>(temperature), static_cast<const void*>(top_k),
                          static_cast<const void*>(top_p), static_cast<const void*>(min_p), static_cast<const void*>(u),
                          static_cast<const void*>(pick), static_cast<const void*>(prob)})
        if (reinterpret_cast<uintptr_t>(x) & 3) return TF_EINVAL;
    if (V > TF_SAMPLE_MAX_VOCAB || R > (1 << 24)) return TF_ERANGE;
    if (!on_this_device(logits)) return TF_EINVAL;
    int rc = prepare();
    if (rc != TF_OK) return rc;
    // CTAs a row: up to 8 while they have an SM each and 16,384 tokens each. 128,000 tokens, temperature alone, us
    // with 1, 2, 4 and 8: one row 18.1, 16.3, 13.8, 13.1; 16 rows 20.7, 17.9, 15.3, 17.4; 38 rows 21.5, 18.3, 19.7,
    // 30.5; 64 rows 21.6, 18.5, 20.9, 35.5; 100 rows 26.6, 25.5, 36.8, 52.6
    int cl = kMaxCluster;
    while (cl > 1 && (int64_t(R) * cl > sm_count() || V < cl * 16384)) cl /= 2;
    Args a = {static_cast<const uint16_t*>(logits), row_stride, temperature, top_k, top_p, min_p, u,
              pick, prob, flag, V, ((V + cl - 1) / cl + 7) / 8 * 8};

    // rows go in grid.y, at most 65,535 a launch
    constexpr int kRowsPerLaunch = 65535;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    for (int r0 = 0; r0 < R; r0 += kRowsPerLaunch) {
        const int nr = R - r0 < kRowsPerLaunch ? R - r0 : kRowsPerLaunch;
        cfg.gridDim = dim3(cl, nr, 1);
        Args b = a;
        b.logits += size_t(r0) * size_t(row_stride);
        for (const float** f : {&b.temperature, &b.top_p, &b.min_p, &b.u})
            if (*f) *f += r0;
        if (b.top_k) b.top_k += r0;
        b.pick += r0;
        if (b.prob) b.prob += r0;
        b.flag += r0;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, sample_rows_kernel, b);
        if (e != cudaSuccess) return cuda_fail(e);
        rc = launch_status();
        if (rc != TF_OK) return rc;
    }
    return TF_OK;
}
