// weight.cuh -- softmax weights as 64-bit integers, and the order of logits.
//
// weight(l) = exp((l - top) / T) in units of 2^-44, rounded to nearest: at most
// 2^44 for the top logit, so 2^19 tokens sum to at most 2^63.  Integer sums are
// exact and do not depend on their order.
//
// The exponential is table-driven (P. T. P. Tang, "Table-driven implementation
// of the exponential function in IEEE floating-point arithmetic", ACM TOMS 15,
// 1989): y = (l - top) log2(e) / T is split into n + j/1024 + g with |g| <=
// 2^-11, and 2^y = 2^n 2^(j/1024) (1 + a + a^2/2 + a^3/6), a = g ln 2.  Plain
// fp32 would lose the small differences (its 2^-24 times a vocabulary of
// borders is a wrong token every few dozen rows) and fp64 runs at 1/64 of the
// fp32 rate here, so the products carry their rounding errors in a second fp32
// (Dekker's and Knuth's error-free sums and products): about 35 fp32 and integer
// instructions per weight, its error below 2^-44.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace gdn {

constexpr uint32_t kNone = 0x007fffffu;       // the key of -inf: a token that cannot be drawn

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// NaN counts as masked, -0 as 0
template <typename L>
__device__ __forceinline__ float clean(L x) {
    const float f = to_float(x);
    return f != f ? -INFINITY : f + 0.0f;
}
// order-preserving 32-bit key of a float that is not NaN, and back
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// 2^(j/1024): x, y = low and high word of the integer nearest to it times 2^46, z, w = its fp32 head and tail
struct WeightRow {
    uint32_t lo, hi;
    float head, tail;
};

struct WeightRows {
    WeightRow r[1024];
};

// by the Taylor series of exp at compile time, in fp64 (the terms fall by 1/n of at most 0.69 each: 24 are ample)
constexpr WeightRows make_weight_rows() {
    WeightRows t{};
    for (int j = 0; j < 1024; ++j) {
        const double x = j * (0.693147180559945309417 / 1024);
        double term = 1, v = 1;
        for (int n = 1; n < 24; ++n) {
            term *= x / n;
            v += term;
        }
        const uint64_t i = uint64_t(v * 70368744177664.0 + 0.5);       // 2^46
        const float h = float(v);
        t.r[j] = {uint32_t(i), uint32_t(i >> 32), h, float(v - double(h))};
    }
    return t;
}

__device__ constexpr WeightRows kWeightRows = make_weight_rows();

struct __align__(16) WeightTable {
    uint4 r[1024];
    // by all threads of a block; a barrier follows before the first use
    __device__ __forceinline__ void fill(int tid, int n) {
        for (int i = tid; i < 1024; i += n) r[i] = reinterpret_cast<const uint4 *>(kWeightRows.r)[i];
    }
};

// log2(e) / T as an fp32 head and tail
struct Scale {
    float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float temp) {
    const double c = 1.4426950408889634074 / double(temp);
    const float h = float(c);
    return {h, float(c - double(h))};
}

__device__ __forceinline__ unsigned long long weight(float l, float top, Scale c, const WeightTable &tab) {
    if (l == top) return 1ull << 44;
    // l - top = s + e exactly
    const float s = l - top, b = s - l, e = (l - (s - b)) - (top + b);
    const float y = s * c.hi;
    if (!(y > -45.5f)) return 0;                             // below half a unit
    const float ye = fmaf(e, c.hi, fmaf(s, c.lo, fmaf(s, c.hi, -y)));
    // y = q + g, q a multiple of 1/1024 (1.5 * 2^13 has a last place of 2^-10); then g + ye as gh + gl
    const float t = y + 12288.0f, g = y - (t - 12288.0f);
    const int m = __float_as_int(t) - __float_as_int(12288.0f);
    const float gh = g + ye, gl = (g - gh) + ye;
    constexpr float L = 0.693147182464599609375f, Ll = -1.90465429995776804525e-9f;   // ln 2 = L + Ll
    const float a = gh * L, ae = fmaf(gl, L, fmaf(gh, Ll, fmaf(gh, L, -a)));
    const float tail = fmaf(a * a, fmaf(a, 0.16666667f, 0.5f), ae);
    const uint4 r = tab.r[m & 1023];
    const float th = __uint_as_float(r.z), tl = __uint_as_float(r.w);
    // th (1 + a + tail) - th = p + q
    const float p = th * a, q = fmaf(th, tail, fmaf(tl, a, fmaf(th, a, -p)));
    // p (below 2^-10) in units of 2^-32, the rest (below 2^-22) in units of 2^-44: the last places of 1.5 * 2^-9
    // and 1.5 * 2^-21
    constexpr float M1 = 0x1.8p-9f, M2 = 0x1.8p-21f;
    const float t1 = p + M1, t2 = ((p - (t1 - M1)) + q) + M2;
    const int i1 = __float_as_int(t1) - __float_as_int(M1), i2 = __float_as_int(t2) - __float_as_int(M2);
    const long long v = ((long long)(((unsigned long long)r.y << 32) | r.x)) + ((long long)i1 << 14) + ((long long)i2 << 2);
    // 2^46 -> units of 2^-44, times 2^n (n <= 0), to nearest
    const int sh = 2 - (m >> 10);
    return (unsigned long long)((v + (1ll << (sh - 1))) >> sh);
}

// ln(exp((l - top) / T) / (total 2^-44)), l - top and the logarithm in fp64: once per row
__device__ __forceinline__ float log_prob(float l, float top, float temp, unsigned long long total) {
    const double x = l == top ? 0.0 : (double(l) - double(top)) / double(temp);
    return float(x - (log(double(total)) - 44 * 0.693147180559945309417));
}

// the smallest integer mass that is at least p of total (at least one unit)
__device__ __forceinline__ unsigned long long mass_target(float p, unsigned long long total) {
    const double t = ceil(double(p) * double(total));
    const unsigned long long v = t < 1.0 ? 1ull : (unsigned long long)t;
    return v < total ? v : total;
}
// floor(u total): the token is the first whose running mass is above it
__device__ __forceinline__ unsigned long long draw_target(float u, unsigned long long total) {
    const unsigned long long v = __umul64hi((unsigned long long)(double(u) * 18446744073709551616.0), total);
    return v < total ? v : total - 1;
}
// the lowest key of a logit with exp((l - top) / T) >= min_p
__device__ __forceinline__ uint32_t min_p_key(float min_p, float temp, float top) {
    if (min_p >= 1.0f) return key_of(top);
    const double border = double(top) + double(temp) * log(double(min_p));
    float f = __double2float_ru(border);
    const uint32_t k = key_of(f + 0.0f), kt = key_of(top);
    return k < kt ? k : kt;
}
// temperature 0 (greedy) or in [2^-20, 2^20], top_p above 0, min_p at most 1; NaN is refused
__device__ __forceinline__ bool sample_params_ok(float temp, float p, float mp) {
    return (temp == 0.0f || (temp >= 0x1p-20f && temp <= 0x1p20f)) && p > 0.0f && mp <= 1.0f;
}

}  // namespace gdn
