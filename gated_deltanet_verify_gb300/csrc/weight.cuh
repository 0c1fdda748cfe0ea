// weight.cuh -- softmax weights as 64-bit integers, and the order of logits.
//
// weight(l) = exp((l - ref) / T) in units of 2^-44, rounded to nearest, where ref is the top logit or a little above:
// at most 2^44, so 2^19 tokens sum to at most 2^63.  Only ratios of weights count, so ref need not be exact.  Integer
// sums are exact and do not depend on their order.  (The choice of the unit: the sum of the largest vocabulary fits 64
// bits.  A weight below half a unit, e^-31.2 of the top one, is 0: with u = 0 too, such a token is not drawn, as the
// masked token that a logit of the type's lowest value stands for must not be.)
//
// The exponential is table-driven (P. T. P. Tang, "Table-driven implementation
// of the exponential function in IEEE floating-point arithmetic", ACM TOMS 15,
// 1989): y = (l - ref) log2(e) / T is split into n + j/1024 + g with |g| near
// 2^-11, and 2^y = 2^n 2^(j/1024) (1 + a + a^2/2 + a^3/6), a = g ln 2.  Plain
// fp32 would lose the small differences (its 2^-24 times a vocabulary of
// borders is a wrong token every few dozen rows) and fp64 runs at 1/64 of the
// fp32 rate here, so the products carry their rounding errors in a second fp32
// (Dekker's and Knuth's error-free sums and products), all of them only for
// weights above 2^-4 of the top one: about 22 instructions for the others, which
// take no sum of two for g and end the series at g^2.  Errors: 2^-43 of the top
// weight, 2^-38 for a few.  (Pairs of fp32 in one instruction, f32x2, took 4 %
// longer: the moves cost more.)  fp64 is kept out of what every thread does: one
// fp64 logarithm in all threads of a CTA costs microseconds.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace gdn {

constexpr uint32_t kNone = 0x007fffffu;       // the key of -inf: a token that cannot be drawn

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// order-preserving 32-bit key of a float that is neither NaN nor -0, and back
__device__ __forceinline__ uint32_t key_of(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// 2^(j/1024) = head (1 + rest), the head an fp32 number, of which j 2^13 is taken off as an integer: with 1024 n + j times
// 2^13 added again it is 2^n head (13 bits below the exponent's)
struct WeightRow {
    int head;
    float rest;
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
        const float h = float(v);                  // in [1, 2): its bits are those of 1 and 23 of (h - 1)
        t.r[j] = {0x3f800000 + int((double(h) - 1) * 8388608) - (j << 13), float((v - double(h)) / double(h))};
    }
    return t;
}

__device__ constexpr WeightRows kWeightRows = make_weight_rows();

struct __align__(16) WeightTable {
    WeightRow r[1024];
    // by all threads of a block; a barrier follows before the first use
    __device__ __forceinline__ void fill(int tid, int n) {
        for (int i = tid; i < 512; i += n)
            reinterpret_cast<uint4 *>(r)[i] = reinterpret_cast<const uint4 *>(kWeightRows.r)[i];
    }
};

// Below 2^kLarge of the top weight, rounding errors of 2^-34 of the weight are let be: they stay below 2^-38 of the top
// weight, and few tokens are near that (all tokens' errors together are near 10^-12 of the sum as a rule; at most
// 2^-34 of it, and 2^-45 of the top weight a token where all round the same way).  At -7, 128 rows of 100003 took 44.7 us,
// at -4 37.0: four tokens a thread share the branch, and seldom is none of 128 large.
constexpr float kLarge = -4.0f;

// What the weights of a row share: y = x c - at with x = l - shift, c = hi + lo = log2(e) / T, and `at` (top - shift) c
// rounded up to a multiple of 2^-10 (by one or two of them, so that y < 0).  With q a multiple of 2^-10 too, at + q is
// exact, and one fused multiply-add takes y - q from l without a difference of logits first.  Where (top - shift) c
// would be too large for that, the shift is the top logit; what counts there lies within 1/40 of it, so l - top is exact.
struct Scale {
    float hi, lo, shift, at, from;                 // from: 12288 - at, where y is rounded to q
    float least;                                   // an x whose weight rounds to 0; lower ones (and NaN) count as it
    float large;                                   // a little below the logits whose y is above kLarge
};
__device__ __forceinline__ Scale scale_of(float temp, float top) {
    constexpr float L = 1.44269502162933349609375f, Ll = 1.92596303350001e-8f;      // log2(e) = L + Ll
    Scale c;
    c.hi = __fdiv_rn(L, temp);                     // the quotient, and the rest of the division over T
    c.lo = __fdiv_rn(fmaf(-c.hi, temp, L) + Ll, temp);
    c.shift = c.at = 0.f;
    if (top == INFINITY) {
        c.shift = c.large = top;                   // only infinite logits are kept, all alike
        c.hi = c.lo = c.least = 0.f;
    } else {
        const float p = __fmul_rn(top, c.hi);
        if (fabsf(p) < 2048.f) c.at = (ceilf(p * 1024.f) + 1.f) * (1.f / 1024);
        else c.shift = top;
        c.least = (top - c.shift) - __fdiv_rn(46.5f, c.hi);
        c.large = __fsub_rd(top, __fdiv_ru(0.01f - kLarge, c.hi));
    }
    c.from = __fsub_rn(12288.0f, c.at);
    return c;
}

// hi * 2^22 + lo units of 2^-44, |lo| at most 2^21: up to 1000 of them add up word by word
struct Weight {
    uint32_t hi;
    int lo;
    __device__ __forceinline__ Weight &operator+=(const Weight &o) {
        hi += o.hi;
        lo += o.lo;
        return *this;
    }
    __device__ __forceinline__ unsigned long long units() const {
        return ((unsigned long long)hi << 22) + (long long)lo;
    }
};

// The weights of N logits (of a masked one: 0), `most` the largest of them.  A token's weight has to be the same wherever
// it is taken, so no product and sum here is left to the compiler to contract or not.  (Several at once, so that they
// share the branch around what only large ones need.)
template <int N>
__device__ __forceinline__ void weights(const float *l, float most, const Scale &c, const WeightTable &tab, Weight *w) {
    constexpr float M = 12288.0f;                  // 1.5 * 2^13: its last place is 2^-10
    constexpr float L = 0.693147182464599609375f, Ll = -1.90465429995776804525e-9f;   // ln 2 = L + Ll
    float x[N], t[N], h[N], lw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = fmaxf(__fsub_rn(l[i], c.shift), c.least);
        t[i] = fmaf(x[i], c.hi, c.from);
        const float at = __fsub_rn(t[i], c.from);  // at + q, exactly
        const int n = __float_as_int(t[i]);        // 1024 q is in its low bits: those of 12288 end in 22 zeros
        const WeightRow r = tab.r[n & 1023];
        const float rx = __int_as_float(r.head + (n << 13));
        // 2^g (1 + rest) = 1 + b to 2^-36, with g = y - q; the weight is rx (1 + b) = h + lw
        const float g = fmaf(x[i], c.lo, fmaf(x[i], c.hi, -at));
        const float b = fmaf(g, fmaf(g, 0.2402265f, L), r.rest);
        h[i] = fmaf(rx, b, rx);
        lw[i] = fmaf(rx, b, __fsub_rn(rx, h[i]));
    }
    if (most > c.large) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            // 2^g = 1 + b, b = a (1 + a / 2 + a^2 / 6) with a = g ln 2; g, a and b as sums of two
            const float at = __fsub_rn(t[i], c.from);
            const int n = __float_as_int(t[i]);
            const WeightRow r = tab.r[n & 1023];
            const float rx = __int_as_float(r.head + (n << 13));
            const float p = __fmul_rn(x[i], c.hi), g0 = __fsub_rn(p, at), ge = fmaf(x[i], c.lo, fmaf(x[i], c.hi, -p));
            const float gh = __fadd_rn(g0, ge), gl = __fadd_rn(__fsub_rn(g0, gh), ge);
            const float ah = __fmul_rn(gh, L), al = fmaf(gl, L, fmaf(gh, Ll, fmaf(gh, L, -ah)));
            const float z = __fmul_rn(__fmul_rn(ah, ah), fmaf(ah, 0.16666667f, 0.5f));
            const float bh = __fadd_rn(ah, z), bl = __fadd_rn(__fadd_rn(__fsub_rn(ah, bh), z), al);
            const float hl = fmaf(rx, bh, rx);
            const float ll = fmaf(rx, __fadd_rn(bl, fmaf(bh, r.rest, r.rest)), fmaf(rx, bh, __fsub_rn(rx, hl)));
            h[i] = t[i] > M + kLarge ? hl : h[i];
            lw[i] = t[i] > M + kLarge ? ll : lw[i];
        }
    }
    // in units of 2^-22 and of 2^-44 (the last places of 1.5 * 2 and of 1.5 * 2^-21), to nearest
    constexpr float M1 = 3.0f, M2 = 0x1.8p-21f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float t1 = __fadd_rn(h[i], M1);
        const float t2 = __fadd_rn(__fadd_rn(lw[i], __fsub_rn(h[i], __fsub_rn(t1, M1))), M2);
        w[i] = {__float_as_uint(t1) - __float_as_uint(M1), __float_as_int(t2) - __float_as_int(M2)};
    }
}

// ln(w / total) for a token of logit l, given the top token's weight, in fp32: (l - top) / T less ln(total / w_top), both
// at most 0, so they do not cancel; the quotient (of a rounded difference), log1pf (at most 1 ulp, of a rounded
// quotient) and their sum are off by at most 2^-22 of it
__device__ __forceinline__ float log_prob(float l, float top, float temp, unsigned long long w_top,
                                          unsigned long long total) {
    const float x = l == top ? 0.0f : __fdiv_rn(l - top, temp);
    return x - log1pf(__fdiv_rn(float(total - w_top), float(w_top)));
}

// ceil(p total), at least one unit: the mass at which top-p ends (p < 1)
__device__ __forceinline__ unsigned long long mass_target(float p, unsigned long long total) {
    const unsigned long long f = (unsigned long long)(p * 18446744073709551616.0f);
    const unsigned long long v = __umul64hi(f, total) + (f * total != 0);
    return v > 1 ? v : 1;
}
// floor(u total): the token is the first whose running mass is above it
__device__ __forceinline__ unsigned long long draw_target(float u, unsigned long long total) {
    return __umul64hi((unsigned long long)(u * 18446744073709551616.0f), total);
}
// the lowest key of a logit with exp((l - top) / T) >= min_p, given T ln(min_p) (at most 0) in fp64
__device__ __forceinline__ uint32_t min_p_key(double t_log_min_p, float top) {
    const uint32_t k = key_of(__double2float_ru(double(top) + t_log_min_p) + 0.0f), k_top = key_of(top);
    return k < k_top ? k : k_top;
}
// temperature 0 (greedy) or in [2^-20, 2^20], top_p above 0, min_p at most 1; NaN is refused
__device__ __forceinline__ bool sample_params_ok(float temp, float p, float mp) {
    return (temp == 0.0f || (temp >= 0x1p-20f && temp <= 0x1p20f)) && p > 0.0f && mp <= 1.0f;
}

}  // namespace gdn
