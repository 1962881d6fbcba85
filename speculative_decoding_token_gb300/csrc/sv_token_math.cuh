// sv_token_math.cuh -- arithmetic of the token log-probability and distillation
// kernel: logits as ordered keys, pairs of floats, exponents and what rounding
// them takes. (A pair h, l stands for the unevaluated sum; see sv_common.cuh.)
#pragma once

#include "sv_token.h"
#include "sv_rows.cuh"

namespace sv {

namespace {

__device__ __forceinline__ uint32_t order_bits(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);  // -0 orders as 0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float from_order_bits(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ unsigned long long order_key(float v, int i) {
    return ((unsigned long long)order_bits(v) << 32) | (uint32_t)~i;
}

// Logits that the same kernel overwrites later, where a gradient takes their place.
template <int DT>
__device__ __forceinline__ float plain_logit(const char *row, int64_t v) {
    if (DT == SV_DT_FP32) return *reinterpret_cast<const volatile float *>(row + 4 * v);
    return __uint_as_float((uint32_t)*reinterpret_cast<const volatile uint16_t *>(row + 2 * v) << 16);
}

__device__ __forceinline__ uint16_t to_bf16(float x) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}

__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ void store_logit(char *row, int64_t v, float x) {
    if (DT == SV_DT_FP32) reinterpret_cast<float *>(row)[v] = x;
    else reinterpret_cast<uint16_t *>(row)[v] = to_bf16(x);
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Pair i of a vector's logits.
template <int DT>
__device__ __forceinline__ float2 pair_of(const uint4 &w, int i) {
    if (DT == SV_DT_FP32)
        return i == 0 ? make_float2(__uint_as_float(w.x), __uint_as_float(w.y))
                      : make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    const uint32_t x = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return make_float2(bf16_lo(x), bf16_hi(x));
}

// d / T for a difference d of logits, as a pair of floats
__device__ __forceinline__ void over_T(const TokenParams &P, float hi, float lo, float &rh, float &rl) {
    rh = hi * P.inv_hi;
    rl = 0.0f;
    if (fabsf(rh) < INFINITY) ff_mul(hi, lo, P.inv_hi, P.inv_lo, rh, rl);
}

// ln x of a positive normal x as a pair of floats, to about 2^-25 of one
__device__ __forceinline__ void ff_log(float x, float &h, float &l) {
    uint32_t b = __float_as_uint(x);
    int e = (int)(b >> 23) - 127;
    float f = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
    if (f > 1.41421356f) {
        f *= 0.5f;
        ++e;
    }
    float eh, el;
    ff_mul((float)e, 0.0f, kLn2Hi, kLn2Lo, eh, el);
    ff_add(eh, el, logf(f), 0.0f, h, l);
}

// ln(2^((z - m) c) / s) = (z - m) / T - ln s, a pair of floats
__device__ __forceinline__ void ff_logprob(const TokenParams &P, float z, float m, float lh, float ll,
                                           float &h, float &l) {
    float d, e, xh, xl;
    two_sum(z, -m, d, e);
    if (!(fabsf(d) < INFINITY)) e = 0.0f;
    over_T(P, d, e, xh, xl);
    if (!(fabsf(xh) < INFINITY)) {
        h = xh;
        l = 0.0f;
        return;
    }
    ff_add(xh, xl, -lh, -ll, h, l);
}

__device__ __forceinline__ float ff_exp(float h, float l) { return h == -INFINITY ? 0.0f : expf(h) * (1.0f + l); }

// 2^(j / 8) as pairs of floats
__device__ const float2 kExp8[8] = {
    {0x1p+0f, 0.0f},
    {0x1.172b84p+0f, -0x1.c15742p-27f},
    {0x1.306fe0p+0f, 0x1.4636e2p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f},
    {0x1.6a09e6p+0f, 0x1.9fcef4p-26f},
    {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f},
    {0x1.d5818ep+0f, -0x1.822dbcp-27f},
};

// e^v of v <= 88 as a pair of floats, to about 2^-40 of itself (0 below e^-86): v = n ln 2 / 8 + x, |x| <= ln 2 / 16, the
// series of e^x with its first three terms as pairs, and 2^(n / 8) from the table (Tang's method, see sv_common.cuh).
__device__ __forceinline__ void ff_exp_near(float v, float &h, float &l) {
    h = l = 0.0f;
    if (!(v > -86.0f)) return;
    const float n = rintf(v * 11.5415603f);
    float ph, pl, xh, xl;
    ff_mul(n * 0.125f, 0.0f, kLn2Hi, kLn2Lo, ph, pl);
    ff_add(v, 0.0f, -ph, -pl, xh, xl);
    const float sq = xh * xh, sl = fmaf(xh, xh, -sq) + 2.0f * xh * xl;
    const float tail = sq * xh * fmaf(xh, fmaf(xh, fmaf(xh, 1.0f / 720.0f, 1.0f / 120.0f), 1.0f / 24.0f), 1.0f / 6.0f);
    float eh, el;
    ff_add(xh, xl, 0.5f * sq, fmaf(0.5f, sl, tail), eh, el);
    ff_add(1.0f, 0.0f, eh, el, eh, el);
    const int i = (int)n;
    const float2 t = kExp8[i & 7];
    ff_mul(eh, el, t.x, t.y, h, l);
    const float scale = __uint_as_float((uint32_t)((i >> 3) + 127) << 23);
    h *= scale;
    l *= scale;
}

// e^(h + l), h <= 0 and l a rounding's worth of it, as a pair good to 2^-31: the same with two constants for ln 2 / 8, the first of
// 13 bits (its products with n are exact), and one pair kept. Half the instructions that wait on one another: a gradient's stores
// wait for this.
__device__ __forceinline__ void ff_exp_pair(float h, float l, float &rh, float &rl) {
    rh = rl = 0.0f;
    if (!(h > -86.0f)) return;
    const float n = rintf(h * 11.5415603f);
    const float d = fmaf(n, -0x1.62ep-4f, h), x = fmaf(n, -0x1.0bfbe8p-18f, d), xl = fmaf(n, -0x1.0bfbe8p-18f, d - x) + l;
    const float tail = fmaf(x * x, fmaf(x, fmaf(x, fmaf(x, 1.0f / 120.0f, 1.0f / 24.0f), 1.0f / 6.0f), 0.5f), xl);
    const float eh = 1.0f + x, el = (x - (eh - 1.0f)) + tail;
    const int i = (int)n;
    const float2 t = kExp8[i & 7];
    const float p = eh * t.x, e = fmaf(el, t.x, fmaf(eh, t.y, fmaf(eh, t.x, -p)));
    const float scale = __uint_as_float((uint32_t)((i >> 3) + 127) << 23);
    rh = p + e;
    rl = (e - (rh - p)) * scale;
    rh *= scale;
}

// ln(x + xl), xl a rounding's worth of x, as a pair of floats good to 2^-40: ff_log's head y, and what x e^-y is more than 1.
__device__ __forceinline__ void ff_log_near(float x, float xl, float &h, float &l) {
    float eh, el;
    ff_log(x, h, l);
    ff_exp_near(-h, eh, el);
    l = fmaf(x, eh, -1.0f) + fmaf(x, el, xl * eh);
}

// a ln(a / b) - a + b, none of it negative, with x = ln(a / b): sums of these have no large terms that cancel. a, b >= 0
__device__ __forceinline__ float divergence_of(float a, float b, float x) {
    if (!(a > 0.0f)) return b;
    if (fabsf(x) > 0.5f) return fmaf(a, x - 1.0f, b);
    // x - 1 + e^-x
    const float c = fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, fmaf(x, -1.0f / 362880.0f, 1.0f / 40320.0f), -1.0f / 5040.0f),
                                                   1.0f / 720.0f), -1.0f / 120.0f), 1.0f / 24.0f), -1.0f / 6.0f);
    return a * (x * x) * fmaf(x, c, 0.5f);
}

// ln(1 + b (e^r - 1)), good where r is small; 0 < b < 1
__device__ __forceinline__ float ln_mixed(float b, float r) { return r > 40.0f ? r + logf(b) : log1pf(b * expm1f(r)); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
    return x;
}

// Logits, and differences of them, are told from -inf down to P.far, -2^25 / c: of no weight either way (with |R| < 2^24), and
// a weight's product with its exponent is 0 and not NaN, also with an entropy's factor between them (below 2^100).

// (z - m) log2(e) / T of a difference
__device__ __forceinline__ float exponent(const TokenParams &P, float d) {
    d = fmaxf(d, P.far);
    return fmaf(d, P.c_lo, d * P.c);
}

// Of a reference nearer to zero than this, exponents are z c - R with R = m c rounded down to a whole number: one FMA, whose product
// is exact, and going from one reference to another multiplies by a power of two. |R| <= 2^24. Others take (z - m) c, with the
// difference first.
__device__ __forceinline__ bool plain(const TokenParams &P, float m) { return fabsf(m) < P.near; }
__device__ __forceinline__ float scaled(const TokenParams &P, float m) { return floorf(__fmul_rn(m, P.c)); }

// What m c is more than R; 0 of others.
__device__ __forceinline__ float off_by(const TokenParams &P, float m) { return plain(P, m) ? fmaf(m, P.c, -scaled(P, m)) + m * P.c_lo : 0.0f; }

// The same times ln 2, as a pair: what the logarithm of a sum is less where it is taken relative to m.
__device__ __forceinline__ void ff_off_by(const TokenParams &P, float m, float &h, float &l) {
    h = l = 0.0f;
    if (!plain(P, m)) return;
    const float p = __fmul_rn(m, P.c);
    float oh, ol;
    ff_add(p - floorf(p), 0.0f, fmaf(m, P.c, -p), m * P.c_lo, oh, ol);
    ff_mul(oh, ol, kLn2Hi, kLn2Lo, h, l);
}

// The exponent x by which sums relative to `from` become sums relative to `to`, not less than it, and 2^x.
__device__ __forceinline__ float between(const TokenParams &P, float from, float to, float &f) {
    float x;
    if (plain(P, from) && plain(P, to)) {
        x = scaled(P, from) - scaled(P, to);
        f = __uint_as_float((uint32_t)(127 + (int)fmaxf(x, -127.0f)) << 23);
    } else {
        x = exponent(P, from - to) - off_by(P, from) + off_by(P, to);
        f = ex2_approx(x);
    }
    return x;
}

// P.far as logits2 takes it
template <int DT>
__device__ __forceinline__ uint32_t far_bits(const TokenParams &P) {
    const uint32_t b = __float_as_uint(P.far);
    return DT == SV_DT_FP32 ? b : b | b >> 16;
}

// The j-th largest of the warp's values (j from 1).
__device__ __forceinline__ uint32_t warp_nth(uint32_t x, int j, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
        for (int i = k >> 1; i > 0; i >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, x, i);
            const bool larger = ((lane & k) == 0) == ((lane & i) == 0);
            x = larger ? max(x, o) : min(x, o);
        }
    }
    return __shfl_sync(0xffffffffu, x, j - 1);
}

}  // namespace

}  // namespace sv
