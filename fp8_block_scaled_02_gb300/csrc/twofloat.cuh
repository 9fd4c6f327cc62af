// twofloat.cuh -- numbers held as the unevaluated sum of two fp32, some 46
// bits, for comparisons that 24 bits cannot decide and this GPU's FP64 rate
// (1/64 of fp32's) is too low for.  Knuth's two-sum and Dekker's fast two-sum
// and products (T. J. Dekker, "A floating-point technique for extending the
// available precision", Numer. Math. 18, 1971), products by fma; 2^f from its
// Taylor series.  Host code includes it too: the test of its error bounds.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define TWOFLOAT_FN __host__ __device__ __forceinline__
#else
#define TWOFLOAT_FN static inline
#endif

namespace fp8bs {

// One rounding each: the compiler may not join them.
TWOFLOAT_FN float add1(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fadd_rn(a, b);
#else
    return a + b;
#endif
}
TWOFLOAT_FN float sub1(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fsub_rn(a, b);
#else
    return a - b;
#endif
}
TWOFLOAT_FN float mul1(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fmul_rn(a, b);
#else
    return a * b;
#endif
}
TWOFLOAT_FN float fma1(float a, float b, float c) {
#ifdef __CUDA_ARCH__
    return __fmaf_rn(a, b, c);
#else
    return fmaf(a, b, c);
#endif
}

struct Two {
    float h, l;  // |l| <= ulp(h) / 2 after norm()
};

// a + b exactly.
TWOFLOAT_FN Two two_sum(float a, float b) {
    const float s = add1(a, b), t = sub1(s, a);
    return Two{s, add1(sub1(a, sub1(s, t)), sub1(b, t))};
}

// The same where |a| >= |b| or a = 0.
TWOFLOAT_FN Two fast_two_sum(float a, float b) {
    const float s = add1(a, b);
    return Two{s, sub1(b, sub1(s, a))};
}

TWOFLOAT_FN Two two_prod(float a, float b) {
    const float p = mul1(a, b);
    return Two{p, fma1(a, b, -p)};
}

TWOFLOAT_FN Two add(Two a, Two b) {
    const Two s = two_sum(a.h, b.h);
    return fast_two_sum(s.h, add1(s.l, add1(a.l, b.l)));
}

TWOFLOAT_FN Two add(Two a, float b) {
    const Two s = two_sum(a.h, b);
    return fast_two_sum(s.h, add1(s.l, a.l));
}

TWOFLOAT_FN Two mul(Two a, Two b) {
    Two p = two_prod(a.h, b.h);
    p.l = fma1(a.h, b.l, p.l);
    p.l = fma1(a.l, b.h, p.l);
    return fast_two_sum(p.h, p.l);
}

// a / b for normal b.h: the quotient of the leading parts and of its remainder.
TWOFLOAT_FN Two div(Two a, Two b) {
    const float q = a.h / b.h;
    const float r = add1(fma1(-q, b.h, a.h), fma1(-q, b.l, a.l));
    return fast_two_sum(q, r / b.h);
}

// x log2(e), within 2^-45 of |x|, for |x| < 2^100: the low part is below
// 2^-22.2 |x| and its two roundings are half a step, 2^-24 of it, each.
TWOFLOAT_FN Two times_log2e(Two x) {
    const float h = 0x1.715476p+0f, m = 0x1.4ae0cp-26f;
    Two p = two_prod(x.h, h);
    p.l = fma1(x.h, m, p.l);
    p.l = fma1(x.l, h, p.l);
    return fast_two_sum(p.h, p.l);
}

// 2^(t.h + t.l) within 2^-45 of itself and 2^-149, for -126 < t < 126; 0 below.
// (Under t = -100 the low part is subnormal, and what counts is the 2^-149.)  With n
// the nearest integer and f the rest, the sum of (f ln 2)^k / k! to k = 12; the
// terms from k = 7 on are below 2^-23 of the sum and need one fp32 each.
TWOFLOAT_FN Two two_exp2(Two t) {
    if (!(t.h > -126.0f)) return Two{t.h != t.h ? t.h : 0.0f, 0.0f};
    const float n = rintf(t.h);
    const Two f = fast_two_sum(sub1(t.h, n), t.l);
    float p = 0x1.c3bd66p-36f;
    p = fma1(p, f.h, 0x1.e8cac8p-32f);
    p = fma1(p, f.h, 0x1.e4cf52p-28f);
    p = fma1(p, f.h, 0x1.b5253ep-24f);
    p = fma1(p, f.h, 0x1.62c022p-20f);
    p = fma1(p, f.h, 0x1.ffcbfcp-17f);
    const float ch[7] = {1.0f,           0x1.62e43p-1f,   0x1.ebfbep-3f,   0x1.c6b08ep-5f,
                         0x1.3b2ab6p-7f, 0x1.5d87fep-10f, 0x1.430912p-13f};
    const float cl[7] = {0.0f,             -0x1.05c61p-29f,  -0x1.f4e9c6p-33f, -0x1.1f6be8p-30f,
                         0x1.f749cep-32f, 0x1.e299ccp-36f, 0x1.f0d8fp-38f};
    Two s{p, 0.0f};
#ifdef __CUDA_ARCH__
#pragma unroll
#endif
    for (int k = 6; k >= 0; --k) {
        Two q = two_prod(s.h, f.h);
        q.l = fma1(s.h, f.l, q.l);
        q.l = fma1(s.l, f.h, q.l);
        const Two c = fast_two_sum(ch[k], q.h);
        s = Two{c.h, add1(add1(c.l, q.l), cl[k])};
    }
    s = fast_two_sum(s.h, s.l);
    union {
        uint32_t u;
        float f;
    } scale;
    scale.u = static_cast<uint32_t>(127 + static_cast<int>(n)) << 23;  // 2^n, n >= -126
    return Two{s.h * scale.f, s.l * scale.f};
}

}  // namespace fp8bs
