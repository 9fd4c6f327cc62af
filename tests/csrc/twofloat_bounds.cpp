/*
 * The error bounds that twofloat.cuh states, against the host's double: prints the largest errors of
 * two_exp2, times_log2e, div and mul over many arguments, in units of 2^-45 of
 * the result (of |x| for times_log2e), and exits non-zero if one is above its bound.
 */
#include <math.h>
#include <stdio.h>

#include "twofloat.cuh"

using namespace fp8bs;

static uint64_t state = 88172645463325252ull;
static double uniform(double lo, double hi)
{
    state ^= state << 13, state ^= state >> 7, state ^= state << 17;
    return lo + (hi - lo) * (double)(state >> 11) * 0x1p-53;
}
static Two split(double v)
{
    const float h = (float)v;
    return Two{h, (float)(v - h)};
}
static double value(Two v) { return (double)v.h + (double)v.l; }

int main(void)
{
    double worst[4] = {0, 0, 0, 0};
    const int n = 4000000;
    for (int i = 0; i < n; ++i) {
        const double t = i & 1 ? uniform(-100, 20) : uniform(-1, 1);
        const Two a = split(t);
        const double want = exp2(value(a));                        /* within an ulp of 2^-53 */
        worst[0] = fmax(worst[0], fabs(value(two_exp2(a)) - want) / want);
        const Two x = split(uniform(-90, 90));
        worst[1] = fmax(worst[1], fabs(value(times_log2e(x)) - value(x) * 1.4426950408889634074) / fabs(value(x)));
        const Two p = split(uniform(1e-3, 1)), q = split(uniform(1, 2));
        worst[2] = fmax(worst[2], fabs(value(div(p, q)) - value(p) / value(q)) / (value(p) / value(q)));
        worst[3] = fmax(worst[3], fabs(value(mul(p, q)) - value(p) * value(q)) / (value(p) * value(q)));
    }
    const double bound[4] = {0x1p-45, 0x1p-45, 0x1p-45, 0x1p-45};
    int bad = 0;
    for (int k = 0; k < 4; ++k) {
        printf("%g of 2^-45\n", worst[k] * 0x1p45);
        bad |= worst[k] > bound[k];
    }
    /* the ends of its range, and equal arguments */
    const Two zero = two_exp2(Two{0.0f, 0.0f}), low = two_exp2(Two{-126.5f, 0.0f}), inf = two_exp2(Two{-INFINITY, 0.0f});
    bad |= zero.h != 1.0f || zero.l != 0.0f || low.h != 0.0f || inf.h != 0.0f || two_exp2(Two{NAN, 0}).h == 0;
    bad |= value(two_exp2(Two{-3.0f, 0.0f})) != 0.125;
    printf("bad %d\n", bad);
    return bad;
}
