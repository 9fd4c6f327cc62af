/*
 * two_exp2 over the whole range that twofloat.cuh states, the smallest results included: within 2^-45 of the result and
 * 2^-149.  Prints the largest share of that bound for each band of arguments; exits non-zero if one is above 1.
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

int main(void)
{
    const double ends[] = {-125.999, -124, -120, -110, -104, -100, -60, -1, 1, 60, 100, 125.99};
    int bad = 0;
    for (int b = 0; b + 1 < (int)(sizeof ends / sizeof *ends); ++b) {
        double worst = 0;
        for (int i = 0; i < 400000; ++i) {
            const double t = uniform(ends[b], ends[b + 1]);
            const float h = (float)t;
            const Two a{h, (float)(t - h)}, r = two_exp2(a);
            const double want = exp2((double)a.h + (double)a.l);   /* within an ulp of 2^-53 */
            worst = fmax(worst, fabs((double)r.h + (double)r.l - want) / (0x1p-45 * want + 0x1p-149));
        }
        printf("[%g, %g] %g\n", ends[b], ends[b + 1], worst);
        bad |= !(worst <= 1);
    }
    return bad;
}
