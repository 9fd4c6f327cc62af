/*
 * The bins of the sampling kernel's histogram of exponents: for many largest logits m and scales c, of every fp32 number
 * from the window's end up to m the bin as the kernel computes it has to be one of kBins.  Prints the largest bin, with
 * the window's end and, for comparison, with m - kWindow / c rounded to the nearest; exits non-zero if one is past the end.
 */
#include <math.h>
#include <stdio.h>

#include "samplebins.cuh"

using namespace fp8bs;

static const float kMagic = 12582912.0f; /* 1.5 * 2^23 */

static int largest_bin(float m, float c, float end)
{
    int most = 0;
    float x = end; /* the bins fall as x rises: the first ones are the largest */
    for (int i = 0; i < 8 && x <= m; ++i, x = nextafterf(x, INFINITY)) {
        const float d = x - m, r = fmaf(d, -c * kPerUnit, kMagic);
        const int bin = (int)(r - kMagic);
        most = bin > most ? bin : most;
    }
    return most;
}

int main(void)
{
    int most = 0, nearest = 0;
    for (int e = -120; e <= 126; ++e)
        for (int s = 0; s < 2; ++s)
            for (int k = 0; k < 41; ++k) {
                const float m = (s ? -1.0f : 1.0f) * ldexpf(1.0f + (float)(k * 977 % 1024) / 1024.0f, e);
                const float ulp = nextafterf(fabsf(m), INFINITY) - fabsf(m);
                for (int j = 0; j < 200; ++j) {
                    /* temperatures from a hundredth of a step of m to 50 steps, and their scales */
                    const double t = ldexp(ulp, -7) * exp2(j / 16.0 + k / 660.0);
                    if (!(t >= 1e-30 && t <= 1e30)) continue;
                    const float c = (float)(1.4426950408889634 / (double)(float)t);
                    const int bin = largest_bin(m, c, window_end(m, c)), other = largest_bin(m, c, m - kWindow / c);
                    most = bin > most ? bin : most;
                    nearest = other > nearest ? other : nearest;
                }
            }
    printf("largest bin %d of %d; rounded to the nearest %d\n", most, kBins, nearest);
    return !(most < kBins && nearest >= kBins); /* the comparison shows that the arguments reach the case */
}
