/*
 * Host-side check of the quotient the 4-bit cache's append uses (Markstein's
 * correction: y = RN(1/d), q0 = RN(x y), r = fma(-d, q0, x), q = RN(q0 + r y))
 * for every divisor mantissa d in [1, 2) and, at each of the seven borders m
 * between e2m1 magnitudes, the bf16 values x next to m d: the only places
 * where the code of q and that of the IEEE quotient RN(x / d) can differ.
 * Scaling d or x by powers of two scales every step exactly within the range
 * the kernel uses it in.  Prints "pairs <n> code_mismatches <m>".
 * Build: -O2 -ffp-contract=off -fopenmp (binary32 IEEE arithmetic).
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float from_bits(uint32_t u)
{
    float f;
    memcpy(&f, &u, 4);
    return f;
}

static uint32_t to_bits(float f)
{
    uint32_t u;
    memcpy(&u, &f, 4);
    return u;
}

static const float border[7] = {0.25f, 0.75f, 1.25f, 1.75f, 2.5f, 3.5f, 5.0f};

/* halfway goes to the even code */
static int enc(float a)
{
    int c = 0;
    for (int i = 0; i < 7; ++i)
        c += (i & 1) ? a >= border[i] : a > border[i];
    return c;
}

int main(void)
{
    long long total = 0, bad = 0;
#pragma omp parallel for schedule(static) reduction(+ : total, bad)
    for (uint32_t mant = 0; mant < (1u << 23); ++mant) {
        const float d = from_bits((127u << 23) | mant), y = 1.0f / d;
        for (int i = 0; i < 7; ++i) {
            const uint32_t below = to_bits((float)((double)border[i] * d)) & 0xFFFF0000u;
            for (uint32_t k = 0; k < 3; ++k) {
                const float x = from_bits(below + (k << 16) - 0x10000u);
                const float q0 = x * y, r = fmaf(-d, q0, x), q = fmaf(r, y, q0);
                ++total;
                bad += enc(q) != enc(x / d);
            }
        }
    }
    printf("pairs %lld code_mismatches %lld\n", total, bad);
    return bad != 0;
}
