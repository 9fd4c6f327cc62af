// samplebins.cuh -- which tokens sample.cu's histogram of exponents takes: those
// within kWindow factors of 2 of the row's largest weight.  Host code includes
// it too: the test that every one of them has a bin.
#pragma once

#include "twofloat.cuh"

namespace fp8bs {

constexpr int kBins = 2048;                     // of the exponents
constexpr float kPerUnit = 32.0f;               // bins in a factor 2 of the weight
constexpr float kWindow = kBins / kPerUnit - 1; // in log2: lighter tokens do not count

// a - b rounded up.
TWOFLOAT_FN float sub_up(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fsub_ru(a, b);
#else
    const Two d = two_sum(a, -b);
    return d.l > 0.0f ? nextafterf(d.h, INFINITY) : d.h;
#endif
}

// No logit below it counts, for the row's largest logit m and weights
// 2^(c (x - m)).  Rounded up: what is taken is at most kWindow / c below m, also
// where that is half a step of m, and its bin at most 32 kWindow + 1.  (To the
// nearest, it can be nearly twice as far below m, and its bin 4032.)
TWOFLOAT_FN float window_end(float m, float c) { return sub_up(m, kWindow / c); }

}  // namespace fp8bs
