// sample_units.hpp -- the row sampler's weights as whole numbers: how fine they are,
// and the constants of their exponential.  Plain C++ with no HIP dependency, so
// that the CPU test suite builds it on its own.
#pragma once
#include <stdint.h>

namespace rt {

// 2^f for |f| <= 2^-6 as 1 + f (kC1 + f (kC2 + f (kC3 + f kC4))).
constexpr double kC4 = 0.009618187552583722, kC3 = 0.055504515561345676, kC2 = 0.24022650695390316,
                 kC1 = 0.693147180535112;

// Weights are multiples of 2^-shift of the largest: v of them stay below 2^63.
constexpr int sample_shift(int64_t v) {
    int log2v = 0;
    while ((int64_t(1) << log2v) < v) ++log2v;
    return 62 - log2v < 46 ? 62 - log2v : 46;
}

// The coefficients and one in units of 2^-shift, to the nearest whole number.  As
// the bits of an fp64 such a number is that multiple of 2^-1074 (below 2^52: they
// are subnormal), which is how the kernels add them.  They are made as whole
// numbers because the calling thread's processor may be set to flush subnormal
// results and operands to zero, where products with 2^-1074 would all be 0.
struct SampleUnits {
    uint64_t c4, c3, c2, c1, one;
};
constexpr SampleUnits sample_units(int shift) {
    const uint64_t one = uint64_t(1) << shift;
    const double unit = static_cast<double>(one);
    return SampleUnits{uint64_t(kC4 * unit + 0.5), uint64_t(kC3 * unit + 0.5), uint64_t(kC2 * unit + 0.5),
                       uint64_t(kC1 * unit + 0.5), one};
}

}  // namespace rt
