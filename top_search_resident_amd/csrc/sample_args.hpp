// sample_args.hpp -- what the row sampling kernels are given (sample_rows.hpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/resident_topk.h"

namespace rt {

// 2^f for |f| <= 2^-6 as 1 + f (kC1 + f (kC2 + f (kC3 + f kC4))).
constexpr double kC4 = 0.009618187552583722, kC3 = 0.055504515561345676, kC2 = 0.24022650695390316,
                 kC1 = 0.693147180535112;

struct SampleArgs {
    const void *logits;
    int64_t r, v, ld;
    const float *u;
    rt_sample_settings set;
    int32_t *out_token;
    float *out_prob;
    int shift;  // weights are multiples of 2^-shift of the largest
    // The quartic of Weights::units with 2^(shift - 1074) multiplied in, one that is
    // 2^(shift - 1074), and 2^-shift: as arguments they reach the fmas in scalar registers.
    double c4, c3, c2, c1, one, per_unit;
};

// One workgroup of 512 threads a row (sample_rows_512.hip).
hipError_t launch_rows_512(const SampleArgs &a, int32_t dtype, hipStream_t s);

}  // namespace rt
