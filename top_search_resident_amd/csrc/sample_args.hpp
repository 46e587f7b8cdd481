// sample_args.hpp -- what the row sampling kernels are given (sample_rows.hpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/resident_topk.h"
#include "sample_units.hpp"

namespace rt {

struct SampleArgs {
    const void *logits;
    int64_t r, v, ld;
    const float *u;
    rt_sample_settings set;
    int32_t *out_token;
    float *out_prob;
    int shift;  // weights are multiples of 2^-shift of the largest
    // The quartic of Weights::units, and 2^-shift: as arguments they reach the fmas in
    // scalar registers.
    SampleUnits units;
    double per_unit;
};

// One workgroup of 512 threads a row (sample_rows_512.hip).
hipError_t launch_rows_512(const SampleArgs &a, int32_t dtype, hipStream_t s);

}  // namespace rt
