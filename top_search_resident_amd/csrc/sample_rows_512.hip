// sample_rows_512.hip -- row sampling by workgroups of 512 threads (sample_rows.hpp),
// two of which share a CU: the one's passes over memory run beside the other's
// searches, which few of a CU's lanes have work in.
#define RT_SAMPLE_THREADS 512
#include "sample_rows.hpp"

namespace rt {

static_assert(sizeof(Shared) <= 80 * 1024, "two workgroups a CU");

hipError_t launch_rows_512(const SampleArgs &a, int32_t dtype, hipStream_t s) {
    switch (dtype) {
        case RT_DTYPE_FLOAT32: return launch_rows<float>(a, s);
        case RT_DTYPE_BFLOAT16: return launch_rows<bf16_t>(a, s);
        default: return launch_rows<fp16_t>(a, s);
    }
}

}  // namespace rt
