// limits.hpp -- the engine limits of the C ABI (include/resident_topk.h), host
// and device independent so that the argument checks also build as plain C++.
#pragma once
#include <stdint.h>

namespace rt {

constexpr int64_t kMaxN = 2147483647LL;  // row / element indices are int32
constexpr int32_t kMaxD = 65536;
constexpr int32_t kMaxK = 1024;
constexpr int32_t kMaxQ = 32;

// int8 rows: a sum of k products of int8 values, each at most 2^14, stays in 32 bits.
constexpr int32_t kMaxRowK = 65536;
constexpr int64_t kMaxLd = 2147483647LL;
// Outputs of one product: keeps every grid below 2^32 threads.
constexpr int64_t kMaxProduct = int64_t(1) << 37;

// Quantised activations in rt_linear_int8's workspace: rows padded with zeros to
// whole 128-byte steps, then the row scales.
constexpr int64_t int8_padded(int32_t k) { return (int64_t(k) + 127) / 128 * 128; }

// Up to here rt_linear_int8 keeps the quantised activations in LDS and runs as
// one kernel without a workspace (int8_rows.hip: few_kernel, stream_kernel for more
// rows b, short_kernel for more activations).
constexpr int kInt8FewRows = 4, kInt8FewBytes = 8192, kInt8FewN = 8192;
constexpr int kInt8StreamRows = 2, kInt8StreamBytes = 1024;
constexpr int64_t kInt8StreamN = int64_t(1) << 29;  // fewer than 2^32 threads
constexpr int kInt8ShortK = 1024, kInt8ShortTiles = 256;
constexpr bool int8_short(int64_t m, int64_t n, int32_t k) {
    return m > kInt8FewRows && k <= kInt8ShortK && (m + 31) / 32 * ((n + 31) / 32) <= kInt8ShortTiles;
}
constexpr bool int8_few(int64_t m, int64_t n, int32_t k) {
    const int64_t bytes = m * int8_padded(k);
    return (m <= kInt8FewRows && bytes <= kInt8FewBytes && n <= kInt8FewN) ||
           (m <= kInt8StreamRows && bytes <= kInt8StreamBytes && n <= kInt8StreamN) || int8_short(m, n, k);
}

// Row sampling: a few long rows are shared by up to kSampleSlices workgroups each
// (sample_rows.hip: split kernels), in slices of `per` chunks of kSplitChunk bytes.
constexpr int kSampleSlices = 32;
constexpr int64_t kSampleSlice = 33 * 1024;  // workspace bytes per slice
constexpr int64_t kSplitChunk = 16384;
constexpr int64_t kSplitLight = 1 << 20;  // bytes of a row from which top-k and greedy rows are shared, too
struct Split {
    int slices, per;
};
constexpr Split sample_split(int64_t r, int64_t v, int64_t element) {
    const int64_t chunks = (v * element + kSplitChunk - 1) / kSplitChunk;
    if (r < 1 || r > 16 || chunks < 16) return Split{1, 0};
    int64_t most = 256 / r;  // one workgroup a CU
    most = most < kSampleSlices ? most : kSampleSlices;
    const int64_t per = (chunks + most - 1) / most;
    return Split{int((chunks + per - 1) / per), int(per)};
}
// For any type of v logits.
constexpr int64_t sample_workspace(int64_t r, int64_t v) {
    const int n = sample_split(r, v, 4).slices;
    const int m = sample_split(r, v, 2).slices;
    const int most = n > m ? n : m;
    return most > 1 ? r * most * kSampleSlice : 0;
}

}  // namespace rt
