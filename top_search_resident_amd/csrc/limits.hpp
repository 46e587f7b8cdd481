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
// one kernel without a workspace (int8_rows.hip: few_kernel).
constexpr int kInt8FewRows = 4, kInt8FewBytes = 8192, kInt8FewN = 8192;
constexpr bool int8_few(int64_t m, int64_t n, int32_t k) {
    return m <= kInt8FewRows && m * int8_padded(k) <= kInt8FewBytes && n <= kInt8FewN;
}

}  // namespace rt
