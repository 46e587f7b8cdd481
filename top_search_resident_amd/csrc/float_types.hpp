// float_types.hpp -- the three floating types of the int8 row products and the
// row sampler, 16 bytes at a time.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rt {

using bf16_t = __bf16;
using fp16_t = _Float16;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A pointer to global memory, said to the compiler: where it cannot see that (a
// pointer out of a struct, through a loop) it reads with flat loads, which wait
// for LDS operations, too, and keep no loads in flight beside them.
template <typename T>
using global_ptr = const __attribute__((address_space(1))) T *;

// 16 bytes from any global address (gfx950 reads unaligned addresses in one load).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ u32x4 load16(const void *p) {
    return *reinterpret_cast<global_ptr<u32x4_any>>((uintptr_t)p);
}

// Element i (a constant after unrolling) of 16 bytes of T, as fp32.
template <typename T>
__device__ __forceinline__ float element(u32x4 v, int i);
template <>
__device__ __forceinline__ float element<float>(u32x4 v, int i) {
    return __uint_as_float(v[i]);
}
template <>
__device__ __forceinline__ float element<bf16_t>(u32x4 v, int i) {
    const uint32_t w = v[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
}
template <>
__device__ __forceinline__ float element<fp16_t>(u32x4 v, int i) {
    const uint32_t w = v[i >> 1];
    const uint16_t h = (i & 1) ? uint16_t(w >> 16) : uint16_t(w);
    return static_cast<float>(__builtin_bit_cast(fp16_t, h));
}

}  // namespace rt
