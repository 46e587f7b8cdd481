// int8_rows.hip -- rows quantised to int8 with an fp32 scale each, and their
// products on the int8 matrix cores (rt_quantize_rows_int8, rt_matmul_int8,
// rt_linear_int8).
//
//   s_i = max_j |x_ij| / 127,  q_ij = nearest whole number to x_ij / s_i
//   out_ij = (sum_l a_il b_jl) sa_i sb_j + bias_j
//
// The sum is exact: v_mfma_i32_16x16x64_i8 multiplies 16 rows by 16 rows over
// 64 values into 32-bit integers, and |sum| <= 65536 * 2^14 = 2^30.  The rows b
// are the first matrix operand and the activations the second, so that a
// lane's four results are four neighbouring columns of one output row.
//
// Two kernels:
//   tile    a workgroup's BM x BN outputs; 128-byte steps of both sides go
//           straight from global memory to LDS (two buffers), swizzled so that
//           the fragment reads spread over all banks.  For many activations.
//   direct  fragments from global memory straight to registers, the depth split
//           over the workgroup's waves and joined in LDS (integers: any order
//           gives the same sum).  For few activations, where the rows b are
//           read once and nothing is reused, and for rows that are not 16-byte
//           aligned, which the LDS loads need.
#include <hip/hip_runtime.h>

#include "../../include/resident_topk.h"
#include "float_types.hpp"
#include "lds_dma.hpp"
#include "limits.hpp"

namespace rt {
namespace {

// ---------------------------------------------------------------- quantise

constexpr int kQuantThreads = 256;
constexpr int kQuantKeep = 4;  // 16-byte chunks a thread keeps between the two passes

// The whole number nearest to x / s, ties to even, for |x| <= 127 s (1 + 2^-24)
// and a normal s.  The product with the rounded reciprocal is at most one off,
// and only next to a half; the remainder d = x - n s is exact in one fma (a
// multiple of ulp(s) / 2 not above s), so comparing 2 |d| with s decides.
__device__ __forceinline__ int nearest_quotient(float x, float s, float inv) {
    float n = __builtin_rintf(x * inv);
    const float d = __builtin_fmaf(-n, s, x);
    const float twice = 2.0f * __builtin_fabsf(d);
    const bool odd = (static_cast<int>(n) & 1) != 0;
    if (twice > s || (twice == s && odd)) n += __builtin_copysignf(1.0f, d);
    return static_cast<int>(n);
}

// One workgroup per row: the largest magnitude, then the codes.  The magnitude
// is compared as the bits of |x|, which also order infinities and NaN above
// every finite value.  Bound by the read of x; the second pass takes up to
// kQuantKeep chunks per thread from registers and the rest from L2.
template <typename T>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(const T *x, int64_t ldx, int64_t m, int k,
                                                                 int8_t *q, int64_t ldq, int kpad, float *scale) {
    constexpr int E = 16 / sizeof(T);
    __shared__ uint32_t wave_max[kQuantThreads / 64];
    const int t = threadIdx.x;
    const int whole = k / E;  // whole 16-byte chunks
    for (int64_t row = blockIdx.x; row < m; row += gridDim.x) {
        const T *xr = x + row * ldx;
        int8_t *qr = q + row * ldq;
        u32x4 keep[kQuantKeep];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < kQuantKeep; ++c) {
            const int i = c * kQuantThreads + t;
            if (i < whole) {
                keep[c] = load16(xr + int64_t(i) * E);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    top = max(top, __float_as_uint(element<T>(keep[c], e)) & 0x7fffffffu);
            }
        }
        for (int i = kQuantKeep * kQuantThreads + t; i < whole; i += kQuantThreads) {
            const u32x4 v = load16(xr + int64_t(i) * E);
#pragma unroll
            for (int e = 0; e < E; ++e) top = max(top, __float_as_uint(element<T>(v, e)) & 0x7fffffffu);
        }
        if (t < k - whole * E)
            top = max(top, __float_as_uint(static_cast<float>(xr[whole * E + t])) & 0x7fffffffu);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), o)));
        __syncthreads();  // the previous row's readers of wave_max are done
        if ((t & 63) == 0) wave_max[t >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQuantThreads / 64; ++w) top = max(top, wave_max[w]);

        float s = __uint_as_float(top) / 127.0f;
        const bool finite = top < 0x7f800000u;
        if (s < 1.17549435e-38f) s = 0.0f;
        const bool live = finite && s > 0.0f;
        if (t == 0) scale[row] = finite ? s : __builtin_nanf("");
        const float inv = live ? 1.0f / s : 0.0f;

        auto codes = [&](int i, u32x4 v) {
            uint32_t w[E / 4];
#pragma unroll
            for (int g = 0; g < E / 4; ++g) {
                w[g] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[g] |= (uint32_t(nearest_quotient(element<T>(v, g * 4 + e), s, inv)) & 0xffu) << (8 * e);
                if (!live) w[g] = 0;
            }
            __builtin_memcpy(qr + int64_t(i) * E, w, E);
        };
#pragma unroll
        for (int c = 0; c < kQuantKeep; ++c)
            if (c * kQuantThreads + t < whole) codes(c * kQuantThreads + t, keep[c]);
        for (int i = kQuantKeep * kQuantThreads + t; i < whole; i += kQuantThreads)
            codes(i, load16(xr + int64_t(i) * E));
        if (t < k - whole * E) {
            const int i = whole * E + t;
            qr[i] = live ? int8_t(nearest_quotient(static_cast<float>(xr[i]), s, inv)) : int8_t(0);
        }
        for (int i = k + t; i < kpad; i += kQuantThreads) qr[i] = 0;
    }
}

// ---------------------------------------------------------------- products

struct Product {
    const int8_t *a, *b;
    int64_t lda, ldb;
    const float *a_scale, *b_scale, *bias;
    void *out;
    int64_t ldo;
    int64_t m, n;
    int k;
    bool vec_out;  // four neighbouring outputs may be stored at once
};

__device__ __forceinline__ i32x4 mfma16(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// Up to 16 bytes at p, of which `valid` (possibly <= 0) exist; zeros elsewhere.
__device__ __forceinline__ i32x4 load_part(const int8_t *p, int valid) {
    if (valid >= 16) return __builtin_bit_cast(i32x4, load16(p));
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < valid) v[i >> 2] |= int(uint32_t(uint8_t(p[i])) << (8 * (i & 3)));
    return v;
}

// Scales, bias and rounding of the sums of output row i, columns j .. j + 3
// (i < m; columns from n on are dropped).
template <typename O>
__device__ __forceinline__ void store4(const Product &p, int64_t i, int64_t j, i32x4 sum) {
    const float sa = p.a_scale[i];
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        y[e] = 0.0f;
        if (j + e < p.n) {
            y[e] = static_cast<float>(sum[e]) * sa * p.b_scale[j + e];
            if (p.bias) y[e] += p.bias[j + e];
        }
    }
    O *o = static_cast<O *>(p.out) + i * p.ldo + j;
    if (p.vec_out && j + 4 <= p.n) {
        O v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = static_cast<O>(y[e]);
        __builtin_memcpy(__builtin_assume_aligned(o, 4 * sizeof(O)), v, sizeof(v));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < p.n) o[e] = static_cast<O>(y[e]);
    }
}

// direct: MF * 16 activations by NF * 16 rows b per workgroup of KW waves; wave w
// takes the 128-value blocks w, w + KW, ... of the depth.
template <int MF, int NF, int KW, typename O>
__global__ __launch_bounds__(64 * KW) void direct_kernel(Product p, int64_t tiles_m, int64_t tiles) {
    __shared__ i32x4 part[KW][MF * NF][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t i0 = tile % tiles_m * (MF * 16), j0 = tile / tiles_m * (NF * 16);
        const int8_t *ap[MF], *bp[NF];
#pragma unroll
        for (int f = 0; f < MF; ++f) ap[f] = p.a + min(i0 + f * 16 + r16, p.m - 1) * p.lda + g * 16;
#pragma unroll
        for (int f = 0; f < NF; ++f) bp[f] = p.b + min(j0 + f * 16 + r16, p.n - 1) * p.ldb + g * 16;
        i32x4 acc[NF][MF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < MF; ++h) acc[f][h] = i32x4{0, 0, 0, 0};
        const int blocks = p.k / 128;
        for (int blk = wave; blk < blocks; blk += KW) {
            i32x4 av[2][MF], bv[2][NF];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    bv[s][f] = __builtin_bit_cast(i32x4, load16(bp[f] + blk * 128 + s * 64));
#pragma unroll
                for (int f = 0; f < MF; ++f)
                    av[s][f] = __builtin_bit_cast(i32x4, load16(ap[f] + blk * 128 + s * 64));
            }
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int h = 0; h < MF; ++h) acc[f][h] = mfma16(bv[s][f], av[s][h], acc[f][h]);
        }
        if (wave == blocks % KW) {  // the values after the last whole block
            for (int k0 = blocks * 128; k0 < p.k; k0 += 64) {
                const int valid = p.k - k0 - g * 16;
                i32x4 av[MF];
#pragma unroll
                for (int f = 0; f < MF; ++f) av[f] = load_part(ap[f] + k0, valid);
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const i32x4 bv = load_part(bp[f] + k0, valid);
#pragma unroll
                    for (int h = 0; h < MF; ++h) acc[f][h] = mfma16(bv, av[h], acc[f][h]);
                }
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f)
#pragma unroll
            for (int h = 0; h < MF; ++h) part[wave][f * MF + h][lane] = acc[f][h];
        __syncthreads();
        for (int x = wave; x < MF * NF; x += KW) {
            i32x4 sum = part[0][x][lane];
#pragma unroll
            for (int w = 1; w < KW; ++w) sum += part[w][x][lane];
            const int64_t i = i0 + x % MF * 16 + r16, j = j0 + x / MF * 16 + g * 4;
            if (i < p.m && j < p.n) store4<O>(p, i, j, sum);
        }
        __syncthreads();  // part is free again
    }
}

// 16 bytes per lane from base + voff to LDS lds + 16 lane (kept in the caches:
// other workgroups read the same rows).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void *base, int voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// All of the wave's LDS reads have returned, then a workgroup barrier (the
// loads to LDS are waited for by wait_vmcnt).
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// tile: BM activations by BN rows b per workgroup of WM x WN waves.
template <int BM, int BN, int WM, int WN, typename O>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(Product p, int tiles_m, int tiles_n) {
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // LDS loads per wave and step
    static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN, "whole loads per wave");
    extern __shared__ __align__(1024) int8_t lds[];  // two buffers of (BM + BN) rows of 128 bytes
    constexpr int kBuf = (BM + BN) * 128;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r16 = lane & 15, g = lane >> 4;

    // Neighbouring workgroup numbers go to different XCDs: give each XCD a
    // contiguous run of tiles, and walk the tiles in groups of 8 tile rows so
    // that the run shares its activations and rows in the XCD's L2.
    const uint32_t total = uint32_t(tiles_m) * uint32_t(tiles_n);  // < 2^31
    uint32_t id = blockIdx.x;
    const uint32_t per = total / 8;
    if (id < per * 8) id = (id % 8) * per + id / 8;
    const uint32_t group = 8 * uint32_t(tiles_n);
    const uint32_t first = id / group * 8;
    const uint32_t rows = min(uint32_t(tiles_m) - first, 8u);
    const int64_t tm = __builtin_amdgcn_readfirstlane(first + id % group % rows);
    const int64_t tn = __builtin_amdgcn_readfirstlane(id % group / rows);
    const int64_t i0 = tm * BM, j0 = tn * BN;

    const int8_t *abase = p.a + i0 * p.lda, *bbase = p.b + j0 * p.ldb;
    int av[LA], bv[LB];  // byte offsets of this lane's 16 bytes; rows past the end repeat the last
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        av[i] = int(min(int64_t(r), p.m - 1 - i0) * p.lda) + (((lane & 7) ^ dma_swizzle(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        bv[i] = int(min(int64_t(r), p.n - 1 - j0) * p.ldb) + (((lane & 7) ^ dma_swizzle(r)) * 16);
    }
    const uint32_t lds0 = lds_addr(lds);
    auto stage = [&](int step, int buf) {
        const uint32_t at = lds0 + buf * kBuf;
#pragma unroll
        for (int i = 0; i < LA; ++i) dma16(abase + step * 128, av[i], at + (i * NW + wave) * 1024);
#pragma unroll
        for (int i = 0; i < LB; ++i) dma16(bbase + step * 128, bv[i], at + BM * 128 + (i * NW + wave) * 1024);
    };

    i32x4 acc[FN][FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int h = 0; h < FM; ++h) acc[f][h] = i32x4{0, 0, 0, 0};

    const int steps = p.k / 128;
    if (steps > 0) stage(0, 0);
    for (int step = 0; step < steps; ++step) {
        if (step + 1 < steps) {
            stage(step + 1, (step + 1) & 1);
            wait_vmcnt<LA + LB>();
        } else {
            wait_vmcnt<0>();
        }
        barrier();  // every wave's loads of this step have landed
        const int8_t *la = lds + (step & 1) * kBuf, *lb = la + BM * 128;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 fa[FM], fb[FN];
#pragma unroll
            for (int h = 0; h < FM; ++h) {
                const int r = wm * TM + h * 16 + r16;
                fa[h] = *reinterpret_cast<const i32x4 *>(la + r * 128 + (((s * 4 + g) ^ dma_swizzle(r)) * 16));
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const int r = wn * TN + f * 16 + r16;
                fb[f] = *reinterpret_cast<const i32x4 *>(lb + r * 128 + (((s * 4 + g) ^ dma_swizzle(r)) * 16));
            }
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int h = 0; h < FM; ++h) acc[f][h] = mfma16(fb[f], fa[h], acc[f][h]);
        }
        barrier();  // this buffer may be overwritten
    }
    // the values after the last whole step, straight from global memory
    for (int k0 = steps * 128; k0 < p.k; k0 += 64) {
        const int valid = p.k - k0 - g * 16;
        i32x4 fa[FM];
#pragma unroll
        for (int h = 0; h < FM; ++h)
            fa[h] = load_part(p.a + min(i0 + wm * TM + h * 16 + r16, p.m - 1) * p.lda + k0 + g * 16, valid);
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const i32x4 fb =
                load_part(p.b + min(j0 + wn * TN + f * 16 + r16, p.n - 1) * p.ldb + k0 + g * 16, valid);
#pragma unroll
            for (int h = 0; h < FM; ++h) acc[f][h] = mfma16(fb, fa[h], acc[f][h]);
        }
    }
#pragma unroll
    for (int h = 0; h < FM; ++h) {
        const int64_t i = i0 + wm * TM + h * 16 + r16;
        if (i >= p.m) continue;
#pragma unroll
        for (int f = 0; f < FN; ++f) {
            const int64_t j = j0 + wn * TN + f * 16 + g * 4;
            if (j < p.n) store4<O>(p, i, j, acc[f][h]);
        }
    }
}

template <int MF, int NF, int KW, typename O>
hipError_t launch_direct(const Product &p, hipStream_t s) {
    const int64_t tiles_m = (p.m + MF * 16 - 1) / (MF * 16), tiles_n = (p.n + NF * 16 - 1) / (NF * 16);
    const int64_t tiles = tiles_m * tiles_n;
    const unsigned grid = unsigned(tiles < (1 << 20) ? tiles : (1 << 20));
    direct_kernel<MF, NF, KW, O><<<grid, 64 * KW, 0, s>>>(p, tiles_m, tiles);
    return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, typename O>
hipError_t launch_tile(const Product &p, hipStream_t s) {
    const int64_t tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
    constexpr int kLds = 2 * (BM + BN) * 128;
    auto *kernel = tile_kernel<BM, BN, WM, WN, O>;
    if (kLds > 64 * 1024) {
        hipError_t err = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
        if (err != hipSuccess) return err;
    }
    kernel<<<unsigned(tiles_m * tiles_n), 64 * WM * WN, kLds, s>>>(p, int(tiles_m), int(tiles_n));
    return hipGetLastError();
}

bool aligned16(const void *ptr, int64_t ld) {
    return ((reinterpret_cast<uintptr_t>(ptr) | uintptr_t(ld)) & 15u) == 0;
}

template <typename O>
hipError_t launch_product(Product p, hipStream_t s) {
    p.vec_out = (reinterpret_cast<uintptr_t>(p.out) % (4 * sizeof(O))) == 0 && p.ldo % 4 == 0;
    // a tile's row offsets are 32-bit: 255 ld + depth
    // and a grid has fewer than 2^32 threads
    const bool tiles = aligned16(p.a, p.lda) && aligned16(p.b, p.ldb) && p.lda <= (1 << 22) && p.ldb <= (1 << 22) &&
                       ((p.m + 127) / 128) * ((p.n + 127) / 128) < (1 << 23);
    if (p.m <= 16) return launch_direct<1, 1, 8, O>(p, s);
    if (p.m <= 32) return launch_direct<2, 2, 8, O>(p, s);
    if (p.m <= 64 || !tiles) return launch_direct<4, 2, 4, O>(p, s);
    const int64_t big = (p.m + 255) / 256 * ((p.n + 255) / 256);
    if (big >= 256) return launch_tile<256, 256, 2, 4, O>(p, s);
    return launch_tile<128, 128, 2, 2, O>(p, s);
}

hipError_t launch_quantize(const void *x, int32_t dtype, int64_t m, int32_t k, int64_t ldx, int8_t *q, int64_t ldq,
                           int kpad, float *scale, hipStream_t s) {
    const unsigned grid = unsigned(m < (1 << 20) ? m : (1 << 20));
    switch (dtype) {
        case RT_DTYPE_FLOAT32:
            quantize_kernel<float><<<grid, kQuantThreads, 0, s>>>(static_cast<const float *>(x), ldx, m, k, q, ldq, kpad, scale);
            break;
        case RT_DTYPE_BFLOAT16:
            quantize_kernel<bf16_t><<<grid, kQuantThreads, 0, s>>>(static_cast<const bf16_t *>(x), ldx, m, k, q, ldq, kpad, scale);
            break;
        default:
            quantize_kernel<fp16_t><<<grid, kQuantThreads, 0, s>>>(static_cast<const fp16_t *>(x), ldx, m, k, q, ldq, kpad, scale);
    }
    return hipGetLastError();
}

hipError_t launch_matmul(const Product &p, int32_t out_dtype, hipStream_t s) {
    switch (out_dtype) {
        case RT_DTYPE_FLOAT32: return launch_product<float>(p, s);
        case RT_DTYPE_BFLOAT16: return launch_product<bf16_t>(p, s);
        default: return launch_product<fp16_t>(p, s);
    }
}

rt_status status_of(hipError_t err) {
    if (err == hipSuccess) return RT_OK;
    (void)hipGetLastError();
    return RT_EHIP;
}

}  // namespace
}  // namespace rt

extern "C" {

rt_status rt_quantize_rows_int8(const void *x, int32_t dtype, int64_t m, int32_t k, int64_t ldx, int8_t *q,
                                int64_t ldq, float *scale, void *stream) {
    rt_status st = rt_check_quantize_rows_int8(x, dtype, m, k, ldx, q, ldq, scale);
    if (st != RT_OK || m == 0) return st;
    return rt::status_of(rt::launch_quantize(x, dtype, m, k, ldx, q, ldq, k, scale, static_cast<hipStream_t>(stream)));
}

rt_status rt_matmul_int8(const int8_t *a, int64_t lda, const float *a_scale, const int8_t *b, int64_t ldb,
                         const float *b_scale, const float *bias, void *out, int32_t out_dtype, int64_t ldo,
                         int64_t m, int64_t n, int32_t k, void *stream) {
    rt_status st = rt_check_matmul_int8(a, lda, a_scale, b, ldb, b_scale, bias, out, out_dtype, ldo, m, n, k);
    if (st != RT_OK || m == 0) return st;
    const rt::Product p{a, b, lda, ldb, a_scale, b_scale, bias, out, ldo, m, n, k, false};
    return rt::status_of(rt::launch_matmul(p, out_dtype, static_cast<hipStream_t>(stream)));
}

rt_status rt_linear_int8(const void *x, int32_t dtype, int64_t ldx, const int8_t *w, int64_t ldw,
                         const float *w_scale, const float *bias, void *out, int32_t out_dtype, int64_t ldo,
                         int64_t m, int64_t n, int32_t k, void *workspace, int64_t workspace_bytes, void *stream) {
    const int64_t need = rt_linear_int8_workspace(m, k);
    if (need < 0) return RT_EINVAL;
    if (m > 0 && (workspace == nullptr || workspace_bytes < need ||
                  (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return RT_EINVAL;
    const int64_t ldq = rt::int8_padded(k);
    int8_t *q = static_cast<int8_t *>(workspace);
    float *scale = m > 0 ? reinterpret_cast<float *>(q + m * ldq) : nullptr;
    rt_status st = rt_check_quantize_rows_int8(x, dtype, m, k, ldx, q, ldq, scale);
    if (st == RT_OK)
        st = rt_check_matmul_int8(q, ldq, scale, w, ldw, w_scale, bias, out, out_dtype, ldo, m, n, k);
    if (st != RT_OK || m == 0) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err = rt::launch_quantize(x, dtype, m, k, ldx, q, ldq, int(ldq), scale, s);
    const rt::Product p{q, w, ldq, ldw, scale, w_scale, bias, out, ldo, m, n, k, false};
    if (err == hipSuccess) err = rt::launch_matmul(p, out_dtype, s);
    return rt::status_of(err);
}

}  // extern "C"
