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
// Products of int8 rows:
//   tile    a workgroup's BM x BN outputs; 128-byte steps of both sides go
//           straight from global memory to LDS (two buffers), swizzled so that
//           the fragment reads spread over all banks.  For many activations.
//   direct  fragments from global memory straight to registers, the depth split
//           over the workgroup's waves and joined in LDS (integers: any order
//           gives the same sum).  For few activations, where the rows b are
//           read once and nothing is reused, and for rows that are not 16-byte
//           aligned, which the LDS loads need.
// Activations still to be quantised (rt_linear_int8): a kernel for that first, or,
// where they are few or short and there is little else to do, in the same one:
//   few     up to 4 activations;  stream  one or two short ones, many rows b;
//   short   up to 1024 values each and 256 workgroups.
#include <hip/hip_runtime.h>

#include "../../include/resident_topk.h"
#include "float_types.hpp"
#include "large_lds.hpp"
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

// A row's scale from the bits of its largest magnitude, which order infinities
// and NaN above every finite value; *inv is 0 where all codes are.
__device__ __forceinline__ float row_scale(uint32_t top, float *inv) {
    float s = __uint_as_float(top) / 127.0f;
    const bool finite = top < 0x7f800000u;
    if (s < 1.17549435e-38f) s = 0.0f;
    *inv = finite && s > 0.0f ? 1.0f / s : 0.0f;
    return finite ? s : __builtin_nanf("");
}
template <typename T>
__device__ __forceinline__ uint32_t magnitude(u32x4 v, uint32_t top) {
#pragma unroll
    for (int e = 0; e < int(16 / sizeof(T)); ++e) top = max(top, __float_as_uint(element<T>(v, e)) & 0x7fffffffu);
    return top;
}
// The codes of 16 bytes of T, 4 to a word (0 where inv is).  Adding 1.5 * 2^23 to x
// inv leaves the whole number n nearest to it in the low byte; it is the nearest
// one to x / s, too, where |x - n s|, exact in one fma, stays below s / 2.  Where
// any does not (a tie, or once in some hundred thousand the one beside it),
// nearest_quotient decides.
template <typename T>
__device__ __forceinline__ void codes16(u32x4 v, float s, float inv, uint32_t (&w)[4 / sizeof(T)]) {
    constexpr float kRound = 12582912.0f;
    float off = 0.0f;
#pragma unroll
    for (int g = 0; g < int(4 / sizeof(T)); ++g) {
        uint32_t n[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = element<T>(v, g * 4 + e), r = __builtin_fmaf(x, inv, kRound);
            n[e] = __float_as_uint(r);
            off = fmaxf(off, __builtin_fabsf(__builtin_fmaf(kRound - r, s, x)));
        }
        w[g] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(n[3], n[2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(n[1], n[0], 0x0c0c0400u), 0x05040100u);
    }
    if (!(2.0f * off < s)) {
#pragma unroll
        for (int g = 0; g < int(4 / sizeof(T)); ++g) {
            w[g] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[g] |= (uint32_t(nearest_quotient(element<T>(v, g * 4 + e), s, inv)) & 0xffu) << (8 * e);
            if (inv == 0.0f) w[g] = 0;
        }
    }
}

// One workgroup per row: the largest magnitude, then the codes; the second pass takes up to kQuantKeep chunks per
// thread from registers and the rest from L2.  Bound by memory for many rows (8192 x 8192 bf16: 35 us, 5.7 TB/s
// read and written, above a large copy's 5.2 because part of the 134 MB stays in the last-level cache from call to
// call; 2048 x 4096: 7.4 us), by latency for few (1 x 768: 2.6 us).
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
                top = magnitude<T>(keep[c], top);
            }
        }
        for (int i = kQuantKeep * kQuantThreads + t; i < whole; i += kQuantThreads)
            top = magnitude<T>(load16(xr + int64_t(i) * E), top);
        if (t < k - whole * E)
            top = max(top, __float_as_uint(static_cast<float>(xr[whole * E + t])) & 0x7fffffffu);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) top = max(top, uint32_t(__shfl_xor(int(top), o)));
        __syncthreads();  // the previous row's readers of wave_max are done
        if ((t & 63) == 0) wave_max[t >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kQuantThreads / 64; ++w) top = max(top, wave_max[w]);

        float inv;
        const float s = row_scale(top, &inv);
        if (t == 0) scale[row] = s;
        auto codes = [&](int i, u32x4 v) {
            uint32_t w[4 / sizeof(T)];
            codes16<T>(v, s, inv, w);
            __builtin_memcpy(qr + int64_t(i) * E, w, E);
        };
#pragma unroll
        for (int c = 0; c < kQuantKeep; ++c)
            if (c * kQuantThreads + t < whole) codes(c * kQuantThreads + t, keep[c]);
        for (int i = kQuantKeep * kQuantThreads + t; i < whole; i += kQuantThreads)
            codes(i, load16(xr + int64_t(i) * E));
        if (t < k - whole * E) {
            const int i = whole * E + t;
            qr[i] = inv != 0.0f ? int8_t(nearest_quotient(static_cast<float>(xr[i]), s, inv)) : int8_t(0);
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
    bool aligned_out;  // every row of out starts at a multiple of 16 bytes

    __device__ __forceinline__ const int8_t *a_end() const { return a + (m - 1) * lda + k; }
    __device__ __forceinline__ const int8_t *b_end() const { return b + (n - 1) * ldb + k; }
};

__device__ __forceinline__ i32x4 mfma16(i32x4 a, i32x4 b, i32x4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// 16 bytes at p, of which the first `valid` (any number) count and the rest read
// as zeros.  They are read whole where they end before `end`, the end of the
// matrix's last row, and byte by byte behind that.
__device__ __forceinline__ i32x4 load_part(const int8_t *p, int valid, const int8_t *end) {
    i32x4 v = {0, 0, 0, 0};
    if (valid <= 0) return v;
    if (p + 16 <= end) {
        v = __builtin_bit_cast(i32x4, load16(p));
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int n = min(max(valid - 4 * d, 0), 4);
            v[d] &= int(uint32_t((uint64_t(1) << (8 * n)) - 1));
        }
        return v;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < valid) v[i >> 2] |= int(uint32_t(uint8_t(p[i])) << (8 * (i & 3)));
    return v;
}

// Scales, bias and rounding of the sums of output row i, columns j .. j + N - 1
// (i < m; columns from n on are dropped).  NT: past the caches' keeping, for
// outputs written in whole 64-byte pieces.
template <int N, bool NT, typename O>
__device__ __forceinline__ void store_row(const Product &p, int64_t i, int64_t j, const int32_t (&sum)[N], float sa) {
    typedef O Piece __attribute__((ext_vector_type(N)));
    Piece v;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        float y = 0.0f;
        if (j + e < p.n) {
            y = static_cast<float>(sum[e]) * sa * p.b_scale[j + e];
            if (p.bias) y += p.bias[j + e];
        }
        v[e] = static_cast<O>(y);
    }
    O *o = static_cast<O *>(p.out) + i * p.ldo + j;
    if (j + N <= p.n) {
        // gfx950 stores to unaligned addresses, too; past the caches only whole pieces of a line
        typedef Piece Anywhere __attribute__((aligned(sizeof(O))));
        if (NT && p.aligned_out)
            __builtin_nontemporal_store(v, reinterpret_cast<Piece *>(o));
        else
            *reinterpret_cast<Anywhere *>(o) = v;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (j + e < p.n) o[e] = v[e];
    }
}
template <typename O>
__device__ __forceinline__ void store4(const Product &p, int64_t i, int64_t j, i32x4 sum) {
    const int32_t s[4] = {sum[0], sum[1], sum[2], sum[3]};
    store_row<4, false, O>(p, i, j, s, p.a_scale[i]);
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
                for (int f = 0; f < MF; ++f) av[f] = load_part(ap[f] + k0, valid, p.a_end());
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    const i32x4 bv = load_part(bp[f] + k0, valid, p.b_end());
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

// m rows of x by the whole workgroup of KW waves: their codes, and zeros up to kpad,
// into LDS, the bits of their largest magnitudes into top.
template <int KW, typename T>
__device__ __forceinline__ void quantize_to_lds(const T *x, int64_t ldx, int m, int k, int kpad, int8_t *codes,
                                                uint32_t *top) {
    constexpr int E = 16 / sizeof(T), kThreads = 64 * KW;
    const int t = threadIdx.x, lane = t & 63, whole = k / E;
    if (t < kInt8FewRows) top[t] = 0;
    __syncthreads();
    for (int i = 0; i < m; ++i) {
        const T *xr = x + i * ldx;
        uint32_t own = 0;
        for (int c = t; c < whole; c += kThreads) own = magnitude<T>(load16(xr + c * E), own);
        if (t < k - whole * E) own = max(own, __float_as_uint(static_cast<float>(xr[whole * E + t])) & 0x7fffffffu);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) own = max(own, uint32_t(__shfl_xor(int(own), o)));
        if (lane == 0) atomicMax(&top[i], own);
    }
    __syncthreads();
    for (int i = 0; i < m; ++i) {
        const T *xr = x + i * ldx;
        float inv;
        const float s = row_scale(top[i], &inv);
        for (int c = t; c < whole; c += kThreads) {
            uint32_t w[4 / sizeof(T)];
            codes16<T>(load16(xr + c * E), s, inv, w);
            __builtin_memcpy(codes + i * kpad + c * E, w, E);
        }
        for (int c = whole * E + t; c < kpad; c += kThreads)
            codes[i * kpad + c] =
                c < k && inv != 0.0f ? int8_t(nearest_quotient(static_cast<float>(xr[c]), s, inv)) : int8_t(0);
    }
    __syncthreads();
}

// few: rt_linear_int8 of a few short activations against not too many rows in
// one launch (limits.hpp: int8_few).  Each workgroup of KW waves quantises all
// of x into LDS while the first of its 16 rows b are on their way, then goes on
// as the direct kernel.  Two launches cost a gap and a round trip of the codes
// through memory: 1 x 4096 x 4096 6.4 us against 8.9, 1 x 1024 x 1024 3.7
// against 5.9; but every workgroup repeats the quantising (4 x 4096 x 4096: 10.9
// against 9.3), hence the limit.
template <int KW, typename T, typename O>
__global__ __launch_bounds__(64 * KW) void few_kernel(const T *x, int64_t ldx, Product p) {
    extern __shared__ __align__(16) int8_t codes[];  // m rows of kpad bytes
    __shared__ i32x4 part[KW][64];
    __shared__ uint32_t top[kInt8FewRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int m = int(p.m), kpad = (p.k + 127) / 128 * 128, blocks = p.k / 128;
    const int8_t *bp = p.b + min(blockIdx.x * int64_t(16) + r16, p.n - 1) * p.ldb + g * 16;

    i32x4 b0 = {0, 0, 0, 0}, b1 = {0, 0, 0, 0};
    if (wave < blocks) {
        b0 = __builtin_bit_cast(i32x4, load16(bp + wave * 128));
        b1 = __builtin_bit_cast(i32x4, load16(bp + wave * 128 + 64));
    }
    quantize_to_lds<KW>(x, ldx, m, p.k, kpad, codes, top);

    const int8_t *ap = codes + min(r16, m - 1) * kpad + g * 16;
    i32x4 acc = {0, 0, 0, 0};
    for (int blk = wave; blk < blocks; blk += KW) {
        if (blk != wave) {
            b0 = __builtin_bit_cast(i32x4, load16(bp + blk * 128));
            b1 = __builtin_bit_cast(i32x4, load16(bp + blk * 128 + 64));
        }
        acc = mfma16(b0, *reinterpret_cast<const i32x4 *>(ap + blk * 128), acc);
        acc = mfma16(b1, *reinterpret_cast<const i32x4 *>(ap + blk * 128 + 64), acc);
    }
    if (wave == blocks % KW)  // the values after the last whole block; the codes behind them are 0
        for (int k0 = blocks * 128; k0 < p.k; k0 += 64)
            acc = mfma16(load_part(bp + k0, p.k - k0 - g * 16, p.b_end()),
                         *reinterpret_cast<const i32x4 *>(ap + k0), acc);
    part[wave][lane] = acc;
    __syncthreads();
    if (wave == 0) {
        i32x4 sum = part[0][lane];
#pragma unroll
        for (int w = 1; w < KW; ++w) sum += part[w][lane];
        const int64_t j = blockIdx.x * int64_t(16) + g * 4;
        float inv;
        if (r16 < m && j < p.n) {
            const int32_t s4[4] = {sum[0], sum[1], sum[2], sum[3]};
            store_row<4, false, O>(p, r16, j, s4, row_scale(top[r16], &inv));
        }
    }
}

// stream: the same against many rows b.  A wave takes 16 of them over the whole
// depth, the first half a KiB of each on its way while x is quantised, so that
// the reads of b start with the kernel and nothing is joined at the end.  Bound by
// them (1 x 262144 x 768: 5.8 TB/s).  For one or two activations of up to 1024
// values together it beats two launches (us, bf16, fp32 out, back to back in a
// graph):
//   m x n x k            stream   quantise + product
//   1 x 16384 x 768      6.2      6.9
//   1 x 100000 x 768     17.3     18.9
//   1 x 100000 x 777     19.4     26.7
//   2 x 100000 x 512     14.0     16.0
//   4 x 100000 x 250     15.5     14.1    not taken
//   1 x 16384 x 4096     18.4     15.2    not taken
template <typename T, typename O>
__global__ __launch_bounds__(512) void stream_kernel(const T *x, int64_t ldx, Product p) {
    constexpr int KW = 8, DEEP = 8;
    extern __shared__ __align__(16) int8_t codes[];  // m rows of kpad bytes
    __shared__ uint32_t top[kInt8FewRows];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r16 = lane & 15, g = lane >> 4;
    const int m = int(p.m), kpad = (p.k + 127) / 128 * 128, steps = p.k / 64;
    const int64_t j0 = (blockIdx.x * int64_t(KW) + wave) * 16;
    const int8_t *bp = p.b + min(j0 + r16, p.n - 1) * p.ldb + g * 16;
    i32x4 b[DEEP];
    const auto fetch = [&](int s0) {
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (s0 + i < steps) b[i] = __builtin_bit_cast(i32x4, load16(bp + (s0 + i) * 64));
    };
    fetch(0);
    quantize_to_lds<KW>(x, ldx, m, p.k, kpad, codes, top);

    const int8_t *ap = codes + min(r16, m - 1) * kpad + g * 16;
    i32x4 acc = {0, 0, 0, 0};
    for (int s0 = 0; s0 < steps; s0 += DEEP) {
        if (s0 > 0) fetch(s0);
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
            if (s0 + i < steps) acc = mfma16(b[i], *reinterpret_cast<const i32x4 *>(ap + (s0 + i) * 64), acc);
    }
    if (steps * 64 < p.k)  // the codes behind the depth are 0
        acc = mfma16(load_part(bp + steps * 64, p.k - steps * 64 - g * 16, p.b_end()),
                     *reinterpret_cast<const i32x4 *>(ap + steps * 64), acc);
    const int64_t j = j0 + g * 4;
    float inv;
    if (r16 < m && j < p.n) {
        const int32_t s4[4] = {acc[0], acc[1], acc[2], acc[3]};
        store_row<4, false, O>(p, r16, j, s4, row_scale(top[r16], &inv));
    }
}

// The largest of the wave's 64 lanes, to all of them.
__device__ __forceinline__ uint32_t wave_most(uint32_t v) {
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x111, 0xf, 0xf, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x112, 0xf, 0xf, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x114, 0xf, 0xf, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x118, 0xf, 0xf, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x142, 0xa, 0xf, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x143, 0xc, 0xf, false)));
    return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}

// short: the same for activations of up to kInt8ShortK values, 32 of them and 32
// rows b per workgroup of 16 waves: a wave takes every sixteenth activation, all of
// whose values it holds at once, and then a 128-value block of the depth with half
// of the rows b.  Up to one workgroup a CU it beats two launches (us, bf16, back to
// back in a graph, with the calling path in brackets; fp32 alike):
//   m x n x k            short         quantise + product
//   8 x 1024 x 256       4.9 [8.4]     5.9 [12.6]
//   77 x 1001 x 777      7.2 [8.5]     10.5 [12.8]
//   256 x 1024 x 1024    7.6 [8.5]     8.2 [12.9]
//   128 x 4096 x 256     7.8 [8.4]     7.0 [12.7]    512 workgroups: not taken
//   512 x 1024 x 777     10.5 [10.5]   10.8 [12.7]   512 workgroups: not taken
// What remains is latency: a launch, a round trip for x and b, the code's own way
// into the instruction cache.
template <typename T, typename O>
__global__ __launch_bounds__(1024) void short_kernel(const T *x, int64_t ldx, Product p, int tiles_n) {
    constexpr int NW = 16, MF = 2, NF = 2, KW = NW / NF, ROWS = MF * 16 / NW;
    constexpr int E = 16 / sizeof(T), CH = kInt8ShortK / E / 64;  // 16-byte chunks a lane of each activation
    extern __shared__ __align__(16) int8_t codes[];  // MF * 16 rows of kpad + 16 bytes
    __shared__ i32x4 part[NW][MF][64];
    __shared__ float scale[MF * 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t i0 = int64_t(blockIdx.x) / tiles_n * (MF * 16);
    const int64_t j0 = int64_t(blockIdx.x) % tiles_n * (NF * 16) + wave / KW * 16;
    const int m = int(min(p.m - i0, int64_t(MF * 16)));
    const int stride = (p.k + 127) / 128 * 128 + 16;  // 16 more: neighbouring rows in other banks
    const int whole = p.k / E, k0 = wave % KW * 128;

    u32x4 keep[ROWS][CH];
    float last[ROWS];  // a lane each for the values behind the whole chunks
#pragma unroll
    for (int h = 0; h < ROWS; ++h) {
        const T *xr = x + (i0 + min(h * NW + wave, m - 1)) * ldx;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            keep[h][c] = u32x4{0, 0, 0, 0};
            if (c * 64 + lane < whole) keep[h][c] = load16(xr + (c * 64 + lane) * E);
        }
        last[h] = lane < p.k - whole * E ? static_cast<float>(xr[whole * E + lane]) : 0.0f;
    }
    const int8_t *bp = p.b + min(j0 + r16, p.n - 1) * p.ldb + g * 16 + k0;
    i32x4 b[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (k0 + 128 <= p.k) {
#pragma unroll
        for (int s = 0; s < 2; ++s) b[s] = __builtin_bit_cast(i32x4, load16(bp + s * 64));
    } else if (k0 < p.k) {
#pragma unroll
        for (int s = 0; s < 2; ++s) b[s] = load_part(bp + s * 64, p.k - k0 - s * 64 - g * 16, p.b_end());
    }
    uint32_t top[ROWS];
#pragma unroll
    for (int h = 0; h < ROWS; ++h) {
        top[h] = __float_as_uint(last[h]) & 0x7fffffffu;
#pragma unroll
        for (int c = 0; c < CH; ++c) top[h] = magnitude<T>(keep[h][c], top[h]);
        top[h] = wave_most(top[h]);
    }
#pragma unroll
    for (int h = 0; h < ROWS; ++h) {
        float inv;
        const float s = row_scale(top[h], &inv);
        int8_t *row = codes + (h * NW + wave) * stride;
        if (lane == 0) scale[h * NW + wave] = s;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint32_t w[4 / sizeof(T)];
            codes16<T>(keep[h][c], s, inv, w);
            if (c * 64 + lane < whole) __builtin_memcpy(row + (c * 64 + lane) * E, w, E);
        }
        for (int c = whole * E + lane; c < stride - 16; c += 64)
            row[c] = c < p.k && inv != 0.0f ? int8_t(nearest_quotient(last[h], s, inv)) : int8_t(0);
    }
    __syncthreads();

#pragma unroll
    for (int h = 0; h < MF; ++h) {
        i32x4 acc = {0, 0, 0, 0};
        if (k0 < p.k) {
            const int8_t *ap = codes + (h * 16 + r16) * stride + k0 + g * 16;
#pragma unroll
            for (int s = 0; s < 2; ++s) acc = mfma16(b[s], *reinterpret_cast<const i32x4 *>(ap + s * 64), acc);
        }
        part[wave][h][lane] = acc;
    }
    __syncthreads();
    if (wave % KW < MF) {
        const int h = wave % KW, w0 = wave - h;
        i32x4 sum = part[w0][h][lane];
#pragma unroll
        for (int w = 1; w < KW; ++w) sum += part[w0 + w][h][lane];
        const int i = h * 16 + r16;
        const int64_t j = j0 + g * 4;
        if (i < m && j < p.n) {
            const int32_t s4[4] = {sum[0], sum[1], sum[2], sum[3]};
            store_row<4, false, O>(p, i0 + i, j, s4, scale[i]);
        }
    }
}

template <typename T, typename O>
hipError_t launch_few(const void *x, int64_t ldx, const Product &p, hipStream_t s) {
    if (int8_short(p.m, p.n, p.k)) {
        // up to 33280 bytes of dynamic LDS beside 32896 that the kernel declares: 66176 of a
        // CU's 163840.  HIP need not be told, as the dynamic part is below 64 KiB.
        const int64_t tiles_n = (p.n + 31) / 32;
        short_kernel<T, O><<<unsigned((p.m + 31) / 32 * tiles_n), 1024, size_t(int8_padded(p.k) + 16) * 32, s>>>(
            static_cast<const T *>(x), ldx, p, int(tiles_n));
        return hipGetLastError();
    }
    if (p.n > kInt8FewN) {
        stream_kernel<T, O><<<unsigned((p.n + 127) / 128), 512, size_t(p.m) * size_t(int8_padded(p.k)), s>>>(
            static_cast<const T *>(x), ldx, p);
        return hipGetLastError();
    }
    const int64_t tiles = (p.n + 15) / 16;
    few_kernel<8, T, O><<<unsigned(tiles), 64 * 8, size_t(p.m) * size_t(int8_padded(p.k)), s>>>(
        static_cast<const T *>(x), ldx, p);
    return hipGetLastError();
}

// 16 bytes per lane from base + voff to LDS lds + 16 lane (kept in the caches:
// other workgroups read the same rows).  A load to LDS must not follow the
// write of M0 at once: it needs one instruction between.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void *base, int voff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(voff), "s"(base), "s"(lds)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// All of the wave's LDS reads have returned, then a workgroup barrier (the
// loads to LDS are waited for by wait_vmcnt).
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The place of 16-byte unit u of a row among its 128 bytes is u ^ unit_swap(row).
// ds_read_b128 serves lanes 0-3, 12-15 and 20-27 together, then 4-11, 16-19 and
// 28-31, and so on: with r & 7 for rows read in order, and with the other for
// the rows a two-byte output reads (row_of), each such 16 lanes hit all 64 banks
// once (4.1 cycles a read; 8.0 with the bound kernels' dma_swizzle).
template <bool PAIRS>
__device__ __forceinline__ int unit_swap(int r) {
    return PAIRS ? ((r >> 1) & 1) | (((r >> 3) & 3) << 1) : r & 7;
}
// Row, within a wave's rows b, of operand row r16 of fragment f.  A lane's four results
// are operand rows 4 g .. 4 g + 3; two-byte outputs take the rows such that
// fragments 2 q and 2 q + 1 give a lane 8 neighbouring columns: 16 bytes a
// lane, and 64 contiguous bytes of a row in one store, for every output type.
template <bool PAIRS>
__device__ __forceinline__ int row_of(int f, int r16) {
    return PAIRS ? (f >> 1) * 32 + (r16 >> 2) * 8 + (f & 1) * 4 + (r16 & 3) : f * 16 + r16;
}

// tile: BM activations by BN rows b per workgroup of WM x WN waves, STAGES
// 128-byte steps of both in LDS.  Measured on 8192^3 (bf16 out): 256 x 256 with
// 16 waves 2.5 PFLOP/s, with 8 waves 2.37 (a wave's LDS reads wait, the more
// waves the better covered), 128 x 128 1.9.
template <int BM, int BN, int WM, int WN, int STAGES, typename O>
__global__ __launch_bounds__(64 * WM * WN) void tile_kernel(Product p, int tiles_m, int tiles_n) {
    constexpr int NW = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
    constexpr int LA = BM / 8 / NW, LB = BN / 8 / NW;  // LDS loads per wave and step
    constexpr bool PAIRS = sizeof(O) == 2;
    static_assert(LA * 8 * NW == BM && LB * 8 * NW == BN, "whole loads per wave");
    static_assert(!PAIRS || FN % 2 == 0, "pairs of fragments");
    extern __shared__ __align__(1024) int8_t lds[];  // STAGES buffers of (BM + BN) rows of 128 bytes
    constexpr int kBuf = (BM + BN) * 128;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r16 = lane & 15, g = lane >> 4;

    // Neighbouring workgroup numbers go to different XCDs: give each XCD a
    // contiguous run of tiles, and walk the tiles in groups of 2048 activations
    // so that the run shares its activations and rows in the XCD's L2.
    const uint32_t total = uint32_t(tiles_m) * uint32_t(tiles_n);  // < 2^31
    uint32_t id = blockIdx.x;
    const uint32_t per = total / 8;
    if (id < per * 8) id = (id % 8) * per + id / 8;
    constexpr uint32_t kGroup = 2048 / BM;
    const uint32_t group = kGroup * uint32_t(tiles_n);
    const uint32_t first = id / group * kGroup;
    const uint32_t rows = min(uint32_t(tiles_m) - first, kGroup);
    const int64_t tm = __builtin_amdgcn_readfirstlane(first + id % group % rows);
    const int64_t tn = __builtin_amdgcn_readfirstlane(id % group / rows);
    const int64_t i0 = tm * BM, j0 = tn * BN;

    const int8_t *abase = p.a + i0 * p.lda, *bbase = p.b + j0 * p.ldb;
    int av[LA], bv[LB];  // byte offsets of this lane's 16 bytes; rows past the end repeat the last
#pragma unroll
    for (int i = 0; i < LA; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        av[i] = int(min(int64_t(r), p.m - 1 - i0) * p.lda) + (((lane & 7) ^ unit_swap<false>(r)) * 16);
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
        const int r = (i * NW + wave) * 8 + (lane >> 3);
        bv[i] = int(min(int64_t(r), p.n - 1 - j0) * p.ldb) + (((lane & 7) ^ unit_swap<PAIRS>(r)) * 16);
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
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < steps) stage(s, s);
    auto multiply = [&](int buf) {
        const int8_t *la = lds + buf * kBuf, *lb = la + BM * 128;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            i32x4 fa[FM], fb[FN];
#pragma unroll
            for (int h = 0; h < FM; ++h) {
                const int r = wm * TM + h * 16 + r16;
                fa[h] = *reinterpret_cast<const i32x4 *>(la + r * 128 + (((s * 4 + g) ^ unit_swap<false>(r)) * 16));
            }
#pragma unroll
            for (int f = 0; f < FN; ++f) {
                const int r = wn * TN + row_of<PAIRS>(f, r16);
                fb[f] = *reinterpret_cast<const i32x4 *>(lb + r * 128 + (((s * 4 + g) ^ unit_swap<PAIRS>(r)) * 16));
            }
#pragma unroll
            for (int f = 0; f < FN; ++f)
#pragma unroll
                for (int h = 0; h < FM; ++h) acc[f][h] = mfma16(fb[f], fa[h], acc[f][h]);
        }
    };
    int buf = 0;
    for (int step = 0; step < steps; ++step) {
        // this step's loads are the oldest of those in flight
        if (step + STAGES - 2 < steps)
            wait_vmcnt<(STAGES - 2) * (LA + LB)>();
        else
            wait_vmcnt<0>();
        barrier();  // every wave's loads of this step have landed, its reads of the step before are done
        if (step + STAGES - 1 < steps) stage(step + STAGES - 1, buf == 0 ? STAGES - 1 : buf - 1);
        multiply(buf);
        if (++buf == STAGES) buf = 0;
    }
    // The values after the last whole step, zeros behind them, through registers
    // into the next buffer: it was last read STAGES steps ago, ahead of a barrier.
    if (steps * 128 < p.k) {
        auto fill = [&](const int8_t *base, const int *offset, int count, const int8_t *end, int8_t *to, bool pairs) {
            for (int i = 0; i < count; ++i) {
                const int r = (i * NW + wave) * 8 + (lane >> 3);
                const int unit = (lane & 7) ^ (pairs ? unit_swap<true>(r) : unit_swap<false>(r));
                *reinterpret_cast<i32x4 *>(to + (i * NW + wave) * 1024 + lane * 16) =
                    load_part(base + offset[i] + steps * 128, p.k - steps * 128 - unit * 16, end);
            }
        };
        int8_t *to = lds + buf * kBuf;
        fill(abase, av, LA, p.a_end(), to, false);
        fill(bbase, bv, LB, p.b_end(), to + BM * 128, PAIRS);
        barrier();
        multiply(buf);
    }
    // 16 bytes a lane: 4 columns of fp32, 8 of a two-byte type
    constexpr int kSide = PAIRS ? 2 : 1;
#pragma unroll
    for (int h = 0; h < FM; ++h) {
        const int64_t i = i0 + wm * TM + h * 16 + r16;
        if (i >= p.m) continue;
        const float sa = p.a_scale[i];
#pragma unroll
        for (int f = 0; f < FN; f += kSide) {
            const int64_t j = j0 + wn * TN + f * 16 + g * 4 * kSide;
            int32_t sum[4 * kSide];
#pragma unroll
            for (int e = 0; e < 4 * kSide; ++e) sum[e] = acc[f + e / 4][h][e % 4];
            if (j < p.n) store_row<4 * kSide, true, O>(p, i, j, sum, sa);
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

template <int BM, int BN, int WM, int WN, int STAGES, typename O>
hipError_t launch_tile(const Product &p, hipStream_t s) {
    const int64_t tiles_m = (p.m + BM - 1) / BM, tiles_n = (p.n + BN - 1) / BN;
    constexpr int kLds = STAGES * (BM + BN) * 128;
    auto *kernel = tile_kernel<BM, BN, WM, WN, STAGES, O>;
    if (kLds > 64 * 1024) {
        static std::atomic<uint64_t> told{0};
        hipError_t err = allow_lds(reinterpret_cast<const void *>(kernel), kLds, told);
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
    p.aligned_out = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 && p.ldo % (16 / sizeof(O)) == 0;
    auto tiles = [&](int64_t bm, int64_t bn) { return ((p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn); };
    // a tile's row offsets are 32-bit: 255 ld + depth; and a grid has fewer than 2^32 threads
    const bool in_tiles = aligned16(p.a, p.lda) && aligned16(p.b, p.ldb) && p.lda <= (1 << 22) && p.ldb <= (1 << 22) &&
                          tiles(128, 128) < (1 << 22);
    if (p.m <= 16 && (p.n <= 8192 || !in_tiles)) return launch_direct<1, 1, 8, O>(p, s);
    // Rows that are not aligned have no other way, for any m: no load to LDS takes them.
    // It is slow, since nothing is reused (us, fp32 out, rows k + 1 bytes apart | aligned):
    //   16 x 8192 x 4096     31 | 10       500 x 4096 x 4096    170 | 18
    //   32 x 8192 x 4096     36 | 10       2048 x 4096 x 4096   667 | 45
    //   77 x 1001 x 777      8.2 | 6.5     500 x 50000 x 768    427 | 47
    if (!in_tiles) return launch_direct<4, 2, 4, O>(p, s);
    // The largest tile, not much higher than m, that still gives each of the 256
    // CUs one.  Measured (us, fp32 out; * is what the rule takes):
    //   m x n x k            256x256 128x128 128x64 64x64  32x128 32x64  32x32  direct
    //   8192 x 8192 x 1024   119*    121     129    291
    //   1024 x 8192 x 4096   53      40.9*   51.4   64.4   71     84     99     173
    //   500 x 50000 x 768    49.4    46.6*   51.8   68.6   71     70     95     138
    //   512 x 4096 x 2048    33.6    12.5    11.0*  10.1   11.2   13.6   14.7   27.0
    //   256 x 4096 x 4096    51.3    18.2    15.5   12.7   13.6*  12.0   11.8   25.7
    //   128 x 8192 x 4096    50.2    25.4    16.3   12.9   13.7*  12.3   13.8   25.9
    //   64 x 16384 x 4096    48.7    24.6    17.6   14.6   14.2*  13.5   14.8   25.9
    //   1024 x 1024 x 1024   24.7    9.0     7.5    6.6    6.8*   6.0    6.0    9.3
    //   64 x 8192 x 4096     48.5    23.5    15.6   12.4   13.4   10.5*  10.8   14.9
    //   32 x 16384 x 4096    44.0    23.5    16.8   13.7   14.0   12.9*  13.0   21.9
    //   77 x 1001 x 777      21.3    8.9     7.5    6.9    6.9    5.7    6.6*   7.0
    //   16 x 100000 x 768    27.0    20.0    21.7   20.0   16.9*  17.2   19.3   28.4
    //   8 x 32768 x 1024             8.5     8.1    6.1    5.7*   5.7    5.8    13.0
    // So 32 x 128 is right for a stream of many rows b past few activations, and up to an
    // eighth slower than 32 x 64 where it takes several tiles of activations.
    if (p.m > 128 && p.k >= 1024 && tiles(256, 256) >= 256) return launch_tile<256, 256, 4, 4, 2, O>(p, s);
    if (p.m > 64 && tiles(128, 128) >= 256) return launch_tile<128, 128, 4, 4, 2, O>(p, s);
    if (p.m > 64 && tiles(128, 64) >= 256) return launch_tile<128, 64, 4, 2, 3, O>(p, s);
    if (p.m > 32 && tiles(64, 64) >= 512) return launch_tile<64, 64, 2, 2, 4, O>(p, s);
    // 1 x 100000 x 768: 32 x 128 17.0, 32 x 64 18.3; 1 x 50000 x 1024: 9.8, 12.2
    if (tiles(32, 128) >= 256) return launch_tile<32, 128, 1, 4, 4, O>(p, s);
    if (tiles(32, 64) >= 256) return launch_tile<32, 64, 2, 2, 4, O>(p, s);
    return launch_tile<32, 32, 2, 1, 4, O>(p, s);
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

template <typename T>
hipError_t launch_few_as(const void *x, int64_t ldx, const Product &p, int32_t out_dtype, hipStream_t s) {
    switch (out_dtype) {
        case RT_DTYPE_FLOAT32: return launch_few<T, float>(x, ldx, p, s);
        case RT_DTYPE_BFLOAT16: return launch_few<T, bf16_t>(x, ldx, p, s);
        default: return launch_few<T, fp16_t>(x, ldx, p, s);
    }
}

hipError_t launch_few_rows(const void *x, int32_t dtype, int64_t ldx, const Product &p, int32_t out_dtype, hipStream_t s) {
    switch (dtype) {
        case RT_DTYPE_FLOAT32: return launch_few_as<float>(x, ldx, p, out_dtype, s);
        case RT_DTYPE_BFLOAT16: return launch_few_as<bf16_t>(x, ldx, p, out_dtype, s);
        default: return launch_few_as<fp16_t>(x, ldx, p, out_dtype, s);
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
    const int64_t need = rt_linear_int8_workspace(m, n, k);
    if (need < 0) return RT_EINVAL;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 15u) != 0))
        return RT_EINVAL;
    // with few rows the codes stay in LDS; the checks only look at their place
    static const float none = 0.0f;
    const int64_t ldq = rt::int8_padded(k);
    int8_t *q = need > 0 ? static_cast<int8_t *>(workspace) : nullptr;
    float *scale = need > 0 ? reinterpret_cast<float *>(q + m * ldq) : nullptr;
    const void *place = need > 0 ? static_cast<const void *>(q) : &none;
    rt_status st = rt_check_quantize_rows_int8(x, dtype, m, k, ldx, place, ldq, need > 0 ? scale : &none);
    if (st == RT_OK)
        st = rt_check_matmul_int8(place, ldq, need > 0 ? scale : &none, w, ldw, w_scale, bias, out, out_dtype, ldo, m,
                                  n, k);
    if (st != RT_OK || m == 0) return st;
    if (need == 0) {
        const rt::Product p{nullptr, w, 0, ldw, nullptr, w_scale, bias, out, ldo, m, n, k, false};
        return rt::status_of(rt::launch_few_rows(x, dtype, ldx, p, out_dtype, static_cast<hipStream_t>(stream)));
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err = rt::launch_quantize(x, dtype, m, k, ldx, q, ldq, int(ldq), scale, s);
    const rt::Product p{q, w, ldq, ldw, scale, w_scale, bias, out, ldo, m, n, k, false};
    if (err == hipSuccess) err = rt::launch_matmul(p, out_dtype, s);
    return rt::status_of(err);
}

}  // extern "C"
