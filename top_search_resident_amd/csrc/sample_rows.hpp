// sample_rows.hpp -- one token per row of logits: temperature, top-k, top-p,
// min-p and a draw with a given random number (rt_sample_rows).
//
// Mathematics.  Order the tokens by (logit down, index up).  Every filter keeps
// a prefix of that order, so a row is settled by one border element: the k-th,
// the first at which the running weight reaches top_p of the whole, or the last
// one at or above the min-p logit.  The draw asks the same in index order: the first kept
// element at which the running weight reaches floor(u S) + 1.  Nothing is
// sorted but short lists of candidates.
//
// Weights are whole multiples of 2^-shift of the largest (shift <= 46; those below
// 2^-47 of it count as 0), from a
// 64-bit exponential, and all sums are 64-bit integers: atomics in any order
// give the same sums, so the same inputs give the same token, and a border
// decided in plain 64-bit floating point falls on the same side unless it is
// within about 2^-43 of the whole.
//
// One workgroup per row, a few passes over it:
//   1. the largest logit, and the largest of each of some thousand groups;
//   2a. top-k up to 1024: k of those reach a value that few elements reach; these
//       go to a list, and the list settles the row;
//   2b. otherwise a histogram of the weights, 32 bins an octave, one for each
//       segment of the row;
//   3. the elements of the one bin that the border cuts go to a list, which
//       finds the border;
//   4. the segments' kept weights (bins before the border's, and the list) say
//       which segment the draw falls into; only that one is read again.
//
// What bounds it, in cycles of one workgroup of 1024 on 131072 bf16, top-p: the
// histogram 33.4k of 73k (16 instructions a logit, 10 of them fp64, 4 cycles each),
// passes 1 and 3 8k each from L2 (64 rows; 20k from the last-level cache with 256
// rows, whose 67 MB pass L2's 4 MB an XCD), the searches 3.5k each (a barrier or a
// memory's round trip after the other, which the waves spend waiting).  Short rows,
// and top-k, are latency throughout: 32000 fp32, top-k 50, 22k cycles, of which the
// passes take 6k.
//
// The including file sets RT_SAMPLE_THREADS, the threads of a workgroup.
#include <hip/hip_runtime.h>

#include "../../include/resident_topk.h"
#include "float_types.hpp"
#include "large_lds.hpp"
#include "limits.hpp"
#include "sample_args.hpp"

namespace rt {
namespace {

constexpr int kThreads = RT_SAMPLE_THREADS;  // 1024 or 512
constexpr int kWaves = kThreads / 64;
constexpr int kList = 2048;   // candidates kept in LDS
constexpr int kSmall = 128;   // lists up to here are settled by comparing all pairs
constexpr int kSegs = kThreads / 128;  // parts of a row with a histogram each
constexpr int kSlices = kSampleSlices;  // most workgroups that share a row
constexpr int kSearch = 2048; // bins of a search
constexpr int kOwn = kSearch / kThreads;   // bins and list elements a thread
constexpr int kTeam = kThreads / kSmall;   // threads that compare one of a small list
constexpr int32_t kMostK = kList / 2;      // top-k up to here is looked for by list
constexpr int kAtOnce = 4;    // chunks on their way in passes that do little
constexpr int kPlaces = 4096; // 16-byte places that hold candidates

// ------------------------------------------------------------------- weights

// exp((x - top) / T) as a whole multiple of 2^-shift.  In octaves, t = (x - top)
// log2(e) / T = 49 (sigma - 1), with sigma clamped to [0, 1], which an fma does
// at no cost: NaN gives 0, as anything 49 octaves or more down.  Adding 1.5 * 2^47
// leaves round(32 t) in the low bits, -bin; the rest f (|f| <= 2^-6) gives 2^f by
// a quartic fitted with its constant fixed at 1 (relative error 2^-43.5), and a
// table in LDS the factor 2^(shift - bin / 32), 0 from 47 octaves on; adding 2^52
// rounds to a whole number.  The largest logit is finite here (a row whose
// largest is +inf takes draw_infinite).
//
// The two octaves without weight are room: elements that have none would all add
// to the last bin of the histogram, one after the other.  Each adds to the lane's
// own of the last 64 bins instead, which takes one maximum of two whole numbers.
constexpr int kPerOctave = 32, kOctaves = 49, kMass = kOctaves * kPerOctave + 1;
constexpr int kNone = kMass - 1 - 64;  // bins from here on have no weight
constexpr double kRound = 211106232532992.0;   // 1.5 * 2^47
constexpr double kWhole = 4503599627370496.0;  // 2^52
typedef const __attribute__((address_space(3))) double *lds_doubles;

// a b + c with c in scalar registers.  Written out because the compiler turns an
// fma with a constant addend into a move of the constant and an fmac: two
// instructions where the passes below are bound by their number.
__device__ __forceinline__ double fma_scalar(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}

// The same for four independent sums at a time: an instruction that needs the
// one before it right after an asm block waits a cycle more (s_nop).
struct Four {
    double v[4];
};
__device__ __forceinline__ void fma_four(Four &d, const Four &a, const Four &b, double c) {
    asm("v_fma_f64 %0, %4, %8, %12\n\tv_fma_f64 %1, %5, %9, %12\n\t"
        "v_fma_f64 %2, %6, %10, %12\n\tv_fma_f64 %3, %7, %11, %12"
        : "=&v"(d.v[0]), "=&v"(d.v[1]), "=&v"(d.v[2]), "=&v"(d.v[3])
        : "v"(a.v[0]), "v"(a.v[1]), "v"(a.v[2]), "v"(a.v[3]), "v"(b.v[0]), "v"(b.v[1]), "v"(b.v[2]), "v"(b.v[3]),
          "s"(c));
}
__device__ __forceinline__ void fma_four(Four &d, const Four &a, double b, double c) {  // b in vector registers
    asm("v_fma_f64 %0, %4, %8, %9\n\tv_fma_f64 %1, %5, %8, %9\n\t"
        "v_fma_f64 %2, %6, %8, %9\n\tv_fma_f64 %3, %7, %8, %9"
        : "=&v"(d.v[0]), "=&v"(d.v[1]), "=&v"(d.v[2]), "=&v"(d.v[3])
        : "v"(a.v[0]), "v"(a.v[1]), "v"(a.v[2]), "v"(a.v[3]), "v"(b), "s"(c));
}

struct Weights {
    double top, rate;  // rate = log2(e) / (kOctaves T)
    lds_doubles zero;  // the factor of bin 0; bin b's is at zero[-b]
    double c4, c3, c2, c1, one, per_unit;

    __device__ __forceinline__ int split(float x, double *f) const {  // -bin
        const double sigma = fmin(fmax(fma(double(x) - top, rate, 1.0), 0.0), 1.0);
        const double m = fma_scalar(sigma, double(kOctaves), kRound - kOctaves);
        *f = fma(sigma, double(kOctaves), (kRound - kOctaves) - m);
        return int(uint32_t(__builtin_bit_cast(uint64_t, m)));
    }
    __device__ __forceinline__ double power(float x, int *bin) const {  // 2^f, and -bin
        double f;
        *bin = split(x, &f);
        return fma(fma_scalar(fma_scalar(fma_scalar(f, kC4, kC3), f, kC2), f, kC1), f, 1.0);
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {
        int bin;
        const double p = power(x, &bin);
        return __builtin_bit_cast(uint64_t, fma_scalar(p, zero[bin], kWhole)) & 0x000fffffffffffffull;
    }
    // For four elements: -bin, and 2^f alone in units of 2^-shift, for sums within
    // one bin.  The polynomial is scaled by 2^-1074 besides (sample_units.hpp): fp64
    // below 2^-1022 are whole multiples of that, and their bits are the multiple itself.
    __device__ __forceinline__ void units(const float *x, int *bin, uint64_t *unit) const {
        double octaves = kOctaves, lead = c4;
        asm("" : "+v"(octaves), "+v"(lead));  // an fma reads at most one scalar pair
        Four sigma, m, f, p;
#pragma unroll
        for (int e = 0; e < 4; ++e) sigma.v[e] = fmin(fmax(fma(double(x[e]) - top, rate, 1.0), 0.0), 1.0);
        fma_four(m, sigma, octaves, kRound - kOctaves);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bin[e] = int(uint32_t(__builtin_bit_cast(uint64_t, m.v[e])));
            f.v[e] = fma(sigma.v[e], octaves, (kRound - kOctaves) - m.v[e]);
        }
        fma_four(p, f, lead, c3);
        fma_four(p, p, f, c2);
        fma_four(p, p, f, c1);
        fma_four(p, p, f, one);
#pragma unroll
        for (int e = 0; e < 4; ++e) unit[e] = __builtin_bit_cast(uint64_t, p.v[e]);
    }
    __device__ __forceinline__ uint64_t whole(uint64_t sum, int bin) const {  // such a sum, with the bin's factor
        return bin ? uint64_t(__builtin_rint(double(sum) * (zero[-bin] * per_unit))) : sum;
    }
};

// fp32 as a whole number that orders the same (-0.0 as +0.0), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ float next_below(float x) {
    const uint32_t o = ordered(x) - 1;
    return unordered(o == 0x7fffffffu ? o - 1 : o);  // below 0.0 is not -0.0
}

// Order of the elements as one 64-bit number, larger first: the logit, then the
// index from the top down.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t idx) {
    return (uint64_t(ordered(x)) << 32) | uint32_t(~idx);
}
__device__ __forceinline__ float key_value(uint64_t key) { return unordered(uint32_t(key >> 32)); }
__device__ __forceinline__ uint32_t key_index(uint64_t key) { return ~uint32_t(key); }

// What is kept by value: logits above `over`, and those equal to `equal` up to index `upto`.
struct Cut {
    float over = -INFINITY, equal = -INFINITY;
    uint32_t upto = 0;

    __device__ __forceinline__ bool operator()(float x, uint32_t i) const {
        return (x > over) | ((x == equal) & (i <= upto));
    }
    __device__ __forceinline__ void from_key(uint64_t key) { over = equal = key_value(key), upto = key_index(key); }
    __device__ __forceinline__ void from_value(float least) {  // and at or above `least`
        if (least > over) over = next_below(least), equal = least, upto = 0xffffffffu;
    }
};

// ------------------------------------------------------------- block helpers

struct Shared {
    uint64_t bin[kSegs * kMass];
    uint64_t list[kList];
    uint64_t weight[kSmall];
    double factor[kMass];
    uint64_t seg[kSlices];
    uint64_t wave_sum[kWaves];
    uint64_t lo, hi, before;
    uint32_t count, found;
    float f[kWaves], g[kWaves];
    float edge[2];
};
static_assert(kSearch <= kSegs * kMass && kPlaces / 2 <= kSegs * kMass, "find_first uses the histograms' memory");

typedef unsigned long long ull;
__device__ __forceinline__ void add64(uint64_t *p, uint64_t v) {
    __hip_atomic_fetch_add(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}

__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d) {
    const uint32_t lo = __shfl_xor(int(uint32_t(v)), d), hi = __shfl_xor(int(uint32_t(v >> 32)), d);
    return (uint64_t(hi) << 32) | lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t dpp64(uint64_t v) {  // 0 where the pattern has no source
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(v)), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(v >> 32)), CTRL, ROWS, 0xf, false);
    return (uint64_t(hi) << 32) | lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp32(float v, float none) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(none), __float_as_int(v), CTRL, ROWS, 0xf, false));
}
// Largest and smallest of the wave's 64 lanes (no NaN).
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp32<0x111, 0xf>(v, -INFINITY));
    v = fmaxf(v, dpp32<0x112, 0xf>(v, -INFINITY));
    v = fmaxf(v, dpp32<0x114, 0xf>(v, -INFINITY));
    v = fmaxf(v, dpp32<0x118, 0xf>(v, -INFINITY));
    v = fmaxf(v, dpp32<0x142, 0xa>(v, -INFINITY));
    v = fmaxf(v, dpp32<0x143, 0xc>(v, -INFINITY));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_min(float v) { return -wave_max(-v); }

__device__ __forceinline__ uint64_t lane64(uint64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(int(uint32_t(v)), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(int(uint32_t(v >> 32)), lane);
    return (uint64_t(hi) << 32) | lo;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t max_dpp64(uint64_t v) {
    const uint64_t o = dpp64<CTRL, ROWS>(v);
    return o > v ? o : v;
}
__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
    v = max_dpp64<0x111, 0xf>(v);
    v = max_dpp64<0x112, 0xf>(v);
    v = max_dpp64<0x114, 0xf>(v);
    v = max_dpp64<0x118, 0xf>(v);
    v = max_dpp64<0x142, 0xa>(v);
    v = max_dpp64<0x143, 0xc>(v);
    return lane64(v, 63);
}

// Running sum over the 16 lanes of each row, over the wave's 64 lanes (row shifts, then
// the last lane of a row to the next one, of the first half to the second).
__device__ __forceinline__ uint64_t row_scan(uint64_t v) {
    v += dpp64<0x111, 0xf>(v);
    v += dpp64<0x112, 0xf>(v);
    v += dpp64<0x114, 0xf>(v);
    v += dpp64<0x118, 0xf>(v);
    return v;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
    v = row_scan(v);
    v += dpp64<0x142, 0xa>(v);
    v += dpp64<0x143, 0xc>(v);
    return v;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ uint32_t wave_scan32(uint32_t v) {
    v += dpp_u32<0x111, 0xf>(v);
    v += dpp_u32<0x112, 0xf>(v);
    v += dpp_u32<0x114, 0xf>(v);
    v += dpp_u32<0x118, 0xf>(v);
    v += dpp_u32<0x142, 0xa>(v);
    v += dpp_u32<0x143, 0xc>(v);
    return v;
}
__device__ __forceinline__ uint64_t wave_add(uint64_t v) { return lane64(wave_scan(v), 63); }

// Running sum over the block's threads: what comes before this thread's `own`,
// and the sum of all.  Whatever all 16 waves do here costs 16 cycles an
// instruction, so the waves' sums are scanned by 16 lanes of each.
__device__ __forceinline__ uint64_t block_scan(Shared &sh, uint64_t own, uint64_t *all) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t scan = wave_scan(own);
    __syncthreads();
    if (lane == 63) sh.wave_sum[wave] = scan;
    __syncthreads();
    const uint64_t waves = row_scan((lane & 15) < kWaves ? sh.wave_sum[lane & 15] : 0);
    *all = lane64(waves, 15);
    const uint64_t base = wave ? lane64(waves, (wave - 1) & 15) : 0;
    return base + scan - own;
}
__device__ __forceinline__ uint64_t block_add(Shared &sh, uint64_t v) {
    uint64_t all;
    (void)block_scan(sh, v, &all);
    return all;
}

// The least number of units that is `part` of `whole`, at least 1.
__device__ __forceinline__ uint64_t at_least(float part, uint64_t whole) {
    const uint64_t n = uint64_t(__builtin_ceil(double(part) * double(whole)));
    return n < 1 ? 1 : (n > whole ? whole : n);
}

// The least number of units above u of `whole`; never more than `whole`, so that
// some running sum always reaches it.
__device__ __forceinline__ uint64_t above(float u, uint64_t whole) {
    if (u >= 1.0f) return whole;
    const uint64_t n = u > 0.0f ? uint64_t(double(u) * double(whole)) + 1 : 1;
    return n > whole ? whole : n;
}

// A thread's share of 2048 bins: bins kOwn t ...
struct alignas(16) Own {
    uint64_t v[kOwn];
};
__device__ __forceinline__ Own own_bins(const Shared &sh) {
    Own own;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own.v[i] = sh.bin[kOwn * threadIdx.x + i];
    return own;
}

// The first bin at which the running sum reaches target(sum of all) (taken as at
// least 1 and at most the sum); *before is the sum ahead of it.
template <typename Target>
__device__ __forceinline__ int find_bin(Shared &sh, const Own &own, Target target_of, uint64_t *before,
                                        uint64_t *target) {
    uint64_t all, mine = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) mine += own.v[i];
    uint64_t run = block_scan(sh, mine, &all);
    uint64_t t = target_of(all);
    t = t > all ? all : t;
    if (run < t && run + mine >= t) {  // exactly one thread, where all > 0
        int at = 0;
#pragma unroll
        for (int i = 0; i + 1 < kOwn; ++i)
            if (at == i && run + own.v[i] < t) run += own.v[i], at = i + 1;
        sh.found = kOwn * threadIdx.x + at;
        sh.before = run;
    }
    __syncthreads();
    *before = sh.before;
    *target = t;
    return all ? int(sh.found) : 0;
}

// The element, among those each(f) presents as f(key, weight), at which the
// weight summed from the largest key down first reaches `target`.  Each round
// narrows to one of 2048 bins of what is left.
template <typename Each>
__device__ __forceinline__ uint64_t find_first(Shared &sh, Each each, uint64_t target) {
    uint64_t lo = 0, hi = ~uint64_t(0);
    for (;;) {
        uint64_t least = ~uint64_t(0), most = 0;
        each([&](uint64_t key, uint64_t) {
            if (key >= lo && key <= hi) {
                least = key < least ? key : least;
                most = key > most ? key : most;
            }
        });
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            const uint64_t a = shfl_xor64(least, o), b = shfl_xor64(most, o);
            least = a < least ? a : least;
            most = b > most ? b : most;
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.lo = ~uint64_t(0), sh.hi = 0;
        for (int i = threadIdx.x; i < kSearch; i += kThreads) sh.bin[i] = 0;
        __syncthreads();
        if ((threadIdx.x & 63) == 0) {
            atomicMin(reinterpret_cast<ull *>(&sh.lo), ull(least));
            atomicMax(reinterpret_cast<ull *>(&sh.hi), ull(most));
        }
        __syncthreads();
        least = sh.lo;
        most = sh.hi;
        if (least >= most) return most;  // one element (or, of an empty range, 0)
        const int bits = 64 - __builtin_clzll(most - least);
        const int drop = bits > 11 ? bits - 11 : 0;
        each([&](uint64_t key, uint64_t w) {
            if (key >= least && key <= most) add64(&sh.bin[(most - key) >> drop], w);
        });
        __syncthreads();
        uint64_t before, t;
        const uint64_t b = find_bin(sh, own_bins(sh), [&](uint64_t) { return target; }, &before, &t);
        if (t == 0) return most;  // no weight at all
        target = t - before;
        hi = most - (b << drop);
        const uint64_t width = (uint64_t(1) << drop) - 1;
        lo = hi - least > width ? hi - width : least;
    }
}

// ------------------------------------------------------------------- the row

// A type's codes as whole numbers, several to a register: nonnegative values order
// as their codes, negative ones the other way round.
template <typename T>
struct CodesOf {
    typedef uint16_t U __attribute__((ext_vector_type(2)));
    typedef int16_t S __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kSign = 0x8000u, kInf = __is_same(T, bf16_t) ? 0x7f80u : 0x7c00u;
    static __device__ __forceinline__ uint32_t most(S v) { return uint32_t(uint16_t(v[0] > v[1] ? v[0] : v[1])); }
    static __device__ __forceinline__ uint32_t least(U v) { return v[0] < v[1] ? v[0] : v[1]; }
    static __device__ __forceinline__ float value(uint32_t code) {
        return static_cast<float>(__builtin_bit_cast(T, uint16_t(code)));
    }
    static __device__ __forceinline__ uint32_t down(float x) {  // of the largest value up to x >= 0
        if constexpr (__is_same(T, bf16_t)) return __float_as_uint(x) >> 16;
        const uint32_t c = __builtin_bit_cast(uint16_t, static_cast<T>(x));
        return value(c) > x ? c - 1 : c;
    }
};
template <>
struct CodesOf<float> {
    typedef uint32_t U;
    typedef int32_t S;
    static constexpr uint32_t kSign = 0x80000000u, kInf = 0x7f800000u;
    static __device__ __forceinline__ uint32_t most(S v) { return uint32_t(v); }
    static __device__ __forceinline__ uint32_t least(U v) { return v; }
    static __device__ __forceinline__ float value(uint32_t code) { return __uint_as_float(code); }
    static __device__ __forceinline__ uint32_t down(float x) { return __float_as_uint(x); }
};

// The largest of many 16 bytes: of the nonnegative ones the largest signed code,
// and where there are none the smallest unsigned one.  Two packed instructions
// for two 2-byte logits, where unpacking, comparing and selecting take six.  A
// positive NaN hides what is below it: nan() says so.
template <typename T>
struct Largest {
    typedef CodesOf<T> C;
    typename C::S most = typename C::S(0) + typename C::S(sizeof(T) == 2 ? -32768 : int32_t(0x80000000u));
    typename C::U least = ~typename C::U(0);

    __device__ __forceinline__ void add(u32x4 x) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            most = __builtin_elementwise_max(most, __builtin_bit_cast(typename C::S, uint32_t(x[d])));
            least = __builtin_elementwise_min(least, __builtin_bit_cast(typename C::U, uint32_t(x[d])));
        }
    }
    __device__ __forceinline__ bool nan() const {
        const uint32_t m = C::most(most);
        return m < C::kSign && m > C::kInf;
    }
    __device__ __forceinline__ float value() const {
        const uint32_t m = C::most(most), n = C::least(least);
        return m < C::kSign ? C::value(m) : (n <= (C::kSign | C::kInf) ? C::value(n) : -INFINITY);
    }
};

// The logits in [lo, last], both of one sign, as a run of codes.
template <typename T>
struct Codes {
    typedef CodesOf<T> C;
    typename C::U first;
    uint32_t width;
    bool usable, empty;  // empty: the type has no value there

    __device__ __forceinline__ Codes(float lo, float last) {
        const bool negative = last < 0.0f;
        const float small = negative ? -last : lo, large = negative ? -lo : last;  // magnitudes
        const uint32_t below = C::down(small), to = C::down(large);
        const uint32_t from = C::value(below) < small ? below + 1 : below;
        usable = small > 0.0f;
        empty = usable && from > to;
        width = to - from;
        first = typename C::U(0) + typename C::U(from | (negative ? C::kSign : 0u));
    }
    __device__ __forceinline__ bool any(u32x4 x) const {
        typename C::U m = ~typename C::U(0);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const typename C::U off = __builtin_bit_cast(typename C::U, uint32_t(x[d])) - first;
            m = __builtin_elementwise_min(m, off);
        }
        return C::least(m) <= width;
    }
};

// Chunk c of thread t holds elements (c * kThreads + t) * E .. of the row; elements
// past its end read as -inf.
template <typename T>
struct Row {
    static constexpr int E = 16 / sizeof(T);
    static constexpr int64_t kChunk = int64_t(kThreads) * E;
    static constexpr uint32_t none =  // -inf
        sizeof(T) == 4 ? 0xff800000u : (__is_same(T, bf16_t) ? 0xff80ff80u : 0xfc00fc00u);
    const T *p;
    int64_t v;
    int begin, end, per;  // the chunks that the passes below go over, and how many make a segment

    __device__ __forceinline__ Row(const SampleArgs &a, int64_t r) : p(static_cast<const T *>(a.logits) + r * a.ld), v(a.v) {
        begin = 0;
        end = int((v + kChunk - 1) / kChunk);
        per = (end + kSegs - 1) / kSegs;
    }
    __device__ __forceinline__ uint32_t index(int c, uint32_t t = threadIdx.x) const {
        return uint32_t(c) * uint32_t(kChunk) + t * E;
    }
    __device__ __forceinline__ int segment(uint32_t idx) const { return int(idx / uint32_t(kChunk)) / per; }
    __device__ __forceinline__ u32x4 load_whole(int64_t c, uint32_t t = threadIdx.x) const {
        return load16(p + c * kChunk + int64_t(t) * E);
    }
    // The chunk that holds the row's last elements: 16 bytes that end with the
    // row, moved down, -inf behind them.
    __device__ __forceinline__ u32x4 load_last(int64_t c, uint32_t t = threadIdx.x) const {
        const int64_t i = c * kChunk + int64_t(t) * E;
        u32x4 x = {none, none, none, none};
        if (i + E <= v) return load16(p + i);
        if (i >= v) return x;
        if (v >= E) x = load16(p + v - E);
        const int n = v >= E ? int(i + E - v) : 0;  // elements to move down by
        if (v < E)
            for (int64_t j = v - 1; j >= 0; --j) {  // a row shorter than 16 bytes, from the last one down
                if constexpr (sizeof(T) == 4) {
                    x = u32x4{*reinterpret_cast<global_ptr<uint32_t>>((uintptr_t)(p + j)), x[0], x[1], x[2]};
                } else {
                    const uint32_t h = *reinterpret_cast<global_ptr<uint16_t>>((uintptr_t)(p + j));
                    x = u32x4{(x[0] << 16) | h, (x[1] << 16) | (x[0] >> 16), (x[2] << 16) | (x[1] >> 16),
                              (x[3] << 16) | (x[2] >> 16)};
                }
            }
        for (int j = 0; j < n; ++j) {
            if constexpr (sizeof(T) == 4)
                x = u32x4{x[1], x[2], x[3], none};
            else
                x = u32x4{(x[0] >> 16) | (x[1] << 16), (x[1] >> 16) | (x[2] << 16), (x[2] >> 16) | (x[3] << 16),
                          (x[3] >> 16) | (none << 16)};
        }
        return x;
    }
    __device__ __forceinline__ u32x4 load(int64_t c, uint32_t t = threadIdx.x) const {
        return (c + 1) * kChunk <= v ? load_whole(c, t) : load_last(c, t);
    }
    // f(16 bytes, chunk) over the row's chunks.  Two chunks are read while two are
    // worked on: the registers are named apart, since handing a load on from one
    // to the next would wait for it.
    template <typename F>
    __device__ __forceinline__ void each_chunk(F f) const {
        const int whole = min(end, int(v / kChunk)), last = whole - 1;
        int c = begin;
        if (c + 4 <= whole) {
            u32x4 a0 = load_whole(c), a1 = load_whole(c + 1);
#pragma unroll 1
            for (; c + 4 <= whole; c += 4) {
                const u32x4 b0 = load_whole(c + 2), b1 = load_whole(c + 3);
                f(a0, c);
                f(a1, c + 1);
                a0 = load_whole(min(c + 4, last));
                a1 = load_whole(min(c + 5, last));
                f(b0, c + 2);
                f(b1, c + 3);
            }
        }
#pragma unroll 1
        for (; c < end; ++c) f(load(c), c);
    }
    // The same for chunks c .. c1 - 1 with kAtOnce on their way at once, for passes that
    // do little with them; behind the last, -inf once more.
    template <typename F>
    __device__ __forceinline__ void each_of_many(F f, int c, int c1) const {
        const int whole = min(c1, int(v / kChunk));
        u32x4 part = {none, none, none, none};
        if (whole < c1) part = load_last(whole);
#pragma unroll 1
        for (; c < whole; c += kAtOnce) {
            u32x4 x[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) x[i] = load_whole(min(c + i, whole - 1));
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const bool in = c + i < whole;
                f(u32x4{in ? x[i][0] : none, in ? x[i][1] : none, in ? x[i][2] : none, in ? x[i][3] : none}, c + i);
            }
        }
        if (whole < c1) f(part, whole);
    }
    // f(value, index) of each element of chunks c .. c1 - 1, one chunk at a time: for
    // the rarely taken paths, where small code matters more
    template <typename F>
    __device__ __forceinline__ void each(F f, int c, int c1) const {
#pragma unroll 1
        for (; c < c1; ++c) {
            const u32x4 x = load(c);
            const uint32_t i = index(c);
#pragma unroll
            for (int e = 0; e < E; ++e) f(element<T>(x, e), i + e);
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        each(f, begin, end);
    }
    __device__ __forceinline__ float largest() const {  // of this thread's elements, NaN passed over
        float m = -INFINITY;
        each([&](float y, uint32_t) { m = y > m ? y : m; });
        return m;
    }
    // The keys of the 16 bytes' elements in [lo, last] (no logit is infinite here) to
    // sh.list, up to kList of them; sh.count counts them all.
    static __device__ __forceinline__ void take(Shared &sh, u32x4 x, uint32_t i, float lo, float last) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float y = element<T>(x, e);
            if (y >= lo && y <= last) {
                const uint32_t at = atomicAdd(&sh.count, 1u);
                if (at < kList) sh.list[at] = order_key(y, i + e);
            }
        }
    }
    // The whole row's; returns sh.count.  First the places of the 16 bytes that hold
    // any (a thread's as bits, noted together), then their elements, a thread each.
    __device__ __forceinline__ uint32_t collect(Shared &sh, float lo, float last) const {
        const Codes<T> codes(lo, last);
        if (codes.empty) return 0;
        uint32_t *places = reinterpret_cast<uint32_t *>(sh.bin);
        __syncthreads();  // sh.bin, sh.found and sh.count have been read
        if (threadIdx.x == 0) sh.count = 0, sh.found = 0;
        __syncthreads();
        for (int c0 = begin; c0 < end; c0 += 32) {
            const int c1 = min(c0 + 32, end);
            uint32_t hit = 0;  // a bit for each of this thread's next 32 places
            if (codes.usable) {
                each_of_many([&](u32x4 x, int c) { hit |= codes.any(x) ? 1u << (c - c0) : 0u; }, c0, c1);
            } else {
                each([&](float y, uint32_t i) { hit |= y >= lo && y <= last ? 1u << (int(i / kChunk) - c0) : 0u; }, c0, c1);
            }
            if (__any(hit != 0)) {
                uint32_t at = places_for(sh.found, __popc(hit));
                for (; hit != 0 && at < kPlaces; hit &= hit - 1, ++at)
                    places[at] = uint32_t(c0 + __builtin_ctz(hit)) * kThreads + threadIdx.x;
            }
        }
        __syncthreads();
        const uint32_t n = sh.found;
        if (n > kPlaces) return kList + 1;
        for (uint32_t j0 = 0; j0 < n; j0 += kThreads) {
            const uint32_t j = j0 + threadIdx.x;
            u32x4 x = {none, none, none, none};
            uint32_t i = 0, hit = 0;
            if (j < n) {
                const uint32_t c = places[j] / kThreads, t = places[j] % kThreads;
                x = load(c, t);
                i = index(c, t);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float y = element<T>(x, e);
                hit |= (y >= lo) & (y <= last) ? 1u << e : 0u;
            }
            if (!__any(hit != 0)) continue;
            uint32_t at = places_for(sh.count, __popc(hit));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if ((hit >> e & 1u) && at < kList) sh.list[at] = order_key(element<T>(x, e), i + e);
                at += hit >> e & 1u;
            }
        }
        __syncthreads();
        return sh.count;
    }
    // The first of `own` places after `count`, which it moves on by the wave's.
    static __device__ __forceinline__ uint32_t places_for(uint32_t &count, uint32_t own) {
        const uint32_t upto = wave_scan32(own);
        uint32_t at = 0;
        if ((threadIdx.x & 63) == 63) at = atomicAdd(&count, upto);
        return __builtin_amdgcn_readlane(int(at), 63) + upto - own;
    }
    // The same without an end, where few threads' largest logit `own` reaches lo:
    // the waves take those threads' places one by one, a chunk a lane.
    __device__ __forceinline__ uint32_t collect_from(Shared &sh, float lo, float own) const {
        uint32_t *threads = reinterpret_cast<uint32_t *>(sh.bin);
        __syncthreads();  // sh.bin, sh.found and sh.count have been read
        if (threadIdx.x == 0) sh.count = 0, sh.found = 0;
        __syncthreads();
        if (own >= lo) threads[atomicAdd(&sh.found, 1u)] = threadIdx.x;
        __syncthreads();
        const uint32_t n = sh.found;
        for (uint32_t h = threadIdx.x >> 6; h < n; h += kWaves) {
            const uint32_t t = threads[h];
            for (int c = begin + (threadIdx.x & 63); c < end; c += 64) {
                take(sh, load(c, t), index(c, t), lo, INFINITY);
            }
        }
        __syncthreads();
        return sh.count;
    }
};

// A row's settings.
struct Settings {
    float temperature, top_p, min_p, u;
    int32_t top_k;
    bool single;  // only the first token of the order is kept

    __device__ __forceinline__ Settings(const SampleArgs &a, int64_t r) {
        temperature = a.set.temperature;
        top_k = a.set.top_k;
        top_p = a.set.top_p;
        min_p = a.set.min_p;
        if (a.set.temperatures) temperature = a.set.temperatures[r];
        if (a.set.top_ks) top_k = a.set.top_ks[r];
        if (a.set.top_ps) top_p = a.set.top_ps[r];
        if (a.set.min_ps) min_p = a.set.min_ps[r];
        u = a.u[r];
        single = !(temperature > 0.0f) || top_k == 1 || !(top_p > 0.0f) || !(min_p <= 1.0f);
        if (top_k < 0 || top_k >= a.v) top_k = 0;
    }
    // min-p as a logit: the smallest fp32 at or above top + T ln(min_p); at an
    // infinite T all weigh the same
    __device__ __forceinline__ float least(float top) const {
        if (!(min_p > 0.0f) || temperature == INFINITY) return -INFINITY;
        const float x = __double2float_ru(double(top) + double(temperature) * log(double(min_p)));
        return x <= top ? x : top;
    }
};

struct Output {
    int32_t *token;
    float *prob;
};

__device__ __forceinline__ void write_row(Output out, int64_t r, uint32_t token, float prob) {
    out.token[r] = int32_t(token);
    if (out.prob) out.prob[r] = prob;
}

// By the thread that found it.
__device__ __forceinline__ void write_drawn(Output out, int64_t r, uint32_t token, float x, uint64_t sum,
                                            const Weights &weight) {
    int bin;
    const double w = weight.power(x, &bin);
    write_row(out, r, token, float(w * weight.zero[bin] / double(sum)));  // not rounded to whole units
}

// f(j) for j = g, g + kTeam, ... below n; what f reads of four at a time is on its way together.
template <typename F>
__device__ __forceinline__ void each_of_small(uint32_t n, uint32_t g, F f) {
    uint32_t j = g;
#pragma unroll 1
    for (; j + 3 * kTeam < n; j += 4 * kTeam) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f(j + e * kTeam);
    }
#pragma unroll 1
    for (; j < n; j += kTeam) f(j);
}

// find_first for at most kOwn elements a thread (weight 0: none), `n` in all, with
// keys in [least, most] (most = 0: anywhere).  Once at most kSmall are left, kTeam threads
// compare one of them with all.  Returns true to the one thread that holds the element
// (the last one, where the weights do not reach the target; key 0, where there
// are none).  Uses sh.list and sh.bin.
struct Share {
    uint64_t key[kOwn], weight[kOwn];
};
__device__ __forceinline__ bool find_in_shares(Shared &sh, Share p, uint32_t n, uint64_t least, uint64_t most,
                                              uint64_t target, uint64_t *found) {
    const int t = threadIdx.x, lane = t & 63;
    for (;;) {
        if (n > kSmall && most != 0) {
            __syncthreads();
            for (int i = t; i < kSearch; i += kThreads) sh.bin[i] = 0;
            __syncthreads();
            const int bits = 64 - __builtin_clzll(most - least);  // more than one key: they differ
            const int drop = bits > 11 ? bits - 11 : 0;
#pragma unroll
            for (int e = 0; e < kOwn; ++e)
                if (p.weight[e]) add64(&sh.bin[(most - p.key[e]) >> drop], p.weight[e]);
            __syncthreads();
            uint64_t before, aim;
            const uint64_t b = find_bin(sh, own_bins(sh), [&](uint64_t) { return target; }, &before, &aim);
            target = aim - before;
#pragma unroll
            for (int e = 0; e < kOwn; ++e)
                if (p.weight[e] && ((most - p.key[e]) >> drop) != b) p.weight[e] = 0;
        }
        // what is left: how many, between which keys, and the first kSmall side by side
        __syncthreads();
        if (t == 0) sh.lo = ~uint64_t(0), sh.hi = 0, sh.count = 0;
        __syncthreads();
        uint64_t held[kOwn], any = 0;
        uint32_t ours = 0;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) {
            held[e] = __ballot(p.weight[e] != 0);
            any |= held[e];
            ours += __popcll(held[e]);
        }
        if (any) {
            uint64_t low = ~uint64_t(0), high = 0;
#pragma unroll
            for (int e = 0; e < kOwn; ++e)
                if (p.weight[e]) {
                    low = p.key[e] < low ? p.key[e] : low;
                    high = p.key[e] > high ? p.key[e] : high;
                }
            low = ~wave_max64(~low);
            high = wave_max64(high);
            uint32_t at = 0;
            if (lane == 0) {
                atomicMin(reinterpret_cast<ull *>(&sh.lo), ull(low));
                atomicMax(reinterpret_cast<ull *>(&sh.hi), ull(high));
                at = atomicAdd(&sh.count, ours);
            }
            at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
            for (int e = 0; e < kOwn; ++e) {
                const uint32_t place = at + __popcll(held[e] & ((uint64_t(1) << lane) - 1));
                if (p.weight[e] && place < kSmall) sh.list[place] = p.key[e], sh.weight[place] = p.weight[e];
                at += __popcll(held[e]);
            }
        }
        __syncthreads();
        n = sh.count;
        least = sh.lo;
        most = sh.hi;
        *found = 0;
        if (n == 0) return t == 0;
        if (n <= kSmall) {
            const uint32_t i = t / kTeam, g = t % kTeam;
            if (i >= n) return false;
            const uint64_t key = sh.list[i], w = sh.weight[i];
            uint64_t run = 0;
            for (uint32_t j = g; j < n; j += kTeam) {
                const uint64_t other = sh.list[j], one = sh.weight[j];
                run += other > key ? one : 0;
            }
#pragma unroll
            for (int o = 1; o < kTeam; o <<= 1) run += shfl_xor64(run, o);
            *found = key;
            return g == 0 && run < target && (run + w >= target || key == least);
        }
    }
}

// sh.list[0, n), kOwn elements a thread, with their weights.
__device__ __forceinline__ Share share_of_list(Shared &sh, uint32_t n, const Weights &weight) {
    Share p;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) {
        const uint32_t j = threadIdx.x + e * kThreads;
        p.key[e] = j < n ? sh.list[j] : 0;
        p.weight[e] = j < n ? weight(key_value(p.key[e])) : 0;
    }
    return p;
}

// The key find_in_shares finds, to all threads (0: no weight at all).
__device__ __forceinline__ uint64_t find_key(Shared &sh, const Share &p, uint32_t n, uint64_t least, uint64_t most,
                                             uint64_t target) {
    uint64_t key;
    if (find_in_shares(sh, p, n, least, most, target, &key)) sh.before = key;
    __syncthreads();
    return sh.before;
}

__device__ __forceinline__ uint64_t weight_of(const Share &p) {
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < kOwn; ++e) sum += p.weight[e];
    return sum;
}

__device__ __forceinline__ void keep_from(Share &p, uint64_t key) {
#pragma unroll
    for (int e = 0; e < kOwn; ++e)
        if (p.key[e] < key) p.weight[e] = 0;
}

// The rest of a row whose kept elements are all in sh.list[0, n): top-k and
// top-p (where on), min-p and the draw.  A barrier has followed the list.
// All its logits reach `from` (-inf: not known); row_value(i) is logit i of v.
template <typename Value>
__device__ __forceinline__ void draw_from_list(Shared &sh, Output out, int64_t r, uint32_t n, const Weights &weight,
                                               const Settings &set, float least, float from, uint32_t v,
                                               Value row_value) {
    const uint32_t t = threadIdx.x;
    const uint32_t limit = set.top_k ? min(n, uint32_t(set.top_k)) : n;
    if (n <= kSmall) {
        // kTeam neighbouring threads compare an element with all of them
        const uint32_t i = t / kTeam, g = t % kTeam;
        const bool mine = i < n && g == 0;
        const uint64_t key = i < n ? sh.list[i] : 0;
        const float x = i < n ? key_value(key) : -INFINITY;
        const uint64_t w = weight(x);
        if (mine) sh.weight[i] = w;
        if (t == 0) sh.hi = 0;
        __syncthreads();
        uint32_t rank = 0;
        uint64_t pre = 0;
        each_of_small(n, g, [&](uint32_t j) {
            const bool ahead = sh.list[j] > key;
            const uint64_t one = sh.weight[j];
            rank += ahead ? 1 : 0;
            pre += ahead ? one : 0;
        });
#pragma unroll
        for (int o = 1; o < kTeam; o <<= 1) {
            rank += uint32_t(__shfl_xor(int(rank), o));
            pre += shfl_xor64(pre, o);
        }
        if (mine && rank == limit - 1) sh.before = pre + w;
        __syncthreads();
        bool kept = i < n && rank < limit && x >= least;
        if (set.top_p < 1.0f) kept = kept && pre < at_least(set.top_p, sh.before);
        if (mine) {
            sh.weight[i] = kept ? w : 0;
            if (kept) atomicMax(reinterpret_cast<ull *>(&sh.hi), ull(pre + w));  // kept ones are first in order
        }
        __syncthreads();
        const uint64_t sum = sh.hi, aim = above(set.u, sum);
        uint64_t run = 0;
        each_of_small(n, g, [&](uint32_t j) {
            const uint64_t other = sh.list[j], one = sh.weight[j];
            run += key_index(other) < key_index(key) ? one : 0;
        });
#pragma unroll
        for (int o = 1; o < kTeam; o <<= 1) run += shfl_xor64(run, o);
        if (mine && kept && run < aim && run + w >= aim) write_drawn(out, r, key_index(key), x, sum, weight);
        return;
    }
    Share p = share_of_list(sh, n, weight);
    const uint64_t first_key = uint64_t(ordered(from)) << 32;
    const uint64_t last_key = from > -INFINITY ? uint64_t(ordered(float(weight.top))) << 32 | 0xffffffffu : 0;
    if (limit < n) {
        Share ones = p;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) ones.weight[e] = p.key[e] ? 1 : 0;
        keep_from(p, find_key(sh, ones, n, first_key, last_key, limit));
    }
    if (set.top_p < 1.0f) {
        const uint64_t z = block_add(sh, weight_of(p));
        keep_from(p, find_key(sh, p, n, first_key, last_key, at_least(set.top_p, z)));
    }
#pragma unroll
    for (int e = 0; e < kOwn; ++e)
        if (!(key_value(p.key[e]) >= least)) p.weight[e] = 0;
    const uint64_t sum = block_add(sh, weight_of(p));
#pragma unroll
    for (int e = 0; e < kOwn; ++e) p.key[e] = uint32_t(p.key[e]);  // by index, the lowest first
    uint64_t key;
    if (find_in_shares(sh, p, n, ~(v - 1), 0xffffffffu, above(set.u, sum), &key)) {
        const uint32_t token = key_index(key);
        write_drawn(out, r, token, row_value(token), sum, weight);
    }
}

// The draw once the segments' kept weights are in sh.seg: the element of the
// row at which the running weight of what `cut` keeps reaches above(u, sum).
template <typename T>
__device__ __forceinline__ void draw_from_row(Shared &sh, Output out, int64_t r, const Row<T> &row,
                                              const Weights &weight, float u, const Cut &cut) {
    // a lane for each segment
    const int lane = threadIdx.x & 63;
    const uint64_t own = lane < kSlices ? sh.seg[lane] : 0;
    const uint64_t upto = wave_scan(own), sum = lane64(upto, 63);
    uint64_t target = above(u, sum);
    const int seg = __builtin_ctzll(__ballot(upto >= target));
    target -= lane64(upto - own, seg);
    const int end = min((seg + 1) * row.per, row.end);
#pragma unroll 1
    for (int c = seg * row.per; c < end; ++c) {
        const u32x4 x = row.load(c);
        const uint32_t i = row.index(c);
        constexpr int E = Row<T>::E;
        uint64_t w[E], mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float y = element<T>(x, e);
            w[e] = cut(y, i + e) ? weight(y) : 0;
            mine += w[e];
        }
        uint64_t all;
        uint64_t run = block_scan(sh, mine, &all);
        if (all >= target) {
            if (run < target && run + mine >= target) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (run < target && run + w[e] >= target)
                        write_drawn(out, r, i + e, element<T>(x, e), sum, weight);
                    run += w[e];
                }
            }
            return;
        }
        target -= all;
    }
    // A segment's sum is its bins', each rounded as one, and can be some units above
    // the sum of its elements': a target up there goes to the last element that
    // weighs a unit, or, where they do so only together, to the last of them.
    uint64_t behind = 0;
    row.each(
        [&](float y, uint32_t i) {
            double f;
            if (cut(y, i) && weight.split(y, &f) > -kNone) {
                const uint64_t key = (uint64_t(weight(y) != 0) << 32) | i;
                behind = key > behind ? key : behind;
            }
        },
        seg * row.per, end);
    behind = wave_max64(behind);
    __syncthreads();
    if (threadIdx.x == 0) sh.hi = 0;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) atomicMax(reinterpret_cast<ull *>(&sh.hi), ull(behind));
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t i = uint32_t(sh.hi);
        write_drawn(out, r, i, static_cast<float>(row.p[i]), sum, weight);
    }
}

// The rarely taken paths, in line like the rest.  They take copies: what they can
// change is no variable of the others.

// The element of the row, from `lo` on and below `hi` (+inf: no end) and kept by
// `cut`, at which the running weight (without `weigh`, their number) reaches `target`.
template <typename T>
__device__ __forceinline__ uint64_t border_in_row(Shared &sh, Row<T> row, bool weigh, Weights weight, float lo, float hi,
                                               Cut cut, uint64_t target) {
    return find_first(
        sh,
        [&](auto f) {
            row.each([&](float x, uint32_t i) {
                if (x >= lo && x < hi && cut(x, i)) f(order_key(x, i), weigh ? weight(x) : 1);
            });
        },
        target);
}

// Any cut at all, where its elements do not fit the list: every element's weight again.
template <typename T>
__device__ __forceinline__ void draw_by_cut(Shared &sh, Output out, int64_t r, Row<T> row, Weights weight, float u,
                                         Cut cut) {
    __syncthreads();
    if (threadIdx.x < kSlices) sh.seg[threadIdx.x] = 0;
    __syncthreads();
    for (int s = 0; s * row.per < row.end; ++s) {
        uint64_t sum = 0;
        row.each(
            [&](float y, uint32_t i) {
                if (cut(y, i)) sum += weight(y);
            },
            s * row.per, min((s + 1) * row.per, row.end));
        sum = wave_add(sum);
        if ((threadIdx.x & 63) == 0 && sum) add64(&sh.seg[s], sum);
    }
    __syncthreads();
    draw_from_row(sh, out, r, row, weight, u, cut);
}

// A row whose largest logit is +inf: the infinite ones weigh the same, the rest nothing.
template <typename T>
__device__ __forceinline__ void draw_infinite(Shared &sh, Output out, int64_t r, Row<T> row, Settings set) {
    uint64_t n = 0;
    row.each([&](float x, uint32_t) { n += x == INFINITY ? 1 : 0; });
    n = block_add(sh, n);
    if (set.top_k && n > uint64_t(set.top_k)) n = set.top_k;
    if (set.top_p < 1.0f) n = at_least(set.top_p, n);
    const uint64_t key = find_first(
        sh,
        [&](auto f) {
            row.each([&](float x, uint32_t i) {
                if (x == INFINITY) f(uint64_t(~i), uint64_t(1));
            });
        },
        above(set.u, n));
    if (threadIdx.x == 0) write_row(out, r, key_index(key), float(1.0 / double(n)));
}

// The smallest fp32 whose bin is at most b < kNone, by one wave, which tries
// 64 values at once: those around where the bin's edge lies in real numbers,
// and, where that fails (next to zero fp32 is finer than the 64-bit logits'
// rounding), a 64th of what is left at a time.
__device__ __forceinline__ float bin_edge(const Weights &weight, float top, int b) {
    const uint32_t lane = threadIdx.x & 63;
    double f;
    uint32_t lo = ordered(-__FLT_MAX__), hi = ordered(top);  // the bin of hi is at most b
    const uint32_t near = ordered(float(weight.top - (b + 0.5) / (kPerOctave * kOctaves) / weight.rate));
    if (near > lo + 64 && near < hi - 64) {
        const uint64_t in = __ballot(-weight.split(unordered(near - 32 + lane), &f) <= b);
        if (in != 0 && !(in & 1)) return unordered(near - 32 + uint32_t(__builtin_ctzll(in)));
    }
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 64 + 1;
        const bool inside = hi - lo >= (lane + 1) * step;
        const uint32_t x = inside ? hi - (lane + 1) * step : lo;
        const uint32_t n = __popcll(__ballot(inside && -weight.split(unordered(x), &f) <= b));  // the first n down from hi
        const uint32_t down = hi - n * step;
        lo = down - lo > step - 1 ? down - (step - 1) : lo;
        hi = down;
        if (step == 1) break;
    }
    return unordered(hi);
}

// The histograms of the weights of what `inside` keeps.
template <int SEGS, typename T, typename Inside>
__device__ __forceinline__ void mass_histogram(Shared &sh, const Row<T> &row, const Weights &weight, Inside inside) {
    for (int i = threadIdx.x; i < SEGS * kMass; i += kThreads) sh.bin[i] = 0;
    __syncthreads();
    // bin b of a segment is at [kMass - 1 - b]
    const int spread = int(threadIdx.x & 63) - (kMass - 1);
    uint64_t *bins = sh.bin + kMass - 1;
    int left = row.per;
    row.each_chunk(
        [&](u32x4 x, int c) {
            const uint32_t i = row.index(c);
#pragma unroll
            for (int h = 0; h < Row<T>::E / 4; ++h) {
                float y[4];
                int b[4];
                uint64_t unit[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = element<T>(x, h * 4 + e);
                weight.units(y, b, unit);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = inside(y[e], i + h * 4 + e) ? b[e] : spread;
                    add64(bins + max(at, spread), unit[e]);
                }
            }
            if (--left == 0) bins += kMass, left = row.per;
        });
    __syncthreads();
}

__device__ __forceinline__ Weights weights_of(Shared &sh, const SampleArgs &args, float top, float temperature) {
    return Weights{double(top), 1.4426950408889634 / kOctaves / double(temperature),
                   (lds_doubles)(sh.factor + kMass - 1),
                   __builtin_bit_cast(double, args.units.c4),
                   __builtin_bit_cast(double, args.units.c3),
                   __builtin_bit_cast(double, args.units.c2),
                   __builtin_bit_cast(double, args.units.c1),
                   __builtin_bit_cast(double, args.units.one),
                   args.per_unit};
}

// The factors' table; a barrier follows before its first use.
__device__ __forceinline__ void fill_factors(Shared &sh, int shift) {
    // a thread's bins are kThreads apart, whole octaves: one power for all of them
    const double part = exp2(double(threadIdx.x % kPerOctave) / -kPerOctave);
    for (int b = threadIdx.x; b < kMass; b += kThreads)
        sh.factor[kMass - 1 - b] = b < kNone ? __builtin_ldexp(part, shift - b / kPerOctave) : 0.0;
}

// Counts x, at least floor, in the bins of [floor, top].
__device__ __forceinline__ void count_logit(Shared &sh, float x, float top, float scale) {
    add64(&sh.bin[min(int(fminf((top - x) * scale, float(kSearch))), kSearch - 1)], 1);
}
__device__ __forceinline__ float count_scale(float top, float floor) {
    return fminf(float(kSearch - 1) / (top - floor), 1e30f);
}
// The lower edge of the bin where that count reaches k (-inf where it does not
// at all): at least k of what was counted reach it.  All threads; after a barrier.
__device__ __forceinline__ float count_edge(Shared &sh, int32_t k, float top, float floor, float scale) {
    uint64_t before, target, all = 0;
    const int last = find_bin(
        sh, own_bins(sh), [&](uint64_t sum) { all = sum; return uint64_t(k); }, &before, &target);
    if (all < uint64_t(k)) return -INFINITY;
    // the roundings of a bin are far below 2^-20 of its distance and 2^-22 of top
    return fmaxf(top - float(last + 1) / scale * 1.000001f - fabsf(top) * 2.4e-7f, floor);
}

// The bin that the border cuts, top-p's or min-p's where that comes first (kMass:
// none, or one without weight), from this thread's bins of the whole row's
// histogram (only looked at where top-p is on).
struct Border {
    int bin;
    bool by_p;                // top-p's border lies in it, at weight target - before within it
    uint64_t before, target;
};
__device__ __forceinline__ Border find_border(Shared &sh, const Weights &weight, const Settings &set, float least,
                                              Own own) {
    Border border{kMass, false, 0, 0};
    if (set.top_p < 1.0f) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
            const int bin = kOwn * threadIdx.x + i;
            own.v[i] = bin < kNone ? weight.whole(own.v[i], bin) : 0;
        }
        border.bin = find_bin(sh, own, [&](uint64_t all) { return at_least(set.top_p, all); }, &border.before,
                              &border.target);
        border.by_p = true;
    }
    if (least > -INFINITY) {
        double f;
        const int l = -weight.split(least, &f);
        if (l < border.bin) border.by_p = false, border.bin = l;
    }
    if (border.bin >= kNone) border.bin = kMass, border.by_p = false;
    return border;
}

// The edges of bin b in sh.edge: logits from [0] on and below [1].  A barrier follows.
__device__ __forceinline__ void find_edges(Shared &sh, const Weights &weight, float top, int b) {
    const int wave = threadIdx.x >> 6;
    if (wave < 2) {
        const float e = b - wave >= 0 ? bin_edge(weight, top, b - wave) : INFINITY;
        if ((threadIdx.x & 63) == 0) sh.edge[wave] = e;
    }
}

// Puts the border among sh.list[0, n), the elements of its bin (logits in [lo, hi]), into
// `cut`, and the weights of those it keeps onto their segments'.
template <typename T>
__device__ __forceinline__ void settle_list(Shared &sh, const Row<T> &row, const Weights &weight, uint32_t n,
                                            const Border &border, float lo, float hi, float least, Cut &cut) {
    const Share p = share_of_list(sh, n, weight);
    if (border.by_p) {
        const uint64_t key = find_key(sh, p, n, uint64_t(ordered(lo)) << 32, (uint64_t(ordered(hi)) << 32) | 0xffffffffu,
                                      border.target - border.before);
        if (key) cut.from_key(key);  // else the bin's weights all round to 0: what it holds cannot be drawn
    }
    cut.from_value(least);
#pragma unroll
    for (int e = 0; e < kOwn; ++e)
        if (p.weight[e] && cut(key_value(p.key[e]), key_index(p.key[e])))
            add64(&sh.seg[row.segment(key_index(p.key[e]))], p.weight[e]);
}

// One row by one workgroup.
template <typename T>
__device__ __forceinline__ void sample_row(Shared &sh, const SampleArgs &args, int64_t r) {
    const int t = threadIdx.x;
    const Row<T> row(args, r);
    const Settings set(args, r);
    const Output out{args.out_token, args.out_prob};

    // the largest logit, and the smallest finite one
    // of the threads' largest, each over every fourth of its chunks
    Largest<T> largest[4];
    row.each_of_many(
        [&](u32x4 x, int c) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if ((c & 3) == g) largest[g].add(x);
        },
        0, row.end);
    float own[4];
    bool again = false;
#pragma unroll
    for (int g = 0; g < 4; ++g) own[g] = largest[g].value(), again |= largest[g].nan();
    if (again) {
        own[0] = row.largest();
        own[1] = own[2] = own[3] = -INFINITY;
    }
    const float mine = fmaxf(fmaxf(own[0], own[1]), fmaxf(own[2], own[3]));
    float top = mine, floor = INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) floor = fminf(floor, own[g] > -INFINITY ? own[g] : INFINITY);
    top = wave_max(top);
    floor = wave_min(floor);
    if ((t & 63) == 0) sh.f[t >> 6] = top, sh.g[t >> 6] = floor;
    if (t == 0) sh.found = 0xffffffffu;
    for (int i = t; i < kSearch; i += kThreads) sh.bin[i] = 0;
    __syncthreads();
    top = wave_max(sh.f[t & (kWaves - 1)]);
    floor = wave_min(sh.g[t & (kWaves - 1)]);
    if (top == -INFINITY) {  // nothing to draw from
        if (t == 0) write_row(out, r, 0xffffffffu, 0.0f);
        return;
    }
    if (set.single) {  // the lowest index that holds it
        if (__any(mine == top)) {
            uint32_t first = 0xffffffffu;
            row.each([&](float x, uint32_t i) {
                if (x >= top && i < first) first = i;
            });
            if (first != 0xffffffffu) atomicMin(&sh.found, first);
        }
        __syncthreads();
        if (t == 0) write_row(out, r, sh.found, 1.0f);
        return;
    }
    if (top == INFINITY) return draw_infinite(sh, out, r, row, set);

    const Weights weight = weights_of(sh, args, top, set.temperature);
    const float least = set.least(top);
    // rows that fit the list, and top-k's elements where a list of few more holds them
    float from = row.v <= kList ? -__FLT_MAX__ : -INFINITY;
    if (row.v > kList && set.top_k && set.top_k <= kMostK && floor < top) {
        // A value that at least k elements reach, and few more: the lower edge of the
        // bin where the count of those 4 kThreads largest logits reaches k (of so many,
        // one seldom hides another of the first k).
        const float scale = count_scale(top, floor);
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (own[g] > -INFINITY) count_logit(sh, own[g], top, scale);
        __syncthreads();
        from = count_edge(sh, set.top_k, top, floor, scale);
    }
    if (from > -INFINITY) {
        // a wave takes about as long for one thread's place as for 64 threads' chunk
        const bool few = row.v > kList && set.top_k <= 128;
        const uint32_t n = few ? row.collect_from(sh, from, mine) : row.collect(sh, from, top);
        if (n <= kList)
            return draw_from_list(sh, out, r, n, weight, set, least, row.v > kList ? from : -INFINITY, uint32_t(row.v),
                                  [&](uint32_t i) { return static_cast<float>(row.p[i]); });
    }
    // Top-k without that list: above kMostK, with fewer live groups than k, or where a
    // mask's low finite value widens the bins until the list overflows.  The border
    // costs two reads of the row for each 11 bits of key, and top-p's below as many.  Measured
    // (us, top-p 0.9; top-k 50 with nothing masked | 99.9 % at -inf | half at the lowest
    // finite value | top-k 2000):
    //   1 x 32000 fp32      10.6 | 38 | 130 | 70
    //   1 x 131072 bf16     12   | 12 | 12  | 211
    //   64 x 50001 fp16     14   | 62 | 209 | 127
    //   256 x 131072 bf16   20   | 19 | 19  | 278
    Cut cut;
    if (set.top_k) {
        cut.from_key(border_in_row<T>(sh, row, false, weight, -__FLT_MAX__, INFINITY, cut, uint64_t(set.top_k)));
        __syncthreads();
    }

    const bool cut_k = set.top_k != 0;
    if (cut_k)
        mass_histogram<kSegs>(sh, row, weight, cut);
    else
        mass_histogram<kSegs>(sh, row, weight, [](float, uint32_t) { return true; });
    Own mass = {};
    if (set.top_p < 1.0f && kOwn * t < kNone) {
#pragma unroll
        for (int s = 0; s < kSegs; ++s)
#pragma unroll
            for (int i = 0; i < kOwn; ++i) mass.v[i] += sh.bin[s * kMass + kMass - 1 - kOwn * t - i];
    }
    const Border border = find_border(sh, weight, set, least, mass);
    const int b = border.bin;
    // about how many elements bin b holds, and the weights kept whole, by segment
    uint64_t in_bin = 0;
    if (b < kMass) {
#pragma unroll
        for (int s = 0; s < kSegs; ++s) in_bin += sh.bin[s * kMass + kMass - 1 - b];
        in_bin >>= args.shift;
    }
    if (t < kSlices) sh.seg[t] = 0;
    __syncthreads();
    {
        // 128 threads a segment, a bin in 128 each, summed in 64-bit floating point in a fixed order
        constexpr int kEach = kThreads / kSegs;
        const int s = t / kEach;
        double sum = 0.0;
        for (int i = t % kEach; i < min(b, kNone); i += kEach)
            sum = fma(double(sh.bin[s * kMass + kMass - 1 - i]), weight.zero[-i] * weight.per_unit, sum);
        const uint64_t all = wave_add(uint64_t(__builtin_rint(sum)));
        if ((t & 63) == 0) add64(&sh.seg[s], all);
    }
    if (b < kMass) {
        find_edges(sh, weight, top, b);
        __syncthreads();
        const float lo = sh.edge[0], hi = sh.edge[1];
        // A bin of more than the list holds its border by reading the row, as above: 16-bit
        // logits far from 0 are that coarse (bf16 from 16 on: steps of four bins).  256 x
        // 131072 bf16, top-p 0.95, normal with deviation 2 around 0 | 24 | 100: 51 | 218 |
        // 231 us; top-p 0.5, whose bins are less full: 51 | 54 | 67.
        const uint32_t n = cut_k || in_bin > 2 * kList ? kList + 1 : row.collect(sh, lo, fminf(next_below(hi), top));
        if (n > kList) {
            if (border.by_p)
                cut.from_key(border_in_row<T>(sh, row, true, weight, lo, hi, cut, border.target - border.before));
            cut.from_value(least);
            return draw_by_cut(sh, out, r, row, weight, set.u, cut);
        }
        settle_list(sh, row, weight, n, border, lo, fminf(hi, top), least, cut);
    }
    __syncthreads();
    draw_from_row(sh, out, r, row, weight, set.u, cut);
}

// (at most 128 registers: 16 waves a CU in either form)
template <typename T>
__global__ __launch_bounds__(kThreads, 4) void row_kernel(SampleArgs args, int64_t first) {
    extern __shared__ __align__(16) char memory[];
    Shared &sh = *reinterpret_cast<Shared *>(memory);
    fill_factors(sh, args.shift);
    sample_row<T>(sh, args, first + blockIdx.x);  // its first barrier is ahead of the factors' first use
}

template <typename T>
hipError_t launch_rows(const SampleArgs &a, hipStream_t s) {
    static std::atomic<uint64_t> told{0};
    hipError_t err = allow_lds(reinterpret_cast<const void *>(row_kernel<T>), int(sizeof(Shared)), told);
    // a workgroup per row: a loop over rows in the kernel would keep what the
    // passes have in common in registers across all of them
    constexpr int64_t kMost = 1 << 20;
    for (int64_t first = 0; first < a.r && err == hipSuccess; first += kMost) {
        const int64_t rows = a.r - first < kMost ? a.r - first : kMost;
        row_kernel<T><<<unsigned(rows), kThreads, sizeof(Shared), s>>>(a, first);
        err = hipGetLastError();
    }
    return err;
}

}  // namespace
}  // namespace rt
