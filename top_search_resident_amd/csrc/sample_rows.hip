// sample_rows.hip -- one token per row of logits: temperature, top-k, top-p,
// min-p and a draw with a given random number (rt_sample_rows).
//
// Mathematics.  Order the tokens by (logit down, index up).  Every filter keeps
// a prefix of that order, so a row is settled by one border element: the k-th,
// or the first at which the running weight reaches top_p of the whole, or the
// min-p logit.  The draw is the same question in index order: the first kept
// element at which the running weight reaches floor(u S) + 1.  All three are
// answered by find_first(): histogram the elements over 2048 bins of a
// monotone key, find the bin in which the running sum crosses the target,
// narrow to it and repeat until one element is left.  No sort.
//
// Weights are whole multiples of 2^-shift of the largest (shift <= 46), from a
// 64-bit exponential, and all sums are 64-bit integers: histogram atomics in
// any order give the same sums, so the same inputs give the same token, and a
// border decided in plain 64-bit floating point falls on the same side except
// within about 2^-45 of the whole.
//
// One workgroup of 1024 threads per row.  It keeps the first kKeep 16-byte chunks of every
// thread in registers (the whole row up to 8192 kKeep bytes... see launch) and
// reads the rest again in each pass.
#include <hip/hip_runtime.h>

#include "../../include/resident_topk.h"
#include "float_types.hpp"
#include "limits.hpp"

namespace rt {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;  // two per thread
constexpr int kList = 2048;  // candidates kept in LDS
constexpr int kSegs = 1024;  // index segments of the draw over a row

struct SampleArgs {
    const void *logits;
    int64_t r, v, ld;
    const float *u;
    rt_sample_settings set;
    int32_t *out_token;
    float *out_prob;
    int shift;  // weights are multiples of 2^-shift of the largest
};

// Order of the elements as one 64-bit number, larger first: the logit's bits
// made monotone, then the index from the top down.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t idx) {
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0.0 becomes +0.0
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return (uint64_t(o) << 32) | uint32_t(~idx);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = uint32_t(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// exp((x - top) / T) as a whole multiple of 2^-shift: 2^t with t = (x - top)
// log2(e) / T, a polynomial of degree 9 for the fraction (relative error
// 2^-46, coefficients fitted for the smallest largest relative error on
// [-1/2, 1/2]) and the exponent added on; adding 2^52 rounds to a whole number.
struct Weights {
    float top;
    double rate;  // log2(e) / T
    int shift;

    __device__ __forceinline__ double power(float x) const {
        const double t = fmax((double(x) - double(top)) * rate, -200.0);  // NaN and -inf give -200
        const double n = __builtin_rint(t), f = t - n;
        double p = 1.0150336908049256e-07;
        p = fma(p, f, 1.3259405616920547e-06);
        p = fma(p, f, 1.5252984837515096e-05);
        p = fma(p, f, 0.00015403434948043135);
        p = fma(p, f, 0.0013333557617606637);
        p = fma(p, f, 0.009618129192067264);
        p = fma(p, f, 0.055504108668685596);
        p = fma(p, f, 0.24022650695649653);
        p = fma(p, f, 0.693147180559871);
        p = fma(p, f, 1.0000000000000127);
        return __builtin_ldexp(p, int(n) + shift);
    }
    __device__ __forceinline__ uint64_t operator()(float x) const {
        const double y = power(x) + 4503599627370496.0;
        const uint64_t w = __builtin_bit_cast(uint64_t, y) & 0x000fffffffffffffull;
        return x >= top ? (uint64_t(1) << shift) : w;
    }
};

struct Shared {
    uint64_t bin[kBins];
    uint64_t list[kList];
    uint64_t wave_sum[kWaves];
    uint64_t lo, hi, before, total;
    uint32_t count, found;
    float f[kWaves];
    float g[kWaves];
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) {
    const uint32_t lo = __shfl_up(int(uint32_t(v)), d), hi = __shfl_up(int(uint32_t(v >> 32)), d);
    return (uint64_t(hi) << 32) | lo;
}
__device__ __forceinline__ uint64_t shfl_xor64(uint64_t v, int d) {
    const uint32_t lo = __shfl_xor(int(uint32_t(v)), d), hi = __shfl_xor(int(uint32_t(v >> 32)), d);
    return (uint64_t(hi) << 32) | lo;
}
__device__ __forceinline__ uint64_t wave_add(uint64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += shfl_xor64(v, o);
    return v;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {  // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint64_t up = shfl_up64(v, o);
        if (lane >= o) v += up;
    }
    return v;
}

__device__ __forceinline__ void clear_bins(Shared &sh) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh.bin[i] = 0;
    __syncthreads();
}

// The first bin at which the running sum reaches `target` (at least 1; a target
// above the sum of all takes the last bin with anything): bin, sum before it.  All
// threads call it after a barrier on the bins; ends with a barrier.
__device__ __forceinline__ int find_bin(Shared &sh, uint64_t target, uint64_t *before, uint64_t *total) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const uint64_t b0 = sh.bin[2 * t], b1 = sh.bin[2 * t + 1];
    const uint64_t own = b0 + b1;
    const uint64_t scan = wave_scan(own);
    if (lane == 63) sh.wave_sum[wave] = scan;
    __syncthreads();
    uint64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint64_t s = sh.wave_sum[w];
        if (w < wave) base += s;
        all += s;
    }
    if (target > all) target = all;
    const uint64_t pre = base + scan - own;
    if (pre < target && pre + own >= target) {  // exactly one thread, where all > 0
        const bool second = pre + b0 < target;
        sh.found = 2 * t + (second ? 1 : 0);
        sh.before = second ? pre + b0 : pre;
    }
    __syncthreads();
    *before = sh.before;
    *total = all;
    return int(sh.found);
}

__device__ __forceinline__ uint64_t block_add(Shared &sh, uint64_t v) {
    v = wave_add(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh.wave_sum[threadIdx.x >> 6] = v;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) all += sh.wave_sum[w];
    return all;
}

// The element, among those each(f) presents as f(key, weight) with lo <= key <=
// hi, at which the weight summed from the largest key down first reaches
// `target`.  Each round narrows [lo, hi] to one of 2048 bins of what is left.
template <typename Each>
__device__ __forceinline__ uint64_t find_first(Shared &sh, Each each, uint64_t target, uint64_t lo, uint64_t hi) {
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
        clear_bins(sh);
        if ((threadIdx.x & 63) == 0) {
            atomicMin(reinterpret_cast<unsigned long long *>(&sh.lo), (unsigned long long)least);
            atomicMax(reinterpret_cast<unsigned long long *>(&sh.hi), (unsigned long long)most);
        }
        __syncthreads();
        least = sh.lo;
        most = sh.hi;
        if (least >= most) return most;  // one element (or, of an empty range, 0)
        const int bits = 64 - __builtin_clzll(most - least);
        const int drop = bits > 11 ? bits - 11 : 0;
        each([&](uint64_t key, uint64_t w) {
            if (key >= least && key <= most)
                atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[(most - key) >> drop]), (unsigned long long)w);
        });
        __syncthreads();
        uint64_t before, total;
        const uint64_t b = find_bin(sh, target, &before, &total);
        if (total == 0) return most;
        target = (target > total ? total : target) - before;
        hi = most - (b << drop);
        const uint64_t width = (uint64_t(1) << drop) - 1;
        lo = hi - least > width ? hi - width : least;
    }
}

// A row: the first KEEP chunks of 16 bytes of each thread in registers, the
// rest read again on each pass.  Chunk c of thread t holds elements
// (c * 1024 + t) * E ..; elements past the row's end read as -inf.
template <typename T, int KEEP>
struct Row {
    static constexpr int E = 16 / sizeof(T);
    static constexpr int64_t kChunk = int64_t(kThreads) * E;
    const T *p;
    int64_t v;
    u32x4 keep[KEEP];

    __device__ __forceinline__ u32x4 load(int64_t c) const {
        const int64_t i = c * kChunk + int64_t(threadIdx.x) * E;
        if (i + E <= v) return load16(p + i);
        constexpr uint32_t none = sizeof(T) == 4 ? 0xff800000u : (__is_same(T, bf16_t) ? 0xff80ff80u : 0xfc00fc00u);
        u32x4 x = {none, none, none, none};
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (i + e < v) {
                if constexpr (sizeof(T) == 4) {
                    x[e] = __float_as_uint(p[i + e]);
                } else {
                    const uint32_t h = __builtin_bit_cast(uint16_t, p[i + e]);
                    x[e >> 1] = (e & 1) ? (x[e >> 1] & 0xffffu) | (h << 16) : (x[e >> 1] & 0xffff0000u) | h;
                }
            }
        return x;
    }
    __device__ __forceinline__ int64_t chunks() const { return (v + kChunk - 1) / kChunk; }
    __device__ __forceinline__ void fill() {
        const int64_t n = chunks();
#pragma unroll
        for (int c = 0; c < KEEP; ++c)
            if (c < n) keep[c] = load(c);
    }
    // f(16 bytes, chunk)
    template <typename F>
    __device__ __forceinline__ void each_chunk(F f) const {
        const int64_t n = chunks();
#pragma unroll
        for (int c = 0; c < KEEP; ++c)
            if (c < n) f(keep[c], int64_t(c));
        for (int64_t c = KEEP; c < n; ++c) f(load(c), c);
    }
    // f(value, index) of each element of a chunk; the loop is kept rolled over
    // the words so that a pass over KEEP register chunks stays small
    template <typename F>
    __device__ __forceinline__ void each_in(u32x4 x, int64_t c, F f) const {
        uint32_t i = uint32_t(c * kChunk + int64_t(threadIdx.x) * E);
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int e = 0; e < E / 4; ++e) f(element<T>(x, e), i + e);
            i += E / 4;
            x = u32x4{x[1], x[2], x[3], x[0]};
        }
    }
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
        each_chunk([&](u32x4 x, int64_t c) { each_in(x, c, f); });
    }
};

// Running sum reaches `part` of `whole` (a fraction in fp32): the least whole
// number of units at or above it.
__device__ __forceinline__ uint64_t at_least(float part, uint64_t whole) {
    const double t = __builtin_ceil(double(part) * double(whole));
    const uint64_t n = uint64_t(t);
    return n < 1 ? 1 : (n > whole ? whole : n);
}

// Running sum exceeds u of `whole`.
__device__ __forceinline__ uint64_t above(float u, uint64_t whole) {
    if (!(u > 0.0f)) return 1;
    if (u >= 1.0f) return whole;
    const uint64_t n = uint64_t(double(u) * double(whole)) + 1;
    return n > whole ? whole : n;
}

template <typename T, int KEEP>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleArgs args) {
    __shared__ Shared sh;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int64_t r = blockIdx.x; r < args.r; r += gridDim.x) {
        __syncthreads();
        Row<T, KEEP> row;
        row.p = static_cast<const T *>(args.logits) + r * args.ld;
        row.v = args.v;
        row.fill();
        const rt_sample_settings &set = args.set;
        const float temperature = set.temperatures ? set.temperatures[r] : set.temperature;
        const int32_t top_k = set.top_ks ? set.top_ks[r] : set.top_k;
        const float top_p = set.top_ps ? set.top_ps[r] : set.top_p;
        const float min_p = set.min_ps ? set.min_ps[r] : set.min_p;
        const float u = args.u[r];

        // the largest logit, and the smallest of the threads' largest
        float own = -INFINITY;
        row.each([&](float x, uint32_t) { own = fmaxf(own, x); });
        float top = own, floor_ = own;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            top = fmaxf(top, __shfl_xor(top, o));
            floor_ = fminf(floor_, __shfl_xor(floor_, o));
        }
        if (lane == 0) sh.f[wave] = top, sh.g[wave] = floor_;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            top = fmaxf(top, sh.f[w]);
            floor_ = fminf(floor_, sh.g[w]);
        }
        if (top == -INFINITY) {  // nothing to draw from
            if (t == 0) {
                args.out_token[r] = -1;
                if (args.out_prob) args.out_prob[r] = 0.0f;
            }
            continue;
        }
        // settings that keep only the first token of the order
        if (!(temperature > 0.0f) || top_k == 1 || !(top_p > 0.0f) || !(min_p <= 1.0f)) {
            uint32_t first = 0xffffffffu;
            row.each([&](float x, uint32_t i) {
                if (x >= top && i < first) first = i;
            });
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) first = min(first, uint32_t(__shfl_xor(int(first), o)));
            if (t == 0) sh.found = 0xffffffffu;
            __syncthreads();
            if (lane == 0) atomicMin(&sh.found, first);
            __syncthreads();
            if (t == 0) {
                args.out_token[r] = int32_t(sh.found);
                if (args.out_prob) args.out_prob[r] = 1.0f;
            }
            continue;
        }
        const Weights weight{top, 1.4426950408889634 / double(temperature), args.shift};
        // min-p as a logit: the smallest fp32 at or above top + T ln(min_p)
        float least = -INFINITY;
        if (min_p > 0.0f) {
            const double cut = double(top) + double(temperature) * log(double(min_p));
            least = __double2float_ru(cut);
            if (!(least <= top)) least = top;
        }

        uint64_t border = 0;  // kept: keys at or above it (and logits at or above `least`)
        bool listed = false;  // every kept element is in sh.list
        uint32_t n_list = 0;
        const bool k_on = top_k > 0 && top_k < args.v, p_on = top_p < 1.0f;

        auto row_keys = [&](auto f) {
            row.each([&](float x, uint32_t i) {
                if (x >= -INFINITY && i < args.v) f(order_key(x, i), uint64_t(1));
            });
        };
        if (k_on) {
            // Bins over [low, top]; everything below goes to the last bin.  At
            // least 1024 elements reach the smallest of the threads' largest.
            float low = (top_k <= kThreads && floor_ > -INFINITY) ? floor_ : top - 22.0f * temperature;
            const float scale = fminf(float(kBins - 2) / (top - low), 1e30f);
            auto bin_of = [&](float x) {
                if (x >= top) return 0;
                return x >= low ? min(int(fminf((top - x) * scale, float(kBins))), kBins - 2) : kBins - 1;
            };
            clear_bins(sh);
            uint32_t below = 0;
            row.each([&](float x, uint32_t i) {
                if (x >= low)
                    atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[bin_of(x)]), 1ull);
                else
                    below += i < args.v ? 1 : 0;  // NaN and -inf, too: the last of the order
            });
            const uint64_t under = wave_add(below);
            if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[kBins - 1]), (unsigned long long)under);
            if (t == 0) sh.count = 0;
            __syncthreads();
            uint64_t before, total;
            const int b = find_bin(sh, uint64_t(top_k), &before, &total);
            const uint64_t upto = before + sh.bin[b];
            if (b == kBins - 1) {
                border = find_first(sh, row_keys, uint64_t(top_k), 0, ~uint64_t(0));
            } else if (upto <= kList) {
                row.each([&](float x, uint32_t i) {
                    if (x >= low && bin_of(x) <= b) {
                        const uint32_t at = atomicAdd(&sh.count, 1u);
                        if (at < kList) sh.list[at] = order_key(x, i);  // always: `upto` of them
                    }
                });
                __syncthreads();
                listed = true;
                n_list = uint32_t(upto);
                border = find_first(
                    sh,
                    [&](auto f) {
                        for (uint32_t j = t; j < n_list; j += kThreads) f(sh.list[j], uint64_t(1));
                    },
                    uint64_t(top_k), 0, ~uint64_t(0));
            } else {
                border = find_first(
                    sh,
                    [&](auto f) {
                        row.each([&](float x, uint32_t i) {
                            if (x >= low && bin_of(x) == b) f(order_key(x, i), uint64_t(1));
                        });
                    },
                    uint64_t(top_k) - before, 0, ~uint64_t(0));
            }
        }
        auto list_weights = [&](auto f) {
            for (uint32_t j = t; j < n_list; j += kThreads) {
                const uint64_t key = sh.list[j];
                if (key >= border) f(key, weight(key_value(key)));
            }
        };
        if (p_on && listed) {
            uint64_t z = 0;
            list_weights([&](uint64_t, uint64_t w) { z += w; });
            z = block_add(sh, z);
            border = find_first(sh, list_weights, at_least(top_p, z), 0, ~uint64_t(0));
        } else if (p_on) {
            // 64 bins an octave of weight, 32 octaves; lighter ones in the last bin
            const float scale = float(fmin(64.0 * weight.rate, 1e30));
            auto bin_of = [&](float x) {
                return x >= top ? 0 : int(fminf((top - x) * scale, float(kBins - 1)));
            };
            const float border_value = border ? key_value(border) : -INFINITY;
            auto inside = [&](float x, uint32_t i) {
                return x > border_value || (x == border_value && order_key(x, i) >= border && x > -INFINITY);
            };
            clear_bins(sh);
            uint64_t light = 0;
            row.each([&](float x, uint32_t i) {
                if (inside(x, i)) {
                    const int b = bin_of(x);
                    const uint64_t w = weight(x);
                    if (b < kBins - 1)
                        atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[b]), (unsigned long long)w);
                    else
                        light += w;
                }
            });
            light = wave_add(light);
            if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[kBins - 1]), (unsigned long long)light);
            if (t == 0) sh.count = 0, sh.total = 0;
            __syncthreads();
            uint64_t before, z;
            (void)find_bin(sh, 1, &before, &z);
            const uint64_t target = at_least(top_p, z);
            const int b = find_bin(sh, target, &before, &z);
            row.each([&](float x, uint32_t i) {
                if (inside(x, i) && bin_of(x) == b) {
                    const uint32_t at = atomicAdd(&sh.count, 1u);
                    if (at < kList) sh.list[at] = order_key(x, i);
                }
            });
            __syncthreads();
            const uint32_t n = sh.count;
            if (n <= kList)
                border = find_first(
                    sh,
                    [&](auto f) {
                        for (uint32_t j = t; j < n; j += kThreads) f(sh.list[j], weight(key_value(sh.list[j])));
                    },
                    target - before, 0, ~uint64_t(0));
            else
                border = find_first(
                    sh,
                    [&](auto f) {
                        row.each([&](float x, uint32_t i) {
                            if (inside(x, i) && bin_of(x) == b) f(order_key(x, i), weight(x));
                        });
                    },
                    target - before, 0, ~uint64_t(0));
        }

        // the draw
        uint32_t token;
        float value;
        uint64_t sum;
        if (listed) {
            auto by_index = [&](auto f) {
                for (uint32_t j = t; j < n_list; j += kThreads) {
                    const uint64_t key = sh.list[j];
                    const float x = key_value(key);
                    if (key >= border && x >= least) f(uint64_t(uint32_t(key)), weight(x));
                }
            };
            uint64_t s = 0;
            by_index([&](uint64_t, uint64_t w) { s += w; });
            sum = block_add(sh, s);
            token = ~uint32_t(find_first(sh, by_index, above(u, sum), 0, ~uint64_t(0)));
        } else {
            const float border_value = border ? key_value(border) : -INFINITY;
            auto kept = [&](float x, uint32_t i) {
                return x >= least && (x > border_value || (x == border_value && order_key(x, i) >= border)) &&
                       x > -INFINITY;
            };
            const int64_t chunks = row.chunks(), per = (chunks + kSegs - 1) / kSegs;
            clear_bins(sh);
            uint64_t s = 0;
            row.each_chunk([&](u32x4 x, int64_t c) {
                row.each_in(x, c, [&](float y, uint32_t i) {
                    if (kept(y, i)) s += weight(y);
                });
                if ((c + 1) % per == 0 || c + 1 == chunks) {
                    const uint64_t all = wave_add(s);
                    if (lane == 0 && all)
                        atomicAdd(reinterpret_cast<unsigned long long *>(&sh.bin[c / per]), (unsigned long long)all);
                    s = 0;
                }
            });
            __syncthreads();
            uint64_t before;
            (void)find_bin(sh, 1, &before, &sum);
            uint64_t target = above(u, sum);
            const int64_t seg = find_bin(sh, target, &before, &sum);
            target -= before;
            token = 0;
            const int64_t last = min((seg + 1) * per, chunks);
            for (int64_t c = seg * per; c < last; ++c) {
                // this chunk again: a bin per 64 / 128 ... threads' own elements
                const u32x4 x = row.load(c);
                uint64_t mine = 0;
                row.each_in(x, c, [&](float y, uint32_t i) {
                    if (kept(y, i)) mine += weight(y);
                });
                const uint64_t scan = wave_scan(mine);
                __syncthreads();
                if (lane == 63) sh.wave_sum[wave] = scan;
                __syncthreads();
                uint64_t base = 0, all = 0;
                for (int w = 0; w < kWaves; ++w) {
                    if (w < wave) base += sh.wave_sum[w];
                    all += sh.wave_sum[w];
                }
                if (all >= target) {
                    uint64_t run = base + scan - mine;
                    if (run < target && run + mine >= target)
                        row.each_in(x, c, [&](float y, uint32_t i) {
                            if (kept(y, i)) {
                                const uint64_t w = weight(y);
                                if (run < target && run + w >= target) sh.found = i;
                                run += w;
                            }
                        });
                    __syncthreads();
                    token = sh.found;
                    break;
                }
                target -= all;
            }
        }
        if (t == 0) {
            token = min(token, uint32_t(args.v - 1));
            args.out_token[r] = int32_t(token);
            if (args.out_prob) {
                value = static_cast<float>(static_cast<const T *>(args.logits)[r * args.ld + token]);
                const double w = value >= top ? __builtin_ldexp(1.0, args.shift) : weight.power(value);
                args.out_prob[r] = float(w / double(sum));
            }
        }
    }
}

template <typename T>
hipError_t launch(const SampleArgs &a, hipStream_t s) {
    const unsigned grid = unsigned(a.r < (1 << 20) ? a.r : (1 << 20));
    sample_kernel<T, 2><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace rt

extern "C" rt_status rt_sample_rows(const void *logits, int32_t dtype, int64_t r, int64_t v, int64_t ld,
                                    const float *u, const rt_sample_settings *settings, int32_t *out_token,
                                    float *out_prob, void *workspace, int64_t workspace_bytes, void *stream) {
    rt_status st = rt_check_sample_rows(logits, dtype, r, v, ld, u, settings, out_token, out_prob, workspace,
                                        workspace_bytes);
    if (st != RT_OK || r == 0) return st;
    int log2v = 0;
    while ((int64_t(1) << log2v) < v) ++log2v;
    const int shift = 62 - log2v < 46 ? 62 - log2v : 46;
    const rt::SampleArgs a{logits, r, v, ld, u, *settings, out_token, out_prob, shift};
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err;
    switch (dtype) {
        case RT_DTYPE_FLOAT32: err = rt::launch<float>(a, s); break;
        case RT_DTYPE_BFLOAT16: err = rt::launch<rt::bf16_t>(a, s); break;
        default: err = rt::launch<rt::fp16_t>(a, s);
    }
    if (err != hipSuccess) {
        (void)hipGetLastError();
        return RT_EHIP;
    }
    return RT_OK;
}
