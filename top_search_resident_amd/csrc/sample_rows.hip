// sample_rows.hip -- rt_sample_rows: a workgroup of 1024 threads a row
// (sample_rows.hpp), or, for a few long rows, several of them.
#define RT_SAMPLE_THREADS 1024
#include "sample_rows.hpp"

namespace rt {
namespace {

// ------------------------------------------------------- few rows, long ones

// A few long rows leave most CUs idle with one workgroup a row: there, `slices`
// workgroups share a row, in four kernels over a workspace (each starts where
// the last has ended: nothing waits inside a kernel):
//   1. each slice's largest logit, and its threads' largest;
//   2. top-k: the value that k of all threads' largest reach, and the slice's
//      elements from it on; else the slice's histogram;
//   3. (not for top-k) the whole row's histogram, the border's bin, the slice's
//      elements of it and its weight before it;
//   4. one workgroup a row: the slices' lists as one, the border, the draw.
struct Slice {
    float top, floor;
    uint32_t first;    // the lowest index that holds `top`
    uint32_t count;    // of list; above kList: the row goes the one-workgroup way
    uint64_t kept;     // weight before the border's bin
    float lo, hi;      // edges of that bin (in the first slice)
    Border border;     // (in the first slice)
    float own[kThreads];       // each thread's largest logit
    alignas(16) uint64_t mass[kMass + kOwn];  // the histogram, bin 0 first
    uint64_t list[kList];
};

template <typename T>
struct SliceOf {
    Row<T> row;
    Slice *all, *own;  // the row's slices, this one
    int slices;
    float top, floor;

    __device__ __forceinline__ SliceOf(const SampleArgs &a, Slice *work, int64_t r, int s, int n, int per)
        : row(a, r), all(work + r * n), own(work + r * n + s), slices(n) {
        row.per = per;
        row.begin = s * per;
        row.end = min(row.begin + per, row.end);
    }
    // use(load(slice)) for each of the row's slices, `none` for a missing one: the
    // loads of eight at a time, since one after the other costs a round trip each.
    template <typename Load, typename V, typename Use>
    __device__ __forceinline__ void each_slice(Load load, V none, Use use) const {
        for (int s = 0; s < slices; s += 8) {
            V v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = s + i < slices ? load(all[min(s + i, slices - 1)]) : none;
#pragma unroll
            for (int i = 0; i < 8; ++i) use(v[i]);
        }
    }
    // The row's largest logit and the smallest of its threads' largest (32 slices at most).
    __device__ __forceinline__ void extremes() {
        const int lane = threadIdx.x & 63;
        top = wave_max(lane < slices ? all[lane].top : -INFINITY);
        floor = wave_min(lane < slices ? all[lane].floor : INFINITY);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void split_top_kernel(SampleArgs args, Slice *work, int slices, int per) {
    extern __shared__ __align__(16) char memory[];
    Shared &sh = *reinterpret_cast<Shared *>(memory);
    const int t = threadIdx.x;
    SliceOf<T> slice(args, work, blockIdx.y, blockIdx.x, slices, per);
    const Settings set(args, blockIdx.y);
    Largest<T> largest;
    slice.row.each_of_many([&](u32x4 x, int) { largest.add(x); }, slice.row.begin, slice.row.end);
    float own = largest.value();
    if (largest.nan()) own = slice.row.largest();
    slice.own->own[t] = own;
    float top = wave_max(own), floor = wave_min(own > -INFINITY ? own : INFINITY);
    if ((t & 63) == 0) sh.f[t >> 6] = top, sh.g[t >> 6] = floor;
    if (t == 0) sh.found = 0xffffffffu;
    __syncthreads();
    top = wave_max(sh.f[t & (kWaves - 1)]);
    floor = wave_min(sh.g[t & (kWaves - 1)]);
    if (set.single && top > -INFINITY) {
        if (own == top) {
            uint32_t first = 0xffffffffu;
            slice.row.each([&](float x, uint32_t i) {
                if (x >= top && i < first) first = i;
            });
            atomicMin(&sh.found, first);
        }
        __syncthreads();
    }
    if (t == 0) {
        slice.own->top = top;
        slice.own->floor = floor;
        slice.own->first = sh.found;
        slice.own->count = 0;
        slice.own->kept = 0;
    }
}

// sh.list[0, n) to the slice's own.
__device__ __forceinline__ void write_list(Shared &sh, Slice *own, uint32_t n) {
    for (uint32_t j = threadIdx.x; j < min(n, uint32_t(kList)); j += kThreads) own->list[j] = sh.list[j];
    if (threadIdx.x == 0) own->count = n;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void split_candidates_kernel(SampleArgs args, Slice *work, int slices, int per) {
    extern __shared__ __align__(16) char memory[];
    Shared &sh = *reinterpret_cast<Shared *>(memory);
    const int t = threadIdx.x;
    SliceOf<T> slice(args, work, blockIdx.y, blockIdx.x, slices, per);
    const Settings set(args, blockIdx.y);
    slice.extremes();
    const float top = slice.top, floor = slice.floor;
    if (set.single || !(fabsf(top) < INFINITY)) return;
    if (set.top_k) {
        float from = -INFINITY;
        if (set.top_k <= kMostK && floor < top) {
            for (int i = t; i < kSearch; i += kThreads) sh.bin[i] = 0;
            __syncthreads();
            const float scale = count_scale(top, floor);
            slice.each_slice([&](const Slice &one) { return one.own[t]; }, -INFINITY, [&](float x) {
                if (x > -INFINITY) count_logit(sh, x, top, scale);
            });
            __syncthreads();
            from = count_edge(sh, set.top_k, top, floor, scale);
        }
        uint32_t n = kList + 1;
        if (from > -INFINITY) n = slice.row.collect(sh, from, top);
        return write_list(sh, slice.own, n);
    }
    const Weights weight = weights_of(sh, args, top, set.temperature);  // no factor is read
    mass_histogram<1>(sh, slice.row, weight, [](float, uint32_t) { return true; });
    for (int b = t; b < kMass; b += kThreads) slice.own->mass[b] = sh.bin[kMass - 1 - b];
}

template <typename T>
__global__ __launch_bounds__(kThreads) void split_border_kernel(SampleArgs args, Slice *work, int slices, int per) {
    extern __shared__ __align__(16) char memory[];
    Shared &sh = *reinterpret_cast<Shared *>(memory);
    const int t = threadIdx.x;
    SliceOf<T> slice(args, work, blockIdx.y, blockIdx.x, slices, per);
    const Settings set(args, blockIdx.y);
    slice.extremes();
    const float top = slice.top;
    if (set.single || set.top_k || !(fabsf(top) < INFINITY)) return;
    fill_factors(sh, args.shift);
    __syncthreads();
    const Weights weight = weights_of(sh, args, top, set.temperature);
    const float least = set.least(top);
    Own mass = {};
    if (set.top_p < 1.0f && kOwn * t < kNone)
        slice.each_slice([&](const Slice &one) { return *reinterpret_cast<const Own *>(one.mass + kOwn * t); }, Own{},
                         [&](const Own &m) {
#pragma unroll
                             for (int i = 0; i < kOwn; ++i) mass.v[i] += m.v[i];
                         });
    const Border border = find_border(sh, weight, set, least, mass);
    double sum = 0.0;  // in a fixed order: 64-bit floating point is as good as whole numbers
    for (int b = t; b < min(border.bin, kNone); b += kThreads)
        sum = fma(double(slice.own->mass[b]), weight.zero[-b] * weight.per_unit, sum);
    const uint64_t kept = block_add(sh, uint64_t(__builtin_rint(sum)));
    if (border.bin < kMass) {
        find_edges(sh, weight, top, border.bin);
        __syncthreads();
        const float lo = sh.edge[0], hi = sh.edge[1];
        write_list(sh, slice.own, slice.row.collect(sh, lo, fminf(next_below(hi), top)));
        if (t == 0) slice.own->lo = lo, slice.own->hi = fminf(hi, top);
    }
    if (t == 0) {
        slice.own->kept = kept;
        slice.own->border = border;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void split_draw_kernel(SampleArgs args, Slice *work, int slices, int per) {
    extern __shared__ __align__(16) char memory[];
    Shared &sh = *reinterpret_cast<Shared *>(memory);
    const int t = threadIdx.x;
    const int64_t r = blockIdx.x;
    SliceOf<T> slice(args, work, r, 0, slices, per);
    const Settings set(args, r);
    const Output out{args.out_token, args.out_prob};
    slice.extremes();
    const float top = slice.top;
    if (top == -INFINITY) {
        if (t == 0) write_row(out, r, 0xffffffffu, 0.0f);
        return;
    }
    if (set.single) {
        uint32_t first = 0xffffffffu;
        if ((t & 63) < slices && slice.all[t & 63].top == top) first = slice.all[t & 63].first;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) first = min(first, uint32_t(__shfl_xor(int(first), o)));
        if (t == 0) write_row(out, r, first, 1.0f);
        return;
    }
    fill_factors(sh, args.shift);
    // the slices' lists side by side
    const uint64_t upto = wave_scan((t & 63) < slices ? slice.all[t & 63].count : 0);
    const uint64_t total = lane64(upto, 63);
    const bool whole = !__any((t & 63) < slices && slice.all[t & 63].count > uint32_t(kList));
    // (sample_row's first barrier is ahead of the factors' use)
    if (!whole || (set.top_k && total > kList) || top == INFINITY) return sample_row<T>(sh, args, r);
    const uint32_t n = uint32_t(total);
    if (n <= kList) {
        if (t < kSlices) sh.bin[t] = upto;
        __syncthreads();
        for (uint32_t j = t; j < n; j += kThreads) {
            int s = 0;
            while (sh.bin[s] <= j) ++s;
            sh.list[j] = slice.all[s].list[j - (s ? uint32_t(sh.bin[s - 1]) : 0)];
        }
    }
    if (t < kSlices) sh.seg[t] = t < slices ? slice.all[t].kept : 0;
    __syncthreads();
    Row<T> row(args, r);
    row.per = per;
    const Weights weight = weights_of(sh, args, top, set.temperature);
    const float least = set.least(top);
    if (set.top_k)
        return draw_from_list(sh, out, r, n, weight, set, least, -INFINITY, uint32_t(row.v),
                              [&](uint32_t i) { return static_cast<float>(row.p[i]); });
    Cut cut;
    const Border border = slice.own->border;
    if (border.bin < kMass && n <= kList) {
        settle_list(sh, row, weight, n, border, slice.own->lo, slice.own->hi, least, cut);
    } else if (border.bin < kMass) {  // more than LDS holds: from where they are
        const auto lists = [&](auto f) {
            for (int s = 0; s < slices; ++s) {
                const uint32_t own = slice.all[s].count;
                for (uint32_t j = t; j < own; j += kThreads) {
                    const uint64_t key = slice.all[s].list[j];
                    f(key, weight(key_value(key)));
                }
            }
        };
        if (border.by_p) {
            const uint64_t key = find_first(sh, lists, border.target - border.before);
            if (key) cut.from_key(key);
        }
        cut.from_value(least);
        lists([&](uint64_t key, uint64_t w) {
            if (cut(key_value(key), key_index(key))) add64(&sh.seg[row.segment(key_index(key))], w);
        });
    }
    __syncthreads();
    draw_from_row(sh, out, r, row, weight, set.u, cut);
}

template <typename T>
hipError_t launch_split(const SampleArgs &a, Split split, void *workspace, hipStream_t s) {
    Slice *work = static_cast<Slice *>(workspace);
    static std::atomic<uint64_t> told[4];
    void (*const kernels[4])(SampleArgs, Slice *, int, int) = {split_top_kernel<T>, split_candidates_kernel<T>,
                                                               split_border_kernel<T>, split_draw_kernel<T>};
    hipError_t err = hipSuccess;
    for (int i = 0; i < 4 && err == hipSuccess; ++i) {
        if (i == 2 && a.set.top_ks == nullptr && a.set.top_k > 0 && a.set.top_k < a.v) continue;  // every row is top-k's
        err = allow_lds(reinterpret_cast<const void *>(kernels[i]), int(sizeof(Shared)), told[i]);
        if (err != hipSuccess) break;
        const dim3 grid = i == 3 ? dim3(unsigned(a.r)) : dim3(unsigned(split.slices), unsigned(a.r));
        kernels[i]<<<grid, kThreads, sizeof(Shared), s>>>(a, work, split.slices, split.per);
        err = hipGetLastError();
    }
    return err;
}

template <typename T>
hipError_t launch(const SampleArgs &a, int32_t dtype, void *workspace, hipStream_t s) {
    // Measured (us, one workgroup a row | slices; bf16, unless said):
    //   r x v                  no filter  top-p 0.95  min-p    top-k 50  greedy
    //   1 x 32000 fp32         13 | 16    19 | 23    15 | 19   11 | 17   7 | 16
    //   1 x 131072             26 | 18    37 | 30    25 | 19   12 | 19   9 | 16
    //   8 x 131072             27 | 19    37 | 33    26 | 20   13 | 21   9 | 15
    //   16 x 131072            27 | 19    38 | 37    26 | 20   13 | 22   9 | 15
    //   64 x 131072            28 | 30    38 | 43    26 | 28   13 | 20   9 | 15
    //   16 x 131072 fp32       30 | 19    39 | 34    34 | 24   14 | 21   13 | 15
    //   1 x 1000000 fp32      163 | 30   685 | 88   169 | 28   41 | 22   75 | 15
    // So top-k and greedy rows are shared from kSplitLight bytes on, the others
    // always; where each row's top-k is its own (some may be off), few rows only.
    const Split split = sample_split(a.r, a.v, sizeof(T));
    const int64_t bytes = a.v * int64_t(sizeof(T));
    const bool light = (a.set.top_ks == nullptr && a.set.top_k > 0) ||
                       (a.set.temperatures == nullptr && !(a.set.temperature > 0.0f));
    const int64_t from = light ? kSplitLight : a.set.top_ks == nullptr ? 0 : 4 * kSplitChunk * a.r;
    if (split.slices > 1 && bytes >= from) return launch_split<T>(a, split, workspace, s);
    // Measured (us, 1024 threads a row | 512, two rows a CU; bf16, unless said):
    //   r x v                 no filter  top-p 0.95  top-k 50  each its own
    //   1 x 500 fp32           9 | 8     13 | 12     12 | 11    7 | 7
    //   300 x 500 fp32        17 | 10    25 | 16     24 | 15   24 | 18
    //   1 x 32000 fp32        13 | 15    19 | 21     11 | 11    7 | 7
    //   256 x 32000           15 | 15    22 | 22     11 | 13   21 | 21
    //   256 x 131072          37 | 42    52 | 58     19 | 21   42 | 48
    //   512 x 32000           28 | 22    41 | 31     22 | 17   40 | 28
    //   512 x 100000 fp32     75 | 78   106 | 107    46 | 48   81 | 80
    if (a.r > 256 || a.v <= kList) return launch_rows_512(a, dtype, s);
    return launch_rows<T>(a, s);
}

static_assert(sizeof(Slice) <= kSampleSlice, "the workspace holds the slices");

}  // namespace
}  // namespace rt

extern "C" rt_status rt_sample_rows(const void *logits, int32_t dtype, int64_t r, int64_t v, int64_t ld,
                                    const float *u, const rt_sample_settings *settings, int32_t *out_token,
                                    float *out_prob, void *workspace, int64_t workspace_bytes, void *stream) {
    rt_status st = rt_check_sample_rows(logits, dtype, r, v, ld, u, settings, out_token, out_prob, workspace,
                                        workspace_bytes);
    if (st != RT_OK || r == 0) return st;
    const int shift = rt::sample_shift(v);
    const rt::SampleArgs a{logits, r, v, ld, u, *settings, out_token, out_prob, shift, rt::sample_units(shift),
                           1.0 / double(int64_t(1) << shift)};
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t err;
    switch (dtype) {
        case RT_DTYPE_FLOAT32: err = rt::launch<float>(a, dtype, workspace, s); break;
        case RT_DTYPE_BFLOAT16: err = rt::launch<rt::bf16_t>(a, dtype, workspace, s); break;
        default: err = rt::launch<rt::fp16_t>(a, dtype, workspace, s);
    }
    if (err != hipSuccess) {
        (void)hipGetLastError();
        return RT_EHIP;
    }
    return RT_OK;
}
