// The global norm of a list of gradient tensors, and their clipping.
//     norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + eps)),  out = g coef
//
// Squares are summed in 64 bits: an fp32 square overflows above 1.8e19 and a sum
// over 10^9 values would lose its small ones.
//
// The list travels in the kernel arguments, so no copy from host memory is
// enqueued and a captured call replays by itself: directly up to kEntries
// tensors, and for longer lists by small kernels that write their share of the
// table into the workspace first, so that the two passes over the gradients stay
// one launch each.
//
// HBM-bound: the tensors are laid end to end, each padded to 1024 elements so that
// a run holds few of them, and every workgroup takes one equal run, whatever
// tensors that crosses (with chunks of 8192 elements
// taken in turn a workgroup spent more time finding its next chunk than reading
// it: 71 us for the sums of 115M bf16 values).  A piece of a tensor is read with
// 16-byte loads from its first aligned address on (gradients are often views into
// one bucket, at any offset); the elements before and after go one by one.  Every
// workgroup leaves one partial sum; the scaling kernel adds them all itself, in
// the same order everywhere, which saves a launch between the two.
//
// The second pass reads what the first has just read, so the loads are ordinary
// ones (non-temporal, the 256 MB last-level cache keeps nothing of them) and the
// stores of the scaled values non-temporal, in whole lines: 115M bf16 values into
// fp32 take 46 us for the sums and 110 us for the scaling (5.0 and 6.3 TB/s).  When
// this was chosen, with other runs, it was 46 + 127 us, against 43 + 155 us with
// non-temporal loads and 82 + 127 us with ordinary stores.
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kSumUnroll = 4, kScaleUnroll = 8;   // vectors in flight per lane
constexpr int kEntries = 120;           // 32 bytes each: a table stays under 4 KB of kernel arguments
constexpr int64_t kMinRun = 4096;       // elements of a workgroup, at least
constexpr int64_t kPad = 1024;          // a tensor counts as whole multiples of this many
constexpr int64_t kSmall = 2048;        // a piece up to here is read by one wave
// Workgroups (8 per CU), and partial sums.  1280 save 4 us where 15M values are read
// and not scaled (14 + 6 us) and cost 8 us at 115M (110 us for the scaling); 4096
// save nothing.
constexpr int kGrid = 2048;

struct Entry {
    const void *in;
    void *out;
    int64_t n_flags;                    // elements * 4 + (in is bf16) + 2 * (out is bf16)
    int64_t first;                      // the padded elements of the entries before
};
struct Table {
    Entry e[kEntries];
};
__host__ __device__ inline int64_t padded(int64_t n) { return (n + kPad - 1) / kPad * kPad; }

// The entry that holds element c of the list: the last with first <= c.  Every
// lane tests one entry, so a list of a few hundred costs one memory latency.
__device__ __forceinline__ int find(const Entry *e, int count, int64_t c) {
    const int lane = threadIdx.x % 64;
    int n = 0;
    for (int i = 0; i < count; i += 64)
        n += __popcll(__ballot(i + lane < count && e[i + lane < count ? i + lane : 0].first <= c));
    return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double tmp[kThreads / 64];
    for (int o = 32; o > 0; o /= 2) v += __shfl_xor(v, o);
    if (threadIdx.x % 64 == 0) tmp[threadIdx.x / 64] = v;
    __syncthreads();
    v = tmp[0];
    for (int w = 1; w < kThreads / 64; ++w) v += tmp[w];
    return v;
}

// V consecutive elements in one access (16 or 8 bytes)
template <typename T, int V> struct Vec {
    static constexpr int kWords = V * static_cast<int>(sizeof(T)) / 4;
    typedef uint32_t raw __attribute__((ext_vector_type(kWords)));
    static __device__ __forceinline__ void widen(raw q, float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (sizeof(T) == 2)
                v[i] = __uint_as_float(i % 2 ? (q[i / 2] & 0xffff0000u) : (q[i / 2] << 16));
            else
                v[i] = __uint_as_float(q[i]);
        }
    }
    static __device__ __forceinline__ raw narrow(const float (&v)[V]) {
        raw q;
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (sizeof(T) == 2)
                q[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                       (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
            else
                q[i] = __float_as_uint(v[i]);
        }
        return q;
    }
};

// The vectors of V elements inside elements [i0, i0 + n) of p, aligned to their
// size: `head` elements come before the first, `vecs` vectors follow, the rest
// comes after.
struct Cut {
    int head;
    int64_t vecs;
};
template <int V, typename T> __device__ __forceinline__ Cut cut(const T *p, int64_t i0, int64_t n) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p + i0) % (V * sizeof(T))) / sizeof(T));
    const int head = off ? static_cast<int>(V - off < n ? V - off : n) : 0;
    return {head, (n - head) / V};
}

template <typename T> __device__ __forceinline__ double sum_piece(const T *p, int64_t i0, int64_t n, int t, int threads) {
    constexpr int V = 16 / sizeof(T);
    using X = Vec<T, V>;
    const Cut c = cut<V>(p, i0, n);
    const typename X::raw *b = reinterpret_cast<const typename X::raw *>(p + i0 + c.head);
    double s = 0.0;
    auto add = [&](typename X::raw w) {
        float v[V];
        X::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
    };
    int64_t k = t;
    for (; k + (kSumUnroll - 1) * threads < c.vecs; k += kSumUnroll * threads) {
        typename X::raw w[kSumUnroll];
#pragma unroll
        for (int i = 0; i < kSumUnroll; ++i) w[i] = b[k + i * threads];
#pragma unroll
        for (int i = 0; i < kSumUnroll; ++i) add(w[i]);
    }
    for (; k < c.vecs; k += threads) add(b[k]);
    auto one = [&](const T *e) {
        const double v = to_f32(*e);
        s = fma(v, v, s);
    };
    if (t < c.head) one(p + i0 + t);
    const int64_t tail = c.head + c.vecs * V + t;
    if (tail < n) one(p + i0 + tail);
    return s;
}

// V elements per lane: 16 bytes of the wider side, so that the lanes of a store
// fill whole lines
template <typename T, typename O> __device__ __forceinline__ void scale_piece(const T *p, O *out, int64_t i0, int64_t n, float coef, int t, int threads) {
    constexpr int V = 16 / (sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));
    using X = Vec<T, V>;
    using Y = Vec<O, V>;
    const Cut c = cut<V>(p, i0, n);
    const typename X::raw *b = reinterpret_cast<const typename X::raw *>(p + i0 + c.head);
    O *o = out + i0 + c.head;
    const bool aligned = reinterpret_cast<uintptr_t>(o) % (V * sizeof(O)) == 0;
    auto scale = [&](typename X::raw w, int64_t k) {
        float v[V];
        X::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= coef;
        if (aligned) {
            const typename Y::raw q = Y::narrow(v);
            __builtin_nontemporal_store(q, reinterpret_cast<typename Y::raw *>(o) + k);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) o[k * V + i] = from_f32<O>(v[i]);
        }
    };
    int64_t k = t;
    for (; k + (kScaleUnroll - 1) * threads < c.vecs; k += kScaleUnroll * threads) {
        typename X::raw w[kScaleUnroll];
#pragma unroll
        for (int i = 0; i < kScaleUnroll; ++i) w[i] = b[k + i * threads];
#pragma unroll
        for (int i = 0; i < kScaleUnroll; ++i) scale(w[i], k + i * threads);
    }
    for (; k < c.vecs; k += threads) scale(b[k], k);
    if (t < c.head) out[i0 + t] = from_f32<O>(to_f32(p[i0 + t]) * coef);
    const int64_t tail = c.head + c.vecs * V + t;
    if (tail < n) out[i0 + tail] = from_f32<O>(to_f32(p[i0 + tail]) * coef);
}

__device__ __forceinline__ uint64_t lane_value(uint64_t v, int lane) {
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(v), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(v >> 32), lane);
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// f(entry, first element, elements, thread, threads) for every piece of the
// workgroup's run.  A wave reads 64 entries at a time, one per lane, so that the
// next piece is found without a trip to memory; a small piece is one wave's, and
// the waves take turns at them.
template <typename F> __device__ __forceinline__ void walk(const Entry *tab, int count, int64_t total, int64_t run, F f) {
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    int64_t c = blockIdx.x * run;
    const int64_t end = c + run < total ? c + run : total;
    for (int i = find(tab, count, c); i < count && c < end; i += 64) {
        const Entry mine = tab[i + lane < count ? i + lane : count - 1];
        const int here = count - i < 64 ? count - i : 64;
        for (int j = 0; j < here && c < end; ++j) {
            Entry e;
            e.in = reinterpret_cast<const void *>(lane_value(reinterpret_cast<uint64_t>(mine.in), j));
            e.out = reinterpret_cast<void *>(lane_value(reinterpret_cast<uint64_t>(mine.out), j));
            e.n_flags = static_cast<int64_t>(lane_value(static_cast<uint64_t>(mine.n_flags), j));
            e.first = static_cast<int64_t>(lane_value(static_cast<uint64_t>(mine.first), j));
            const int64_t size = e.n_flags >> 2, i0 = c - e.first, stop = end - e.first < size ? end - e.first : size;
            c = e.first + padded(size);              // where the next entry starts
            if (i0 >= stop) continue;
            if (stop - i0 > kSmall)
                f(e, i0, stop - i0, static_cast<int>(threadIdx.x), kThreads);
            else if ((i + j) % (kThreads / 64) == w)
                f(e, i0, stop - i0, lane, 64);
        }
    }
}

__device__ __forceinline__ void sumsq(const Entry *tab, int count, int64_t total, int64_t run, double *part) {
    double s = 0.0;
    walk(tab, count, total, run, [&](const Entry &e, int64_t i0, int64_t n, int t, int threads) {
        s += e.n_flags & 1 ? sum_piece(static_cast<const bf16_t *>(e.in), i0, n, t, threads)
                           : sum_piece(static_cast<const float *>(e.in), i0, n, t, threads);
    });
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// every workgroup adds the partial sums, in the same order
__device__ __forceinline__ double norm_of(const double *part, int parts) {
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    return sqrt(block_sum(s));
}

__device__ __forceinline__ void clip(const Entry *tab, int count, int64_t total, int64_t run, const double *part, int parts,
                                     float max_norm, float eps, float *norm, int in_place) {
    const double wide = norm_of(part, parts);
    const float value = static_cast<float>(wide);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = value;
    // finite gradients may have a norm past fp32; at or below the limit nothing is
    // divided, so no 0 / 0 or inf / inf; a NaN norm fails both tests and stays
    const float coef = value + eps <= max_norm         ? 1.0f
                       : value == __builtin_inff()     ? static_cast<float>(max_norm / wide)
                                                       : max_norm / (value + eps);
    if (coef == 1.0f && in_place) return;              // nothing changes
    walk(tab, count, total, run, [&](const Entry &e, int64_t i0, int64_t n, int t, int threads) {
        if (coef == 1.0f && e.out == e.in) return;
        switch (e.n_flags & 3) {
        case 0: scale_piece(static_cast<const float *>(e.in), static_cast<float *>(e.out), i0, n, coef, t, threads); break;
        case 1: scale_piece(static_cast<const bf16_t *>(e.in), static_cast<float *>(e.out), i0, n, coef, t, threads); break;
        case 2: scale_piece(static_cast<const float *>(e.in), static_cast<bf16_t *>(e.out), i0, n, coef, t, threads); break;
        default: scale_piece(static_cast<const bf16_t *>(e.in), static_cast<bf16_t *>(e.out), i0, n, coef, t, threads);
        }
    });
}

__global__ __launch_bounds__(kThreads) void sumsq_kernel(Table t, int count, int64_t total, int64_t run, double *part) {
    sumsq(t.e, count, total, run, part);
}
__global__ __launch_bounds__(kThreads) void sumsq_long_kernel(const Entry *tab, int count, int64_t total, int64_t run, double *part) {
    sumsq(tab, count, total, run, part);
}
__global__ __launch_bounds__(kThreads) void clip_kernel(Table t, int count, int64_t total, int64_t run, const double *part,
                                                        int parts, float max_norm, float eps, float *norm, int in_place) {
    clip(t.e, count, total, run, part, parts, max_norm, eps, norm, in_place);
}
__global__ __launch_bounds__(kThreads) void clip_long_kernel(const Entry *tab, int count, int64_t total, int64_t run,
                                                             const double *part, int parts, float max_norm, float eps,
                                                             float *norm, int in_place) {
    clip(tab, count, total, run, part, parts, max_norm, eps, norm, in_place);
}
__global__ __launch_bounds__(kThreads) void norm_kernel(const double *part, int parts, float *norm) {
    const double v = norm_of(part, parts);
    if (threadIdx.x == 0) *norm = static_cast<float>(v);
}
__global__ __launch_bounds__(kThreads) void table_kernel(Table t, int count, Entry *tab) {
    if (static_cast<int>(threadIdx.x) < count) tab[threadIdx.x] = t.e[threadIdx.x];
}
static_assert(kEntries <= kThreads, "one thread writes one entry");

// the next entries of the list that hold anything, from index i on
int64_t fill(Table &t, int &count, int64_t &total, const ClipArgs &a, int64_t i) {
    for (count = 0; i < a.count && count < kEntries; ++i) {
        const int64_t n = a.numel[i];
        if (n == 0) continue;
        Entry &e = t.e[count++];
        e.in = a.grads[i];
        e.out = a.outs ? a.outs[i] : const_cast<void *>(a.grads[i]);
        e.n_flags = n * 4 + (a.dtypes[i] != 0 ? 1 : 0) + (a.out_dtypes[i] != 0 ? 2 : 0);
        e.first = total;
        total += padded(n);
    }
    return i;
}

}  // namespace

// the partial sums, then the table of a long list
size_t grad_norm_workspace(int64_t count) {
    return kGrid * sizeof(double) + static_cast<size_t>(count > kEntries ? count : 0) * sizeof(Entry);
}

hipError_t launch_grad_clip(const ClipArgs &a, hipStream_t s) {
    Table t;
    double *part = static_cast<double *>(a.workspace);
    Entry *tab = reinterpret_cast<Entry *>(part + kGrid);
    int count = 0, entries = 0;
    int64_t total = 0;
    const bool is_long = a.count > kEntries;
    const int in_place = a.outs ? 0 : 1;               // every tensor
    for (int64_t i = 0; i < a.count;) {
        i = fill(t, count, total, a, i);
        if (is_long && count > 0)
            hipLaunchKernelGGL(table_kernel, dim3(1), dim3(kThreads), 0, s, t, count, tab + entries);
        entries += count;
    }
    // equal runs, of whole 16-byte vectors from the start of an aligned tensor
    const int64_t wgs = (total + kMinRun - 1) / kMinRun;
    const int64_t run = wgs <= kGrid ? kMinRun : ((total + kGrid - 1) / kGrid + 7) / 8 * 8;
    const int grid = static_cast<int>((total + run - 1) / run);
    if (grid > 0) {
        if (is_long)
            hipLaunchKernelGGL(sumsq_long_kernel, dim3(grid), dim3(kThreads), 0, s, tab, entries, total, run, part);
        else
            hipLaunchKernelGGL(sumsq_kernel, dim3(grid), dim3(kThreads), 0, s, t, entries, total, run, part);
    }
    if (!a.scale || grid == 0)
        hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, grid, a.norm);
    else if (is_long)
        hipLaunchKernelGGL(clip_long_kernel, dim3(grid), dim3(kThreads), 0, s, tab, entries, total, run, part, grid,
                           a.max_norm, a.eps, a.norm, in_place);
    else
        hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(kThreads), 0, s, t, entries, total, run, part, grid, a.max_norm,
                           a.eps, a.norm, in_place);
    return hipGetLastError();
}

}  // namespace ssm
