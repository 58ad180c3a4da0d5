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
// HBM-bound: a workgroup takes chunks of kChunk elements in turn and reads each
// with 16-byte loads from the first aligned address on (gradients are often
// views into one bucket, at any offset); the elements before and after go one
// by one.  Every workgroup leaves one partial sum; the scaling kernel adds them
// all itself, in the same order everywhere, which saves a launch between the two.
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kEntries = 120;           // 32 bytes each: a table stays under 4 KB of kernel arguments
constexpr int64_t kChunk = 8192;        // elements
constexpr int kGrid = 2048;             // workgroups (8 per CU), and partial sums

struct Entry {
    const void *in;
    void *out;
    int64_t n_flags;                    // elements * 4 + (in is bf16) + 2 * (out is bf16)
    int64_t first;                      // index of the entry's first chunk
};
struct Table {
    Entry e[kEntries];
};

// The entry whose chunks hold chunk c: the last with first <= c.  Every lane
// tests one entry, so a list of a few hundred costs one memory latency.
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

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// V consecutive elements of 16 bytes as fp32
template <typename T> struct Vec {
    static constexpr int V = 16 / sizeof(T);
    static __device__ __forceinline__ void widen(u4 q, float (&v)[V]) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (V == 8)
                v[i] = __uint_as_float(i % 2 ? (q[i / 2] & 0xffff0000u) : (q[i / 2] << 16));
            else
                v[i] = __uint_as_float(q[i]);
        }
    }
};

// The 16-byte vectors inside elements [i0, i1) of p: `head` elements come
// before the first, `vecs` vectors follow, the rest comes after.
struct Cut {
    int head, vecs;
};
template <typename T> __device__ __forceinline__ Cut cut(const T *p, int64_t i0, int n) {
    constexpr int V = Vec<T>::V;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(p + i0) % 16) / sizeof(T));
    const int head = off ? (V - off < n ? V - off : n) : 0;
    return {head, (n - head) / V};
}

template <typename T> __device__ __forceinline__ double sum_chunk(const T *p, int64_t i0, int n) {
    constexpr int V = Vec<T>::V, kUnroll = 4;
    const Cut c = cut(p, i0, n);
    const T *q = p + i0 + c.head;
    const u4 *b = reinterpret_cast<const u4 *>(q);
    double s = 0.0;
    auto add = [&](u4 w) {
        float v[V];
        Vec<T>::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), s);
    };
    int k = threadIdx.x;
    for (; k + (kUnroll - 1) * kThreads < c.vecs; k += kUnroll * kThreads) {
        u4 w[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) w[i] = b[k + i * kThreads];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) add(w[i]);
    }
    for (; k < c.vecs; k += kThreads) add(b[k]);
    auto one = [&](const T *e) {
        const double v = to_f32(*e);
        s = fma(v, v, s);
    };
    if (static_cast<int>(threadIdx.x) < c.head) one(p + i0 + threadIdx.x);
    const int tail = c.head + c.vecs * V + threadIdx.x;
    if (tail < n) one(p + i0 + tail);
    return s;
}

template <typename O> __device__ __forceinline__ void put(O *p, float v) { *p = from_f32<O>(v); }
// V fp32 values at out: 16-byte stores when its address allows them
template <typename O, int V> __device__ __forceinline__ void put_vec(O *out, const float (&v)[V], bool aligned) {
    constexpr int VO = 16 / sizeof(O);
    if (!aligned) {
#pragma unroll
        for (int i = 0; i < V; ++i) put(out + i, v[i]);
        return;
    }
    if constexpr (V >= VO) {
#pragma unroll
        for (int h = 0; h < V / VO; ++h) {
            u4 q;
            if constexpr (VO == 8) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                           (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = __float_as_uint(v[4 * h + i]);
            }
            reinterpret_cast<u4 *>(out)[h] = q;
        }
    } else {                                           // four fp32 values to bf16: 8 bytes
        typedef uint32_t u2 __attribute__((ext_vector_type(2)));
        u2 q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            q[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                   (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
        *reinterpret_cast<u2 *>(out) = q;
    }
}

template <typename T, typename O> __device__ __forceinline__ void scale_chunk(const T *p, O *out, int64_t i0, int n, float coef) {
    constexpr int V = Vec<T>::V, kUnroll = 4;
    constexpr int kOutBytes = V * sizeof(O) < 16 ? V * sizeof(O) : 16;
    const Cut c = cut(p, i0, n);
    const u4 *b = reinterpret_cast<const u4 *>(p + i0 + c.head);
    O *o = out + i0 + c.head;
    const bool aligned = reinterpret_cast<uintptr_t>(o) % kOutBytes == 0;
    auto scale = [&](u4 w, int k) {
        float v[V];
        Vec<T>::widen(w, v);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= coef;
        put_vec<O, V>(o + static_cast<int64_t>(k) * V, v, aligned);
    };
    int k = threadIdx.x;
    for (; k + (kUnroll - 1) * kThreads < c.vecs; k += kUnroll * kThreads) {
        u4 w[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) w[i] = b[k + i * kThreads];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) scale(w[i], k + i * kThreads);
    }
    for (; k < c.vecs; k += kThreads) scale(b[k], k);
    if (static_cast<int>(threadIdx.x) < c.head) put(out + i0 + threadIdx.x, to_f32(p[i0 + threadIdx.x]) * coef);
    const int tail = c.head + c.vecs * V + threadIdx.x;
    if (tail < n) put(out + i0 + tail, to_f32(p[i0 + tail]) * coef);
}

__device__ __forceinline__ void sumsq(const Entry *tab, int count, int64_t chunks, double *part) {
    double s = 0.0;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        const Entry &e = tab[find(tab, count, c)];
        const int64_t i0 = (c - e.first) * kChunk, left = (e.n_flags >> 2) - i0;
        const int n = static_cast<int>(left < kChunk ? left : kChunk);
        s += e.n_flags & 1 ? sum_chunk(static_cast<const bf16_t *>(e.in), i0, n)
                           : sum_chunk(static_cast<const float *>(e.in), i0, n);
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// every workgroup adds the partial sums, in the same order
__device__ __forceinline__ float norm_of(const double *part, int parts) {
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    return static_cast<float>(sqrt(block_sum(s)));
}

// Chunks are taken from the last one down: the sums have just been over them,
// so the last ones read are the likeliest to be in a cache still.
__device__ __forceinline__ void clip(const Entry *tab, int count, int64_t chunks, const double *part, int parts,
                                     float max_norm, float eps, float *norm) {
    const float total = norm_of(part, parts);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    float coef = max_norm / (total + eps);
    coef = coef > 1.0f ? 1.0f : coef;                  // false for NaN, which stays
    for (int64_t c = chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const Entry &e = tab[find(tab, count, c)];
        if (coef == 1.0f && e.out == e.in) continue;   // nothing changes
        const int64_t i0 = (c - e.first) * kChunk, left = (e.n_flags >> 2) - i0;
        const int n = static_cast<int>(left < kChunk ? left : kChunk);
        switch (e.n_flags & 3) {
        case 0: scale_chunk(static_cast<const float *>(e.in), static_cast<float *>(e.out), i0, n, coef); break;
        case 1: scale_chunk(static_cast<const bf16_t *>(e.in), static_cast<float *>(e.out), i0, n, coef); break;
        case 2: scale_chunk(static_cast<const float *>(e.in), static_cast<bf16_t *>(e.out), i0, n, coef); break;
        default: scale_chunk(static_cast<const bf16_t *>(e.in), static_cast<bf16_t *>(e.out), i0, n, coef);
        }
    }
}

__global__ __launch_bounds__(kThreads) void sumsq_kernel(Table t, int count, int64_t chunks, double *part) {
    sumsq(t.e, count, chunks, part);
}
__global__ __launch_bounds__(kThreads) void sumsq_long_kernel(const Entry *tab, int count, int64_t chunks, double *part) {
    sumsq(tab, count, chunks, part);
}
__global__ __launch_bounds__(kThreads) void clip_kernel(Table t, int count, int64_t chunks, const double *part, int parts,
                                                        float max_norm, float eps, float *norm) {
    clip(t.e, count, chunks, part, parts, max_norm, eps, norm);
}
__global__ __launch_bounds__(kThreads) void clip_long_kernel(const Entry *tab, int count, int64_t chunks, const double *part,
                                                             int parts, float max_norm, float eps, float *norm) {
    clip(tab, count, chunks, part, parts, max_norm, eps, norm);
}
__global__ __launch_bounds__(kThreads) void norm_kernel(const double *part, int parts, float *norm) {
    const float v = norm_of(part, parts);
    if (threadIdx.x == 0) *norm = v;
}
__global__ __launch_bounds__(kThreads) void table_kernel(Table t, int count, Entry *tab) {
    if (static_cast<int>(threadIdx.x) < count) tab[threadIdx.x] = t.e[threadIdx.x];
}
static_assert(kEntries <= kThreads, "one thread writes one entry");

// the next entries of the list that hold anything, from index i on
int64_t fill(Table &t, int &count, int64_t &chunks, const ClipArgs &a, int64_t i) {
    for (count = 0; i < a.count && count < kEntries; ++i) {
        const int64_t n = a.numel[i];
        if (n == 0) continue;
        Entry &e = t.e[count++];
        e.in = a.grads[i];
        e.out = a.outs ? a.outs[i] : const_cast<void *>(a.grads[i]);
        e.n_flags = n * 4 + (a.dtypes[i] != 0 ? 1 : 0) + (a.out_dtypes[i] != 0 ? 2 : 0);
        e.first = chunks;
        chunks += (n + kChunk - 1) / kChunk;
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
    int count = 0, total = 0;
    int64_t chunks = 0;
    const bool is_long = a.count > kEntries;
    for (int64_t i = 0; i < a.count;) {
        i = fill(t, count, chunks, a, i);
        if (is_long && count > 0)
            hipLaunchKernelGGL(table_kernel, dim3(1), dim3(kThreads), 0, s, t, count, tab + total);
        total += count;
    }
    const int grid = static_cast<int>(chunks < kGrid ? chunks : kGrid);
    if (grid > 0) {
        if (is_long)
            hipLaunchKernelGGL(sumsq_long_kernel, dim3(grid), dim3(kThreads), 0, s, tab, total, chunks, part);
        else
            hipLaunchKernelGGL(sumsq_kernel, dim3(grid), dim3(kThreads), 0, s, t, total, chunks, part);
    }
    if (!a.scale || grid == 0)
        hipLaunchKernelGGL(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, grid, a.norm);
    else if (is_long)
        hipLaunchKernelGGL(clip_long_kernel, dim3(grid), dim3(kThreads), 0, s, tab, total, chunks, part, grid, a.max_norm,
                           a.eps, a.norm);
    else
        hipLaunchKernelGGL(clip_kernel, dim3(grid), dim3(kThreads), 0, s, t, total, chunks, part, grid, a.max_norm, a.eps,
                           a.norm);
    return hipGetLastError();
}

}  // namespace ssm
