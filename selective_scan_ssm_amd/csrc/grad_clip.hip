// The global norm of a list of gradient tensors, and their clipping.
//     norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + eps)),  out = g coef
//
// The list travels in the kernel arguments, up to kEntries tensors per launch,
// so nothing is copied to the device beforehand and a captured call replays by
// itself.  Squares are summed in 64 bits: an fp32 square overflows above 1.8e19
// and a sum over 10^9 values would lose its small ones.
// First form: a workgroup takes chunks of kChunk elements in turn.
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kEntries = 112;           // 32 bytes each: the table stays under 4 KB of kernel arguments
constexpr int64_t kChunk = 16384;       // elements
constexpr int kGrid = 1024;             // workgroups, and partial sums, per launch

struct Entry {
    const void *in;
    void *out;
    int64_t n_flags;                    // elements * 4 + (in is bf16) + 2 * (out is bf16)
    int64_t first;                      // index of the entry's first chunk in this launch
};
struct Table {
    Entry e[kEntries];
    int count;
    int grid;
    int64_t chunks;
};

// the entry whose chunks hold chunk c
__device__ __forceinline__ int find(const Table &t, int64_t c) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    return lo;
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

__device__ __forceinline__ float load(const void *p, int64_t i, bool bf16) {
    return bf16 ? to_f32(static_cast<const bf16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}

__global__ __launch_bounds__(kThreads) void sumsq_kernel(Table t, double *part) {
    double s = 0.0;
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry &e = t.e[find(t, c)];
        const int64_t n = e.n_flags >> 2, i0 = (c - e.first) * kChunk, i1 = i0 + kChunk < n ? i0 + kChunk : n;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const double v = load(e.in, i, e.n_flags & 1);
            s = fma(v, v, s);
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// every workgroup adds the partial sums, in the same order
__device__ __forceinline__ float norm_of(const double *part, int64_t parts) {
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    return static_cast<float>(sqrt(block_sum(s)));
}

__global__ __launch_bounds__(kThreads) void norm_only_kernel(const double *part, int64_t parts, float *norm) {
    const float v = norm_of(part, parts);
    if (threadIdx.x == 0) *norm = v;
}

__global__ __launch_bounds__(kThreads) void clip_kernel(Table t, const double *part, int64_t parts, float max_norm,
                                                        float eps, float *norm) {
    const float total = norm_of(part, parts);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    float coef = max_norm / (total + eps);
    coef = coef > 1.0f ? 1.0f : coef;                  // false for NaN, which stays
    for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
        const Entry &e = t.e[find(t, c)];
        if (coef == 1.0f && e.out == e.in) continue;   // nothing changes
        const int64_t n = e.n_flags >> 2, i0 = (c - e.first) * kChunk, i1 = i0 + kChunk < n ? i0 + kChunk : n;
        for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const float v = load(e.in, i, e.n_flags & 1) * coef;
            if (e.n_flags & 2)
                static_cast<bf16_t *>(e.out)[i] = from_f32<bf16_t>(v);
            else
                static_cast<float *>(e.out)[i] = v;
        }
    }
}

// the next entries of the list that hold anything, from index i on
int64_t fill(Table &t, const ClipArgs &a, int64_t i) {
    t.count = 0;
    t.chunks = 0;
    for (; i < a.count && t.count < kEntries; ++i) {
        const int64_t n = a.numel[i];
        if (n == 0) continue;
        Entry &e = t.e[t.count++];
        e.in = a.grads[i];
        e.out = a.outs ? a.outs[i] : const_cast<void *>(a.grads[i]);
        e.n_flags = n * 4 + (a.dtypes[i] != 0 ? 1 : 0) + (a.out_dtypes[i] != 0 ? 2 : 0);
        e.first = t.chunks;
        t.chunks += (n + kChunk - 1) / kChunk;
    }
    t.grid = static_cast<int>(t.chunks < kGrid ? t.chunks : kGrid);
    return i;
}

}  // namespace

size_t grad_norm_workspace(int64_t count) {
    return static_cast<size_t>((count + kEntries - 1) / kEntries * kGrid) * sizeof(double);
}

hipError_t launch_grad_clip(const ClipArgs &a, hipStream_t s) {
    Table t;
    double *part = static_cast<double *>(a.workspace);
    int64_t parts = 0;
    for (int64_t i = 0; i < a.count;) {
        i = fill(t, a, i);
        if (t.count == 0) break;
        hipLaunchKernelGGL(sumsq_kernel, dim3(t.grid), dim3(kThreads), 0, s, t, part + parts);
        parts += t.grid;
    }
    if (!a.scale || parts == 0) {
        hipLaunchKernelGGL(norm_only_kernel, dim3(1), dim3(kThreads), 0, s, part, parts, a.norm);
        return hipGetLastError();
    }
    float *norm = a.norm;
    for (int64_t i = 0; i < a.count;) {
        i = fill(t, a, i);
        if (t.count == 0) break;
        hipLaunchKernelGGL(clip_kernel, dim3(t.grid), dim3(kThreads), 0, s, t, part, parts, a.max_norm, a.eps, norm);
        norm = nullptr;                                // the first launch writes it
    }
    return hipGetLastError();
}

}  // namespace ssm
