// RMS norm with the residual's addition, with an output in the io dtype or in
// 8 bits with a scale per row, and its gradient.
// First form: one workgroup per row, the row kept in LDS between the sum of
// squares and the output.
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.1754943508222875e-38f;   // 2^-126: scales stay normal numbers
constexpr int kPartRows = 64;                          // rows per workgroup of the gradient

template <typename F> __device__ __forceinline__ float block_reduce(float v, float *tmp, F f) {
    for (int o = 32; o > 0; o /= 2) v = f(v, __shfl_xor(v, o));
    __syncthreads();
    if (threadIdx.x % 64 == 0) tmp[threadIdx.x / 64] = v;
    __syncthreads();
    v = tmp[0];
    for (int w = 1; w < kThreads / 64; ++w) v = f(v, tmp[w]);
    return v;
}
struct Add {
    __device__ float operator()(float a, float b) const { return a + b; }
};
// the larger of two magnitudes, a NaN above everything (its bits are)
struct MaxAbs {
    __device__ float operator()(float a, float b) const {
        const uint32_t i = __float_as_uint(a) & 0x7fffffffu, j = __float_as_uint(b) & 0x7fffffffu;
        return __uint_as_float(i > j ? i : j);
    }
};

__device__ __forceinline__ uint8_t to_e4m3(float v) {
    return static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v, v, 0, false) & 0xff);
}

template <typename T, typename R> __global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs p) {
    extern __shared__ float row[];
    __shared__ float tmp[kThreads / 64];
    const int64_t r = blockIdx.x;
    const int dim = static_cast<int>(p.dim);
    const T *x = static_cast<const T *>(p.x) + r * p.ldx;
    const R *res = p.residual ? static_cast<const R *>(p.residual) + r * p.dim : nullptr;
    R *res_out = p.residual_out ? static_cast<R *>(p.residual_out) + r * p.dim : nullptr;
    float ss = 0.0f;
    for (int i = threadIdx.x; i < dim; i += kThreads) {
        float v = to_f32(x[i]);
        if (res) v += to_f32(res[i]);
        if (res_out) res_out[i] = from_f32<R>(v);
        row[i] = v;
        ss = fmaf(v, v, ss);
    }
    ss = block_reduce(ss, tmp, Add());
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(dim) + p.eps);
    if (!p.scale) {
        for (int i = threadIdx.x; i < dim; i += kThreads)
            (static_cast<T *>(p.y) + r * p.dim)[i] = from_f32<T>(row[i] * rstd * p.weight[i]);
        return;
    }
    float m = 0.0f;
    for (int i = threadIdx.x; i < dim; i += kThreads) {
        row[i] = row[i] * rstd * p.weight[i];
        m = MaxAbs()(m, row[i]);
    }
    m = block_reduce(m, tmp, MaxAbs());
    float scale = m / kE4m3Max;
    scale = scale < kMinScale ? kMinScale : scale;     // false for NaN, which stays
    if (threadIdx.x == 0) p.scale[r] = scale;
    for (int i = threadIdx.x; i < dim; i += kThreads)
        (static_cast<uint8_t *>(p.y) + r * p.dim)[i] = to_e4m3(row[i] / scale);
}

template <typename T, typename R> __global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormBwdArgs p) {
    __shared__ float tmp[kThreads / 64];
    const int dim = static_cast<int>(p.dim);
    float *part = static_cast<float *>(p.workspace) + static_cast<int64_t>(blockIdx.x) * p.dim;
    for (int i = threadIdx.x; i < dim; i += kThreads) part[i] = 0.0f;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kPartRows;
    for (int64_t r = r0; r < r0 + kPartRows && r < p.rows; ++r) {
        const T *dy = static_cast<const T *>(p.dy) + r * p.dim;
        const R *rr = static_cast<const R *>(p.r) + r * p.dim;
        const R *add = p.dres_out ? static_cast<const R *>(p.dres_out) + r * p.dim : nullptr;
        float ss = 0.0f, dot = 0.0f;
        for (int i = threadIdx.x; i < dim; i += kThreads) {
            const float v = to_f32(rr[i]);
            ss = fmaf(v, v, ss);
            dot = fmaf(v, p.weight[i] * to_f32(dy[i]), dot);
        }
        ss = block_reduce(ss, tmp, Add());
        dot = block_reduce(dot, tmp, Add());
        const float rstd = 1.0f / sqrtf(ss / static_cast<float>(dim) + p.eps);
        const float c = dot * rstd / static_cast<float>(dim);
        for (int i = threadIdx.x; i < dim; i += kThreads) {
            const float n = to_f32(rr[i]) * rstd, g = to_f32(dy[i]);
            float v = rstd * (p.weight[i] * g - n * c);
            if (add) v += to_f32(add[i]);
            static_cast<T *>(p.dx)[r * p.dim + i] = from_f32<T>(v);
            if (p.dres) static_cast<R *>(p.dres)[r * p.dim + i] = from_f32<R>(v);
            part[i] += g * n;
        }
    }
}

__global__ __launch_bounds__(kThreads) void norm_dweight_kernel(const float *part, float *out, int64_t parts, int64_t dim) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (d >= dim) return;
    float s = 0.0f;
    for (int64_t i = 0; i < parts; ++i) s += part[i * dim + d];
    out[d] = s;
}

int64_t parts_of(int64_t rows) { return (rows + kPartRows - 1) / kPartRows; }

}  // namespace

size_t norm_bwd_workspace(int64_t rows, int64_t dim) { return static_cast<size_t>(parts_of(rows) * dim) * 4; }

hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.rows)), block(kThreads);
    const size_t lds = static_cast<size_t>(a.dim) * 4;
    const void *f = a.bf16 ? (a.res_bf16 ? reinterpret_cast<const void *>(norm_kernel<bf16_t, bf16_t>)
                                         : reinterpret_cast<const void *>(norm_kernel<bf16_t, float>))
                           : reinterpret_cast<const void *>(norm_kernel<float, float>);
    if (lds > 60000)
        if (hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(lds)))
            return e;
    NormArgs p = a;
    void *args[] = {&p};
    return hipLaunchKernel(f, grid, block, args, lds, s);
}

hipError_t launch_add_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s) {
    const int64_t parts = parts_of(a.rows);
    if (parts > 0) {
        const dim3 grid(static_cast<unsigned>(parts)), block(kThreads);
        if (a.bf16 && a.res_bf16)
            hipLaunchKernelGGL((norm_bwd_kernel<bf16_t, bf16_t>), grid, block, 0, s, a);
        else if (a.bf16)
            hipLaunchKernelGGL((norm_bwd_kernel<bf16_t, float>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((norm_bwd_kernel<float, float>), grid, block, 0, s, a);
    }
    hipLaunchKernelGGL(norm_dweight_kernel, dim3(static_cast<unsigned>((a.dim + kThreads - 1) / kThreads)), dim3(kThreads),
                       0, s, static_cast<const float *>(a.workspace), a.dweight, parts, a.dim);
    return hipGetLastError();
}

}  // namespace ssm
