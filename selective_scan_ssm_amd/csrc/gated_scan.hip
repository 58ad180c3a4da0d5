// The gated linear recurrence, its gradient and its one-token form:
//     a = sigmoid(g + bias),  h <- a h + (1 - a) x,  y = h SiLU(z)
// First form: one lane walks one (batch, channel) chain through time.
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

// a = sigmoid(v) and s = 1 - a = sigmoid(-v).  The smaller of the two is
// e / (1 + e) with e = exp(-|v|), to a relative accuracy of a few ulp; the
// larger is 1 minus it, rounded once, so neither a decay near 1 nor its
// complement carries a bias.  v log2(e) is taken in two parts, as its rounding
// alone would cost |v| / 2 ulp.  The clamp keeps infinite gates exact (e = 0).
struct Gate {
    float a, s;
};
__device__ __forceinline__ Gate gate(float v) {
    constexpr float kLog2eLo = 1.925963033500411e-08f;   // log2(e) - float(log2(e))
    float av = fabsf(v);
    av = av > 128.0f ? 128.0f : av;                       // false for NaN, which stays
    const float t = av * kLog2e;
    const float lo = fmaf(av, kLog2eLo, fmaf(av, kLog2e, -t));
    const float e = fast_exp2(-t) * fmaf(-lo, kLn2, 1.0f);
    const float small = e / (1.0f + e);
    const float large = 1.0f - small;
    return v >= 0.0f ? Gate{large, small} : Gate{small, large};
}

struct FwdParams {
    const void *x, *g, *z;
    int64_t ldx, ldg, ldz;
    const float *bias, *h0;
    void *y;
    float *last, *ckpt, *before;      // before: every state entering a step (workspace), or null
    int64_t batch, seqlen, dim;
};

template <typename T> __global__ __launch_bounds__(64) void gated_fwd_kernel(FwdParams p) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.dim) return;
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.g), *z = static_cast<const T *>(p.z);
    T *y = static_cast<T *>(p.y);
    const float bias = p.bias ? p.bias[d] : 0.0f;
    float h = p.h0 ? p.h0[b * p.dim + d] : 0.0f;
    const int64_t blocks = (p.seqlen + kGatedBlock - 1) / kGatedBlock;
    for (int64_t t = 0; t < p.seqlen; ++t) {
        const int64_t row = b * p.seqlen + t;
        if (p.ckpt && t % kGatedBlock == 0) p.ckpt[(b * blocks + t / kGatedBlock) * p.dim + d] = h;
        if (p.before) p.before[row * p.dim + d] = h;
        const Gate k = gate(to_f32(g[row * p.ldg + d]) + bias);
        h = fmaf(k.a, h, k.s * to_f32(x[row * p.ldx + d]));
        if (y) y[row * p.dim + d] = from_f32<T>(z ? h * silu(to_f32(z[row * p.ldz + d])) : h);
    }
    if (p.last) p.last[b * p.dim + d] = h;
}

struct BwdParams {
    const void *x, *g, *z, *dout;
    int64_t ldx, ldg, ldz;
    const float *bias, *dlast, *before;
    void *dx, *dg, *dz;
    float *dbias_part, *dh0;
    int64_t batch, seqlen, dim;
};

template <typename T> __global__ __launch_bounds__(64) void gated_bwd_kernel(BwdParams p) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    const int64_t b = blockIdx.y;
    if (d >= p.dim) return;
    const T *x = static_cast<const T *>(p.x), *g = static_cast<const T *>(p.g), *z = static_cast<const T *>(p.z);
    const T *dout = static_cast<const T *>(p.dout);
    T *dx = static_cast<T *>(p.dx), *dg = static_cast<T *>(p.dg), *dz = static_cast<T *>(p.dz);
    const float bias = p.bias ? p.bias[d] : 0.0f;
    float carry = p.dlast ? p.dlast[b * p.dim + d] : 0.0f;
    double db = 0.0;
    for (int64_t t = p.seqlen - 1; t >= 0; --t) {
        const int64_t row = b * p.seqlen + t, i = row * p.dim + d;
        const Gate k = gate(to_f32(g[row * p.ldg + d]) + bias);
        const float hb = p.before[i], xv = to_f32(x[row * p.ldx + d]);
        float e = to_f32(dout[i]);
        if (z) {
            const float zv = to_f32(z[row * p.ldz + d]);
            const Gate s = gate(zv);
            const float h = fmaf(k.a, hb, k.s * xv);
            dz[i] = from_f32<T>(e * h * (s.a * fmaf(zv, s.s, 1.0f)));
            e *= zv * s.a;
        }
        e += carry;
        const float dgv = e * (hb - xv) * (k.a * k.s);
        dx[i] = from_f32<T>(k.s * e);
        dg[i] = from_f32<T>(dgv);
        db += dgv;
        carry = k.a * e;
    }
    p.dbias_part[b * p.dim + d] = static_cast<float>(db);
    if (p.dh0) p.dh0[b * p.dim + d] = carry;
}

__global__ __launch_bounds__(64) void gated_dbias_kernel(const float *part, float *out, int64_t rows, int64_t dim) {
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x;
    if (d >= dim) return;
    float s = 0.0f;
    for (int64_t r = 0; r < rows; ++r) s += part[r * dim + d];
    out[d] = s;
}

template <typename T> __global__ __launch_bounds__(256) void gated_update_kernel(GatedStepArgs p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.batch * p.dim) return;
    const float bias = p.gate_bias ? p.gate_bias[i % p.dim] : 0.0f;
    const Gate k = gate(to_f32(static_cast<const T *>(p.g)[i]) + bias);
    const float h = fmaf(k.a, p.state[i], k.s * to_f32(static_cast<const T *>(p.x)[i]));
    p.state[i] = h;
    static_cast<T *>(p.y)[i] = from_f32<T>(p.z ? h * silu(to_f32(static_cast<const T *>(p.z)[i])) : h);
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T> hipError_t launch_fwd(const GatedArgs &a, float *before, hipStream_t s) {
    FwdParams p{a.x, a.g, a.z, a.ldx, a.ldg, a.ldz, a.gate_bias, a.h0, a.y, a.last_state, a.ckpt, before,
                a.batch, a.seqlen, a.dim};
    const dim3 grid(static_cast<unsigned>((a.dim + 63) / 64), static_cast<unsigned>(a.batch));
    hipLaunchKernelGGL(gated_fwd_kernel<T>, grid, dim3(64), 0, s, p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_bwd(const GatedBwdArgs &a, hipStream_t s) {
    const GatedArgs &f = a.fwd;
    char *ws = static_cast<char *>(f.workspace);
    float *part = reinterpret_cast<float *>(ws);
    float *before = reinterpret_cast<float *>(ws + round256(f.batch * f.dim * 4));
    const unsigned cols = static_cast<unsigned>((f.dim + 63) / 64);
    if (f.batch > 0) {
        GatedArgs g = f;
        g.y = nullptr; g.last_state = nullptr; g.ckpt = nullptr;
        if (hipError_t e = launch_fwd<T>(g, before, s)) return e;
        BwdParams p{f.x, f.g, f.z, a.dout, f.ldx, f.ldg, f.ldz, f.gate_bias, a.dlast, before, a.dx, a.dg, a.dz,
                    part, a.dh0, f.batch, f.seqlen, f.dim};
        hipLaunchKernelGGL(gated_bwd_kernel<T>, dim3(cols, static_cast<unsigned>(f.batch)), dim3(64), 0, s, p);
    }
    if (a.dgate_bias)
        hipLaunchKernelGGL(gated_dbias_kernel, dim3(cols), dim3(64), 0, s, part, a.dgate_bias, f.batch, f.dim);
    return hipGetLastError();
}

}  // namespace

size_t gated_scan_workspace(int64_t, int64_t, int64_t, int) { return 0; }

size_t gated_scan_bwd_workspace(int64_t batch, int64_t seqlen, int64_t dim, int) {
    return round256(batch * dim * 4) + round256(batch * seqlen * dim * 4);
}

hipError_t launch_gated_scan(const GatedArgs &a, hipStream_t s) {
    return a.bf16 ? launch_fwd<bf16_t>(a, nullptr, s) : launch_fwd<float>(a, nullptr, s);
}
hipError_t launch_gated_scan_bwd(const GatedBwdArgs &a, hipStream_t s) {
    return a.fwd.bf16 ? launch_bwd<bf16_t>(a, s) : launch_bwd<float>(a, s);
}
hipError_t launch_gated_update(const GatedStepArgs &a, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>((a.batch * a.dim + 255) / 256);
    if (a.bf16)
        hipLaunchKernelGGL(gated_update_kernel<bf16_t>, dim3(grid), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL(gated_update_kernel<float>, dim3(grid), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace ssm
