// RMS norm with the residual's addition, with an output in the io dtype or in
// 8 bits with a scale per row, and its gradient:
//     r = x + residual,  y = r / sqrt(mean(r^2) + eps) w
//     dr = rstd (w dy - n mean(n w dy)) + dresidual,  dw = sum over rows of dy n,  n = r rstd
//
// HBM-bound: a row is read once, kept in registers across the reduction(s), and
// written once.  R waves share a row (1 where a row fits one wave's registers)
// and each lane holds P chunks of V consecutive elements (16 bytes of the widest
// tensor; V = 1 where the width or an address does not allow that), so nothing
// but the reduction crosses lanes.  Waves walk the rows with a grid stride and
// keep the weight in registers; the gradient also keeps its lane's share of dw
// there, and one partial sum per workgroup goes through the workspace.
#include "column_sum.h"
#include "ssm_device.h"
#include "ssm_kernels.h"
#include "wave_fold.h"

namespace ssm {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kMinScale = 1.1754943508222875e-38f;   // 2^-126: scales stay normal numbers

// y / scale rounded to nearest, from inv = 1 / scale rounded to nearest: y inv is
// off by at most two units, one correction leaves a neighbour of the quotient, and
// from a neighbour, whose remainder is exact, the second rounds correctly
// (P. Markstein's theorem on division by a correctly rounded reciprocal, 1990).  A
// product with inv alone puts values beside the middle of two e4m3 numbers on the
// wrong side.  From kExactScale on, the remainder of every quotient that e4m3 does
// not round to 0 is exact: at least 2^-34 2^(-90 - 23) in its last place.
// Time, us, beside the product alone / the compiler's division: 16384 x 2560 bf16 55
// (54 / 55), 32768 x 1537 88 (83 / 95), 400000 x 63 115 (108 / 121).
constexpr float kExactScale = 0x1p-90f;
__device__ __forceinline__ float quotient(float y, float scale, float inv) {
    float q = y * inv;
    q = fmaf(fmaf(-q, scale, y), inv, q);
    return fmaf(fmaf(-q, scale, y), inv, q);
}

// the larger of two magnitudes, a NaN above everything (its bits are)
struct MaxAbs {
    __device__ __forceinline__ float operator()(float a, float b) const {
        const uint32_t i = __float_as_uint(a) & 0x7fffffffu, j = __float_as_uint(b) & 0x7fffffffu;
        return __uint_as_float(i > j ? i : j);
    }
};

// f over the row's R waves, or its L lanes; one barrier, tmp of the calls alternating
template <int R, int L, typename F> __device__ __forceinline__ float row_fold(float v, float *tmp, F f) {
    v = wave_fold<L>(v, f);
    if constexpr (R > 1) {
        if (threadIdx.x % 64 == 0) tmp[threadIdx.x / 64] = v;
        __syncthreads();
        v = tmp[0];
#pragma unroll
        for (int w = 1; w < R; ++w) v = f(v, tmp[w]);
    }
    return v;
}

// -------------------------------------------- V consecutive elements of a row
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

template <typename T, int V> struct Chunk;
template <> struct Chunk<bf16_t, 8> {
    u4 q;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t e) { q = __builtin_amdgcn_raw_buffer_load_b128(r, e * 2, 0, kStream); }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i % 2 ? (q[i / 2] & 0xffff0000u) : (q[i / 2] << 16));
    }
    static __device__ __forceinline__ void store(const float *v, rsrc_t r, uint32_t e) {
        u4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                   (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
        __builtin_amdgcn_raw_buffer_store_b128(q, r, e * 2, 0, kStream);
    }
};
template <> struct Chunk<bf16_t, 4> {
    u2 q;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t e) { q = __builtin_amdgcn_raw_buffer_load_b64(r, e * 2, 0, kStream); }
    __device__ __forceinline__ float get(int i) const {
        return __uint_as_float(i % 2 ? (q[i / 2] & 0xffff0000u) : (q[i / 2] << 16));
    }
    static __device__ __forceinline__ void store(const float *v, rsrc_t r, uint32_t e) {
        u2 q;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            q[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                   (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
        __builtin_amdgcn_raw_buffer_store_b64(q, r, e * 2, 0, kStream);
    }
};
template <> struct Chunk<float, 4> {
    u4 q;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t e) { q = __builtin_amdgcn_raw_buffer_load_b128(r, e * 4, 0, kStream); }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(q[i]); }
    static __device__ __forceinline__ void store(const float *v, rsrc_t r, uint32_t e) {
        const u4 q = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        __builtin_amdgcn_raw_buffer_store_b128(q, r, e * 4, 0, kStream);
    }
};
// the weight and its gradient beside eight bf16 values: two accesses of 16 bytes
template <> struct Chunk<float, 8> {
    Chunk<float, 4> h[2];
    __device__ __forceinline__ void load(rsrc_t r, uint32_t e) {
        h[0].load(r, e);
        h[1].load(r, e + 4);
    }
    __device__ __forceinline__ float get(int i) const { return h[i / 4].get(i % 4); }
    static __device__ __forceinline__ void store(const float *v, rsrc_t r, uint32_t e) {
        Chunk<float, 4>::store(v, r, e);
        Chunk<float, 4>::store(v + 4, r, e + 4);
    }
};
template <typename T> struct Chunk<T, 1> {
    typename Io<T>::raw q;
    __device__ __forceinline__ void load(rsrc_t r, uint32_t e) { q = Io<T>::template load<kStream>(r, e * sizeof(T), 0); }
    __device__ __forceinline__ float get(int) const { return Io<T>::f32(q); }
    static __device__ __forceinline__ void store(const float *v, rsrc_t r, uint32_t e) {
        Io<T>::template store<kStream>(v[0], r, e * sizeof(T), 0);
    }
};

template <int V> __device__ __forceinline__ void store_e4m3(const float *v, rsrc_t r, uint32_t e) {
    if constexpr (V == 8) {
        u2 q;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
            q[i] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], p, true));
        }
        __builtin_amdgcn_raw_buffer_store_b64(q, r, e, 0, kStream);
    } else if constexpr (V == 4) {
        const int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        __builtin_amdgcn_raw_buffer_store_b32(static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], p, true)), r, e,
                                              0, kStream);
    } else {
        __builtin_amdgcn_raw_buffer_store_b8(
            static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[0], 0, false) & 0xff), r, e, 0, kStream);
    }
}

// n rows of a (rows, dim) tensor with rows ld apart, from row `row` on: accesses
// past the last one's end read 0 and store nothing
template <typename T> __device__ __forceinline__ rsrc_t row_rsrc(const void *p, int64_t row, int64_t ld, int dim, int n = 1) {
    return make_rsrc(static_cast<const char *>(p) + row * ld * static_cast<int64_t>(sizeof(T)),
                     static_cast<uint32_t>(((n - 1) * ld + dim) * static_cast<int64_t>(sizeof(T))));
}
// an element index past every such range, in bytes too (rows that share a wave span under 2^29 bytes)
constexpr uint32_t kNoElem = 0x30000000u;
constexpr int64_t kMaxSharedLd = int64_t(1) << 24;

// ----------------------------------------------------------------- forward
// T: io dtype; S: the residual's; Q: 8-bit output.  A workgroup is R waves on
// one row, or (R = 1) four waves on a row each, or (L < 64) on 64 / L rows each:
// narrow rows, as of a norm per head, would leave most lanes idle.
template <typename T, typename S, bool Q, int V, int P, int R, int L>
__global__ __launch_bounds__(R == 1 ? 256 : R * 64) void norm_kernel(NormArgs p) {
    __shared__ float tmp[2][2][R];
    const int lane = threadIdx.x % 64;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int dim = static_cast<int>(p.dim);
    static_assert(L == 64 || (P == 1 && R == 1), "rows that share a wave");
    constexpr int G = 64 / L;                                        // rows of a wave
    constexpr int per_wg = (R == 1 ? 4 : 1) * G;
    const int sub = lane / L;
    const uint32_t e0 = static_cast<uint32_t>(((R == 1 ? 0 : w) * 64 + lane % L) * V);   // the lane's first element
    constexpr uint32_t step = R * 64 * V;
    const bool inside = L == 64 || static_cast<int>(e0) < dim;       // L = 64: past dim is past the descriptor
    const uint32_t ed = inside ? sub * static_cast<uint32_t>(dim) + e0 : kNoElem;
    const uint32_t ex = inside ? sub * static_cast<uint32_t>(p.ldx) + e0 : kNoElem;
    float wt[P][V];
    const rsrc_t rw = make_rsrc(p.weight, static_cast<uint32_t>(dim * 4));
#pragma unroll
    for (int c = 0; c < P; ++c) {
        Chunk<float, V> q;
        q.load(rw, e0 + c * step);
#pragma unroll
        for (int i = 0; i < V; ++i) wt[c][i] = q.get(i);
    }
    const float inv_dim = 1.0f / static_cast<float>(dim);
    int par = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_wg + (R == 1 ? w * G : 0); row < p.rows;
         row += static_cast<int64_t>(gridDim.x) * per_wg, par ^= 1) {
        const int n = L == 64 ? 1 : static_cast<int>(p.rows - row < G ? p.rows - row : G);
        Chunk<T, V> x[P];
        Chunk<S, V> res[P];
        const rsrc_t rx = row_rsrc<T>(p.x, row, p.ldx, dim, n);
#pragma unroll
        for (int c = 0; c < P; ++c) x[c].load(rx, ex + c * step);
        if (p.residual) {
            const rsrc_t rr = row_rsrc<S>(p.residual, row, p.dim, dim, n);
#pragma unroll
            for (int c = 0; c < P; ++c) res[c].load(rr, ed + c * step);
        }
        float v[P][V], ss = 0.0f;
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[c][i] = x[c].get(i);
                if (p.residual) v[c][i] += res[c].get(i);
                ss = fmaf(v[c][i], v[c][i], ss);
            }
        if (p.residual_out) {
            const rsrc_t ro = row_rsrc<S>(p.residual_out, row, p.dim, dim, n);
#pragma unroll
            for (int c = 0; c < P; ++c) Chunk<S, V>::store(v[c], ro, ed + c * step);
        }
        ss = row_fold<R, L>(ss, tmp[0][par], AddOp());
        const float rstd = 1.0f / sqrtf(fmaf(ss, inv_dim, p.eps));
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[c][i] = v[c][i] * rstd * wt[c][i];         // in the formula's order
                if constexpr (Q) m = MaxAbs()(m, v[c][i]);
            }
        if constexpr (Q) {
            m = row_fold<R, L>(m, tmp[1][par], MaxAbs());
            float scale = m / kE4m3Max;
            scale = scale < kMinScale ? kMinScale : scale;     // false for NaN, which stays
            if (lane % L == 0 && (R == 1 || w == 0) && sub < n) p.scale[row + sub] = scale;
            const rsrc_t ry = row_rsrc<uint8_t>(p.y, row, p.dim, dim, n);
            // a row of zeros or nearly so is raised by 2^64 first; finite values over an infinite scale are 0
            const float up = scale < kExactScale ? 0x1p64f : 1.0f, raised = scale * up, inv = 1.0f / raised;
            const float b = raised == __builtin_inff() ? 1.0f : raised;
#pragma unroll
            for (int c = 0; c < P; ++c) {
#pragma unroll
                for (int i = 0; i < V; ++i) v[c][i] = quotient(v[c][i] * up, b, inv);
                store_e4m3<V>(v[c], ry, ed + c * step);
            }
        } else {
            const rsrc_t ry = row_rsrc<T>(p.y, row, p.dim, dim, n);
#pragma unroll
            for (int c = 0; c < P; ++c) Chunk<T, V>::store(v[c], ry, ed + c * step);
        }
    }
}

// ---------------------------------------------------------------- gradient
// Workgroups as in the forward; a workgroup's sum of dy n over its rows is one
// row of `part`.
template <typename T, typename S, int V, int P, int R, int L>
__global__ __launch_bounds__(R == 1 ? 256 : R * 64) void norm_bwd_kernel(NormBwdArgs p) {
    constexpr int NW = R == 1 ? 4 : R;
    __shared__ float tmp[2][2][NW];
    __shared__ float sW[R == 1 ? NW : 1][R == 1 ? 64 * V * P : 1];
    const int lane = threadIdx.x % 64;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int dim = static_cast<int>(p.dim);
    static_assert(L == 64 || (P == 1 && R == 1), "rows that share a wave");
    constexpr int G = 64 / L;                                        // rows of a wave
    constexpr int per_wg = (R == 1 ? 4 : 1) * G;
    const int sub = lane / L;
    const uint32_t e0 = static_cast<uint32_t>(((R == 1 ? 0 : w) * 64 + lane % L) * V);   // the lane's first element
    constexpr uint32_t step = R * 64 * V;
    const bool inside = L == 64 || static_cast<int>(e0) < dim;       // L = 64: past dim is past the descriptor
    const uint32_t ed = inside ? sub * static_cast<uint32_t>(dim) + e0 : kNoElem;
    const uint32_t er = inside ? sub * static_cast<uint32_t>(p.ldr) + e0 : kNoElem;
    float wt[P][V], dw[P][V];
    const rsrc_t rw = make_rsrc(p.weight, static_cast<uint32_t>(dim * 4));
#pragma unroll
    for (int c = 0; c < P; ++c) {
        Chunk<float, V> q;
        q.load(rw, e0 + c * step);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            wt[c][i] = q.get(i);
            dw[c][i] = 0.0f;
        }
    }
    const float inv_dim = 1.0f / static_cast<float>(dim);
    int par = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * per_wg + (R == 1 ? w * G : 0); row < p.rows;
         row += static_cast<int64_t>(gridDim.x) * per_wg, par ^= 1) {
        const int n = L == 64 ? 1 : static_cast<int>(p.rows - row < G ? p.rows - row : G);
        Chunk<T, V> dy[P];
        Chunk<S, V> r[P], add[P];
        const rsrc_t rr = row_rsrc<S>(p.r, row, p.ldr, dim, n), rd = row_rsrc<T>(p.dy, row, p.dim, dim, n);
#pragma unroll
        for (int c = 0; c < P; ++c) r[c].load(rr, er + c * step);
#pragma unroll
        for (int c = 0; c < P; ++c) dy[c].load(rd, ed + c * step);
        if (p.dres_out) {
            const rsrc_t ra = row_rsrc<S>(p.dres_out, row, p.dim, dim, n);
#pragma unroll
            for (int c = 0; c < P; ++c) add[c].load(ra, ed + c * step);
        }
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = r[c].get(i);
                ss = fmaf(v, v, ss);
                dot = fmaf(v, wt[c][i] * dy[c].get(i), dot);
            }
        ss = row_fold<R, L>(ss, tmp[0][par], AddOp());
        dot = row_fold<R, L>(dot, tmp[1][par], AddOp());
        // a row past the last one has no part in dw, whatever eps
        const float rstd = L == 64 || sub < n ? 1.0f / sqrtf(fmaf(ss, inv_dim, p.eps)) : 0.0f;
        const float k = dot * inv_dim * rstd * rstd;           // mean(n w dy) rstd
        const rsrc_t wx = row_rsrc<T>(p.dx, row, p.dim, dim, n);
        const rsrc_t wr = p.dres ? row_rsrc<S>(p.dres, row, p.dim, dim, n) : make_rsrc(p.dx, 0u);
#pragma unroll
        for (int c = 0; c < P; ++c) {
            float o[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float g = dy[c].get(i), v = r[c].get(i);
                o[i] = rstd * fmaf(-v, k, wt[c][i] * g);
                if (p.dres_out) o[i] += add[c].get(i);
                dw[c][i] = fmaf(g, v * rstd, dw[c][i]);
            }
            Chunk<T, V>::store(o, wx, ed + c * step);
            if (p.dres) Chunk<S, V>::store(o, wr, ed + c * step);
        }
    }
    if constexpr (R == 1) {                            // the waves' sums, in wave and row order
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) sW[w][(c * V + i) * 64 + lane] = dw[c][i];
        __syncthreads();
        if (w > 0 || lane >= L) return;
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dw[c][i] = 0.0f;
                for (int u = 0; u < NW; ++u)
                    for (int q = 0; q < G; ++q) dw[c][i] += sW[u][(c * V + i) * 64 + q * L + lane];
            }
    }
    const rsrc_t rp = row_rsrc<float>(p.workspace, blockIdx.x, p.dim, dim);
#pragma unroll
    for (int c = 0; c < P; ++c) Chunk<float, V>::store(dw[c], rp, (inside ? e0 : kNoElem) + c * step);
}

__global__ __launch_bounds__(kSumThreads) void norm_dweight_kernel(const float *part, float *out, int64_t parts, int64_t dim) {
    column_sums(part, out, parts, dim);
}

// ------------------------------------------------------------------- host
// accesses of V elements stay aligned in every row (and end with it)
template <int V, typename T> bool wide(const void *p, int64_t ld) {
    return reinterpret_cast<uintptr_t>(p) % (V * sizeof(T)) == 0 && ld % V == 0;
}

// Workgroups: 16 of four waves per CU (2048 instead: 16384 x 2561 fp32 148 us
// against 143 us, 32768 x 2560 bf16 178 against 176 us).
constexpr int64_t kMaxGrid = 4096;
// Workgroups of the gradient, each with a partial sum of dw: few where a sum is
// long (with 1024, 16384 x 768 takes 37 + 5.5 us instead of 36 + 4, 2000 x 12001
// 115 us instead of 95), enough to fill the chip where it is short (100000 x 130:
// 50 us with 512, 36 us with 1024).
int64_t max_parts(int64_t dim) { return dim <= 256 ? 1024 : 512; }

template <typename T, typename S, bool Q, int V, int P, int R, int L = 64>
hipError_t launch_fwd(const NormArgs &a, hipStream_t s) {
    const int per_wg = (R == 1 ? 4 : 1) * (64 / L);
    const int64_t wgs = (a.rows + per_wg - 1) / per_wg;
    hipLaunchKernelGGL((norm_kernel<T, S, Q, V, P, R, L>), dim3(static_cast<unsigned>(wgs < kMaxGrid ? wgs : kMaxGrid)),
                       dim3(R == 1 ? 256 : R * 64), 0, s, a);
    return hipGetLastError();
}
int64_t parts_of(int64_t rows, int64_t dim, int per_wg) {
    const int64_t wgs = (rows + per_wg - 1) / per_wg;
    return wgs < max_parts(dim) ? wgs : max_parts(dim);
}
template <typename T, typename S, int V, int P, int R, int L = 64>
hipError_t launch_bwd(const NormBwdArgs &a, hipStream_t s) {
    const int parts = static_cast<int>(parts_of(a.rows, a.dim, (R == 1 ? 4 : 1) * (64 / L)));
    if (parts > 0)
        hipLaunchKernelGGL((norm_bwd_kernel<T, S, V, P, R, L>), dim3(parts), dim3(R == 1 ? 256 : R * 64), 0, s, a);
    hipLaunchKernelGGL(norm_dweight_kernel, dim3(static_cast<unsigned>((a.dim + kSumCols - 1) / kSumCols)),
                       dim3(kSumThreads), 0, s, static_cast<const float *>(a.workspace), a.dweight,
                       static_cast<int64_t>(parts), a.dim);
    return hipGetLastError();
}

// Rows of up to 32 V elements share a wave (200000 x 64 bf16: 19 us against 50 us
// with a wave each).
#define SSM_NARROW(CALL, V)                                                        \
    if (a.dim <= 8 * V) return CALL(V, 1, 1, 8);                                   \
    if (a.dim <= 16 * V) return CALL(V, 1, 1, 16);                                 \
    if (a.dim <= 32 * V) return CALL(V, 1, 1, 32)

// The chunks per lane and waves per row for a width, in units of 512 elements
// (V = 8 or 4) or 64 (V = 1).  Few waves to a row as far as the registers go, as
// waves that share one wait for each other at every reduction.  44M elements, us,
// aligned rows (bf16 / the same to 8 bits / fp32):
//   forward   1536 wide                  one wave 63 / 57 / 123   four 70 / 87 / 129
//             2048 wide                  one 62 / 57 / 121        four 66 / 62 / 122
//             2560 wide                  one 64 / 57 / 123        four 67 / 61 / 124
//             3584 wide                  one 65 / 59 / 122        four 64 / 58 / 124
//             4096 wide                  one 64 / 58 / 137        four 62 / 56 / 118
// 40M elements, us:
//             1537 wide, bf16            one 70         four 87    sixteen 110
//             2561 wide, bf16 / 8 bits   four 86 / 77   sixteen 81 / 92
//   gradient  1280 wide, bf16            one 46         four 81
//             5120 wide, bf16            four 52        sixteen 71
//             401 wide, bf16             one 66         four 208
//             2561 wide, fp32            four 91        sixteen 103
//             2048 wide, fp32            one 89         four 81
// Above 16384 wide sixteen waves do not hold a gradient's row: up to 92 registers
// are spilled, and 44M elements take 225 us (bf16, 32768 wide) instead of 72 (16384
// wide), in fp32 240 instead of 107.
#define SSM_FWD_PICK(CALL, V)                                                      \
    return units <= 1    ? CALL(V, 8 / V, 1)                                       \
           : units <= 2  ? CALL(V, 16 / V, 1)                                      \
           : units <= 3  ? CALL(V, 24 / V, 1)                                      \
           : units <= 4  ? CALL(V, 32 / V, 1)                                      \
           : units <= 5  ? CALL(V, 40 / V, 1)                                      \
           : units <= 8  ? CALL(V, 16 / V, 4)                                      \
           : units <= 12 ? CALL(V, 24 / V, 4)                                      \
           : units <= 16 ? CALL(V, 32 / V, 4)                                      \
           : units <= 32 ? CALL(V, 16 / V, 16)                                     \
                         : CALL(V, 32 / V, 16)
#define SSM_BWD_PICK(CALL, V)                                                      \
    return units <= 1    ? CALL(V, 8 / V, 1)                                       \
           : units <= 2  ? CALL(V, 16 / V, 1)                                      \
           : units <= 3  ? CALL(V, 24 / V, 1)                                      \
           : units <= 4  ? CALL(V, (V == 8 ? 32 : 8) / V, V == 8 ? 1 : 4)          \
           : units <= 8  ? CALL(V, 16 / V, 4)                                      \
           : units <= 16 ? CALL(V, 32 / V, 4)                                      \
           : units <= 32 ? CALL(V, 16 / V, 16)                                     \
                         : CALL(V, 32 / V, 16)
#define SSM_FWD_PICK1(CALL, Q)                                                     \
    return units <= 4     ? CALL(1, 4, 1)                                          \
           : units <= 8   ? CALL(1, 8, 1)                                          \
           : units <= 16  ? CALL(1, 16, 1)                                         \
           : units <= 32  ? CALL(1, 32, 1)                                         \
           : units <= 64  ? CALL(1, Q ? 16 : 4, Q ? 4 : 16)                        \
           : units <= 128 ? CALL(1, 8, 16)                                         \
           : units <= 256 ? CALL(1, 16, 16)                                        \
                          : CALL(1, 32, 16)
#define SSM_BWD_PICK1(CALL)                                                        \
    return units <= 4     ? CALL(1, 4, 1)                                          \
           : units <= 8   ? CALL(1, 8, 1)                                          \
           : units <= 16  ? CALL(1, 16, 1)                                         \
           : units <= 32  ? CALL(1, 8, 4)                                          \
           : units <= 64  ? CALL(1, 16, 4)                                         \
           : units <= 128 ? CALL(1, 8, 16)                                         \
           : units <= 256 ? CALL(1, 16, 16)                                        \
                          : CALL(1, 32, 16)

// 16 bytes of the widest tensor: the lanes of a store then fill whole lines (a row
// of fp32 written as two 16-byte halves per lane took 195 us instead of 179 us at
// 32768 x 2560)
template <typename T, typename S> constexpr int kVec = sizeof(T) == 4 || sizeof(S) == 4 ? 4 : 8;

// Whether accesses of V elements suit every tensor of a call.
template <typename T, typename S, int V> bool fits(const NormArgs &a) {
    return wide<V, T>(a.x, a.ldx) && wide<V, S>(a.residual, a.dim) && wide<V, S>(a.residual_out, a.dim) &&
           wide<4, float>(a.weight, a.dim) && (a.scale ? wide<V, uint8_t>(a.y, a.dim) : wide<V, T>(a.y, a.dim));
}
template <typename T, typename S, int V> bool fits(const NormBwdArgs &a) {
    return wide<V, T>(a.dy, a.dim) && wide<V, T>(a.dx, a.dim) && wide<V, S>(a.r, a.ldr) && wide<V, S>(a.dres_out, a.dim) &&
           wide<V, S>(a.dres, a.dim) && wide<4, float>(a.weight, a.dim);
}

template <typename T, typename S, bool Q, int V> hipError_t pick_fwd_v(const NormArgs &a, hipStream_t s) {
#define SSM_CALL(V, ...) (launch_fwd<T, S, Q, V, __VA_ARGS__>(a, s))
    if (a.ldx < kMaxSharedLd) {
        SSM_NARROW(SSM_CALL, V);
    }
    const int64_t units = (a.dim + (V == 1 ? 63 : 511)) / (V == 1 ? 64 : 512);
    if constexpr (V == 1)
        SSM_FWD_PICK1(SSM_CALL, Q);
    else
        SSM_FWD_PICK(SSM_CALL, V);
#undef SSM_CALL
}
template <typename T, typename S, int V> hipError_t pick_bwd_v(const NormBwdArgs &a, hipStream_t s) {
#define SSM_CALL(V, ...) (launch_bwd<T, S, V, __VA_ARGS__>(a, s))
    if (a.ldr < kMaxSharedLd) {
        SSM_NARROW(SSM_CALL, V);
    }
    const int64_t units = (a.dim + (V == 1 ? 63 : 511)) / (V == 1 ? 64 : 512);
    if constexpr (V == 1)
        SSM_BWD_PICK1(SSM_CALL);
    else
        SSM_BWD_PICK(SSM_CALL, V);
#undef SSM_CALL
}
template <typename T, typename S, bool Q> hipError_t pick_fwd(const NormArgs &a, hipStream_t s) {
    constexpr int W = kVec<T, S>;
    if (fits<T, S, W>(a)) return pick_fwd_v<T, S, Q, W>(a, s);
    if constexpr (W == 8)
        if (fits<T, S, 4>(a)) return pick_fwd_v<T, S, Q, 4>(a, s);
    return pick_fwd_v<T, S, Q, 1>(a, s);
}
template <typename T, typename S> hipError_t pick_bwd(const NormBwdArgs &a, hipStream_t s) {
    constexpr int W = kVec<T, S>;
    if (fits<T, S, W>(a)) return pick_bwd_v<T, S, W>(a, s);
    if constexpr (W == 8)
        if (fits<T, S, 4>(a)) return pick_bwd_v<T, S, 4>(a, s);
    return pick_bwd_v<T, S, 1>(a, s);
}
template <typename T, typename S> hipError_t pick_fwd_q(const NormArgs &a, hipStream_t s) {
    return a.scale ? pick_fwd<T, S, true>(a, s) : pick_fwd<T, S, false>(a, s);
}

}  // namespace

size_t norm_bwd_workspace(int64_t rows, int64_t dim) {
    return static_cast<size_t>(parts_of(rows, dim, 1) * ((dim + 3) / 4 * 4)) * 4;
}

hipError_t launch_add_rms_norm(const NormArgs &a, hipStream_t s) {
    if (!a.bf16) return pick_fwd_q<float, float>(a, s);
    return a.res_bf16 ? pick_fwd_q<bf16_t, bf16_t>(a, s) : pick_fwd_q<bf16_t, float>(a, s);
}

hipError_t launch_add_rms_norm_bwd(const NormBwdArgs &a, hipStream_t s) {
    if (!a.bf16) return pick_bwd<float, float>(a, s);
    return a.res_bf16 ? pick_bwd<bf16_t, bf16_t>(a, s) : pick_bwd<bf16_t, float>(a, s);
}

}  // namespace ssm
