// Group norm over channels-last tensors, with an activation and a gate, and its
// gradient.  x is (batch, rows, dim); a group is dim / groups neighbouring channels
// over all rows of one batch entry:
//     n = (x - mean) rstd,  a = n w + b,  y = act(a) SiLU(z)        (act: none or SiLU; z optional)
//     da = dy SiLU(z) act'(a),  dz = dy act(a) SiLU'(z),  dw = sum da n,  db = sum da
//     dx = rstd (w da - mean(w da) - n mean(w da n))                (means over the group)
//
// HBM-bound.  With one row to a statistic (a norm per token and head) a group lies
// in the registers of a few lanes, and every tensor is read once and written once.
// Otherwise a batch entry is cut into runs of rows; the first pass leaves partial
// sums of each run in the workspace, a small kernel adds them in a fixed order, and
// the second pass reads the inputs again.  The forward's sums of x and x^2 are
// taken in fp64, so that a mean far from 0 costs the variance nothing.
#include "ssm_device.h"
#include "ssm_kernels.h"
#include "wave_fold.h"

namespace ssm {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kRunGroups = 2048;        // workgroups that the runs of rows are cut for: eight per CU

// V consecutive io elements
template <typename T, int V> struct Vec;
template <> struct Vec<bf16_t, 8> { using raw = u4; };
template <> struct Vec<bf16_t, 4> { using raw = u2; };
template <> struct Vec<bf16_t, 2> { using raw = uint32_t; };
template <> struct Vec<bf16_t, 1> { using raw = uint16_t; };
template <> struct Vec<float, 4> { using raw = u4; };
template <> struct Vec<float, 2> { using raw = u2; };
template <> struct Vec<float, 1> { using raw = uint32_t; };
template <typename T, int V> __device__ __forceinline__ typename Vec<T, V>::raw load_vec(const T *p) {
    return *reinterpret_cast<const typename Vec<T, V>::raw *>(p);
}
__device__ __forceinline__ uint32_t word(u4 q, int i) { return q[i]; }
__device__ __forceinline__ uint32_t word(u2 q, int i) { return q[i]; }
__device__ __forceinline__ uint32_t word(uint32_t q, int) { return q; }
__device__ __forceinline__ uint32_t word(uint16_t q, int) { return q; }
template <typename T, int V> __device__ __forceinline__ void unpack(typename Vec<T, V>::raw q, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(word(q, i));
        else v[i] = __uint_as_float(i % 2 ? word(q, i / 2) & 0xffff0000u : word(q, i / 2) << 16);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
        typename Vec<T, V>::raw q;
        if constexpr (V == 1) q = __float_as_uint(v[0]);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) q[i] = __float_as_uint(v[i]);
        *reinterpret_cast<typename Vec<T, V>::raw *>(p) = q;
    } else if constexpr (V == 1) {
        *reinterpret_cast<uint16_t *>(p) = from_f32<bf16_t>(v[0]).bits;
    } else {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            u[i] = static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i]).bits) |
                   (static_cast<uint32_t>(from_f32<bf16_t>(v[2 * i + 1]).bits) << 16);
        typename Vec<T, V>::raw q;
        if constexpr (V == 2) q = u[0];
        else
#pragma unroll
            for (int i = 0; i < V / 2; ++i) q[i] = u[i];
        *reinterpret_cast<typename Vec<T, V>::raw *>(p) = q;
    }
}

__device__ __forceinline__ float sigmoid(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }
// SiLU and its slope
__device__ __forceinline__ float silu_slope(float v, float s) { return s * fmaf(v, 1.0f - s, 1.0f); }

// what y is of n, element by element
struct Affine {
    float w, b;
};
__device__ __forceinline__ float forward(float n, Affine p, bool act, bool gate, float z) {
    const float a = fmaf(n, p.w, p.b);
    float y = act ? silu(a) : a;
    return gate ? y * silu(z) : y;
}
// da, and dz into dz
__device__ __forceinline__ float backward(float n, float dy, Affine p, bool act, bool gate, float z, float &dz) {
    const float a = fmaf(n, p.w, p.b), s = sigmoid(a);
    float da = dy;
    if (gate) {
        const float sz = sigmoid(z);
        dz = dy * (act ? a * s : a) * silu_slope(z, sz);
        da = dy * (z * sz);
    }
    return act ? da * silu_slope(a, s) : da;
}

// ---------------------------------------------------- one row to a statistic
// L lanes share a group (P chunks of V channels each), 64 / L neighbouring groups a
// wave; a wave keeps its channels and walks the rows.
template <typename T, int V, int P, int L, bool BWD> __global__ __launch_bounds__(kThreads) void group_row_kernel(GroupNormBwdArgs b, float *part) {
    const GroupNormArgs &a = b.fwd;
    constexpr int GW = 64 / L;
    __shared__ float sW[BWD ? 4 : 1][BWD ? 2 * V * P : 1][BWD ? 64 : 1];
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int D = static_cast<int>(a.dim / a.groups);
    const int64_t nunit = (a.groups + GW - 1) / GW;
    const int64_t unit = blockIdx.x % nunit, first = blockIdx.x / nunit, step = gridDim.x / nunit;
    const int64_t group = unit * GW + lane / L;
    const int e0 = (lane % L) * V;
    bool in[P];
    Affine p[P][V];
    float dw[P][V], db[P][V];
#pragma unroll
    for (int c = 0; c < P; ++c) {
        const int e = e0 + c * L * V;
        in[c] = group < a.groups && e < D;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[c][i].w = a.weight && in[c] ? a.weight[group * D + e + i] : 1.0f;
            p[c][i].b = a.bias && in[c] ? a.bias[group * D + e + i] : 0.0f;
            dw[c][i] = db[c][i] = 0.0f;
        }
    }
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const float inv = 1.0f / static_cast<float>(D);
    using raw = typename Vec<T, V>::raw;
    for (int64_t row = first * 4 + w; row < a.batch; row += step * 4) {
        const T *const px = static_cast<const T *>(a.x) + row * a.ldx + group * D;
        const T *const pz = static_cast<const T *>(a.z) + row * a.ldz + group * D;
        const T *const pd = static_cast<const T *>(b.dy) + row * a.dim + group * D;
        raw rx[P], rz[P], rd[P];
#pragma unroll
        for (int c = 0; c < P; ++c) {
            const int e = e0 + c * L * V;
            rx[c] = rz[c] = rd[c] = raw{};
            if (in[c]) {
                rx[c] = load_vec<T, V>(px + e);
                if (gate) rz[c] = load_vec<T, V>(pz + e);
                if constexpr (BWD) rd[c] = load_vec<T, V>(pd + e);
            }
        }
        float x[P][V];
#pragma unroll
        for (int c = 0; c < P; ++c) unpack<T, V>(rx[c], x[c]);
        float mean, rstd;
        if constexpr (BWD) {
            const bool any = group < a.groups;
            mean = any ? a.mean[row * a.groups + group] : 0.0f;
            rstd = any ? a.rstd[row * a.groups + group] : 0.0f;
        } else {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < P; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) s += x[c][i];
            mean = wave_fold<L>(s, AddOp()) * inv;
            s = 0.0f;
#pragma unroll
            for (int c = 0; c < P; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = in[c] ? x[c][i] - mean : 0.0f;
                    s = fmaf(d, d, s);
                }
            rstd = 1.0f / sqrtf(fmaf(wave_fold<L>(s, AddOp()), inv, a.eps));
            if (lane % L == 0 && group < a.groups) {
                if (a.mean) a.mean[row * a.groups + group] = mean;
                if (a.rstd) a.rstd[row * a.groups + group] = rstd;
            }
        }
        float out[P][V], dz[P][V], n[P][V];
        float m1 = 0.0f, m2 = 0.0f;
#pragma unroll
        for (int c = 0; c < P; ++c) {
            float z[V], dy[V];
            unpack<T, V>(rz[c], z);
            unpack<T, V>(rd[c], dy);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[c][i] = (x[c][i] - mean) * rstd;
                if constexpr (BWD) {
                    const float da = in[c] ? backward(n[c][i], dy[i], p[c][i], act, gate, z[i], dz[c][i]) : 0.0f;
                    out[c][i] = da * p[c][i].w;
                    dw[c][i] = in[c] ? fmaf(da, n[c][i], dw[c][i]) : 0.0f;
                    db[c][i] += da;
                    m1 += out[c][i];
                    m2 = in[c] ? fmaf(out[c][i], n[c][i], m2) : m2;
                } else {
                    out[c][i] = forward(n[c][i], p[c][i], act, gate, z[i]);
                }
            }
        }
        if constexpr (BWD) {
            m1 = wave_fold<L>(m1, AddOp()) * inv;
            m2 = wave_fold<L>(m2, AddOp()) * inv;
#pragma unroll
            for (int c = 0; c < P; ++c)
#pragma unroll
                for (int i = 0; i < V; ++i) out[c][i] = rstd * (out[c][i] - fmaf(n[c][i], m2, m1));
        }
        T *const po = static_cast<T *>(BWD ? b.dx : a.y) + row * a.dim + group * D;
        T *const pzo = static_cast<T *>(b.dz) + row * a.dim + group * D;
#pragma unroll
        for (int c = 0; c < P; ++c)
            if (in[c]) {
                store_vec<T, V>(po + e0 + c * L * V, out[c]);
                if constexpr (BWD)
                    if (gate) store_vec<T, V>(pzo + e0 + c * L * V, dz[c]);
            }
    }
    if constexpr (BWD) {                                   // the waves' sums, in wave order
#pragma unroll
        for (int c = 0; c < P; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sW[w][2 * (c * V + i)][lane] = dw[c][i];
                sW[w][2 * (c * V + i) + 1][lane] = db[c][i];
            }
        __syncthreads();
        if (w == 0) {
            float *const row = part + first * 2 * a.dim + group * D;
#pragma unroll
            for (int c = 0; c < P; ++c)
                if (in[c])
#pragma unroll
                    for (int i = 0; i < V; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int o = 2 * (c * V + i) + h;
                            row[h * a.dim + e0 + c * L * V + i] = (sW[0][o][lane] + sW[1][o][lane]) + (sW[2][o][lane] + sW[3][o][lane]);
                        }
        }
    }
}

// ------------------------------------------------------ many rows to a statistic
// A block is up to 256 vectors of V channels of a row (whole groups, or a part of
// one); a workgroup takes one run of rows of one block.
struct Runs {
    int64_t runs, per;            // of a batch entry; rows of a run
    int64_t blocks;               // of a row
    int bc;                       // channels of a block
    int per_group;                // blocks of a group where one is wider than a block, else 1
    int64_t total;                // workgroups' worth of work
};
// channels of a block: as many whole groups as 256 lanes hold, or an even part of a group
Runs runs_of(int64_t batch, int64_t rows, int64_t dim, int64_t groups, int V) {
    const int64_t D = dim / groups, most = static_cast<int64_t>(kThreads) * V;
    Runs r{};
    if (D <= most) {
        r.bc = static_cast<int>(most / D * D < dim ? most / D * D : dim);
        r.per_group = 1;
        r.blocks = (dim + r.bc - 1) / r.bc;
    } else {
        r.per_group = static_cast<int>((D + most - 1) / most);
        r.bc = static_cast<int>(most);
        r.blocks = groups * r.per_group;
    }
    const int64_t lanes = (r.bc + V - 1) / V, ty = kThreads / lanes;
    int64_t n = kRunGroups / (batch * r.blocks > 0 ? batch * r.blocks : 1);
    const int64_t most_runs = (rows + 4 * ty - 1) / (4 * ty);
    n = n < 1 ? 1 : (n > most_runs ? most_runs : n);
    r.per = (rows + n - 1) / n;
    r.runs = r.per > 0 ? (rows + r.per - 1) / r.per : 0;
    r.total = batch * r.runs * r.blocks;
    return r;
}
// where a workgroup's item lies and what a thread has of it
struct Item {
    int64_t n, run, block, row0, row1;
    int lanes, ty_count, tx, ty, ch;       // lanes of a row, rows at a time, the thread's place, its first channel
    int64_t group;                         // of the thread's channels
    bool in;
};
template <int V> __device__ __forceinline__ Item item_of(const GroupNormArgs &a, const Runs &r, int64_t id) {
    Item t;
    t.block = id % r.blocks;
    t.run = id / r.blocks % r.runs;
    t.n = id / r.blocks / r.runs;
    t.row0 = t.run * r.per;
    t.row1 = t.row0 + r.per < a.rows ? t.row0 + r.per : a.rows;
    const int64_t D = a.dim / a.groups;
    int64_t c0 = t.block * r.bc, c1 = c0 + r.bc < a.dim ? c0 + r.bc : a.dim;
    if (r.per_group > 1) {
        const int64_t g = t.block / r.per_group;
        c0 = g * D + t.block % r.per_group * r.bc;
        c1 = c0 + r.bc < (g + 1) * D ? c0 + r.bc : (g + 1) * D;
    }
    t.lanes = static_cast<int>((c1 - c0) / V);
    t.ty_count = kThreads / t.lanes;
    t.tx = threadIdx.x % t.lanes;
    t.ty = threadIdx.x / t.lanes;
    t.in = t.ty < t.ty_count;
    t.ch = static_cast<int>(c0) + t.tx * V;
    t.group = t.ch / D;
    return t;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// sums of x and x^2 of each run and group (part of a group): part[(n, run), block's groups]
template <typename T, int V> __global__ __launch_bounds__(kThreads) void group_stats_kernel(GroupNormArgs a, Runs r, double *part) {
    __shared__ double s1[kThreads], s2[kThreads];
    const int lane = threadIdx.x % 64, w = threadIdx.x / 64;
    const int64_t slots = a.groups * r.per_group;
    const int D = static_cast<int>(a.dim / a.groups);
    for (int64_t id = blockIdx.x; id < r.total; id += gridDim.x) {
        const Item t = item_of<V>(a, r, id);
        double u = 0.0, v = 0.0;
        if (t.in) {
            const T *const p = static_cast<const T *>(a.x) + t.n * a.rows * a.ldx + t.ch;
#pragma unroll 4
            for (int64_t row = t.row0 + t.ty; row < t.row1; row += t.ty_count) {
                float x[V];
                unpack<T, V>(load_vec<T, V>(p + row * a.ldx), x);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const double d = x[i];
                    u += d;
                    v = fma(d, d, v);
                }
            }
        }
        __syncthreads();
        s1[threadIdx.x] = u;
        s2[threadIdx.x] = v;
        __syncthreads();
        // a wave per group of the block: its lanes of every row of threads
        const int dv = r.per_group > 1 ? t.lanes : D / V, ngr = t.lanes / dv;
        for (int q = w; q < ngr; q += 4) {
            double x = 0.0, y = 0.0;
            for (int e = lane; e < dv * t.ty_count; e += 64) {
                const int o = e / dv * t.lanes + q * dv + e % dv;
                x += s1[o];
                y += s2[o];
            }
            x = wave_sum(x);
            y = wave_sum(y);
            if (lane == 0) {
                const int64_t slot = r.per_group > 1 ? t.block : t.block * (r.bc / D) + q;
                double *const o = part + 2 * ((t.n * r.runs + t.run) * slots + slot);
                o[0] = x;
                o[1] = y;
            }
        }
    }
}
// mean and rstd of a group, a wave each
__global__ __launch_bounds__(kThreads) void group_stats_end_kernel(GroupNormArgs a, Runs r, const double *part, float *mean, float *rstd) {
    const int lane = threadIdx.x % 64;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(a.dim / a.groups));
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64; id < a.batch * a.groups; id += gridDim.x * 4ll) {
        const int64_t n = id / a.groups, g = id % a.groups;
        double x = 0.0, y = 0.0;
        for (int64_t e = lane; e < r.runs * r.per_group; e += 64) {
            const double *const o = part + 2 * (((n * r.runs + e / r.per_group) * a.groups + g) * r.per_group + e % r.per_group);
            x += o[0];
            y += o[1];
        }
        x = wave_sum(x) * inv;
        y = wave_sum(y) * inv - x * x;
        if (lane == 0) {
            const float rs = static_cast<float>(1.0 / sqrt((y < 0.0 ? 0.0 : y) + static_cast<double>(a.eps)));
            mean[id] = static_cast<float>(x);
            rstd[id] = rs;
            if (a.mean && a.mean != mean) a.mean[id] = static_cast<float>(x);
            if (a.rstd && a.rstd != rstd) a.rstd[id] = rs;
        }
    }
}
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void group_apply_kernel(GroupNormArgs a, Runs r, const float *mean, const float *rstd) {
    const bool act = a.silu != 0, gate = a.z != nullptr;
    for (int64_t id = blockIdx.x; id < r.total; id += gridDim.x) {
        const Item t = item_of<V>(a, r, id);
        if (!t.in) continue;
        Affine p[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = {a.weight ? a.weight[t.ch + i] : 1.0f, a.bias ? a.bias[t.ch + i] : 0.0f};
        const float m = mean[t.n * a.groups + t.group], s = rstd[t.n * a.groups + t.group];
        const T *const px = static_cast<const T *>(a.x) + t.n * a.rows * a.ldx + t.ch;
        const T *const pz = static_cast<const T *>(a.z) + t.n * a.rows * a.ldz + t.ch;
        T *const py = static_cast<T *>(a.y) + t.n * a.rows * a.dim + t.ch;
#pragma unroll 4
        for (int64_t row = t.row0 + t.ty; row < t.row1; row += t.ty_count) {
            float x[V], z[V] = {};
            unpack<T, V>(load_vec<T, V>(px + row * a.ldx), x);
            if (gate) unpack<T, V>(load_vec<T, V>(pz + row * a.ldz), z);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = forward((x[i] - m) * s, p[i], act, gate, z[i]);
            store_vec<T, V>(py + row * a.dim, x);
        }
    }
}

// the gradient's sums of da and da n of each run and channel: part[(n, run), 2, dim]
template <typename T, int V> __global__ __launch_bounds__(kThreads) void group_sums_kernel(GroupNormBwdArgs b, Runs r, float *part) {
    const GroupNormArgs &a = b.fwd;
    __shared__ float sA[kThreads][V + 1], sB[kThreads][V + 1];
    const bool act = a.silu != 0, gate = a.z != nullptr;
    for (int64_t id = blockIdx.x; id < r.total; id += gridDim.x) {
        const Item t = item_of<V>(a, r, id);
        float u[V] = {}, v[V] = {};
        if (t.in) {
            Affine p[V];
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = {a.weight ? a.weight[t.ch + i] : 1.0f, a.bias ? a.bias[t.ch + i] : 0.0f};
            const float m = a.mean[t.n * a.groups + t.group], s = a.rstd[t.n * a.groups + t.group];
            const T *const px = static_cast<const T *>(a.x) + t.n * a.rows * a.ldx + t.ch;
            const T *const pz = static_cast<const T *>(a.z) + t.n * a.rows * a.ldz + t.ch;
            const T *const pd = static_cast<const T *>(b.dy) + t.n * a.rows * a.dim + t.ch;
#pragma unroll 4
            for (int64_t row = t.row0 + t.ty; row < t.row1; row += t.ty_count) {
                float x[V], z[V] = {}, d[V], dz = 0.0f;
                unpack<T, V>(load_vec<T, V>(px + row * a.ldx), x);
                unpack<T, V>(load_vec<T, V>(pd + row * a.dim), d);
                if (gate) unpack<T, V>(load_vec<T, V>(pz + row * a.ldz), z);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float n = (x[i] - m) * s, da = backward(n, d[i], p[i], act, gate, z[i], dz);
                    u[i] += da;
                    v[i] = fmaf(da, n, v[i]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sA[threadIdx.x][i] = u[i];
            sB[threadIdx.x][i] = v[i];
        }
        __syncthreads();
        float *const o = part + (t.n * r.runs + t.run) * 2 * a.dim + (t.ch - t.tx * V);
        for (int c = threadIdx.x; c < t.lanes * V; c += kThreads) {
            float x = 0.0f, y = 0.0f;
            for (int q = 0; q < t.ty_count; ++q) {
                x += sA[q * t.lanes + c / V][c % V];
                y += sB[q * t.lanes + c / V][c % V];
            }
            o[c] = x;
            o[a.dim + c] = y;
        }
    }
}
// mean(w da) and mean(w da n) of a group, a wave each
__global__ __launch_bounds__(kThreads) void group_sums_end_kernel(GroupNormArgs a, int64_t runs, const float *part, float *coef) {
    const int lane = threadIdx.x % 64;
    const int64_t D = a.dim / a.groups;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(D));
    for (int64_t id = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64; id < a.batch * a.groups; id += gridDim.x * 4ll) {
        const int64_t n = id / a.groups, g = id % a.groups;
        double x = 0.0, y = 0.0;
        for (int64_t e = lane; e < runs * D; e += 64) {
            const int64_t c = g * D + e % D;
            const float *const o = part + (n * runs + e / D) * 2 * a.dim + c;
            const double wc = a.weight ? a.weight[c] : 1.0f;
            x += wc * o[0];
            y += wc * o[a.dim];
        }
        x = wave_sum(x) * inv;
        y = wave_sum(y) * inv;
        if (lane == 0) {
            coef[2 * id] = static_cast<float>(x);
            coef[2 * id + 1] = static_cast<float>(y);
        }
    }
}
template <typename T, int V> __global__ __launch_bounds__(kThreads) void group_grad_kernel(GroupNormBwdArgs b, Runs r, const float *coef) {
    const GroupNormArgs &a = b.fwd;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    for (int64_t id = blockIdx.x; id < r.total; id += gridDim.x) {
        const Item t = item_of<V>(a, r, id);
        if (!t.in) continue;
        Affine p[V];
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = {a.weight ? a.weight[t.ch + i] : 1.0f, a.bias ? a.bias[t.ch + i] : 0.0f};
        const int64_t ng = t.n * a.groups + t.group;
        const float m = a.mean[ng], s = a.rstd[ng], m1 = coef[2 * ng], m2 = coef[2 * ng + 1];
        const int64_t row = t.n * a.rows;
        const T *const px = static_cast<const T *>(a.x) + row * a.ldx + t.ch, *const pz = static_cast<const T *>(a.z) + row * a.ldz + t.ch;
        const T *const pd = static_cast<const T *>(b.dy) + row * a.dim + t.ch;
        T *const po = static_cast<T *>(b.dx) + row * a.dim + t.ch, *const pzo = static_cast<T *>(b.dz) + row * a.dim + t.ch;
#pragma unroll 4
        for (int64_t q = t.row0 + t.ty; q < t.row1; q += t.ty_count) {
            float x[V], z[V] = {}, d[V], dz[V];
            unpack<T, V>(load_vec<T, V>(px + q * a.ldx), x);
            unpack<T, V>(load_vec<T, V>(pd + q * a.dim), d);
            if (gate) unpack<T, V>(load_vec<T, V>(pz + q * a.ldz), z);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = (x[i] - m) * s, da = backward(n, d[i], p[i], act, gate, z[i], dz[i]);
                x[i] = s * (da * p[i].w - fmaf(n, m2, m1));
            }
            store_vec<T, V>(po + q * a.dim, x);
            if (gate) store_vec<T, V>(pzo + q * a.dim, dz);
        }
    }
}
// dweight and dbias from (rows, 2, dim) partial sums (da first, or da n first), in a
// fixed order: 16 columns to a workgroup, 64 stripes of rows
__global__ __launch_bounds__(1024) void group_params_kernel(const float *part, float *first, float *second, int64_t rows, int64_t dim) {
    __shared__ float sums[64][17];
    const int col = threadIdx.x % 16, stripe = threadIdx.x / 16;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 16 + col;
    float s = 0.0f;
    if (d < 2 * dim) {
#pragma unroll 8
        for (int64_t r = stripe; r < rows; r += 64) s += part[r * 2 * dim + d];
    }
    sums[stripe][col] = s;
    __syncthreads();
    const int w = threadIdx.x / 64, lane = threadIdx.x % 64;
    s = wave_fold(sums[lane][w], AddOp());
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 16 + w;
    if (lane == 0 && o < 2 * dim) {
        float *const to = o < dim ? first : second;
        if (to) to[o < dim ? o : o - dim] = s;
    }
}

// ------------------------------------------------------------------- dispatch
constexpr int64_t kRowWorkgroups = 2048;
size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
bool at(const void *p, int64_t bytes) { return !p || reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// elements of the widest access that the group, the strides and the addresses allow
int width(const GroupNormBwdArgs &b) {
    const GroupNormArgs &a = b.fwd;
    const int64_t es = a.bf16 ? 2 : 4, D = a.dim / a.groups;
    for (int v = a.bf16 ? 8 : 4; v > 1; v /= 2) {
        const int64_t n = es * v;
        if (D % v == 0 && a.ldx % v == 0 && (!a.z || a.ldz % v == 0) && at(a.x, n) && at(a.z, n) && at(a.y, n) && at(b.dy, n) &&
            at(b.dx, n) && at(b.dz, n))
            return v;
    }
    return 1;
}
// Whether a group fits the registers of a wave at every width that may be chosen
// for it (the workspace's size does not know the addresses).
constexpr int kMaxChunks = 4;
bool row_form(int64_t rows, int64_t dim, int64_t groups, int v) { return rows == 1 && dim / groups <= 64 * v * kMaxChunks; }
int64_t row_first(int64_t batch, int64_t units) {          // workgroups that share a unit's rows
    const int64_t most = (batch + 3) / 4, n = kRowWorkgroups / units > 0 ? kRowWorkgroups / units : 1;
    return n < most ? n : most;
}

template <typename T, int V, int P, int L, bool BWD> hipError_t run_rows(const GroupNormBwdArgs &b, hipStream_t s) {
    const GroupNormArgs &a = b.fwd;
    constexpr int GW = 64 / L;
    const int64_t units = (a.groups + GW - 1) / GW, first = row_first(a.batch, units);
    float *const part = static_cast<float *>(a.workspace);
    hipLaunchKernelGGL((group_row_kernel<T, V, P, L, BWD>), dim3(static_cast<unsigned>(units * first)), dim3(kThreads), 0, s, b, part);
    if (hipError_t e = hipGetLastError()) return e;
    if (!BWD || (!b.dweight && !b.dbias)) return hipSuccess;
    hipLaunchKernelGGL(group_params_kernel, dim3(static_cast<unsigned>((2 * a.dim + 15) / 16)), dim3(1024), 0, s, part, b.dweight, b.dbias,
                       first, a.dim);
    return hipGetLastError();
}
template <typename T, int V, bool BWD> hipError_t run_rows_of(const GroupNormBwdArgs &b, hipStream_t s) {
    const int64_t n = (b.fwd.dim / b.fwd.groups + V - 1) / V;          // lanes that a group needs
    if (n <= 8) return run_rows<T, V, 1, 8, BWD>(b, s);
    if (n <= 16) return run_rows<T, V, 1, 16, BWD>(b, s);
    if (n <= 32) return run_rows<T, V, 1, 32, BWD>(b, s);
    if (n <= 64) return run_rows<T, V, 1, 64, BWD>(b, s);
    if (n <= 128) return run_rows<T, V, 2, 64, BWD>(b, s);
    return run_rows<T, V, 4, 64, BWD>(b, s);
}
unsigned grid_of(int64_t items) { return static_cast<unsigned>(items < (1 << 20) ? items : (1 << 20)); }

template <typename T, int V> hipError_t run_fwd(const GroupNormArgs &a, hipStream_t s) {
    if (row_form(a.rows, a.dim, a.groups, V)) {
        GroupNormBwdArgs b{};
        b.fwd = a;
        return run_rows_of<T, V, false>(b, s);
    }
    const Runs r = runs_of(a.batch, a.rows, a.dim, a.groups, V);
    char *const ws = static_cast<char *>(a.workspace);
    const size_t ng = static_cast<size_t>(a.batch * a.groups);
    float *const mean = reinterpret_cast<float *>(ws), *const rstd = reinterpret_cast<float *>(ws + align256(ng * 4));
    double *const part = reinterpret_cast<double *>(ws + 2 * align256(ng * 4));
    hipLaunchKernelGGL((group_stats_kernel<T, V>), dim3(grid_of(r.total)), dim3(kThreads), 0, s, a, r, part);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL(group_stats_end_kernel, dim3(grid_of((a.batch * a.groups + 3) / 4)), dim3(kThreads), 0, s, a, r, part, mean, rstd);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((group_apply_kernel<T, V>), dim3(grid_of(r.total)), dim3(kThreads), 0, s, a, r, mean, rstd);
    return hipGetLastError();
}
template <typename T, int V> hipError_t run_bwd(const GroupNormBwdArgs &b, hipStream_t s) {
    const GroupNormArgs &a = b.fwd;
    if (row_form(a.rows, a.dim, a.groups, V)) return run_rows_of<T, V, true>(b, s);
    const Runs r = runs_of(a.batch, a.rows, a.dim, a.groups, V);
    char *const ws = static_cast<char *>(a.workspace);
    float *const coef = reinterpret_cast<float *>(ws), *const part = reinterpret_cast<float *>(ws + align256(a.batch * a.groups * 8));
    hipLaunchKernelGGL((group_sums_kernel<T, V>), dim3(grid_of(r.total)), dim3(kThreads), 0, s, b, r, part);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL(group_sums_end_kernel, dim3(grid_of((a.batch * a.groups + 3) / 4)), dim3(kThreads), 0, s, a, r.runs, part, coef);
    if (hipError_t e = hipGetLastError()) return e;
    if (b.dweight || b.dbias) {
        hipLaunchKernelGGL(group_params_kernel, dim3(static_cast<unsigned>((2 * a.dim + 15) / 16)), dim3(1024), 0, s, part, b.dbias, b.dweight,
                           a.batch * r.runs, a.dim);
        if (hipError_t e = hipGetLastError()) return e;
    }
    hipLaunchKernelGGL((group_grad_kernel<T, V>), dim3(grid_of(r.total)), dim3(kThreads), 0, s, b, r, coef);
    return hipGetLastError();
}

}  // namespace

// The largest over the widths that a call may choose.
size_t group_norm_workspace(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    size_t most = 0;
    const size_t ng = static_cast<size_t>(batch * groups);
    for (int v = 1; v <= 8; v *= 2) {
        if (row_form(rows, dim, groups, v)) continue;
        const Runs r = runs_of(batch, rows, dim, groups, v);
        const size_t n = 2 * align256(ng * 4) + align256(static_cast<size_t>(batch * r.runs * groups * r.per_group) * 16);
        most = n > most ? n : most;
    }
    return most;
}
size_t group_norm_bwd_workspace(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    size_t most = 0;
    for (int v = 1; v <= 8; v *= 2) {
        size_t n;
        if (row_form(rows, dim, groups, v)) {
            n = static_cast<size_t>(row_first(batch, (groups + 7) / 8)) * 2 * dim * 4;      // at most 8 groups to a wave
        } else {
            const Runs r = runs_of(batch, rows, dim, groups, v);
            n = align256(static_cast<size_t>(batch * groups) * 8) + static_cast<size_t>(batch * r.runs) * 2 * dim * 4;
        }
        most = n > most ? n : most;
    }
    return align256(most);
}

hipError_t launch_group_norm(const GroupNormArgs &a, hipStream_t s) {
    GroupNormBwdArgs b{};
    b.fwd = a;
    switch (width(b)) {
    case 8: return run_fwd<bf16_t, 8>(a, s);
    case 4: return a.bf16 ? run_fwd<bf16_t, 4>(a, s) : run_fwd<float, 4>(a, s);
    case 2: return a.bf16 ? run_fwd<bf16_t, 2>(a, s) : run_fwd<float, 2>(a, s);
    default: return a.bf16 ? run_fwd<bf16_t, 1>(a, s) : run_fwd<float, 1>(a, s);
    }
}
hipError_t launch_group_norm_bwd(const GroupNormBwdArgs &b, hipStream_t s) {
    if (b.fwd.batch == 0 || b.fwd.rows == 0) {             // sums of nothing
        hipLaunchKernelGGL(group_params_kernel, dim3(static_cast<unsigned>((2 * b.fwd.dim + 15) / 16)), dim3(1024), 0, s, nullptr, b.dweight,
                           b.dbias, 0, b.fwd.dim);
        return hipGetLastError();
    }
    switch (width(b)) {
    case 8: return run_bwd<bf16_t, 8>(b, s);
    case 4: return b.fwd.bf16 ? run_bwd<bf16_t, 4>(b, s) : run_bwd<float, 4>(b, s);
    case 2: return b.fwd.bf16 ? run_bwd<bf16_t, 2>(b, s) : run_bwd<float, 2>(b, s);
    default: return b.fwd.bf16 ? run_bwd<bf16_t, 1>(b, s) : run_bwd<float, 1>(b, s);
    }
}

}  // namespace ssm
