// Group norm over channels-last tensors, with an activation and a gate, and its
// gradient.  x is (batch, rows, dim); a group is dim / groups neighbouring channels
// over all rows of one batch entry:
//     n = (x - mean) rstd,  a = n w + b,  y = act(a) SiLU(z)        (act: none or SiLU; z optional)
//     da = dy SiLU(z) act'(a),  dz = dy act(a) SiLU'(z),  dw = sum da n,  db = sum da
//     dx = rstd (w da - mean(w da) - n mean(w da n))                (means over the group)
//
// HBM-bound.  With one row to a statistic (a norm per token and head) a group lies
// in the registers of a few lanes, and every tensor is read once and written once.
// Otherwise, where a few groups of a batch entry fit a workgroup's registers, it keeps
// them there over both passes.  Else a batch entry is cut into runs of rows; the
// first pass leaves each run's sums in the workspace, and the second adds them up, in a
// fixed order, and reads the inputs again.
//
// Measured (a copy: 5.6 TB/s): 16384 tokens of 40 heads of 128, bf16 with a gate, 503 MB 103 us
// (4.9 TB/s; 114 without the next row's loads ahead), its gradient at 12 heads 252 MB 53 us; 16 maps of
// 8192 x 512 27 us for the sums and 59 for the second pass (268 MB); 196 x 96 fp32 in one launch 7 us, in
// three 14.
#include "ssm_device.h"
#include "ssm_kernels.h"
#include "wave_fold.h"

#include <type_traits>

namespace ssm {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

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
        __builtin_nontemporal_store(q, reinterpret_cast<typename Vec<T, V>::raw *>(p));
    } else if constexpr (V == 1) {
        *reinterpret_cast<uint16_t *>(p) = from_f32<bf16_t>(v[0]).bits;
    } else {
        uint32_t u[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            u[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{v[2 * i], v[2 * i + 1]}, bf2));
        typename Vec<T, V>::raw q;
        if constexpr (V == 2) q = u[0];
        else
#pragma unroll
            for (int i = 0; i < V / 2; ++i) q[i] = u[i];
        __builtin_nontemporal_store(q, reinterpret_cast<typename Vec<T, V>::raw *>(p));
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
    struct Row {
        raw x[P], z[P], d[P];
    } next;
    auto load = [&](int64_t row) {
        const T *const px = static_cast<const T *>(a.x) + row * a.ldx + group * D;
        const T *const pz = static_cast<const T *>(a.z) + row * a.ldz + group * D;
        const T *const pd = static_cast<const T *>(b.dy) + row * a.dim + group * D;
#pragma unroll
        for (int c = 0; c < P; ++c) {
            const int e = e0 + c * L * V;
            next.x[c] = next.z[c] = next.d[c] = raw{};
            if (in[c]) {
                next.x[c] = load_vec<T, V>(px + e);
                if (gate) next.z[c] = load_vec<T, V>(pz + e);
                if constexpr (BWD) next.d[c] = load_vec<T, V>(pd + e);
            }
        }
    };
    if (first * 4 + w < a.batch) load(first * 4 + w);
    for (int64_t row = first * 4 + w; row < a.batch; row += step * 4) {
        raw rx[P], rz[P], rd[P];
#pragma unroll
        for (int c = 0; c < P; ++c) {
            rx[c] = next.x[c];
            rz[c] = next.z[c];
            rd[c] = next.d[c];
        }
        if (row + step * 4 < a.batch) load(row + step * 4);
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
            rstd = rsqrtf(fmaf(wave_fold<L>(s, AddOp()), inv, a.eps));
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
// Runs are cut for as many workgroups as the CUs hold at once: four of 8 waves a CU in 64
// registers a lane, two in the 128 that the gradient of wide vectors needs.
constexpr int kRunGroups = 1024;
constexpr int grad_waves(int V) { return V > 2 ? 4 : 8; }
constexpr int grad_groups(int V) { return 128 * grad_waves(V); }
constexpr int kRunThreads = 512, kRunWaves = kRunThreads / 64, kLanes = 256;
// The gradient's sums over rows: a thread adds at most kSumRows rows in fp32 before a sum moves
// on, into fp64 where it is a group's and where threads, runs and entries meet, into a second fp32
// sum of at most kSumRows where it is a channel's: one-signed terms lose 2 kSumRows U at most, not U per row.
constexpr int kSumRows = 128;
struct Runs {
    int64_t per;                  // rows of a run
    int runs;                     // of a batch entry
    int blocks;                   // of a row
    int bc;                       // channels of a block
    int per_group;                // blocks of a group where one is wider than a block, else 1
    int D;                        // channels of a group
    bool whole;                   // a run is a whole batch entry, and fits the workgroup's registers
    int64_t fold;                 // batch entries whose channel sums a workgroup of the gradient adds up
};
// Whole entries: a thread holds up to kHeld vectors of x (and z), the gradient half as
// many (beside dy's, and the sums), and a block is the fewest groups that are eight
// vectors wide (128 bytes at full width: a cache line) and, of few rows, give every thread one.
constexpr int kHeld = 8, kHeldGrad = 4;
constexpr int64_t kAnyRows = int64_t(1) << 40, kMostGradRows = kSumRows * kSumRows;
// most_rows: the rows that a thread may take of a run.
Runs runs_of(int64_t batch, int64_t rows, int64_t dim, int64_t groups, int V, int held, int target, int64_t most_rows) {
    const int D = static_cast<int>(dim / groups), most = kLanes * V;
    Runs r{};
    r.D = D;
    r.per_group = 1;
    const int64_t lanes1 = (D + V - 1) / V, busy = rows > 0 ? (kRunThreads < kLanes * rows ? kRunThreads / rows : kLanes) / lanes1 : 0;
    int64_t few = (8 * V + D - 1) / D;
    few = few > busy ? few : busy;
    few = few < groups ? few : groups;
    const int64_t few_lanes = few * lanes1;
    if (few_lanes <= kLanes && rows <= kRunThreads / few_lanes * held) {
        r.bc = static_cast<int>(few * D);
        r.blocks = static_cast<int>((groups + few - 1) / few);
        r.runs = 1;
        r.per = rows;
        r.whole = true;
        return r;
    }
    if (D <= most) {
        r.bc = static_cast<int>(most / D * D < dim ? most / D * D : dim);
        r.blocks = static_cast<int>((dim + r.bc - 1) / r.bc);
    } else {
        r.per_group = (D + most - 1) / most;
        r.bc = most;
        r.blocks = static_cast<int>(groups * r.per_group);
    }
    const int64_t lanes = (r.bc + V - 1) / V, ty = kRunThreads / lanes;
    int64_t n = target / (batch * r.blocks > 0 ? batch * r.blocks : 1);
    const int64_t most_runs = (rows + 4 * ty - 1) / (4 * ty);
    const int64_t least = (rows + most_rows * ty - 1) / (most_rows * ty);
    n = n < least ? least : (n > most_runs ? most_runs : n);
    n = n < 1 ? 1 : n;
    r.per = (rows + n - 1) / n;
    r.runs = r.per > 0 ? static_cast<int>((rows + r.per - 1) / r.per) : 0;
    return r;
}
// The gradient's runs.  Where entries have fewer rows than kSumRows and are more than fill the GPU, a
// workgroup takes several one after the other, kSumRows rows at most, and leaves one partial sum per channel of
// them all.  (With one per entry, 16384 x 5120 of one row took 676 MB of them, four times a bf16 x, and 1820 us
// a call; this way 1280.  Long entries are better spread: 600 x 1024 x 2048 2900 us one by one, 3060 two by two.)
Runs grad_runs_of(int64_t batch, int64_t rows, int64_t dim, int64_t groups, int V) {
    Runs r = runs_of(batch, rows, dim, groups, V, kHeldGrad, grad_groups(V), kMostGradRows);
    const int64_t full = (batch * r.blocks * r.runs + grad_groups(V) - 1) / grad_groups(V), most = rows > 0 ? kSumRows / rows : 1;
    r.fold = full < most ? full : most;
    r.fold = r.fold > 1 ? r.fold : 1;
    return r;
}
int64_t folds(int64_t batch, const Runs &r) { return (batch + r.fold - 1) / r.fold; }
// where a workgroup's item lies and what a thread has of it
struct Item {
    int64_t row0, rows;                    // the run's first row (of all batch entries'), its rows
    int run, block;
    int lanes, ty_count, tx, ty, ch;       // lanes of a row, rows at a time, the thread's place, its first channel
    int groups, dv, q;                     // groups of the block, lanes of each, the thread's
    int slot, group;                       // the first of the block's partial sums; the thread's group
    bool in;
};
template <int V> __device__ __forceinline__ Item item_of(const GroupNormArgs &a, const Runs &r, int64_t n) {
    Item t;
    const int dim = static_cast<int>(a.dim), id = static_cast<int>(blockIdx.x);
    t.block = id % r.blocks;
    t.run = id / r.blocks;
    t.row0 = t.run * r.per;
    t.rows = t.row0 + r.per < a.rows ? r.per : a.rows - t.row0;
    t.row0 += n * a.rows;
    int c0 = t.block * r.bc, c1 = c0 + r.bc < dim ? c0 + r.bc : dim;
    t.slot = t.block * (r.bc / r.D);
    if (r.per_group > 1) {
        const int g = t.block / r.per_group;
        c0 = g * r.D + t.block % r.per_group * r.bc;
        c1 = c0 + r.bc < (g + 1) * r.D ? c0 + r.bc : (g + 1) * r.D;
        t.slot = t.block;
    }
    t.lanes = (c1 - c0) / V;
    t.ty_count = kRunThreads / t.lanes;
    t.tx = static_cast<int>(threadIdx.x) % t.lanes;
    t.ty = static_cast<int>(threadIdx.x) / t.lanes;
    t.in = t.ty < t.ty_count;
    t.ch = c0 + t.tx * V;
    t.dv = r.per_group > 1 ? t.lanes : r.D / V;
    t.groups = t.lanes / t.dv;
    t.q = t.tx / t.dv;
    t.group = t.ch / r.D;
    return t;
}
// A thread's vectors of a tensor: its first row's, rows apart by `step` elements
template <typename T> struct Walk {
    T *p;
    int64_t step;
    __device__ __forceinline__ Walk(void *base, int64_t ld, const Item &t)
        : p(static_cast<T *>(base) + (t.row0 + t.ty) * ld + t.ch), step(t.ty_count * ld) {}
    __device__ __forceinline__ Walk(const void *base, int64_t ld, const Item &t) : Walk(const_cast<void *>(base), ld, t) {}
    __device__ __forceinline__ T *next() {
        T *const q = p;
        p += step;
        return q;
    }
};
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}
template <int V> __device__ __forceinline__ void params_of(const GroupNormArgs &a, int ch, Affine (&p)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = {a.weight ? a.weight[ch + i] : 1.0f, a.bias ? a.bias[ch + i] : 0.0f};
}

// Two sums over the threads of each group of a block, in a fixed order: a wave per
// group adds its lanes of every row of threads.
struct Totals {
    double s1[kRunThreads], s2[kRunThreads], t1[kLanes], t2[kLanes];
};
__device__ __forceinline__ void group_totals(Totals &m, const Item &t, double u, double v) {
    const int lane = threadIdx.x % 64;
    __syncthreads();
    m.s1[threadIdx.x] = u;
    m.s2[threadIdx.x] = v;
    __syncthreads();
    for (int q = threadIdx.x / 64; q < t.groups; q += kRunWaves) {
        double x = 0.0, y = 0.0;
        for (int e = lane; e < t.dv * t.ty_count; e += 64) {
            const int o = e / t.dv * t.lanes + q * t.dv + e % t.dv;
            x += m.s1[o];
            y += m.s2[o];
        }
        x = wave_sum(x);
        y = wave_sum(y);
        if (lane == 0) {
            m.t1[q] = x;
            m.t2[q] = y;
        }
    }
    __syncthreads();
}
__device__ __forceinline__ void put_totals(const Totals &m, const GroupNormArgs &a, const Runs &r, const Item &t, int64_t n, double *part) {
    const int q = static_cast<int>(threadIdx.x);
    if (q >= t.groups) return;
    double *const o = part + 2 * ((n * r.runs + t.run) * a.groups * r.per_group + t.slot + q);
    o[0] = m.t1[q];
    o[1] = m.t2[q];
}
// The runs' sums of the block's groups, added by each workgroup that needs them for
// itself: a launch less, for a few KB out of the L2.  Up to 64 lanes to a group.
__device__ __forceinline__ void add_runs(Totals &m, const GroupNormArgs &a, const Runs &r, const Item &t, int64_t n, const double *part) {
    int lg = 64;
    while (lg * t.groups > kRunThreads) lg /= 2;
    const int q = static_cast<int>(threadIdx.x) / lg, l = static_cast<int>(threadIdx.x) % lg, row = static_cast<int>(a.groups) * r.per_group;
    double x = 0.0, y = 0.0;
    if (q < t.groups) {
        const double *const p = part + 2 * (n * r.runs * row + (r.per_group > 1 ? t.block / r.per_group * r.per_group : t.slot + q));
        if (r.per_group == 1) {
#pragma unroll 4
            for (int e = l; e < r.runs; e += lg) {
                x += p[2ll * e * row];
                y += p[2ll * e * row + 1];
            }
        } else {
            for (int e = l; e < r.runs * r.per_group; e += lg) {
                const double *const o = p + 2ll * (e / r.per_group * row + e % r.per_group);
                x += o[0];
                y += o[1];
            }
        }
    }
    for (int o = lg / 2; o > 0; o /= 2) {
        x += __shfl_xor(x, o);
        y += __shfl_xor(y, o);
    }
    __syncthreads();
    if (l == 0 && q < t.groups) {
        m.t1[q] = x;
        m.t2[q] = y;
    }
    __syncthreads();
}
__device__ __forceinline__ void put_stats(const GroupNormArgs &a, const Runs &r, const Item &t, int64_t n, float mean, float rstd) {
    if (t.run != 0 || t.ty != 0 || t.tx % t.dv != 0 || (r.per_group > 1 && t.block % r.per_group != 0)) return;
    if (a.mean) a.mean[n * a.groups + t.group] = mean;
    if (a.rstd) a.rstd[n * a.groups + t.group] = rstd;
}

// The first value of the thread's group in batch entry n.
template <typename T> __device__ __forceinline__ float pivot_of(const GroupNormArgs &a, const Item &t, int D, int64_t n) {
    return to_f32(static_cast<const T *>(a.x)[n * a.rows * a.ldx + static_cast<int64_t>(t.group) * D]);
}
// Sums of x - x0 and its square over a run, x0 the thread's first value, in fp32 over
// a vector and fp64 beyond, then about the group's first value instead, which all runs and
// threads share: x - x0 is about as large as the group's spread, and a mean far from 0 costs
// the variance nothing (sums of x^2 themselves would cost it mean^2 2^-52, beside eps).  (All in
// fp64 the pass took 35 us over 134 MB instead of 27.)
template <typename T, int V> __global__ __launch_bounds__(kRunThreads) void group_stats_kernel(GroupNormArgs a, Runs r, double *part) {
    __shared__ Totals m;
    for (int64_t n = blockIdx.y; n < a.batch; n += gridDim.y) {
        const Item t = item_of<V>(a, r, n);
        double u = 0.0, v = 0.0;
        if (t.in && t.ty < t.rows) {
            Walk<const T> px(a.x, a.ldx, t);
            const T *const first = px.p;
            const float x0 = to_f32(*first);
            for (int64_t left = t.rows - t.ty; left > 0; left -= 4 * t.ty_count) {
                typename Vec<T, V>::raw q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const T *const at = px.next();
                    q[j] = load_vec<T, V>(left > j * t.ty_count ? at : first);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x[V], su = 0.0f, sv = 0.0f;
                    unpack<T, V>(q[j], x);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float d = left > j * t.ty_count ? x[i] - x0 : 0.0f;
                        su += d;
                        sv = fmaf(d, d, sv);
                    }
                    u += su;
                    v += sv;
                }
            }
            const double count = static_cast<double>((t.rows - t.ty + t.ty_count - 1) / t.ty_count * V), z = static_cast<double>(x0) - pivot_of<T>(a, t, r.D, n);
            v += z * (2.0 * u + count * z);
            u += count * z;
        }
        group_totals(m, t, u, v);
        put_totals(m, a, r, t, n, part);
    }
}
template <typename T, int V> __global__ __launch_bounds__(kRunThreads) __attribute__((amdgpu_waves_per_eu(8, 8))) void group_apply_kernel(GroupNormArgs a, Runs r, const double *part) {
    __shared__ Totals m;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(a.dim / a.groups));
    for (int64_t n = blockIdx.y; n < a.batch; n += gridDim.y) {
        const Item t = item_of<V>(a, r, n);
        add_runs(m, a, r, t, n, part);
        if (!t.in) continue;
        const double mu = m.t1[t.q] * inv, var = m.t2[t.q] * inv - mu * mu;      // about the pivot
        const float mean = static_cast<float>(pivot_of<T>(a, t, r.D, n) + mu);
        const float rstd = static_cast<float>(1.0 / sqrt((var < 0.0 ? 0.0 : var) + static_cast<double>(a.eps)));
        put_stats(a, r, t, n, mean, rstd);
        Affine p[V];
        params_of<V>(a, t.ch, p);
        Walk<const T> px(a.x, a.ldx, t), pz(a.z, a.ldz, t);
        Walk<T> py(a.y, a.dim, t);
#pragma unroll 2
        for (int64_t left = t.rows - t.ty; left > 0; left -= t.ty_count) {
            float x[V], z[V] = {};
            unpack<T, V>(load_vec<T, V>(px.next()), x);
            if (gate) unpack<T, V>(load_vec<T, V>(pz.next()), z);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = forward((x[i] - mean) * rstd, p[i], act, gate, z[i]);
            store_vec<T, V>(py.next(), x);
        }
    }
}
// Whole batch entries in registers: one launch, one pass
template <typename T, int V> __global__ __launch_bounds__(kRunThreads) void group_whole_kernel(GroupNormArgs a, Runs r) {
    __shared__ Totals m;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(a.dim / a.groups));
    using raw = typename Vec<T, V>::raw;
    for (int64_t n = blockIdx.y; n < a.batch; n += gridDim.y) {
        const Item t = item_of<V>(a, r, n);
        Walk<const T> px(a.x, a.ldx, t), pz(a.z, a.ldz, t);
        Walk<T> py(a.y, a.dim, t);
        raw qx[kHeld], qz[kHeld];
        Affine p[V];
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            const bool in = t.in && t.ty + j * t.ty_count < t.rows;
            qx[j] = qz[j] = raw{};
            const T *const ax = px.next(), *const az = pz.next();
            if (in) qx[j] = load_vec<T, V>(ax);
            if (in && gate) qz[j] = load_vec<T, V>(az);
        }
        params_of<V>(a, t.ch, p);
        double u = 0.0, v = 0.0;                             // fp32 over a vector, fp64 beyond
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            float x[V], s = 0.0f;
            unpack<T, V>(qx[j], x);
#pragma unroll
            for (int i = 0; i < V; ++i) s += x[i];
            u += s;
        }
        group_totals(m, t, u, 0.0);
        const float mean = static_cast<float>(m.t1[t.q] * inv);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            float x[V], s = 0.0f;
            unpack<T, V>(qx[j], x);
            const bool in = t.in && t.ty + j * t.ty_count < t.rows;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = in ? x[i] - mean : 0.0f;
                s = fmaf(d, d, s);
            }
            v += s;
        }
        group_totals(m, t, v, 0.0);
        const float rstd = static_cast<float>(1.0 / sqrt(m.t1[t.q] * inv + static_cast<double>(a.eps)));
        if (t.in) put_stats(a, r, t, n, mean, rstd);
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            T *const ay = py.next();
            if (!t.in || t.ty + j * t.ty_count >= t.rows) continue;
            float x[V], z[V];
            unpack<T, V>(qx[j], x);
            unpack<T, V>(qz[j], z);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = forward((x[i] - mean) * rstd, p[i], act, gate, z[i]);
            store_vec<T, V>(ay, x);
        }
    }
}

// Sums over a workgroup's rows of each channel of the block, to o and o + dim
template <int V> struct ChannelSums {
    float a[kRunThreads][V + 1], b[kRunThreads][V + 1];
};
template <int V> __device__ __forceinline__ void channel_sums(ChannelSums<V> &m, const Item &t, const float (&u)[V], const float (&v)[V], float *o, int64_t dim) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        m.a[threadIdx.x][i] = u[i];
        m.b[threadIdx.x][i] = v[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < t.lanes * V; c += kRunThreads) {
        double x = 0.0, y = 0.0;
        for (int q = 0; q < t.ty_count; ++q) {
            x += m.a[q * t.lanes + c / V][c % V];
            y += m.b[q * t.lanes + c / V][c % V];
        }
        o[c] = static_cast<float>(x);
        o[dim + c] = static_cast<float>(y);
    }
}
// A thread's sums of w da and w da n, added to x and y
template <int V> __device__ __forceinline__ void weighted(const Affine (&p)[V], const float (&u)[V], const float (&v)[V], double &x, double &y) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x += static_cast<double>(p[i].w) * u[i];
        y += static_cast<double>(p[i].w) * v[i];
    }
}
// The gradient's sums of da and da n of each run and channel over r.fold entries, (fold, run), 2, dim, and of
// w da and w da n of each entry, run and group
// FOLD: r.fold is more than 1; else the loop over a fold costs registers (12 x 3025 x 192 41 us a call, with it 44)
template <typename T, int V, bool FOLD> __global__ __launch_bounds__(kRunThreads) __attribute__((amdgpu_waves_per_eu(grad_waves(V), grad_waves(V)))) void group_sums_kernel(GroupNormBwdArgs b, Runs r, double *part, float *chan) {
    const GroupNormArgs &a = b.fwd;
    __shared__ union { ChannelSums<V> c; Totals t; } m;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const int64_t fold = FOLD ? r.fold : 1;
    for (int64_t n0 = blockIdx.y * fold; n0 < a.batch; n0 += gridDim.y * fold) {
        Item t = item_of<V>(a, r, n0);
        Affine p[V];
        params_of<V>(a, t.ch, p);
        float u[V] = {}, v[V] = {};
        const int64_t n1 = FOLD ? (n0 + fold < a.batch ? n0 + fold : a.batch) : n0 + 1;
        for (int64_t n = n0; n < n1; ++n, t.row0 += a.rows) {
            double s1 = 0.0, s2 = 0.0;
            if (t.in) {
                const float mean = a.mean[n * a.groups + t.group], rstd = a.rstd[n * a.groups + t.group];
                Walk<const T> px(a.x, a.ldx, t), pz(a.z, a.ldz, t), pd(b.dy, a.dim, t);
                for (int64_t left = t.rows - t.ty; left > 0;) {
                    const int64_t stop = left > kSumRows * t.ty_count ? left - kSumRows * t.ty_count : 0;
                    float su[V] = {}, sv[V] = {};
#pragma unroll 2
                    for (; left > stop; left -= t.ty_count) {
                        float x[V], z[V] = {}, d[V], dz = 0.0f;
                        unpack<T, V>(load_vec<T, V>(px.next()), x);
                        unpack<T, V>(load_vec<T, V>(pd.next()), d);
                        if (gate) unpack<T, V>(load_vec<T, V>(pz.next()), z);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            const float nx = (x[i] - mean) * rstd, da = backward(nx, d[i], p[i], act, gate, z[i], dz);
                            su[i] += da;
                            sv[i] = fmaf(da, nx, sv[i]);
                        }
                    }
                    weighted<V>(p, su, sv, s1, s2);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        u[i] += su[i];
                        v[i] += sv[i];
                    }
                }
            }
            group_totals(m.t, t, s1, s2);
            put_totals(m.t, a, r, t, n, part);
        }
        if (chan) channel_sums<V>(m.c, t, u, v, chan + (n0 / fold * r.runs + t.run) * 2 * a.dim + (t.ch - t.tx * V), a.dim);
    }
}
template <typename T, int V> __global__ __launch_bounds__(kRunThreads) __attribute__((amdgpu_waves_per_eu(grad_waves(V), grad_waves(V)))) void group_grad_kernel(GroupNormBwdArgs b, Runs r, const double *part) {
    const GroupNormArgs &a = b.fwd;
    __shared__ Totals m;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(a.dim / a.groups));
    for (int64_t n = blockIdx.y; n < a.batch; n += gridDim.y) {
        const Item t = item_of<V>(a, r, n);
        add_runs(m, a, r, t, n, part);
        if (!t.in) continue;
        Affine p[V];
        params_of<V>(a, t.ch, p);
        const int64_t ng = n * a.groups + t.group;
        const float mean = a.mean[ng], rstd = a.rstd[ng], m1 = static_cast<float>(m.t1[t.q] * inv), m2 = static_cast<float>(m.t2[t.q] * inv);
        Walk<const T> px(a.x, a.ldx, t), pz(a.z, a.ldz, t), pd(b.dy, a.dim, t);
        Walk<T> po(b.dx, a.dim, t), pzo(b.dz, a.dim, t);
#pragma unroll 2
        for (int64_t left = t.rows - t.ty; left > 0; left -= t.ty_count) {
            float x[V], z[V] = {}, d[V], dz[V];
            unpack<T, V>(load_vec<T, V>(px.next()), x);
            unpack<T, V>(load_vec<T, V>(pd.next()), d);
            if (gate) unpack<T, V>(load_vec<T, V>(pz.next()), z);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float nx = (x[i] - mean) * rstd, da = backward(nx, d[i], p[i], act, gate, z[i], dz[i]);
                x[i] = rstd * (da * p[i].w - fmaf(nx, m2, m1));
            }
            store_vec<T, V>(po.next(), x);
            if (gate) store_vec<T, V>(pzo.next(), dz);
        }
    }
}
// The gradient of whole batch entries in registers; the channels' sums are (fold, 2, dim)
template <typename T, int V, bool FOLD> __global__ __launch_bounds__(kRunThreads) void group_whole_grad_kernel(GroupNormBwdArgs b, Runs r, float *chan) {
    const GroupNormArgs &a = b.fwd;
    __shared__ union { ChannelSums<V> c; Totals t; } m;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const double inv = 1.0 / (static_cast<double>(a.rows) * static_cast<double>(a.dim / a.groups));
    using raw = typename Vec<T, V>::raw;
    const int64_t fold = FOLD ? r.fold : 1;
    for (int64_t n0 = blockIdx.y * fold; n0 < a.batch; n0 += gridDim.y * fold) {
        Item t = item_of<V>(a, r, n0);
        Affine p[V];
        params_of<V>(a, t.ch, p);
        float cu[V] = {}, cv[V] = {};
        const int64_t n1 = FOLD ? (n0 + fold < a.batch ? n0 + fold : a.batch) : n0 + 1;
        for (int64_t n = n0; n < n1; ++n, t.row0 += a.rows) {
            const int64_t ng = n * a.groups + t.group;
            Walk<const T> px(a.x, a.ldx, t), pz(a.z, a.ldz, t), pd(b.dy, a.dim, t);
            Walk<T> po(b.dx, a.dim, t), pzo(b.dz, a.dim, t);
            raw qx[kHeldGrad], qz[kHeldGrad], qd[kHeldGrad];
#pragma unroll
            for (int j = 0; j < kHeldGrad; ++j) {
                const bool in = t.in && t.ty + j * t.ty_count < t.rows;
                qx[j] = qz[j] = qd[j] = raw{};
                const T *const ax = px.next(), *const az = pz.next(), *const ad = pd.next();
                if (in) qx[j] = load_vec<T, V>(ax);
                if (in) qd[j] = load_vec<T, V>(ad);
                if (in && gate) qz[j] = load_vec<T, V>(az);
            }
            const float mean = a.mean[ng], rstd = a.rstd[ng];
            float u[V] = {}, v[V] = {};
#pragma unroll
            for (int j = 0; j < kHeldGrad; ++j) {
                float x[V], z[V], d[V], dz = 0.0f;
                unpack<T, V>(qx[j], x);
                unpack<T, V>(qd[j], d);
                unpack<T, V>(qz[j], z);
                const bool in = t.in && t.ty + j * t.ty_count < t.rows;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float nx = in ? (x[i] - mean) * rstd : 0.0f, da = in ? backward(nx, d[i], p[i], act, gate, z[i], dz) : 0.0f;
                    u[i] += da;
                    v[i] = fmaf(da, nx, v[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                cu[i] += u[i];
                cv[i] += v[i];
            }
            double s1 = 0.0, s2 = 0.0;
            weighted<V>(p, u, v, s1, s2);
            group_totals(m.t, t, s1, s2);
            const float m1 = static_cast<float>(m.t.t1[t.q] * inv), m2 = static_cast<float>(m.t.t2[t.q] * inv);
#pragma unroll
            for (int j = 0; j < kHeldGrad; ++j) {
                T *const ao = po.next(), *const az = pzo.next();
                if (!t.in || t.ty + j * t.ty_count >= t.rows) continue;
                float x[V], z[V], d[V], dz[V];
                unpack<T, V>(qx[j], x);
                unpack<T, V>(qd[j], d);
                unpack<T, V>(qz[j], z);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float nx = (x[i] - mean) * rstd, da = backward(nx, d[i], p[i], act, gate, z[i], dz[i]);
                    x[i] = rstd * (da * p[i].w - fmaf(nx, m2, m1));
                }
                store_vec<T, V>(ao, x);
                if (gate) store_vec<T, V>(az, dz);
            }
        }
        if (chan) channel_sums<V>(m.c, t, cu, cv, chan + n0 / fold * 2 * a.dim + (t.ch - t.tx * V), a.dim);
    }
}
// dweight and dbias from (rows, 2, dim) partial sums (da first, or da n first), in a
// fixed order: 16 columns to a workgroup, 64 stripes of rows (column_sum.h's way, but in fp64 and to two outputs)
__global__ __launch_bounds__(1024) void group_params_kernel(const float *part, float *first, float *second, int64_t rows, int64_t dim) {
    __shared__ double sums[64][17];
    const int col = threadIdx.x % 16, stripe = threadIdx.x / 16;
    const int64_t d = static_cast<int64_t>(blockIdx.x) * 16 + col;
    double s = 0.0;
    if (d < 2 * dim) {
#pragma unroll 8
        for (int64_t r = stripe; r < rows; r += 64) s += part[r * 2 * dim + d];
    }
    sums[stripe][col] = s;
    __syncthreads();
    const int w = threadIdx.x / 64, lane = threadIdx.x % 64;
    s = wave_sum(sums[lane][w]);
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 16 + w;
    if (lane == 0 && o < 2 * dim) {
        float *const to = o < dim ? first : second;
        if (to) to[o < dim ? o : o - dim] = static_cast<float>(s);
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
// Workgroups that share a unit's rows: as many as fill the GPU; for the gradient at least so many
// that a wave adds up kSumRows rows at most, as far as a launch's 2^32 lanes go.
int64_t row_first(int64_t batch, int64_t units, bool bwd) {
    const int64_t most = (batch + 3) / 4, lanes = ((int64_t(1) << 32) - 1) / kThreads / units;
    int64_t n = kRowWorkgroups / units, least = bwd ? (batch + 4 * kSumRows - 1) / (4 * kSumRows) : 1;
    least = least < lanes ? least : lanes;
    n = n > least ? n : least;
    return n < most ? n : most;
}

template <typename T, int V, int P, int L, bool BWD> hipError_t run_rows(const GroupNormBwdArgs &b, hipStream_t s) {
    const GroupNormArgs &a = b.fwd;
    constexpr int GW = 64 / L;
    const int64_t units = (a.groups + GW - 1) / GW, first = row_first(a.batch, units, BWD);
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
size_t chan_bytes(int64_t batch, const Runs &r, int64_t dim) { return align256(static_cast<size_t>(folds(batch, r) * r.runs) * 2 * dim * 4); }
size_t part_bytes(int64_t batch, const Runs &r, int64_t groups) {
    return r.whole ? 0 : align256(static_cast<size_t>(batch * r.runs * groups * r.per_group) * 16);
}
// batch entries (folds) on y, as many as a launch's 2^32 lanes allow
dim3 grid_of(int64_t batch, const Runs &r) {
    const int64_t x = static_cast<int64_t>(r.blocks) * r.runs, fit = ((int64_t(1) << 32) - 1) / (x * kRunThreads), most = fit < 65535 ? fit : 65535;
    return dim3(static_cast<unsigned>(x), static_cast<unsigned>(batch < most ? batch : most));
}

template <typename T, int V> hipError_t run_fwd(const GroupNormArgs &a, hipStream_t s) {
    if (row_form(a.rows, a.dim, a.groups, V)) {
        GroupNormBwdArgs b{};
        b.fwd = a;
        return run_rows_of<T, V, false>(b, s);
    }
    const Runs r = runs_of(a.batch, a.rows, a.dim, a.groups, V, kHeld, kRunGroups, kAnyRows);
    if (r.whole) {
        hipLaunchKernelGGL((group_whole_kernel<T, V>), grid_of(a.batch, r), dim3(kRunThreads), 0, s, a, r);
        return hipGetLastError();
    }
    double *const part = static_cast<double *>(a.workspace);
    hipLaunchKernelGGL((group_stats_kernel<T, V>), grid_of(a.batch, r), dim3(kRunThreads), 0, s, a, r, part);
    if (hipError_t e = hipGetLastError()) return e;
    hipLaunchKernelGGL((group_apply_kernel<T, V>), grid_of(a.batch, r), dim3(kRunThreads), 0, s, a, r, part);
    return hipGetLastError();
}
template <typename T, int V> hipError_t run_bwd(const GroupNormBwdArgs &b, hipStream_t s) {
    const GroupNormArgs &a = b.fwd;
    if (row_form(a.rows, a.dim, a.groups, V)) return run_rows_of<T, V, true>(b, s);
    const Runs r = grad_runs_of(a.batch, a.rows, a.dim, a.groups, V);
    const bool params = b.dweight || b.dbias;
    float *const chan = params ? static_cast<float *>(a.workspace) : nullptr;
    double *const part = reinterpret_cast<double *>(static_cast<char *>(a.workspace) + chan_bytes(a.batch, r, a.dim));
    const dim3 grid = grid_of(folds(a.batch, r), r);
    auto first = [&](auto fold) {
        constexpr bool FOLD = decltype(fold)::value;
        if (r.whole) hipLaunchKernelGGL((group_whole_grad_kernel<T, V, FOLD>), grid, dim3(kRunThreads), 0, s, b, r, chan);
        else hipLaunchKernelGGL((group_sums_kernel<T, V, FOLD>), grid, dim3(kRunThreads), 0, s, b, r, part, chan);
    };
    if (r.fold > 1) first(std::true_type{});
    else first(std::false_type{});
    if (hipError_t e = hipGetLastError()) return e;
    if (!r.whole) {
        hipLaunchKernelGGL((group_grad_kernel<T, V>), grid_of(a.batch, r), dim3(kRunThreads), 0, s, b, r, part);
        if (hipError_t e = hipGetLastError()) return e;
    }
    if (!params) return hipSuccess;
    hipLaunchKernelGGL(group_params_kernel, dim3(static_cast<unsigned>((2 * a.dim + 15) / 16)), dim3(1024), 0, s, chan, b.dbias, b.dweight,
                       folds(a.batch, r) * r.runs, a.dim);
    return hipGetLastError();
}

}  // namespace

// The largest over the widths that a call may choose.
size_t group_norm_workspace(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    size_t most = 0;
    for (int v = 1; v <= 8; v *= 2) {
        if (dim / groups % v || row_form(rows, dim, groups, v)) continue;
        const size_t n = part_bytes(batch, runs_of(batch, rows, dim, groups, v, kHeld, kRunGroups, kAnyRows), groups);
        most = n > most ? n : most;
    }
    return most;
}
size_t group_norm_bwd_workspace(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    size_t most = 0;
    for (int v = 1; v <= 8; v *= 2) {
        if (dim / groups % v) continue;
        size_t n;
        if (row_form(rows, dim, groups, v)) {
            n = static_cast<size_t>(row_first(batch, (groups + 7) / 8, true)) * 2 * dim * 4;      // at most 8 groups to a wave
        } else {
            const Runs r = grad_runs_of(batch, rows, dim, groups, v);
            n = chan_bytes(batch, r, dim) + part_bytes(batch, r, groups);
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
