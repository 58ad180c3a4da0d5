// Matrix-core building blocks of the gated delta rule's kernels (delta_scan.hip,
// delta_bwd.hip): operands and accumulator tiles, staging into LDS, the chunks of
// a sequence.
//
// A 16x16 accumulator tile gives lane (g = lane / 16, c = lane % 16) rows 4 g + i
// (i < 4) of column c.  An operand of a product over K = 32 gives it elements
// 8 g .. 8 g + 7 of row (A) or column (B) c.  Rows of accumulator tiles are named
// so that one turns into the other in place: in a pair of tiles that stand for 32
// indices, tile 0's row 4 g + i is index 8 g + i and tile 1's index 8 g + 4 + i, so
// the eight values that a lane holds of the pair are its eight elements of an
// operand, and a product's result is the next product's operand without leaving
// the registers.
//
// bf16 io multiplies in bf16 with fp32 sums.  Operands that are inputs are exact;
// computed ones (states, the solve's results, the decayed products) are carried
// as two bf16 terms, hi = bf16(v) and lo = bf16(v - hi): one term would cost a
// relative 2^-9 in each, two leave 2^-17.  The product of two computed operands drops
// lo x lo (2^-18).  fp32 io multiplies in fp32.
#pragma once

#include "ssm_device.h"
#include "ssm_kernels.h"
#include "wave_fold.h"

namespace ssm {
namespace delta {

constexpr int kC = kDeltaChunk;        // steps of a chunk
constexpr int kThreads = 256, kWaves = 4;
static_assert(kC == 64, "four tiles of 16 steps, one step per lane");

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// index (of 64) that row c of tile `tile` stands for
__device__ __forceinline__ int row_index(int tile, int c) { return 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4; }

// ------------------------------------------------------------------ operands
template <typename T> struct Op;                  // exact values
template <> struct Op<bf16_t> { u32x4 v; };
template <> struct Op<float> { f32x4 a, b; };
template <typename T> struct Op2;                 // computed values
template <> struct Op2<bf16_t> { u32x4 hi, lo; };
template <> struct Op2<float> { f32x4 a, b; };
template <typename T> constexpr int kOpBytes = 64 * sizeof(Op<T>);
constexpr int kOp2Bytes = 64 * 32;

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// fp32: eight products over K = 4, lane group g's slot being its element i
__device__ __forceinline__ f32x4 mfma(f32x4 a0, f32x4 a1, f32x4 b0, f32x4 b1, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[i], b0[i], c, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[i], b1[i], c, 0, 0, 0);
    return c;
}
__device__ __forceinline__ f32x4 mma(const Op<bf16_t> &a, const Op<bf16_t> &b, f32x4 c) { return mfma(a.v, b.v, c); }
__device__ __forceinline__ f32x4 mma(const Op<bf16_t> &a, const Op2<bf16_t> &b, f32x4 c) {
    return mfma(a.v, b.hi, mfma(a.v, b.lo, c));
}
__device__ __forceinline__ f32x4 mma(const Op2<bf16_t> &a, const Op<bf16_t> &b, f32x4 c) {
    return mfma(a.hi, b.v, mfma(a.lo, b.v, c));
}
__device__ __forceinline__ f32x4 mma(const Op2<bf16_t> &a, const Op2<bf16_t> &b, f32x4 c) {
    return mfma(a.hi, b.hi, mfma(a.hi, b.lo, mfma(a.lo, b.hi, c)));
}
template <typename A, typename B> __device__ __forceinline__ f32x4 mma32(const A &a, const B &b, f32x4 c) {
    return mfma(a.a, a.b, b.a, b.b, c);
}
__device__ __forceinline__ f32x4 mma(const Op<float> &a, const Op<float> &b, f32x4 c) { return mma32(a, b, c); }
__device__ __forceinline__ f32x4 mma(const Op<float> &a, const Op2<float> &b, f32x4 c) { return mma32(a, b, c); }
__device__ __forceinline__ f32x4 mma(const Op2<float> &a, const Op<float> &b, f32x4 c) { return mma32(a, b, c); }
__device__ __forceinline__ f32x4 mma(const Op2<float> &a, const Op2<float> &b, f32x4 c) { return mma32(a, b, c); }

// eight computed values (a pair of tiles' registers) as an operand
template <typename T> __device__ __forceinline__ Op2<T> computed(f32x4 a, f32x4 b);
template <> __device__ __forceinline__ Op2<float> computed<float>(f32x4 a, f32x4 b) { return {a, b}; }
template <> __device__ __forceinline__ Op2<bf16_t> computed<bf16_t>(f32x4 a, f32x4 b) {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    Op2<bf16_t> o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o.hi[i] = pack2(v[2 * i], v[2 * i + 1]);
        o.lo[i] = pack2(v[2 * i] - low(o.hi[i]), v[2 * i + 1] - high(o.hi[i]));
    }
    return o;
}
// eight exact values held as floats
template <typename T> __device__ __forceinline__ Op<T> exact(f32x4 a, f32x4 b);
template <> __device__ __forceinline__ Op<float> exact<float>(f32x4 a, f32x4 b) { return {a, b}; }
template <> __device__ __forceinline__ Op<bf16_t> exact<bf16_t>(f32x4 a, f32x4 b) {
    return {u32x4{pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])}};
}

// an operand's bytes in memory (LDS or the workspace), each half 16 bytes a lane
__device__ __forceinline__ Op<bf16_t> get_op(const char *p, int lane, bf16_t) {
    return {*reinterpret_cast<const u32x4 *>(p + lane * 16)};
}
__device__ __forceinline__ Op<float> get_op(const char *p, int lane, float) {
    return {*reinterpret_cast<const f32x4 *>(p + lane * 16), *reinterpret_cast<const f32x4 *>(p + 1024 + lane * 16)};
}
__device__ __forceinline__ Op2<bf16_t> get_op2(const char *p, int lane, bf16_t) {
    return {*reinterpret_cast<const u32x4 *>(p + lane * 16), *reinterpret_cast<const u32x4 *>(p + 1024 + lane * 16)};
}
__device__ __forceinline__ Op2<float> get_op2(const char *p, int lane, float) {
    return {*reinterpret_cast<const f32x4 *>(p + lane * 16), *reinterpret_cast<const f32x4 *>(p + 1024 + lane * 16)};
}
__device__ __forceinline__ void put_op(char *p, int lane, const Op<bf16_t> &o) { *reinterpret_cast<u32x4 *>(p + lane * 16) = o.v; }
__device__ __forceinline__ void put_op(char *p, int lane, const Op<float> &o) {
    *reinterpret_cast<f32x4 *>(p + lane * 16) = o.a;
    *reinterpret_cast<f32x4 *>(p + 1024 + lane * 16) = o.b;
}
__device__ __forceinline__ void put_op(char *p, int lane, const Op2<bf16_t> &o) {
    *reinterpret_cast<u32x4 *>(p + lane * 16) = o.hi;
    *reinterpret_cast<u32x4 *>(p + 1024 + lane * 16) = o.lo;
}
__device__ __forceinline__ void put_op(char *p, int lane, const Op2<float> &o) {
    *reinterpret_cast<f32x4 *>(p + lane * 16) = o.a;
    *reinterpret_cast<f32x4 *>(p + 1024 + lane * 16) = o.b;
}

// Rows of keys and queries in LDS, operands with channels along K.  bf16: lane
// groups lie 320 bytes apart, so that the transposing read of a 4 x 16 block (lane l
// of 16 names row l / 4, piece l % 4 of four channels, and gets column l of the four
// rows) finds its 16 pieces in different banks.
template <typename T> constexpr int kRowBytes = kOpBytes<T>;
template <> inline constexpr int kRowBytes<bf16_t> = 4 * 320;
__device__ __forceinline__ Op<bf16_t> get_row(const char *p, int lane, bf16_t) {
    return {*reinterpret_cast<const u32x4 *>(p + lane / 16 * 320 + lane % 16 * 16)};
}
__device__ __forceinline__ Op<float> get_row(const char *p, int lane, float) { return get_op(p, lane, 0.0f); }
__device__ __forceinline__ void put_row(char *p, int lane, const Op<bf16_t> &o) {
    *reinterpret_cast<u32x4 *>(p + lane / 16 * 320 + lane % 16 * 16) = o.v;
}
__device__ __forceinline__ void put_row(char *p, int lane, const Op<float> &o) { put_op(p, lane, o); }

// ------------------------------------------------------------- global memory
__device__ __forceinline__ f32x4 load4(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void store4(f32x4 v, rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
}
// past the L2, for what a later kernel reads once (a training chunk's state, R, dX: 189 us -> 165 in the forward walk of
// 8 x 2048 steps of 12 heads)
__device__ __forceinline__ void stream4(f32x4 v, rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 2);
}
// eight consecutive io elements
__device__ __forceinline__ Op<bf16_t> load_op(rsrc_t r, uint32_t off, bf16_t) {
    return {__builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0)};
}
__device__ __forceinline__ Op<float> load_op(rsrc_t r, uint32_t off, float) { return {load4(r, off), load4(r, off + 16)}; }
// four consecutive io elements from floats
__device__ __forceinline__ void store_io4(f32x4 v, rsrc_t r, uint32_t off, bf16_t) {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])}, r, off, 0, 0);
}
__device__ __forceinline__ void store_io4(f32x4 v, rsrc_t r, uint32_t off, float) { store4(v, r, off); }

// Eight rows of two neighbouring fp32 columns, as the two columns' operand elements.
struct Columns {
    f32x2 w[8];
    __device__ __forceinline__ void load(rsrc_t r, int j, uint32_t off) {
        w[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
    __device__ __forceinline__ void put(char *p, int lane) const {
        put_op(p, lane, Op<float>{f32x4{w[0][0], w[1][0], w[2][0], w[3][0]}, f32x4{w[4][0], w[5][0], w[6][0], w[7][0]}});
        put_op(p, lane + 1, Op<float>{f32x4{w[0][1], w[1][1], w[2][1], w[3][1]}, f32x4{w[4][1], w[5][1], w[6][1], w[7][1]}});
    }
};

// ---------------------------------------------------------- decay of the steps
// Prefix sums of g over a chunk are fp64, and their differences rounded only relative
// to themselves: a sum behind a few restarts or strong decays is in the thousands, and in
// fp32 each difference would lose |G| U of it for good (behind 48 restarts 4e-4 of a decay).
// bf16 io takes them in log2 units, for the hardware's exponential, and the gradient's
// per-chunk part, which has no registers left, as two floats (8 x 2048 steps of 12 heads 226 to 233 us,
// as with fp32 sums alone; with fp64 ones 248).  A step's g is taken as at least kMinLog: exp(-104) is
// already 0 in fp32, so nothing changes, and -inf (a restart) leaves finite sums.
constexpr float kMinLog = -104.0f;
__device__ __forceinline__ float step_log(float g) { return g < kMinLog ? kMinLog : g; }   // NaN stays

// e^d to 4 U relative (U = 2^-24) down to fp32's subnormals: d = k ln 2 + r with |r| <= ln 2 / 2, r taken in fp64
// (d itself in fp32 would cost |d| / 2 U), e^r by its Taylor series through r^7 (truncation < 6e-9), scaled by 2^k.
// expm1(d) + 1 is no substitute: near -1 expm1 has steps of U, which at d = -10 are 4e-4 of the result and at -17 all of it.
__device__ __forceinline__ float exp_accurate(double d) {
    const double k = __builtin_rint(d * 1.4426950408889634);
    const float r = static_cast<float>(fma(-k, 0.6931471805599453, d));
    float q = fmaf(r, 1.0f / 5040.0f, 1.0f / 720.0f);
    q = fmaf(r, q, 1.0f / 120.0f);
    q = fmaf(r, q, 1.0f / 24.0f);
    q = fmaf(r, q, 1.0f / 6.0f);
    q = fmaf(r, q, 0.5f);
    q = fmaf(r, q, 1.0f);
    return __builtin_amdgcn_ldexpf(fmaf(r, q, 1.0f), static_cast<int>(k));
}

template <typename T> struct Decay;
template <> struct Decay<bf16_t> {
    using Sum = f32x2;                                 // hi + lo
    static __device__ __forceinline__ double scaled(float g) { return g * 1.4426950408889634; }
    static __device__ __forceinline__ Sum sum(double G) {
        const float hi = static_cast<float>(G);
        return {hi, static_cast<float>(G - hi)};
    }
    static __device__ __forceinline__ float minus(Sum a, Sum b) { return (a[0] - b[0]) + (a[1] - b[1]); }
    static __device__ __forceinline__ float ex(float d) { return fast_exp2(d); }
    static __device__ __forceinline__ float ex(double d) { return fast_exp2(static_cast<float>(d)); }
};
template <> struct Decay<float> {
    using Sum = double;
    static __device__ __forceinline__ double scaled(float g) { return static_cast<double>(g); }
    static __device__ __forceinline__ Sum sum(double G) { return G; }
    static __device__ __forceinline__ double minus(Sum a, Sum b) { return a - b; }
    static __device__ __forceinline__ float ex(double d) { return exp_accurate(d); }
};
__device__ __forceinline__ double lane_prefix(double v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double u = __shfl_up(v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// ------------------------------------------------------- sequences and chunks
// Sequence i's first row, its length and the slot of its first chunk.  Packed
// sequences: slot floor(start / 64) + i, which leaves every sequence room for its
// chunks whatever the lengths.  Starts that are out of order or out of range are
// brought into it, so that no access leaves the tensors.
struct Span {
    int64_t row0;
    int len;
    int64_t slot0;
};
__device__ __forceinline__ int clamp_start(const DeltaShape &s, int64_t i) {
    const int v = s.starts[i], total = static_cast<int>(s.seqlen);
    return v < 0 ? 0 : (v > total ? total : v);
}
__device__ __forceinline__ Span span_of(const DeltaShape &s, int64_t i) {
    if (!s.starts) return {i * s.seqlen, static_cast<int>(s.seqlen), i * ((s.seqlen + kC - 1) / kC)};
    const int a = clamp_start(s, i), b = clamp_start(s, i + 1);
    return {a, b > a ? b - a : 0, (a >> 6) + i};
}
// the sequence that a chunk's slot belongs to
__device__ __forceinline__ int64_t sequence_of(const DeltaShape &s, int64_t slot) {
    if (!s.starts) return slot / ((s.seqlen + kC - 1) / kC);
    int64_t lo = 0, hi = s.nseq - 1;
    while (lo < hi) {                                  // the last one whose first slot is not behind this one
        const int64_t mid = (lo + hi + 1) / 2;
        if ((clamp_start(s, mid) >> 6) + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Time segments: a sequence's chunks cut into runs of cps.  Between two neighbouring
// segments of a sequence lies a border, where a state and a transition are kept; packed
// sequence i's first one is (its first chunk's slot) / cps, which leaves every sequence room
// for its own.  A walk over all segments takes, packed, those behind a border first and then the first
// ones of all sequences: long ones start early, and what is not cut lies side by side.  (A slot for every
// segment a sequence might have, used or not, let the used ones meet unevenly on the XCDs: 30 sequences of 300
// steps, 16 heads of 128 x 128 in bf16, 119 us; now 100, uncut 84.)  A pass over the ends has the borders alone.
struct Segment {
    int64_t seq, edge;                                 // edge: the border before it, edge + 1: the one behind it
    int s, j0, j1;                                     // of the sequence; its chunks
    bool used, last;
};
enum Part { kAllSegments, kBeforeEdges, kBehindEdges };
__device__ __forceinline__ int64_t first_edge(const DeltaShape &sh, int64_t seq, int64_t slot0, int segments, int cps) {
    return sh.starts ? slot0 / cps : seq * (segments - 1);
}
template <Part PART> __device__ __forceinline__ Segment segment_of(const DeltaShape &sh, int64_t id, int64_t edges, int cps, Span &sp) {
    Segment g;
    int64_t s = 0;
    if (!sh.starts) {
        const int64_t nc = (sh.seqlen + kC - 1) / kC, ns = nc > cps ? (nc + cps - 1) / cps : 1;
        const int64_t per = PART == kAllSegments ? ns : ns - 1;        // a pass over the ends has two segments at least
        g.seq = id / per;
        s = id - g.seq * per + (PART == kBehindEdges ? 1 : 0);
        g.edge = g.seq * (ns - 1) + s - 1;
        sp = span_of(sh, g.seq);
    } else if (PART == kAllSegments && id >= edges) {
        g.seq = id - edges;
        sp = span_of(sh, g.seq);
        g.edge = sp.slot0 / cps - 1;
    } else {
        int64_t lo = 0, hi = sh.nseq - 1;
        while (lo < hi) {                              // the last one whose first border is not behind this one
            const int64_t mid = (lo + hi + 1) / 2;
            if (((clamp_start(sh, mid) >> 6) + mid) / cps <= id) lo = mid;
            else hi = mid - 1;
        }
        g.seq = lo;
        sp = span_of(sh, lo);
        g.edge = id;
        s = id - sp.slot0 / cps + 1;                   // behind the border
        if (s <= 0 || s * cps >= (sp.len + kC - 1) / kC) s = -1;       // it is no sequence's
        else if (PART == kBeforeEdges) {
            --s;
            --g.edge;
        }
    }
    const int nc = (sp.len + kC - 1) / kC;
    g.used = s >= 0;
    g.s = static_cast<int>(s);
    g.j0 = g.used ? g.s * cps : 0;
    g.j1 = g.j0 + cps < nc ? g.j0 + cps : nc;
    g.last = g.j1 == nc;
    return g;
}

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// What a workgroup of the recurrence holds of a chunk in LDS.  Each part is loaded
// into registers (load) a chunk ahead of the LDS writes (put), so the memory
// latency runs beside the chunk before.

// A chunk's n steps of one head, from its first element: what lies behind the last
// step reads as 0, so offsets inside a chunk do not depend on how long it is.
__device__ __forceinline__ rsrc_t chunk_rsrc(const void *p, int n, int64_t ld, int width, int size) {
    return make_rsrc(p, n > 0 ? static_cast<uint32_t>(((n - 1) * static_cast<int>(ld) + width) * size) : 0u);
}
// Rows of q or k as operands: slot (tile, kk) holds steps row_index(tile, c),
// channels 32 kk + 8 g ...  Channels from K on are zeros.  ld in elements.
template <typename T, int KP> struct Rows {
    static constexpr int KK = KP / 32, N = 4 * KK * 64 / kThreads, kBytes = 4 * KK * kRowBytes<T>;
    static constexpr int kTiles = kWaves / KK;                 // tiles that the threads cover at a time
    Op<T> v[N];
    // the thread's offset in the first tiles; the others are whole rows further on
    static __device__ __forceinline__ uint32_t offset(int64_t ld, int K, int thread) {
        const int lane = thread % 64, f = thread / 64;
        const int t = row_index(f / KK, lane % 16), k = 32 * (f % KK) + 8 * (lane / 16);
        return k < K ? static_cast<uint32_t>((t * static_cast<int>(ld) + k) * static_cast<int>(sizeof(T))) : kOffNone;
    }
    __device__ __forceinline__ void load(rsrc_t r, int64_t ld, uint32_t off) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = load_op(r, off + static_cast<uint32_t>(row_index(i * kTiles, 0) * static_cast<int>(ld) * static_cast<int>(sizeof(T))), T());
    }
    __device__ __forceinline__ void put(char *dst, int thread) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = i * kThreads + thread;
            put_row(dst + s / 64 * kRowBytes<T>, s % 64, v[i]);
        }
    }
};
// The same chunk with steps along K: slot (tile, kk) holds channels row_index (of
// each 32) as rows, steps 32 kk + 8 g ...  fp32 only: bf16 reads the rows' copy
// transposed.
template <int KP> struct Cols {
    using T = float;
    static constexpr int KT = KP / 16, N = KT * 2 * 32 / kThreads, kBytes = 2 * KT * kOpBytes<T>;
    Columns v[N];
    static __device__ __forceinline__ uint32_t offset(int64_t ld, int i, int K, int thread) {
        const int s = i * kThreads + thread, f = s / 32, c = 2 * (s % 8), g = (s / 8) % 4;
        const int tile = f / 2, k = 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4, t0 = 32 * (f % 2) + 8 * g;
        return k < K ? static_cast<uint32_t>((t0 * static_cast<int>(ld) + k) * static_cast<int>(sizeof(T))) : kOffNone;
    }
    struct Offsets {
        uint32_t at[N];
    };
    static __device__ __forceinline__ Offsets offsets(int64_t ld, int K, int thread) {
        Offsets o;
#pragma unroll
        for (int i = 0; i < N; ++i) o.at[i] = offset(ld, i, K, thread);
        return o;
    }
    __device__ __forceinline__ void load(rsrc_t r, int64_t ld, const Offsets &o) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].load(r, j, o.at[i] + static_cast<uint32_t>(j * static_cast<int>(ld) * static_cast<int>(sizeof(T))));
    }
    __device__ __forceinline__ void put(char *dst, int thread) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = i * kThreads + thread, f = s / 32;
            v[i].put(dst + f * kOpBytes<T>, 16 * ((s / 8) % 4) + 2 * (s % 8));
        }
    }
};
// channels of tile kt as rows, steps 32 kk + 8 g ... along K, from the rows or the columns in LDS
template <int KP> __device__ __forceinline__ Op<bf16_t> get_col(const char *rows, const char *, int kt, int kk, int lane, bf16_t) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    using lds = __attribute__((address_space(3))) s16x4 *;
    const int l = lane % 16;
    const char *const p = rows + (l % 4) * 320 + (4 * (lane / 16) + l / 4) * 16 + (2 * kk * (KP / 32) + kt / 2) * kRowBytes<bf16_t> + kt % 2 * 8;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(const_cast<char *>(p)));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(const_cast<char *>(p + KP / 32 * kRowBytes<bf16_t>)));
    const u32x2 u = __builtin_bit_cast(u32x2, a), v = __builtin_bit_cast(u32x2, b);
    return {u32x4{u[0], u[1], v[0], v[1]}};
}
template <int KP> __device__ __forceinline__ Op<float> get_col(const char *, const char *cols, int kt, int kk, int lane, float) {
    return get_op(cols + (kt * 2 + kk) * kOpBytes<float>, lane, 0.0f);
}
// A chunk's steps of a wave's 16 fp32 value channels, as the columns of accumulator
// tiles, or as an operand with steps along K.  V: channels from the workgroup's first on.
struct Values {
    float v[16];
    static __device__ __forceinline__ uint32_t offset(int ld, int V, int w, int lane) {
        const int c = 16 * w + lane % 16;
        return c < V ? static_cast<uint32_t>((8 * (lane / 16) * ld + c) * 4) : kOffNone;
    }
    __device__ __forceinline__ void load(rsrc_t r, int ld, uint32_t off) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = Io<float>::f32(Io<float>::load(r, off + static_cast<uint32_t>((32 * (i / 8) + i % 8) * ld * 4), 0));
    }
    __device__ __forceinline__ Op<float> op(int p) const {
        return {f32x4{v[8 * p], v[8 * p + 1], v[8 * p + 2], v[8 * p + 3]}, f32x4{v[8 * p + 4], v[8 * p + 5], v[8 * p + 6], v[8 * p + 7]}};
    }
};
// an operand's eight elements as the registers of a pair of tiles
__device__ __forceinline__ void tiles(const Op<bf16_t> &o, f32x4 &a, f32x4 &b) {
    a = f32x4{low(o.v[0]), high(o.v[0]), low(o.v[1]), high(o.v[1])};
    b = f32x4{low(o.v[2]), high(o.v[2]), low(o.v[3]), high(o.v[3])};
}
__device__ __forceinline__ void tiles(const Op<float> &o, f32x4 &a, f32x4 &b) {
    a = o.a;
    b = o.b;
}
// bytes from the workspace as they are
template <int BYTES> struct Copy {
    static constexpr int N = BYTES / (16 * kThreads);
    static_assert(BYTES % (16 * kThreads) == 0, "whole pieces");
    u32x4 v[N];
    __device__ __forceinline__ void load(const char *src) {
        const rsrc_t r = make_rsrc(src, BYTES);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, (i * kThreads + threadIdx.x) * 16, 0, 0);
    }
    __device__ __forceinline__ void put(char *dst) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *reinterpret_cast<u32x4 *>(dst + (i * kThreads + threadIdx.x) * 16) = v[i];
    }
};

// A wave's 16 columns of a state, (V, K) in memory with K contiguous, as tiles
// whose rows are K: columns v0 + c, pairs of tiles of 32 channels.
template <int KP> __device__ __forceinline__ void load_state(f32x4 (&S)[KP / 16], const float *p, int v0, int V, int K, int lane) {
    const rsrc_t r = make_rsrc(p, static_cast<uint32_t>(static_cast<int64_t>(V) * K * 4));
    const int v = v0 + lane % 16, g = lane / 16;
#pragma unroll
    for (int q = 0; q < KP / 32; ++q) {
        const int k = 32 * q + 8 * g;
        const uint32_t off = v < V && k < K ? static_cast<uint32_t>((v * K + k) * 4) : kOffNone;
        S[2 * q] = load4(r, off);
        S[2 * q + 1] = load4(r, off == kOffNone ? off : off + 16);
    }
}
template <int KP> __device__ __forceinline__ void store_state(const f32x4 (&S)[KP / 16], float *p, int v0, int V, int K, int lane) {
    const rsrc_t r = make_rsrc(p, static_cast<uint32_t>(static_cast<int64_t>(V) * K * 4));
    const int v = v0 + lane % 16, g = lane / 16;
#pragma unroll
    for (int q = 0; q < KP / 32; ++q) {
        const int k = 32 * q + 8 * g;
        const uint32_t off = v < V && k < K ? static_cast<uint32_t>((v * K + k) * 4) : kOffNone;
        stream4(S[2 * q], r, off);
        stream4(S[2 * q + 1], r, off == kOffNone ? off : off + 16);
    }
}

// ------------------------------------------------- what the chunks share
// Per (chunk slot, head) in the workspace: the six operands of the solve's inverse
// T and of P, or of their transposes, and exp(G), exp(G_end - G), beta per step.
constexpr int kTriBytes = 6 * kOp2Bytes;
// Lower-triangular: tile rows tb, K pair kk <= tb / 2.  Upper: kk >= tb / 2.
__device__ __forceinline__ constexpr int tri_low(int tile, int kk) { return tile < 2 ? tile : 2 * tile - 2 + kk; }
__device__ __forceinline__ constexpr int tri_up(int tile, int kk) { return tile < 2 ? 2 * tile + kk : 2 + tile; }

}  // namespace delta
}  // namespace ssm
