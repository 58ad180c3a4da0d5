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

// ------------------------------------------------------------- global memory
__device__ __forceinline__ f32x4 load4(rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void store4(f32x4 v, rsrc_t r, uint32_t off) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 0);
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

// Eight rows of two neighbouring columns, as the two columns' operand elements.
template <typename T> struct Columns;
template <> struct Columns<bf16_t> {
    uint32_t w[8];
    __device__ __forceinline__ void load(rsrc_t r, int j, uint32_t off) { w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0); }
    __device__ __forceinline__ void put(char *p, int lane) const {
        u32x4 a, b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = (w[2 * i] & 0xffffu) | (w[2 * i + 1] << 16);
            b[i] = (w[2 * i] >> 16) | (w[2 * i + 1] & 0xffff0000u);
        }
        put_op(p, lane, Op<bf16_t>{a});
        put_op(p, lane + 1, Op<bf16_t>{b});
    }
};
template <> struct Columns<float> {
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
// Prefix sums of g over a chunk and exponentials of their differences: fp32 in
// log2 units for bf16 io, fp64 for fp32 io, where |G| 2^-24 lost in each
// difference would show.  A step's g is taken as at least kMinLog: exp(-104) is
// already 0 in fp32, so nothing changes, and -inf (a restart) leaves finite sums.
constexpr float kMinLog = -104.0f;
__device__ __forceinline__ float step_log(float g) { return g < kMinLog ? kMinLog : g; }   // NaN stays

template <typename T> struct Decay;
template <> struct Decay<bf16_t> {
    using real = float;
    static __device__ __forceinline__ float scaled(float g) { return g * kLog2e; }
    static __device__ __forceinline__ float ex(float d) { return fast_exp2(d); }
};
template <> struct Decay<float> {
    using real = double;
    static __device__ __forceinline__ double scaled(float g) { return static_cast<double>(g); }
    static __device__ __forceinline__ float ex(double d) { return expm1_accurate(static_cast<float>(d)) + 1.0f; }
};
template <typename R> __device__ __forceinline__ R lane_prefix(R v, int lane) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const R u = __shfl_up(v, o);
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

__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Rows of a chunk of q or k as operands in LDS: slot (tile, kk) holds steps
// row_index(tile, c), channels 32 kk + 8 g ...  Rows from n on and channels from K
// on are zeros.  ld in elements; r starts at the chunk's first row.
template <typename T, int KP> __device__ __forceinline__ void stage_rows(char *dst, rsrc_t r, int64_t ld, int n, int K) {
    constexpr int KK = KP / 32;
#pragma unroll
    for (int i = 0; i < 4 * KK * 64 / kThreads; ++i) {
        const int s = i * kThreads + threadIdx.x, lane = s % 64, f = s / 64;
        const int t = row_index(f / KK, lane % 16), k = 32 * (f % KK) + 8 * (lane / 16);
        const uint32_t off = t < n && k < K ? static_cast<uint32_t>((t * ld + k) * static_cast<int64_t>(sizeof(T))) : kOffNone;
        put_op(dst + f * kOpBytes<T>, lane, load_op(r, off, T()));
    }
}
// The same chunk with steps along K: slot (tile, kk) holds channels (rows)
// row_index within 32-channel pairs of tiles, steps 32 kk + 8 g ...
template <typename T, int KP> __device__ __forceinline__ void stage_columns(char *dst, rsrc_t r, int64_t ld, int n, int K) {
    constexpr int KT = KP / 16;
#pragma unroll
    for (int i = 0; i < KT * 2 * 32 / kThreads; ++i) {
        const int s = i * kThreads + threadIdx.x, f = s / 32, pair = s % 8, g = (s / 8) % 4;
        const int tile = f / 2, kk = f % 2, c = 2 * pair;
        const int k = 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4, t0 = 32 * kk + 8 * g;
        Columns<T> w;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w.load(r, j, t0 + j < n && k < K ? static_cast<uint32_t>(((t0 + j) * ld + k) * static_cast<int64_t>(sizeof(T))) : kOffNone);
        w.put(dst + f * kOpBytes<T>, 16 * g + c);
    }
}
// bytes from the workspace as they are
template <int BYTES> __device__ __forceinline__ void stage_copy(char *dst, const char *src) {
    static_assert(BYTES % (16 * kThreads) == 0, "whole pieces");
#pragma unroll
    for (int i = 0; i < BYTES / (16 * kThreads); ++i)
        *reinterpret_cast<u32x4 *>(dst + (i * kThreads + threadIdx.x) * 16) =
            *reinterpret_cast<const u32x4 *>(src + (i * kThreads + threadIdx.x) * 16);
}

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
        store4(S[2 * q], r, off);
        store4(S[2 * q + 1], r, off == kOffNone ? off : off + 16);
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
