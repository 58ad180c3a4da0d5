// The gated linear recurrence, its gradient and its one-token form:
//     a = sigmoid(g + bias),  h <- a h + (1 - a) x,  y = h SiLU(z)
//
// One step is the affine map h -> a h + u, u = (1 - a) x, and such maps compose:
// (A1, U1) then (A2, U2) = (A2 A1, A2 U1 + U2).  There are only batch x d_inner
// chains, so time is cut into tiles of 128 steps x 64 lanes of channels.  A
// workgroup of W waves takes one tile; wave w holds S = 128 / W consecutive
// steps in registers, so every tensor is read once and written once:
//   1. each wave discretises its steps and folds them into its (A, U);
//   2. the waves' aggregates meet in LDS and give every wave its prefix and the
//      tile its own (A, U), which is published in the workspace;
//   3. the state entering the tile is the state entering its group of 8 tiles,
//      folded over the published aggregates of the tiles before it in the
//      group (one wave waits for one of them); the last tile of a group
//      publishes the state leaving it.  The order of every fold is fixed, so
//      results do not depend on who was first;
//   4. each wave replays its steps from its own entering state and writes y.
// A tile waits only for tiles with lower tickets, which are running or done; a
// wait is bounded as in the row scan (error word, NaN state).
// The gradient is the same scan backwards over c_t = a_t e_t, with e the
// gradient of h: e_t = d_t + c_{t+1}, tiles in falling order.  It needs the
// states h_{t-1}: they are recomputed inside a tile from the state entering it,
// which the forward saves (one fp32 per channel and 128 steps).
#include "column_sum.h"
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kBlock = kGatedBlock;        // steps of a tile
constexpr int kGroup = 8;                  // tiles of a group
constexpr uint32_t kSpinLimit = 1u << 22;  // polls before a wait gives up
constexpr uint32_t kReady = 0x80000000u;   // set in a published word: a decay is never negative
#ifndef SSM_GATED_FWD_WAVES
#define SSM_GATED_FWD_WAVES 8              // waves of a tile, forward and gradient
#endif
#ifndef SSM_GATED_BWD_WAVES
#define SSM_GATED_BWD_WAVES 16
#endif
constexpr size_t kHeader = 256;            // ticket and error word

// ------------------------------------------------------------------- gates
// a = sigmoid(v) and 1 - a = sigmoid(-v) are carried as one number: the smaller
// of the two, e / (1 + e) with e = exp(-|v|), with v's sign.  The larger is 1
// minus it, rounded once, so neither a decay near 1 nor its complement loses
// its leading digits.  An infinite v gives exactly 0 and 1.
template <bool Precise> __device__ __forceinline__ float signed_gate(float v) {
    float e, small;
    if constexpr (Precise) {
        // v log2(e) in two parts, as its rounding alone would cost |v| units in
        // the last place; the quotient corrected by one Newton step
        constexpr float kLog2eLo = 1.925963033500411e-08f;   // log2(e) - float(log2(e))
        float av = fabsf(v);
        av = av > 128.0f ? 128.0f : av;                       // false for NaN, which stays
        const float t = av * kLog2e;
        const float lo = fmaf(av, kLog2eLo, fmaf(av, kLog2e, -t));
        e = fast_exp2(-t);
        e = fmaf(e * -kLn2, lo, e);
        const float q = 1.0f + e, r = fast_rcp(q);
        small = e * r;
        small = fmaf(fmaf(-q, small, e), r, small);
    } else {
        e = fast_exp2(-fabsf(v) * kLog2e);
        small = e * fast_rcp(1.0f + e);
    }
    return copysignf(small, v);
}
struct Gate {
    float a, s;
};
__device__ __forceinline__ Gate split(float sg) {
    const float small = fabsf(sg), large = 1.0f - small;
    const bool neg = static_cast<int>(__float_as_uint(sg)) < 0;
    return {neg ? small : large, neg ? large : small};
}

// Makes the compiler take a register as new, so that what was derived from it
// before a barrier is derived again after it (a few instructions) and not kept
// in registers across.
template <typename V> __device__ __forceinline__ void renew(V &v) { asm volatile("" : "+v"(v)); }

// ------------------------------------------------- VEC channels of one row
template <typename T, int VEC> struct Cell;
template <> struct Cell<bf16_t, 2> {
    using raw = uint32_t;
    static __device__ __forceinline__ raw load(rsrc_t r, uint32_t off) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, kStream);
    }
    static __device__ __forceinline__ float get(raw v, int i) { return __uint_as_float(i ? (v & 0xffff0000u) : (v << 16)); }
    static __device__ __forceinline__ void store(const float (&v)[2], rsrc_t r, uint32_t off) {
        const uint32_t lo = from_f32<bf16_t>(v[0]).bits, hi = from_f32<bf16_t>(v[1]).bits;
        __builtin_amdgcn_raw_buffer_store_b32(lo | (hi << 16), r, off, 0, kStream);
    }
};
template <typename T> struct Cell<T, 1> {
    using raw = typename Io<T>::raw;
    static __device__ __forceinline__ raw load(rsrc_t r, uint32_t off) { return Io<T>::template load<kStream>(r, off, 0); }
    static __device__ __forceinline__ float get(raw v, int) { return Io<T>::f32(v); }
    static __device__ __forceinline__ void store(const float (&v)[1], rsrc_t r, uint32_t off) {
        Io<T>::template store<kStream>(v[0], r, off, 0);
    }
};

// --------------------------------------------------------------- hand-over
struct Link {
    uint32_t *words;             // [0] ticket, [1] error
    uint64_t *agg, *state;       // per (chain, tile) and per (chain, group): 64 VEC words each
    uint32_t spin_limit;
    int publish;
};

// one word once it is ready; 0 when the wait gave up
__device__ __forceinline__ uint64_t wait_word(const uint64_t *p, const Link &k) {
    uint64_t v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    uint32_t spins = 0;
    while (!(static_cast<uint32_t>(v) & kReady)) {
        if (++spins > k.spin_limit) {
            __hip_atomic_store(&k.words[1], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            return 0;
        }
        __builtin_amdgcn_s_sleep(1);
        v = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    return v;
}
__device__ __forceinline__ void publish_word(uint64_t *p, float decay, float offset) {
    const uint64_t v = (static_cast<uint64_t>(__float_as_uint(offset)) << 32) | (__float_as_uint(decay) | kReady);
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float word_decay(uint64_t v) {
    return __uint_as_float(static_cast<uint32_t>(v) & ~kReady);
}
__device__ __forceinline__ float word_offset(uint64_t v) {
    const float f = __uint_as_float(static_cast<uint32_t>(v >> 32));
    return (static_cast<uint32_t>(v) & kReady) ? f : __builtin_nanf("");   // gave up: poison
}

// The carry entering tile k of a chain (k counts in scan order): `first` for
// the chain's first group, else the published state of the group before, folded
// over the group's tiles before k.  All W >= kGroup waves take part; `h` is the
// result in every wave.  Publishes this tile's aggregate beforehand, and the
// state leaving the group when k is its last tile.
template <int W, int VEC>
__device__ __forceinline__ void chain_carry(const Link &lk, int64_t chain, int n_tiles, int k, const float (&A)[VEC],
                                            const float (&U)[VEC], const float (&first)[VEC],
                                            float2 (*slot)[64 * VEC], int w, int lane, float (&h)[VEC]) {
    static_assert(W >= kGroup, "one wave waits for one tile");
    constexpr int kW = 64 * VEC;
    const int in_group = k % kGroup, n_groups = (n_tiles + kGroup - 1) / kGroup;
    uint64_t *mine = lk.agg + (chain * n_tiles + k) * kW;
    uint64_t *states = lk.state + chain * n_groups * kW;
    const bool more = k + 1 < n_tiles;
    if (w == 0 && more && in_group != kGroup - 1 && lk.publish) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) publish_word(mine + e * 64 + lane, A[e], U[e]);
    }
    // wave w < in_group: the aggregate of the group's tile w; wave kGroup - 1: the
    // state before the group
    if (w < in_group) {
        const uint64_t *p = lk.agg + (chain * n_tiles + (k - in_group + w)) * kW;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const uint64_t v = wait_word(p + e * 64 + lane, lk);
            slot[w][e * 64 + lane] = make_float2(word_decay(v), word_offset(v));
        }
    } else if (w == kGroup - 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float s = first[e];
            if (k >= kGroup) s = word_offset(wait_word(states + (k / kGroup - 1) * kW + e * 64 + lane, lk));
            slot[w][e * 64 + lane] = make_float2(0.0f, s);
        }
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = slot[kGroup - 1][e * 64 + lane].y;
    for (int i = 0; i < in_group; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 m = slot[i][e * 64 + lane];
            h[e] = fmaf(m.x, h[e], m.y);
        }
    }
    if (w == 0 && more && in_group == kGroup - 1 && lk.publish) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            publish_word(states + (k / kGroup) * kW + e * 64 + lane, 0.0f, fmaf(A[e], h[e], U[e]));
    }
}

// ----------------------------------------------------------------- forward
struct FwdParams {
    const void *x, *g, *z;
    int64_t ldx, ldg, ldz;
    const float *bias, *h0;
    void *y;
    float *last, *ckpt;
    int64_t seqlen;
    int dim, n_ct, n_tiles;
    uint32_t chains;             // batch x column tiles
    Link link;
};

// the rows of a strided tensor that a wave holds, from (row, column c0) on
template <typename T> __device__ __forceinline__ rsrc_t rows_rsrc(const void *p, int64_t row, int64_t ld, int c0, int dim, int n) {
    const uint32_t bytes = n > 0 ? static_cast<uint32_t>(((n - 1) * ld + (dim - c0)) * static_cast<int64_t>(sizeof(T))) : 0u;
    return make_rsrc(static_cast<const char *>(p) + (row * ld + c0) * static_cast<int64_t>(sizeof(T)), bytes);
}

template <typename T, int VEC, int W, bool Z, bool Multi>
__global__ __launch_bounds__(W * 64) void gated_fwd_kernel(FwdParams p) {
    using C = Cell<T, VEC>;
    using raw = typename C::raw;
    constexpr int S = kBlock / W;
    constexpr bool Precise = sizeof(T) == 4;
    __shared__ float2 sAgg[W][64 * VEC];
    __shared__ float2 sLink[Multi ? kGroup : 1][64 * VEC];
    __shared__ uint32_t sTicket;

    const int tid = threadIdx.x, lane = tid % 64;
    const int w = __builtin_amdgcn_readfirstlane(tid / 64);
    uint32_t ticket = blockIdx.x;
    if constexpr (Multi) {
        if (tid == 0) sTicket = atomicAdd(&p.link.words[0], 1u);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(sTicket);
    }
    const uint32_t chain = ticket % p.chains;
    const int k = static_cast<int>(ticket / p.chains);
    const int64_t b = chain / p.n_ct;
    const int c0 = static_cast<int>(chain % p.n_ct) * 64 * VEC;
    const int ch = c0 + lane * VEC;
    const bool active = ch < p.dim;
    const int64_t t0 = static_cast<int64_t>(k) * kBlock + w * S;     // first step of the wave
    const int64_t left = p.seqlen - t0;
    const int n = static_cast<int>(left < 0 ? 0 : (left < S ? left : S));
    const int64_t row = b * p.seqlen + t0;

    const uint32_t col = active ? static_cast<uint32_t>(lane * VEC * sizeof(T)) : kOffNone;
    const rsrc_t rx = rows_rsrc<T>(p.x, row, p.ldx, c0, p.dim, n), rg = rows_rsrc<T>(p.g, row, p.ldg, c0, p.dim, n);
    const uint32_t bx = static_cast<uint32_t>(p.ldx * sizeof(T)), bg = static_cast<uint32_t>(p.ldg * sizeof(T));
    raw xr[S], gr[S], zr[Z ? S : 1];
#pragma unroll
    for (int i = 0; i < S; ++i) gr[i] = C::load(rg, col + i * bg);
#pragma unroll
    for (int i = 0; i < S; ++i) xr[i] = C::load(rx, col + i * bx);
    if constexpr (Z) {
        const rsrc_t rz = rows_rsrc<T>(p.z, row, p.ldz, c0, p.dim, n);
        const uint32_t bz = static_cast<uint32_t>(p.ldz * sizeof(T));
#pragma unroll
        for (int i = 0; i < S; ++i) zr[i] = C::load(rz, col + i * bz);
    }
    float bias[VEC], first[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        bias[e] = (p.bias && active) ? p.bias[ch + e] : 0.0f;
        first[e] = (p.h0 && active) ? p.h0[b * p.dim + ch + e] : 0.0f;
    }

    // discretise and fold; steps past the sequence are the identity
    float a[S][VEC], u[S][VEC], A[VEC], U[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = 1.0f;
        U[e] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const Gate q = split(signed_gate<Precise>(C::get(gr[i], e) + bias[e]));
            a[i][e] = i < n ? q.a : 1.0f;
            u[i][e] = i < n ? q.s * C::get(xr[i], e) : 0.0f;
            U[e] = fmaf(a[i][e], U[e], u[i][e]);
            A[e] *= a[i][e];
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sAgg[w][e * 64 + lane] = make_float2(A[e], U[e]);
    __syncthreads();
    float Ap[VEC], Up[VEC];                          // the waves before this one
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = 1.0f;
        U[e] = 0.0f;
    }
#pragma unroll 4
    for (int i = 0; i < W; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (i == w) {
                Ap[e] = A[e];
                Up[e] = U[e];
            }
            const float2 m = sAgg[i][e * 64 + lane];
            U[e] = fmaf(m.x, U[e], m.y);
            A[e] *= m.x;
        }
    }
    float h[VEC];
    if constexpr (Multi) {
        chain_carry<W, VEC>(p.link, chain, p.n_tiles, k, A, U, first, sLink, w, lane, h);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = first[e];
    }
    if (w == 0 && active) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (p.ckpt) p.ckpt[(b * p.n_tiles + k) * p.dim + ch + e] = h[e];
            if (p.last && k + 1 == p.n_tiles) p.last[b * p.dim + ch + e] = fmaf(A[e], h[e], U[e]);
        }
    }
    if (!p.y) return;
    const rsrc_t ry = rows_rsrc<T>(p.y, row, p.dim, c0, p.dim, n);
    const uint32_t by = static_cast<uint32_t>(p.dim * sizeof(T));
#pragma unroll
    for (int e = 0; e < VEC; ++e) h[e] = fmaf(Ap[e], h[e], Up[e]);
#pragma unroll
    for (int i = 0; i < S; ++i) {
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            h[e] = fmaf(a[i][e], h[e], u[i][e]);
            o[e] = Z ? h[e] * silu(C::get(zr[i], e)) : h[e];
        }
        C::store(o, ry, col + i * by);
    }
}

// ---------------------------------------------------------------- gradient
struct BwdParams {
    const void *x, *g, *z, *dout;
    int64_t ldx, ldg, ldz;
    const float *bias, *ckpt, *dlast;
    void *dx, *dg, *dz;
    float *part, *dh0;           // part: dgate_bias of each (batch row, tile), or null
    int64_t seqlen;
    int dim, n_ct, n_tiles;
    uint32_t chains;
    Link link;
};

template <typename T, int VEC, int W, bool Z, bool Multi>
__global__ __launch_bounds__(W * 64) void gated_bwd_kernel(BwdParams p) {
    using C = Cell<T, VEC>;
    using raw = typename C::raw;
    constexpr int S = kBlock / W;
    constexpr bool Precise = sizeof(T) == 4;
    __shared__ float2 sAgg[W][64 * VEC];             // (A, U) of the waves, forward
    __shared__ float sRev[W][64 * VEC];              // offset of the reverse map (its decay is A too)
    __shared__ float2 sLink[Multi ? kGroup : 1][64 * VEC];
    __shared__ uint32_t sTicket;

    const int tid = threadIdx.x, lane = tid % 64;
    const int w = __builtin_amdgcn_readfirstlane(tid / 64);
    uint32_t ticket = blockIdx.x;
    if constexpr (Multi) {
        if (tid == 0) sTicket = atomicAdd(&p.link.words[0], 1u);
        __syncthreads();
        ticket = __builtin_amdgcn_readfirstlane(sTicket);
    }
    const uint32_t chain = ticket % p.chains;
    const int k = static_cast<int>(ticket / p.chains);               // in scan order: from the last tile down
    const int j = p.n_tiles - 1 - k;
    const int64_t b = chain / p.n_ct;
    const int c0 = static_cast<int>(chain % p.n_ct) * 64 * VEC;
    const int ch = c0 + lane * VEC;
    const bool active = ch < p.dim;
    const int64_t t0 = static_cast<int64_t>(j) * kBlock + w * S;
    const int64_t left = p.seqlen - t0;
    const int n = static_cast<int>(left < 0 ? 0 : (left < S ? left : S));
    const int64_t row = b * p.seqlen + t0;

    const uint32_t col = active ? static_cast<uint32_t>(lane * VEC * sizeof(T)) : kOffNone;
    const rsrc_t rx = rows_rsrc<T>(p.x, row, p.ldx, c0, p.dim, n), rg = rows_rsrc<T>(p.g, row, p.ldg, c0, p.dim, n);
    const rsrc_t rd = rows_rsrc<T>(p.dout, row, p.dim, c0, p.dim, n);
    const uint32_t bx = static_cast<uint32_t>(p.ldx * sizeof(T)), bg = static_cast<uint32_t>(p.ldg * sizeof(T));
    const uint32_t bd = static_cast<uint32_t>(p.dim * sizeof(T));
    raw xr[S], gr[S], dr[S], zr[Z ? S : 1];
#pragma unroll
    for (int i = 0; i < S; ++i) gr[i] = C::load(rg, col + i * bg);
#pragma unroll
    for (int i = 0; i < S; ++i) xr[i] = C::load(rx, col + i * bx);
    if constexpr (Z) {
        const rsrc_t rz = rows_rsrc<T>(p.z, row, p.ldz, c0, p.dim, n);
        const uint32_t bz = static_cast<uint32_t>(p.ldz * sizeof(T));
#pragma unroll
        for (int i = 0; i < S; ++i) zr[i] = C::load(rz, col + i * bz);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) dr[i] = C::load(rd, col + i * bd);
    float bias[VEC], first[VEC], h[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        bias[e] = (p.bias && active) ? p.bias[ch + e] : 0.0f;
        first[e] = (p.dlast && active) ? p.dlast[b * p.dim + ch + e] : 0.0f;
        h[e] = active ? p.ckpt[(b * p.n_tiles + j) * p.dim + ch + e] : 0.0f;
    }

    // the forward map of the wave's steps and, from its last step down, the
    // offset of c -> a (d + c).  A step past the sequence is the identity: its
    // gate is +inf (kept as 0), and its x and dout were read as 0.
    float sg[S][VEC], A[VEC], U[VEC], R[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = 1.0f;
        U[e] = 0.0f;
        R[e] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float v = signed_gate<Precise>(C::get(gr[i], e) + bias[e]);
            sg[i][e] = i < n ? v : 0.0f;
            const Gate q = split(sg[i][e]);
            U[e] = fmaf(q.a, U[e], q.s * C::get(xr[i], e));
            A[e] *= q.a;
        }
    }
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float d = C::get(dr[i], e);
            if constexpr (Z) d *= silu(C::get(zr[i], e));
            R[e] = split(sg[i][e]).a * (d + R[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        sAgg[w][e * 64 + lane] = make_float2(A[e], U[e]);
        sRev[w][e * 64 + lane] = R[e];
    }
    __syncthreads();
    float Ap[VEC], Rp[VEC];                          // the reverse map of the waves after this one
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = 1.0f;
        R[e] = 0.0f;
    }
#pragma unroll 4
    for (int i = W - 1; i >= 0; --i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (i == w) {
                Ap[e] = A[e];
                Rp[e] = R[e];
            }
            const float m = sAgg[i][e * 64 + lane].x;
            R[e] = fmaf(m, R[e], sRev[i][e * 64 + lane]);
            A[e] *= m;
        }
    }
#pragma unroll 4
    for (int i = 0; i < w; ++i) {                    // the state entering this wave's steps
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 m = sAgg[i][e * 64 + lane];
            h[e] = fmaf(m.x, h[e], m.y);
        }
    }
    float c[VEC];
    if constexpr (Multi) {
        chain_carry<W, VEC>(p.link, chain, p.n_tiles, k, A, R, first, sLink, w, lane, c);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) c[e] = first[e];
    }
    if (w == 0 && active && p.dh0 && j == 0) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p.dh0[b * p.dim + ch + e] = fmaf(A[e], c[e], R[e]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = fmaf(Ap[e], c[e], Rp[e]);

#pragma unroll
    for (int i = 0; i < S; ++i) {
        if constexpr (Z) renew(zr[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) renew(sg[i][e]);
    }
    float hb[S][VEC];                                // the state before each step
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            hb[i][e] = h[e];
            const Gate q = split(sg[i][e]);
            h[e] = fmaf(q.a, h[e], q.s * C::get(xr[i], e));
        }
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) renew(sg[i][e]);
    const rsrc_t wx = rows_rsrc<T>(p.dx, row, p.dim, c0, p.dim, n), wg = rows_rsrc<T>(p.dg, row, p.dim, c0, p.dim, n);
    const rsrc_t wz = rows_rsrc<T>(Z ? p.dz : p.dx, row, p.dim, c0, p.dim, n);
    float db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) db[e] = 0.0f;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
        float ox[VEC], og[VEC], oz[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const Gate q = split(sg[i][e]);
            const float xv = C::get(xr[i], e);
            float d = C::get(dr[i], e);
            if constexpr (Z) {
                const float zv = C::get(zr[i], e), hv = i + 1 < S ? hb[i + 1 < S ? i + 1 : i][e] : h[e];
                const Gate y = split(signed_gate<Precise>(zv));
                oz[e] = d * hv * (y.a * fmaf(zv, y.s, 1.0f));
                d *= zv * y.a;
            }
            const float ev = d + c[e];
            ox[e] = q.s * ev;
            og[e] = ev * (hb[i][e] - xv) * (q.a * q.s);
            db[e] += og[e];
            c[e] = q.a * ev;
        }
        C::store(ox, wx, col + i * bd);
        C::store(og, wg, col + i * bd);
        if constexpr (Z) C::store(oz, wz, col + i * bd);
    }
    if (p.part) {                                    // the waves' sums, added in wave order
        __syncthreads();                             // sRev was last read before the fold
#pragma unroll
        for (int e = 0; e < VEC; ++e) sRev[w][e * 64 + lane] = db[e];
        __syncthreads();
        if (w == 0 && active) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float s = 0.0f;
                for (int i = 0; i < W; ++i) s += sRev[i][e * 64 + lane];
                p.part[(b * p.n_tiles + j) * p.dim + ch + e] = s;
            }
        }
    }
}

// dgate_bias: the sum of the tiles' partial sums
__global__ __launch_bounds__(kSumThreads) void gated_dbias_kernel(const float *part, float *out, int64_t rows, int64_t dim) {
    column_sums(part, out, rows, dim);
}

// an empty sequence: the carry passes through
__global__ __launch_bounds__(256) void gated_copy_kernel(const float *in, float *out, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) out[i] = in ? in[i] : 0.0f;
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint64_t *p, int64_t n, uint32_t *words, int keep_error) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i == 0) {                                    // the header: ticket and error word
        words[0] = 0;
        if (!keep_error) words[1] = 0;
    }
    if (i < n) p[i] = 0;
}

template <typename T> __global__ __launch_bounds__(256) void gated_update_kernel(GatedStepArgs p) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= p.batch * p.dim) return;
    const float bias = p.gate_bias ? p.gate_bias[i % p.dim] : 0.0f;
    const Gate k = split(signed_gate<sizeof(T) == 4>(to_f32(static_cast<const T *>(p.g)[i]) + bias));
    const float h = fmaf(k.a, p.state[i], k.s * to_f32(static_cast<const T *>(p.x)[i]));
    p.state[i] = h;
    static_cast<T *>(p.y)[i] = from_f32<T>(p.z ? h * silu(to_f32(static_cast<const T *>(p.z)[i])) : h);
}

// ------------------------------------------------------------------- host
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Sizes do not depend on the vector width: column tiles are counted in lanes of
// one channel, of which a tile of 2 per lane takes two.
struct Layout {
    int64_t n_tiles, n_groups, cols;     // cols: d_inner rounded up to whole tiles
    size_t agg, state, total;
};
Layout layout(int64_t batch, int64_t seqlen, int64_t dim) {
    Layout l;
    l.n_tiles = (seqlen + kBlock - 1) / kBlock;
    l.n_groups = (l.n_tiles + kGroup - 1) / kGroup;
    l.cols = (dim + 127) / 128 * 128;
    l.agg = kHeader;
    l.state = l.agg + static_cast<size_t>(batch * l.cols * l.n_tiles) * 8;
    l.total = l.n_tiles > 1 ? round256(l.state + static_cast<size_t>(batch * l.cols * l.n_groups) * 8) : 0;
    return l;
}

Link make_link(const Layout &l, void *ws, uint32_t test_spin_limit) {
    char *p = static_cast<char *>(ws);
    Link k;
    k.words = reinterpret_cast<uint32_t *>(p);
    k.agg = reinterpret_cast<uint64_t *>(p + l.agg);
    k.state = reinterpret_cast<uint64_t *>(p + l.state);
    k.spin_limit = test_spin_limit ? test_spin_limit : kSpinLimit;
    k.publish = test_spin_limit ? 0 : 1;
    return k;
}
void clear(const Layout &l, const Link &k, bool keep_error, hipStream_t s) {
    const int64_t n = static_cast<int64_t>((l.total - kHeader) / 8);
    hipLaunchKernelGGL(gated_clear_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, k.agg, n,
                       k.words, keep_error ? 1 : 0);
}

bool even(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; }

template <typename T, int VEC, int W> hipError_t launch_fwd(const GatedArgs &a, hipStream_t s) {
    const Layout l = layout(a.batch, a.seqlen, a.dim);
    FwdParams p{};
    p.x = a.x; p.g = a.g; p.z = a.z; p.ldx = a.ldx; p.ldg = a.ldg; p.ldz = a.ldz;
    p.bias = a.gate_bias; p.h0 = a.h0; p.y = a.y; p.last = a.last_state; p.ckpt = a.ckpt;
    p.seqlen = a.seqlen; p.dim = static_cast<int>(a.dim);
    p.n_ct = static_cast<int>((a.dim + 64 * VEC - 1) / (64 * VEC));
    p.n_tiles = static_cast<int>(l.n_tiles);
    p.chains = static_cast<uint32_t>(a.batch * p.n_ct);
    const dim3 grid(static_cast<unsigned>(p.chains * l.n_tiles)), block(W * 64);
    const bool z = a.z && a.y;
    if (l.n_tiles > 1) {
        p.link = make_link(l, a.workspace, a.test_spin_limit);
        clear(l, p.link, false, s);
        if (z)
            hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, true, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, false, true>), grid, block, 0, s, p);
    } else if (z) {
        hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, true, false>), grid, block, 0, s, p);
    } else {
        hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, false, false>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

// the partial sums and checkpoints of the gradient, behind the hand-over words
size_t part_bytes(int64_t batch, int64_t n_tiles, int64_t dim) { return round256(static_cast<size_t>(batch * n_tiles * dim) * 4); }

template <typename T, int VEC, int W> hipError_t launch_bwd(const GatedBwdArgs &a, hipStream_t s) {
    const GatedArgs &f = a.fwd;
    const Layout l = layout(f.batch, f.seqlen, f.dim);
    char *ws = static_cast<char *>(f.workspace);
    BwdParams p{};
    float *part = reinterpret_cast<float *>(ws + l.total);
    float *ckpt = reinterpret_cast<float *>(ws + l.total + part_bytes(f.batch, l.n_tiles, f.dim));
    if (!a.ckpt) {                                   // the states entering the tiles, y unwritten
        GatedArgs q = f;
        q.y = nullptr; q.last_state = nullptr; q.ckpt = ckpt; q.z = nullptr;
        if (hipError_t e = launch_fwd<T, VEC, SSM_GATED_FWD_WAVES>(q, s)) return e;
    }
    p.x = f.x; p.g = f.g; p.z = f.z; p.dout = a.dout; p.ldx = f.ldx; p.ldg = f.ldg; p.ldz = f.ldz;
    p.bias = f.gate_bias; p.ckpt = a.ckpt ? a.ckpt : ckpt; p.dlast = a.dlast;
    p.dx = a.dx; p.dg = a.dg; p.dz = a.dz; p.dh0 = a.dh0;
    p.part = a.dgate_bias ? part : nullptr;
    p.seqlen = f.seqlen; p.dim = static_cast<int>(f.dim);
    p.n_ct = static_cast<int>((f.dim + 64 * VEC - 1) / (64 * VEC));
    p.n_tiles = static_cast<int>(l.n_tiles);
    p.chains = static_cast<uint32_t>(f.batch * p.n_ct);
    const dim3 grid(static_cast<unsigned>(p.chains * l.n_tiles)), block(W * 64);
    if (l.n_tiles > 1) {
        p.link = make_link(l, ws, f.test_spin_limit);
        clear(l, p.link, !a.ckpt, s);
        if (f.z)
            hipLaunchKernelGGL((gated_bwd_kernel<T, VEC, W, true, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((gated_bwd_kernel<T, VEC, W, false, true>), grid, block, 0, s, p);
    } else if (f.z) {
        hipLaunchKernelGGL((gated_bwd_kernel<T, VEC, W, true, false>), grid, block, 0, s, p);
    } else {
        hipLaunchKernelGGL((gated_bwd_kernel<T, VEC, W, false, false>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

size_t gated_scan_workspace(int64_t batch, int64_t seqlen, int64_t dim, int) { return layout(batch, seqlen, dim).total; }

size_t gated_scan_bwd_workspace(int64_t batch, int64_t seqlen, int64_t dim, int) {
    const Layout l = layout(batch, seqlen, dim);
    return l.total + 2 * part_bytes(batch, l.n_tiles, dim);
}

hipError_t launch_gated_scan(const GatedArgs &a, hipStream_t s) {
    constexpr int W = SSM_GATED_FWD_WAVES;
    if (a.seqlen == 0) {
        const int64_t n = a.batch * a.dim;
        if (a.last_state)
            hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, a.h0,
                               a.last_state, n);
        return hipGetLastError();
    }
    if (!a.bf16) return launch_fwd<float, 1, W>(a, s);
    const bool two = even(a.x, a.ldx) && even(a.g, a.ldg) && even(a.z, a.z ? a.ldz : 0) && even(a.y, a.dim);
    return two ? launch_fwd<bf16_t, 2, W>(a, s) : launch_fwd<bf16_t, 1, W>(a, s);
}

hipError_t launch_gated_scan_bwd(const GatedBwdArgs &a, hipStream_t s) {
    constexpr int W = SSM_GATED_BWD_WAVES;
    const GatedArgs &f = a.fwd;
    hipError_t e = hipSuccess;
    if (f.batch > 0 && f.seqlen > 0) {
        const bool two = even(f.x, f.ldx) && even(f.g, f.ldg) && even(f.z, f.z ? f.ldz : 0) && even(a.dout, f.dim) &&
                         even(a.dx, f.dim) && even(a.dg, f.dim) && even(a.dz, f.dim);
        e = !f.bf16 ? launch_bwd<float, 1, W>(a, s) : two ? launch_bwd<bf16_t, 2, W>(a, s) : launch_bwd<bf16_t, 1, W>(a, s);
    } else if (a.dh0 && f.batch > 0) {
        const int64_t n = f.batch * f.dim;
        hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, a.dlast,
                           a.dh0, n);
    }
    if (e != hipSuccess) return e;
    if (a.dgate_bias) {
        const Layout l = layout(f.batch, f.seqlen, f.dim);
        hipLaunchKernelGGL(gated_dbias_kernel, dim3(static_cast<unsigned>((f.dim + kSumCols - 1) / kSumCols)), dim3(kSumThreads), 0, s,
                           reinterpret_cast<const float *>(static_cast<char *>(f.workspace) + l.total), a.dgate_bias,
                           f.batch * l.n_tiles, f.dim);
    }
    return hipGetLastError();
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
