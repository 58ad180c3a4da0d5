// The gated linear recurrence, its gradient and its one-token form:
//     a = sigmoid(g + bias),  h <- a h + (1 - a) x,  y = h SiLU(z)
//
// One step is the affine map h -> a h + u, u = (1 - a) x, and such maps compose:
// (A1, U1) then (A2, U2) = (A2 A1, A2 U1 + U2).  There are only batch x d_inner
// chains, so time is cut into tiles of 128 steps x 64 lanes of channels.  A
// workgroup of 8 waves takes one tile; each wave holds S = 16 consecutive steps
// in registers, so every tensor is read once and written once (up to 64 steps
// take a workgroup of 1, 2 or 4 waves):
//   1. each wave discretises its steps and folds them into its (A, U);
//   2. the waves' aggregates meet in LDS and give every wave its prefix and the
//      tile its own (A, U), which is published in the workspace;
//   3. the state entering the tile is folded from what the tiles before it
//      published, on three levels (tiles, groups of 8 tiles, states after 8
//      groups); one wave waits for one of them.  The order of every fold is
//      fixed, so results do not depend on who was first;
//   4. each wave replays its steps from its own entering state and writes y.
// A tile waits only for tiles with lower tickets, which are running or done; a
// wait is bounded as in the row scan (error word, NaN state).
// The gradient is the same scan backwards over c_t = a_t e_t, with e the
// gradient of h: e_t = d_t + c_{t+1}, tiles in falling order.  It needs the
// states h_{t-1}: they are recomputed inside a tile from the state entering it,
// which the forward saves (one fp32 per channel and 128 steps).
// Bound by HBM where the tiles fill the chip: the 2.8b layer (4 x 8192 x 5120 bf16
// with z, 1342 MB) takes 237 to 243 us, 5.5 to 5.7 TB/s, as a 16-byte copy does.
// The 130m layer (8 x 2048 x 1536), 8 x 16 x 24 tiles, is a few rounds of what the chip
// holds and spends a part of its 45 + 80 us starting and draining them (4.5 TB/s).
// Tiles of 16 waves: 328 us at the 2.8b layer, as one workgroup then fills a CU.
#include <type_traits>

#include "column_sum.h"
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

constexpr int kBlock = kGatedBlock;        // steps of a tile
constexpr int kGroup = 8;                  // tiles of a group, and groups of a state
constexpr uint32_t kSpinLimit = 1u << 22;  // polls before a wait gives up
constexpr uint32_t kReady = 0x80000000u;   // set in a published word: a decay is never negative
constexpr int kWaves = 8;                  // waves of a tile
constexpr int kSteps = kGatedSteps;        // steps of a wave
static_assert(kWaves * kSteps == kBlock, "the waves hold a tile");
constexpr int kCounters = 8;               // ticket counters, each on a cache line of its own
constexpr int kCounterWords = 32;
constexpr size_t kHeader = 1280;           // word 1: the error word; from word kCounterWords on: the counters

// ------------------------------------------------------------------- gates
// a = sigmoid(v) and s = 1 - a = sigmoid(-v) from e = exp(-|v|): the smaller of
// the two is e / (1 + e), the larger 1 / (1 + e), so neither a decay near 1 nor
// its complement loses its leading digits.  An infinite v gives exactly 0 and 1.
struct Gate {
    float a, s;
};
// fp32 io: a few ulp.  v log2(e) is taken in two parts, as its rounding alone
// would cost |v| ulp; the quotient is corrected by one Newton step; the larger
// side is 1 minus the smaller, rounded once: a biased decay near 1 would
// compound over thousands of steps.
struct PreciseGate {
    static __device__ __forceinline__ float prep_bias(float b) { return b; }
    static __device__ __forceinline__ Gate eval(float g, float bias) {
        constexpr float kLog2eLo = 1.925963033500411e-08f;   // log2(e) - float(log2(e))
        const float v = g + bias;
        float av = fabsf(v);
        av = av > 128.0f ? 128.0f : av;                       // false for NaN, which stays
        const float t = av * kLog2e;
        const float lo = fmaf(av, kLog2eLo, fmaf(av, kLog2e, -t));
        float e = fast_exp2(-t);
        e = fmaf(e * -kLn2, lo, e);
        const float q = 1.0f + e, r = fast_rcp(q);
        float small = e * r;
        small = fmaf(fmaf(-q, small, e), r, small);
        const float large = 1.0f - small;
        return v < 0.0f ? Gate{small, large} : Gate{large, small};
    }
};
// bf16 io: the hardware exponential and reciprocal as they are (1 ulp each, the
// output rounds at 2^-9), log2(e) folded into the sum with the bias.
struct FastGate {
    static __device__ __forceinline__ float prep_bias(float b) { return b * kLog2e; }
    static __device__ __forceinline__ Gate eval(float g, float bias) {
        const float v = fmaf(g, kLog2e, bias);
        const float e = fast_exp2(-fabsf(v));
        const float r = fast_rcp(1.0f + e), small = e * r;
        return v < 0.0f ? Gate{small, r} : Gate{r, small};
    }
};
template <typename T> struct GateFor;
template <> struct GateFor<float> { using type = PreciseGate; };
template <> struct GateFor<bf16_t> { using type = FastGate; };

// Makes the compiler take a register as new: its value is computed here and not
// sunk to where it is used, and what was derived from it before is derived again
// and not kept.
template <typename V> __device__ __forceinline__ void renew(V &v) { asm volatile("" : "+v"(v)); }

// ------------------------------------------------- VEC channels of one row
template <typename T, int VEC> struct Cell;
template <> struct Cell<bf16_t, 2> {
    using raw = uint32_t;
    static __device__ __forceinline__ raw load(rsrc_t r, uint32_t col, uint32_t row) {
        return __builtin_amdgcn_raw_buffer_load_b32(r, col, row, kStream);
    }
    static __device__ __forceinline__ float get(raw v, int i) { return __uint_as_float(i ? (v & 0xffff0000u) : (v << 16)); }
    template <int CP> static __device__ __forceinline__ void store(const float (&v)[2], rsrc_t r, uint32_t col, uint32_t row) {
        const uint32_t lo = from_f32<bf16_t>(v[0]).bits, hi = from_f32<bf16_t>(v[1]).bits;
        __builtin_amdgcn_raw_buffer_store_b32(lo | (hi << 16), r, col, row, CP);
    }
};
template <typename T> struct Cell<T, 1> {
    using raw = typename Io<T>::raw;
    static __device__ __forceinline__ raw load(rsrc_t r, uint32_t col, uint32_t row) {
        return Io<T>::template load<kStream>(r, col, row);
    }
    static __device__ __forceinline__ float get(raw v, int) { return Io<T>::f32(v); }
    template <int CP> static __device__ __forceinline__ void store(const float (&v)[1], rsrc_t r, uint32_t col, uint32_t row) {
        Io<T>::template store<CP>(v[0], r, col, row);
    }
};

// --------------------------------------------------------------- hand-over
struct Link {
    uint32_t *error, *tickets;       // the error word, the ticket counters
    uint64_t *agg, *group, *state;   // 64 VEC words per (chain, tile), (chain, group), (chain, 8 groups)
    uint32_t spin_limit;
    int publish;
    uint32_t counters;
};

// one word (seen as v before) once it is ready; 0 when the wait gave up
__device__ __forceinline__ uint64_t wait_word(const uint64_t *p, uint64_t v, const Link &k) {
    uint32_t spins = 0;
    while (!(static_cast<uint32_t>(v) & kReady)) {
        if (++spins > k.spin_limit) {
            __hip_atomic_store(k.error, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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

// A workgroup's tile: chain and position k in scan order.  Tickets are taken in
// order, so a tile only ever waits for tiles that are running or done, whatever
// else runs on the GPU.  One counter serves one ticket in about 17 ns (a pass of
// some 3000 tiles that reads 200 MB took 58 us), so the chains are dealt to up to
// eight counters (48 us) in runs of neighbours: with every eighth chain to a
// counter the 2.8b layer took 258 us instead of 237, as workgroups then no longer
// read neighbouring columns together.  Fewer counters where the shares would not
// come out even (a short share runs ahead and leaves the rest to few workgroups).
// A workgroup starts at the counter of its XCD's number and goes on to the next
// when that one has no tiles left; as many workgroups as tiles: each finds one
// (k = n_tiles, and the workgroup leaves, only where another call runs on the same
// workspace, against the rules).
struct Tile {
    uint32_t chain;
    int k;
};
__device__ __forceinline__ Tile take_tile(const Link &lk, uint32_t chains, int n_tiles, uint32_t (&shared)[2]) {
    if (threadIdx.x == 0) {
        shared[0] = 0;
        shared[1] = static_cast<uint32_t>(n_tiles);
        const uint32_t n = lk.counters;                              // a power of two, at most `chains`
        for (uint32_t i = 0; i < n; ++i) {
            const uint32_t c = (blockIdx.x + i) & (n - 1);
            const uint32_t first = chains * c / n, mine = chains * (c + 1) / n - first;
            const uint32_t t = atomicAdd(&lk.tickets[c * kCounterWords], 1u);
            const uint32_t k = t / mine;
            if (k < static_cast<uint32_t>(n_tiles)) {
                shared[0] = first + (t - k * mine);
                shared[1] = k;
                break;
            }
        }
    }
    __syncthreads();
    return {static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(shared[0])),
            static_cast<int>(__builtin_amdgcn_readfirstlane(shared[1]))};
}

// Where a wave looks for the maps that its tile waits for: a tile of its own
// group, a group of its own state's 8 groups (or, for the last wave, that state).
// The first look is taken before the waves' folds: mostly the words are there by
// then, and their round trip is hidden.
template <int VEC> struct Ahead {
    const uint64_t *tile, *group;                    // this wave's words, or null (uniform)
    uint64_t *tiles, *groups, *states;               // of the chain, group and state at hand, to publish
    uint64_t tv[VEC], gv[VEC];
};
template <int VEC>
__device__ __forceinline__ void look_ahead(Ahead<VEC> &q, const Link &lk, int64_t chain, int n_tiles, int k, int w, int lane) {
    constexpr int kW = 64 * VEC, kSuper = kGroup * kGroup;
    const int in_group = k % kGroup, group = k / kGroup, in_super = group % kGroup, super = k / kSuper;
    const int n_groups = (n_tiles + kGroup - 1) / kGroup, n_supers = (n_tiles + kSuper - 1) / kSuper;
    q.tiles = lk.agg + (chain * n_tiles + (k - in_group)) * kW;
    q.groups = lk.group + (chain * n_groups + (group - in_super)) * kW;
    q.states = lk.state + (chain * n_supers + super) * kW;
    q.tile = w < in_group ? q.tiles + w * kW : nullptr;
    q.group = w < in_super ? q.groups + w * kW : w == kGroup - 1 && super > 0 ? q.states - kW : nullptr;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        q.tv[e] = q.gv[e] = 0;
        if (q.tile) q.tv[e] = __hip_atomic_load(q.tile + e * 64 + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (q.group) q.gv[e] = __hip_atomic_load(q.group + e * 64 + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
template <int VEC>
__device__ __forceinline__ void wait_map(const uint64_t *p, const uint64_t (&seen)[VEC], const Link &lk, int lane, float2 *slot) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const uint64_t v = wait_word(p + e * 64 + lane, seen[e], lk);
        slot[e * 64 + lane] = make_float2(word_decay(v), word_offset(v));
    }
}
// slot[0 .. n) composed onto (A, U), first to last
template <int VEC>
__device__ __forceinline__ void fold_maps(const float2 (*slot)[64 * VEC], int n, int lane, float (&A)[VEC], float (&U)[VEC]) {
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float2 m = slot[i][e * 64 + lane];
            U[e] = fmaf(m.x, U[e], m.y);
            A[e] *= m.x;
        }
    }
}

// The carry entering tile k of a chain (k counts in scan order).  Three levels:
// the tiles of a group of 8 publish their maps, the last tile of a group the
// group's map, and the last tile of 8 groups the state leaving them.  So a tile
// waits for at most 7 maps of tiles, 7 of groups and one state, each by a wave of
// its own, and only the states form a chain, one link per 64 tiles.  (With group
// states only, one link per 8 tiles, 65536 steps took 122 us.)
// (A, U) is the tile's own map, known to the wave that `publishes`, `first` the
// chain's initial carry, `h` the result, the same in every wave.
template <int W, int VEC>
__device__ __forceinline__ void chain_carry(const Link &lk, const Ahead<VEC> &q, int n_tiles, int k, const float (&A)[VEC],
                                            const float (&U)[VEC], const float (&first)[VEC],
                                            float2 (*slot)[64 * VEC], bool publishes, int w, int lane,
                                            float (&h)[VEC]) {
    static_assert(W >= kGroup, "one wave waits for one map of each level");
    constexpr int kW = 64 * VEC, kSuper = kGroup * kGroup;
    const int in_group = k % kGroup, in_super = k / kGroup % kGroup, super = k / kSuper;
    const bool more = k + 1 < n_tiles && lk.publish, last = in_group == kGroup - 1;
    float2 (*slot_g)[64 * VEC] = slot + kGroup;
    if (publishes && more && !last) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) publish_word(q.tiles + in_group * kW + e * 64 + lane, A[e], U[e]);
    }
    if (q.tile) wait_map<VEC>(q.tile, q.tv, lk, lane, slot[w]);
    if (last && in_super != kGroup - 1 && more) {    // the group's map, before anything else is waited for
        __syncthreads();
        if (publishes) {
            float Ag[VEC], Ug[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                Ag[e] = 1.0f;
                Ug[e] = 0.0f;
            }
            fold_maps<VEC>(slot, in_group, lane, Ag, Ug);
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                publish_word(q.groups + in_super * kW + e * 64 + lane, Ag[e] * A[e], fmaf(A[e], Ug[e], U[e]));
        }
    }
    if (q.group) wait_map<VEC>(q.group, q.gv, lk, lane, slot_g[w]);
    __syncthreads();
    float unused[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        h[e] = super > 0 ? slot_g[kGroup - 1][e * 64 + lane].y : first[e];
        unused[e] = 0.0f;
    }
    fold_maps<VEC>(slot_g, in_super, lane, unused, h);
    fold_maps<VEC>(slot, in_group, lane, unused, h);
    if (publishes && last && in_super == kGroup - 1 && more) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) publish_word(q.states + e * 64 + lane, 0.0f, fmaf(A[e], h[e], U[e]));
    }
}

// Row i of a wave's steps, in the scalar offset of its accesses: a step past the
// sequence reads the last valid row again (its values are replaced) and its stores
// are dropped by their lane offset, so both stay in range however the buffer unit
// counts the scalar offset.  No lane register holds a row's address.
struct RowPick {
    int n;
    __device__ __forceinline__ uint32_t operator()(int i) const {
        const int last = (n > 1 ? n : 1) - 1;        // a maximum first: a clamped subtraction is not scalar
        return static_cast<uint32_t>(i < last ? i : last);
    }
};

// ----------------------------------------------------------------- forward
struct FwdParams {
    const void *x, *g, *z;
    int64_t ldx, ldg, ldz;
    const float *bias, *h0;
    void *y;
    float *last, *ckpt;
    int seqlen, dim, n_ct, n_tiles;
    uint32_t chains;             // batch x column tiles
    Link link;
};

// the rows of a strided tensor that a wave holds, from (row, column c0) on
template <typename T> __device__ __forceinline__ rsrc_t rows_rsrc(const void *p, int64_t row, int64_t ld, int c0, int dim, int n) {
    const uint32_t bytes = n > 0 ? static_cast<uint32_t>(((n - 1) * ld + (dim - c0)) * static_cast<int64_t>(sizeof(T))) : 0u;
    return make_rsrc(static_cast<const char *>(p) + (row * ld + c0) * static_cast<int64_t>(sizeof(T)), bytes);
}

template <typename T, int VEC, int W, bool Z, bool Multi, int Store>
__global__ __launch_bounds__(W * 64) void gated_fwd_kernel(FwdParams p) {
    using C = Cell<T, VEC>;
    using G = typename GateFor<T>::type;
    using raw = typename C::raw;
    constexpr int S = kSteps;
    __shared__ float2 sAgg[W][64 * VEC];
    __shared__ float2 sLink[Multi ? 2 * kGroup : 1][64 * VEC];
    __shared__ uint32_t sTile[2];

    const int tid = threadIdx.x, lane = tid % 64;
    const int w = __builtin_amdgcn_readfirstlane(tid / 64);
    Tile tile{blockIdx.x, 0};
    if constexpr (Multi) {
        tile = take_tile(p.link, p.chains, p.n_tiles, sTile);
        if (tile.k >= p.n_tiles) return;
    }
    const uint32_t chain = tile.chain;
    const int k = tile.k;
    const int b = static_cast<int>(chain / static_cast<uint32_t>(p.n_ct));
    const int c0 = static_cast<int>(chain % static_cast<uint32_t>(p.n_ct)) * 64 * VEC;
    const int ch = c0 + lane * VEC;
    const bool active = ch < p.dim;
    const int t0 = k * kBlock + w * S;     // first step of the wave
    const int left = p.seqlen - t0;                  // 32-bit: 64-bit compares would leave the scalar unit
    const int n = left < 0 ? 0 : (left < S ? left : S);
    const int64_t row = static_cast<int64_t>(b) * p.seqlen + t0;

    const uint32_t col = active ? static_cast<uint32_t>(lane * VEC * sizeof(T)) : kOffNone;
    const RowPick at{n};
    auto keep = [&](int i) { return i < n ? col : kOffNone; };
    const rsrc_t rx = rows_rsrc<T>(p.x, row, p.ldx, c0, p.dim, n), rg = rows_rsrc<T>(p.g, row, p.ldg, c0, p.dim, n);
    const uint32_t bx = static_cast<uint32_t>(p.ldx * sizeof(T)), bg = static_cast<uint32_t>(p.ldg * sizeof(T));
    raw xr[S], gr[S], zr[Z ? S : 1];
#pragma unroll
    for (int i = 0; i < S; ++i) gr[i] = C::load(rg, col, at(i) * bg);
#pragma unroll
    for (int i = 0; i < S; ++i) xr[i] = C::load(rx, col, at(i) * bx);
    if constexpr (Z) {
        const rsrc_t rz = rows_rsrc<T>(p.z, row, p.ldz, c0, p.dim, n);
        const uint32_t bz = static_cast<uint32_t>(p.ldz * sizeof(T));
#pragma unroll
        for (int i = 0; i < S; ++i) zr[i] = C::load(rz, col, at(i) * bz);
    }
    float bias[VEC], first[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        bias[e] = (p.bias && active) ? G::prep_bias(p.bias[ch + e]) : 0.0f;
        first[e] = (p.h0 && active) ? p.h0[static_cast<int64_t>(b) * p.dim + ch + e] : 0.0f;
    }

    // discretise and fold; steps past the sequence are the identity
    float a[S][VEC], u[S][VEC], A[VEC], U[VEC];
#pragma unroll
    for (int i = 0; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const Gate q = G::eval(C::get(gr[i], e), bias[e]);
            a[i][e] = q.a;
            u[i][e] = q.s * C::get(xr[i], e);
        }
    }
    if (n < S) {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                a[i][e] = i < n ? a[i][e] : 1.0f;
                u[i][e] = i < n ? u[i][e] : 0.0f;
            }
    }
    Ahead<VEC> ahead;
    if constexpr (Multi) look_ahead<VEC>(ahead, p.link, chain, p.n_tiles, k, w, lane);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        A[e] = a[0][e];
        U[e] = u[0][e];
    }
#pragma unroll
    for (int i = 1; i < S; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
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
        Ap[e] = 1.0f;
        Up[e] = 0.0f;
    }
    fold_maps<VEC>(sAgg, w, lane, Ap, Up);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {                  // up to this wave's end; the last wave's is the tile's
        U[e] = fmaf(A[e], Up[e], U[e]);
        A[e] *= Ap[e];
    }
    float h[VEC];
    if constexpr (Multi) {
        chain_carry<W, VEC>(p.link, ahead, p.n_tiles, k, A, U, first, sLink, w == W - 1, w, lane, h);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[e] = first[e];
    }
    if (w == W - 1 && active) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            if (p.ckpt) p.ckpt[(static_cast<int64_t>(b) * p.n_tiles + k) * p.dim + ch + e] = h[e];
            if (p.last && k + 1 == p.n_tiles) p.last[static_cast<int64_t>(b) * p.dim + ch + e] = fmaf(A[e], h[e], U[e]);
        }
    }
    if (!p.y) return;
    if constexpr (Z) {                               // or SiLU(z) is held from before the carry, in twice the registers
#pragma unroll
        for (int i = 0; i < S; ++i) renew(zr[i]);
    }
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
        C::template store<Store>(o, ry, keep(i), at(i) * by);
    }
}

// ---------------------------------------------------------------- gradient
struct BwdParams {
    const void *x, *g, *z, *dout;
    int64_t ldx, ldg, ldz;
    const float *bias, *ckpt, *dlast;
    void *dx, *dg, *dz;
    float *part, *dh0;           // part: dgate_bias of each (batch row, tile), or null
    int seqlen, dim, n_ct, n_tiles;
    uint32_t chains;
    Link link;
};

// One channel per lane: a step's values (a, 1 - a, x, the two factors of dout and
// the state) take six registers per step and channel, and two workgroups per CU
// overlap better than wider lanes at one (at the 130m layer 80 us against 96 us).
template <typename T, int W, bool Z, bool Multi, int Store>
__global__ __launch_bounds__(W * 64) void gated_bwd_kernel(BwdParams p) {
    using C = Cell<T, 1>;
    using G = typename GateFor<T>::type;
    using raw = typename C::raw;
    constexpr int S = kSteps;
    __shared__ float2 sAgg[W][64];                   // (A, U) of the waves, forward
    __shared__ float2 sRev[W][64];                   // the reverse maps (the same A, R)
    __shared__ float2 sLink[Multi ? 2 * kGroup : 1][64];
    __shared__ uint32_t sTile[2];

    const int tid = threadIdx.x, lane = tid % 64;
    const int w = __builtin_amdgcn_readfirstlane(tid / 64);
    Tile tile{blockIdx.x, 0};
    if constexpr (Multi) {
        tile = take_tile(p.link, p.chains, p.n_tiles, sTile);
        if (tile.k >= p.n_tiles) return;
    } else if (blockIdx.x == 0 && threadIdx.x == 0) {
        *p.link.error = 0;                           // no wait, no clear launch before this one
    }
    const uint32_t chain = tile.chain;
    const int k = tile.k;                            // in scan order: from the last tile down
    const int j = p.n_tiles - 1 - k;
    const int b = static_cast<int>(chain / static_cast<uint32_t>(p.n_ct));
    const int c0 = static_cast<int>(chain % static_cast<uint32_t>(p.n_ct)) * 64;
    const int ch = c0 + lane;
    const bool active = ch < p.dim;
    const int t0 = j * kBlock + w * S;
    const int left = p.seqlen - t0;                  // 32-bit: 64-bit compares would leave the scalar unit
    const int n = left < 0 ? 0 : (left < S ? left : S);
    const int64_t row = static_cast<int64_t>(b) * p.seqlen + t0;

    const uint32_t col = active ? static_cast<uint32_t>(lane * sizeof(T)) : kOffNone;
    const RowPick at{n};
    auto keep = [&](int i) { return i < n ? col : kOffNone; };
    const rsrc_t rx = rows_rsrc<T>(p.x, row, p.ldx, c0, p.dim, n), rg = rows_rsrc<T>(p.g, row, p.ldg, c0, p.dim, n);
    const rsrc_t rd = rows_rsrc<T>(p.dout, row, p.dim, c0, p.dim, n);
    const uint32_t bx = static_cast<uint32_t>(p.ldx * sizeof(T)), bg = static_cast<uint32_t>(p.ldg * sizeof(T));
    const uint32_t bd = static_cast<uint32_t>(p.dim * sizeof(T));
    raw xr[S], gr[S], dr[S], zr[Z ? S : 1];
#pragma unroll
    for (int i = 0; i < S; ++i) gr[i] = C::load(rg, col, at(i) * bg);
#pragma unroll
    for (int i = 0; i < S; ++i) xr[i] = C::load(rx, col, at(i) * bx);
    if constexpr (Z) {
        const rsrc_t rz = rows_rsrc<T>(p.z, row, p.ldz, c0, p.dim, n);
        const uint32_t bz = static_cast<uint32_t>(p.ldz * sizeof(T));
#pragma unroll
        for (int i = 0; i < S; ++i) zr[i] = C::load(rz, col, at(i) * bz);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) dr[i] = C::load(rd, col, at(i) * bd);
    const float bias = (p.bias && active) ? G::prep_bias(p.bias[ch]) : 0.0f;
    const float first[1] = {(p.dlast && active) ? p.dlast[static_cast<int64_t>(b) * p.dim + ch] : 0.0f};
    float h = active ? p.ckpt[(static_cast<int64_t>(b) * p.n_tiles + j) * p.dim + ch] : 0.0f;

    // The gates, x, and dout's factors: dh = dout SiLU(z) (dout without z) and
    // dz / h = dout SiLU'(z), SiLU' = s + SiLU (1 - s) with s = sigmoid(z).  A
    // step past the sequence is the identity: a = 1 and no gradient of its own.
    float a[S], s[S], x[S], dh[S], dzh[Z ? S : 1];
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const Gate q = G::eval(C::get(gr[i], 0), bias);
        a[i] = q.a;
        s[i] = q.s;
        x[i] = C::get(xr[i], 0);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
        dh[i] = C::get(dr[i], 0);
        if constexpr (Z) {
            const float zv = C::get(zr[i], 0);
            const Gate y = G::eval(zv, 0.0f);
            const float sl = zv * y.a;
            dzh[i] = dh[i] * fmaf(sl, y.s, y.a);
            dh[i] *= sl;
            renew(dzh[i]);                           // or its factors wait for the last loop in two registers
            renew(dh[i]);
        }
    }
    if (n < S) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
            a[i] = i < n ? a[i] : 1.0f;
            s[i] = i < n ? s[i] : 0.0f;
            x[i] = i < n ? x[i] : 0.0f;
            dh[i] = i < n ? dh[i] : 0.0f;
        }
    }
    Ahead<1> ahead;
    if constexpr (Multi) look_ahead<1>(ahead, p.link, chain, p.n_tiles, k, w, lane);
    // the forward map of the wave's steps, and the reverse map c -> a (dh + c)
    // from its last step down
    float A[1] = {a[0]}, U = s[0] * x[0], R[1] = {a[S - 1] * dh[S - 1]};
#pragma unroll
    for (int i = 1; i < S; ++i) {
        U = fmaf(a[i], U, s[i] * x[i]);
        A[0] *= a[i];
    }
#pragma unroll
    for (int i = S - 2; i >= 0; --i) R[0] = a[i] * (dh[i] + R[0]);
    sAgg[w][lane] = make_float2(A[0], U);
    sRev[w][lane] = make_float2(A[0], R[0]);
    __syncthreads();
    float Ap = 1.0f, Rp = 0.0f;                      // the reverse map of the waves after this one
#pragma unroll 4
    for (int i = W - 1; i > w; --i) {
        const float2 m = sRev[i][lane];
        Rp = fmaf(m.x, Rp, m.y);
        Ap *= m.x;
    }
    R[0] = fmaf(A[0], Rp, R[0]);                     // down to this wave's first step; wave 0's is the tile's
    A[0] *= Ap;
#pragma unroll 4
    for (int i = 0; i < w; ++i) {                    // the state entering this wave's steps
        const float2 m = sAgg[i][lane];
        h = fmaf(m.x, h, m.y);
    }
    float c[1];
    if constexpr (Multi)
        chain_carry<W, 1>(p.link, ahead, p.n_tiles, k, A, R, first, sLink, w == 0, w, lane, c);
    else
        c[0] = first[0];
    if (w == 0 && active && p.dh0 && j == 0) p.dh0[static_cast<int64_t>(b) * p.dim + ch] = fmaf(A[0], c[0], R[0]);
    float cc = fmaf(Ap, c[0], Rp);

#pragma unroll
    for (int i = 0; i < S; ++i) renew(x[i]);
    float hb[S];                                     // the state before each step
#pragma unroll
    for (int i = 0; i < S; ++i) {
        hb[i] = h;
        h = fmaf(a[i], h, s[i] * x[i]);
    }
    const rsrc_t wx = rows_rsrc<T>(p.dx, row, p.dim, c0, p.dim, n), wg = rows_rsrc<T>(p.dg, row, p.dim, c0, p.dim, n);
    const rsrc_t wz = rows_rsrc<T>(Z ? p.dz : p.dx, row, p.dim, c0, p.dim, n);
    float db = 0.0f;
#pragma unroll
    for (int i = S - 1; i >= 0; --i) {
        const float ev = dh[i] + cc;
        const float ox[1] = {s[i] * ev}, og[1] = {ev * (hb[i] - x[i]) * (a[i] * s[i])};
        db += og[0];
        cc = a[i] * ev;
        C::template store<Store>(ox, wx, keep(i), at(i) * bd);
        C::template store<Store>(og, wg, keep(i), at(i) * bd);
        if constexpr (Z) {
            const float oz[1] = {dzh[i] * (i + 1 < S ? hb[i + 1 < S ? i + 1 : i] : h)};
            C::template store<Store>(oz, wz, keep(i), at(i) * bd);
        }
    }
    if (p.part) {                                    // the waves' sums, added in wave order
        __syncthreads();                             // sRev was last read before the carry
        sRev[w][lane].x = db;
        __syncthreads();
        if (w == 0 && active) {
            float sum = 0.0f;
            for (int i = 0; i < W; ++i) sum += sRev[i][lane].x;
            p.part[(static_cast<int64_t>(b) * p.n_tiles + j) * p.dim + ch] = sum;
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

// clears header and hand-over words, 16 bytes at a time
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
__global__ __launch_bounds__(256) void gated_clear_kernel(u4 *p, int64_t n) {
    const u4 zero = {0, 0, 0, 0};
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
        p[i] = zero;
}

// One token: V channels per lane (4 where the width and the addresses allow 8- and
// 16-byte accesses).
template <typename T, int V> __global__ __launch_bounds__(256) void gated_update_kernel(GatedStepArgs p) {
    using G = typename GateFor<T>::type;
    struct alignas(V * sizeof(T)) Io4 {
        T v[V];
    };
    struct alignas(V * 4) F4 {
        float v[V];
    };
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, n = static_cast<uint32_t>(p.batch * p.dim / V);
    if (i >= n) return;
    const uint32_t d = i % static_cast<uint32_t>(p.dim / V);
    const Io4 g = static_cast<const Io4 *>(p.g)[i], x = static_cast<const Io4 *>(p.x)[i];
    F4 h = reinterpret_cast<const F4 *>(p.state)[i], bias{};
    Io4 z{}, y;
    if (p.z) z = static_cast<const Io4 *>(p.z)[i];
    if (p.gate_bias) bias = reinterpret_cast<const F4 *>(p.gate_bias)[d];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const Gate k = G::eval(to_f32(g.v[e]), G::prep_bias(bias.v[e]));
        h.v[e] = fmaf(k.a, h.v[e], k.s * to_f32(x.v[e]));
        y.v[e] = from_f32<T>(p.z ? h.v[e] * silu(to_f32(z.v[e])) : h.v[e]);
    }
    reinterpret_cast<F4 *>(p.state)[i] = h;
    static_cast<Io4 *>(p.y)[i] = y;
}

// ------------------------------------------------------------------- host
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Sizes do not depend on the vector width: column tiles are counted in lanes of
// one channel, of which a tile of 2 per lane takes two.
struct Layout {
    int64_t n_tiles, cols;               // cols: d_inner rounded up to whole tiles
    size_t agg, group, state, total;
};
Layout layout(int64_t batch, int64_t seqlen, int64_t dim) {
    Layout l;
    l.n_tiles = batch * dim > 0 ? (seqlen + kBlock - 1) / kBlock : 0;
    const int64_t n_groups = (l.n_tiles + kGroup - 1) / kGroup, n_supers = (n_groups + kGroup - 1) / kGroup;
    l.cols = (dim + 127) / 128 * 128;
    l.agg = kHeader;
    l.group = l.agg + static_cast<size_t>(batch * l.cols * l.n_tiles) * 8;
    l.state = l.group + static_cast<size_t>(batch * l.cols * n_groups) * 8;
    l.total = l.n_tiles > 1 ? round256(l.state + static_cast<size_t>(batch * l.cols * n_supers) * 8) : 0;
    return l;
}

// error: the workspace's error word, in its first region
Link make_link(const Layout &l, char *region, uint32_t *error, uint32_t chains, uint32_t test_spin_limit) {
    Link k;
    k.counters = kCounters;
    // shares of at least 6 chains (12 chains on four counters: 127 us for 65536
    // steps, on two: 122 us), and even ones below 20
    while (k.counters > 1 && (chains < 6 * k.counters || (chains % k.counters != 0 && chains < 20 * k.counters)))
        k.counters /= 2;
    k.error = error;
    k.tickets = reinterpret_cast<uint32_t *>(region) + kCounterWords;
    k.agg = reinterpret_cast<uint64_t *>(region + l.agg);
    k.group = reinterpret_cast<uint64_t *>(region + l.group);
    k.state = reinterpret_cast<uint64_t *>(region + l.state);
    k.spin_limit = test_spin_limit ? test_spin_limit : kSpinLimit;
    k.publish = test_spin_limit ? 0 : 1;
    return k;
}
uint32_t *error_word(void *workspace) { return static_cast<uint32_t *>(workspace) + 1; }
void clear(void *region, size_t bytes, hipStream_t s) {
    const int64_t n = static_cast<int64_t>(bytes / 16), wgs = (n + 255) / 256;
    hipLaunchKernelGGL(gated_clear_kernel, dim3(static_cast<unsigned>(wgs < 1024 ? wgs : 1024)), dim3(256), 0, s,
                       static_cast<u4 *>(region), n);
}

bool even(const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 4 == 0 && ld % 2 == 0; }

// launch(waves, whether there are several tiles to a chain): as many waves as the
// steps of a sequence need, in powers of two (1024 x 16 x 1536 bf16 with z: 39 us
// instead of 168 us with eight waves to every workgroup, its gradient 80 us instead
// of 380 us).
template <typename F> void with_waves(int64_t seqlen, F launch) {
    if (seqlen > kBlock) return launch(std::integral_constant<int, kWaves>(), std::true_type());
    switch (gated_waves(seqlen)) {
    case 8: return launch(std::integral_constant<int, 8>(), std::false_type());
    case 4: return launch(std::integral_constant<int, 4>(), std::false_type());
    case 2: return launch(std::integral_constant<int, 2>(), std::false_type());
    default: return launch(std::integral_constant<int, 1>(), std::false_type());
    }
}

template <typename T, int VEC, int Store> hipError_t launch_fwd(const GatedArgs &a, bool cleared, hipStream_t s) {
    const Layout l = layout(a.batch, a.seqlen, a.dim);
    FwdParams p{};
    p.x = a.x; p.g = a.g; p.z = a.z; p.ldx = a.ldx; p.ldg = a.ldg; p.ldz = a.ldz;
    p.bias = a.gate_bias; p.h0 = a.h0; p.y = a.y; p.last = a.last_state; p.ckpt = a.ckpt;
    p.seqlen = static_cast<int>(a.seqlen); p.dim = static_cast<int>(a.dim);
    p.n_ct = static_cast<int>((a.dim + 64 * VEC - 1) / (64 * VEC));
    p.n_tiles = static_cast<int>(l.n_tiles);
    p.chains = static_cast<uint32_t>(a.batch * p.n_ct);
    const dim3 grid(static_cast<unsigned>(p.chains * l.n_tiles));
    const bool z = a.z && a.y;
    if (l.n_tiles > 1) {
        p.link = make_link(l, static_cast<char *>(a.workspace), error_word(a.workspace), p.chains, a.test_spin_limit);
        if (!cleared) clear(a.workspace, l.total, s);
    }
    with_waves(a.seqlen, [&](auto waves, auto multi) {
        constexpr int W = decltype(waves)::value;
        constexpr bool M = decltype(multi)::value;
        if (z)
            hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, true, M, Store>), grid, dim3(W * 64), 0, s, p);
        else
            hipLaunchKernelGGL((gated_fwd_kernel<T, VEC, W, false, M, Store>), grid, dim3(W * 64), 0, s, p);
    });
    return hipGetLastError();
}

// Whether a wave's row segments fill whole 128-byte lines of an output, row after
// row.  Non-temporal stores then spare the caches; where a line is shared by two
// tiles they would write it to memory twice in part, so those go through the L2
// (4 x 4096 x 2561 bf16 with z: gradient 174 us against 235 us, forward 96 against
// 121 us; at 2560 channels the other way round, 133 against 128 us).  Pairs of channels
// go by the same rule: 4 x 8192 x 2562 bf16 with z 159 us through the L2 against 174 us,
// 5120 channels 252 against 247 us.
bool whole_lines(const void *p, int64_t row_bytes) { return reinterpret_cast<uintptr_t>(p) % 128 == 0 && row_bytes % 128 == 0; }

// bf16 in pairs of channels where every row starts on 4 bytes: whole-line accesses
// of a wave (the 2.8b layer 243 us against 248 us with one channel per lane), unless
// the tiles are then too few for more than a few rounds on the chip (8 x 2048 x 1536,
// 1536 tiles of pairs, 48.6 us against 45.1 us; 32768 steps of 64 channels 18.4
// against 15.0 us).
constexpr int64_t kPairTiles = 4096;
hipError_t dispatch_fwd(const GatedArgs &a, bool cleared, hipStream_t s) {
    const bool lines = whole_lines(a.y, a.dim * (a.bf16 ? 2 : 4));
    if (!a.bf16) return lines ? launch_fwd<float, 1, kStream>(a, cleared, s) : launch_fwd<float, 1, kCached>(a, cleared, s);
    const bool two = even(a.x, a.ldx) && even(a.g, a.ldg) && even(a.z, a.z ? a.ldz : 0) && even(a.y, a.dim);
    const int64_t pair_tiles = a.batch * ((a.dim + 127) / 128) * layout(a.batch, a.seqlen, a.dim).n_tiles;
    if (two && pair_tiles >= kPairTiles)
        return lines ? launch_fwd<bf16_t, 2, kStream>(a, cleared, s) : launch_fwd<bf16_t, 2, kCached>(a, cleared, s);
    return lines ? launch_fwd<bf16_t, 1, kStream>(a, cleared, s) : launch_fwd<bf16_t, 1, kCached>(a, cleared, s);
}

// The workspace of the gradient: the hand-over of the pass that computes the
// checkpoints, the gradient's own, partial sums, checkpoints.  With one tile per
// chain there is nothing to hand over, but the error word keeps its place.
size_t parts_at(const Layout &l) { return l.n_tiles > 1 ? 2 * l.total : l.n_tiles * 256; }
size_t part_bytes(int64_t batch, int64_t n_tiles, int64_t dim) { return round256(static_cast<size_t>(batch * n_tiles * dim) * 4); }

template <typename T, int Store> hipError_t launch_bwd(const GatedBwdArgs &a, hipStream_t s) {
    const GatedArgs &f = a.fwd;
    const Layout l = layout(f.batch, f.seqlen, f.dim);
    char *ws = static_cast<char *>(f.workspace);
    BwdParams p{};
    float *part = reinterpret_cast<float *>(ws + parts_at(l));
    float *ckpt = reinterpret_cast<float *>(ws + parts_at(l) + part_bytes(f.batch, l.n_tiles, f.dim));
    // one region of hand-over words for each pass, cleared together
    char *region = a.ckpt ? ws : ws + l.total;
    if (l.total) clear(ws, (a.ckpt ? 1 : 2) * l.total, s);
    if (!a.ckpt) {                                   // the states entering the tiles, y unwritten
        GatedArgs q = f;
        q.y = nullptr; q.last_state = nullptr; q.ckpt = ckpt; q.z = nullptr;
        if (hipError_t e = dispatch_fwd(q, true, s)) return e;
    }
    p.x = f.x; p.g = f.g; p.z = f.z; p.dout = a.dout; p.ldx = f.ldx; p.ldg = f.ldg; p.ldz = f.ldz;
    p.bias = f.gate_bias; p.ckpt = a.ckpt ? a.ckpt : ckpt; p.dlast = a.dlast;
    p.dx = a.dx; p.dg = a.dg; p.dz = a.dz; p.dh0 = a.dh0;
    p.part = a.dgate_bias ? part : nullptr;
    p.seqlen = static_cast<int>(f.seqlen); p.dim = static_cast<int>(f.dim);
    p.n_ct = static_cast<int>((f.dim + 63) / 64);
    p.n_tiles = static_cast<int>(l.n_tiles);
    p.chains = static_cast<uint32_t>(f.batch * p.n_ct);
    p.link.error = error_word(ws);
    const dim3 grid(static_cast<unsigned>(p.chains * l.n_tiles));
    if (l.n_tiles > 1) p.link = make_link(l, region, error_word(ws), p.chains, f.test_spin_limit);
    with_waves(f.seqlen, [&](auto waves, auto multi) {
        constexpr int W = decltype(waves)::value;
        constexpr bool M = decltype(multi)::value;
        if (f.z)
            hipLaunchKernelGGL((gated_bwd_kernel<T, W, true, M, Store>), grid, dim3(W * 64), 0, s, p);
        else
            hipLaunchKernelGGL((gated_bwd_kernel<T, W, false, M, Store>), grid, dim3(W * 64), 0, s, p);
    });
    return hipGetLastError();
}

}  // namespace

size_t gated_scan_workspace(int64_t batch, int64_t seqlen, int64_t dim, int) { return layout(batch, seqlen, dim).total; }

size_t gated_scan_bwd_workspace(int64_t batch, int64_t seqlen, int64_t dim, int) {
    const Layout l = layout(batch, seqlen, dim);
    return parts_at(l) + 2 * part_bytes(batch, l.n_tiles, dim);
}

hipError_t launch_gated_scan(const GatedArgs &a, hipStream_t s) {
    if (a.seqlen == 0) {
        const int64_t n = a.batch * a.dim;
        if (a.last_state)
            hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, a.h0,
                               a.last_state, n);
        return hipGetLastError();
    }
    return dispatch_fwd(a, false, s);
}

hipError_t launch_gated_scan_bwd(const GatedBwdArgs &a, hipStream_t s) {
    const GatedArgs &f = a.fwd;
    hipError_t e = hipSuccess;
    if (f.batch > 0 && f.seqlen > 0) {
        const int64_t row = f.dim * (f.bf16 ? 2 : 4);
        const bool lines = whole_lines(a.dx, row) && whole_lines(a.dg, row) && whole_lines(a.dz, row);
        if (f.bf16)
            e = lines ? launch_bwd<bf16_t, kStream>(a, s) : launch_bwd<bf16_t, kCached>(a, s);
        else
            e = lines ? launch_bwd<float, kStream>(a, s) : launch_bwd<float, kCached>(a, s);
    } else if (a.dh0 && f.batch > 0) {
        const int64_t n = f.batch * f.dim;
        hipLaunchKernelGGL(gated_copy_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, a.dlast,
                           a.dh0, n);
    }
    if (e != hipSuccess) return e;
    if (a.dgate_bias) {
        const Layout l = layout(f.batch, f.seqlen, f.dim);
        hipLaunchKernelGGL(gated_dbias_kernel, dim3(static_cast<unsigned>((f.dim + kSumCols - 1) / kSumCols)), dim3(kSumThreads), 0, s,
                           reinterpret_cast<const float *>(static_cast<char *>(f.workspace) + parts_at(l)), a.dgate_bias,
                           f.batch * l.n_tiles, f.dim);
    }
    return hipGetLastError();
}

namespace {
template <typename T> hipError_t launch_update(const GatedStepArgs &a, hipStream_t s) {
    const uintptr_t io = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.g) |
                         reinterpret_cast<uintptr_t>(a.z) | reinterpret_cast<uintptr_t>(a.y);
    const uintptr_t f32 = reinterpret_cast<uintptr_t>(a.state) | reinterpret_cast<uintptr_t>(a.gate_bias);
    const bool four = a.dim % 4 == 0 && io % (4 * sizeof(T)) == 0 && f32 % 16 == 0;
    const int64_t lanes = a.batch * a.dim / (four ? 4 : 1);
    const dim3 grid(static_cast<unsigned>((lanes + 255) / 256)), block(256);
    if (four)
        hipLaunchKernelGGL((gated_update_kernel<T, 4>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((gated_update_kernel<T, 1>), grid, block, 0, s, a);
    return hipGetLastError();
}
}  // namespace

hipError_t launch_gated_update(const GatedStepArgs &a, hipStream_t s) {
    return a.bf16 ? launch_update<bf16_t>(a, s) : launch_update<float>(a, s);
}

}  // namespace ssm
