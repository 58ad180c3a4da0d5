// The gradient of the gated delta rule.  With dS' = dL/dS' of the state S' that a
// chunk leaves, per chunk (all of delta_chunk.h's names; F, E lower triangular):
//     dU = scale P^T dY + exp(G_end - G) K dS',   dX = T^T (beta dU) = dV
//     dS = exp(G_end) dS' + scale Q^T (exp(G) dY) - K^T (exp(G) dX)
//     F = scale (dY R^T) o Gam,   E = (dX R^T) o Gam below the diagonal,   M = -E diag(beta)
//     dQ = scale exp(G) dY S^T + F diag(beta) K
//     dK = dKe + beta Z,  dKe = M K - exp(G) dX S^T,  Z = F^T Q - E^T K + exp(G_end - G) R dS'^T
//     dbeta_t = k_t . Z_t
//     dg_t = sum over t' >= t of (q . dq + k . dke - beta k . z)_t'  + <S', dS'>
// dg's form: G_t enters every product as exp(G_t) beside q_t and the key that is
// read with, and as exp(-G_t) beside the key that is written with, so the
// derivative by G_t is the product with what stands beside it.  <S', dS'> =
// exp(G_end) <S, dS'> + sum_t beta k_t . (exp(G_end - G) R dS'^T)_t.  Z is the gradient by
// the key that is written with, before beta; dbeta needs neither dU nor a division.
//
// Launches: the chunks' preparation; without saved ones, the states entering the
// chunks and R, in a walk over the chunks; dS' and dX, in a walk backwards, cut into
// time segments as the forward is; the rest, all chunks at once.
#include "delta_flow.h"

namespace ssm {
namespace delta {
namespace {

struct BwdParams {
    DeltaBwdArgs b;
    ChunkWs ws;
    float *dX, *dS;                // per (slot, head): (64, V), (V, K)
    SeqParams seq;                 // the time segments, their ends and transitions
};
// A segment of the walk backwards: where it starts and what it has to do.
struct RevPart {
    int64_t head, kh, seq, edge, lastrow, lastunit;
    int tile, vt, nch, n;          // n: steps of the chunk that it starts with
    bool first, last, transition, used;
};
template <int KP, bool ENDS, int NW> __device__ __forceinline__ RevPart rev_part(const BwdParams &p) {
    constexpr int wide = 16 * NW;
    const DeltaShape &sh = p.b.fwd.s;
    const int64_t H = sh.heads;
    const int nvt = (static_cast<int>(sh.dv) + wide - 1) / wide, tiles = ENDS ? nvt + (KP + wide - 1) / wide : nvt;
    const int64_t per_tile = gridDim.x / tiles, rest = blockIdx.x % per_tile;
    RevPart r{};
    r.tile = static_cast<int>(blockIdx.x / per_tile);
    r.head = rest % H;
    r.kh = r.head / (H / sh.kheads);
    Span sp;
    const Segment sg = segment_of<ENDS ? kBehindEdges : kAllSegments>(sh, rest / H, p.seq.edges, p.seq.cps, sp);
    r.seq = sg.seq;
    r.edge = sg.edge;
    r.first = sg.s == 0;
    r.last = sg.last;
    r.transition = ENDS && r.tile >= nvt;
    r.used = sg.used && !(ENDS && r.last && r.transition);
    r.vt = r.transition ? 0 : r.tile;
    r.tile -= nvt;
    r.nch = sg.j1 - sg.j0;
    r.n = sp.len - (sg.j1 - 1) * kC < kC ? sp.len - (sg.j1 - 1) * kC : kC;
    r.lastrow = sp.row0 + static_cast<int64_t>(sg.j1 - 1) * kC;
    r.lastunit = (sp.slot0 + sg.j1 - 1) * H + r.head;
    return r;
}
template <int KP, bool ENDS> __device__ __forceinline__ void rev_start(f32x4 (&dS)[KP / 16], const BwdParams &p, const RevPart &r, int wide, int v0, int w, int lane) {
    const DeltaArgs &a = p.b.fwd;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const size_t VK = static_cast<size_t>(V) * K;
    if (r.transition) {
        unit_columns<KP>(dS, r.tile * wide + w * 16, lane);
    } else if (!ENDS && !r.last) {
        load_state<KP>(dS, p.seq.ends + ((r.edge + 1) * a.s.heads + r.head) * VK, v0, V, K, lane);
    } else if (r.last && p.b.dlast) {
        load_state<KP>(dS, p.b.dlast + (r.seq * a.s.heads + r.head) * VK, v0, V, K, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KP / 16; ++i) dS[i] = f32x4{0, 0, 0, 0};
    }
}
template <typename T, int KP, bool ENDS, int NW>
__device__ __forceinline__ void rev_end(const f32x4 (&dS)[KP / 16], const BwdParams &p, const RevPart &r, char *smem, int v0, int w, int lane) {
    const DeltaArgs &a = p.b.fwd;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const size_t VK = static_cast<size_t>(V) * K;
    const int64_t unit = r.edge * a.s.heads + r.head;
    if constexpr (ENDS) {
        if (r.transition) store_map<T, KP, NW>(dS, smem, w, lane, p.seq.maps + unit * kMapBytes<KP>, r.tile * 16 * NW);
        else store_state<KP>(dS, p.seq.ends + unit * VK, v0, V, K, lane);
    } else if (r.first && p.b.dh0) {
        store_state<KP>(dS, p.b.dh0 + (r.seq * a.s.heads + r.head) * VK, v0, V, K, lane);
    }
}

// What get_col reads of a chunk that is used with steps along K only.
template <typename T, int KP> struct QSide : Cols<KP> {};
template <int KP> struct QSide<bf16_t, KP> : Rows<bf16_t, KP> {
    static __device__ __forceinline__ uint32_t offsets(int64_t ld, int K, int thread) { return Rows<bf16_t, KP>::offset(ld, K, thread); }
};

// --------------------------------------------------------- dS and dX, in reverse
template <int KP, bool ENDS> __global__ __launch_bounds__(kThreads) void delta_rev_kernel(BwdParams p) {
    using T = float;
    constexpr int KT = KP / 16, KK = KP / 32, RB = kRowBytes<T>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    // rows and columns of the keys, columns of the queries
    char *const sK = smem, *const sC = sK + Rows<T, KP>::kBytes, *const sQ = sC + Cols<KP>::kBytes,
         *const sT = sQ + QSide<T, KP>::kBytes, *const sP = sT + kTriBytes;
    float *const sS = reinterpret_cast<float *>(sP + kTriBytes);
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    const RevPart r = rev_part<KP, ENDS, kWaves>(p);
    if (!r.used) return;
    const int64_t head = r.head, kh = r.kh;
    const int v0 = r.vt * 64 + w * 16;
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    constexpr int es = sizeof(T);
    f32x4 dS[KT];
    rev_start<KP, ENDS>(dS, p, r, 64, v0, w, lane);
    // the next chunk's data, a chunk ahead, as in the forward
    Rows<T, KP> nK;
    Cols<KP> nC;
    QSide<T, KP> nQ;
    Copy<kTriBytes> nT, nP;
    float nS;
    Values nY;
    const uint32_t okr = Rows<T, KP>::offset(a.ldk, K, threadIdx.x);
    const auto okc = Cols<KP>::offsets(a.ldk, K, threadIdx.x);
    const auto oqc = QSide<T, KP>::offsets(a.ldq, K, threadIdx.x);
    const int ldy = static_cast<int>(H * V);
    const uint32_t oy = Values::offset(ldy, V - r.vt * 64, w, lane);
    auto prefetch = [&](int j) {                           // the j-th chunk from the end; past the first one nothing is read
        const int jj = j < r.nch ? j : r.nch - 1, n = j < r.nch ? (j == 0 ? r.n : kC) : 0;
        const int64_t row0 = r.lastrow - static_cast<int64_t>(jj) * kC, unit = r.lastunit - jj * H;
        const rsrc_t rk = chunk_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, n, a.ldk, K, es);
        const rsrc_t rd = chunk_rsrc(static_cast<const T *>(p.b.dout) + (row0 * H + head) * V + r.vt * 64, r.transition ? 0 : n, ldy, V - r.vt * 64, es);
        nK.load(rk, a.ldk, okr);
        nY.load(rd, ldy, oy);
        nT.load(p.ws.tt + unit * kTriBytes);
        nP.load(p.ws.p + unit * kTriBytes);
        nS = p.ws.scal[unit * 3 * kC + (threadIdx.x < 3 * kC ? threadIdx.x : 0)];
        nC.load(rk, a.ldk, okc);
        nQ.load(chunk_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K, n, a.ldq, K, es), a.ldq, oqc);
    };
    if (r.nch > 0) prefetch(0);
    for (int j = 0; j < r.nch; ++j) {
        const int64_t row0 = r.lastrow - static_cast<int64_t>(j) * kC, unit = r.lastunit - j * H;
        const int n = j == 0 ? r.n : kC;
        __syncthreads();                                   // the chunk before is done with LDS
        nK.put(sK, threadIdx.x);
        nC.put(sC, threadIdx.x);
        nQ.put(sQ, threadIdx.x);
        nT.put(sT);
        nP.put(sP);
        if (threadIdx.x < 3 * kC) sS[threadIdx.x] = nS;
        const Values cY = nY;
        __syncthreads();
        if constexpr (!ENDS) store_state<KP>(dS, p.dS + unit * VK, v0, V, K, lane);
        prefetch(j + 1);
        const Op<T> yo[2] = {cY.op(0), cY.op(1)};
        Op2<T> so[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) so[kk] = computed<T>(dS[2 * kk], dS[2 * kk + 1]);
        f32x4 dU[4] = {zero, zero, zero, zero}, pd[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) dU[tb] = mma(get_row(sK + (tb * KK + kk) * RB, lane, T()), so[kk], dU[tb]);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 0; tb < 2 * kk + 2; ++tb) pd[tb] = mma(get_op2(sP + tri_up(tb, kk) * kOp2Bytes, lane, T()), yo[kk], pd[tb]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = 32 * (tb / 2) + 8 * g + 4 * (tb % 2);
            dU[tb] = dU[tb] * *reinterpret_cast<const f32x4 *>(&sS[kC + t]) + pd[tb] * a.scale;
            dU[tb] = dU[tb] * *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t]);
        }
        const Op2<T> uo[2] = {computed<T>(dU[0], dU[1]), computed<T>(dU[2], dU[3])};
        const rsrc_t rv = chunk_rsrc(static_cast<T *>(p.b.dv) + (row0 * H + head) * V, n, ldy, V, es);
        const rsrc_t rx = make_rsrc(p.dX + unit * kC * V, static_cast<uint32_t>(kC * V * 4));
        // dX for the state, and transposed for stores of four channels
        f32x4 dX[4] = {zero, zero, zero, zero}, xt[4] = {zero, zero, zero, zero}, dY[4];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 0; tb < 2 * kk + 2; ++tb) {
                const Op2<T> tt = get_op2(sT + tri_up(tb, kk) * kOp2Bytes, lane, T());
                dX[tb] = mma(tt, uo[kk], dX[tb]);
                if constexpr (!ENDS) xt[tb] = mma(uo[kk], tt, xt[tb]);
            }
        tiles(yo[0], dY[0], dY[1]);
        tiles(yo[1], dY[2], dY[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            if constexpr (!ENDS) {
                const int t = row_index(tb, c), v = v0 + 4 * g;
                store_io4(xt[tb], rv, v < V ? static_cast<uint32_t>((t * ldy + v) * es) : kOffNone, T());
                stream4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
            }
            const f32x4 eg = *reinterpret_cast<const f32x4 *>(&sS[32 * (tb / 2) + 8 * g + 4 * (tb % 2)]);
            dY[tb] = dY[tb] * eg * a.scale;
            dX[tb] = dX[tb] * -eg;
        }
        const Op2<T> qo[2] = {computed<T>(dY[0], dY[1]), computed<T>(dY[2], dY[3])};
        const Op2<T> xo[2] = {computed<T>(dX[0], dX[1]), computed<T>(dX[2], dX[3])};
        const float end = sS[kC - 1];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) dS[kt] = dS[kt] * end;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) dS[kt] = mma(get_col<KP>(sQ, sQ, kt, kk, lane, T()), qo[kk], dS[kt]);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) dS[kt] = mma(get_col<KP>(sK, sC, kt, kk, lane, T()), xo[kk], dS[kt]);
    }
    rev_end<T, KP, ENDS, kWaves>(dS, p, r, smem, v0, w, lane);
}

template <int KP> constexpr size_t rev_lds() {
    using T = float;
    return Rows<T, KP>::kBytes + Cols<KP>::kBytes + QSide<T, KP>::kBytes + 2 * kTriBytes + 3 * kC * 4;
}

// The same in bf16 io, as in delta_flow.h: a fifth (ninth) wave loads.  The buffer's
// parts hold T^T, P^T and the columns of dY where the forward has T, P and V.
template <int KP, bool ENDS, int NW>
__global__ __launch_bounds__(kFlowThreads<NW>) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 3 : 2, NW == 8 ? 3 : 2))) void delta_rev_flow_kernel(BwdParams p) {
    using T = bf16_t;
    using B = FlowBuf<KP, NW>;
    constexpr int KT = KP / 16, KK = KP / 32, kWide = 16 * NW;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    const RevPart r = rev_part<KP, ENDS, NW>(p);
    if (!r.used) return;
    const int64_t head = r.head, kh = r.kh, lastrow = r.lastrow, lastunit = r.lastunit;
    const int vt = r.vt, nch = r.nch, ldy = static_cast<int>(H) * V;

    if (w == NW) {                                         // the loading wave
        const FlowLoader<KP, NW> ld(a.ldk, a.ldq, ldy, K, V - vt * kWide);
        const T *pk = static_cast<const T *>(a.k) + lastrow * a.ldk + kh * K, *pq = static_cast<const T *>(a.q) + lastrow * a.ldq + kh * K;
        const T *pv = static_cast<const T *>(p.b.dout) + (lastrow * H + head) * V + vt * kWide;
        const char *pt = p.ws.tt + lastunit * kTriBytes, *pp = p.ws.p + lastunit * kTriBytes;
        const float *ps = p.ws.scal + lastunit * 3 * kC;
        for (int j = 0; j < nch; ++j) {
            char *const buf = smem + j % 2 * B::bytes;
            const int n = j == 0 ? r.n : kC;
            ld.template rows<KK>(buf, chunk_rsrc(pk, n, a.ldk, K, 2), ld.k, ld.ldk);
            ld.template rows<B::kv>(buf + B::v, chunk_rsrc(pv, r.transition ? 0 : n, ldy, V - vt * kWide, 2), ld.v, ld.ldv);
            ld.template copy<kTriBytes>(buf + B::p, pp);
            ld.scalars(buf + B::s, ps);
            ld.template copy<kTriBytes>(buf + B::t, pt);
            ld.template rows<KK>(buf + B::q, chunk_rsrc(pq, n, a.ldq, K, 2), ld.q, ld.ldq);
            pk -= kC * a.ldk;
            pq -= kC * a.ldq;
            pv -= static_cast<int64_t>(kC) * ldy;
            pt -= H * kTriBytes;
            pp -= H * kTriBytes;
            ps -= H * 3 * kC;
            flow_loaded();
            flow_barrier();
        }
        if (r.transition) {
            flow_barrier();
            flow_barrier();
        }
        return;
    }

    const int v0 = vt * kWide + w * 16;
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    const int at = flow_at(lane), tat = flow_tr_at(lane);
    constexpr bool AHEAD = NW == 4;
    auto fence = [] {
        if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 dS[KT];
    rev_start<KP, ENDS>(dS, p, r, kWide, v0, w, lane);
    int64_t unit = lastunit;
    T *pdv = static_cast<T *>(p.b.dv) + (lastrow * H + head) * V;
    for (int j = 0; j < nch; ++j, unit -= H, pdv -= static_cast<int64_t>(kC) * ldy) {
        const char *const buf = smem + j % 2 * B::bytes;
        const float *const sS = reinterpret_cast<const float *>(buf + B::s);
        const int n = j == 0 ? r.n : kC;
        flow_barrier();
        if constexpr (!ENDS) store_state<KP>(dS, p.dS + unit * VK, v0, V, K, lane);
        Op<T> fk[2][4], yo[2];
        Op2<T> so[2], fp[AHEAD ? 6 : 1], ft[AHEAD ? 6 : 1];
        auto read_rows = [&](int kk) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) fk[kk % 2][tb] = flow_row(buf + (tb * KK + kk) * 1024, at);
        };
        f32x4 dU[4] = {zero, zero, zero, zero}, pd[4] = {zero, zero, zero, zero};
        if constexpr (AHEAD) {
            read_rows(0);
#pragma unroll
            for (int f = 0; f < 6; ++f) fp[f] = get_op2(buf + B::p + f * kOp2Bytes, lane, T());
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) yo[q] = flow_value<B::kv>(buf + B::v, lane, q, w);
        fence();
        so[0] = computed<T>(dS[0], dS[1]);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if constexpr (!AHEAD) read_rows(kk);
            else if (kk + 1 < KK) read_rows(kk + 1);
            fence();
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) dU[tb] = mma(fk[kk % 2][tb], so[kk % 2], dU[tb]);
            if (kk + 1 < KK) so[(kk + 1) % 2] = computed<T>(dS[2 * kk + 2], dS[2 * kk + 3]);
            fence();
        }
#pragma unroll
        for (int f = 0; f < (AHEAD ? 6 : 0); ++f) ft[f] = get_op2(buf + B::t + f * kOp2Bytes, lane, T());
        f32x4 eg[4], ew[4], eb[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = 32 * (tb / 2) + 8 * g + 4 * (tb % 2);
            eg[tb] = *reinterpret_cast<const f32x4 *>(&sS[t]);
            ew[tb] = *reinterpret_cast<const f32x4 *>(&sS[kC + t]);
            eb[tb] = *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t]);
        }
        const float end = sS[kC - 1];
        fence();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 0; tb < 2 * kk + 2; ++tb) {
                Op2<T> f;
                if constexpr (AHEAD) f = fp[tri_up(tb, kk)];
                else f = get_op2(buf + B::p + tri_up(tb, kk) * kOp2Bytes, lane, T());
                pd[tb] = mma(f, yo[kk], pd[tb]);
            }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) dU[tb] = (dU[tb] * ew[tb] + pd[tb] * a.scale) * eb[tb];
        const Op2<T> uo[2] = {computed<T>(dU[0], dU[1]), computed<T>(dU[2], dU[3])};
        f32x4 dY[4];
        tiles(yo[0], dY[0], dY[1]);
        tiles(yo[1], dY[2], dY[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) dY[tb] = dY[tb] * eg[tb] * a.scale;
        const Op2<T> qo[2] = {computed<T>(dY[0], dY[1]), computed<T>(dY[2], dY[3])};
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) dS[kt] = dS[kt] * end;
        fence();
        Op<T> fc[KT];
        auto read_cols = [&](const char *rows, int kk) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) fc[kt] = flow_col<KP>(rows, tat, kt, kk);
        };
        if constexpr (AHEAD) read_cols(buf + B::q, 0);
        fence();
        // dX for the state, and transposed for stores of four channels
        f32x4 dX[4] = {zero, zero, zero, zero}, xt[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 0; tb < 2 * kk + 2; ++tb) {
                Op2<T> f;
                if constexpr (AHEAD) f = ft[tri_up(tb, kk)];
                else f = get_op2(buf + B::t + tri_up(tb, kk) * kOp2Bytes, lane, T());
                dX[tb] = mma(f, uo[kk], dX[tb]);
                if constexpr (!ENDS) xt[tb] = mma(uo[kk], f, xt[tb]);
            }
        auto add_cols = [&](const char *rows, int kk, const Op2<T> &o) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                if constexpr (!AHEAD) fc[kt] = flow_col<KP>(rows, tat, kt, kk);
                dS[kt] = mma(fc[kt], o, dS[kt]);
            }
        };
        add_cols(buf + B::q, 0, qo[0]);
        fence();
        if constexpr (AHEAD) read_cols(buf + B::q, 1);
        fence();
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) dX[tb] = dX[tb] * -eg[tb];
        const Op2<T> xo[2] = {computed<T>(dX[0], dX[1]), computed<T>(dX[2], dX[3])};
        if constexpr (!ENDS) {
            const rsrc_t rv = chunk_rsrc(pdv, n, ldy, V, 2), rx = make_rsrc(p.dX + unit * kC * V, static_cast<uint32_t>(kC * V * 4));
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const int t = row_index(tb, c);
                store_io4(xt[tb], rv, v < V ? static_cast<uint32_t>((t * ldy + v) * 2) : kOffNone, T());
                stream4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
            }
        }
        add_cols(buf + B::q, 1, qo[1]);
        fence();
        if constexpr (AHEAD) read_cols(buf, 0);
        fence();
        add_cols(buf, 0, xo[0]);
        fence();
        if constexpr (AHEAD) read_cols(buf, 1);
        fence();
        add_cols(buf, 1, xo[1]);
    }
    rev_end<T, KP, ENDS, NW>(dS, p, r, smem, v0, w, lane);
}

// -------------------------------------------------------------------- the rest
// A workgroup takes (chunk, key head) after (chunk, key head), over the value heads that
// share it; a pair of waves (w, w + 4) owns 16 of the chunk's steps as columns of
// transposed results (rows are the K channels), each wave half of the channels: a lane
// holds eight neighbouring channels of one step, so stores have 16 bytes and the row
// sums of dg and dbeta are sums inside a lane.  Of the chunk's four decayed products
// wave w makes the two with the pair's steps as t, wave w + 4 the two with them as s;
// they exchange them through LDS.
//
// The value channels are taken 32 at a time.  Four more waves bring them from global
// memory, as operands, into one of two LDS buffers: a wave that computes and loads
// stands still for as long as its loads queue, which at the memory's rate is longer than
// all it computes.  8 x 2048 steps of 12 heads of 128 x 128 (bytes: 148 us at a copy's rate): every wave
// loading for itself 404 us with four waves, 267 with eight; now 227.
constexpr int kGradThreads = 768, kGradWaves = 8;

// What a loading thread holds of 32 value channels: two channels of eight rows of S and of
// dS', one row's eight channels of dX, R and dY.
template <typename T, int KP> struct GradStage {
    static constexpr int kSlots = 2 * KP;
    f32x2 s[8], d[8];
    f32x4 x[2], r[2];
    Op<T> y;
    int i, v8;                                             // of the 256 threads; the first value channel
    uint32_t state, row, value, out;                       // offsets of value channel 0
    __device__ __forceinline__ GradStage(int thread, int64_t ldy, int K, int V) : i(thread) {
        const int c = 2 * (i % 8), tile = i / 32, k = 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4;
        const int t = row_index(i / 64, i % 16);
        v8 = 8 * (i / 16 % 4);
        state = i < kSlots && k < K ? static_cast<uint32_t>((8 * (i / 8 % 4) * K + k) * 4) : kOffNone;
        row = static_cast<uint32_t>(K * 4);
        value = static_cast<uint32_t>((t * V + v8) * 4);
        out = static_cast<uint32_t>((t * ldy + v8) * static_cast<int64_t>(sizeof(T)));
    }
    __device__ __forceinline__ void load(rsrc_t rs, rsrc_t rd, rsrc_t rx, rsrc_t rr, rsrc_t ry, int v0, int V) {
        const int v = v0 + 8 * (i / 8 % 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t off = state != kOffNone && v + j < V ? state + (v0 + j) * row : kOffNone;
            s[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
            d[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rd, off, 0, 0));
        }
        const bool in = v0 + v8 < V;
        const uint32_t off = in ? value + static_cast<uint32_t>(v0 * 4) : kOffNone;
        x[0] = load4(rx, off);
        x[1] = load4(rx, off + 16);
        r[0] = load4(rr, off);
        r[1] = load4(rr, off + 16);
        y = load_op(ry, in ? out + static_cast<uint32_t>(v0 * static_cast<int>(sizeof(T))) : kOffNone, T());
    }
    // into LDS as operands; the thread's part of <S, dS'>
    __device__ __forceinline__ float put(char *sX, char *sR, char *sS, char *sD, char *sY) const {
        const int lane = i % 64, w = i / 64;
        float dot = 0.0f;
        if (i < kSlots) {
            const int to = i / 32 * kOp2Bytes, at = 16 * (i / 8 % 4) + 2 * (i % 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) dot = fmaf(s[j][0], d[j][0], fmaf(s[j][1], d[j][1], dot));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                put_op(sS + to, at + h, computed<T>(f32x4{s[0][h], s[1][h], s[2][h], s[3][h]}, f32x4{s[4][h], s[5][h], s[6][h], s[7][h]}));
                put_op(sD + to, at + h, computed<T>(f32x4{d[0][h], d[1][h], d[2][h], d[3][h]}, f32x4{d[4][h], d[5][h], d[6][h], d[7][h]}));
            }
        }
        put_op(sX + w * kOp2Bytes, lane, computed<T>(x[0], x[1]));
        put_op(sR + w * kOp2Bytes, lane, computed<T>(r[0], r[1]));
        put_op(sY + w * kOpBytes<T>, lane, y);
        return dot;
    }
};
// the eight elements of an operand as floats
__device__ __forceinline__ void floats(const Op<bf16_t> &o, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = low(o.v[i]);
        v[2 * i + 1] = high(o.v[i]);
    }
}
__device__ __forceinline__ void floats(const Op<float> &o, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = o.a[i];
        v[4 + i] = o.b[i];
    }
}
__device__ __forceinline__ void store_io8(f32x4 a, f32x4 b, rsrc_t r, uint32_t off, bf16_t) {
    __builtin_amdgcn_raw_buffer_store_b128(exact<bf16_t>(a, b).v, r, off, 0, 0);
}
__device__ __forceinline__ void store_io8(f32x4 a, f32x4 b, rsrc_t r, uint32_t off, float) {
    store4(a, r, off);
    store4(b, r, off + 16);
}
// over the four lane groups that hold one column
__device__ __forceinline__ float column_total(float v) {
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <typename T, int KP>
__device__ __forceinline__ void store_keys(const BwdParams &p, const f32x4 *dq, const f32x4 *dk, int64_t row0, int64_t kh, int t, int wh,
                                           int g, int n) {
    constexpr int KK = KP / 64;
    const int64_t Hk = p.b.fwd.s.kheads, K = p.b.fwd.s.dk;
    const rsrc_t wq = make_rsrc(static_cast<T *>(p.b.dq) + (row0 * Hk + kh) * K), wk = make_rsrc(static_cast<T *>(p.b.dk) + (row0 * Hk + kh) * K);
#pragma unroll
    for (int kp = 0; kp < KK; ++kp) {
        const int k0 = 32 * (wh * KK + kp) + 8 * g;
        const uint32_t off = t < n && k0 < K ? static_cast<uint32_t>((t * Hk * K + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
        store_io8(dq[2 * kp], dq[2 * kp + 1], wq, off, T());
        store_io8(dk[2 * kp], dk[2 * kp + 1], wk, off, T());
    }
}

// LDS: buffers of 32 value channels, the decayed products in place of the last; the
// chunk's keys and queries.  Two buffers but for the widest fp32 form.
template <typename T, int KP> struct GradBuf {
    static constexpr int x = 0, r = 4 * kOp2Bytes, s = 8 * kOp2Bytes, d = s + KP / 16 * kOp2Bytes, y = d + KP / 16 * kOp2Bytes;
    static constexpr int loop = y + 4 * kOpBytes<T>, bytes = loop > 24 * kOp2Bytes ? loop : 24 * kOp2Bytes;
    static constexpr int ft = 0, et = 6 * kOp2Bytes, f = 12 * kOp2Bytes, e = 18 * kOp2Bytes;
    static constexpr int n = sizeof(T) == 4 && KP > 64 ? 1 : 2;
    static constexpr int k = n * bytes, q = k + QSide<T, KP>::kBytes, all = q + QSide<T, KP>::kBytes;
};
// eight channels of one step, channels 32 kk + 8 g ..: bf16 has them as rows in LDS
__device__ __forceinline__ Op<bf16_t> own_row(const char *rows, int tile, int lane, rsrc_t, uint32_t, bf16_t) {
    return get_row(rows + tile * kRowBytes<bf16_t>, lane, bf16_t());
}
__device__ __forceinline__ Op<float> own_row(const char *, int, int, rsrc_t r, uint32_t off, float) { return load_op(r, off, 0.0f); }

template <typename T, int KP, bool SHARED>
__global__ __launch_bounds__(kGradThreads) __attribute__((amdgpu_waves_per_eu(3, 3))) void delta_grad_kernel(BwdParams p) {
    using D = Decay<T>;
    using B = GradBuf<T, KP>;
    constexpr int KT = KP / 32, KK = KP / 64, OB = kOpBytes<T>;    // a wave's half of the channels
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char *const sC = smem + B::k, *const sQ = smem + B::q;
    __shared__ typename D::Sum sG[kC];
    __shared__ float sScal[3 * kC], sQK[2][kC], sZ[2][kC], sTot[kGradWaves], sDot[4];
    const float *const sB = sScal + 2 * kC;
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv), stages = (V + 31) / 32;
    const int64_t H = a.s.heads, units = a.s.slots * a.s.kheads;
    const int group = static_cast<int>(H / a.s.kheads);
    const size_t VK = static_cast<size_t>(V) * K;
    struct Place {
        int64_t id, slot, kh, row0;                        // id < 0: none
        int n;
    };
    auto find = [&](int64_t id) {                            // the workgroup's next (chunk, key head)
        Place c{};
        for (; id < units; id += gridDim.x) {
            c.slot = id / a.s.kheads;
            c.kh = id % a.s.kheads;
            const Span sp = span_of(a.s, sequence_of(a.s, c.slot));
            const int64_t step0 = (c.slot - sp.slot0) * kC;
            if (step0 < 0 || step0 >= sp.len) continue;
            c.n = sp.len - step0 < kC ? static_cast<int>(sp.len - step0) : kC;
            c.row0 = sp.row0 + step0;
            c.id = id;
            return c;
        }
        c.id = -1;
        return c;
    };
    auto rows_of = [&](const void *t, int64_t ld, const Place &c) {
        return chunk_rsrc(static_cast<const T *>(t) + c.row0 * ld + c.kh * K, c.n, ld, K, sizeof(T));
    };
    auto buffer = [&](int i) { return smem + (B::n == 2 ? i % 2 : 0) * B::bytes; };
    Place here = find(blockIdx.x);
    if (here.id < 0) return;
    int at = 0;                                              // stages so far

    // Barriers of a head, which all twelve waves pass: one per stage (it is in LDS, and the one before done with; with
    // one buffer a second, done with this one), the loop's end, the decayed products, the end.
    if (wave >= kGradWaves) {                                // the loading waves
        const int thread = threadIdx.x - 64 * kGradWaves, pw = wave - kGradWaves;
        GradStage<T, KP> st(thread, H * V, K, V);
        auto load = [&](const Place &c, int64_t head, int v0) {
            const int64_t unit = c.slot * H + head;
            const float *const saved = a.ckpt + unit * (VK + kC * V);
            st.load(make_rsrc(saved, static_cast<uint32_t>(VK * 4)), make_rsrc(p.dS + unit * VK, static_cast<uint32_t>(VK * 4)),
                    make_rsrc(p.dX + unit * kC * V), make_rsrc(saved + VK),
                    chunk_rsrc(static_cast<const T *>(p.b.dout) + (c.row0 * H + head) * V, c.n, H * V, V, sizeof(T)), v0, V);
        };
        auto put = [&](int i) {
            char *const to = buffer(i);
            return st.put(to + B::x, to + B::r, to + B::s, to + B::d, to + B::y);
        };
        const auto ok = QSide<T, KP>::offsets(a.ldk, K, thread), oq = QSide<T, KP>::offsets(a.ldq, K, thread);
        load(here, here.kh * group, 0);
        float tot = put(0);
        while (true) {
            const Place next = find(here.id + gridDim.x);
            QSide<T, KP> k, q;
            k.load(rows_of(a.k, a.ldk, here), a.ldk, ok);
            q.load(rows_of(a.q, a.ldq, here), a.ldq, oq);
            for (int hh = 0; hh < group; ++hh) {
                const int64_t head = here.kh * group + hh, unit = here.slot * H + head;
                const bool more = hh + 1 < group || next.id >= 0;
                float step = 0.0f, scal[3];
                if (pw == 0) {
                    if (lane < here.n) step = a.g[(here.row0 + lane) * H + head];
#pragma unroll
                    for (int i = 0; i < 3; ++i) scal[i] = p.ws.scal[unit * 3 * kC + i * kC + lane];
                }
                for (int i = 0; i < stages; ++i, ++at) {
                    if (i + 1 < stages) load(here, head, 32 * (i + 1));
                    else if (hh + 1 < group) load(here, head + 1, 0);
                    else if (next.id >= 0) load(next, next.kh * group, 0);
                    flow_barrier();
                    // what the head's end needs, now that everyone is done with the head before
                    if (i + 1 == stages) {
                        tot = wave_fold(tot, AddOp());
                        if (lane == 0) sDot[pw] = tot;
                    }
                    if (i == 0) {
                        if (hh == 0) {
                            k.put(sC, thread);
                            q.put(sQ, thread);
                        }
                        if (pw == 0) {
                            sG[lane] = D::sum(lane_prefix(lane < here.n ? D::scaled(step_log(step)) : 0.0, lane));
#pragma unroll
                            for (int j = 0; j < 3; ++j) sScal[j * kC + lane] = scal[j];
                        }
                    }
                    if (B::n == 1) flow_barrier();
                    if (i + 1 < stages) tot += put(at + 1);
                }
                if (B::n == 2) flow_barrier();
                flow_barrier();
                if (B::n == 2 && more) tot = put(at);
                flow_barrier();
                if (B::n == 1 && more) tot = put(at);
            }
            if (next.id < 0) return;
            here = next;
        }
    }

    const int w = wave % 4, wh = wave / 4, g = lane / 16, c = lane % 16, t = row_index(w, c);
    const f32x4 zero = {0, 0, 0, 0};
    while (true) {
        const Place next = find(here.id + gridDim.x);
        f32x4 dqs[SHARED ? KT : 1], dks[SHARED ? KT : 1];
        if constexpr (SHARED) {
#pragma unroll
            for (int i = 0; i < KT; ++i) dqs[i] = dks[i] = zero;
        }
        for (int hh = 0; hh < group; ++hh) {
            const int64_t head = here.kh * group + hh;
            // A: (F diag(beta))^T or F, B: M^T or -E
            f32x4 dq[KT], ke[KT], kw[KT], A[4], E[4];
#pragma unroll
            for (int i = 0; i < KT; ++i) dq[i] = ke[i] = kw[i] = zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) A[i] = E[i] = zero;
            for (int i = 0; i < stages; ++i, ++at) {
                const char *const from = buffer(at);
                flow_barrier();
                // operands are read from LDS a product ahead of their use
                Op2<T> sd[2][2];
                auto read = [&](int kt) {
                    sd[kt % 2][0] = get_op2(from + B::s + (wh * KT + kt) * kOp2Bytes, lane, T());
                    sd[kt % 2][1] = get_op2(from + B::d + (wh * KT + kt) * kOp2Bytes, lane, T());
                };
                const Op<T> y = get_op(from + B::y + w * OB, lane, T());
                const Op2<T> x = get_op2(from + B::x + w * kOp2Bytes, lane, T()), r = get_op2(from + B::r + w * kOp2Bytes, lane, T());
                read(0);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    if (kt + 1 < KT) read(kt + 1);
                    __builtin_amdgcn_sched_barrier(0);
                    dq[kt] = mma(sd[kt % 2][0], y, dq[kt]);
                    ke[kt] = mma(sd[kt % 2][0], x, ke[kt]);
                    kw[kt] = mma(sd[kt % 2][1], r, kw[kt]);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if (wh == 0 && kk <= w / 2) {            // rows s at or before the pair's steps
                        const char *const f = from + B::r + 2 * kk * kOp2Bytes;
                        const Op2<T> r0 = get_op2(f, lane, T()), r1 = get_op2(f + kOp2Bytes, lane, T());
                        A[2 * kk] = mma(r0, y, A[2 * kk]);
                        A[2 * kk + 1] = mma(r1, y, A[2 * kk + 1]);
                        E[2 * kk] = mma(r0, x, E[2 * kk]);
                        E[2 * kk + 1] = mma(r1, x, E[2 * kk + 1]);
                    }
                    if (wh == 1 && kk >= w / 2) {            // rows t at or behind them
                        const char *const f = from + B::x + 2 * kk * kOp2Bytes, *const fy = from + B::y + 2 * kk * OB;
                        const Op<T> y0 = get_op(fy, lane, T()), y1 = get_op(fy + OB, lane, T());
                        const Op2<T> x0 = get_op2(f, lane, T()), x1 = get_op2(f + kOp2Bytes, lane, T());
                        A[2 * kk] = mma(y0, r, A[2 * kk]);
                        A[2 * kk + 1] = mma(y1, r, A[2 * kk + 1]);
                        E[2 * kk] = mma(x0, r, E[2 * kk]);
                        E[2 * kk + 1] = mma(x1, r, E[2 * kk + 1]);
                    }
                }
                if (B::n == 1) flow_barrier();
            }
            if (B::n == 2) flow_barrier();
            char *const to = buffer(at - 1);
            const float eg = sScal[t], wt = sScal[kC + t], beta = sB[t], end = sScal[kC - 1];
            const typename D::Sum gt = sG[t];
#pragma unroll
            for (int ob = 0; ob < 4; ++ob)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int o = 32 * (ob / 2) + 8 * g + 4 * (ob % 2) + i;      // the row: s or t
                    const bool in = wh ? o >= t : o <= t;
                    const typename D::Sum go = sG[o];                   // no branch: the reads of LDS side by side
                    const float bo = sB[o], d = D::ex(in ? (wh ? D::minus(go, gt) : D::minus(gt, go)) : 0.0f) * (wh ? 1.0f : bo);
                    A[ob][i] = in ? A[ob][i] * (a.scale * d) : 0.0f;
                    E[ob][i] = in && o != t ? E[ob][i] * -d : 0.0f;
                }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                if (wh == 0 && kk <= w / 2) {
                    put_op(to + B::ft + tri_low(w, kk) * kOp2Bytes, lane, computed<T>(A[2 * kk], A[2 * kk + 1]));
                    put_op(to + B::et + tri_low(w, kk) * kOp2Bytes, lane, computed<T>(E[2 * kk], E[2 * kk + 1]));
                }
                if (wh == 1 && kk >= w / 2) {
                    put_op(to + B::f + tri_up(w, kk) * kOp2Bytes, lane, computed<T>(A[2 * kk], A[2 * kk + 1]));
                    put_op(to + B::e + tri_up(w, kk) * kOp2Bytes, lane, computed<T>(E[2 * kk], E[2 * kk + 1]));
                }
            }
            float qd = 0.0f, kd = 0.0f, kz = 0.0f, kc = 0.0f;
            const float fq = a.scale * eg;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                dq[kt] = dq[kt] * fq;
                ke[kt] = ke[kt] * -eg;
                kw[kt] = kw[kt] * wt;                        // Z
            }
            flow_barrier();
            float kv[KK][8], qv[KK][8];
#pragma unroll
            for (int kp = 0; kp < KK; ++kp) {
                const int kk = wh * KK + kp, k0 = 32 * kk + 8 * g, tile = w * (KP / 32) + kk;
                const uint32_t ok = k0 < K ? static_cast<uint32_t>((t * a.ldk + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
                const uint32_t oq = k0 < K ? static_cast<uint32_t>((t * a.ldq + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
                floats(own_row(sC, tile, lane, rows_of(a.k, a.ldk, here), ok, T()), kv[kp]);
                floats(own_row(sQ, tile, lane, rows_of(a.q, a.ldq, here), oq, T()), qv[kp]);
            }
#pragma unroll
            for (int kp = 0; kp < KK; ++kp)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i) kc = fmaf(kv[kp][4 * h + i], kw[2 * kp + h][i], kc);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                if (kk <= w / 2) {
                    const Op2<T> ft = get_op2(to + B::ft + tri_low(w, kk) * kOp2Bytes, lane, T()), et = get_op2(to + B::et + tri_low(w, kk) * kOp2Bytes, lane, T());
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        const Op<T> kcol = get_col<KP>(sC, sC, wh * KT + kt, kk, lane, T());
                        dq[kt] = mma(kcol, ft, dq[kt]);
                        ke[kt] = mma(kcol, et, ke[kt]);
                    }
                }
                if (kk >= w / 2) {
                    const Op2<T> f = get_op2(to + B::f + tri_up(w, kk) * kOp2Bytes, lane, T()), e = get_op2(to + B::e + tri_up(w, kk) * kOp2Bytes, lane, T());
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt) {
                        kw[kt] = mma(get_col<KP>(sQ, sQ, wh * KT + kt, kk, lane, T()), f, kw[kt]);
                        kw[kt] = mma(get_col<KP>(sC, sC, wh * KT + kt, kk, lane, T()), e, kw[kt]);
                    }
                }
            }
#pragma unroll
            for (int kp = 0; kp < KK; ++kp)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int kt = 2 * kp + h;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        qd = fmaf(qv[kp][4 * h + i], dq[kt][i], qd);
                        kd = fmaf(kv[kp][4 * h + i], ke[kt][i], kd);
                        kz = fmaf(kv[kp][4 * h + i], kw[kt][i], kz);
                    }
                    ke[kt] = ke[kt] + kw[kt] * beta;
                }
            const float qk = column_total(qd + kd), z = column_total(kz);
            kc = wave_fold(beta * kc, AddOp());
            if (lane == 0) sTot[wave] = kc;
            if (g == 0) {
                sQK[wh][t] = qk;
                sZ[wh][t] = z;
            }
            flow_barrier();
            if (wave == 0) {                                 // lane l is step 63 - l: sums from the end
                const int l = 63 - lane;
                const float zl = sZ[0][l] + sZ[1][l];
                double v = static_cast<double>(sQK[0][l]) + sQK[1][l] - static_cast<double>(sB[l]) * zl;
                if (lane == 0) {
                    v += static_cast<double>(end) * (static_cast<double>(sDot[0]) + sDot[1] + sDot[2] + sDot[3]);
                    for (int i = 0; i < kGradWaves; ++i) v += sTot[i];
                }
                v = lane_prefix(v, lane);
                if (l < here.n) {
                    p.b.dg[(here.row0 + l) * H + head] = static_cast<float>(v);
                    p.b.dbeta[(here.row0 + l) * H + head] = zl;
                }
            }
            if constexpr (SHARED) {
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    dqs[i] = dqs[i] + dq[i];
                    dks[i] = dks[i] + ke[i];
                }
            } else {
                store_keys<T, KP>(p, dq, ke, here.row0, here.kh, t, wh, g, here.n);
            }
        }
        if constexpr (SHARED) store_keys<T, KP>(p, dqs, dks, here.row0, here.kh, t, wh, g, here.n);
        if (next.id < 0) return;
        here = next;
    }
}

// bf16: 64 value channels to a workgroup, 128 where only those let every CU have one.
// Gradient calls, 128 x 128: 8 x 2048 steps of 12 heads (192 narrow workgroups), this kernel 175 us
// against 247 wide; 16 x 2048 of 12 (384), the call 944 against 899; 24 x 1024 of 12 (576) 656 against 701.
template <typename T, int KP, bool ENDS> hipError_t launch_rev(const BwdParams &p, hipStream_t s) {
    const DeltaShape &sh = p.b.fwd.s;
    auto groups = [&](int wide) { return ((sh.dv + wide - 1) / wide + (ENDS ? (KP + wide - 1) / wide : 0)) * sh.heads * (ENDS ? p.seq.edges : p.seq.segments); };
    if constexpr (sizeof(T) == 4) {
        constexpr size_t lds = rev_lds<KP>();
        hipLaunchKernelGGL((delta_rev_kernel<KP, ENDS>), dim3(static_cast<unsigned>(groups(64))), dim3(kThreads), lds, s, p);
    } else if (sh.dv > 64 && groups(64) > 256 && groups(128) <= 256) {
        constexpr size_t lds = 2 * FlowBuf<KP, 8>::bytes;
        hipLaunchKernelGGL((delta_rev_flow_kernel<KP, ENDS, 8>), dim3(static_cast<unsigned>(groups(128))), dim3(kFlowThreads<8>), lds, s, p);
    } else {
        constexpr size_t lds = 2 * FlowBuf<KP, 4>::bytes;
        hipLaunchKernelGGL((delta_rev_flow_kernel<KP, ENDS, 4>), dim3(static_cast<unsigned>(groups(64))), dim3(kFlowThreads<4>), lds, s, p);
    }
    return hipGetLastError();
}
// The walk backwards, cut in time where the forward is.  The gradient call with saved chunks,
// uncut and cut: 65536 steps of 8 heads of 64 x 64 bf16 3004 and 769 us, 16384 of 4 of 128 x 128 886 and 292, 8192 of 4
// of 64 x 64 fp32 1060 and 177.
template <typename T, int KP> hipError_t launch_back(const BwdParams &p, hipStream_t s) {
    if (p.seq.segments != p.b.fwd.s.nseq) {
        if (hipError_t e = launch_rev<T, KP, true>(p, s)) return e;
        if (hipError_t e = launch_carry<T, KP, true>(p.seq, s)) return e;
    }
    return launch_rev<T, KP, false>(p, s);
}

struct BwdWs {
    size_t t, tt, p, scal, dX, dS, ckpt, ends, maps, total;
};
BwdWs bwd_ws(const DeltaShape &s, const Plan &plan, bool saved) {
    const size_t units = static_cast<size_t>(s.slots * s.heads), V = s.dv, K = s.dk;
    BwdWs w{};
    w.tt = w.t + (saved ? 0 : align256(units * kTriBytes));
    w.p = w.tt + align256(units * kTriBytes);
    w.scal = w.p + align256(units * kTriBytes);
    w.dX = w.scal + align256(units * 3 * kC * 4);
    w.dS = w.dX + align256(units * kC * V * 4);
    w.ckpt = w.dS + align256(units * V * K * 4);
    w.ends = w.ckpt + (saved ? 0 : align256(units * static_cast<size_t>(delta_ckpt_stride(K, V)) * 4));
    w.maps = w.ends + ends_bytes(s, plan);
    w.total = w.maps + maps_bytes(s, plan);
    return w;
}

template <typename T, int KP> hipError_t run(const DeltaBwdArgs &b, hipStream_t s) {
    const DeltaShape &sh = b.fwd.s;
    const Plan plan = plan_of(sh, b.fwd.bf16);
    const BwdWs w = bwd_ws(sh, plan, b.fwd.ckpt != nullptr);
    char *const base = static_cast<char *>(b.fwd.workspace);
    BwdParams p{};
    p.b = b;
    p.b.fwd.last_state = nullptr;
    p.ws = {b.fwd.ckpt ? nullptr : base + w.t, base + w.p, base + w.tt, reinterpret_cast<float *>(base + w.scal)};
    p.dX = reinterpret_cast<float *>(base + w.dX);
    p.dS = reinterpret_cast<float *>(base + w.dS);
    SeqParams &q = p.seq;
    q.a = b.fwd;
    q.a.last_state = nullptr;
    q.ws = p.ws;
    q.cps = plan.cps;
    q.wide = plan.wide;
    q.wide_ends = plan.wide_ends;
    q.segments = plan.segments;
    q.edges = plan.edges;
    q.ends = reinterpret_cast<float *>(base + w.ends);
    q.maps = base + w.maps;
    if (sh.slots > 0) {
        if (hipError_t e = launch_prep<T, KP, true>(b.fwd, p.ws, s)) return e;
        if (!b.fwd.ckpt) {
            q.a.ckpt = p.b.fwd.ckpt = reinterpret_cast<float *>(base + w.ckpt);
            if (hipError_t e = launch_segments<T, KP>(q, s)) return e;
            if (hipError_t e = launch_walk<T, KP, kSave>(q, s)) return e;
        }
    }
    if (hipError_t e = launch_back<T, KP>(p, s)) return e;
    if (sh.slots == 0) return hipSuccess;
    constexpr size_t glds = GradBuf<T, KP>::all;
    const int64_t units = sh.slots * sh.kheads;
    const dim3 grid(static_cast<unsigned>(units < 256 ? units : 256));       // one to a CU
    if (sh.heads == sh.kheads) hipLaunchKernelGGL((delta_grad_kernel<T, KP, false>), grid, dim3(kGradThreads), glds, s, p);
    else hipLaunchKernelGGL((delta_grad_kernel<T, KP, true>), grid, dim3(kGradThreads), glds, s, p);
    return hipGetLastError();
}

}  // namespace
}  // namespace delta

size_t delta_scan_bwd_workspace(const DeltaShape &s, int bf16, bool saved) {
    return s.slots * s.heads > 0 ? delta::bwd_ws(s, delta::plan_of(s, bf16), saved).total : 0;
}
hipError_t launch_delta_scan_bwd(const DeltaBwdArgs &b, hipStream_t s) {
    using namespace delta;
    if (b.fwd.bf16) return b.fwd.s.dk > 64 ? run<bf16_t, 128>(b, s) : run<bf16_t, 64>(b, s);
    return b.fwd.s.dk > 64 ? run<float, 128>(b, s) : run<float, 64>(b, s);
}

}  // namespace ssm
