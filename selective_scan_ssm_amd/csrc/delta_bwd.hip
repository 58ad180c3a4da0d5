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
// chunks and R, in a walk over the chunks; dS' and dX, in reverse; the rest, all
// chunks at once.
#include "delta_flow.h"

namespace ssm {
namespace delta {
namespace {

struct BwdParams {
    DeltaBwdArgs b;
    ChunkWs ws;
    float *dX, *dS;                // per (slot, head): (64, V), (V, K)
};

// What get_col reads of a chunk that is used with steps along K only.
template <typename T, int KP> struct QSide : Cols<T, KP> {};
template <int KP> struct QSide<bf16_t, KP> : Rows<bf16_t, KP> {
    static __device__ __forceinline__ uint32_t offsets(int64_t ld, int K) { return Rows<bf16_t, KP>::offset(ld, K); }
};

// --------------------------------------------------------- dS and dX, in reverse
template <int KP> __global__ __launch_bounds__(kThreads) void delta_rev_kernel(BwdParams p) {
    using T = float;
    constexpr int KT = KP / 16, KK = KP / 32, RB = kRowBytes<T>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    // rows and columns of the keys, columns of the queries
    char *const sK = smem, *const sC = sK + Rows<T, KP>::kBytes, *const sQ = sC + Cols<T, KP>::kBytes,
         *const sT = sQ + QSide<T, KP>::kBytes, *const sP = sT + kTriBytes;
    char *const sY = sP + kTriBytes;
    float *const sS = reinterpret_cast<float *>(sY + Values<T, 1>::kBytes);
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    const int nvt = (V + 63) / 64, vt = blockIdx.x % nvt;
    const int64_t rest = blockIdx.x / nvt, head = rest % H, kh = head / (H / a.s.kheads), seq = rest / H;
    const Span sp = span_of(a.s, seq);
    const int nchunks = (sp.len + kC - 1) / kC;
    const int v0 = vt * 64 + w * 16;
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    constexpr int es = sizeof(T);
    f32x4 dS[KT];
    if (p.b.dlast) {
        load_state<KP>(dS, p.b.dlast + (seq * H + head) * VK, v0, V, K, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) dS[i] = zero;
    }
    // the next chunk's data, a chunk ahead, as in the forward
    Rows<T, KP> nK;
    Cols<T, KP> nC;
    QSide<T, KP> nQ;
    Copy<kTriBytes> nT, nP;
    float nS;
    Values<T, 1> nY;
    const uint32_t okr = Rows<T, KP>::offset(a.ldk, K);
    const auto okc = Cols<T, KP>::offsets(a.ldk, K);
    const auto oqc = QSide<T, KP>::offsets(a.ldq, K);
    const int ldy = static_cast<int>(H * V);
    const uint32_t oy = Values<T, 1>::offset(ldy, V - vt * 64, w, lane);
    auto prefetch = [&](int j) {
        const int jj = j >= 0 ? j : 0;
        const int64_t row0 = sp.row0 + static_cast<int64_t>(jj) * kC, unit = (sp.slot0 + jj) * H + head;
        const int n = j >= 0 ? (sp.len - j * kC < kC ? sp.len - j * kC : kC) : 0;
        const rsrc_t rk = chunk_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, n, a.ldk, K, es);
        const rsrc_t rd = chunk_rsrc(static_cast<const T *>(p.b.dout) + (row0 * H + head) * V + vt * 64, n, ldy, V - vt * 64, es);
        nK.load(rk, a.ldk, okr);
        nY.load(rd, ldy, oy);
        nT.load(p.ws.tt + unit * kTriBytes);
        nP.load(p.ws.p + unit * kTriBytes);
        nS = p.ws.scal[unit * 3 * kC + (threadIdx.x < 3 * kC ? threadIdx.x : 0)];
        nC.load(rk, a.ldk, okc);
        nQ.load(chunk_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K, n, a.ldq, K, es), a.ldq, oqc);
    };
    if (nchunks > 0) prefetch(nchunks - 1);
    for (int j = nchunks - 1; j >= 0; --j) {
        const int64_t row0 = sp.row0 + static_cast<int64_t>(j) * kC, unit = (sp.slot0 + j) * H + head;
        const int n = sp.len - j * kC < kC ? sp.len - j * kC : kC;
        __syncthreads();                                   // the chunk before is done with LDS
        nK.put(sK);
        nC.put(sC);
        nQ.put(sQ);
        nT.put(sT);
        nP.put(sP);
        if (threadIdx.x < 3 * kC) sS[threadIdx.x] = nS;
        nY.put(sY);
        const Values<T, 1> cY = nY;
        __syncthreads();
        store_state<KP>(dS, p.dS + unit * VK, v0, V, K, lane);
        prefetch(j - 1);
        const Op<T> yo[2] = {cY.op(sY, 0, w, lane), cY.op(sY, 1, w, lane)};
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
                xt[tb] = mma(uo[kk], tt, xt[tb]);
            }
        tiles(yo[0], dY[0], dY[1]);
        tiles(yo[1], dY[2], dY[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = row_index(tb, c), v = v0 + 4 * g;
            store_io4(xt[tb], rv, v < V ? static_cast<uint32_t>((t * ldy + v) * es) : kOffNone, T());
            store4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
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
    if (p.b.dh0) store_state<KP>(dS, p.b.dh0 + (seq * H + head) * VK, v0, V, K, lane);
}

template <int KP> constexpr size_t rev_lds() {
    using T = float;
    return Rows<T, KP>::kBytes + Cols<T, KP>::kBytes + QSide<T, KP>::kBytes + 2 * kTriBytes + 3 * kC * 4 + Values<T, 1>::kBytes;
}

// The same in bf16 io, as in delta_flow.h: a fifth (ninth) wave loads.  The buffer's
// parts hold T^T, P^T and the columns of dY where the forward has T, P and V.
template <int KP, int NW>
__global__ __launch_bounds__(kFlowThreads<NW>) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 3 : 2, NW == 8 ? 3 : 2))) void delta_rev_flow_kernel(BwdParams p) {
    using T = bf16_t;
    using B = FlowBuf<KP, 1, NW>;
    constexpr int KT = KP / 16, KK = KP / 32, kWide = 16 * NW;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads, per_tile = H * a.s.nseq;
    const int vt = static_cast<int>(blockIdx.x / per_tile);
    const int64_t rest = blockIdx.x % per_tile, head = rest % H, kh = head / (H / a.s.kheads), seq = rest / H;
    const Span sp = span_of(a.s, seq);
    const int nch = (sp.len + kC - 1) / kC;
    const int64_t lastrow = sp.row0 + static_cast<int64_t>(nch - 1) * kC, lastunit = (sp.slot0 + nch - 1) * H + head;
    const int ldy = static_cast<int>(H) * V;

    if (w == NW) {                                         // the loading wave
        const FlowLoader<KP, 1, NW> ld(a.ldk, a.ldq, ldy, K, V - vt * kWide);
        const T *pk = static_cast<const T *>(a.k) + lastrow * a.ldk + kh * K, *pq = static_cast<const T *>(a.q) + lastrow * a.ldq + kh * K;
        const T *pv = static_cast<const T *>(p.b.dout) + (lastrow * H + head) * V + vt * kWide;
        const char *pt = p.ws.tt + lastunit * kTriBytes, *pp = p.ws.p + lastunit * kTriBytes;
        const float *ps = p.ws.scal + lastunit * 3 * kC;
        for (int j = 0; j < nch; ++j) {
            char *const buf = smem + j % 2 * B::bytes;
            const int n = j == 0 ? sp.len - (nch - 1) * kC : kC;
            ld.template rows<KK>(buf, chunk_rsrc(pk, n, a.ldk, K, 2), ld.k, ld.ldk);
            ld.template rows<B::kv>(buf + B::v, chunk_rsrc(pv, n, ldy, V - vt * kWide, 2), ld.v, ld.ldv);
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
    if (p.b.dlast) {
        load_state<KP>(dS, p.b.dlast + (seq * H + head) * VK, v0, V, K, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) dS[i] = zero;
    }
    int64_t unit = lastunit;
    T *pdv = static_cast<T *>(p.b.dv) + (lastrow * H + head) * V;
    for (int j = 0; j < nch; ++j, unit -= H, pdv -= static_cast<int64_t>(kC) * ldy) {
        const char *const buf = smem + j % 2 * B::bytes;
        const float *const sS = reinterpret_cast<const float *>(buf + B::s);
        const int n = j == 0 ? sp.len - (nch - 1) * kC : kC;
        flow_barrier();
        store_state<KP>(dS, p.dS + unit * VK, v0, V, K, lane);
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
                xt[tb] = mma(uo[kk], f, xt[tb]);
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
        const rsrc_t rv = chunk_rsrc(pdv, n, ldy, V, 2), rx = make_rsrc(p.dX + unit * kC * V, static_cast<uint32_t>(kC * V * 4));
        const int v = v0 + 4 * g;
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = row_index(tb, c);
            store_io4(xt[tb], rv, v < V ? static_cast<uint32_t>((t * ldy + v) * 2) : kOffNone, T());
            store4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
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
    if (p.b.dh0) store_state<KP>(dS, p.b.dh0 + (seq * H + head) * VK, v0, V, K, lane);
}

// -------------------------------------------------------------------- the rest
// A workgroup per (chunk, key head), over the value heads that share it; a wave
// owns 16 of the chunk's steps as columns of transposed results (rows are the K
// channels), so a lane holds eight neighbouring channels of one step: 16-byte
// stores, and the row sums of dg and dbeta are sums inside a lane.  The value
// channels are taken 32 at a time.

// 32 rows (value channels v0 ..) of a (V, K) state as operands with K channels as
// rows and the value channels along K, and the sum of products of two of them
template <typename T, int KP> __device__ __forceinline__ float stage_states(char *dst, char *dst2, const float *S, const float *dS,
                                                                          int v0, int V, int K) {
    constexpr int KT = KP / 16;
    const rsrc_t r = make_rsrc(S, static_cast<uint32_t>(static_cast<int64_t>(V) * K * 4));
    const rsrc_t r2 = make_rsrc(dS, static_cast<uint32_t>(static_cast<int64_t>(V) * K * 4));
    float dot = 0.0f;
    for (int s = threadIdx.x; s < KT * 32; s += kThreads) {
        const int tile = s / 32, c = 2 * (s % 8), g = (s / 8) % 4;
        const int k = 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4;
        f32x2 x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int v = v0 + 8 * g + j;
            const uint32_t off = v < V && k < K ? static_cast<uint32_t>((v * K + k) * 4) : kOffNone;
            x[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
            y[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(r2, off, 0, 0));
            dot = fmaf(x[j][0], y[j][0], fmaf(x[j][1], y[j][1], dot));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            put_op(dst + tile * kOp2Bytes, 16 * g + c + h,
                   computed<T>(f32x4{x[0][h], x[1][h], x[2][h], x[3][h]}, f32x4{x[4][h], x[5][h], x[6][h], x[7][h]}));
            put_op(dst2 + tile * kOp2Bytes, 16 * g + c + h,
                   computed<T>(f32x4{y[0][h], y[1][h], y[2][h], y[3][h]}, f32x4{y[4][h], y[5][h], y[6][h], y[7][h]}));
        }
    }
    return dot;
}
// a chunk's rows of a (64, V) fp32 workspace tensor, 32 columns from v0 on
template <typename T> __device__ __forceinline__ void stage_values(char *dst, const float *src, int v0, int V) {
    const rsrc_t r = make_rsrc(src);
    const int lane = threadIdx.x % 64, f = threadIdx.x / 64;
    const int t = row_index(f, lane % 16), v = v0 + 8 * (lane / 16);
    const uint32_t off = v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone;
    put_op(dst + f * kOp2Bytes, lane, computed<T>(load4(r, off), load4(r, off + 16)));
}
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

template <typename T, int KP> constexpr size_t grad_lds() {
    constexpr size_t loop = 4 * kOpBytes<T> + 8 * kOp2Bytes + 2 * (KP / 16) * kOp2Bytes, tail = 2 * QSide<T, KP>::kBytes;
    return loop > tail ? loop : tail;
}

template <typename T, int KP, bool SHARED>
__global__ __launch_bounds__(kThreads) void delta_grad_kernel(BwdParams p) {
    using D = Decay<T>;
    using real = typename D::real;
    constexpr int KT = KP / 16, KK = KP / 32, OB = kOpBytes<T>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char *const sY = smem, *const sX = sY + 4 * OB, *const sR = sX + 4 * kOp2Bytes, *const sS = sR + 4 * kOp2Bytes,
         *const sD = sS + KT * kOp2Bytes;
    char *const sC = smem, *const sQ = sC + QSide<T, KP>::kBytes;      // after the loop over the value channels
    __shared__ real sG[kC];
    __shared__ float sB[kC], sDG[kC], sTot[kWaves];
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16, t = row_index(w, c);
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads, slot = blockIdx.x / a.s.kheads, kh = blockIdx.x % a.s.kheads;
    const int group = static_cast<int>(H / a.s.kheads);
    const int64_t seq = sequence_of(a.s, slot);
    const Span sp = span_of(a.s, seq);
    const int64_t step0 = (slot - sp.slot0) * kC;
    if (step0 < 0 || step0 >= sp.len) return;
    const int n = sp.len - step0 < kC ? static_cast<int>(sp.len - step0) : kC;
    const int64_t row0 = sp.row0 + step0;
    const f32x4 zero = {0, 0, 0, 0};
    const rsrc_t rk = chunk_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, n, a.ldk, K, sizeof(T));
    const rsrc_t rq = chunk_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K, n, a.ldq, K, sizeof(T));
    const size_t VK = static_cast<size_t>(V) * K;
    f32x4 dqs[SHARED ? KT : 1], dks[SHARED ? KT : 1];
    if constexpr (SHARED) {
#pragma unroll
        for (int i = 0; i < KT; ++i) dqs[i] = dks[i] = zero;
    }
    for (int hh = 0; hh < group; ++hh) {
        const int64_t head = kh * group + hh, unit = slot * H + head;
        const float *const scal = p.ws.scal + unit * 3 * kC, *const saved = a.ckpt + unit * (VK + kC * V);
        __syncthreads();                                     // the head before is done with sG, sB, sDG
        if (w == 0) {
            const real G = lane_prefix<real>(lane < n ? D::scaled(step_log(a.g[(row0 + lane) * H + head])) : real(0), lane);
            sG[lane] = G;
            sB[lane] = scal[2 * kC + lane];
        }
        f32x4 dq[KT], ke[KT], kw[KT], FT[4], F[4], ET[4], E[4];
#pragma unroll
        for (int i = 0; i < KT; ++i) dq[i] = ke[i] = kw[i] = zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) FT[i] = F[i] = ET[i] = E[i] = zero;
        float tot = 0.0f;
        const rsrc_t rd = make_rsrc(static_cast<const T *>(p.b.dout) + (row0 * H + head) * V);
        for (int v0 = 0; v0 < V; v0 += 32) {
            __syncthreads();
            const int f = threadIdx.x / 64, tr = row_index(f, c), v = v0 + 8 * g;
            put_op(sY + f * OB, lane, load_op(rd, tr < n && v < V ? static_cast<uint32_t>((tr * H * V + v) * static_cast<int64_t>(sizeof(T))) : kOffNone, T()));
            stage_values<T>(sX, p.dX + unit * kC * V, v0, V);
            stage_values<T>(sR, saved + VK, v0, V);
            tot += stage_states<T, KP>(sS, sD, saved, p.dS + unit * VK, v0, V, K);
            __syncthreads();
            const Op<T> y = get_op(sY + w * OB, lane, T());
            const Op2<T> x = get_op2(sX + w * kOp2Bytes, lane, T()), r = get_op2(sR + w * kOp2Bytes, lane, T());
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Op2<T> s = get_op2(sS + kt * kOp2Bytes, lane, T()), d = get_op2(sD + kt * kOp2Bytes, lane, T());
                dq[kt] = mma(s, y, dq[kt]);
                ke[kt] = mma(s, x, ke[kt]);
                kw[kt] = mma(d, r, kw[kt]);
            }
#pragma unroll
            for (int ob = 0; ob < 4; ++ob) {
                if (ob / 2 <= w / 2) {                       // rows s at or before this wave's steps
                    const Op2<T> ro = get_op2(sR + ob * kOp2Bytes, lane, T());
                    FT[ob] = mma(ro, y, FT[ob]);
                    ET[ob] = mma(ro, x, ET[ob]);
                }
                if (ob / 2 >= w / 2) {                       // rows t at or behind them
                    F[ob] = mma(get_op(sY + ob * OB, lane, T()), r, F[ob]);
                    E[ob] = mma(get_op2(sX + ob * kOp2Bytes, lane, T()), r, E[ob]);
                }
            }
        }
        __syncthreads();
        QSide<T, KP> side;
        side.load(rk, a.ldk, QSide<T, KP>::offsets(a.ldk, K));
        side.put(sC);
        side.load(rq, a.ldq, QSide<T, KP>::offsets(a.ldq, K));
        side.put(sQ);
        const float eg = scal[t], wt = scal[kC + t], beta = sB[t], end = scal[kC - 1];
        const real gt = sG[t];
#pragma unroll
        for (int ob = 0; ob < 4; ++ob)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = 32 * (ob / 2) + 8 * g + 4 * (ob % 2) + i;      // the row: s for FT, ET, t for F, E
                const float before = o <= t ? D::ex(gt - sG[o]) : 0.0f, behind = o >= t ? D::ex(sG[o] - gt) : 0.0f;
                FT[ob][i] = o <= t ? FT[ob][i] * (a.scale * before * sB[o]) : 0.0f;    // (F diag(beta))^T
                ET[ob][i] = o < t ? ET[ob][i] * (-before * sB[o]) : 0.0f;      // M^T
                F[ob][i] = o >= t ? F[ob][i] * (a.scale * behind) : 0.0f;
                E[ob][i] = o > t ? E[ob][i] * -behind : 0.0f;
            }
        float qd = 0.0f, kd = 0.0f, kz = 0.0f, kc = 0.0f;
        const float fq = a.scale * eg;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            dq[kt] = dq[kt] * fq;
            ke[kt] = ke[kt] * -eg;
            kw[kt] = kw[kt] * wt;                            // Z
        }
        __syncthreads();
#pragma unroll
        for (int kp = 0; kp < KK; ++kp) {                    // pairs of channel tiles
            const int k0 = 32 * kp + 8 * g;
            const uint32_t off = t < n && k0 < K ? static_cast<uint32_t>((t * a.ldk + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
            const uint32_t offq = t < n && k0 < K ? static_cast<uint32_t>((t * a.ldq + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
            float kv[8], qv[8];
            floats(load_op(rk, off, T()), kv);
            floats(load_op(rq, offq, T()), qv);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kt = 2 * kp + h;
#pragma unroll
                for (int i = 0; i < 4; ++i) kc = fmaf(kv[4 * h + i], kw[kt][i], kc);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    const Op<T> kcol = get_col<KP>(sC, sC, kt, kk, lane, T()), qcol = get_col<KP>(sQ, sQ, kt, kk, lane, T());
                    if (kk <= w / 2) {
                        dq[kt] = mma(kcol, computed<T>(FT[2 * kk], FT[2 * kk + 1]), dq[kt]);
                        ke[kt] = mma(kcol, computed<T>(ET[2 * kk], ET[2 * kk + 1]), ke[kt]);
                    }
                    if (kk >= w / 2) {
                        kw[kt] = mma(qcol, computed<T>(F[2 * kk], F[2 * kk + 1]), kw[kt]);
                        kw[kt] = mma(kcol, computed<T>(E[2 * kk], E[2 * kk + 1]), kw[kt]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    qd = fmaf(qv[4 * h + i], dq[kt][i], qd);
                    kd = fmaf(kv[4 * h + i], ke[kt][i], kd);
                    kz = fmaf(kv[4 * h + i], kw[kt][i], kz);
                }
                ke[kt] = ke[kt] + kw[kt] * beta;
            }
        }
        const float dG = column_total(fmaf(-beta, kz, qd + kd));
        kz = column_total(kz);
        if (g == 0 && t < n) p.b.dbeta[(row0 + t) * H + head] = kz;
        tot = wave_fold(fmaf(end, tot, beta * kc), AddOp());
        if (lane == 0) sTot[w] = tot;
        if (g == 0) sDG[t] = dG;
        __syncthreads();
        if (w == 0) {                                        // lane l is step 63 - l: sums from the end
            double v = sDG[63 - lane];
            if (lane == 0) v += static_cast<double>(sTot[0]) + sTot[1] + sTot[2] + sTot[3];
            v = lane_prefix<double>(v, lane);
            if (63 - lane < n) p.b.dg[(row0 + 63 - lane) * H + head] = static_cast<float>(v);
        }
        if constexpr (SHARED) {
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                dqs[i] = dqs[i] + dq[i];
                dks[i] = dks[i] + ke[i];
            }
        } else {
            const int64_t Hk = a.s.kheads;
            const rsrc_t wq = make_rsrc(static_cast<T *>(p.b.dq) + (row0 * Hk + kh) * K), wk = make_rsrc(static_cast<T *>(p.b.dk) + (row0 * Hk + kh) * K);
#pragma unroll
            for (int kp = 0; kp < KK; ++kp) {
                const int k0 = 32 * kp + 8 * g;
                const uint32_t off = t < n && k0 < K ? static_cast<uint32_t>((t * Hk * K + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
                store_io8(dq[2 * kp], dq[2 * kp + 1], wq, off, T());
                store_io8(ke[2 * kp], ke[2 * kp + 1], wk, off, T());
            }
        }
    }
    if constexpr (SHARED) {
        const int64_t Hk = a.s.kheads;
        const rsrc_t wq = make_rsrc(static_cast<T *>(p.b.dq) + (row0 * Hk + kh) * K), wk = make_rsrc(static_cast<T *>(p.b.dk) + (row0 * Hk + kh) * K);
#pragma unroll
        for (int kp = 0; kp < KK; ++kp) {
            const int k0 = 32 * kp + 8 * g;
            const uint32_t off = t < n && k0 < K ? static_cast<uint32_t>((t * Hk * K + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone;
            store_io8(dqs[2 * kp], dqs[2 * kp + 1], wq, off, T());
            store_io8(dks[2 * kp], dks[2 * kp + 1], wk, off, T());
        }
    }
}

// bf16: 64 value channels to a workgroup while the CUs hold them all, else 128
template <int KP, int NW> hipError_t launch_rev_flow(const BwdParams &p, hipStream_t s) {
    constexpr int wide = 16 * NW;
    const DeltaShape &sh = p.b.fwd.s;
    constexpr size_t lds = 2 * FlowBuf<KP, 1, NW>::bytes;
    hipLaunchKernelGGL((delta_rev_flow_kernel<KP, NW>), dim3(static_cast<unsigned>((sh.dv + wide - 1) / wide * sh.heads * sh.nseq)),
                       dim3(kFlowThreads<NW>), lds, s, p);
    return hipGetLastError();
}
template <typename T, int KP> hipError_t launch_rev(const BwdParams &p, hipStream_t s) {
    const DeltaShape &sh = p.b.fwd.s;
    const int64_t n = (sh.dv + 63) / 64 * sh.heads * sh.nseq;
    if constexpr (sizeof(T) == 2) {
        return sh.dv > 64 && n > 256 ? launch_rev_flow<KP, 8>(p, s) : launch_rev_flow<KP, 4>(p, s);
    } else {
        constexpr size_t lds = rev_lds<KP>();
        hipLaunchKernelGGL((delta_rev_kernel<KP>), dim3(static_cast<unsigned>(n)), dim3(kThreads), lds, s, p);
        return hipGetLastError();
    }
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
    w.maps = w.ends + (saved ? 0 : ends_bytes(s, plan));
    w.total = w.maps + (saved ? 0 : maps_bytes(s, plan));
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
    if (sh.slots > 0) {
        if (hipError_t e = launch_prep<T, KP, true>(b.fwd, p.ws, s)) return e;
        if (!b.fwd.ckpt) {
            SeqParams q{};
            q.a = b.fwd;
            q.a.last_state = nullptr;
            q.ws = p.ws;
            q.cps = plan.cps;
            q.wide = plan.wide;
            q.wide_ends = plan.wide_ends;
            q.segments = plan.segments;
            q.ends = reinterpret_cast<float *>(base + w.ends);
            q.maps = base + w.maps;
            q.a.ckpt = p.b.fwd.ckpt = reinterpret_cast<float *>(base + w.ckpt);
            if (hipError_t e = launch_segments<T, KP>(q, s)) return e;
            if (hipError_t e = launch_walk<T, KP, kSave>(q, s)) return e;
        }
    }
    if (hipError_t e = launch_rev<T, KP>(p, s)) return e;
    if (sh.slots == 0) return hipSuccess;
    const dim3 grid(static_cast<unsigned>(sh.slots * sh.kheads));
    constexpr size_t glds = grad_lds<T, KP>();
    if (sh.heads == sh.kheads) hipLaunchKernelGGL((delta_grad_kernel<T, KP, false>), grid, dim3(kThreads), glds, s, p);
    else hipLaunchKernelGGL((delta_grad_kernel<T, KP, true>), grid, dim3(kThreads), glds, s, p);
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
