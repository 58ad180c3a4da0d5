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
template <typename T, int KP> struct QSide : Cols<KP> {};
template <int KP> struct QSide<bf16_t, KP> : Rows<bf16_t, KP> {
    static __device__ __forceinline__ uint32_t offsets(int64_t ld, int K, int thread) { return Rows<bf16_t, KP>::offset(ld, K, thread); }
};

// --------------------------------------------------------- dS and dX, in reverse
template <int KP> __global__ __launch_bounds__(kThreads) void delta_rev_kernel(BwdParams p) {
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
    Cols<KP> nC;
    QSide<T, KP> nQ;
    Copy<kTriBytes> nT, nP;
    float nS;
    Values nY;
    const uint32_t okr = Rows<T, KP>::offset(a.ldk, K, threadIdx.x);
    const auto okc = Cols<KP>::offsets(a.ldk, K, threadIdx.x);
    const auto oqc = QSide<T, KP>::offsets(a.ldq, K, threadIdx.x);
    const int ldy = static_cast<int>(H * V);
    const uint32_t oy = Values::offset(ldy, V - vt * 64, w, lane);
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
        nK.put(sK, threadIdx.x);
        nC.put(sC, threadIdx.x);
        nQ.put(sQ, threadIdx.x);
        nT.put(sT);
        nP.put(sP);
        if (threadIdx.x < 3 * kC) sS[threadIdx.x] = nS;
        const Values cY = nY;
        __syncthreads();
        store_state<KP>(dS, p.dS + unit * VK, v0, V, K, lane);
        prefetch(j - 1);
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
                xt[tb] = mma(uo[kk], tt, xt[tb]);
            }
        tiles(yo[0], dY[0], dY[1]);
        tiles(yo[1], dY[2], dY[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = row_index(tb, c), v = v0 + 4 * g;
            store_io4(xt[tb], rv, v < V ? static_cast<uint32_t>((t * ldy + v) * es) : kOffNone, T());
            stream4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
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
    return Rows<T, KP>::kBytes + Cols<KP>::kBytes + QSide<T, KP>::kBytes + 2 * kTriBytes + 3 * kC * 4;
}

// The same in bf16 io, as in delta_flow.h: a fifth (ninth) wave loads.  The buffer's
// parts hold T^T, P^T and the columns of dY where the forward has T, P and V.
template <int KP, int NW>
__global__ __launch_bounds__(kFlowThreads<NW>) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 3 : 2, NW == 8 ? 3 : 2))) void delta_rev_flow_kernel(BwdParams p) {
    using T = bf16_t;
    using B = FlowBuf<KP, NW>;
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
        const FlowLoader<KP, NW> ld(a.ldk, a.ldq, ldy, K, V - vt * kWide);
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
            stream4(xt[tb], rx, v < V ? static_cast<uint32_t>((t * V + v) * 4) : kOffNone);
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
// A workgroup per (chunk, key head), over the value heads that share it; a pair of
// waves (w, w + 4) owns 16 of the chunk's steps as columns of transposed results (rows
// are the K channels), each wave half of the channels: a lane holds eight neighbouring
// channels of one step, so stores have 16 bytes and the row sums of dg and dbeta are sums
// inside a lane.  Of the chunk's four decayed products wave w makes the two with the
// pair's steps as t, wave w + 4 the two with them as s; they exchange them through LDS.
// The value channels are taken 32 at a time, the next ones loaded meanwhile.
constexpr int kGradThreads = 512;

// half of a computed operand's eight elements in LDS
template <typename T> __device__ __forceinline__ void put_half(char *p, int lane, int half, f32x4 v);
template <> __device__ __forceinline__ void put_half<float>(char *p, int lane, int half, f32x4 v) {
    *reinterpret_cast<f32x4 *>(p + half * 1024 + lane * 16) = v;
}
template <> __device__ __forceinline__ void put_half<bf16_t>(char *p, int lane, int half, f32x4 v) {
    const u32x2 hi = {pack2(v[0], v[1]), pack2(v[2], v[3])};
    *reinterpret_cast<u32x2 *>(p + lane * 16 + half * 8) = hi;
    *reinterpret_cast<u32x2 *>(p + 1024 + lane * 16 + half * 8) =
        u32x2{pack2(v[0] - low(hi[0]), v[1] - high(hi[0])), pack2(v[2] - low(hi[1]), v[3] - high(hi[1]))};
}

// What a thread holds of 32 value channels: two channels of four rows of S and of dS', one
// row's eight channels of dX (waves 0 .. 3) or R (waves 4 .. 7) and of dY (waves 0 .. 3).
template <typename T, int KP> struct GradStage {
    static constexpr int kSlots = 2 * KP;                  // two channels of eight rows each, in halves
    f32x2 s[4], d[4];
    f32x4 x[2];
    Op<T> y;
    struct At {
        uint32_t state, value, out, row;                   // offsets of value channel 0
        int v4, v8;                                        // the first value channels of the halves and the eights
    };
    static __device__ __forceinline__ At at(int64_t ldy, int K, int V, int n) {
        const int i = threadIdx.x % kSlots, tile = i / 32, c = 2 * (i % 8), half = threadIdx.x / kSlots;
        const int k = 32 * (tile / 2) + 8 * (c / 4) + 4 * (tile % 2) + c % 4;
        const int lane = threadIdx.x % 64, t = row_index(threadIdx.x / 64 % 4, lane % 16);
        At o;
        o.v4 = 8 * ((i / 8) % 4) + 4 * half;
        o.v8 = 8 * (lane / 16);
        o.state = half < 2 && k < K ? static_cast<uint32_t>((o.v4 * K + k) * 4) : kOffNone;
        o.row = static_cast<uint32_t>(K * 4);
        o.value = static_cast<uint32_t>((t * V + o.v8) * 4);
        o.out = t < n && threadIdx.x < 256 ? static_cast<uint32_t>((t * ldy + o.v8) * static_cast<int64_t>(sizeof(T))) : kOffNone;
        return o;
    }
    __device__ __forceinline__ void load(rsrc_t rs, rsrc_t rd, rsrc_t rx, rsrc_t ry, const At &o, int v0, int V) {
        const uint32_t state = o.state == kOffNone ? kOffNone : o.state + static_cast<uint32_t>(v0) * o.row;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t off = v0 + o.v4 + j < V ? state + j * o.row : kOffNone;
            s[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
            d[j] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(rd, off, 0, 0));
        }
        const bool in = v0 + o.v8 < V;
        const uint32_t off = in ? o.value + static_cast<uint32_t>(v0 * 4) : kOffNone;
        x[0] = load4(rx, off);
        x[1] = load4(rx, off + 16);
        y = load_op(ry, in && o.out != kOffNone ? o.out + static_cast<uint32_t>(v0 * static_cast<int>(sizeof(T))) : kOffNone, T());
    }
    // into LDS as operands; the thread's part of <S, dS'>
    __device__ __forceinline__ float put(char *sS, char *sD, char *sX, char *sY) const {
        const int i = threadIdx.x % kSlots, half = threadIdx.x / kSlots, lane = threadIdx.x % 64, w = threadIdx.x / 64;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(s[j][0], d[j][0], fmaf(s[j][1], d[j][1], dot));
        if (half < 2) {
            const int to = i / 32 * kOp2Bytes, at = 16 * ((i / 8) % 4) + 2 * (i % 8);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                put_half<T>(sS + to, at + h, half, f32x4{s[0][h], s[1][h], s[2][h], s[3][h]});
                put_half<T>(sD + to, at + h, half, f32x4{d[0][h], d[1][h], d[2][h], d[3][h]});
            }
        }
        put_op(sX + w * kOp2Bytes, lane, computed<T>(x[0], x[1]));
        if (w < 4) put_op(sY + w * kOpBytes<T>, lane, y);
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

// LDS: what the loop over the value channels reads, then the decayed products in its
// place; the chunk's keys and queries
template <typename T, int KP> constexpr int grad_loop() { return 4 * kOpBytes<T> + 8 * kOp2Bytes + 2 * (KP / 16) * kOp2Bytes; }
template <typename T, int KP> constexpr int grad_main() { return grad_loop<T, KP>() > 24 * kOp2Bytes ? grad_loop<T, KP>() : 24 * kOp2Bytes; }
template <typename T, int KP> constexpr size_t grad_lds() { return grad_main<T, KP>() + 2 * QSide<T, KP>::kBytes; }

template <typename T, int KP, bool SHARED>
__global__ __launch_bounds__(kGradThreads) void delta_grad_kernel(BwdParams p) {
    using D = Decay<T>;
    using real = typename D::real;
    constexpr int KT = KP / 32, KK = KP / 64, OB = kOpBytes<T>;    // a wave's half of the channels
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char *const sX = smem, *const sR = sX + 4 * kOp2Bytes, *const sS = sR + 4 * kOp2Bytes, *const sD = sS + 2 * KT * kOp2Bytes,
         *const sY = sD + 2 * KT * kOp2Bytes;
    char *const sFT = smem, *const sET = sFT + 6 * kOp2Bytes, *const sF = sET + 6 * kOp2Bytes, *const sE = sF + 6 * kOp2Bytes;
    char *const sC = smem + grad_main<T, KP>(), *const sQ = sC + QSide<T, KP>::kBytes;
    __shared__ real sG[kC];
    __shared__ float sB[kC], sQK[2][kC], sZ[2][kC], sTot[8];
    const DeltaArgs &a = p.b.fwd;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), w = wave % 4, wh = wave / 4;
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
    const size_t VK = static_cast<size_t>(V) * K;
    const rsrc_t rk = chunk_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, n, a.ldk, K, sizeof(T));
    const rsrc_t rq = chunk_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K, n, a.ldq, K, sizeof(T));
    const auto at = GradStage<T, KP>::at(H * V, K, V, n);
    GradStage<T, KP> st;
    auto load = [&](int64_t head, int v0) {
        const int64_t unit = slot * H + head;
        const float *const saved = a.ckpt + unit * (VK + kC * V);
        st.load(make_rsrc(saved, static_cast<uint32_t>(VK * 4)), make_rsrc(p.dS + unit * VK, static_cast<uint32_t>(VK * 4)),
                make_rsrc(wh ? saved + VK : p.dX + unit * kC * V), make_rsrc(static_cast<const T *>(p.b.dout) + (row0 * H + head) * V), at, v0, V);
    };
    {
        QSide<T, KP> side;
        const int64_t ld = wh ? a.ldq : a.ldk;
        side.load(wh ? rq : rk, ld, QSide<T, KP>::offsets(ld, K, threadIdx.x % kThreads));
        load(kh * group, 0);
        side.put(wh ? sQ : sC, threadIdx.x % kThreads);
    }
    f32x4 dqs[SHARED ? KT : 1], dks[SHARED ? KT : 1];
    if constexpr (SHARED) {
#pragma unroll
        for (int i = 0; i < KT; ++i) dqs[i] = dks[i] = zero;
    }
    for (int hh = 0; hh < group; ++hh) {
        const int64_t head = kh * group + hh, unit = slot * H + head;
        const float *const scal = p.ws.scal + unit * 3 * kC;
        if (wave == 0) {
            const real G = lane_prefix<real>(lane < n ? D::scaled(step_log(a.g[(row0 + lane) * H + head])) : real(0), lane);
            sG[lane] = G;
            sB[lane] = scal[2 * kC + lane];
        }
        const float eg = scal[t], wt = scal[kC + t], end = scal[kC - 1];
        // A: (F diag(beta))^T or F, B: M^T or -E
        f32x4 dq[KT], ke[KT], kw[KT], A[4], B[4];
#pragma unroll
        for (int i = 0; i < KT; ++i) dq[i] = ke[i] = kw[i] = zero;
#pragma unroll
        for (int i = 0; i < 4; ++i) A[i] = B[i] = zero;
        float tot = 0.0f;
        for (int v0 = 0; v0 < V; v0 += 32) {
            tot += st.put(sS, sD, sX, sY);                   // sX's waves 4 .. 7 write sR
            if (v0 + 32 < V) load(head, v0 + 32);
            else if (hh + 1 < group) load(head + 1, 0);
            __syncthreads();
            const Op<T> y = get_op(sY + w * OB, lane, T());
            const Op2<T> x = get_op2(sX + w * kOp2Bytes, lane, T()), r = get_op2(sR + w * kOp2Bytes, lane, T());
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Op2<T> s = get_op2(sS + (wh * KT + kt) * kOp2Bytes, lane, T()), d = get_op2(sD + (wh * KT + kt) * kOp2Bytes, lane, T());
                dq[kt] = mma(s, y, dq[kt]);
                ke[kt] = mma(s, x, ke[kt]);
                kw[kt] = mma(d, r, kw[kt]);
            }
#pragma unroll
            for (int ob = 0; ob < 4; ++ob) {
                if (wh == 0 && ob / 2 <= w / 2) {            // rows s at or before the pair's steps
                    const Op2<T> ro = get_op2(sR + ob * kOp2Bytes, lane, T());
                    A[ob] = mma(ro, y, A[ob]);
                    B[ob] = mma(ro, x, B[ob]);
                }
                if (wh == 1 && ob / 2 >= w / 2) {            // rows t at or behind them
                    A[ob] = mma(get_op(sY + ob * OB, lane, T()), r, A[ob]);
                    B[ob] = mma(get_op2(sX + ob * kOp2Bytes, lane, T()), r, B[ob]);
                }
            }
            __syncthreads();
        }
        const float beta = sB[t];
        const real gt = sG[t];
#pragma unroll
        for (int ob = 0; ob < 4; ++ob)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = 32 * (ob / 2) + 8 * g + 4 * (ob % 2) + i;      // the row: s or t
                const bool in = wh ? o >= t : o <= t;
                const float d = in ? D::ex(wh ? sG[o] - gt : gt - sG[o]) * (wh ? 1.0f : sB[o]) : 0.0f;
                A[ob][i] = in ? A[ob][i] * (a.scale * d) : 0.0f;
                B[ob][i] = in && o != t ? B[ob][i] * -d : 0.0f;
            }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            if (wh == 0 && kk <= w / 2) {
                put_op(sFT + tri_low(w, kk) * kOp2Bytes, lane, computed<T>(A[2 * kk], A[2 * kk + 1]));
                put_op(sET + tri_low(w, kk) * kOp2Bytes, lane, computed<T>(B[2 * kk], B[2 * kk + 1]));
            }
            if (wh == 1 && kk >= w / 2) {
                put_op(sF + tri_up(w, kk) * kOp2Bytes, lane, computed<T>(A[2 * kk], A[2 * kk + 1]));
                put_op(sE + tri_up(w, kk) * kOp2Bytes, lane, computed<T>(B[2 * kk], B[2 * kk + 1]));
            }
        }
        float qd = 0.0f, kd = 0.0f, kz = 0.0f, kc = 0.0f;
        const float fq = a.scale * eg;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            dq[kt] = dq[kt] * fq;
            ke[kt] = ke[kt] * -eg;
            kw[kt] = kw[kt] * wt;                            // Z
        }
        float kv[KK][8], qv[KK][8];
#pragma unroll
        for (int kp = 0; kp < KK; ++kp) {
            const int k0 = 32 * (wh * KK + kp) + 8 * g;
            floats(load_op(rk, k0 < K ? static_cast<uint32_t>((t * a.ldk + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone, T()), kv[kp]);
            floats(load_op(rq, k0 < K ? static_cast<uint32_t>((t * a.ldq + k0) * static_cast<int64_t>(sizeof(T))) : kOffNone, T()), qv[kp]);
        }
        __syncthreads();
#pragma unroll
        for (int kp = 0; kp < KK; ++kp)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) kc = fmaf(kv[kp][4 * h + i], kw[2 * kp + h][i], kc);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            if (kk <= w / 2) {
                const Op2<T> ft = get_op2(sFT + tri_low(w, kk) * kOp2Bytes, lane, T()), et = get_op2(sET + tri_low(w, kk) * kOp2Bytes, lane, T());
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    const Op<T> kcol = get_col<KP>(sC, sC, wh * KT + kt, kk, lane, T());
                    dq[kt] = mma(kcol, ft, dq[kt]);
                    ke[kt] = mma(kcol, et, ke[kt]);
                }
            }
            if (kk >= w / 2) {
                const Op2<T> f = get_op2(sF + tri_up(w, kk) * kOp2Bytes, lane, T()), e = get_op2(sE + tri_up(w, kk) * kOp2Bytes, lane, T());
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
        tot = wave_fold(fmaf(end, tot, beta * kc), AddOp());
        if (lane == 0) sTot[wave] = tot;
        if (g == 0) {
            sQK[wh][t] = qk;
            sZ[wh][t] = z;
        }
        __syncthreads();
        if (wave == 0) {                                     // lane l is step 63 - l: sums from the end
            const int l = 63 - lane;
            const float zl = sZ[0][l] + sZ[1][l];
            double v = static_cast<double>(sQK[0][l]) + sQK[1][l] - static_cast<double>(sB[l]) * zl;
            if (lane == 0)
                for (int i = 0; i < 8; ++i) v += sTot[i];
            v = lane_prefix<double>(v, lane);
            if (l < n) {
                p.b.dg[(row0 + l) * H + head] = static_cast<float>(v);
                p.b.dbeta[(row0 + l) * H + head] = zl;
            }
        }
        if constexpr (SHARED) {
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                dqs[i] = dqs[i] + dq[i];
                dks[i] = dks[i] + ke[i];
            }
        } else {
            store_keys<T, KP>(p, dq, ke, row0, kh, t, wh, g, n);
        }
    }
    if constexpr (SHARED) store_keys<T, KP>(p, dqs, dks, row0, kh, t, wh, g, n);
}

// bf16: 64 value channels to a workgroup while the CUs hold them all, else 128
template <int KP, int NW> hipError_t launch_rev_flow(const BwdParams &p, hipStream_t s) {
    constexpr int wide = 16 * NW;
    const DeltaShape &sh = p.b.fwd.s;
    constexpr size_t lds = 2 * FlowBuf<KP, NW>::bytes;
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
