// The two passes that the gated delta rule and its gradient share: what a chunk
// needs of its keys and queries alone (delta_prep_kernel), and the recurrence over
// the chunks (delta_seq_kernel).
#pragma once

#include "delta_tile.h"

namespace ssm {
namespace delta {
namespace {

// The workspace's parts per (chunk slot, head).
struct ChunkWs {
    char *t, *p;                    // T and P as operands (kTriBytes each); in the gradient T, T^T and P^T
    char *tt;
    float *scal;                    // 3 x 64: exp(G), exp(G_end - G), beta
};

struct SeqParams {
    DeltaArgs a;
    ChunkWs ws;
    float *R;                       // per (slot, head): (64, V) fp32, or null
};

// ---------------------------------------------------------------- preparation
// A wave per (chunk, head).  With Gam_ts = exp(G_t - G_s) (s <= t):
//     N = stril(K K^T o Gam) diag(beta),  T = (I + N)^-1,  P = tril(Q K^T o Gam)
// T is found column by column, one column per lane, by forward substitution: the
// rows of N are the same for all lanes (LDS broadcasts), T never leaves the
// registers until it is done.
template <typename T, int KP, bool BWD> __global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs a, ChunkWs ws) {
    using D = Decay<T>;
    using real = typename D::real;
    constexpr int KK = KP / 32;
    constexpr int LN = 68;                             // floats of a row of N: 16-byte rows, four banks apart
    __shared__ __attribute__((aligned(16))) float sN[kWaves][kC][LN];
    __shared__ real sG[kWaves][kC];
    __shared__ float sB[kWaves][kC];
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWaves + w;
    if (unit >= a.s.slots * a.s.heads) return;
    const int64_t slot = unit / a.s.heads, head = unit % a.s.heads, kh = head / (a.s.heads / a.s.kheads);
    const Span sp = span_of(a.s, sequence_of(a.s, slot));
    const int64_t step0 = (slot - sp.slot0) * kC;
    if (step0 < 0 || step0 >= sp.len) return;          // a slot that no sequence uses
    const int n = sp.len - step0 < kC ? static_cast<int>(sp.len - step0) : kC;
    const int K = static_cast<int>(a.s.dk);
    const int64_t row0 = sp.row0 + step0;

    const int64_t at = (row0 + (lane < n ? lane : 0)) * a.s.heads + head;
    const real G = lane_prefix<real>(lane < n ? D::scaled(step_log(a.g[at])) : real(0), lane);
    const float beta = lane < n ? a.beta[at] : 0.0f;
    const real end = __shfl(G, 63);
    float *scal = ws.scal + unit * 3 * kC;
    scal[lane] = D::ex(G);
    scal[kC + lane] = D::ex(end - G);
    scal[2 * kC + lane] = beta;
    sG[w][lane] = G;
    sB[w][lane] = beta;

    const rsrc_t rk = make_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K);
    const rsrc_t rq = make_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K);
    Op<T> k[4][KK];
    auto load = [&](Op<T>(&dst)[4][KK], rsrc_t r, int64_t ld) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const int t = row_index(tb, c), ch = 32 * kk + 8 * g;
                dst[tb][kk] = load_op(r, t < n && ch < K ? static_cast<uint32_t>((t * ld + ch) * static_cast<int64_t>(sizeof(T))) : kOffNone, T());
            }
    };
    load(k, rk, a.ldk);
    wave_sync();
    const f32x4 zero = {0, 0, 0, 0};
    // N by rows: a lane holds four neighbouring s of one t
#pragma unroll
    for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int sb = 0; sb < 2 * (tb / 2) + 2; ++sb) {
            f32x4 acc = zero;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) acc = mma(k[sb][kk], k[tb][kk], acc);
            const int t = row_index(tb, c), s0 = 32 * (sb / 2) + 8 * g + 4 * (sb % 2);
            const real gt = sG[w][t];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = s0 + i < t ? acc[i] * D::ex(gt - sG[w][s0 + i]) * sB[w][s0 + i] : 0.0f;
            *reinterpret_cast<f32x4 *>(&sN[w][t][s0]) = acc;
        }
    wave_sync();
    // column `lane` of T: x_t = [t == lane] - sum_{s < t} N_ts x_s
    float x[kC];
#pragma unroll
    for (int t = 0; t < kC; ++t) {
        float v = t == lane ? 1.0f : 0.0f;
#pragma unroll
        for (int s = 0; s < t; s += 4) {
            const f32x4 nrow = *reinterpret_cast<const f32x4 *>(&sN[w][t][s]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s + i < t) v = fmaf(-nrow[i], x[s + i], v);
        }
        x[t] = v;
    }
    wave_sync();
#pragma unroll
    for (int t = 0; t < kC; ++t) sN[w][t][lane] = x[t];
    wave_sync();
    char *const to = ws.t + unit * kTriBytes;
#pragma unroll
    for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int kk = 0; kk <= tb / 2; ++kk) {
            const float *row = &sN[w][row_index(tb, c)][32 * kk + 8 * g];
            put_op(to + tri_low(tb, kk) * kOp2Bytes, lane,
                   computed<T>(*reinterpret_cast<const f32x4 *>(row), *reinterpret_cast<const f32x4 *>(row + 4)));
        }
    if constexpr (BWD) {
        char *const tto = ws.tt + unit * kTriBytes;
#pragma unroll
        for (int sb = 0; sb < 4; ++sb)
#pragma unroll
            for (int kk = sb / 2; kk < 2; ++kk) {
                const int s = row_index(sb, c), t0 = 32 * kk + 8 * g;
                f32x4 u, v;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    u[i] = sN[w][t0 + i][s];
                    v[i] = sN[w][t0 + 4 + i][s];
                }
                put_op(tto + tri_up(sb, kk) * kOp2Bytes, lane, computed<T>(u, v));
            }
    }
    // P as operands: rows t and steps s along K, or (gradient) rows s and steps t along K
    Op<T> q[4][KK];
    load(q, rq, a.ldq);
    char *const po = ws.p + unit * kTriBytes;
#pragma unroll
    for (int rb = 0; rb < 4; ++rb)                     // the operand's row tile
#pragma unroll
        for (int kk = BWD ? rb / 2 : 0; kk < (BWD ? 2 : rb / 2 + 1); ++kk) {
            f32x4 acc[2];
            const int r = row_index(rb, c);
            const real gr = sG[w][r];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                acc[h] = zero;
#pragma unroll
                for (int ks = 0; ks < KK; ++ks)
                    acc[h] = BWD ? mma(q[2 * kk + h][ks], k[rb][ks], acc[h]) : mma(k[2 * kk + h][ks], q[rb][ks], acc[h]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int o = 32 * kk + 8 * g + 4 * h + i;         // the other index
                    const bool in = BWD ? r <= o : o <= r;
                    const real d = BWD ? sG[w][o] - gr : gr - sG[w][o];
                    acc[h][i] = in ? acc[h][i] * D::ex(d) : 0.0f;
                }
            }
            put_op(po + (BWD ? tri_up(rb, kk) : tri_low(rb, kk)) * kOp2Bytes, lane, computed<T>(acc[0], acc[1]));
        }
}

// ------------------------------------------------------------------ recurrence
// A workgroup owns (sequence, head, 64 value channels) and walks the chunks; a wave
// keeps 16 channels' state (K x 16, fp32) in accumulator tiles.  A chunk, with S
// the state entering it:
//     X = V - exp(G) K S,  R = T X,  U = beta R
//     Y = scale (exp(G) Q S + P U),  S <- exp(G_end) S + K^T (exp(G_end - G) U)
// Every product's computed operand comes from the accumulators of the one before;
// K, K^T, Q, T and P are shared by the waves through LDS.
//   OUT: y is computed (else the states, and R, alone).
//   ONE: a workgroup does a single chunk from its checkpoint (R of all chunks at once).
template <typename T, int KP, bool OUT, bool ONE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 2 : 1))) void delta_seq_kernel(SeqParams p) {
    constexpr int KT = KP / 16, KK = KP / 32, RB = kRowBytes<T>;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char *const sK = smem, *const sC = sK + Rows<T, KP>::kBytes, *const sT = sC + Cols<T, KP>::kBytes;
    float *const sS = reinterpret_cast<float *>(sT + kTriBytes);
    char *const sV = sT + kTriBytes + 3 * kC * 4, *const sP = sV + Values<T>::kBytes, *const sQ = sP + kTriBytes;
    const DeltaArgs &a = p.a;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    const int nvt = (V + 63) / 64;
    const int vt = blockIdx.x % nvt;
    const int64_t rest = blockIdx.x / nvt, head = rest % H, kh = head / (H / a.s.kheads);
    const int64_t seq = ONE ? sequence_of(a.s, rest / H) : rest / H;
    const Span sp = span_of(a.s, seq);
    const int nchunks = (sp.len + kC - 1) / kC;
    int j0 = 0, j1 = nchunks;
    if constexpr (ONE) {
        const int64_t j = rest / H - sp.slot0;
        if (j < 0 || j >= nchunks) return;
        j0 = static_cast<int>(j);
        j1 = j0 + 1;
    }
    const int v0 = vt * 64 + w * 16;
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    f32x4 S[KT];
    if constexpr (ONE) {
        load_state<KP>(S, a.ckpt + ((sp.slot0 + j0) * H + head) * VK, v0, V, K, lane);
    } else if (a.h0) {
        load_state<KP>(S, a.h0 + (seq * H + head) * VK, v0, V, K, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) S[i] = zero;
    }
    // the next chunk's data, a chunk ahead; past the last one all of it is out of range
    Rows<T, KP> nK, nQ;
    Cols<T, KP> nC;
    Copy<kTriBytes> nT, nP;
    float nS;
    Values<T> nV;
    const uint32_t okr = Rows<T, KP>::offset(a.ldk, K), oqr = Rows<T, KP>::offset(a.ldq, K);
    const auto okc = Cols<T, KP>::offsets(a.ldk, K);
    const int ldv = static_cast<int>(a.ldv);
    const uint32_t ov = Values<T>::offset(ldv, V - vt * 64, w, lane);
    auto prefetch = [&](int j) {
        const int jj = j < j1 ? j : j1 - 1;
        const int64_t row0 = sp.row0 + static_cast<int64_t>(jj) * kC, unit = (sp.slot0 + jj) * H + head;
        const int n = j < j1 ? (sp.len - j * kC < kC ? sp.len - j * kC : kC) : 0;
        const rsrc_t rk = chunk_rsrc(static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, n, a.ldk, K, sizeof(T));
        const rsrc_t rv = chunk_rsrc(static_cast<const T *>(a.v) + row0 * a.ldv + head * V + vt * 64, n, a.ldv, V - vt * 64, sizeof(T));
        nK.load(rk, a.ldk, okr);
        nV.load(rv, ldv, ov);
        nT.load(p.ws.t + unit * kTriBytes);
        nS = p.ws.scal[unit * 3 * kC + (threadIdx.x < 3 * kC ? threadIdx.x : 0)];
        if constexpr (OUT) {
            nQ.load(chunk_rsrc(static_cast<const T *>(a.q) + row0 * a.ldq + kh * K, n, a.ldq, K, sizeof(T)), a.ldq, oqr);
            nP.load(p.ws.p + unit * kTriBytes);
        }
        if constexpr (!ONE) nC.load(rk, a.ldk, okc);
    };
    if (j0 < j1) prefetch(j0);
    for (int j = j0; j < j1; ++j) {
        const int64_t row0 = sp.row0 + static_cast<int64_t>(j) * kC, unit = (sp.slot0 + j) * H + head;
        const int n = sp.len - j * kC < kC ? sp.len - j * kC : kC;
        __syncthreads();                                   // the chunk before is done with LDS
        nK.put(sK);
        nT.put(sT);
        if (threadIdx.x < 3 * kC) sS[threadIdx.x] = nS;
        if constexpr (OUT) {
            nQ.put(sQ);
            nP.put(sP);
        }
        if constexpr (!ONE) nC.put(sC);
        nV.put(sV);
        const Values<T> cV = nV;
        __syncthreads();
        if constexpr (!ONE) {
            if (a.ckpt) store_state<KP>(S, a.ckpt + unit * VK, v0, V, K, lane);
            prefetch(j + 1);
        }
        Op2<T> so[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) so[kk] = computed<T>(S[2 * kk], S[2 * kk + 1]);
        f32x4 ks[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) ks[tb] = mma(get_row(sK + (tb * KK + kk) * RB, lane, T()), so[kk], ks[tb]);
        f32x4 X[4];
        tiles(cV.op(sV, 0, w, lane), X[0], X[1]);
        tiles(cV.op(sV, 1, w, lane), X[2], X[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const f32x4 eg = *reinterpret_cast<const f32x4 *>(&sS[32 * (tb / 2) + 8 * g + 4 * (tb % 2)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) X[tb][i] = fmaf(-eg[i], ks[tb][i], X[tb][i]);
        }
        f32x4 y[OUT ? 4 : 1];                              // transposed: rows are channels, columns steps
        if constexpr (OUT) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) y[tb] = zero;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) y[tb] = mma(so[kk], get_row(sQ + (tb * KK + kk) * RB, lane, T()), y[tb]);
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) y[tb] = y[tb] * sS[row_index(tb, c)];
        }
        const Op2<T> xo[2] = {computed<T>(X[0], X[1]), computed<T>(X[2], X[3])};
        if constexpr (!OUT) {                              // R, transposed, for stores of four channels
            const rsrc_t rr = make_rsrc(p.R + unit * kC * V, static_cast<uint32_t>(kC * V * 4));
            f32x4 rt[4] = {zero, zero, zero, zero};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb) rt[tb] = mma(xo[kk], get_op2(sT + tri_low(tb, kk) * kOp2Bytes, lane, T()), rt[tb]);
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) store4(rt[tb], rr, v < V ? static_cast<uint32_t>((row_index(tb, c) * V + v) * 4) : kOffNone);
        }
        if constexpr (ONE) return;
        f32x4 R[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 2 * kk; tb < 4; ++tb) R[tb] = mma(get_op2(sT + tri_low(tb, kk) * kOp2Bytes, lane, T()), xo[kk], R[tb]);
        f32x4 W[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = 32 * (tb / 2) + 8 * g + 4 * (tb % 2);
            R[tb] = R[tb] * *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t]);       // U
            W[tb] = R[tb] * *reinterpret_cast<const f32x4 *>(&sS[kC + t]);
        }
        if constexpr (OUT) {
            const Op2<T> uo[2] = {computed<T>(R[0], R[1]), computed<T>(R[2], R[3])};
            const rsrc_t ry = make_rsrc(static_cast<T *>(a.y) + (row0 * H + head) * V);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb) y[tb] = mma(uo[kk], get_op2(sP + tri_low(tb, kk) * kOp2Bytes, lane, T()), y[tb]);
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const int t = row_index(tb, c), v = v0 + 4 * g;
                store_io4(y[tb] * a.scale, ry, t < n && v < V ? static_cast<uint32_t>((t * H * V + v) * static_cast<int64_t>(sizeof(T))) : kOffNone, T());
            }
        }
        const Op2<T> wo[2] = {computed<T>(W[0], W[1]), computed<T>(W[2], W[3])};
        const float end = sS[kC - 1];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = S[kt] * end;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) S[kt] = mma(get_col<KP>(sK, sC, kt, kk, lane, T()), wo[kk], S[kt]);
    }
    if constexpr (!ONE)
        if (a.last_state) store_state<KP>(S, a.last_state + (seq * H + head) * VK, v0, V, K, lane);
}

template <typename T, int KP, bool OUT> constexpr size_t seq_lds() {
    return Rows<T, KP>::kBytes + Cols<T, KP>::kBytes + kTriBytes + 3 * kC * 4 + Values<T>::kBytes + (OUT ? kTriBytes + Rows<T, KP>::kBytes : 0);
}

inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <typename T, int KP, bool BWD> hipError_t launch_prep(const DeltaArgs &a, const ChunkWs &ws, hipStream_t s) {
    const int64_t units = a.s.slots * a.s.heads;
    hipLaunchKernelGGL((delta_prep_kernel<T, KP, BWD>), dim3(static_cast<unsigned>((units + kWaves - 1) / kWaves)), dim3(kThreads),
                       0, s, a, ws);
    return hipGetLastError();
}
template <typename T, int KP, bool OUT, bool ONE> hipError_t launch_seq(const SeqParams &p, hipStream_t s) {
    const int64_t nvt = (p.a.s.dv + 63) / 64;
    const int64_t grid = nvt * p.a.s.heads * (ONE ? p.a.s.slots : p.a.s.nseq);
    constexpr size_t lds = seq_lds<T, KP, OUT>();
    hipLaunchKernelGGL((delta_seq_kernel<T, KP, OUT, ONE>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), lds, s, p);
    return hipGetLastError();
}

}  // namespace
}  // namespace delta
}  // namespace ssm
