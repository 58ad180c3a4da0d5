// The two passes that the gated delta rule and its gradient share: what a chunk
// needs of its keys and queries alone (delta_prep_kernel), and the recurrence over
// the chunks (delta_seq_kernel for fp32, delta_flow.h for bf16).
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
    int cps;                        // chunks of a time segment
    bool wide, wide_ends;           // see Plan
    int64_t segments, edges;        // and their borders (see Segment)
    float *ends;                    // per (border, head): (V, K) fp32, the state that passes it
    char *maps;                     // per (border, head): the transition of the segment that ends there, as operands
};
// Operands of a segment's transition: (KP / 32, KP / 16) of them.
template <int KP> constexpr int64_t kMapBytes = static_cast<int64_t>(KP / 32) * (KP / 16) * kOp2Bytes;

// ---------------------------------------------------------------- preparation
// A wave per (chunk, head).  With Gam_ts = exp(G_t - G_s) (s <= t):
//     N = stril(K K^T o Gam) diag(beta),  T = (I + N)^-1,  P = tril(Q K^T o Gam)
// T's 16 x 16 diagonal blocks come from forward substitution, one column to a lane, the
// others from them in fp32 products on the matrix cores: stable whatever the keys,
// unlike powers of N.  One column of all 64 steps to a lane instead, with 2016
// multiplications and 504 LDS broadcasts: 10240 chunks of 64 x 128 145 us, this way 109 (253 MB
// of T and P are written).
template <typename T, int KP, bool BWD> __global__ __launch_bounds__(kThreads) void delta_prep_kernel(DeltaArgs a, ChunkWs ws) {
    using D = Decay<T>;
    constexpr int KK = KP / 32;
    constexpr int LN = 68;                             // floats of a row of N: 16-byte rows, four banks apart
    __shared__ __attribute__((aligned(16))) float sN[kWaves][kC][LN];
    __shared__ double sG[kWaves][kC];
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
    const double G = lane_prefix(lane < n ? D::scaled(step_log(a.g[at])) : 0.0, lane);
    const float beta = lane < n ? a.beta[at] : 0.0f;
    const double end = __shfl(G, 63);
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
            const double gt = sG[w][t];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = s0 + i < t ? acc[i] * D::ex(gt - sG[w][s0 + i]) * sB[w][s0 + i] : 0.0f;
            *reinterpret_cast<f32x4 *>(&sN[w][t][s0]) = acc;
        }
    wave_sync();
    // the diagonal blocks' inverses D, one block to 16 lanes, one column to a lane:
    // x_t = [t == c] - sum_{s < t} N_ts x_s; each takes its block's place in sN
    {
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
            float v = t == c ? 1.0f : 0.0f;
#pragma unroll
            for (int s = 0; s < t; s += 4) {
                const f32x4 nrow = *reinterpret_cast<const f32x4 *>(&sN[w][16 * g + t][16 * g + s]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s + i < t) v = fmaf(-nrow[i], x[s + i], v);
            }
            x[t] = v;
        }
        wave_sync();
#pragma unroll
        for (int t = 0; t < 16; ++t) sN[w][16 * g + t][16 * g + c] = x[t];
    }
    wave_sync();
    // T_ij = -D_i sum_{j <= m < i} N_im T_mj, in fp32 products of 16 x 16 blocks: the right factor is always an
    // accumulator tile (rows 4 g + i, column c), taken along K in that order; the left one is four floats of a row
    {
        auto left = [&](int i, int m) { return *reinterpret_cast<const f32x4 *>(&sN[w][16 * i + c][16 * m + 4 * g]); };
        auto product = [](f32x4 l, f32x4 r, f32x4 acc) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(l[i], r[i], acc, 0, 0, 0);
            return acc;
        };
        f32x4 t[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 4; ++h) t[i][i][h] = sN[w][16 * i + 4 * g + h][16 * i + c];
#pragma unroll
        for (int d = 1; d < 4; ++d)
#pragma unroll
            for (int j = 0; j + d < 4; ++j) {
                const int i = j + d;
                f32x4 z = zero;
#pragma unroll
                for (int m = j; m < i; ++m) z = product(left(i, m), t[m][j], z);
                t[i][j] = product(-left(i, i), z, zero);
            }
        wave_sync();
#pragma unroll
        for (int i = 1; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < i; ++j)
#pragma unroll
                for (int h = 0; h < 4; ++h) sN[w][16 * i + 4 * g + h][16 * j + c] = t[i][j][h];
    }
    wave_sync();
    char *const to = ws.t + unit * kTriBytes;
    if (!BWD || ws.t)                                  // the gradient needs T itself only where it walks forward first
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
            const double gr = sG[w][r];
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
                    const double d = BWD ? sG[w][o] - gr : gr - sG[w][o];
                    acc[h][i] = in ? acc[h][i] * D::ex(d) : 0.0f;
                }
            }
            put_op(po + (BWD ? tri_up(rb, kk) : tri_low(rb, kk)) * kOp2Bytes, lane, computed<T>(acc[0], acc[1]));
        }
}

// ------------------------------------------------------------------ recurrence
// A workgroup owns (sequence's time segment, head, 64 value channels) and walks the
// chunks; a wave keeps 16 channels' state (K x 16, fp32) in accumulator tiles.  This
// kernel is fp32's; bf16's has a wave that loads (delta_flow.h).  A chunk, with S the
// state entering it:
//     X = V - exp(G) K S,  R = T X,  U = beta R
//     Y = scale (exp(G) Q S + P U),  S <- exp(G_end) S + K^T (exp(G_end - G) U)
// Every product's computed operand comes from the accumulators of the one before;
// K, Q, T and P are shared by the waves through LDS.
//
// A sequence is one segment where there are heads enough to fill the GPU.  Else it
// is cut: kEnds finds what every segment but the last leaves from zero, and its
// transition (the state is an affine function of the one entering: 64 channels more
// that start as columns of the identity, with V = 0); delta_carry_kernel joins them,
// and the pass proper starts every segment from the state it is entered with.
enum Mode {
    kOut,       // y
    kTrain,     // y, and for the gradient to come the states entering the chunks, and R
    kSave,      // these alone
    kEnds       // the segments' ends
};
constexpr bool has_out(Mode m) { return m == kOut || m == kTrain; }
constexpr bool has_save(Mode m) { return m == kTrain || m == kSave; }
// A wave's 16 columns n of a segment's transition, as operands with n along K; by all
// waves of a workgroup whose first column is n0.
template <typename T, int KP, int NW> __device__ __forceinline__ void store_map(const f32x4 (&S)[KP / 16], char *smem, int w, int lane, char *out, int n0) {
    constexpr int KT = KP / 16, LM = KP + 4, kWide = 16 * NW;
    float *const sM = reinterpret_cast<float *>(smem);
    const int g = lane / 16, c = lane % 16;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < KT; ++q) *reinterpret_cast<f32x4 *>(&sM[(16 * w + c) * LM + 32 * (q / 2) + 8 * g + 4 * (q % 2)]) = S[q];
    __syncthreads();
    const int nk = KP - n0 < kWide ? (KP - n0) / 32 : kWide / 32;
    for (int f = w; f < nk * KT; f += NW) {
        const int kk = f / KT, kt = f % KT, k = row_index(kt, c);
        f32x4 x, y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = sM[(32 * kk + 8 * g + i) * LM + k];
            y[i] = sM[(32 * kk + 8 * g + 4 + i) * LM + k];
        }
        put_op(out + ((n0 / 32 + kk) * KT + kt) * kOp2Bytes, lane, computed<T>(x, y));
    }
}
// columns col0 + c of the identity
template <int KP> __device__ __forceinline__ void unit_columns(f32x4 (&S)[KP / 16], int col0, int lane) {
    const int g = lane / 16, col = col0 + lane % 16;
#pragma unroll
    for (int q = 0; q < KP / 32; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            S[2 * q][i] = 32 * q + 8 * g + i == col ? 1.0f : 0.0f;
            S[2 * q + 1][i] = 32 * q + 8 * g + 4 + i == col ? 1.0f : 0.0f;
        }
}
template <int KP, Mode MODE> __global__ __launch_bounds__(kThreads) void delta_seq_kernel(SeqParams p) {
    using T = float;
    constexpr int KT = KP / 16, KK = KP / 32, RB = kRowBytes<T>;
    constexpr bool OUT = has_out(MODE), SAVE = has_save(MODE);
    extern __shared__ __attribute__((aligned(16))) char smem[];
    char *const sK = smem, *const sC = sK + Rows<T, KP>::kBytes, *const sT = sC + Cols<KP>::kBytes;
    float *const sS = reinterpret_cast<float *>(sT + kTriBytes);
    char *const sP = sT + kTriBytes + 3 * kC * 4, *const sQ = sP + kTriBytes;
    const DeltaArgs &a = p.a;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    constexpr int kWide = 64;
    const int nvt = (V + kWide - 1) / kWide, tiles_n = MODE == kEnds ? nvt + (KP + kWide - 1) / kWide : nvt;
    const int tile = blockIdx.x % tiles_n;
    const int64_t rest = blockIdx.x / tiles_n, head = rest % H, kh = head / (H / a.s.kheads), id = rest / H;
    Span sp;
    const Segment sg = segment_of<MODE == kEnds ? kBeforeEdges : kAllSegments>(a.s, id, p.edges, p.cps, sp);
    if (!sg.used) return;
    const int64_t seq = sg.seq;
    const int j0 = sg.j0, j1 = sg.j1;
    const bool first = sg.s == 0, last = sg.last;
    const bool transition = MODE == kEnds && tile >= nvt;
    if (MODE == kEnds && first && transition) return;
    const int vt = transition ? 0 : tile;
    const int v0 = vt * kWide + w * 16;                    // the wave's first channel
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    f32x4 S[KT];
    if (transition) {
        unit_columns<KP>(S, (tile - nvt) * kWide + w * 16, lane);
    } else if (MODE != kEnds && !first) {
        load_state<KP>(S, p.ends + (sg.edge * H + head) * VK, v0, V, K, lane);
    } else if (first && a.h0) {
        load_state<KP>(S, a.h0 + (seq * H + head) * VK, v0, V, K, lane);
    } else {
#pragma unroll
        for (int i = 0; i < KT; ++i) S[i] = zero;
    }
    // the next chunk's data, a chunk ahead; past the last one all of it is out of range
    Rows<T, KP> nK, nQ;
    Cols<KP> nC;
    Copy<kTriBytes> nT, nP;
    float nS;
    Values nV;
    const uint32_t okr = Rows<T, KP>::offset(a.ldk, K, threadIdx.x), oqr = Rows<T, KP>::offset(a.ldq, K, threadIdx.x);
    const auto okc = Cols<KP>::offsets(a.ldk, K, threadIdx.x);
    const int ldv = static_cast<int>(a.ldv);
    const uint32_t ov = Values::offset(ldv, V - vt * kWide, w, lane);
    // addresses move on by whole chunks; loads are issued in two parts, each beside products, as a chunk's loads take
    // the memory pipe longer than the waves can queue them
    const T *pk = static_cast<const T *>(a.k) + (sp.row0 + static_cast<int64_t>(j0) * kC) * a.ldk + kh * K;
    const T *pq = static_cast<const T *>(a.q) + (sp.row0 + static_cast<int64_t>(j0) * kC) * a.ldq + kh * K;
    const T *pv = static_cast<const T *>(a.v) + (sp.row0 + static_cast<int64_t>(j0) * kC) * a.ldv + head * V + vt * kWide;
    int64_t unit = (sp.slot0 + j0) * H + head;             // of the chunk at hand
    const char *pt = p.ws.t + unit * kTriBytes, *pp = p.ws.p + unit * kTriBytes;
    const float *ps = p.ws.scal + unit * 3 * kC;
    int left = sp.len - j0 * kC;
    const int tS = threadIdx.x < 3 * kC ? threadIdx.x : 0;
    auto prefetch1 = [&]() {
        const int n = left < kC ? left : kC;
        const rsrc_t rk = chunk_rsrc(pk, n, a.ldk, K, sizeof(T));
        nK.load(rk, a.ldk, okr);
        nC.load(rk, a.ldk, okc);
        nT.load(pt);
    };
    auto prefetch2 = [&]() {
        const int n = left < kC ? left : kC;
        nV.load(chunk_rsrc(pv, transition ? 0 : n, a.ldv, V - vt * kWide, sizeof(T)), ldv, ov);
        nS = ps[tS];
        if constexpr (OUT) {
            nQ.load(chunk_rsrc(pq, n, a.ldq, K, sizeof(T)), a.ldq, oqr);
            nP.load(pp);
        }
        left -= kC;
        if (left > 0) {                                    // else what is loaded is not used: the last chunk's again
            pk += kC * a.ldk;
            pq += kC * a.ldq;
            pv += kC * a.ldv;
            pt += H * kTriBytes;
            pp += H * kTriBytes;
            ps += H * 3 * kC;
        }
    };
    if (j0 < j1) {
        prefetch1();
        prefetch2();
    }
    for (int j = j0; j < j1; ++j, unit += H) {
        const int64_t row0 = sp.row0 + static_cast<int64_t>(j) * kC;
        const int n = sp.len - j * kC < kC ? sp.len - j * kC : kC;
        __syncthreads();                                   // the chunk before is done with LDS
        nK.put(sK, threadIdx.x);
        nT.put(sT);
        if (threadIdx.x < 3 * kC) sS[threadIdx.x] = nS;
        if constexpr (OUT) {
            nQ.put(sQ, threadIdx.x);
            nP.put(sP);
        }
        nC.put(sC, threadIdx.x);
        const Values cV = nV;
        __syncthreads();
        if constexpr (SAVE) store_state<KP>(S, a.ckpt + unit * (VK + kC * V), v0, V, K, lane);
        Op2<T> so[KK];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
            so[kk] = computed<T>(S[2 * kk], S[2 * kk + 1]);
        f32x4 ks[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) ks[tb] = zero;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const Op<T> f = get_row(sK + (tb * KK + kk) * RB, lane, T());
                ks[tb] = mma(f, so[kk], ks[tb]);
            }
        __builtin_amdgcn_sched_barrier(0);
        prefetch1();
        __builtin_amdgcn_sched_barrier(0);
        f32x4 y[4];                          // transposed: rows are channels, columns steps
        if constexpr (OUT) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) y[tb] = zero;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) {
                    const Op<T> f = get_row(sQ + (tb * KK + kk) * RB, lane, T());
                    y[tb] = mma(so[kk], f, y[tb]);
                }
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const float e = sS[row_index(tb, c)];
                y[tb] = y[tb] * e;
            }
        }
        Op2<T> xo[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {                      // 32 steps
            const f32x4 e0 = *reinterpret_cast<const f32x4 *>(&sS[32 * q + 8 * g]), e1 = *reinterpret_cast<const f32x4 *>(&sS[32 * q + 8 * g + 4]);
            f32x4 x0, x1;
            tiles(cV.op(q), x0, x1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x0[i] = fmaf(-e0[i], ks[2 * q][i], x0[i]);
                x1[i] = fmaf(-e1[i], ks[2 * q + 1][i], x1[i]);
            }
            xo[q] = computed<T>(x0, x1);
        }
        __builtin_amdgcn_sched_barrier(0);
        prefetch2();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (SAVE) {                              // R, transposed, for stores of four channels
            const rsrc_t rr = make_rsrc(a.ckpt + unit * (VK + kC * V) + VK, static_cast<uint32_t>(kC * V * 4));
            f32x4 rt[4];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) rt[tb] = zero;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb)
                    rt[tb] = mma(xo[kk], get_op2(sT + tri_low(tb, kk) * kOp2Bytes, lane, T()), rt[tb]);
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) stream4(rt[tb], rr, v < V ? static_cast<uint32_t>((row_index(tb, c) * V + v) * 4) : kOffNone);
        }
        f32x4 R[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) R[tb] = zero;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 2 * kk; tb < 4; ++tb) {
                const Op2<T> f = get_op2(sT + tri_low(tb, kk) * kOp2Bytes, lane, T());
                R[tb] = mma(f, xo[kk], R[tb]);
            }
        Op2<T> uo[2], wo[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = 32 * q + 8 * g;
            const f32x4 b0 = *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t]), b1 = *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t + 4]);
            const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&sS[kC + t]), w1 = *reinterpret_cast<const f32x4 *>(&sS[kC + t + 4]);
            const f32x4 u0 = R[2 * q] * b0, u1 = R[2 * q + 1] * b1;
            if constexpr (OUT) uo[q] = computed<T>(u0, u1);
            wo[q] = computed<T>(u0 * w0, u1 * w1);
        }
        if constexpr (OUT) {
            const rsrc_t ry = chunk_rsrc(static_cast<T *>(a.y) + (row0 * H + head) * V, n, H * V, V, sizeof(T));
            const int ldy = static_cast<int>(H) * V;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb) {
                    const Op2<T> f = get_op2(sP + tri_low(tb, kk) * kOp2Bytes, lane, T());
                    y[tb] = mma(uo[kk], f, y[tb]);
                }
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb)
                store_io4(y[tb] * a.scale, ry, v < V ? static_cast<uint32_t>((row_index(tb, c) * ldy + v) * static_cast<int>(sizeof(T))) : kOffNone, T());
        }
        const float end = sS[kC - 1];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = S[kt] * end;
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                const Op<T> f = get_col<KP>(sK, sC, kt, kk, lane, T());
                S[kt] = mma(f, wo[kk], S[kt]);
            }
    }
    if constexpr (MODE == kEnds) {
        if (!transition) {
            store_state<KP>(S, p.ends + ((sg.edge + 1) * H + head) * VK, v0, V, K, lane);
            return;
        }
        store_map<T, KP, kWaves>(S, smem, w, lane, p.maps + ((sg.edge + 1) * H + head) * kMapBytes<KP>, (tile - nvt) * kWide);
    } else {
        if (last && a.last_state) {
            store_state<KP>(S, a.last_state + (seq * H + head) * VK, v0, V, K, lane);
        }
    }
}

template <int KP, Mode MODE> constexpr size_t seq_lds() {
    using T = float;
    constexpr size_t n = Rows<T, KP>::kBytes + Cols<KP>::kBytes + kTriBytes + 3 * kC * 4 +
                         (has_out(MODE) ? kTriBytes + Rows<T, KP>::kBytes : 0), m = MODE == kEnds ? 64 * (KP + 4) * 4 : 0;
    return n > m ? n : m;
}

// What the segments leave, one after the other: from the state that the one before
// leaves, through the transition, plus what it leaves from zero.  REV: from the last one
// on, for the gradient.  A wave per (sequence, head, 16 value channels).
template <typename T, int KP, bool REV> __global__ __launch_bounds__(64) void delta_carry_kernel(SeqParams p) {
    constexpr int KT = KP / 16, KK = KP / 32;
    const DeltaArgs &a = p.a;
    const int lane = threadIdx.x, K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    const int nt = (V + 15) / 16, v0 = blockIdx.x % nt * 16;
    const int64_t rest = blockIdx.x / nt, head = rest % H, seq = rest / H;
    const Span sp = span_of(a.s, seq);
    const int nc = (sp.len + kC - 1) / kC, ns = (nc + p.cps - 1) / p.cps;
    if (ns < 3) return;
    const int64_t first = first_edge(a.s, seq, sp.slot0, ns, p.cps);
    const size_t VK = static_cast<size_t>(V) * K;
    f32x4 S[KT];
    auto unit = [&](int s) { return (first + (REV ? ns - 2 - s : s)) * H + head; };
    load_state<KP>(S, p.ends + unit(0) * VK, v0, V, K, lane);
    // a step is little more than the latency of its loads: as many steps ahead as registers hold
    constexpr int AHEAD = KP > 64 ? 1 : 3;
    struct Step {
        Op2<T> map[KK][KT];
        f32x4 end[KT];
    } next[AHEAD];
    auto fetch = [&](Step &f, int s) {
        const int64_t at = unit(s < ns - 1 ? s : ns - 2);
        const char *const m = p.maps + at * kMapBytes<KP>;
        load_state<KP>(f.end, p.ends + at * VK, v0, V, K, lane);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) f.map[kk][kt] = get_op2(m + (kk * KT + kt) * kOp2Bytes, lane, T());
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(next[d], 1 + d);
    for (int s0 = 1; s0 < ns - 1; s0 += AHEAD) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            const int s = s0 + d;
            if (s >= ns - 1) return;
            Op2<T> so[KK];
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) so[kk] = computed<T>(S[2 * kk], S[2 * kk + 1]);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) S[kt] = next[d].end[kt];
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) S[kt] = mma(next[d].map[kk][kt], so[kk], S[kt]);
            store_state<KP>(S, p.ends + unit(s) * VK, v0, V, K, lane);
            fetch(next[d], s + AHEAD);
        }
    }
}

inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

template <typename T, int KP, bool BWD> hipError_t launch_prep(const DeltaArgs &a, const ChunkWs &ws, hipStream_t s) {
    const int64_t units = a.s.slots * a.s.heads;
    hipLaunchKernelGGL((delta_prep_kernel<T, KP, BWD>), dim3(static_cast<unsigned>((units + kWaves - 1) / kWaves)), dim3(kThreads),
                       0, s, a, ws);
    return hipGetLastError();
}
template <int KP, Mode MODE> hipError_t launch_seq(const SeqParams &p, hipStream_t s) {
    constexpr int wide = 64;
    const int64_t nvt = (p.a.s.dv + wide - 1) / wide;
    const int64_t grid = (MODE == kEnds ? (nvt + (KP + wide - 1) / wide) * p.edges : nvt * p.segments) * p.a.s.heads;
    constexpr size_t lds = seq_lds<KP, MODE>();
    hipLaunchKernelGGL((delta_seq_kernel<KP, MODE>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), lds, s, p);
    return hipGetLastError();
}
template <typename T, int KP, bool REV> hipError_t launch_carry(const SeqParams &p, hipStream_t s) {
    const int64_t grid = (p.a.s.dv + 15) / 16 * p.a.s.heads * p.a.s.nseq;
    hipLaunchKernelGGL((delta_carry_kernel<T, KP, REV>), dim3(static_cast<unsigned>(grid)), dim3(64), 0, s, p);
    return hipGetLastError();
}

// ----------------------------------------------------------------- time segments
// The chunks of a segment (INT32_MAX: sequences are not cut), the segments' slots and their borders', and
// whether bf16's workgroups hold 128 value channels (eight waves) instead of 64.
struct Plan {
    int cps;
    int64_t segments, edges;
    bool wide, wide_ends;
};
// The cheapest of some ways to cut, by what a chunk takes a workgroup alone on its CU
// (us, at 128 and at 64 key channels): 64 value channels 2.75 and 1.95, 128 of them 5
// and 3.2; without the output 1.8 and 1.3, 4 and 2.5; fp32 11.5 and 5.4, 7.5 and
// 3.6; a step of the join 7.5 and 1.  Packed sequences count as equally long
// at first.
// Measured, us a call, bf16: 2 x 8192 steps of 40 heads of 128 x 128, 64 channels to a
// workgroup, 1 / 2 / 3 segments 511 / 629 / 626, 128 channels 588 / 574 / 495 to 590 (the clock
// gives way when every CU is at work for long); 65536 steps of 8 heads of 64 x 64,
// 1 / 8 / 16 / 32 / 64 segments 2002 / 565 / 367 / 334 / 369.  Short sequences, 4 heads of 64 x 64: 12 chunks
// in bf16 35 whole, 33 in four, 31 in six, 16 in fp32 120 whole, 75 in four, 61 in sixteen, their gradients 258, 167,
// 129; 128 x 128 in bf16, 12 chunks, 42 whole, 48 in two.  Under 12 chunks a sequence stays whole, so that its results
// are to the bit what they are between others: for bf16 the model would leave it so, in fp32 it costs
// 59 us instead of 46 at 6 chunks, 83 instead of 55 at 10.  The gradient's walk backwards is cut alike.
inline int64_t map_bytes(const DeltaShape &s) { return s.dk > 64 ? kMapBytes<128> : kMapBytes<64>; }
inline int64_t edge_bytes(const DeltaShape &s) { return s.dv * s.dk * 4 + map_bytes(s); }      // of a border and head
inline Plan plan_of(const DeltaShape &s, int bf16) {
    const bool big = s.dk > 64;
    const double c4 = bf16 ? (big ? 2.75 : 1.95) : (big ? 11.5 : 5.4), c8 = big ? 5.0 : 3.2;
    const double e4 = bf16 ? (big ? 1.8 : 1.3) : (big ? 7.5 : 3.6), e8 = big ? 4.0 : 2.5, step = big ? 7.5 : 1.0;
    const int64_t nc = s.nseq > 0 ? (s.slots + s.nseq - 1) / s.nseq : 0, units = s.heads * s.nseq;
    const int64_t t4 = (s.dv + 63) / 64, t8 = (s.dv + 127) / 128, k4 = big ? 2 : 1, k8 = 1;
    const bool may = bf16 && s.dv > 64;
    // what a launch holds: the walk over the segments, the pass over their ends
    auto fits = [&](int64_t edges) { return t4 * s.heads * (s.nseq + edges) <= kDeltaMaxGroups && (t4 + k4) * s.heads * edges <= kDeltaMaxGroups; };
    auto rounds = [](int64_t n) { return static_cast<double>((n + 255) / 256); };
    Plan best{0x7fffffff, s.nseq, 0, false, false};
    double least = -1.0;
    for (int64_t n : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128}) {
        if (n > 1 && (nc < 12 || n > nc)) break;
        const int64_t cps = (nc + n - 1) / n;
        const double out4 = rounds(t4 * units * n) * c4, out8 = rounds(t8 * units * n) * c8;
        const double ends4 = rounds(units * (t4 * (n - 1) + k4 * (n - 2))) * e4, ends8 = rounds(units * (t8 * (n - 1) + k8 * (n - 2))) * e8;
        Plan p{0x7fffffff, s.nseq, 0, may && out8 < out4, may && ends8 < ends4};
        double cost = cps * (p.wide ? out8 : out4);
        if (n > 1) {
            cost += cps * (p.wide_ends ? ends8 : ends4) + (n - 2) * step + 15.0;
            p.cps = static_cast<int>(cps);
            p.edges = s.packed ? s.slots / cps : s.nseq * ((nc + cps - 1) / cps - 1);
            p.segments = s.nseq + p.edges;
            if (!fits(p.edges)) break;
        }
        if (least < 0.0 || cost < least) {
            least = cost;
            best = p;
        }
    }
    // Packed sequences of which one may be much longer than the average would all wait for that one: those beyond the
    // average, beyond what keeps every CU at work and beyond 8 chunks are cut, if what the borders keep takes no more memory
    // than T and P.  9 sequences of 1 to 24 chunks, 12 heads of 96 x 80, fp32: 293 us a call whole, 238 cut at 9 chunks, 275 at 7.
    if (s.packed && best.segments == s.nseq && s.nseq > 0) {
        const int64_t longest = (s.seqlen + kC - 1) / kC, work = (s.slots * s.heads * (best.wide ? t8 : t4) + 255) / 256;
        int64_t cps = nc > work ? nc : work;
        cps = cps > 8 ? cps : 8;
        const int64_t edges = s.slots / cps, segments = s.nseq + edges;
        // the lengths are on the device; taken that the longest is half of all: its chunks beyond cps against the ends' pass
        // and the join.  What is wrong with that costs two launches and some workgroups that find nothing: 4 heads of 128 x 128
        // in bf16, 64 sequences of 64 steps 27 whole, 33 so planned, 8 of 512 38 and 41; with a 65th one of 3000 130 and 101
        // (fp32 567 and 241), one of 4000 with 20 of 16 144 and 103
        const double won = (longest / 2 - cps) * (best.wide ? c8 : c4), lost = cps * e4 + 15.0 + longest / (2 * cps) * step;
        if (won > lost && fits(edges) && edges * edge_bytes(s) <= s.slots * 2 * kTriBytes) {
            best.cps = static_cast<int>(cps);
            best.segments = segments;
            best.edges = edges;
        }
    }
    return best;
}
inline size_t ends_bytes(const DeltaShape &s, const Plan &p) {
    return align256(static_cast<size_t>(p.edges * s.heads * s.dv * s.dk) * 4);
}
inline size_t maps_bytes(const DeltaShape &s, const Plan &p) {
    return align256(static_cast<size_t>(p.edges * s.heads * map_bytes(s)));
}

}  // namespace
}  // namespace delta
}  // namespace ssm
