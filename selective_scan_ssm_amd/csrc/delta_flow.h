// The recurrence over the chunks in bf16 io: four (or eight) waves compute, one more loads.
//
// A chunk's keys, queries, values and shared operands are 50 to 73 KB, which take the
// memory pipe one to two thousand clocks; waves that also compute stood still for
// as long, since a wave's instructions issue in order.  The extra wave moves them
// from global memory into one of two LDS buffers directly (no registers, no LDS
// writes), a chunk ahead, and one barrier per chunk hands them over.
//
// 2 x 8192 steps of 40 heads of 128 x 128 (160 workgroups), the walk: the four waves loading
// for themselves 636 us a call, with the fifth wave 467; now 350 us of kernel, 2.75 us a
// chunk.  What bounds it: each wave reads the chunk's 91 KB of operands from LDS (four waves
// 2900 clocks of the CU's LDS) and issues 132 products (2100 clocks), in a chain from S to
// the next S that leaves little of them side by side.  32 columns to a wave, for half of the
// reads, 3.9 to 6 us a chunk: one wave to a SIMD has no one to cover its waits.
#pragma once

#include "delta_chunk.h"

namespace ssm {
namespace delta {
namespace {

template <int NW> constexpr int kFlowThreads = 64 * (NW + 1);

// One LDS buffer: rows of keys and queries and columns of values as 1 KB operands.
// In an operand lane (g, c) finds its 16 bytes at 256 g + 16 (c ^ 4 g): the
// transposing read of a 4 x 16 block then touches 16 different places, and a plain
// one is a permutation of each 256 bytes.
template <int KP, int NW> struct FlowBuf {
    static constexpr int KK = KP / 32, KT = KP / 16;
    static constexpr int rows = 4 * KK * 1024, kv = NW / 2, values = 4 * kv * 1024;
    static constexpr int q = rows, t = 2 * rows, p = t + kTriBytes, v = p + kTriBytes, s = v + values, bytes = s + 3 * kC * 4;
};
__device__ __forceinline__ int flow_at(int lane) { return lane / 16 * 256 + ((lane % 16) ^ (lane / 16 * 4)) * 16; }
__device__ __forceinline__ Op<bf16_t> flow_row(const char *p, int at) { return {*reinterpret_cast<const u32x4 *>(p + at)}; }
// where a lane's part of a transposing read lies: row l / 4 of four, piece l % 4 (of channels), lane groups four rows apart
__device__ __forceinline__ u32x2 flow_tr(const char *p) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    using lds = __attribute__((address_space(3))) s16x4 *;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds)(const_cast<char *>(p))));
}
__device__ __forceinline__ int flow_tr_at(int lane) {
    const int l = lane % 16, piece = l % 4;
    return piece * 256 + ((4 * (lane / 16) + l / 4) ^ (4 * piece)) * 16;
}
// channels of tile kt as rows, steps 32 kk + 8 g ... along K
template <int KP> __device__ __forceinline__ Op<bf16_t> flow_col(const char *rows, int at, int kt, int kk) {
    const char *const p = rows + at + (2 * kk * (KP / 32) + kt / 2) * 1024 + kt % 2 * 8;
    const u32x2 a = flow_tr(p), b = flow_tr(p + KP / 32 * 1024);
    return {u32x4{a[0], a[1], b[0], b[1]}};
}
// value channels of column tile ct, steps 32 q ... along K
template <int KV> __device__ __forceinline__ Op<bf16_t> flow_value(const char *v, int lane, int q, int ct) {
    const int l = lane % 16, piece = l % 4, grp = 2 * (ct % 2) + piece / 2;
    const char *const p = v + (2 * q * KV + ct / 2) * 1024 + grp * 256 + ((4 * (lane / 16) + l / 4) ^ (4 * grp)) * 16 + piece % 2 * 8;
    const u32x2 a = flow_tr(p), b = flow_tr(p + KV * 1024);
    return {u32x4{a[0], a[1], b[0], b[1]}};
}

// every LDS read before the barrier has its data, whatever of global memory is under way
__device__ __forceinline__ void flow_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }
__device__ __forceinline__ void flow_loaded() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// The loading wave's part.
template <int KP, int NW> struct FlowLoader {
    using B = FlowBuf<KP, NW>;
    using lds = __attribute__((address_space(3))) void *;
    static constexpr int KK = B::KK;
    int lane, r;                                   // r: the step that lane's 16 bytes belong to, in tile 0
    int g;
    uint32_t k[KK], q[KK], v[B::kv];              // offsets in tile 0
    int ldk, ldq, ldv;                             // bytes
    __device__ __forceinline__ FlowLoader(int64_t lk, int64_t lq, int64_t lv, int K, int V)
        : lane(threadIdx.x % 64), ldk(static_cast<int>(lk) * 2), ldq(static_cast<int>(lq) * 2), ldv(static_cast<int>(lv) * 2) {
        g = lane / 16;
        r = row_index(0, (lane % 16) ^ (4 * g));
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            const int ch = 32 * kk + 8 * g;
            k[kk] = ch < K ? static_cast<uint32_t>(r * ldk + ch * 2) : kOffNone;
            q[kk] = ch < K ? static_cast<uint32_t>(r * ldq + ch * 2) : kOffNone;
        }
#pragma unroll
        for (int kk = 0; kk < B::kv; ++kk) {
            const int ch = 32 * kk + 8 * g;
            v[kk] = ch < V ? static_cast<uint32_t>(r * ldv + ch * 2) : kOffNone;
        }
    }
    template <int N> __device__ __forceinline__ void rows(char *dst, rsrc_t src, const uint32_t *off, int ld) const {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb)
#pragma unroll
            for (int kk = 0; kk < N; ++kk)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(src, (lds)(dst + (tb * N + kk) * 1024), 16,
                                                         off[kk] + static_cast<uint32_t>(row_index(tb, 0) * ld), 0, 0, 0);
    }
    template <int BYTES> __device__ __forceinline__ void copy(char *dst, const void *src) const {
        const rsrc_t s = make_rsrc(src, BYTES);
#pragma unroll
        for (int i = 0; i < BYTES / 1024; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s, (lds)(dst + i * 1024), 16, i * 1024 + lane * 16, 0, 0, 0);
    }
    __device__ __forceinline__ void scalars(char *dst, const float *src) const {
        const rsrc_t s = make_rsrc(src, 3 * kC * 4);
#pragma unroll
        for (int i = 0; i < 3; ++i) __builtin_amdgcn_raw_ptr_buffer_load_lds(s, (lds)(dst + i * 256), 4, i * 256 + lane * 4, 0, 0, 0);
    }
};

template <int KP, Mode MODE, int NW>
__global__ __launch_bounds__(kFlowThreads<NW>) __attribute__((amdgpu_waves_per_eu(NW == 8 ? 3 : 2, NW == 8 ? 3 : 2))) void delta_flow_kernel(SeqParams p) {
    using T = bf16_t;
    using B = FlowBuf<KP, NW>;
    constexpr int KT = KP / 16, KK = KP / 32;
    constexpr bool OUT = has_out(MODE), SAVE = has_save(MODE);
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const DeltaArgs &a = p.a;
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 16, c = lane % 16;
    const int K = static_cast<int>(a.s.dk), V = static_cast<int>(a.s.dv);
    const int64_t H = a.s.heads;
    constexpr int kWide = 16 * NW;
    const int nvt = (V + kWide - 1) / kWide, tiles_n = MODE == kEnds ? nvt + (KP + kWide - 1) / kWide : nvt;
    // a segment's tiles lie a whole number of segments apart: on the same XCD where that is a multiple of eight
    const int64_t per_tile = gridDim.x / tiles_n;
    const int tile = static_cast<int>(blockIdx.x / per_tile);
    const int64_t rest = blockIdx.x % per_tile, head = rest % H, kh = head / (H / a.s.kheads), id = rest / H;
    Span sp;
    const Segment sg = segment_of<MODE == kEnds ? kBeforeEdges : kAllSegments>(a.s, id, p.edges, p.cps, sp);
    if (!sg.used) return;
    const int64_t seq = sg.seq;
    const bool first = sg.s == 0, last = sg.last, transition = MODE == kEnds && tile >= nvt;
    if (MODE == kEnds && first && transition) return;
    const int vt = transition ? 0 : tile;
    const int64_t row0 = sp.row0 + static_cast<int64_t>(sg.j0) * kC, unit0 = (sp.slot0 + sg.j0) * H + head;
    const int nch = sg.j1 - sg.j0;

    if (w == NW) {                                     // the loading wave
        const FlowLoader<KP, NW> ld(a.ldk, a.ldq, a.ldv, K, V - vt * kWide);
        const T *pk = static_cast<const T *>(a.k) + row0 * a.ldk + kh * K, *pq = static_cast<const T *>(a.q) + row0 * a.ldq + kh * K;
        const T *pv = static_cast<const T *>(a.v) + row0 * a.ldv + head * V + vt * kWide;
        const char *pt = p.ws.t + unit0 * kTriBytes, *pp = p.ws.p + unit0 * kTriBytes;
        const float *ps = p.ws.scal + unit0 * 3 * kC;
        int left = sp.len - sg.j0 * kC;
        for (int j = 0; j < nch; ++j) {
            char *const buf = smem + j % 2 * B::bytes;
            const int n = left < kC ? left : kC;
            ld.template rows<KK>(buf, chunk_rsrc(pk, n, a.ldk, K, 2), ld.k, ld.ldk);
            ld.template copy<kTriBytes>(buf + B::t, pt);
            ld.scalars(buf + B::s, ps);
            ld.template rows<B::kv>(buf + B::v, chunk_rsrc(pv, transition ? 0 : n, a.ldv, V - vt * kWide, 2), ld.v, ld.ldv);
            if constexpr (OUT) {
                ld.template rows<KK>(buf + B::q, chunk_rsrc(pq, n, a.ldq, K, 2), ld.q, ld.ldq);
                ld.template copy<kTriBytes>(buf + B::p, pp);
            }
            left -= kC;
            pk += kC * a.ldk;
            pq += kC * a.ldq;
            pv += kC * a.ldv;
            pt += H * kTriBytes;
            pp += H * kTriBytes;
            ps += H * 3 * kC;
            flow_loaded();
            flow_barrier();                                // chunk j is there, and everyone is done with chunk j - 1
        }
        if (transition) {
            flow_barrier();
            flow_barrier();
        }
        return;
    }

    const int v0 = vt * kWide + w * 16;                    // the wave's first channel
    const f32x4 zero = {0, 0, 0, 0};
    const size_t VK = static_cast<size_t>(V) * K;
    const int at = flow_at(lane), tat = flow_tr_at(lane);
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
    int64_t unit = unit0;
    const int ldy = static_cast<int>(H) * V;
    T *py = static_cast<T *>(a.y) + (row0 * H + head) * V;
    int left = sp.len - sg.j0 * kC;
    for (int j = 0; j < nch; ++j, unit += H, left -= kC, py += static_cast<int64_t>(kC) * ldy) {
        const char *const buf = smem + j % 2 * B::bytes;
        const float *const sS = reinterpret_cast<const float *>(buf + B::s);
        flow_barrier();
        if constexpr (SAVE) store_state<KP>(S, a.ckpt + unit * (VK + kC * V), v0, V, K, lane);
        // With a wave to a SIMD the reads of LDS are issued a product ahead of their use, and held there by `fence`: left
        // to itself the compiler reads each operand where it is used and waits for it.  Eight waves cover one another's
        // waits, and have not the registers.
        constexpr bool AHEAD = NW == 4;
        auto fence = [] {
            if constexpr (AHEAD) __builtin_amdgcn_sched_barrier(0);
        };
        f32x4 ks[4], y[4];                                 // y transposed: rows are channels, columns steps
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            ks[tb] = zero;
            if constexpr (OUT) y[tb] = zero;
        }
        Op<T> fk[2][4], fq[2][4], fv[2];
        Op2<T> ft[AHEAD ? 6 : 1], so[2];
        f32x4 e[4];
        auto t_op = [&](int f) {
            if constexpr (AHEAD) return ft[f];
            else return get_op2(buf + B::t + f * kOp2Bytes, lane, T());
        };
        auto read_rows = [&](int kk) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                fk[kk % 2][tb] = flow_row(buf + (tb * KK + kk) * 1024, at);
                if constexpr (OUT) fq[kk % 2][tb] = flow_row(buf + B::q + (tb * KK + kk) * 1024, at);
            }
        };
        if constexpr (AHEAD) read_rows(0);
        fence();
        so[0] = computed<T>(S[0], S[1]);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            if constexpr (!AHEAD) read_rows(kk);
            if (kk + 1 < KK) {
                if constexpr (AHEAD) read_rows(kk + 1);
            } else {
#pragma unroll
                for (int f = 0; f < (AHEAD ? 6 : 0); ++f) ft[f] = get_op2(buf + B::t + f * kOp2Bytes, lane, T());
#pragma unroll
                for (int q = 0; q < 2; ++q) fv[q] = flow_value<B::kv>(buf + B::v, lane, q, w);
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) e[tb] = *reinterpret_cast<const f32x4 *>(&sS[32 * (tb / 2) + 8 * g + 4 * (tb % 2)]);
            }
            fence();
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) ks[tb] = mma(fk[kk % 2][tb], so[kk % 2], ks[tb]);
            if constexpr (OUT) {
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) y[tb] = mma(so[kk % 2], fq[kk % 2][tb], y[tb]);
            }
            if (kk + 1 < KK) so[(kk + 1) % 2] = computed<T>(S[2 * kk + 2], S[2 * kk + 3]);
            fence();
        }
        Op2<T> fp[OUT && AHEAD ? 6 : 1], xo[2];
        float ey[OUT ? 4 : 1];
        f32x4 eb[4], ew[4];
        const float end = sS[kC - 1];
        if constexpr (OUT) {
#pragma unroll
            for (int f = 0; f < (AHEAD ? 6 : 0); ++f) fp[f] = get_op2(buf + B::p + f * kOp2Bytes, lane, T());
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) ey[tb] = sS[row_index(tb, c)];
        }
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            const int t = 32 * (tb / 2) + 8 * g + 4 * (tb % 2);
            eb[tb] = *reinterpret_cast<const f32x4 *>(&sS[2 * kC + t]);
            ew[tb] = *reinterpret_cast<const f32x4 *>(&sS[kC + t]);
        }
        fence();
#pragma unroll
        for (int q = 0; q < 2; ++q) {                      // 32 steps
            f32x4 x0, x1;
            tiles(fv[q], x0, x1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x0[i] = fmaf(-e[2 * q][i], ks[2 * q][i], x0[i]);
                x1[i] = fmaf(-e[2 * q + 1][i], ks[2 * q + 1][i], x1[i]);
            }
            xo[q] = computed<T>(x0, x1);
        }
        f32x4 R[4];
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) R[tb] = zero;
        if constexpr (SAVE) {                              // R, transposed, for stores of four channels
            const rsrc_t rr = make_rsrc(a.ckpt + unit * (VK + kC * V) + VK, static_cast<uint32_t>(kC * V * 4));
            f32x4 rt[4] = {zero, zero, zero, zero};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb) rt[tb] = mma(xo[kk], t_op(tri_low(tb, kk)), rt[tb]);
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) stream4(rt[tb], rr, v < V ? static_cast<uint32_t>((row_index(tb, c) * V + v) * 4) : kOffNone);
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
            for (int tb = 2 * kk; tb < 4; ++tb) {
                const Op2<T> f = t_op(tri_low(tb, kk));
                R[tb] = mma(f, xo[kk], R[tb]);
            }
        if constexpr (OUT) {
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) y[tb] = y[tb] * ey[tb];
        }
        fence();
        Op<T> fc[KT];                                      // the first 32 steps' columns
#pragma unroll
        for (int kt = 0; kt < (AHEAD ? KT : 0); ++kt) fc[kt] = flow_col<KP>(buf, tat, kt, 0);
        fence();
        Op2<T> uo[2], wo[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const f32x4 u0 = R[2 * q] * eb[2 * q], u1 = R[2 * q + 1] * eb[2 * q + 1];
            if constexpr (OUT) uo[q] = computed<T>(u0, u1);
            wo[q] = computed<T>(u0 * ew[2 * q], u1 * ew[2 * q + 1]);
        }
        if constexpr (OUT) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int tb = 2 * kk; tb < 4; ++tb) {
                    Op2<T> f;
                    if constexpr (AHEAD) f = fp[tri_low(tb, kk)];
                    else f = get_op2(buf + B::p + tri_low(tb, kk) * kOp2Bytes, lane, T());
                    y[tb] = mma(uo[kk], f, y[tb]);
                }
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = S[kt] * end;
        fence();
        Op<T> fd[KT];
#pragma unroll
        for (int kt = 0; kt < (AHEAD ? KT : 0); ++kt) fd[kt] = flow_col<KP>(buf, tat, kt, 1);
        fence();
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if constexpr (!AHEAD) fc[kt] = flow_col<KP>(buf, tat, kt, 0);
            S[kt] = mma(fc[kt], wo[0], S[kt]);
        }
        if constexpr (OUT) {
            const rsrc_t ry = chunk_rsrc(py, left < kC ? left : kC, ldy, V, 2);
            const int v = v0 + 4 * g;
#pragma unroll
            for (int tb = 0; tb < 4; ++tb)
                store_io4(y[tb] * a.scale, ry, v < V ? static_cast<uint32_t>((row_index(tb, c) * ldy + v) * 2) : kOffNone, T());
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
            if constexpr (!AHEAD) fd[kt] = flow_col<KP>(buf, tat, kt, 1);
            S[kt] = mma(fd[kt], wo[1], S[kt]);
        }
    }
    if constexpr (MODE == kEnds) {
        if (!transition) {
            store_state<KP>(S, p.ends + ((sg.edge + 1) * H + head) * VK, v0, V, K, lane);
            return;
        }
        store_map<T, KP, NW>(S, smem, w, lane, p.maps + ((sg.edge + 1) * H + head) * kMapBytes<KP>, (tile - nvt) * kWide);
    } else if (last && a.last_state) {
        store_state<KP>(S, a.last_state + (seq * H + head) * VK, v0, V, K, lane);
    }
}

template <int KP, Mode MODE, int NW> hipError_t launch_flow(const SeqParams &p, hipStream_t s) {
    constexpr int wide = 16 * NW;
    const int64_t nvt = (p.a.s.dv + wide - 1) / wide;
    const int64_t grid = (MODE == kEnds ? (nvt + (KP + wide - 1) / wide) * p.edges : nvt * p.segments) * p.a.s.heads;
    constexpr size_t lds = 2 * FlowBuf<KP, NW>::bytes;
    hipLaunchKernelGGL((delta_flow_kernel<KP, MODE, NW>), dim3(static_cast<unsigned>(grid)), dim3(kFlowThreads<NW>), lds, s, p);
    return hipGetLastError();
}

// A walk over all chunks: bf16 with a loading wave, fp32 without.
template <typename T, int KP, Mode MODE> hipError_t launch_walk(const SeqParams &p, hipStream_t s) {
    if constexpr (sizeof(T) == 4) return launch_seq<KP, MODE>(p, s);
    else return (MODE == kEnds ? p.wide_ends : p.wide) ? launch_flow<KP, MODE, 8>(p, s) : launch_flow<KP, MODE, 4>(p, s);
}
// the states that the segments are entered with, where there is more than one
template <typename T, int KP> hipError_t launch_segments(const SeqParams &p, hipStream_t s) {
    if (p.segments == p.a.s.nseq) return hipSuccess;
    if (hipError_t e = launch_walk<T, KP, kEnds>(p, s)) return e;
    return launch_carry<T, KP, false>(p, s);
}

}  // namespace
}  // namespace delta
}  // namespace ssm
