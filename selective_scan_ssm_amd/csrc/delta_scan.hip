// The gated delta rule: whole sequences (chunks of 64 steps on the matrix cores)
// and one decode token.  Per value head, with its state S (V x K, fp32):
//     S <- exp(g_t) S,  r = v_t - S k_t,  S <- S + beta_t r k_t^T,  y_t = scale S q_t
#include "delta_flow.h"

namespace ssm {
namespace delta {
namespace {

struct FwdWs {
    size_t t, p, scal, ends, maps, total;
};
FwdWs fwd_ws(const DeltaShape &s, const Plan &plan) {
    const size_t units = static_cast<size_t>(s.slots * s.heads);
    FwdWs w{};
    w.p = w.t + align256(units * kTriBytes);
    w.scal = w.p + align256(units * kTriBytes);
    w.ends = w.scal + align256(units * 3 * kC * 4);
    w.maps = w.ends + ends_bytes(s, plan);
    w.total = w.maps + maps_bytes(s, plan);
    return w;
}

template <typename T, int KP> hipError_t run(const DeltaArgs &a, hipStream_t s) {
    const Plan plan = plan_of(a.s, a.bf16);
    const FwdWs w = fwd_ws(a.s, plan);
    char *const base = static_cast<char *>(a.workspace);
    SeqParams p{};
    p.a = a;
    p.ws = {base + w.t, base + w.p, nullptr, reinterpret_cast<float *>(base + w.scal)};
    p.cps = plan.cps;
    p.wide = plan.wide;
    p.wide_ends = plan.wide_ends;
    p.segments = plan.segments;
    p.edges = plan.edges;
    p.ends = reinterpret_cast<float *>(base + w.ends);
    p.maps = base + w.maps;
    if (a.s.slots > 0) {
        if (hipError_t e = launch_prep<T, KP, false>(a, p.ws, s)) return e;
        if (hipError_t e = launch_segments<T, KP>(p, s)) return e;
    }
    return a.ckpt && a.s.slots > 0 ? launch_walk<T, KP, kTrain>(p, s) : launch_walk<T, KP, kOut>(p, s);
}

// ------------------------------------------------------------------- one token
// A row of the state (K values of one value channel) lies across L lanes, four
// values each, so a wave holds 64 / L rows at a time and M of them after one
// another.  The state is read once and written once; both of its products with a
// vector are taken of the values read:
//     a = S k, b = S q;  u = beta (v - alpha a);  y = scale (alpha b + u (k . q))
// HBM-bound: 5120 states of 128 x 128, 671 MB, 116 us (5.8 TB/s).
template <typename T, int L, int M> __global__ __launch_bounds__(kThreads) void delta_update_kernel(DeltaStepArgs a) {
    const int lane = threadIdx.x % 64, w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int sub = lane / L, l = lane % L;
    const int K = static_cast<int>(a.dk), V = static_cast<int>(a.dv);
    constexpr int kRows = 64 / L * M;                      // of a wave
    const int nvt = (V + kRows * kWaves - 1) / (kRows * kWaves);
    const int64_t bh = blockIdx.x / nvt, b = bh / a.heads, head = bh % a.heads, kh = head / (a.heads / a.kheads);
    const int v0 = (static_cast<int>(blockIdx.x % nvt) * kWaves + w) * kRows + sub * M;
    const bool in = 4 * l < K;
    float *const st = a.state + bh * V * K;
    const rsrc_t rs = make_rsrc(st, static_cast<uint32_t>(static_cast<int64_t>(V) * K * 4));
    f32x4 S[M];
#pragma unroll
    for (int m = 0; m < M; ++m) S[m] = load4(rs, in ? static_cast<uint32_t>(((v0 + m) * K + 4 * l) * 4) : kOffNone);
    f32x4 k = {0, 0, 0, 0}, q = {0, 0, 0, 0};
    const T *const pk = static_cast<const T *>(a.k) + (b * a.kheads + kh) * K, *const pq = static_cast<const T *>(a.q) + (b * a.kheads + kh) * K;
    if (in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            k[i] = to_f32(pk[4 * l + i]);
            q[i] = to_f32(pq[4 * l + i]);
        }
    }
    const float alpha = exp_accurate(step_log(a.g[bh])), beta = a.beta[bh];
    float kq = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) kq = fmaf(k[i], q[i], kq);
    kq = wave_fold<L>(kq, AddOp());
    const T *const pv = static_cast<const T *>(a.v) + bh * V;
    float y = 0.0f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const int v = v0 + m;
        float sk = 0.0f, sq = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sk = fmaf(S[m][i], k[i], sk);
            sq = fmaf(S[m][i], q[i], sq);
        }
        sk = wave_fold<L>(sk, AddOp());
        sq = wave_fold<L>(sq, AddOp());
        const float u = beta * fmaf(-alpha, sk, v < V ? to_f32(pv[v]) : 0.0f);
        const float out = a.scale * fmaf(alpha, sq, u * kq);
        if (l == m) y = out;
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = fmaf(alpha, S[m][i], u * k[i]);
        store4(o, rs, in ? static_cast<uint32_t>((v * K + 4 * l) * 4) : kOffNone);
    }
    static_assert(M <= L, "a lane per output");
    if (l < M && v0 + l < V) static_cast<T *>(a.y)[bh * V + v0 + l] = from_f32<T>(y);
}

template <typename T, int L, int M> hipError_t launch_update_of(const DeltaStepArgs &a, hipStream_t s) {
    constexpr int rows = 64 / L * M * kWaves;
    const int64_t grid = a.batch * a.heads * ((a.dv + rows - 1) / rows);
    hipLaunchKernelGGL((delta_update_kernel<T, L, M>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <typename T> hipError_t update(const DeltaStepArgs &a, hipStream_t s) {
    if (a.dk > 64) return launch_update_of<T, 32, 8>(a, s);
    if (a.dk > 32) return launch_update_of<T, 16, 4>(a, s);
    return launch_update_of<T, 8, 4>(a, s);
}

}  // namespace
}  // namespace delta

size_t delta_scan_workspace(const DeltaShape &s, int bf16) { return s.slots * s.heads > 0 ? delta::fwd_ws(s, delta::plan_of(s, bf16)).total : 0; }

hipError_t launch_delta_scan(const DeltaArgs &a, hipStream_t s) {
    using namespace delta;
    if (a.bf16) return a.s.dk > 64 ? run<bf16_t, 128>(a, s) : run<bf16_t, 64>(a, s);
    return a.s.dk > 64 ? run<float, 128>(a, s) : run<float, 64>(a, s);
}
hipError_t launch_delta_update(const DeltaStepArgs &a, hipStream_t s) {
    return a.bf16 ? delta::update<bf16_t>(a, s) : delta::update<float>(a, s);
}

}  // namespace ssm
