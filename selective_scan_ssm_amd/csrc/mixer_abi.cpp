// C ABI of the gated delta rule and of the channels-last group norm (declared in
// include/ssm_scan.h).  As in ssm_abi.cpp, arguments are validated before the HIP
// runtime is touched.
#include "ssm_scan.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "ssm_abi_check.h"
#include "ssm_kernels.h"

using namespace ssm::abi;

namespace {

constexpr int64_t kMaxSpan = (int64_t(1) << 31) - 1;   // 32-bit buffer offsets
constexpr int64_t kMaxLanes = (int64_t(1) << 32) - 1;  // a launch counts its lanes in 32 bits
constexpr size_t kBad = static_cast<size_t>(-1);

// elements a strided (rows, dim) view spans
int64_t span(int64_t rows, int64_t ld, int64_t dim) { return rows > 0 ? (rows - 1) * ld + dim : 0; }

// outs against ins and against one another
template <int NO, int NI> int check_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (const Range &r : ins)
            if (overlap(outs[i], r)) return SSM_ERR_ALIAS;
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return SSM_ERR_ALIAS;
    }
    return SSM_OK;
}
int check_workspace(size_t need, const void *ws, size_t bytes) {
    if (need && (!ws || bytes < need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(ws, 256)) return SSM_ERR_ALIGN;
    return SSM_OK;
}
template <int N> bool all_aligned(const void *const (&p)[N], size_t a) {
    for (const void *q : p)
        if (!aligned(q, a)) return false;
    return true;
}

// ------------------------------------------------------------- gated delta rule
int check_heads(int64_t kheads, int64_t heads, int64_t dk, int64_t dv, int io) {
    if (int r = check_dtype(io)) return r;
    if (kheads < 1 || heads < 1 || heads % kheads != 0) return SSM_ERR_SHAPE;
    if (dk < 8 || dk > ssm::kDeltaMaxState || dk % 8 != 0 || dv < 8 || dv % 8 != 0) return SSM_ERR_SHAPE;
    // a chunk of y and of the fp32 workspace, and a state, are addressed with 32-bit byte offsets
    if (mul3(heads, dv, 4 * ssm::kDeltaChunk) < 0 || mul3(heads, dv, 4 * ssm::kDeltaChunk) > kMaxSpan ||
        mul3(dv, dk, 4) > kMaxSpan || mul3(heads, dk, 4 * ssm::kDeltaChunk) > kMaxSpan || mul3(heads, dk, 4 * ssm::kDeltaChunk) < 0)
        return SSM_ERR_SHAPE;
    return SSM_OK;
}
// Fills `s`; packed: whether starts are given.
int check_delta(ssm::DeltaShape &s, int64_t batch, int64_t seqlen, bool packed, int64_t nseq, int64_t kheads, int64_t heads,
                int64_t dk, int64_t dv, int io) {
    if (int r = check_heads(kheads, heads, dk, dv, io)) return r;
    if (batch < 0 || seqlen < 0 || seqlen > kMaxSpan || (packed && (batch != 1 || nseq < 0))) return SSM_ERR_SHAPE;
    s.packed = packed ? 1 : 0;
    s.nseq = packed ? nseq : batch;
    s.seqlen = seqlen;
    s.kheads = kheads; s.heads = heads; s.dk = dk; s.dv = dv;
    const int64_t C = ssm::kDeltaChunk;
    if (s.nseq > kMaxSpan) return SSM_ERR_SHAPE;
    if (packed) s.slots = nseq > 0 ? seqlen / C + nseq : 0;
    else s.slots = batch * ((seqlen + C - 1) / C);
    if (seqlen == 0) s.slots = 0;
    const int64_t tiles = (dv + 63) / 64;
    const int64_t slots = s.slots > s.nseq ? s.slots : s.nseq;
    // workgroups per chunk (sequence), head and 64 channels
    const int64_t groups = mul3(slots, heads, tiles);
    if (groups < 0 || groups > ssm::kDeltaMaxGroups) return SSM_ERR_SHAPE;
    if (mul3(groups, 64 * 64, 8) < 0 || mul3(mul3(slots, heads, dv), dk + C, 8) < 0 || mul3(batch * seqlen, heads, (dk > dv ? dk : dv) * 4) < 0)
        return SSM_ERR_SHAPE;
    return SSM_OK;
}

struct DeltaIn {
    int64_t rows;                         // batch * seqlen
    size_t es;
    int64_t ends;                         // elements of a state tensor
    Range q, k, v, g, beta, h0, starts;
};
int check_delta_inputs(ssm::DeltaArgs &a, DeltaIn &in, int64_t batch, int64_t seqlen, int io) {
    const ssm::DeltaShape &s = a.s;
    in.es = io_size(io);
    in.rows = batch * seqlen;
    in.ends = s.nseq * s.heads * s.dv * s.dk;
    const int64_t per = 16 / static_cast<int64_t>(in.es);
    const int64_t width[3] = {s.kheads * s.dk, s.kheads * s.dk, s.heads * s.dv};
    int64_t *const ld[3] = {&a.ldq, &a.ldk, &a.ldv};
    for (int i = 0; i < 3; ++i) {
        if (in.rows <= 1) {               // a single step has no row stride to speak of
            *ld[i] = width[i];
            continue;
        }
        if (*ld[i] < width[i] || *ld[i] % per != 0) return SSM_ERR_SHAPE;
        const int64_t c = mul3(ssm::kDeltaChunk, *ld[i], static_cast<int64_t>(in.es));
        if (c < 0 || c > kMaxSpan || mul3(in.rows, *ld[i], static_cast<int64_t>(in.es)) < 0) return SSM_ERR_SHAPE;
    }
    if (!std::isfinite(a.scale)) return SSM_ERR_VALUE;
    if (in.rows > 0 && (!a.q || !a.k || !a.v || !a.g || !a.beta)) return SSM_ERR_NULL;
    const void *wide[] = {a.q, a.k, a.v, a.h0, a.ckpt};
    const void *words[] = {a.g, a.beta, s.starts};
    if (!all_aligned(wide, 16) || !all_aligned(words, 4)) return SSM_ERR_ALIGN;
    in.q = range(a.q, span(in.rows, a.ldq, width[0]), in.es);
    in.k = range(a.k, span(in.rows, a.ldk, width[1]), in.es);
    in.v = range(a.v, span(in.rows, a.ldv, width[2]), in.es);
    in.g = range(a.g, in.rows * s.heads, 4);
    in.beta = range(a.beta, in.rows * s.heads, 4);
    in.h0 = range(a.h0, in.ends, 4);
    in.starts = range(s.starts, s.starts ? s.nseq + 1 : 0, 4);
    return SSM_OK;
}

// ------------------------------------------------------------------- group norm
int check_group(int64_t batch, int64_t rows, int64_t dim, int64_t groups, int io) {
    if (int r = check_dtype(io)) return r;
    if (batch < 0 || rows < 0 || dim < 1 || dim > SSM_MAX_GROUP_DIM || groups < 1 || dim % groups != 0) return SSM_ERR_SHAPE;
    if (mul3(batch, rows, dim * 8) < 0 || mul3(batch, groups, 64) < 0) return SSM_ERR_SHAPE;
    return SSM_OK;
}
int check_group_ld(int64_t n, int64_t ld, int64_t dim) { return n > 1 && (ld < dim || mul3(n, ld, 4) < 0) ? SSM_ERR_SHAPE : SSM_OK; }

}  // namespace

extern "C" {

size_t ssm_delta_ckpt_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nseq, int64_t nheads, int64_t dstate,
                            int64_t headdim) {
    ssm::DeltaShape s{};
    if (check_delta(s, batch, seqlen, packed != 0, nseq, nheads, nheads, dstate, headdim, SSM_F32)) return kBad;
    return static_cast<size_t>(s.slots * s.heads) * static_cast<size_t>(ssm::delta_ckpt_stride(dstate, headdim)) * 4;
}

size_t ssm_delta_scan_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nseq, int64_t nkheads, int64_t nheads,
                                      int64_t dstate, int64_t headdim, int io_dtype) {
    ssm::DeltaShape s{};
    if (check_delta(s, batch, seqlen, packed != 0, nseq, nkheads, nheads, dstate, headdim, io_dtype)) return kBad;
    return ssm::delta_scan_workspace(s, io_dtype == SSM_BF16);
}

int ssm_delta_scan_fwd(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const float *g,
                       const float *beta, float scale, const float *h0, const int32_t *starts, int64_t nseq, void *y,
                       float *last_state, float *ckpt, int64_t batch, int64_t seqlen, int64_t nkheads, int64_t nheads,
                       int64_t dstate, int64_t headdim, int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    ssm::DeltaArgs a{};
    a.s.starts = starts;
    if (int r = check_delta(a.s, batch, seqlen, starts != nullptr, nseq, nkheads, nheads, dstate, headdim, io_dtype)) return r;
    if (a.s.nseq == 0) return SSM_OK;
    a.q = q; a.k = k; a.v = v; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.g = g; a.beta = beta; a.h0 = h0; a.scale = scale; a.ckpt = ckpt;
    a.bf16 = io_dtype == SSM_BF16;
    DeltaIn in;
    if (int r = check_delta_inputs(a, in, batch, seqlen, io_dtype)) return r;
    if (in.rows > 0 && !y) return SSM_ERR_NULL;
    const void *wide[] = {y, last_state};
    if (!all_aligned(wide, 16)) return SSM_ERR_ALIGN;
    const size_t need = ssm::delta_scan_workspace(a.s, a.bf16);
    const Range ins[] = {in.q, in.k, in.v, in.g, in.beta, in.h0, in.starts};
    const Range outs[] = {range(y, in.rows * nheads * headdim, in.es), range(last_state, in.ends, 4),
                          range(ckpt, a.s.slots * nheads * ssm::delta_ckpt_stride(dstate, headdim), 4),
                          range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    a.y = y; a.last_state = last_state; a.workspace = workspace;
    return hip_status(ssm::launch_delta_scan(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_delta_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int packed, int64_t nseq, int64_t nkheads, int64_t nheads,
                                          int64_t dstate, int64_t headdim, int saved, int io_dtype) {
    ssm::DeltaShape s{};
    if (check_delta(s, batch, seqlen, packed != 0, nseq, nkheads, nheads, dstate, headdim, io_dtype)) return kBad;
    return ssm::delta_scan_bwd_workspace(s, io_dtype == SSM_BF16, saved != 0);
}

int ssm_delta_scan_bwd(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const float *g,
                       const float *beta, float scale, const float *h0, const int32_t *starts, int64_t nseq, const void *dout,
                       const float *dlast, const float *ckpt, void *dq, void *dk, void *dv, float *dg, float *dbeta, float *dh0,
                       int64_t batch, int64_t seqlen, int64_t nkheads, int64_t nheads, int64_t dstate, int64_t headdim,
                       int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    ssm::DeltaBwdArgs b{};
    ssm::DeltaArgs &a = b.fwd;
    a.s.starts = starts;
    if (int r = check_delta(a.s, batch, seqlen, starts != nullptr, nseq, nkheads, nheads, dstate, headdim, io_dtype)) return r;
    if (a.s.nseq == 0) return SSM_OK;
    a.q = q; a.k = k; a.v = v; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
    a.g = g; a.beta = beta; a.h0 = h0; a.scale = scale; a.ckpt = const_cast<float *>(ckpt);
    a.bf16 = io_dtype == SSM_BF16;
    DeltaIn in;
    if (int r = check_delta_inputs(a, in, batch, seqlen, io_dtype)) return r;
    if (in.rows > 0 && (!dout || !dq || !dk || !dv || !dg || !dbeta)) return SSM_ERR_NULL;
    const void *wide[] = {dout, dlast, dq, dk, dv, dh0};
    const void *words[] = {dg, dbeta};
    if (!all_aligned(wide, 16) || !all_aligned(words, 4)) return SSM_ERR_ALIGN;
    const size_t need = ssm::delta_scan_bwd_workspace(a.s, a.bf16, ckpt != nullptr);
    const int64_t nk = in.rows * nkheads * dstate, nv = in.rows * nheads * headdim, nh = in.rows * nheads;
    const Range ins[] = {in.q, in.k, in.v, in.g, in.beta, in.h0, in.starts, range(dout, nv, in.es), range(dlast, in.ends, 4),
                         range(ckpt, a.s.slots * nheads * ssm::delta_ckpt_stride(dstate, headdim), 4)};
    const Range outs[] = {range(dq, nk, in.es), range(dk, nk, in.es), range(dv, nv, in.es), range(dg, nh, 4), range(dbeta, nh, 4),
                          range(dh0, in.ends, 4), range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    a.workspace = workspace;
    b.dout = dout; b.dlast = dlast;
    b.dq = dq; b.dk = dk; b.dv = dv; b.dg = dg; b.dbeta = dbeta; b.dh0 = dh0;
    return hip_status(ssm::launch_delta_scan_bwd(b, static_cast<hipStream_t>(stream)));
}

int ssm_delta_state_update(float *state, const void *q, const void *k, const void *v, const float *g, const float *beta, float scale,
                           void *y, int64_t batch, int64_t nkheads, int64_t nheads, int64_t dstate, int64_t headdim, int io_dtype,
                           void *stream) {
    if (int r = check_heads(nkheads, nheads, dstate, headdim, io_dtype)) return r;
    // workgroups of 256 lanes take 32 rows of a state at least
    const int64_t groups = mul3(batch, nheads, (headdim + 31) / 32);
    if (groups < 0 || groups > kMaxLanes / 256 || mul3(batch * nheads, headdim, dstate * 4) < 0) return SSM_ERR_SHAPE;
    if (!std::isfinite(scale)) return SSM_ERR_VALUE;
    if (batch == 0) return SSM_OK;
    if (!state || !q || !k || !v || !g || !beta || !y) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    const void *wide[] = {state, q, k, v, y}, *words[] = {g, beta};
    if (!all_aligned(wide, 16) || !all_aligned(words, 4)) return SSM_ERR_ALIGN;
    const int64_t nk = batch * nkheads * dstate, nv = batch * nheads * headdim, nh = batch * nheads;
    const Range ins[] = {range(q, nk, es), range(k, nk, es), range(v, nv, es), range(g, nh, 4), range(beta, nh, 4)};
    const Range outs[] = {range(state, nv * dstate, 4), range(y, nv, es)};
    if (int r = check_overlap(outs, ins)) return r;
    ssm::DeltaStepArgs a{};
    a.state = state; a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.y = y;
    a.batch = batch; a.kheads = nkheads; a.heads = nheads; a.dk = dstate; a.dv = headdim;
    a.scale = scale; a.bf16 = io_dtype == SSM_BF16;
    return hip_status(ssm::launch_delta_update(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_group_norm_workspace_bytes(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    if (check_group(batch, rows, dim, groups, SSM_F32)) return kBad;
    return batch == 0 || rows == 0 ? 0 : ssm::group_norm_workspace(batch, rows, dim, groups);
}

int ssm_group_norm_fwd(const void *x, int64_t ldx, const void *z, int64_t ldz, const float *weight, const float *bias, void *y,
                       float *mean, float *rstd, int64_t batch, int64_t rows, int64_t dim, int64_t groups, float eps, int silu,
                       int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (int r = check_group(batch, rows, dim, groups, io_dtype)) return r;
    const int64_t n = batch * rows;
    if (check_group_ld(n, ldx, dim) || (z && check_group_ld(n, ldz, dim))) return SSM_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return SSM_ERR_VALUE;
    if (n == 0) return SSM_OK;
    if (!x || !y) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    const void *io_ptrs[] = {x, z, y}, *words[] = {weight, bias, mean, rstd};
    if (!all_aligned(io_ptrs, es) || !all_aligned(words, 4)) return SSM_ERR_ALIGN;
    ssm::GroupNormArgs a{};
    a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.ldx = n > 1 ? ldx : dim; a.ldz = n > 1 ? ldz : dim;
    a.batch = batch; a.rows = rows; a.dim = dim; a.groups = groups; a.eps = eps; a.silu = silu != 0;
    a.bf16 = io_dtype == SSM_BF16; a.workspace = workspace;
    const size_t need = ssm::group_norm_workspace(batch, rows, dim, groups);
    const Range ins[] = {range(x, span(n, a.ldx, dim), es), range(z, span(n, a.ldz, dim), es), range(weight, dim, 4), range(bias, dim, 4)};
    const Range outs[] = {range(y, n * dim, es), range(mean, batch * groups, 4), range(rstd, batch * groups, 4),
                          range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    return hip_status(ssm::launch_group_norm(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_group_norm_bwd_workspace_bytes(int64_t batch, int64_t rows, int64_t dim, int64_t groups) {
    if (check_group(batch, rows, dim, groups, SSM_F32)) return kBad;
    return batch == 0 || rows == 0 ? 0 : ssm::group_norm_bwd_workspace(batch, rows, dim, groups);
}

int ssm_group_norm_bwd(const void *dy, const void *x, int64_t ldx, const void *z, int64_t ldz, const float *weight, const float *bias,
                       const float *mean, const float *rstd, void *dx, void *dz, float *dweight, float *dbias, int64_t batch,
                       int64_t rows, int64_t dim, int64_t groups, int silu, int io_dtype, void *workspace, size_t workspace_bytes,
                       void *stream) {
    if (int r = check_group(batch, rows, dim, groups, io_dtype)) return r;
    const int64_t n = batch * rows;
    if (check_group_ld(n, ldx, dim) || (z && check_group_ld(n, ldz, dim))) return SSM_ERR_SHAPE;
    if (n > 0 && (!dy || !x || !mean || !rstd || !dx || (z && !dz))) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    const void *io_ptrs[] = {dy, x, z, dx, dz}, *words[] = {weight, bias, mean, rstd, dweight, dbias};
    if (!all_aligned(io_ptrs, es) || !all_aligned(words, 4)) return SSM_ERR_ALIGN;
    ssm::GroupNormBwdArgs b{};
    ssm::GroupNormArgs &a = b.fwd;
    a.x = x; a.z = z; a.weight = weight; a.bias = bias;
    a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
    a.ldx = n > 1 ? ldx : dim; a.ldz = n > 1 ? ldz : dim;
    a.batch = batch; a.rows = rows; a.dim = dim; a.groups = groups; a.silu = silu != 0;
    a.bf16 = io_dtype == SSM_BF16; a.workspace = workspace;
    b.dy = dy; b.dx = dx; b.dz = z ? dz : nullptr; b.dweight = dweight; b.dbias = dbias;
    const size_t need = n > 0 ? ssm::group_norm_bwd_workspace(batch, rows, dim, groups) : 0;
    const Range ins[] = {range(dy, n * dim, es), range(x, span(n, a.ldx, dim), es), range(z, span(n, a.ldz, dim), es), range(weight, dim, 4),
                         range(bias, dim, 4), range(mean, batch * groups, 4), range(rstd, batch * groups, 4)};
    const Range outs[] = {range(dx, n * dim, es), range(b.dz, n * dim, es), range(dweight, dim, 4), range(dbias, dim, 4),
                          range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    return hip_status(ssm::launch_group_norm_bwd(b, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
