// C ABI of the operators around and beside the scan: the gated linear
// recurrence, the RMS norm with residual, gradient clipping (declared in
// include/ssm_scan.h).  As in ssm_abi.cpp, arguments are validated before the
// HIP runtime is touched.
#include "ssm_scan.h"
#include "ssm_scan_testing.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "ssm_abi_check.h"
#include "ssm_kernels.h"

using namespace ssm::abi;

namespace {

constexpr int64_t kMaxSpan = (int64_t(1) << 31) - 1;   // 32-bit buffer offsets

bool bad_dtype2(int io, int res) { return check_dtype(io) || (res != SSM_F32 && res != io); }

// elements a strided (rows, dim) view spans
int64_t span(int64_t rows, int64_t ld, int64_t dim) { return rows > 0 ? (rows - 1) * ld + dim : 0; }

int check_gated_sizes(int64_t batch, int64_t seqlen, int64_t dim, int io) {
    if (int r = check_dtype(io)) return r;
    if (batch < 0 || seqlen < 0 || dim < 0 || batch > kMaxGridY) return SSM_ERR_SHAPE;
    if (mul3(batch, seqlen, dim) < 0 || mul3(batch, dim, 4) < 0) return SSM_ERR_SHAPE;
    // one block of steps is addressed with 32-bit byte offsets
    if (mul3(ssm::kGatedBlock, dim, 4) < 0 || mul3(ssm::kGatedBlock, dim, 4) > kMaxSpan) return SSM_ERR_SHAPE;
    // a launch counts its lanes in 32 bits: those of a tile's waves (no tile at all:
    // a copy of the states, 256 to a workgroup), which also keeps seqlen under 2^30
    const int64_t blocks = seqlen / ssm::kGatedBlock + (seqlen % ssm::kGatedBlock != 0);
    const int64_t lanes = seqlen == 0 ? 256 : 64 * ssm::gated_waves(seqlen);
    const int64_t tiles = mul3(batch, (dim + 63) / 64, blocks > 0 ? blocks : 1);
    if (tiles < 0 || tiles > (int64_t(1) << 32) / lanes - 1) return SSM_ERR_SHAPE;
    return SSM_OK;
}

// The inputs shared by the recurrence and its gradient.
int check_gated_inputs(const ssm::GatedArgs &a, int io) {
    const size_t es = io_size(io);
    const int64_t steps = a.batch * a.seqlen;
    const int64_t lds[] = {a.ldx, a.ldg, a.z ? a.ldz : a.dim};
    const int64_t block = a.seqlen < ssm::kGatedBlock ? a.seqlen : ssm::kGatedBlock;
    for (int64_t ld : lds) {
        if (steps > 1 && ld < a.dim) return SSM_ERR_SHAPE;
        if (steps > 1 && (mul3(block, ld, es) < 0 || mul3(block, ld, es) > kMaxSpan || mul3(steps, ld, es) < 0))
            return SSM_ERR_SHAPE;
    }
    if (steps > 0 && (!a.x || !a.g)) return SSM_ERR_NULL;
    const void *io_ptrs[] = {a.x, a.g, a.z};
    for (const void *p : io_ptrs)
        if (p && !aligned(p, es)) return SSM_ERR_ALIGN;
    const void *f_ptrs[] = {a.gate_bias, a.h0};
    for (const void *p : f_ptrs)
        if (p && !aligned(p, 4)) return SSM_ERR_ALIGN;
    return SSM_OK;
}

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

ssm::GatedArgs gated_args(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *bias, const void *z,
                          int64_t ldz, const float *h0, int64_t batch, int64_t seqlen, int64_t dim, int io, void *ws,
                          size_t ws_bytes) {
    ssm::GatedArgs a{};
    a.x = x; a.g = g; a.z = z;
    a.batch = batch; a.seqlen = seqlen; a.dim = dim;
    // a single step has no row stride to speak of
    const bool one = batch * seqlen <= 1;
    a.ldx = one ? dim : ldx; a.ldg = one ? dim : ldg; a.ldz = one ? dim : ldz;
    a.gate_bias = bias; a.h0 = h0;
    a.bf16 = io == SSM_BF16 ? 1 : 0;
    a.workspace = ws; a.workspace_bytes = ws_bytes;
    return a;
}

int check_workspace(size_t need, const void *ws, size_t bytes) {
    if (need && (!ws || bytes < need)) return SSM_ERR_WORKSPACE;
    if (need && !aligned(ws, 256)) return SSM_ERR_ALIGN;
    return SSM_OK;
}

int check_norm(const void *x, int64_t ldx, const void *residual, const float *weight, const void *y, size_t y_es,
               const float *scale, const void *residual_out, int64_t rows, int64_t dim, float eps, int io, int res) {
    if (bad_dtype2(io, res)) return SSM_ERR_DTYPE;
    if (rows < 0 || dim < 1 || dim > SSM_MAX_NORM_DIM) return SSM_ERR_SHAPE;
    if (rows > 1 && (ldx < dim || mul3(rows, ldx, 4) < 0)) return SSM_ERR_SHAPE;
    if (rows > kMaxSpan || mul3(rows, dim, 4) < 0) return SSM_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return SSM_ERR_VALUE;
    if (rows == 0) return SSM_OK;
    if (!x || !weight || !y) return SSM_ERR_NULL;
    const size_t es = io_size(io), rs = io_size(res);
    if (!aligned(x, es) || !aligned(y, y_es) || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(residual, rs) ||
        !aligned(residual_out, rs))
        return SSM_ERR_ALIGN;
    const Range ins[] = {range(x, span(rows, rows > 1 ? ldx : dim, dim), es), range(weight, dim, 4),
                         range(residual_out == residual ? nullptr : residual, rows * dim, rs)};
    const Range outs[] = {range(y, rows * dim, y_es), range(residual_out, rows * dim, rs), range(scale, rows, 4)};
    return check_overlap(outs, ins);
}

int norm_bwd(const void *dy, const void *r, int64_t ldr, const float *weight, const void *dresidual_out, void *dx,
             void *dresidual, float *dweight, int64_t rows, int64_t dim, float eps, int io_dtype, int residual_dtype,
             void *workspace, size_t workspace_bytes, void *stream) {
    if (bad_dtype2(io_dtype, residual_dtype)) return SSM_ERR_DTYPE;
    if (rows < 0 || rows > kMaxSpan || dim < 1 || dim > SSM_MAX_NORM_DIM || mul3(rows, dim, 4) < 0)
        return SSM_ERR_SHAPE;
    if (rows > 1 && (ldr < dim || mul3(rows, ldr, 4) < 0)) return SSM_ERR_SHAPE;
    if (!(eps >= 0.0f) || std::isinf(eps)) return SSM_ERR_VALUE;
    if (!dweight || (rows > 0 && (!dy || !r || !weight || !dx))) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype), rs = io_size(residual_dtype);
    if (!aligned(dy, es) || !aligned(dx, es) || !aligned(r, rs) || !aligned(dresidual_out, rs) ||
        !aligned(dresidual, rs) || !aligned(weight, 4) || !aligned(dweight, 4))
        return SSM_ERR_ALIGN;
    const int64_t n = rows * dim;
    const size_t need = ssm::norm_bwd_workspace(rows, dim);
    const Range ins[] = {range(dy, n, es), range(r, span(rows, rows > 1 ? ldr : dim, dim), rs), range(weight, dim, 4),
                         range(dresidual_out == dresidual ? nullptr : dresidual_out, n, rs)};
    const Range outs[] = {range(dx, n, es), range(dresidual, n, rs), range(dweight, dim, 4),
                          range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int rc = check_overlap(outs, ins)) return rc;
    if (int rc = check_workspace(need, workspace, workspace_bytes)) return rc;
    ssm::NormBwdArgs a{};
    a.dy = dy; a.r = r; a.dres_out = dresidual_out; a.weight = weight;
    a.dx = dx; a.dres = dresidual; a.dweight = dweight;
    a.rows = rows; a.dim = dim; a.ldr = rows > 1 ? ldr : dim; a.eps = eps;
    a.bf16 = io_dtype == SSM_BF16; a.res_bf16 = residual_dtype == SSM_BF16;
    a.workspace = workspace;
    return hip_status(ssm::launch_add_rms_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

// Checks a gradient list; an output may be its own input with the same dtype
// and otherwise overlaps nothing.
int check_list(const void *const *grads, void *const *outs, const int64_t *numel, const int *dtypes,
               const int *out_dtypes, int64_t count, bool scale, const float *norm, const void *ws, size_t ws_need) {
    if (count < 0 || count > (int64_t(1) << 20)) return SSM_ERR_SHAPE;
    if (!norm || (count > 0 && (!grads || !numel || !dtypes || (outs && !out_dtypes)))) return SSM_ERR_NULL;
    if (!aligned(norm, 4)) return SSM_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        if (check_dtype(dtypes[i]) || (outs && check_dtype(out_dtypes[i]))) return SSM_ERR_DTYPE;
        if (numel[i] < 0 || numel[i] >= (int64_t(1) << 40)) return SSM_ERR_SHAPE;
        if (numel[i] == 0) continue;
        if (!grads[i] || (outs && !outs[i])) return SSM_ERR_NULL;
        if (!aligned(grads[i], io_size(dtypes[i])) || (outs && !aligned(outs[i], io_size(out_dtypes[i]))))
            return SSM_ERR_ALIGN;
        if (outs && outs[i] == grads[i] && out_dtypes[i] != dtypes[i]) return SSM_ERR_ALIAS;
    }
    // every range once, sorted by its start: an output overlaps another range
    // if it overlaps one that starts before it and reaches furthest, or one that
    // starts inside it
    struct Item {
        uintptr_t lo, hi;
        bool out;
    };
    Item *items = new (std::nothrow) Item[static_cast<size_t>(2 * count + 2)];
    if (!items) return SSM_ERR_HOST;
    int64_t m = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (numel[i] == 0) continue;
        const bool in_place = scale && (!outs || outs[i] == grads[i]);
        const Range gi = range(grads[i], numel[i], io_size(dtypes[i]));
        items[m++] = {gi.lo, gi.hi, in_place};
        if (scale && !in_place) {
            const Range ro = range(outs[i], numel[i], io_size(out_dtypes[i]));
            items[m++] = {ro.lo, ro.hi, true};
        }
    }
    const Range own[] = {range(norm, 1, 4), range(ws, static_cast<int64_t>(ws_need), 1)};
    for (const Range &r : own)
        if (r.lo && r.lo != r.hi) items[m++] = {r.lo, r.hi, true};
    std::sort(items, items + m, [](const Item &p, const Item &q) { return p.lo < q.lo; });
    uintptr_t far_any = 0, far_out = 0;     // how far the ranges before this one reach
    int rc = SSM_OK;
    for (int64_t i = 0; i < m && rc == SSM_OK; ++i) {
        if (items[i].lo < (items[i].out ? far_any : far_out)) rc = SSM_ERR_ALIAS;
        far_any = std::max(far_any, items[i].hi);
        if (items[i].out) far_out = std::max(far_out, items[i].hi);
    }
    delete[] items;
    return rc;
}

int run_list(const void *const *grads, void *const *outs, const int64_t *numel, const int *dtypes,
             const int *out_dtypes, int64_t count, bool scale, float max_norm, float eps, float *norm,
             void *workspace, size_t workspace_bytes, void *stream) {
    const size_t need = count < 0 ? 0 : ssm::grad_norm_workspace(count);
    if (int r = check_list(grads, outs, numel, dtypes, out_dtypes, count, scale, norm, workspace, need)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    ssm::ClipArgs a{};
    a.grads = grads; a.outs = outs; a.numel = numel; a.dtypes = dtypes;
    a.out_dtypes = outs ? out_dtypes : dtypes;
    a.count = count; a.max_norm = max_norm; a.eps = eps; a.norm = norm; a.scale = scale;
    a.workspace = workspace;
    return hip_status(ssm::launch_grad_clip(a, static_cast<hipStream_t>(stream)));
}

// spin_limit: 0, or the error-path tests' (every hand-over withheld)
int gated_fwd(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
              const void *z, int64_t ldz, const float *h0, void *y, float *last_state,
              float *ckpt, int64_t batch, int64_t seqlen, int64_t d_inner, int io_dtype,
              void *workspace, size_t workspace_bytes, uint32_t spin_limit, void *stream) {
    if (int r = check_gated_sizes(batch, seqlen, d_inner, io_dtype)) return r;
    if (batch == 0 || d_inner == 0) return SSM_OK;
    ssm::GatedArgs a = gated_args(x, ldx, g, ldg, gate_bias, z, ldz, h0, batch, seqlen, d_inner, io_dtype, workspace,
                                  workspace_bytes);
    if (int r = check_gated_inputs(a, io_dtype)) return r;
    if (seqlen > 0 && !y) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    if (!aligned(y, es) || !aligned(last_state, 4) || !aligned(ckpt, 4)) return SSM_ERR_ALIGN;
    const int64_t steps = batch * seqlen, n_bd = batch * d_inner;
    const int64_t n_ck = batch * ((seqlen + ssm::kGatedBlock - 1) / ssm::kGatedBlock) * d_inner;
    const size_t need = ssm::gated_scan_workspace(batch, seqlen, d_inner, a.bf16);
    const Range ins[] = {range(x, span(steps, a.ldx, d_inner), es), range(g, span(steps, a.ldg, d_inner), es),
                         range(z, span(steps, a.ldz, d_inner), es), range(gate_bias, d_inner, 4), range(h0, n_bd, 4)};
    const Range outs[] = {range(y, steps * d_inner, es), range(last_state, n_bd, 4), range(ckpt, n_ck, 4),
                          range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    a.test_spin_limit = spin_limit;
    a.y = y; a.last_state = last_state; a.ckpt = ckpt;
    return hip_status(ssm::launch_gated_scan(a, static_cast<hipStream_t>(stream)));
}

int gated_bwd(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
              const void *z, int64_t ldz, const float *h0, const void *dout,
              const float *dlast, const float *ckpt, void *dx, void *dg, void *dz,
              float *dgate_bias, float *dh0, int64_t batch, int64_t seqlen, int64_t d_inner,
              int io_dtype, void *workspace, size_t workspace_bytes, uint32_t spin_limit, void *stream) {
    if (int r = check_gated_sizes(batch, seqlen, d_inner, io_dtype)) return r;
    if (d_inner == 0) return SSM_OK;
    ssm::GatedBwdArgs b{};
    b.fwd = gated_args(x, ldx, g, ldg, gate_bias, z, ldz, h0, batch, seqlen, d_inner, io_dtype, workspace,
                       workspace_bytes);
    if (int r = check_gated_inputs(b.fwd, io_dtype)) return r;
    const int64_t steps = batch * seqlen, n_bd = batch * d_inner;
    if (steps > 0 && (!dout || !dx || !dg || (z && !dz))) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    const void *io_ptrs[] = {dout, dx, dg, dz};
    for (const void *p : io_ptrs)
        if (!aligned(p, es)) return SSM_ERR_ALIGN;
    const void *f_ptrs[] = {dlast, ckpt, dgate_bias, dh0};
    for (const void *p : f_ptrs)
        if (!aligned(p, 4)) return SSM_ERR_ALIGN;
    const int64_t n_ck = batch * ((seqlen + ssm::kGatedBlock - 1) / ssm::kGatedBlock) * d_inner;
    const size_t need = ssm::gated_scan_bwd_workspace(batch, seqlen, d_inner, b.fwd.bf16);
    const Range ins[] = {range(x, span(steps, b.fwd.ldx, d_inner), es), range(g, span(steps, b.fwd.ldg, d_inner), es),
                         range(z, span(steps, b.fwd.ldz, d_inner), es), range(gate_bias, d_inner, 4),
                         range(h0, n_bd, 4), range(dout, steps * d_inner, es), range(dlast, n_bd, 4),
                         range(ckpt, n_ck, 4)};
    const Range outs[] = {range(dx, steps * d_inner, es), range(dg, steps * d_inner, es),
                          range(z ? dz : nullptr, steps * d_inner, es), range(dgate_bias, d_inner, 4),
                          range(dh0, n_bd, 4), range(need ? workspace : nullptr, static_cast<int64_t>(need), 1)};
    if (int r = check_overlap(outs, ins)) return r;
    if (int r = check_workspace(need, workspace, workspace_bytes)) return r;
    b.fwd.test_spin_limit = spin_limit;
    b.dout = dout; b.dlast = dlast; b.ckpt = ckpt;
    b.dx = dx; b.dg = dg; b.dz = z ? dz : nullptr;
    b.dgate_bias = dgate_bias; b.dh0 = dh0;
    return hip_status(ssm::launch_gated_scan_bwd(b, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t ssm_gated_ckpt_bytes(int64_t batch, int64_t seqlen, int64_t d_inner) {
    if (batch < 0 || seqlen < 0 || d_inner < 0) return static_cast<size_t>(-1);
    const int64_t n = mul3(batch, seqlen / ssm::kGatedBlock + (seqlen % ssm::kGatedBlock != 0), d_inner);
    return n < 0 ? static_cast<size_t>(-1) : static_cast<size_t>(n) * 4;
}

size_t ssm_gated_scan_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, int io_dtype) {
    if (check_gated_sizes(batch, seqlen, d_inner, io_dtype)) return static_cast<size_t>(-1);
    return ssm::gated_scan_workspace(batch, seqlen, d_inner, io_dtype == SSM_BF16);
}

int ssm_gated_scan_fwd(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
                       const void *z, int64_t ldz, const float *h0, void *y, float *last_state,
                       float *ckpt, int64_t batch, int64_t seqlen, int64_t d_inner, int io_dtype,
                       void *workspace, size_t workspace_bytes, void *stream) {
    return gated_fwd(x, ldx, g, ldg, gate_bias, z, ldz, h0, y, last_state, ckpt, batch, seqlen, d_inner, io_dtype, workspace,
                     workspace_bytes, 0, stream);
}

size_t ssm_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t d_inner, int io_dtype) {
    if (check_gated_sizes(batch, seqlen, d_inner, io_dtype)) return static_cast<size_t>(-1);
    return ssm::gated_scan_bwd_workspace(batch, seqlen, d_inner, io_dtype == SSM_BF16);
}

int ssm_gated_scan_bwd(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
                       const void *z, int64_t ldz, const float *h0, const void *dout,
                       const float *dlast, const float *ckpt, void *dx, void *dg, void *dz,
                       float *dgate_bias, float *dh0, int64_t batch, int64_t seqlen, int64_t d_inner,
                       int io_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return gated_bwd(x, ldx, g, ldg, gate_bias, z, ldz, h0, dout, dlast, ckpt, dx, dg, dz, dgate_bias, dh0, batch, seqlen, d_inner,
                     io_dtype, workspace, workspace_bytes, 0, stream);
}

int ssm_testing_gated_fwd_no_handoff(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
                       const void *z, int64_t ldz, const float *h0, void *y, float *last_state,
                       float *ckpt, int64_t batch, int64_t seqlen, int64_t d_inner, int io_dtype,
                       void *workspace, size_t workspace_bytes, uint32_t spin_limit, void *stream) {
    if (spin_limit < 1 || spin_limit > 65536) return SSM_ERR_SHAPE;
    return gated_fwd(x, ldx, g, ldg, gate_bias, z, ldz, h0, y, last_state, ckpt, batch, seqlen, d_inner, io_dtype, workspace,
                     workspace_bytes, spin_limit, stream);
}

int ssm_testing_gated_bwd_no_handoff(const void *x, int64_t ldx, const void *g, int64_t ldg, const float *gate_bias,
                       const void *z, int64_t ldz, const float *h0, const void *dout,
                       const float *dlast, const float *ckpt, void *dx, void *dg, void *dz,
                       float *dgate_bias, float *dh0, int64_t batch, int64_t seqlen, int64_t d_inner,
                       int io_dtype, void *workspace, size_t workspace_bytes, uint32_t spin_limit, void *stream) {
    if (spin_limit < 1 || spin_limit > 65536) return SSM_ERR_SHAPE;
    return gated_bwd(x, ldx, g, ldg, gate_bias, z, ldz, h0, dout, dlast, ckpt, dx, dg, dz, dgate_bias, dh0, batch, seqlen, d_inner,
                     io_dtype, workspace, workspace_bytes, spin_limit, stream);
}

int ssm_gated_state_update(float *state, const void *x, const void *g, const float *gate_bias,
                           const void *z, void *y, int64_t batch, int64_t d_inner, int io_dtype,
                           void *stream) {
    if (int r = check_dtype(io_dtype)) return r;
    const int64_t n = mul3(batch, d_inner, 1);
    if (n < 0 || n > kMaxSpan) return SSM_ERR_SHAPE;
    if (n == 0) return SSM_OK;
    if (!state || !x || !g || !y) return SSM_ERR_NULL;
    const size_t es = io_size(io_dtype);
    const void *io_ptrs[] = {x, g, z, y};
    for (const void *p : io_ptrs)
        if (!aligned(p, es)) return SSM_ERR_ALIGN;
    if (!aligned(state, 4) || !aligned(gate_bias, 4)) return SSM_ERR_ALIGN;
    const Range ins[] = {range(x, n, es), range(g, n, es), range(z, n, es), range(gate_bias, d_inner, 4)};
    const Range outs[] = {range(state, n, 4), range(y, n, es)};
    if (int r = check_overlap(outs, ins)) return r;
    ssm::GatedStepArgs a{};
    a.state = state; a.x = x; a.g = g; a.z = z; a.gate_bias = gate_bias; a.y = y;
    a.batch = batch; a.dim = d_inner;
    a.bf16 = io_dtype == SSM_BF16 ? 1 : 0;
    return hip_status(ssm::launch_gated_update(a, static_cast<hipStream_t>(stream)));
}

int ssm_add_rms_norm_fwd(const void *x, int64_t ldx, const void *residual, const float *weight, void *y,
                         void *residual_out, int64_t rows, int64_t dim, float eps, int io_dtype,
                         int residual_dtype, void *stream) {
    if (int r = check_norm(x, ldx, residual, weight, y, io_size(io_dtype), nullptr, residual_out, rows, dim, eps,
                           io_dtype, residual_dtype))
        return r;
    if (rows == 0) return SSM_OK;
    ssm::NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.residual_out = residual_out;
    a.rows = rows; a.dim = dim; a.ldx = rows > 1 ? ldx : dim; a.eps = eps;
    a.bf16 = io_dtype == SSM_BF16; a.res_bf16 = residual_dtype == SSM_BF16;
    return hip_status(ssm::launch_add_rms_norm(a, static_cast<hipStream_t>(stream)));
}

int ssm_add_rms_norm_quant(const void *x, int64_t ldx, const void *residual, const float *weight, void *q,
                           float *scale, void *residual_out, int64_t rows, int64_t dim, float eps,
                           int io_dtype, int residual_dtype, void *stream) {
    if (int r = check_norm(x, ldx, residual, weight, q, 1, scale, residual_out, rows, dim, eps, io_dtype,
                           residual_dtype))
        return r;
    if (rows == 0) return SSM_OK;
    if (!scale) return SSM_ERR_NULL;
    ssm::NormArgs a{};
    a.x = x; a.residual = residual; a.weight = weight; a.y = q; a.scale = scale; a.residual_out = residual_out;
    a.rows = rows; a.dim = dim; a.ldx = rows > 1 ? ldx : dim; a.eps = eps;
    a.bf16 = io_dtype == SSM_BF16; a.res_bf16 = residual_dtype == SSM_BF16;
    return hip_status(ssm::launch_add_rms_norm(a, static_cast<hipStream_t>(stream)));
}

size_t ssm_add_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t dim) {
    if (rows < 0 || rows > kMaxSpan || dim < 1 || dim > SSM_MAX_NORM_DIM) return static_cast<size_t>(-1);
    return ssm::norm_bwd_workspace(rows, dim);
}

int ssm_add_rms_norm_bwd(const void *dy, const void *r, const float *weight, const void *dresidual_out,
                         void *dx, void *dresidual, float *dweight, int64_t rows, int64_t dim, float eps,
                         int io_dtype, int residual_dtype, void *workspace, size_t workspace_bytes,
                         void *stream) {
    return norm_bwd(dy, r, dim, weight, dresidual_out, dx, dresidual, dweight, rows, dim, eps, io_dtype, residual_dtype,
                    workspace, workspace_bytes, stream);
}

int ssm_add_rms_norm_bwd_strided(const void *dy, const void *r, int64_t ldr, const float *weight,
                                 const void *dresidual_out, void *dx, void *dresidual, float *dweight, int64_t rows,
                                 int64_t dim, float eps, int io_dtype, int residual_dtype, void *workspace,
                                 size_t workspace_bytes, void *stream) {
    return norm_bwd(dy, r, ldr, weight, dresidual_out, dx, dresidual, dweight, rows, dim, eps, io_dtype, residual_dtype,
                    workspace, workspace_bytes, stream);
}

size_t ssm_grad_norm_workspace_bytes(int64_t count) {
    if (count < 0 || count > (int64_t(1) << 20)) return static_cast<size_t>(-1);
    return ssm::grad_norm_workspace(count);
}

int ssm_grad_norm(const void *const *grads, const int64_t *numel, const int *dtypes, int64_t count,
                  float *norm, void *workspace, size_t workspace_bytes, void *stream) {
    return run_list(grads, nullptr, numel, dtypes, nullptr, count, false, 0.0f, 0.0f, norm, workspace,
                    workspace_bytes, stream);
}

int ssm_grad_clip(const void *const *grads, void *const *outs, const int64_t *numel, const int *dtypes,
                  const int *out_dtypes, int64_t count, float max_norm, float eps, float *norm,
                  void *workspace, size_t workspace_bytes, void *stream) {
    if (!(max_norm >= 0.0f) || !(eps >= 0.0f) || std::isinf(eps)) return SSM_ERR_VALUE;
    return run_list(grads, outs, numel, dtypes, out_dtypes, count, true, max_norm, eps, norm, workspace,
                    workspace_bytes, stream);
}

}  // extern "C"
