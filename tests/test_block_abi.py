"""The C ABI of the gated recurrent block's operators, checked on the CPU: bad
arguments are refused before the HIP runtime is touched, empty problems are
no-ops, and workspace sizes are what the header says.  Nothing here launches."""
import ctypes
import os

import pytest

from selective_scan_ssm_amd import _lib

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EALIAS, EVALUE = 0, -1, -2, -3, -4, -5, -7, -10
F32, BF16 = 0, 1
BAD = (1 << 64) - 1
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from selective_scan_ssm_amd import build
        build.build()
    return _lib.load()


class FakeDev:
    """Distinct, aligned device addresses that are never dereferenced."""

    def __init__(self):
        self.at = 0x7f0000000000

    def __call__(self, nbytes=64 * MB):
        p = self.at
        self.at += (nbytes + 4095) & ~4095
        return p


def scan_args(**over):
    f = FakeDev()
    a = dict(x=f(), ldx=8, g=f(), ldg=8, bias=f(), z=f(), ldz=8, h0=f(), y=f(), last=f(), ckpt=f(), batch=2, seqlen=300,
             dim=8, io=F32, ws=f(), ws_bytes=64 * MB, dout=f(), dlast=f(), dx=f(), dg=f(), dz=f(), dbias=f(), dh0=f())
    a.update(over)
    return a


def fwd(lib, a):
    return lib.ssm_gated_scan_fwd(a["x"], a["ldx"], a["g"], a["ldg"], a["bias"], a["z"], a["ldz"], a["h0"], a["y"],
                                  a["last"], a["ckpt"], a["batch"], a["seqlen"], a["dim"], a["io"], a["ws"],
                                  a["ws_bytes"], None)


def bwd(lib, a):
    return lib.ssm_gated_scan_bwd(a["x"], a["ldx"], a["g"], a["ldg"], a["bias"], a["z"], a["ldz"], a["h0"], a["dout"],
                                  a["dlast"], a["ckpt"], a["dx"], a["dg"], a["dz"], a["dbias"], a["dh0"], a["batch"],
                                  a["seqlen"], a["dim"], a["io"], a["ws"], a["ws_bytes"], None)


BOTH = [(dict(x=None), ENULL), (dict(g=None), ENULL), (dict(io=2), EDTYPE), (dict(batch=-1), ESHAPE),
        (dict(seqlen=-1), ESHAPE), (dict(dim=-1), ESHAPE), (dict(batch=65536), ESHAPE), (dict(ldx=7), ESHAPE),
        (dict(ldg=0), ESHAPE), (dict(ldz=-8), ESHAPE), (dict(ldx=1 << 23), ESHAPE), (dict(dim=1 << 23, ldx=1 << 23), ESHAPE),
        (dict(batch=1 << 15, seqlen=1 << 62), ESHAPE), (dict(x=0x7f0000000002), EALIGN),
        (dict(io=BF16, g=0x7f0000000001), EALIGN), (dict(bias=0x7f0000000002), EALIGN), (dict(h0=0x7f0000000001), EALIGN)]


@pytest.mark.parametrize("over,code", BOTH + [(dict(y=None), ENULL), (dict(last=0x7f0000000002), EALIGN),
                                              (dict(ckpt=0x7f0000000001), EALIGN)])
def test_gated_fwd_refuses(lib, over, code):
    assert fwd(lib, scan_args(**over)) == code


@pytest.mark.parametrize("over,code", BOTH + [(dict(dout=None), ENULL), (dict(dx=None), ENULL), (dict(dg=None), ENULL),
                                              (dict(dz=None), ENULL), (dict(dlast=0x7f0000000002), EALIGN),
                                              (dict(ws=None), EWS), (dict(ws_bytes=16), EWS)])
def test_gated_bwd_refuses(lib, over, code):
    assert bwd(lib, scan_args(**over)) == code


def test_gated_overlaps(lib):
    a = scan_args()
    for over in (dict(y=a["x"] + 64), dict(y=a["g"]), dict(last=a["h0"]), dict(ckpt=a["y"]), dict(last=a["y"])):
        assert fwd(lib, scan_args(**over)) == EALIAS, over
    for over in (dict(dx=a["x"]), dict(dg=a["dx"]), dict(dz=a["dout"]), dict(dh0=a["dlast"]), dict(dbias=a["bias"]),
                 dict(ws=a["dx"])):
        assert bwd(lib, scan_args(**over)) == EALIAS, over


def test_gated_strided_views_may_interleave(lib):
    # thirds of one projection: ranges overlap one another, the output sits behind them
    a = scan_args(ldx=24, ldg=24, ldz=24)
    a["g"], a["z"] = a["x"] + 32, a["x"] + 64
    a["y"] = a["x"] + 4 * (24 * 599 + 16)          # inside the last row of z
    assert fwd(lib, a) == EALIAS


def test_gated_empty(lib):
    assert fwd(lib, scan_args(batch=0, x=None, y=None)) == OK
    assert fwd(lib, scan_args(dim=0, ldx=0, ldg=0, ldz=0)) == OK
    assert bwd(lib, scan_args(dim=0)) == OK


def test_gated_sizes(lib):
    assert lib.ssm_gated_ckpt_bytes(2, 300, 8) == 2 * 3 * 8 * 4
    assert lib.ssm_gated_ckpt_bytes(2, 0, 8) == 0
    assert lib.ssm_gated_ckpt_bytes(-1, 1, 1) == BAD
    assert lib.ssm_gated_ckpt_bytes(1 << 40, 1 << 40, 8) == BAD
    assert lib.ssm_gated_scan_workspace_bytes(1, 1, 1, F32) == 0
    assert lib.ssm_gated_scan_workspace_bytes(1, 1, 1, 9) == BAD
    assert lib.ssm_gated_scan_bwd_workspace_bytes(1, 100, -4, F32) == BAD
    assert lib.ssm_gated_scan_bwd_workspace_bytes(2, 300, 8, F32) > 0
    # an error word and its line come before the sums; nothing is run, nothing needed, without a row or a channel
    assert lib.ssm_gated_scan_bwd_workspace_bytes(1, 1, 1, F32) >= 512
    assert lib.ssm_gated_scan_bwd_workspace_bytes(0, 300, 8, F32) == lib.ssm_gated_scan_workspace_bytes(0, 300, 8, F32) == 0


@pytest.mark.parametrize("limit", [0, 65537])
def test_testing_entries_bound_their_limit(lib, limit):
    a = scan_args()
    head = (a["x"], 8, a["g"], 8, a["bias"], a["z"], 8, a["h0"])
    tail = (2, 300, 8, F32, a["ws"], a["ws_bytes"], limit, None)
    assert lib.ssm_testing_gated_fwd_no_handoff(*head, a["y"], a["last"], a["ckpt"], *tail) == ESHAPE
    assert lib.ssm_testing_gated_bwd_no_handoff(*head, a["dout"], a["dlast"], a["ckpt"], a["dx"], a["dg"], a["dz"], a["dbias"],
                                                a["dh0"], *tail) == ESHAPE


def update(lib, **over):
    f = FakeDev()
    a = dict(state=f(), x=f(), g=f(), bias=f(), z=f(), y=f(), batch=2, dim=8, io=F32)
    a.update(over)
    return lib.ssm_gated_state_update(a["state"], a["x"], a["g"], a["bias"], a["z"], a["y"], a["batch"], a["dim"],
                                      a["io"], None)


@pytest.mark.parametrize("over,code", [
    (dict(state=None), ENULL), (dict(x=None), ENULL), (dict(g=None), ENULL), (dict(y=None), ENULL), (dict(io=3), EDTYPE),
    (dict(batch=-1), ESHAPE), (dict(batch=1 << 16, dim=1 << 16), ESHAPE), (dict(state=0x7f0000000002), EALIGN),
    (dict(y=0x7f0000000000), EALIAS), (dict(batch=0), OK), (dict(dim=0, x=None), OK)])
def test_update_refuses(lib, over, code):
    assert update(lib, **over) == code


def norm_args(**over):
    f = FakeDev()
    a = dict(x=f(), ldx=16, res=f(), w=f(), y=f(), scale=f(), res_out=f(), rows=4, dim=16, eps=1e-5, io=F32, rt=F32,
             dy=f(), r=f(), dro=f(), dx=f(), dres=f(), dw=f(), ws=f(), ws_bytes=64 * MB)
    a.update(over)
    return a


def norm_fwd(lib, a):
    return lib.ssm_add_rms_norm_fwd(a["x"], a["ldx"], a["res"], a["w"], a["y"], a["res_out"], a["rows"], a["dim"],
                                    a["eps"], a["io"], a["rt"], None)


def norm_quant(lib, a):
    return lib.ssm_add_rms_norm_quant(a["x"], a["ldx"], a["res"], a["w"], a["y"], a["scale"], a["res_out"], a["rows"],
                                      a["dim"], a["eps"], a["io"], a["rt"], None)


def norm_bwd(lib, a):
    return lib.ssm_add_rms_norm_bwd(a["dy"], a["r"], a["w"], a["dro"], a["dx"], a["dres"], a["dw"], a["rows"], a["dim"],
                                    a["eps"], a["io"], a["rt"], a["ws"], a["ws_bytes"], None)


NORM = [(dict(io=7), EDTYPE), (dict(io=F32, rt=BF16), EDTYPE), (dict(rt=5), EDTYPE), (dict(rows=-1), ESHAPE),
        (dict(dim=0), ESHAPE), (dict(dim=32769, ldx=40000), ESHAPE), (dict(rows=1 << 31), ESHAPE), (dict(eps=-1.0), EVALUE),
        (dict(eps=float("nan")), EVALUE), (dict(eps=float("inf")), EVALUE), (dict(w=None), ENULL),
        (dict(w=0x7f0000000002), EALIGN)]


@pytest.mark.parametrize("over,code", NORM + [(dict(x=None), ENULL), (dict(y=None), ENULL), (dict(ldx=15), ESHAPE),
                                              (dict(x=0x7f0000000002), EALIGN), (dict(res=0x7f0000000001), EALIGN)])
def test_norm_refuses(lib, over, code):
    assert norm_fwd(lib, norm_args(**over)) == code
    if "y" not in over:
        assert norm_quant(lib, norm_args(**over)) == code


def test_norm_quant_needs_its_scale(lib):
    assert norm_quant(lib, norm_args(scale=None)) == ENULL
    assert norm_quant(lib, norm_args(scale=0x7f0000000002)) == EALIGN


@pytest.mark.parametrize("over,code", NORM + [(dict(dy=None), ENULL), (dict(r=None), ENULL), (dict(dx=None), ENULL),
                                              (dict(dw=None), ENULL), (dict(ws=None), EWS), (dict(ws_bytes=8), EWS),
                                              (dict(dro=0x7f0000000002), EALIGN)])
def test_norm_bwd_refuses(lib, over, code):
    assert norm_bwd(lib, norm_args(**over)) == code


def test_norm_overlaps(lib):
    a = norm_args()
    for over in (dict(y=a["x"]), dict(y=a["res"]), dict(res_out=a["x"]), dict(res_out=a["res"] + 4), dict(res_out=a["y"]),
                 dict(y=a["w"])):
        assert norm_fwd(lib, norm_args(**over)) == EALIAS, over
    assert norm_quant(lib, norm_args(scale=a["y"])) == EALIAS
    for over in (dict(dx=a["dy"]), dict(dx=a["r"]), dict(dres=a["dro"] + 4), dict(dres=a["dx"]), dict(dw=a["w"]),
                 dict(ws=a["r"])):
        assert norm_bwd(lib, norm_args(**over)) == EALIAS, over


def test_norm_empty(lib):
    assert norm_fwd(lib, norm_args(rows=0, x=None)) == OK
    assert norm_quant(lib, norm_args(rows=0, x=None)) == OK
    assert lib.ssm_add_rms_norm_bwd_workspace_bytes(1, 0) == BAD
    assert lib.ssm_add_rms_norm_bwd_workspace_bytes(-1, 4) == BAD
    assert lib.ssm_add_rms_norm_bwd_workspace_bytes(100, 64) > 0


def clip(lib, ptrs, numel, dtypes, outs=None, out_dtypes=None, max_norm=1.0, eps=1e-6, norm=0x7e0000000000,
         ws=0x7d0000000000, ws_bytes=64 * MB, count=None, norm_only=False):
    n = len(ptrs)
    arr = lambda t, v: None if v is None else (t * n)(*v)
    args = [arr(ctypes.c_void_p, ptrs)]
    count = n if count is None else count
    if norm_only:
        return lib.ssm_grad_norm(*args, arr(ctypes.c_int64, numel), arr(ctypes.c_int, dtypes), count, norm, ws, ws_bytes,
                                 None)
    return lib.ssm_grad_clip(*args, arr(ctypes.c_void_p, outs), arr(ctypes.c_int64, numel), arr(ctypes.c_int, dtypes),
                             arr(ctypes.c_int, out_dtypes), count, max_norm, eps, norm, ws, ws_bytes, None)


P, Q = 0x7f0000000000, 0x7f0000100000


@pytest.mark.parametrize("norm_only", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(ptrs=[P, None], numel=[4, 4], dtypes=[0, 0]), ENULL), (dict(ptrs=[P], numel=[4], dtypes=[2]), EDTYPE),
    (dict(ptrs=[P], numel=[-1], dtypes=[0]), ESHAPE), (dict(ptrs=[P], numel=[1 << 40], dtypes=[0]), ESHAPE),
    (dict(ptrs=[P + 2], numel=[4], dtypes=[0]), EALIGN), (dict(ptrs=[P + 1], numel=[4], dtypes=[1]), EALIGN),
    (dict(ptrs=[P], numel=[4], dtypes=[0], norm=None), ENULL), (dict(ptrs=[P], numel=[4], dtypes=[0], norm=P + 8), EALIAS),
    (dict(ptrs=[P], numel=[4], dtypes=[0], ws=None), EWS), (dict(ptrs=[P], numel=[4], dtypes=[0], ws_bytes=8), EWS),
    (dict(ptrs=[P], numel=[4], dtypes=[0], ws=0x7d0000000010), EALIGN), (dict(ptrs=[P], numel=[4], dtypes=[0], count=-1), ESHAPE),
    (dict(ptrs=[P], numel=[1 << 20], dtypes=[0], ws=P + 4096), EALIAS),
    (dict(ptrs=[P], numel=[4], dtypes=[0], count=(1 << 20) + 1), ESHAPE)])
def test_clip_refuses(lib, kw, code, norm_only):
    assert clip(lib, norm_only=norm_only, **kw) == code


@pytest.mark.parametrize("kw", [dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1e-6), dict(eps=float("inf"))])
def test_clip_values(lib, kw):
    assert clip(lib, [P], [4], [0], **kw) == EVALUE


def test_clip_overlaps(lib):
    one = dict(numel=[16, 16], dtypes=[0, 0])
    assert clip(lib, [P, P], **one) == EALIAS                                        # the same tensor twice, in place
    assert clip(lib, [P, P + 32], **one) == EALIAS
    assert clip(lib, [P, Q], outs=[P, P], out_dtypes=[0, 0], **one) == EALIAS        # one output twice
    assert clip(lib, [P, Q], outs=[Q, P], out_dtypes=[0, 0], **one) == EALIAS        # outputs on other inputs
    assert clip(lib, [P, Q], outs=[P, Q], out_dtypes=[1, 0], **one) == EALIAS        # in place, another dtype
    assert clip(lib, [P, Q], outs=[P + 4096, Q + 4096], out_dtypes=[0, 9], **one) == EDTYPE
    assert clip(lib, [P, Q], outs=[P + 4096, None], out_dtypes=[0, 0], **one) == ENULL


def test_clip_workspace(lib):
    assert lib.ssm_grad_norm_workspace_bytes(-1) == BAD and lib.ssm_grad_norm_workspace_bytes((1 << 20) + 1) == BAD
    assert lib.ssm_grad_norm_workspace_bytes(1) > 0


def test_status_strings_of_the_new_codes(lib):
    for code in (-10, -11):
        assert lib.ssm_status_string(code).decode().startswith("SSM_ERR_")


def norm_bwd_strided(lib, ldr, **over):
    a = norm_args(**over)
    return lib.ssm_add_rms_norm_bwd_strided(a["dy"], a["r"], ldr, a["w"], a["dro"], a["dx"], a["dres"], a["dw"], a["rows"],
                                            a["dim"], a["eps"], a["io"], a["rt"], a["ws"], a["ws_bytes"], None)


def test_norm_bwd_strided_refuses(lib):
    for over, code in NORM + [(dict(r=None), ENULL), (dict(r=0x7f0000000002), EALIGN), (dict(ws_bytes=8), EWS)]:
        assert norm_bwd_strided(lib, 40000, **over) == code, over
    for ldr in (15, 0, -16, 1 << 60):
        assert norm_bwd_strided(lib, ldr) == ESHAPE, ldr
    # an output between the rows of r, in the span of the last one
    a = norm_args()
    assert norm_bwd_strided(lib, 48, dx=a["r"] + 4 * 20) == EALIAS
    assert norm_bwd_strided(lib, 48, dw=a["r"] + 4 * (3 * 48 + 15)) == EALIAS


# one tile below and at 2^32 lanes: 64 to a workgroup up to 16 steps, then 128, 256, 512
@pytest.mark.parametrize("batch,seqlen,dim,code", [
    (40000, 16, 4096, OK), (65535, 1, 64, OK), (65535, 128, 4096, OK), (65535, 16, 65536, OK), (65535, 16, 65537, ESHAPE),
    (32767, 17, 65536, OK), (32768, 17, 65536, ESHAPE), (16383, 64, 65536, OK), (16384, 33, 65536, ESHAPE),
    (8191, 128, 65536, OK), (8192, 65, 65536, ESHAPE), (4095, 129, 65536, OK), (4096, 129, 65536, ESHAPE),
    (1, (1 << 30) - 128, 64, OK), (1, (1 << 30) - 127, 64, ESHAPE), (1, 1 << 62, 64, ESHAPE), (65536, 1, 1, ESHAPE)])
def test_gated_largest_sizes(lib, batch, seqlen, dim, code):
    for need in (lib.ssm_gated_scan_workspace_bytes, lib.ssm_gated_scan_bwd_workspace_bytes):
        assert (need(batch, seqlen, dim, BF16) == BAD) == (code == ESHAPE)
    if code == ESHAPE:
        a = scan_args(batch=batch, seqlen=seqlen, dim=dim, ldx=dim, ldg=dim, ldz=dim)
        assert fwd(lib, a) == bwd(lib, a) == ESHAPE


def test_the_value_status_says_what_is_refused(lib):
    """An infinite max_norm is no limit and accepted; a NaN or negative one, and an eps that is not finite, are not."""
    said = lib.ssm_status_string(EVALUE).decode()
    assert "eps is negative or not finite" in said and "max_norm is negative or NaN" in said
    header = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ssm_scan.h")).read()
    assert "eps is negative or not finite, or max_norm negative or NaN" in header
    kw = dict(ptrs=[P], numel=[4], dtypes=[0], ws=None)
    assert clip(lib, max_norm=float("inf"), **kw) == EWS                  # past the check of values
    assert clip(lib, max_norm=float("nan"), **kw) == clip(lib, eps=float("nan"), **kw) == EVALUE


def test_gated_row_strides_of_short_sequences(lib):
    """The first step of each of a batch's long rows is far from the next one's; a sequence itself spans little."""
    far = dict(batch=2, dim=8, ws=None, last=None, ckpt=0x7f0000000001)          # refused after the sizes are accepted
    for seqlen, ld, code in ((1, (1 << 29) - 1, EALIGN), (1, 1 << 29, ESHAPE), (5, 107374182, EALIGN), (5, 107374183, ESHAPE),
                             (128, (1 << 22) - 1, EALIGN), (128, 1 << 22, ESHAPE), (4000, (1 << 22) - 1, EALIGN),
                             (4000, 1 << 22, ESHAPE)):
        a = scan_args(seqlen=seqlen, ldx=ld, ldg=ld, ldz=ld, **far)
        assert fwd(lib, a) == code and bwd(lib, a) == code, (seqlen, ld)
