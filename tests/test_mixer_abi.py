"""The C ABI of the gated delta rule and of the group norm, checked on the CPU:
bad arguments are refused before the HIP runtime is touched, empty problems are
no-ops, and workspace sizes are what the header says.  Nothing here launches."""
import os

import pytest

from selective_scan_ssm_amd import _lib

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS, EALIAS, EVALUE = 0, -1, -2, -3, -4, -5, -7, -10
F32, BF16 = 0, 1
BAD = (1 << 64) - 1
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


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


def delta_args(**over):
    f = FakeDev()
    a = dict(q=f(), ldq=16, k=f(), ldk=16, v=f(), ldv=64, g=f(), beta=f(), scale=0.25, h0=f(), starts=None, nseq=0, y=f(),
             last=f(), ckpt=f(), batch=2, seqlen=130, kheads=2, heads=4, dk=8, dv=16, io=F32, ws=f(256 * MB), ws_bytes=256 * MB,
             dout=f(), dlast=f(), dq=f(), dkey=f(), dval=f(), dg=f(), dbeta=f(), dh0=f())
    a.update(over)
    return a


def heads_in(a):
    return (a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["g"], a["beta"], a["scale"], a["h0"], a["starts"], a["nseq"])


def tail(a):
    return (a["batch"], a["seqlen"], a["kheads"], a["heads"], a["dk"], a["dv"], a["io"], a["ws"], a["ws_bytes"], None)


def fwd(lib, a):
    return lib.ssm_delta_scan_fwd(*heads_in(a), a["y"], a["last"], a["ckpt"], *tail(a))


def bwd(lib, a):
    return lib.ssm_delta_scan_bwd(*heads_in(a), a["dout"], a["dlast"], a["ckpt"], a["dq"], a["dkey"], a["dval"], a["dg"], a["dbeta"],
                                  a["dh0"], *tail(a))


BOTH = [(dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(g=None), ENULL), (dict(beta=None), ENULL),
        (dict(io=2), EDTYPE), (dict(batch=-1), ESHAPE), (dict(seqlen=-1), ESHAPE), (dict(seqlen=1 << 31), ESHAPE),
        (dict(kheads=0), ESHAPE), (dict(kheads=3), ESHAPE), (dict(heads=0), ESHAPE), (dict(dk=12), ESHAPE), (dict(dk=0), ESHAPE),
        (dict(dk=136, ldq=512, ldk=512), ESHAPE), (dict(dv=12), ESHAPE), (dict(dv=0), ESHAPE), (dict(ldq=12), ESHAPE),
        (dict(ldk=18), ESHAPE), (dict(ldv=60), ESHAPE), (dict(io=BF16, ldv=68), ESHAPE), (dict(ldq=1 << 23), ESHAPE),
        (dict(batch=1 << 40), ESHAPE), (dict(batch=1 << 20, seqlen=1 << 14), ESHAPE), (dict(dv=1 << 30, ldv=1 << 40), ESHAPE),
        (dict(starts=0x7f0000100000, nseq=3), ESHAPE), (dict(starts=0x7f0000100000, nseq=-1, batch=1), ESHAPE),
        (dict(starts=0x7f0000100002, nseq=1, batch=1), EALIGN), (dict(scale=NAN), EVALUE), (dict(scale=INF), EVALUE),
        (dict(q=0x7f0000000008), EALIGN), (dict(h0=0x7f0000000004), EALIGN), (dict(g=0x7f0000000002), EALIGN),
        (dict(beta=0x7f0000000001), EALIGN), (dict(ckpt=0x7f0000000008), EALIGN), (dict(ws=None), EWS), (dict(ws_bytes=64), EWS),
        (dict(ws=0x7f0100000010), EALIGN)]


@pytest.mark.parametrize("over,code", BOTH + [(dict(y=None), ENULL), (dict(y=0x7f0000000008), EALIGN),
                                              (dict(last=0x7f0000000004), EALIGN)])
def test_delta_fwd_refuses(lib, over, code):
    assert fwd(lib, delta_args(**over)) == code


@pytest.mark.parametrize("over,code", BOTH + [(dict(dout=None), ENULL), (dict(dq=None), ENULL), (dict(dkey=None), ENULL),
                                              (dict(dval=None), ENULL), (dict(dg=None), ENULL), (dict(dbeta=None), ENULL),
                                              (dict(dh0=0x7f0000000004), EALIGN), (dict(dlast=0x7f0000000004), EALIGN)])
def test_delta_bwd_refuses(lib, over, code):
    assert bwd(lib, delta_args(**over)) == code


def test_delta_overlaps(lib):
    a = delta_args()
    for over in (dict(y=a["v"]), dict(y=a["q"] + 64), dict(last=a["h0"]), dict(ckpt=a["y"]), dict(last=a["y"]), dict(ws=a["k"])):
        assert fwd(lib, delta_args(**over)) == EALIAS, over
    for over in (dict(dq=a["q"]), dict(dkey=a["dq"]), dict(dval=a["dout"]), dict(dg=a["g"]), dict(dbeta=a["dg"]),
                 dict(dh0=a["dlast"]), dict(ws=a["dkey"]), dict(dg=a["ckpt"])):
        assert bwd(lib, delta_args(**over)) == EALIAS, over
    # ranges of one projection overlap one another; an output inside the last step of v is found
    p = delta_args(ldq=96, ldk=96, ldv=96)
    p["k"], p["v"] = p["q"] + 64, p["q"] + 128
    p["y"] = p["v"] + 4 * 96 * 259 + 128
    assert fwd(lib, p) == EALIAS


def test_delta_empty(lib):
    assert fwd(lib, delta_args(batch=0, q=None, y=None)) == OK
    assert bwd(lib, delta_args(batch=0, q=None, dq=None)) == OK
    assert fwd(lib, delta_args(batch=1, starts=0x7f0000100000, nseq=0)) == OK


def test_delta_sizes(lib):
    assert lib.ssm_delta_ckpt_bytes(2, 130, 0, 0, 4, 8, 16) == 2 * 3 * 4 * 16 * (8 + 64) * 4
    assert lib.ssm_delta_ckpt_bytes(1, 130, 1, 5, 4, 8, 16) == (2 + 5) * 4 * 16 * (8 + 64) * 4
    assert lib.ssm_delta_ckpt_bytes(2, 130, 1, 5, 4, 8, 16) == BAD
    assert lib.ssm_delta_ckpt_bytes(2, 0, 0, 0, 4, 8, 16) == 0
    for fn, extra in ((lib.ssm_delta_scan_workspace_bytes, ()), (lib.ssm_delta_scan_bwd_workspace_bytes, (0,)),
                      (lib.ssm_delta_scan_bwd_workspace_bytes, (1,))):
        assert fn(2, 0, 0, 0, 2, 4, 8, 16, *extra, F32) == 0
        assert 0 < fn(2, 130, 0, 0, 2, 4, 8, 16, *extra, F32) < BAD
        assert fn(2, 130, 0, 0, 3, 4, 8, 16, *extra, F32) == BAD
        assert fn(2, 130, 0, 0, 2, 4, 8, 16, *extra, 7) == BAD
    free, saved = (lib.ssm_delta_scan_bwd_workspace_bytes(2, 130, 0, 0, 2, 4, 8, 16, s, F32) for s in (0, 1))
    assert free >= saved + lib.ssm_delta_ckpt_bytes(2, 130, 0, 0, 4, 8, 16)


def update(lib, **over):
    f = FakeDev()
    a = dict(state=f(), q=f(), k=f(), v=f(), g=f(), beta=f(), scale=1.0, y=f(), batch=2, kheads=2, heads=4, dk=8, dv=16, io=F32)
    a.update(over)
    return lib.ssm_delta_state_update(*(a[n] for n in ("state", "q", "k", "v", "g", "beta", "scale", "y", "batch", "kheads", "heads",
                                                       "dk", "dv", "io")), None)


@pytest.mark.parametrize("over,code", [(dict([(n, None)]), ENULL) for n in ("state", "q", "k", "v", "g", "beta", "y")] + [
    (dict(io=3), EDTYPE), (dict(batch=-1), ESHAPE), (dict(batch=1 << 40), ESHAPE), (dict(heads=5), ESHAPE), (dict(dk=4), ESHAPE),
    (dict(dv=20), ESHAPE), (dict(scale=NAN), EVALUE), (dict(state=0x7f0000000008), EALIGN), (dict(v=0x7f0000000002), EALIGN),
    (dict(g=0x7f0000000002), EALIGN), (dict(y=0x7f0000000000), EALIAS), (dict(batch=0, state=None), OK)])
def test_update_refuses(lib, over, code):
    assert update(lib, **over) == code


def norm_args(**over):
    f = FakeDev()
    a = dict(x=f(), ldx=24, z=f(), ldz=24, w=f(), b=f(), y=f(), mean=f(), rstd=f(), batch=3, rows=5000, dim=24, groups=4, eps=1e-5, silu=1,
             io=F32, ws=f(), ws_bytes=64 * MB, dy=f(), dx=f(), dz=f(), dw=f(), db=f())
    a.update(over)
    return a


def nfwd(lib, a):
    return lib.ssm_group_norm_fwd(a["x"], a["ldx"], a["z"], a["ldz"], a["w"], a["b"], a["y"], a["mean"], a["rstd"], a["batch"], a["rows"],
                                  a["dim"], a["groups"], a["eps"], a["silu"], a["io"], a["ws"], a["ws_bytes"], None)


def nbwd(lib, a):
    return lib.ssm_group_norm_bwd(a["dy"], a["x"], a["ldx"], a["z"], a["ldz"], a["w"], a["b"], a["mean"], a["rstd"], a["dx"], a["dz"],
                                  a["dw"], a["db"], a["batch"], a["rows"], a["dim"], a["groups"], a["silu"], a["io"], a["ws"],
                                  a["ws_bytes"], None)


NORM = [(dict(x=None), ENULL), (dict(io=2), EDTYPE), (dict(batch=-1), ESHAPE), (dict(rows=-1), ESHAPE), (dict(dim=0), ESHAPE),
        (dict(groups=0), ESHAPE), (dict(groups=5), ESHAPE), (dict(groups=-4), ESHAPE), (dict(dim=1 << 21, groups=1), ESHAPE),
        (dict(ldx=23), ESHAPE), (dict(ldz=8), ESHAPE), (dict(batch=1 << 60), ESHAPE), (dict(rows=1 << 50, batch=1 << 12), ESHAPE),
        (dict(x=0x7f0000000002), EALIGN), (dict(io=BF16, z=0x7f0000000001), EALIGN), (dict(w=0x7f0000000002), EALIGN),
        (dict(mean=0x7f0000000001), EALIGN), (dict(ws=None), EWS), (dict(ws_bytes=8), EWS), (dict(ws=0x7f0100000040), EALIGN)]


@pytest.mark.parametrize("over,code", NORM + [(dict(y=None), ENULL), (dict(eps=-1.0), EVALUE), (dict(eps=NAN), EVALUE),
                                              (dict(eps=INF), EVALUE)])
def test_norm_fwd_refuses(lib, over, code):
    assert nfwd(lib, norm_args(**over)) == code


@pytest.mark.parametrize("over,code", NORM + [(dict(dy=None), ENULL), (dict(dx=None), ENULL), (dict(dz=None), ENULL),
                                              (dict(mean=None), ENULL), (dict(rstd=None), ENULL), (dict(dw=0x7f0000000002), EALIGN)])
def test_norm_bwd_refuses(lib, over, code):
    assert nbwd(lib, norm_args(**over)) == code


def test_norm_overlaps_and_empty(lib):
    a = norm_args()
    for over in (dict(y=a["x"]), dict(y=a["z"] + 16), dict(mean=a["w"]), dict(rstd=a["mean"]), dict(ws=a["x"])):
        assert nfwd(lib, norm_args(**over)) == EALIAS, over
    for over in (dict(dx=a["dy"]), dict(dz=a["dx"]), dict(dw=a["w"]), dict(db=a["dw"]), dict(ws=a["dx"])):
        assert nbwd(lib, norm_args(**over)) == EALIAS, over
    assert nfwd(lib, norm_args(batch=0, x=None, y=None)) == OK
    assert nfwd(lib, norm_args(rows=0, x=None, y=None)) == OK


def test_norm_sizes(lib):
    for fn in (lib.ssm_group_norm_workspace_bytes, lib.ssm_group_norm_bwd_workspace_bytes):
        assert fn(3, 5, 24, 5) == BAD and fn(-1, 5, 24, 4) == BAD and fn(0, 5, 24, 4) == 0
        assert 0 < fn(3, 5000, 24, 4) < BAD
    for rows in (1, 5):                                                     # the groups stay in registers
        assert lib.ssm_group_norm_workspace_bytes(4096, rows, 24, 4) == 0
    assert lib.ssm_group_norm_bwd_workspace_bytes(4096, 1, 24, 4) > 0
