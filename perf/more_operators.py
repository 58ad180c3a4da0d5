"""What is measured of the gated delta rule and of the channels-last group norm, and their plain forms.

The operators: the gated delta rule (whole sequences, packed ones, its gradient,
one decode token) and the group norm with an activation or a gate (and its
gradient).  With `own` set, run() calls the library's entry points; otherwise it
computes the same in elementary torch operations, in 32 bits (the delta rule in
chunks of 64 steps).  exact() evaluates the definitions in 64 bits, the delta rule
one step after the other.
"""
import math

import torch

own = False

EPS = 1e-5                      # of the norm
CHUNK = 64                      # steps of the plain form's chunks
_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_ES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # the mixer of a 2.8b-shaped layer (5120 channels as 40 heads of 128), prefill: q, k and v are column ranges
        # of one convolution's output, two value heads to a key head
        dict(name="delta_fwd_2.8b_layer", op="delta", mode="fwd", batch=2, seqlen=8192, kheads=20, heads=40, dk=128,
             dv=128, dtype="bf16", packed=True, state=False, lens=""),
        # one long document, few heads: the state from the part before goes in and the next one out
        dict(name="delta_fwd_long", op="delta", mode="fwd", batch=1, seqlen=65536, kheads=8, heads=8, dk=64, dv=64,
             dtype="bf16", packed=False, state=True, lens=""),
        # prompts of different lengths one after the other, odd head sizes, full precision
        dict(name="delta_fwd_prompts", op="delta", mode="fwd", batch=1, seqlen=4200, kheads=4, heads=12, dk=96, dv=80,
             dtype="fp32", packed=True, state=True, lens="1,700,63,64,65,1500,7,1117,500"),
        # a training step through a 130m-shaped layer (1536 channels as 12 heads of 128): the forward and all gradients
        dict(name="delta_train_130m_layer", op="delta", mode="train", batch=8, seqlen=2048, kheads=12, heads=12, dk=128,
             dv=128, dtype="bf16", packed=True, state=False, lens=""),
        # the gradient alone in full precision, odd length, shared key heads, through the states at both ends
        dict(name="delta_bwd_odd", op="delta", mode="bwd", batch=2, seqlen=777, kheads=3, heads=6, dk=64, dv=64,
             dtype="fp32", packed=False, state=True, lens=""),
        # one token of a large decode batch
        dict(name="delta_update_decode", op="delta", mode="update", batch=128, seqlen=1, kheads=20, heads=40, dk=128,
             dv=128, dtype="bf16", packed=False, state=True, lens=""),
        # one token of one request
        dict(name="delta_update_one", op="delta", mode="update", batch=1, seqlen=1, kheads=12, heads=12, dk=128, dv=128,
             dtype="bf16", packed=False, state=True, lens=""),
        # the mixer's output norm in prefill: each token's 40 heads normalised apart and multiplied by the gate
        dict(name="norm_heads_2.8b", op="norm", mode="fwd", batch=16384, rows=1, dim=5120, groups=40, dtype="bf16",
             act="none", gate=True),
        # its gradient in training at the 130m-shaped layer
        dict(name="norm_heads_bwd_130m", op="norm", mode="bwd", batch=16384, rows=1, dim=1536, groups=12, dtype="bf16",
             act="none", gate=True),
        # a patch grid's feature maps, statistics over whole images, SiLU behind
        dict(name="norm_images", op="norm", mode="fwd", batch=16, rows=64 * 128, dim=512, groups=32, dtype="bf16",
             act="silu", gate=False),
        # the gradient at a smaller stage of odd sizes
        dict(name="norm_images_bwd", op="norm", mode="bwd", batch=12, rows=55 * 55, dim=192, groups=32, dtype="bf16",
             act="silu", gate=False),
        # one small image in full precision
        dict(name="norm_small", op="norm", mode="fwd", batch=1, rows=14 * 14, dim=96, groups=8, dtype="fp32", act="silu",
             gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "norm"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "delta":
        mode = rng.choice(["fwd", "fwd", "train", "bwd", "update"])
        kheads, group = _log(rng, 1, 20), rng.choice([1, 1, 2, 3, 4])
        dk, dv = rng.choice([(128, 128), (64, 64), (128, 64), (64, 128), (96, 96), (8 * rng.randint(2, 16), 8 * rng.randint(1, 24))])
        case = dict(op=op, mode=mode, kheads=kheads, heads=kheads * group, dk=dk, dv=dv, dtype=dtype,
                    packed=rng.random() < 0.5, state=rng.random() < 0.5, lens="")
        if mode == "update":
            while True:
                case.update(batch=_log(rng, 1, 512), seqlen=1, packed=False, state=True)
                if case["batch"] * case["heads"] * dk * dv <= (64 << 20):
                    return case
        # full precision and gradients at the smaller end: about as long a pass
        most = (16384 * 5120) // ({"fwd": 1, "train": 4, "bwd": 4}[mode] * {"bf16": 1, "fp32": 4}[dtype])
        while True:
            if rng.random() < 0.35:
                lens = [_log(rng, 1, 4096) for _ in range(rng.randint(2, 12))]
                case.update(batch=1, seqlen=sum(lens) + rng.choice([0, 3]), lens=",".join(map(str, lens)))
            else:
                case.update(batch=_log(rng, 1, 16), seqlen=_log(rng, 2, 65536), lens="")
            if case["batch"] * case["seqlen"] * case["heads"] * max(dk, dv) <= most:
                return case
    while True:
        heads = rng.random() < 0.5
        groups = _log(rng, 1, 48)
        dim = groups * (rng.choice([64, 96, 128, 256]) if heads and rng.random() < 0.7 else _log(rng, 1, 160))
        batch, rows = (_log(rng, 1, 65536), 1) if heads else (_log(rng, 1, 32), _log(rng, 2, 16384))
        if dim <= 8192 and batch * rows * dim <= (80 << 20):
            return dict(op=op, mode=rng.choice(["fwd", "bwd"]), batch=batch, rows=rows, dim=dim, groups=groups, dtype=dtype,
                        act=rng.choice(["none", "silu"]), gate=heads and rng.random() < 0.7)


def _lengths(case):
    return [int(n) for n in case["lens"].split(",")] if case["lens"] else []


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    dt = _DT[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "delta":
        B, T, Hk, H, K, V = (case[n] for n in ("batch", "seqlen", "kheads", "heads", "dk", "dv"))
        lens = _lengths(case)
        # as behind a short convolution: SiLU of normal values, queries and keys of length one
        key = lambda: torch.nn.functional.silu(normal(B, T, Hk, K))
        q, k = (t / t.norm(dim=-1, keepdim=True).clamp_min(1e-6) for t in (key(), key()))
        v = torch.nn.functional.silu(normal(B, T, H, V))
        if case["packed"]:
            all_ = torch.cat([q.flatten(2), k.flatten(2), v.flatten(2)], -1).to(dt)
            q, k, v = all_.split([Hk * K, Hk * K, H * V], -1)
            q, k, v = q.unflatten(-1, (Hk, K)), k.unflatten(-1, (Hk, K)), v.unflatten(-1, (H, V))
        else:
            q, k, v = q.to(dt), k.to(dt), v.to(dt)
        # a head's memory of 2 to 1000 steps, varied by the token; beta a sigmoid
        tau = torch.exp(uniform(H) * math.log(500.0)) * 2.0
        g = -torch.nn.functional.softplus(normal(B, T, H) + torch.log(torch.expm1(1.0 / tau)))
        beta = torch.sigmoid(normal(B, T, H))
        if case["mode"] == "update":
            q, k, v, g, beta = (t[:, 0].contiguous() for t in (q, k, v, g, beta))
        s.update(q=q, k=k, v=v, g=g.contiguous(), beta=beta.contiguous(), scale=K ** -0.5)
        n = len(lens) or B
        s["h0"] = 0.3 * normal(n, H, V, K) if case["state"] else None
        s["starts"] = None
        if lens:
            s["starts"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
        if case["mode"] in ("train", "bwd"):
            s["dout"] = normal(B, T, H, V, dtype=dt)
            s["dlast"] = normal(n, H, V, K) if case["state"] else None
        return s
    N, R, C, G = case["batch"], case["rows"], case["dim"], case["groups"]
    # channels of different means and spreads
    s["x"] = (normal(N, R, C) * (0.5 + uniform(C)) + 0.5 * normal(C)).to(dt)
    s["weight"], s["bias"] = 1.0 + 0.1 * normal(C), 0.1 * normal(C)
    s["z"] = normal(N, R, 2 * C, dtype=dt)[..., :C] if case["gate"] else None      # one half of a projection's output
    if case["mode"] == "bwd":
        s["dy"] = normal(N, R, C, dtype=dt)
        x = s["x"].double().reshape(N, R, G, C // G)
        mean = x.mean((1, 3))
        s["mean"] = mean.float()
        s["rstd"] = (1.0 / ((x - mean[:, None, :, None]).square().mean((1, 3)) + EPS).sqrt()).float()
    return s


# ------------------------------------------------------------- plain forms
def _rows_of(case):
    """For packed sequences, the rows of each, padded to equal lengths with row 0, and which are real."""
    lens = _lengths(case)
    top = max(lens)
    idx, real, at = [], [], 0
    for n in lens:
        idx.append(list(range(at, at + n)) + [0] * (top - n))
        real.append([1.0] * n + [0.0] * (top - n))
        at += n
    return torch.tensor(idx, device="cuda"), torch.tensor(real, device="cuda")


def _chunks(t, fill=0):
    """(B, T, H, ...) as (B, H, chunks, 64, ...), padded with zeros, in 32 bits."""
    B, T = t.shape[:2]
    n = -(-T // CHUNK)
    full = torch.zeros((B, n * CHUNK) + tuple(t.shape[2:]), device=t.device)
    full[:, :T] = t
    full = full.unflatten(1, (n, CHUNK))
    return full.movedim(3, 1).contiguous()


def _unchunk(t, T):
    """(B, H, chunks, 64, ...) back to (B, T, H, ...)."""
    return t.movedim(1, 3).flatten(1, 2)[:, :T]


def _delta_parts(q, k, v, g, beta, H):
    """What a chunk's products need: the decays, L = stril(K K' o Gamma), the solve's inverse, P = tril(Q K' o Gamma)."""
    group = H // q.shape[2]
    p = dict(q=_chunks(q).repeat_interleave(group, 1), k=_chunks(k).repeat_interleave(group, 1), v=_chunks(v),
             beta=_chunks(beta)[..., None])
    G = torch.cumsum(_chunks(g).double(), -1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    gam = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf"))).float()
    p["eg"], p["w"] = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    p["end"] = torch.exp(G[..., -1]).float()[..., None, None]
    p["gam"] = gam
    kt = p["k"].transpose(-1, -2).contiguous()
    p["L"] = (p["k"] @ kt * gam).tril(-1)
    p["P"] = p["q"] @ kt * gam
    N = p["L"] * p["beta"].transpose(-1, -2)
    inv = torch.eye(CHUNK, device="cuda").expand_as(N).clone()
    for i in range(1, CHUNK):
        inv[..., i, :i] = -(N[..., i:i + 1, :i] @ inv[..., :i, :i])[..., 0, :]
    p["T"] = inv
    return p


def _delta_states(p, h0):
    """R of every chunk, the state (K x V) entering each, and the one behind the last."""
    B, H, n, _, V = p["v"].shape
    S = torch.zeros(B, H, p["k"].shape[-1], V, device="cuda") if h0 is None else h0.transpose(-1, -2).contiguous()
    TV, TK = p["T"] @ p["v"], p["T"] @ (p["eg"] * p["k"])
    kw = (p["w"] * p["k"]).transpose(-1, -2).contiguous()
    Rs, Ss = torch.empty_like(p["v"]), torch.empty((B, H, n) + S.shape[2:], device="cuda")
    for c in range(n):
        Ss[:, :, c] = S
        R = TV[:, :, c] - TK[:, :, c] @ S
        Rs[:, :, c] = R
        S = p["end"][:, :, c] * S + kw[:, :, c] @ (p["beta"][:, :, c] * R)
    return Rs, Ss, S


def _delta_grads(p, Rs, Ss, last, dy, dlast, scale):
    n = Rs.shape[2]
    dS = torch.zeros_like(last) if dlast is None else dlast.transpose(-1, -2).contiguous()
    U = p["beta"] * Rs
    PtdY = scale * (p["P"].transpose(-1, -2).contiguous() @ dy)
    Tt = p["T"].transpose(-1, -2).contiguous()
    qe = scale * (p["eg"] * p["q"]).transpose(-1, -2).contiguous()
    ke = (p["eg"] * p["k"]).transpose(-1, -2).contiguous()
    dUs, dXs, dSs, dot = torch.empty_like(Rs), torch.empty_like(Rs), torch.empty_like(Ss), torch.empty_like(p["end"])
    after = last
    for c in range(n - 1, -1, -1):
        dSs[:, :, c] = dS
        dot[:, :, c] = (dS * after).sum((-1, -2), keepdim=True)
        after = Ss[:, :, c]
        dU = PtdY[:, :, c] + p["w"][:, :, c] * (p["k"][:, :, c] @ dS)
        dX = Tt[:, :, c] @ (p["beta"][:, :, c] * dU)
        dUs[:, :, c], dXs[:, :, c] = dU, dX
        dS = p["end"][:, :, c] * dS + qe[:, :, c] @ dy[:, :, c] - ke[:, :, c] @ dX
    tr = lambda t: t.transpose(-1, -2).contiguous()
    F = scale * (dy @ tr(U)) * p["gam"]
    E = (dXs @ tr(Rs)).tril(-1)
    M = -(E * p["gam"]) * tr(p["beta"])
    dq = scale * p["eg"] * (dy @ tr(Ss)) + F @ p["k"]
    write = tr(F) @ p["q"] + p["w"] * (U @ tr(dSs)) + tr(M) @ p["k"]
    erase = M @ p["k"] - p["eg"] * (dXs @ tr(Ss))
    dbeta = (Rs * dUs).sum(-1) - (p["L"] * E).sum(-2)
    dG = (p["q"] * dq).sum(-1) + (p["k"] * (erase - write)).sum(-1)
    dG[..., -1] += dot[..., 0, 0]
    dg = dG.double().flip(-1).cumsum(-1).flip(-1).float()
    return dq, write + erase, dXs, dg, dbeta, tr(dS)


def _plain_delta(s):
    case, scale, H, T = s["case"], s["scale"], s["case"]["heads"], s["case"]["seqlen"]
    dt, names = s["v"].dtype, ("q", "k", "v", "g", "beta")
    if case["mode"] == "update":
        q, k, v, g, beta = (s[n].float() for n in names)
        q, k = (t.repeat_interleave(H // t.shape[1], 1) for t in (q, k))
        S = s["h0"] * torch.exp(g)[..., None, None]
        u = beta[..., None] * (v - (S * k[:, :, None]).sum(-1))
        S = S + u[..., None] * k[:, :, None]
        s["h0"].copy_(S)
        return {"y": (scale * (S * q[:, :, None]).sum(-1)).to(dt), "state": s["h0"]}
    t = {n: s[n].float() for n in names}
    dy = s["dout"].float() if "dout" in s else None
    if case["lens"]:
        idx, real = _rows_of(case)
        spread = lambda a: a[0][idx] * real.reshape(real.shape + (1,) * (a.dim() - 2))
        t = {n: spread(a) for n, a in t.items()}
        dy = None if dy is None else spread(dy)
        valid = real.bool()

    def back(a, heads=None):
        """A chunked result as the tensors lie, in the io type or as it is."""
        a = _unchunk(a, idx.shape[1] if case["lens"] else T)
        if heads is not None:                        # shared heads: the sum over those that share one
            a = a.unflatten(2, (heads, H // heads)).sum(3)
        if case["lens"]:
            full = torch.zeros((1, T) + tuple(a.shape[2:]), device="cuda")
            full[0, :sum(_lengths(case))] = a[valid]
            a = full
        return a

    p = _delta_parts(H=H, **t)
    Rs, Ss, last = _delta_states(p, s["h0"])
    out = {}
    if case["mode"] != "bwd":
        y = scale * (p["eg"] * (p["q"] @ Ss) + p["P"] @ (p["beta"] * Rs))
        out["y"] = back(y).to(dt)
        if s["h0"] is not None:
            out["last"] = last.transpose(-1, -2).contiguous()
    if case["mode"] != "fwd":
        dq, dk, dv, dg, dbeta, dh0 = _delta_grads(p, Rs, Ss, last, _chunks(dy), s["dlast"], scale)
        Hk = case["kheads"]
        out.update(dq=back(dq, Hk).to(dt), dk=back(dk, Hk).to(dt), dv=back(dv).to(dt), dg=back(dg), dbeta=back(dbeta))
        if s["h0"] is not None:
            out["dh0"] = dh0
    return out


def _plain_norm(s):
    case = s["case"]
    N, R, C, G = case["batch"], case["rows"], case["dim"], case["groups"]
    dt, w = s["x"].dtype, s["weight"].reshape(G, C // G)
    b = s["bias"].reshape(G, C // G)
    x = s["x"].float().reshape(N, R, G, C // G)
    if case["mode"] == "fwd":
        mean = x.mean((1, 3), keepdim=True)
        rstd = torch.rsqrt((x - mean).square().mean((1, 3), keepdim=True) + EPS)
    else:
        mean, rstd = s["mean"][:, None, :, None], s["rstd"][:, None, :, None]
    n = (x - mean) * rstd
    a = n * w + b
    sa = torch.sigmoid(a) if case["act"] == "silu" else None
    val = a if sa is None else a * sa
    if s["z"] is not None:
        z = s["z"].float().reshape(x.shape)
        sz = torch.sigmoid(z)
    if case["mode"] == "fwd":
        y = val if s["z"] is None else val * (z * sz)
        return {"y": y.reshape(N, R, C).to(dt), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0]}
    dy = s["dy"].float().reshape(x.shape)
    out = {}
    da = dy
    if s["z"] is not None:
        out["dz"] = (dy * val * (sz * (1.0 + z * (1.0 - sz)))).reshape(N, R, C).to(dt)
        da = dy * (z * sz)
    if sa is not None:
        da = da * (sa * (1.0 + a * (1.0 - sa)))
    out["dweight"] = (da * n).sum((0, 1), dtype=torch.float64).float().reshape(C)
    out["dbias"] = da.sum((0, 1), dtype=torch.float64).float().reshape(C)
    wda = da * w
    dx = rstd * (wda - wda.mean((1, 3), keepdim=True) - n * (wda * n).mean((1, 3), keepdim=True))
    out["dx"] = dx.reshape(N, R, C).to(dt)
    return out


# ------------------------------------------------------ the library's calls
def _own(s):
    from selective_scan_ssm_amd import ops
    case = s["case"]
    if case["op"] == "norm":
        act = None if case["act"] == "none" else case["act"]
        if case["mode"] == "fwd":
            y, mean, rstd = ops.group_norm(s["x"], case["groups"], s["weight"], s["bias"], z=s["z"], activation=act, eps=EPS,
                                           return_stats=True)
            return {"y": y, "mean": mean, "rstd": rstd}
        got = ops.group_norm_bwd(s["dy"], s["x"], s["mean"], s["rstd"], case["groups"], s["weight"], s["bias"], z=s["z"],
                                 activation=act)
        return {k: v for k, v in got.items() if v is not None}
    args = [s[n] for n in ("q", "k", "v", "g", "beta")]
    if case["mode"] == "update":
        return {"y": ops.delta_state_update(s["h0"], *args, scale=s["scale"]), "state": s["h0"]}
    kw = dict(scale=s["scale"], h0=s["h0"], starts=s["starts"])
    out, ckpt, state = {}, None, s["h0"] is not None
    total = sum(_lengths(case)) if case["lens"] else case["seqlen"]
    if case["mode"] == "train":
        ckpt = torch.empty(ops.delta_ckpt_shape(s["q"], s["v"], s["starts"]), device=s["q"].device)
    if case["mode"] != "bwd":
        y = torch.zeros_like(s["v"], memory_format=torch.contiguous_format) if total < case["seqlen"] else None
        got = ops.delta_scan_fwd(*args, return_last_state=state, ckpt_out=ckpt, out=y, **kw)
        out.update({"y": got[0], "last": got[1]} if state else {"y": got})
    if case["mode"] != "fwd":
        got = ops.delta_scan_bwd(*args, s["dout"], dlast=s["dlast"], ckpt=ckpt, **kw)
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            if total < case["seqlen"]:
                got[name][:, total:] = 0             # rows behind the last sequence are not written
        out.update({k: v for k, v in got.items() if k != "dh0" or state})
    return out


def run(state):
    if own:
        return _own(state)
    return {"delta": _plain_delta, "norm": _plain_norm}[state["case"]["op"]](state)


def work(case):
    es = _ES[case["dtype"]]
    if case["op"] == "norm":
        n, C = case["batch"] * case["rows"] * case["dim"], case["dim"]
        z, stats = int(case["gate"]), 8 * case["batch"] * case["groups"]
        if case["mode"] == "fwd":
            return {"bytes": n * es * (2 + z) + 8 * C + stats, "flops": n * (8 + 5 * z + 5 * (case["act"] == "silu"))}
        return {"bytes": n * es * (3 + 2 * z) + 16 * C + stats, "flops": n * (18 + 12 * z + 10 * (case["act"] == "silu"))}
    K, V, H, st = case["dk"], case["dv"], case["heads"], int(case["state"])
    rows = (sum(_lengths(case)) if case["lens"] else case["seqlen"]) * case["batch"]
    ends = 4 * (len(_lengths(case)) or case["batch"]) * H * K * V
    qk, v, gb = 2 * rows * case["kheads"] * K * es, rows * H * V * es, 8 * rows * H
    if case["mode"] == "fwd" or case["mode"] == "update":
        return {"bytes": qk + 2 * v + gb + 2 * ends * st, "flops": 7 * rows * H * K * V}
    if case["mode"] == "bwd":
        return {"bytes": 2 * qk + 3 * v + 2 * gb + 3 * ends * st, "flops": 20 * rows * H * K * V}
    return {"bytes": 2 * qk + 4 * v + 2 * gb + 4 * ends * st, "flops": 22 * rows * H * K * V}


# ------------------------------------------------------------ in 64 bits
def _steps(S, q, k, v, g, beta, scale, keep=None):
    """The definition, one step after the other, on (B, T, H, ...) in 64 bits; S (B, H, V, K)."""
    ys = torch.empty_like(v)
    for t in range(v.shape[1]):
        if keep is not None:
            keep[t] = S
        kt = k[:, t, :, :, None]
        S = S * torch.exp(g[:, t])[..., None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.matmul(S, kt)[..., 0])
        S = torch.addcmul(S, u[..., None], kt.transpose(-1, -2))
        ys[:, t] = scale * torch.matmul(S, q[:, t, :, :, None])[..., 0]
    return ys, S


def _steps_back(starts, q, k, v, g, beta, scale, dy, dS):
    """The gradient, the steps in reverse, from the states that each step starts at."""
    out = [torch.empty_like(t) for t in (q, k, v, g, beta)]
    for t in range(v.shape[1] - 1, -1, -1):
        kt, qt, dyt = k[:, t, :, None], q[:, t, :, None], scale * dy[:, t, :, :, None]
        alpha = torch.exp(g[:, t])
        dec = starts[t] * alpha[..., None, None]
        r = v[:, t] - (dec * kt).sum(-1)
        u = beta[:, t, :, None] * r
        S = dec + u[..., None] * kt
        out[0][:, t] = (S * dyt).sum(-2)
        dS = dS + dyt * qt
        du = (dS * kt).sum(-1)
        dr = beta[:, t, :, None] * du
        out[1][:, t] = (dS * u[..., None]).sum(-2) - (dec * dr[..., None]).sum(-2)
        out[2][:, t] = dr
        out[4][:, t] = (du * r).sum(-1)
        dS = dS - dr[..., None] * kt
        out[3][:, t] = (dS * dec).sum((-1, -2))
        dS = dS * alpha[..., None, None]
    return out, dS


def _exact_sequence(s, at, n, h0, dlast):
    """One run of n steps from row `at` on, of every batch row."""
    case, H = s["case"], s["case"]["heads"]
    cut = lambda t: t[:, at:at + n].double()
    group = H // case["kheads"]
    q, k = (cut(s[m]).repeat_interleave(group, 2) for m in ("q", "k"))
    v, g, beta = (cut(s[m]) for m in ("v", "g", "beta"))
    S = torch.zeros(v.shape[0], H, v.shape[-1], k.shape[-1], device="cuda", dtype=torch.float64) if h0 is None else h0.double()
    out = {}
    if case["mode"] == "fwd":
        out["y"], out["last"] = _steps(S, q, k, v, g, beta, s["scale"])
        return out
    # states at every 64th step first, then block by block from the end
    block, marks, ys = 64, [], []
    for a in range(0, n, block):
        marks.append(S)
        y, S = _steps(S, *(t[:, a:a + block] for t in (q, k, v, g, beta)), s["scale"])
        ys.append(y)
    if case["mode"] == "train":
        out["y"], out["last"] = torch.cat(ys, 1), S
    dy = cut(s["dout"])
    dS = torch.zeros_like(S) if dlast is None else dlast.double()
    parts = []
    for i in range(len(marks) - 1, -1, -1):
        sl = [t[:, i * block:(i + 1) * block] for t in (q, k, v, g, beta)]
        keep = torch.empty((sl[0].shape[1],) + S.shape, device="cuda", dtype=torch.float64)
        _steps(marks[i], *sl, s["scale"], keep=keep)
        got, dS = _steps_back(keep, *sl, s["scale"], dy[:, i * block:(i + 1) * block], dS)
        parts.insert(0, got)
    for j, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        out[name] = torch.cat([p[j] for p in parts], 1)
    for name in ("dq", "dk"):
        out[name] = out[name].unflatten(2, (case["kheads"], group)).sum(3)
    out["dh0"] = dS
    return out


def _exact_delta(s):
    case, H = s["case"], s["case"]["heads"]
    if case["mode"] == "update":
        group = H // case["kheads"]
        q, k = (s[m].double().repeat_interleave(group, 1)[:, None] for m in ("q", "k"))
        v, g, beta = (s[m].double()[:, None] for m in ("v", "g", "beta"))
        y, S = _steps(s["h0"].double(), q, k, v, g, beta, s["scale"])
        return {"y": y[:, 0], "state": S}
    lens = _lengths(case)
    # about 0.25 ms a step forward, 1 ms with its gradient
    if (max(lens) if lens else case["seqlen"]) * (1 if case["mode"] == "fwd" else 4) > 70000:
        return None
    if not lens:
        out = _exact_sequence(s, 0, case["seqlen"], s["h0"], s.get("dlast"))
    else:
        runs, at = [], 0
        for i, n in enumerate(lens):
            one = lambda t: None if t is None else t[i:i + 1]
            runs.append(_exact_sequence(s, at, n, one(s["h0"]), one(s.get("dlast"))))
            at += n
        out = {}
        for name in runs[0]:
            ends = name in ("last", "dh0")
            out[name] = torch.cat([r[name] for r in runs], 0 if ends else 1)
            if not ends and at < case["seqlen"]:
                t = out[name]
                out[name] = torch.cat([t, t.new_zeros((1, case["seqlen"] - at) + tuple(t.shape[2:]))], 1)
    if s["h0"] is None:
        out.pop("last", None)
        out.pop("dh0", None)
    return out


def _exact_norm(s):
    case = s["case"]
    N, R, C, G = case["batch"], case["rows"], case["dim"], case["groups"]
    per_channel = lambda t: t.double().repeat_interleave(C // G, -1)[:, None]        # (N, G) -> (N, 1, C)
    group_mean = lambda t: t.sum(1).unflatten(-1, (G, C // G)).sum(-1) / (R * (C // G))
    x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
    if case["mode"] == "fwd":
        mean = group_mean(x)
        rstd = 1.0 / (group_mean((x - per_channel(mean)) ** 2) + EPS) ** 0.5
    else:
        mean, rstd = s["mean"], s["rstd"]
    n = (x - per_channel(mean)) * per_channel(rstd)
    a = n * w + b
    silu = lambda t: t / (1.0 + torch.exp(-t))

    def slope(t):
        e = 1.0 / (1.0 + torch.exp(-t))
        return e + t * e * (1.0 - e)

    val = silu(a) if case["act"] == "silu" else a
    z = None if s["z"] is None else s["z"].double()
    if case["mode"] == "fwd":
        return {"y": val if z is None else val * silu(z), "mean": mean, "rstd": rstd}
    da, out = s["dy"].double(), {}
    if z is not None:
        out["dz"] = da * val * slope(z)
        da = da * silu(z)
    if case["act"] == "silu":
        da = da * slope(a)
    out["dweight"], out["dbias"] = (da * n).sum((0, 1)), da.sum((0, 1))
    out["dx"] = per_channel(rstd) * (w * da - per_channel(group_mean(w * da)) - n * per_channel(group_mean(w * da * n)))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_delta(s) if case["op"] == "delta" else _exact_norm(s)
