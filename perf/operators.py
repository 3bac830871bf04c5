"""Workloads of the mixer operators around a recurrent state: the short causal
convolution, the selective scan and the group norm with its gate.

Each case is one call: ``op`` is ``conv``, ``scan`` or ``norm``; ``pass`` is
``fwd``, ``bwd`` or ``step`` (one token a sequence, state in place).  Token
tensors are bf16 or fp32, parameters and scan states fp32.  With ``own`` the
call goes to the library; without, it is written in elementary torch
operations in fp32 (fp64 for the sums of log decays).
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64


# ---- cases ------------------------------------------------------------------------
def _conv(name, pas, dt, n, t, d, w=4, bias=True, act="silu", packed=False, state=False, lens=0):
    return {"name": name, "op": "conv", "pass": pas, "dtype": dt, "n": n, "t": t, "d": d, "w": w, "bias": bias,
            "act": act, "packed": packed, "state": state, "lens": lens}


def _scan(name, pas, dt, n, t, h, g, k, p, packed=False, state=False, softplus=True, skip=True, lens=0):
    return {"name": name, "op": "scan", "pass": pas, "dtype": dt, "n": n, "t": t, "h": h, "g": g, "k": k, "p": p,
            "packed": packed, "state": state, "softplus": softplus, "skip": skip, "lens": lens}


def _norm(name, pas, dt, rows, c, groups, act="silu", gate=True, gate_first=False, center=False, affine=True):
    return {"name": name, "op": "norm", "pass": pas, "dtype": dt, "rows": rows, "c": c, "groups": groups, "act": act,
            "gate": gate, "gate_first": gate_first, "center": center, "affine": affine}


def listed():
    return [
        # q, k and v of one 8K prompt on 32 heads of 128, convolved together
        _conv("conv prompt 8k", "fwd", "bf16", 1, 8192, 12288, bias=False),
        # gradient over packed documents of ragged lengths (x, B, C of 32 heads of 64, state 128)
        _conv("conv packed grad", "bwd", "bf16", 48, 777, 2304, packed=True, state=True, lens=1),
        # the convolution of one decode step of 256 sequences
        _conv("conv step 256", "step", "bf16", 256, 1, 2304),
        # one 8K prompt on 32 heads
        _scan("scan prompt 8k", "fwd", "bf16", 1, 8192, 32, 1, 128, 64),
        # eight 32K prompts resumed from cached states: the largest prefill
        _scan("scan prompt 32k x8", "fwd", "bf16", 8, 32768, 32, 1, 128, 64, state=True),
        # a packed batch of ragged prompts in full precision, one group a head
        _scan("scan packed fp32", "fwd", "fp32", 37, 700, 5, 5, 64, 64, packed=True, state=True, lens=2),
        # training step of an 8K sequence
        _scan("scan grad 8k", "bwd", "bf16", 1, 8192, 32, 1, 128, 64),
        # training step over packed documents, wide heads, two groups
        _scan("scan packed grad", "bwd", "bf16", 16, 901, 6, 2, 64, 128, packed=True, state=True, lens=3),
        # one decode step of 256 sequences x 32 heads, and of a single sequence
        _scan("scan step 256", "step", "bf16", 256, 1, 32, 1, 128, 64),
        _scan("scan step 1", "step", "bf16", 1, 1, 32, 1, 128, 64),
        # per-head norm and output gate of an 8K prompt, 32 heads of 128
        _norm("norm heads 8k", "fwd", "bf16", 8192, 4096, 32, act="sigmoid"),
        # gradient of the whole-row norm behind a gate, 16K tokens
        _norm("norm gate grad", "bwd", "bf16", 16384, 2048, 1, gate_first=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dt = rng.choice(["bf16", "bf16", "fp32"])
    op = rng.choice(["conv", "scan", "scan", "norm"])
    if op == "norm":
        groups = rng.choice([1, 2, 7, 8, 32])
        c = groups * (_log(rng, 8, 512) if groups > 1 else _log(rng, 33, 4096))
        if rng.random() < 0.6:
            c = -(-c // (8 * groups)) * 8 * groups
        gate = rng.random() < 0.6
        case = _norm("", rng.choice(["fwd", "bwd"]), dt, _log(rng, 1, 16384), c, groups,
                     act=rng.choice(["silu", "sigmoid"]), gate=gate, gate_first=gate and rng.random() < 0.5,
                     center=rng.random() < 0.5, affine=rng.random() < 0.8)
    else:
        pas = rng.choice(["fwd", "bwd", "step"])
        packed = pas != "step" and rng.random() < 0.5
        if pas == "step":
            n, t = _log(rng, 1, 256), 1
        elif packed:
            n, t = _log(rng, 2, 48), _log(rng, 3, 700)
        else:
            n = rng.choice([1, 1, 2, 3])
            t = _log(rng, 1, 8192 // n)
        more = {"packed": packed, "state": rng.random() < 0.5, "lens": rng.randrange(1 << 20) if packed else 0}
        if op == "conv":
            d = _log(rng, 1, 4096)
            if rng.random() < 0.6:
                d = -(-d // 64) * 64
            case = _conv("", pas, dt, n, t, d, w=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5,
                         act=rng.choice(["silu", "silu", "none"]), **more)
        else:
            g = rng.choice([1, 1, 2, 3])
            h = g * rng.randint(1, 32 // g // (2 if pas == "bwd" else 1))
            case = _scan("", pas, dt, n, t, h, g, rng.choice([64, 128]), rng.choice([64, 128]),
                         softplus=rng.random() < 0.7, skip=rng.random() < 0.7, **more)
    del case["name"]
    return case


def _lengths(case):
    """Lengths of the sequences of a packed case, from one token up to ``t``."""
    rng = random.Random(case["lens"])
    return [case["t"]] + [rng.randint(1, case["t"]) for _ in range(case["n"] - 1)]


def _tokens(case):
    if case["op"] == "norm":
        return case["rows"]
    return sum(_lengths(case)) if case["packed"] else case["n"] * case["t"]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    m = _tokens(case)
    bwd = case["pass"] == "bwd"
    if case["op"] == "norm":
        v = m * case["c"]
        tensors = 2 + case["gate"] + bwd * (1 + case["gate"])
        return {"bytes": tensors * v * e + (1 + bwd) * 8 * case["c"] * case["affine"], "flops": (30 if bwd else 12) * v}
    if case["op"] == "conv":
        v, rows = m * case["d"], case["n"] * (case["w"] - 1) * case["d"]
        states = 2 if case["pass"] == "step" else (2 * case["state"] + bwd * case["state"]) or 1
        par = case["d"] * (case["w"] + case["bias"]) * 4 * (1 + bwd)
        return {"bytes": (3 if bwd else 2) * v * e + states * rows * e + par,
                "flops": ((6 if bwd else 2) * case["w"] + 6) * v}
    h, g, k, p = case["h"], case["g"], case["k"], case["p"]
    x, bc, dts = m * h * p * e, m * g * k * e, m * h * e
    state = case["n"] * h * k * p * 4
    if bwd:
        return {"bytes": 3 * x + 4 * bc + 2 * dts + (3 if case["state"] else 0) * state,
                "flops": 10 * m * h * k * p}
    states = 2 if case["pass"] == "step" else 1 + case["state"]
    return {"bytes": 2 * x + 2 * bc + dts + states * state, "flops": 4 * m * h * k * p}


# ---- inputs -----------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(n, lo, hi):
        return torch.rand(n, generator=gen, device=dev) * (hi - lo) + lo

    s = dict(case)
    bwd, step = case["pass"] == "bwd", case["pass"] == "step"
    if case["op"] == "norm":
        shape = (case["rows"], case["c"])
        s["x"] = normal(*shape) * 2 + (0.5 if case["center"] else 0.0)
        s["z"] = normal(*shape) if case["gate"] else None
        s["weight"] = 1 + 0.1 * normal(case["c"], dtype=torch.float32) if case["affine"] else None
        s["bias"] = 0.1 * normal(case["c"], dtype=torch.float32) if case["affine"] else None
        s["d_y"] = normal(*shape) if bwd else None
        return s
    n = case["n"]
    lead = (n,) if step else (_tokens(case),) if case["packed"] else (n, case["t"])
    s["cu"] = None
    if case["packed"]:
        lens = torch.tensor([0] + _lengths(case), device=dev)
        s["cu"] = lens.cumsum(0).to(torch.int32)
    if case["op"] == "conv":
        d, w = case["d"], case["w"]
        s["x"] = normal(*lead, d)
        s["weight"] = normal(d, w, std=w ** -0.5, dtype=torch.float32)
        s["bias"] = normal(d, std=0.1, dtype=torch.float32) if case["bias"] else None
        s["state0"] = normal(n, w - 1, d) if case["state"] or step else None
        if bwd:
            s["d_y"] = normal(*lead, d)
            s["d_final"] = normal(n, w - 1, d) if case["state"] else None
        return s
    h, g, k, p = case["h"], case["g"], case["k"], case["p"]
    s["x"] = normal(*lead, h, p)
    s["B"], s["C"] = normal(*lead, g, k), normal(*lead, g, k)
    s["A"] = -uniform(h, 1.0, 16.0)
    # step sizes between 1e-3 and 1e-1 a head, varied by the token
    size = torch.exp(uniform(h, math.log(1e-3), math.log(1e-1)))
    if case["softplus"]:
        s["dt_bias"] = size + torch.log(-torch.expm1(-size))
        s["dt"] = normal(*lead, h, std=0.5)
    else:
        s["dt_bias"] = None
        s["dt"] = (size * torch.exp(normal(*lead, h, std=0.5, dtype=torch.float32))).to(dt)
    s["D"] = normal(h, dtype=torch.float32) if case["skip"] else None
    s["state0"] = normal(n, h, k, p, dtype=torch.float32) if case["state"] or step else None
    if bwd:
        s["d_y"] = normal(*lead, h, p)
        s["d_final"] = normal(n, h, k, p, dtype=torch.float32) if case["state"] else None
    return s


# ---- one pass ---------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[state["op"]](state)


def _run_own(s):
    import gated_delta_rule_66_amd as lib
    if s["op"] == "norm":
        how = {"activation": s["act"], "gate_first": s["gate_first"], "center": s["center"]}
        if s["pass"] == "fwd":
            return {"y": lib.group_norm_fwd(s["x"], s["groups"], s["weight"], s["bias"], s["z"], **how)}
        dx, dw, db, dz = lib.group_norm_bwd(s["x"], s["groups"], s["weight"], s["bias"], s["z"], s["d_y"], **how)
        return {"dx": dx, "dweight": dw, "dbias": db, "dz": dz}
    if s["op"] == "conv":
        act = None if s["act"] == "none" else s["act"]
        if s["pass"] == "step":
            y = lib.short_conv_step(s["x"], s["weight"], s["bias"], s["state0"], activation=act)
            return {"y": y, "state": s["state0"]}
        if s["pass"] == "fwd":
            y, final = lib.short_conv_fwd(s["x"], s["weight"], s["bias"], s["state0"], activation=act,
                                          cu_seqlens=s["cu"])
            return {"y": y, "state": final}
        dx, dw, db, ds = lib.short_conv_bwd(s["x"], s["weight"], s["bias"], s["d_y"], s["state0"], s["d_final"],
                                            activation=act, cu_seqlens=s["cu"], want_d_initial_state=s["state"])
        return {"dx": dx, "dweight": dw, "dbias": db, "dstate": ds}
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dt_bias"])
    if s["pass"] == "step":
        y = lib.selective_scan_step(*args, s["state0"], dt_softplus=s["softplus"])
        return {"y": y, "state": s["state0"]}
    if s["pass"] == "fwd":
        y, final = lib.selective_scan_fwd(*args, s["state0"], dt_softplus=s["softplus"], cu_seqlens=s["cu"])
        return {"y": y, "state": final}
    got = lib.selective_scan_bwd(*args, s["d_y"], s["state0"], s["d_final"], dt_softplus=s["softplus"],
                                 cu_seqlens=s["cu"], want_d_initial_state=s["state"])
    return dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dstate"), got))


# ---- plain forms ------------------------------------------------------------------
def _act(v, name):
    return v if name == "none" else torch.sigmoid(v) if name == "sigmoid" else v * torch.sigmoid(v)


def _dact(v, name):
    if name == "none":
        return torch.ones_like(v)
    sg = torch.sigmoid(v)
    return sg * (1 - sg) if name == "sigmoid" else sg * (1 + v * (1 - sg))


def _rows(s):
    """Row of the packed axis behind each place of the padded batch, and which places hold a token."""
    cu = s["cu"].long()
    at = torch.arange(s["t"], device=cu.device)
    there = at < (cu[1:] - cu[:-1])[:, None]
    return torch.where(there, cu[:-1, None] + at, 0), there


def _pad(s, v, rows):
    """[T_total, ...] as an fp32 batch [N, t, ...] with zeros behind each sequence; a regular batch as it is."""
    if rows is None:
        return v.float()
    index, there = rows
    v = v.float()[index]
    return torch.where(there.reshape(there.shape + (1,) * (v.dim() - 2)), v, 0.0)


def _unpad(v, rows, dt):
    return v.to(dt) if rows is None else v[rows[1]].to(dt)


def _plain_norm(s):
    dt, c, groups, eps = DTYPES[s["dtype"]], s["c"], s["groups"], 1e-5
    x = s["x"].float()
    z = s["z"].float() if s["gate"] else None
    u = x * _act(z, s["act"]) if s["gate_first"] else x
    u = u.view(-1, groups, c // groups)
    mid = u - u.mean(-1, keepdim=True) if s["center"] else u
    rstd = torch.rsqrt(mid.square().mean(-1, keepdim=True) + eps)
    hat = (mid * rstd).view(-1, c)
    v = hat * s["weight"] + s["bias"] if s["affine"] else hat
    outer = s["gate"] and not s["gate_first"]
    if s["pass"] == "fwd":
        return {"y": (v * _act(z, s["act"]) if outer else v if s["gate"] else _act(v, s["act"])).to(dt)}
    dy = s["d_y"].float()
    dv = dy * _act(z, s["act"]) if outer else dy if s["gate"] else dy * _dact(v, s["act"])
    dz = dy * v * _dact(z, s["act"]) if outer else None
    dw = (dv * hat).sum(0) if s["affine"] else None
    db = dv.sum(0) if s["affine"] else None
    dhat = (dv * s["weight"] if s["affine"] else dv).view(-1, groups, c // groups)
    hat = hat.view(-1, groups, c // groups)
    du = dhat - hat * (dhat * hat).mean(-1, keepdim=True)
    if s["center"]:
        du = du - dhat.mean(-1, keepdim=True)
    du = (du * rstd).view(-1, c)
    if s["gate_first"]:
        dz = du * x * _dact(z, s["act"])
        du = du * _act(z, s["act"])
    return {"dx": du.to(dt), "dweight": dw, "dbias": db, "dz": None if dz is None else dz.to(dt)}


def _plain_conv(s):
    dt, w = DTYPES[s["dtype"]], s["w"]
    weight, bias = s["weight"], s["bias"]
    if s["pass"] == "step":
        window = torch.cat([s["state0"].float(), s["x"].float()[:, None]], 1)
        pre = (window * weight.t()).sum(1) + (bias if bias is not None else 0.0)
        s["state0"].copy_(window[:, 1:])
        return {"y": _act(pre, s["act"]).to(dt), "state": s["state0"]}
    rows = _rows(s) if s["packed"] else None
    x = _pad(s, s["x"], rows)
    n, t, d = x.shape
    before = s["state0"].float() if s["state0"] is not None else x.new_zeros(n, w - 1, d)
    full = torch.cat([before, x], 1)
    window = full.unfold(1, w, 1)                       # [N, t, D, W]
    pre = (window * weight).sum(-1) + (bias if bias is not None else 0.0)
    # the last W - 1 rows of each sequence with its state before it
    ends = (s["cu"][1:] - s["cu"][:-1]).long() if s["packed"] else torch.full((n,), t, device=x.device)
    last = ends[:, None] + torch.arange(w - 1, device=x.device)
    last = last[..., None].expand(-1, -1, d)
    if s["pass"] == "fwd":
        return {"y": _unpad(_act(pre, s["act"]), rows, dt), "state": full.gather(1, last).to(dt)}
    p = _pad(s, s["d_y"], rows) * _dact(pre, s["act"])
    dfull = (torch.cat([p.new_zeros(n, w - 1, d), p, p.new_zeros(n, w - 1, d)], 1).unfold(1, w, 1)
             * weight.flip(1)).sum(-1)                  # [N, t + W - 1, D]
    if s["d_final"] is not None:
        dfull.scatter_add_(1, last, s["d_final"].float())
    return {"dx": _unpad(dfull[:, w - 1:], rows, dt), "dweight": (p[..., None] * window).sum((0, 1)),
            "dbias": p.sum((0, 1)) if bias is not None else None,
            "dstate": dfull[:, :w - 1].to(dt) if s["state"] else None}


def _softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0)


def _chunks(v, nc):
    """[N, t, ...] as [N, NC, 64, ...], zeros behind the last token."""
    short = nc * CHUNK - v.shape[1]
    if short:
        v = torch.cat([v, v.new_zeros(v.shape[0], short, *v.shape[2:])], 1)
    return v.view(v.shape[0], nc, CHUNK, *v.shape[2:])


def _plain_scan(s):
    dt, h, g, k, p = DTYPES[s["dtype"]], s["h"], s["g"], s["k"], s["p"]
    A, D = s["A"], s["D"]
    if s["pass"] == "step":
        raw = s["dt"].float() + (s["dt_bias"] if s["dt_bias"] is not None else 0.0)
        delta = _softplus(raw) if s["softplus"] else raw
        x = s["x"].float()
        Bh = s["B"].float().repeat_interleave(h // g, 1)
        Ch = s["C"].float().repeat_interleave(h // g, 1)
        st = s["state0"]
        st.mul_(torch.exp(delta * A)[..., None, None])
        st.add_((delta[..., None] * Bh)[..., None] * x[:, :, None])
        y = (st * Ch[..., None]).sum(2)
        return {"y": (y + D[:, None] * x if D is not None else y).to(dt), "state": st}
    rows = _rows(s) if s["packed"] else None
    x = _pad(s, s["x"], rows)
    n, t = x.shape[:2]
    nc = -(-t // CHUNK)
    raw = _pad(s, s["dt"], rows) + (s["dt_bias"] if s["dt_bias"] is not None else 0.0)
    delta = _softplus(raw) if s["softplus"] else raw
    if rows is not None:
        delta = torch.where(rows[1][..., None], delta, 0.0)
    # heads before tokens: [N, NC, H, 64, .]
    xs = _chunks(x, nc).transpose(2, 3)
    Bs = _chunks(_pad(s, s["B"], rows), nc).transpose(2, 3)
    Cs = _chunks(_pad(s, s["C"], rows), nc).transpose(2, 3)
    ds = _chunks(delta, nc).transpose(2, 3)             # [N, NC, H, 64]
    ca = (ds.double() * A[:, None].double()).cumsum(-1)  # log decay from the chunk's start
    tot = ca[..., -1]                                   # [N, NC, H]
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    decay = torch.where(causal, ca[..., :, None] - ca[..., None, :], -torch.inf).exp_().float()
    into = torch.exp(ca).float()[..., None]             # from the chunk's start to the token
    out = torch.exp(tot[..., None] - ca).float()[..., None]   # from the token to the chunk's end
    per = h // g
    score = (Cs @ Bs.transpose(-1, -2).contiguous()).repeat_interleave(per, 2)   # [N, NC, H, 64, 64]
    Bh, Ch = Bs.repeat_interleave(per, 2), Cs.repeat_interleave(per, 2)
    # the state before each chunk and behind the last: decays between chunks times what each chunk adds
    w = out * ds[..., None]
    adds = (Bh * w).transpose(-1, -2).contiguous() @ xs   # [N, NC, H, K, P]
    s0 = s["state0"] if s["state0"] is not None else x.new_zeros(n, h, k, p)
    upto = torch.cat([tot.new_zeros(n, 1, h), tot.cumsum(1)], 1).transpose(1, 2)    # [N, H, NC + 1]
    ones = torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril()
    between = torch.where(ones, upto[..., :, None] - upto[..., None, :], -torch.inf).exp_().float()
    adds = torch.cat([s0[:, None], adds], 1).transpose(1, 2).reshape(n, h, nc + 1, k * p)
    states = (between @ adds).view(n, h, nc + 1, k, p)
    start = states[:, :, :-1].transpose(1, 2)           # [N, NC, H, K, P]
    if s["pass"] == "fwd":
        y = (score * decay * ds[..., None, :]) @ xs + into * (Ch @ start)
        if D is not None:
            y = y + D[:, None, None] * xs
        y = y.transpose(2, 3).reshape(n, nc * CHUNK, h, p)[:, :t]
        return {"y": _unpad(y, rows, dt), "state": states[:, :, -1].contiguous()}
    dy = _chunks(_pad(s, s["d_y"], rows), nc).transpose(2, 3)
    # gradient of the state behind each chunk
    back = (Ch * into).transpose(-1, -2).contiguous() @ dy   # [N, NC, H, K, P]: what a chunk gives its start state
    dS_T = s["d_final"] if s["d_final"] is not None else x.new_zeros(n, h, k, p)
    back = torch.cat([back, dS_T[:, None]], 1).transpose(1, 2).reshape(n, h, nc + 1, k * p)
    ahead = between.transpose(-1, -2)                   # row c: decay from state c to state c' >= c
    dstates = (ahead.contiguous() @ back).view(n, h, nc + 1, k, p)
    dend = dstates[:, :, 1:].transpose(1, 2)
    dM = dy @ xs.transpose(-1, -2).contiguous()
    dG = dM * decay * ds[..., None, :]
    pairs = dM * score * decay
    U = Bh @ dend                                       # [N, NC, H, 64, P]
    V = dy @ start.transpose(-1, -2).contiguous()       # [N, NC, H, 64, K]
    dxs = (score * decay * ds[..., None, :]).transpose(-1, -2).contiguous() @ dy + w * U
    if D is not None:
        dxs = dxs + D[:, None, None] * dy
    dBh = dG.transpose(-1, -2).contiguous() @ Ch + w * (xs @ dend.transpose(-1, -2).contiguous())
    dCh = dG @ Bh + into * V
    z = (U * xs).sum(-1)                                # [N, NC, H, 64]
    wz = w[..., 0] * z
    ddelta = pairs.sum(-2) + out[..., 0] * z
    # log decay of token t: everything that passes from before t to t or later
    below = (pairs * ds[..., None, :]).tril(-1).double()
    later = (below.sum(-1) - below.sum(-2) + (into[..., 0] * (Ch * V).sum(-1)).double()).flip(-1).cumsum(-1).flip(-1)
    through = torch.exp(tot) * (start * dend).sum((-1, -2), dtype=torch.float64)
    dla = later + wz.double().cumsum(-1) - wz + through[..., None]
    ddelta = ddelta.double() + A[:, None] * dla
    raws = _chunks(raw, nc).transpose(2, 3)
    draw_ = ddelta * torch.sigmoid(raws) if s["softplus"] else ddelta

    def tokens(v):
        return _unpad(v.transpose(2, 3).reshape(n, nc * CHUNK, *v.shape[2:3], *v.shape[4:])[:, :t], rows, dt)

    there = _chunks(rows[1][..., None] if rows is not None else raw.new_ones(n, t, 1, dtype=torch.bool), nc)
    draw_ = torch.where(there.transpose(2, 3), draw_, 0.0)
    return {"dx": tokens(dxs), "ddt": tokens(draw_), "dA": (dla * ds).sum((0, 1, 3)).float(),
            "dB": tokens(dBh.view(n, nc, g, per, CHUNK, k).sum(3)), "dC": tokens(dCh.view(n, nc, g, per, CHUNK, k).sum(3)),
            "dD": (dy * xs).sum((0, 1, 3, 4)) if D is not None else None,
            "ddt_bias": draw_.sum((0, 1, 3)).float() if s["dt_bias"] is not None else None,
            "dstate": dstates[:, :, 0].contiguous() if s["state"] else None}


# ---- the definitions in 64 bits ---------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    with torch.enable_grad():
        return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](s)


def _leaf(v):
    return None if v is None else v.detach().double().requires_grad_()


def _grad(loss, leaf):
    return None if leaf is None else torch.autograd.grad(loss, leaf, retain_graph=True)[0]


def _exact_act(v, name):
    return v if name == "none" else (v if name == "silu" else 1.0) / (1 + torch.exp(-v))


def _exact_norm(s):
    x, z, w, b = (_leaf(s[k]) for k in ("x", "z", "weight", "bias"))
    u = x * _exact_act(z, s["act"]) if s["gate_first"] else x
    parts = []
    for part in u.chunk(s["groups"], -1):
        if s["center"]:
            part = part - part.sum(-1, keepdim=True) / part.shape[-1]
        parts.append(part / (part.pow(2).sum(-1, keepdim=True) / part.shape[-1] + 1e-5).sqrt())
    y = torch.cat(parts, -1)
    if w is not None:
        y = y * w + b
    if not s["gate"]:
        y = _exact_act(y, s["act"])
    elif not s["gate_first"]:
        y = y * _exact_act(z, s["act"])
    if s["pass"] == "fwd":
        return {"y": y.detach()}
    loss = (y * s["d_y"].double()).sum()
    return {"dx": _grad(loss, x), "dweight": _grad(loss, w), "dbias": _grad(loss, b), "dz": _grad(loss, z)}


def _sequences(s):
    """Slices of the tokens of each sequence in the flattened token axis."""
    lens = _lengths(s) if s["packed"] else [s["t"]] * s["n"]
    at, got = 0, []
    for n in lens:
        got.append(slice(at, at + n))
        at += n
    return got


def _exact_conv(s):
    d, w = s["d"], s["w"]
    x, weight, bias, state = (_leaf(s[k]) for k in ("x", "weight", "bias", "state0"))
    flat = x.reshape(-1, d)
    ys, finals = [], []
    for i, at in enumerate(_sequences(s) if s["pass"] != "step" else [slice(i, i + 1) for i in range(s["n"])]):
        before = state[i] if state is not None else flat.new_zeros(w - 1, d)
        seq = torch.cat([before, flat[at]])
        y = 0 if bias is None else bias
        for j in range(w):
            y = y + weight[:, j] * seq[j:len(seq) - (w - 1 - j)]
        ys.append(_exact_act(y, s["act"]))
        finals.append(seq[len(seq) - (w - 1):])
    y, final = torch.cat(ys).view(x.shape), torch.stack(finals)
    if s["pass"] != "bwd":
        return {"y": y.detach(), "state": final.detach()}
    loss = (y * s["d_y"].double()).sum()
    if s["d_final"] is not None:
        loss = loss + (final * s["d_final"].double()).sum()
    return {"dx": _grad(loss, x), "dweight": _grad(loss, weight), "dbias": _grad(loss, bias),
            "dstate": _grad(loss, state)}


def _exact_scan(s):
    """The recurrence token by token, every sequence at once; tokens behind a sequence's end change nothing."""
    h, g, k, p, n = s["h"], s["g"], s["k"], s["p"], s["n"]
    dev = s["x"].device
    step = s["pass"] == "step"
    seqs = [slice(i, i + 1) for i in range(n)] if step else _sequences(s)
    t = max(at.stop - at.start for at in seqs)
    index = torch.zeros(t, n, dtype=torch.long, device=dev)
    there = torch.zeros(t, n, dtype=torch.bool, device=dev)
    for i, at in enumerate(seqs):
        size = at.stop - at.start
        index[:size, i] = torch.arange(at.start, at.stop, device=dev)
        there[:size, i] = True

    def by_time(v, *tail):
        return v.double().reshape(-1, *tail)[index]

    x, Bt, Ct = by_time(s["x"], h, p), by_time(s["B"], g, k), by_time(s["C"], g, k)
    raw = by_time(s["dt"], h)
    if s["dt_bias"] is not None:
        raw = raw + s["dt_bias"].double()
    delta = torch.logaddexp(raw, torch.zeros_like(raw)) if s["softplus"] else raw
    delta = torch.where(there[..., None], delta, 0.0)
    A = s["A"].double()
    a = torch.exp(delta * A)
    D = s["D"].double() if s["D"] is not None else torch.zeros(h, dtype=torch.float64, device=dev)
    S = s["state0"].double() if s["state0"] is not None else torch.zeros(n, h, k, p, dtype=torch.float64, device=dev)
    S = S.view(n, g, h // g, k, p)
    xg, dg, ag = x.view(t, n, g, -1, p), delta.view(t, n, g, -1), a.view(t, n, g, -1)
    bwd = s["pass"] == "bwd"
    kept = torch.empty(t + 1, *S.shape, dtype=torch.float64, device=dev) if bwd else None
    ys = torch.empty_like(xg)
    if bwd:
        kept[0] = S
    dx_in = dg[..., None] * xg
    for i in range(t):
        S = torch.addcmul(S * ag[i][..., None, None], Bt[i][:, :, None, :, None], dx_in[i][..., None, :])
        if bwd:
            kept[i + 1] = S
        else:
            ys[i] = torch.matmul(Ct[i][:, :, None, None, :], S)[..., 0, :]

    def packed(v, like):
        flat = torch.zeros(like.numel() // v[0, 0].numel(), *v.shape[2:], dtype=torch.float64, device=dev)
        flat[index[there]] = v[there]
        return flat.view(like.shape)

    if not bwd:
        y = ys.view(t, n, h, p) + D[:, None] * x
        return {"y": packed(y, s["x"]), "state": S.reshape(n, h, k, p)}
    dy = torch.where(there[..., None, None], by_time(s["d_y"], h, p), 0.0).view(t, n, g, -1, p)
    dS = s["d_final"].double().view(S.shape) if s["d_final"] is not None else torch.zeros_like(S)
    dx, dB, dC = torch.zeros_like(xg), torch.zeros_like(Bt), torch.zeros_like(Ct)
    ddelta, dla = torch.zeros_like(dg), torch.zeros_like(dg)
    for i in reversed(range(t)):
        dS = torch.addcmul(dS, Ct[i][:, :, None, :, None], dy[i][..., None, :])
        u = torch.matmul(Bt[i][:, :, None, None, :], dS)[..., 0, :]
        dx[i] = dg[i][..., None] * u
        dB[i] = torch.matmul(dS, dx_in[i][..., None])[..., 0].sum(2)
        dC[i] = torch.matmul(kept[i + 1], dy[i][..., None])[..., 0].sum(2)
        ddelta[i] = (u * xg[i]).sum(-1)
        dS = dS * ag[i][..., None, None]
        dla[i] = (dS * kept[i]).sum((-1, -2))
    dx = dx.view(t, n, h, p) + D[:, None] * dy.view(t, n, h, p)
    dla, ddelta = dla.view(t, n, h), ddelta.view(t, n, h)
    draw_ = ddelta + A * dla
    if s["softplus"]:
        draw_ = draw_ / (1 + torch.exp(-raw))
    draw_ = torch.where(there[..., None], draw_, 0.0)
    return {"dx": packed(dx, s["x"]), "ddt": packed(draw_, s["dt"]), "dA": (dla * delta).sum((0, 1)),
            "dB": packed(dB, s["B"]), "dC": packed(dC, s["C"]),
            "dD": (dy.view(t, n, h, p) * x).sum((0, 1, 3)) if s["D"] is not None else None,
            "ddt_bias": draw_.sum((0, 1)) if s["dt_bias"] is not None else None,
            "dstate": dS.reshape(n, h, k, p) if s["state"] else None}
