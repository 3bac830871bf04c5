"""The mixer operators on the GPU against 64-bit references.

Bounds.  An output rounded once to its dtype is off by half a step (2^-8
relative for bf16, 2^-24 for fp32).  fp32 arithmetic inside is held to
2^-20 .. 2^-18 of the sum of absolute values of the terms it adds (a chain of n
fp32 operations is off by at most n 2^-24 of that sum; the hardware exp2 and
reciprocal by 1 ulp).  The chunked bf16 scan rounds each score (decay and step
size included) and the chunk's start state once to bf16 before its products:
2^-8 more of the sum of absolute values.  States are carried in fp32 through
exact three-way splits.
"""
import pytest
import torch

import gated_delta_rule_66_amd as kda
import mixer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]


def rnd(gen, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def up(t):
    """float64 on the CPU"""
    return None if t is None else t.detach().cpu().double()


def dev(t):
    return None if t is None else t.to(DEV)


def packed(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32)


# ---- short convolution ------------------------------------------------------------------
CONV = [
    # (n, t, lens, d, w, bias, state, act)
    (1, 1, None, 1, 2, True, True, "silu"),
    (2, 2, None, 8, 4, False, True, "silu"),
    (3, 17, None, 7, 3, True, False, None),
    (2, 130, None, 72, 4, True, True, "silu"),
    (1, 300, None, 2304, 4, False, False, "silu"),
    (0, 0, [5, 0, 1, 2, 40, 0, 33, 3], 40, 4, True, True, "silu"),
    (0, 0, [1, 1, 1, 200], 33, 3, False, True, "sigmoid"),
    (0, 0, [0, 0], 16, 4, True, True, "silu"),
    (0, 0, [97], 264, 2, True, False, "silu"),
    (0, 0, [0] * 150 + [3] + [0] * 100 + [1, 9] + [0] * 60, 24, 4, True, True, "silu"),
]


def conv_case(case, dtype, seed=0):
    n, t, lens, d, w, bias, state, act = case
    gen = torch.Generator().manual_seed(seed)
    cu = packed(lens) if lens is not None else None
    n = len(lens) if lens is not None else n
    m = sum(lens) if lens is not None else n * t
    shape = (m, d) if lens is not None else (n, t, d)
    c = {"x": rnd(gen, *shape, dtype=dtype), "w": rnd(gen, d, w), "b": rnd(gen, d) if bias else None,
         "s": rnd(gen, n, w - 1, d, dtype=dtype) if state else None, "cu": cu, "act": act,
         "dy": rnd(gen, *shape, dtype=dtype), "ds": rnd(gen, n, w - 1, d, dtype=dtype), "n": n,
         "ranges": R.seqs(n, t, cu), "shape": shape}
    return c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CONV, ids=[str(i) for i in range(len(CONV))])
def test_short_conv_forward(case, dtype):
    c = conv_case(case, dtype)
    y, fin = kda.short_conv_fwd(dev(c["x"]), dev(c["w"]), dev(c["b"]), dev(c["s"]), activation=c["act"],
                                cu_seqlens=dev(c["cu"]))
    D = c["x"].shape[-1]
    x = up(c["x"]).reshape(-1, D)
    want, wfin = R.conv(x, up(c["w"]), up(c["b"]), up(c["s"]), c["ranges"], c["act"])
    size, _ = R.conv(x.abs(), up(c["w"]).abs(), None if c["b"] is None else up(c["b"]).abs(),
                     None if c["s"] is None else up(c["s"]).abs(), c["ranges"], None)
    R.close(y.reshape(-1, D), want, R.HALF[dtype] * want.abs() + 2.0 ** -20 * (size + want.abs()), "y")
    assert torch.equal(up(fin), wfin)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", CONV, ids=[str(i) for i in range(len(CONV))])
def test_short_conv_backward(case, dtype):
    c = conv_case(case, dtype, 1)
    dx, dw, db, ds = kda.short_conv_bwd(dev(c["x"]), dev(c["w"]), dev(c["b"]), dev(c["dy"]), dev(c["s"]), dev(c["ds"]),
                                        activation=c["act"], cu_seqlens=dev(c["cu"]), want_d_initial_state=True)
    D = c["x"].shape[-1]
    zero = torch.zeros(c["n"], c["w"].shape[1] - 1, D, dtype=torch.float64)

    def grads(x, w, b, s, gy, gs, act):
        leaves = [v.requires_grad_() for v in (x, w, b, s)]
        y, fin = R.conv(x, w, b, s, c["ranges"], act)
        loss = (y * gy).sum() + (fin * gs).sum()
        return torch.autograd.grad(loss, leaves, allow_unused=True, materialize_grads=True)

    x, w = up(c["x"]).reshape(-1, D), up(c["w"])
    b = up(c["b"]) if c["b"] is not None else torch.zeros(D, dtype=torch.float64)
    s = up(c["s"]) if c["s"] is not None else zero
    dy, dsT = up(c["dy"]).reshape(-1, D), up(c["ds"])
    want = grads(x.clone(), w.clone(), b.clone(), s.clone(), dy, dsT, c["act"])
    # |act'| <= 1.1 and |act''| <= 0.5: the terms' sizes, with the error of the
    # recomputed convolution in act'
    size, _ = R.conv(x.abs(), w.abs(), b.abs(), s.abs(), c["ranges"], None)
    q = dy.abs() * (1.1 + size)
    sizes = grads(x.abs(), w.abs(), b.abs(), s.abs(), q, dsT.abs(), None)
    m = x.shape[0]
    R.close(dx.reshape(-1, D), want[0], R.HALF[dtype] * want[0].abs() + 2.0 ** -19 * sizes[0], "dx")
    R.close(dw, want[1], (2.0 ** -19 + m * 2.0 ** -24) * sizes[1], "dweight")
    if c["b"] is None:
        assert db is None
    else:
        R.close(db, want[2], (2.0 ** -19 + m * 2.0 ** -24) * sizes[2], "dbias")
    R.close(ds, want[3], R.HALF[dtype] * want[3].abs() + 2.0 ** -19 * sizes[3], "d_initial_state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,w", [(1, 2), (40, 3), (2304, 4), (33, 4)])
def test_short_conv_step_is_the_forward_token_by_token(dtype, d, w):
    gen = torch.Generator().manual_seed(2)
    n, t = 5, 6
    x, weight, bias = rnd(gen, n, t, d, dtype=dtype), rnd(gen, d, w), rnd(gen, d)
    s = rnd(gen, n, w - 1, d, dtype=dtype)
    y, fin = kda.short_conv_fwd(dev(x), dev(weight), dev(bias), dev(s))
    state = dev(s).clone()
    wide = torch.zeros(n, t, d + 8, dtype=dtype, device=DEV)
    wide[..., :d] = dev(x)
    size, _ = R.conv(up(x).reshape(-1, d).abs(), up(weight).abs(), up(bias).abs(), up(s).abs(), R.seqs(n, t, None), None)
    size = size.reshape(n, t, d)
    for i in range(t):
        # a row of a wider projection
        yi = kda.short_conv_step(wide[:, i, :d], dev(weight), dev(bias), state)
        # the same sum in another order, each rounded once
        R.close(yi, up(y[:, i]), 2 * R.HALF[dtype] * up(y[:, i]).abs() + 2.0 ** -19 * (size[:, i] + 1e-3), "step")
    assert torch.equal(state, fin)


def test_short_conv_leaves_padding_and_reads_strided_rows():
    gen = torch.Generator().manual_seed(3)
    lens, d = [9, 0, 20], 64
    cu = packed(lens)
    wide = rnd(gen, 50, 3 * d, dtype=torch.bfloat16).to(DEV)
    wide[29:] = float("nan")                       # rows behind the last sequence
    w, b = dev(rnd(gen, d, 4)), dev(rnd(gen, d))
    x = wide[:, d:2 * d]
    out = torch.full((50, d), 7.0, dtype=torch.bfloat16, device=DEV)
    y, fin = kda.short_conv_fwd(x, w, b, cu_seqlens=dev(cu), out=out)
    y2, fin2 = kda.short_conv_fwd(x[:29].contiguous(), w, b, cu_seqlens=dev(cu))
    assert torch.equal(y[:29], y2) and torch.equal(fin, fin2)
    assert (y[29:] == 7.0).all()
    dy = torch.full((50, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    dy[:29] = rnd(gen, 29, d, dtype=torch.bfloat16)
    dx = torch.full((50, d), 7.0, dtype=torch.bfloat16, device=DEV)
    got = kda.short_conv_bwd(x, w, b, dy, cu_seqlens=dev(cu), dx=dx)
    ref = kda.short_conv_bwd(x[:29].contiguous(), w, b, dy[:29].contiguous(), cu_seqlens=dev(cu))
    assert torch.equal(got[0][:29], ref[0]) and (got[0][29:] == 7.0).all()
    # the tiles of the longer axis are summed in another grouping
    assert torch.allclose(got[1], ref[1], rtol=1e-4, atol=1e-4) and torch.allclose(got[2], ref[2], rtol=1e-4, atol=1e-4)


# ---- group norm -------------------------------------------------------------------------
NORM = [
    # (rows, C, groups, act, gate, gate_first, center, affine)
    (1, 1, 1, None, False, False, False, True),
    (5, 7, 7, "silu", False, False, True, True),
    (3, 64, 1, "silu", True, False, False, True),
    (33, 4096, 32, "sigmoid", True, False, False, True),
    (17, 2048, 1, "silu", True, True, False, True),
    (9, 8192, 1, "silu", True, True, True, False),
    (4, 16384, 1, None, False, False, True, True),
    (6, 4095, 1, "silu", True, False, True, True),
    (130, 120, 5, "silu", False, False, False, False),
    (300, 264, 3, "sigmoid", True, True, True, True),
    (7, 350, 2, "silu", True, False, False, True),
    (0, 64, 2, "silu", True, False, False, True),
]


def norm_case(case, dtype, seed=0):
    rows, C, groups, act, gate, first, center, affine = case
    gen = torch.Generator().manual_seed(seed)
    return {"x": rnd(gen, rows, C, dtype=dtype, std=2.0) + 0.5, "z": rnd(gen, rows, C, dtype=dtype) if gate else None,
            "w": rnd(gen, C) if affine else None, "b": rnd(gen, C) if affine else None,
            "dy": rnd(gen, rows, C, dtype=dtype), "groups": groups,
            "how": dict(activation=act, gate_first=first, center=center, eps=1e-5)}


def norm_sizes(c):
    """hat's size: |u| and the mean it may lose, over the deviation; and the pieces."""
    x, z, g, how = up(c["x"]), up(c["z"]), c["groups"], c["how"]
    az = R.act(z, how["activation"]) if z is not None else None
    u = x * az if z is not None and how["gate_first"] else x
    ug = u.reshape(u.shape[0], g, u.shape[1] // g)
    mid = ug - ug.mean(-1, keepdim=True) if how["center"] else ug
    rstd = 1 / torch.sqrt(mid.square().mean(-1, keepdim=True) + how["eps"])
    hat = ((ug.abs() + ug.abs().mean(-1, keepdim=True)) * rstd).reshape(x.shape)
    return hat, rstd.expand(ug.shape).reshape(x.shape), az


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", NORM, ids=[str(i) for i in range(len(NORM))])
def test_group_norm_forward(case, dtype):
    c = norm_case(case, dtype)
    y = kda.group_norm_fwd(dev(c["x"]), c["groups"], dev(c["w"]), dev(c["b"]), dev(c["z"]), **c["how"])
    want = R.norm(up(c["x"]), c["groups"], up(c["w"]), up(c["b"]), up(c["z"]), **c["how"])
    hat, _, az = norm_sizes(c)
    size = hat * (up(c["w"]).abs() if c["w"] is not None else 1) + (up(c["b"]).abs() if c["b"] is not None else 0)
    if az is not None and not c["how"]["gate_first"]:
        size = size * az.abs()
    R.close(y, want, R.HALF[dtype] * want.abs() + 2.0 ** -18 * (size + want.abs()), "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", NORM, ids=[str(i) for i in range(len(NORM))])
def test_group_norm_backward(case, dtype):
    c = norm_case(case, dtype, 1)
    dx, dw, db, dz = kda.group_norm_bwd(dev(c["x"]), c["groups"], dev(c["w"]), dev(c["b"]), dev(c["z"]), dev(c["dy"]),
                                        **c["how"])
    leaves = [None if c[k] is None else up(c[k]).requires_grad_() for k in ("x", "w", "b", "z")]
    y = R.norm(leaves[0], c["groups"], leaves[1], leaves[2], leaves[3], **c["how"])
    used = [v for v in leaves if v is not None]
    got = iter(torch.autograd.grad((y * up(c["dy"])).sum(), used, allow_unused=True, materialize_grads=True))
    want = [None if v is None else next(got) for v in leaves]
    hat, rstd, az = norm_sizes(c)
    how, act = c["how"], c["how"]["activation"]
    w = up(c["w"]).abs() if c["w"] is not None else torch.ones(c["x"].shape[-1], dtype=torch.float64)
    b = up(c["b"]).abs() if c["b"] is not None else torch.zeros_like(w)
    dn = up(c["dy"]).abs()
    if az is None:
        # the activation's derivative sees the error of n: |act''| <= 0.5
        dn = dn * ((1.1 + hat * w + b) if act else 1.0)
    elif not how["gate_first"]:
        dn = dn * az.abs()
    g = (dn * w).reshape(dn.shape[0], c["groups"], dn.shape[1] // c["groups"])
    hg = hat.reshape(g.shape)
    du = (g + hg * (g * hg).mean(-1, keepdim=True) + g.mean(-1, keepdim=True)).reshape(dn.shape) * rstd
    half, rows = R.HALF[dtype], dn.shape[0]
    if az is not None and how["gate_first"]:
        R.close(dx, want[0], half * want[0].abs() + 2.0 ** -17 * du * az.abs(), "dx")
        R.close(dz, want[3], half * want[3].abs() + 2.0 ** -17 * du * up(c["x"]).abs() * 1.1, "dz")
    else:
        R.close(dx, want[0], half * want[0].abs() + 2.0 ** -17 * du, "dx")
        if az is not None:
            R.close(dz, want[3], half * want[3].abs() + 2.0 ** -17 * up(c["dy"]).abs() * (hat * w + b) * 1.1, "dz")
        else:
            assert dz is None
    if c["w"] is None:
        assert dw is None and db is None
    else:
        R.close(dw, want[1], (2.0 ** -17 + rows * 2.0 ** -24) * (dn * hat).sum(0), "dweight")
        R.close(db, want[2], (2.0 ** -17 + rows * 2.0 ** -24) * dn.sum(0), "dbias")


def test_group_norm_in_place_and_strided():
    gen = torch.Generator().manual_seed(5)
    wide = rnd(gen, 6, 5, 512, dtype=torch.bfloat16).to(DEV)
    x, z = wide[..., :256], wide[..., 256:]
    w = dev(rnd(gen, 256))
    want = kda.group_norm_fwd(x.contiguous(), 4, w, None, z.contiguous())
    assert torch.equal(kda.group_norm_fwd(x, 4, w, None, z), want)
    xc = x.contiguous()
    assert torch.equal(kda.group_norm_fwd(xc, 4, w, None, z, out=xc), want)
    with pytest.raises(kda.KDAError):
        kda.group_norm_bwd(x, 3, w, None, z, want)


# ---- selective scan ---------------------------------------------------------------------
SCAN = [
    # (n, t, lens, h, g, k, p, state, softplus, skip)
    (1, 1, None, 1, 1, 64, 64, True, True, True),
    (2, 5, None, 2, 1, 128, 64, False, True, True),
    (1, 64, None, 3, 1, 64, 128, True, False, False),
    (2, 65, None, 4, 2, 128, 128, True, True, True),
    (1, 200, None, 3, 3, 128, 64, True, True, False),
    (1, 700, None, 2, 1, 64, 64, False, False, True),
    (0, 0, [3, 0, 64, 1, 130, 0, 63], 4, 2, 64, 64, True, True, True),
    (0, 0, [1, 1, 2, 300], 2, 2, 128, 64, False, True, True),
    (0, 0, [0, 0, 0], 2, 1, 64, 128, True, True, True),
    (3, 0, None, 2, 1, 64, 64, True, True, True),
    (0, 0, [1, 0, 2] * 110, 2, 1, 64, 64, True, True, True),
]
SCAN_IDS = [str(i) for i in range(len(SCAN))]


def scan_case(case, dtype, seed=0, decay=16.0):
    n, t, lens, h, g, k, p, state, softplus, skip = case
    gen = torch.Generator().manual_seed(seed)
    cu = packed(lens) if lens is not None else None
    n = len(lens) if lens is not None else n
    lead = (sum(lens),) if lens is not None else (n, t)
    c = {"x": rnd(gen, *lead, h, p, dtype=dtype), "B": rnd(gen, *lead, g, k, dtype=dtype),
         "C": rnd(gen, *lead, g, k, dtype=dtype), "A": -torch.rand(h, generator=gen) * decay - 0.5,
         "D": rnd(gen, h) if skip else None, "s": rnd(gen, n, h, k, p) if state else None,
         "dy": rnd(gen, *lead, h, p, dtype=dtype), "ds": rnd(gen, n, h, k, p),
         "cu": cu, "n": n, "softplus": softplus, "ranges": R.seqs(n, t, cu), "lead": lead}
    if softplus:
        c["dt"], c["bias"] = rnd(gen, *lead, h, dtype=dtype), rnd(gen, h) - 3.0
    else:
        c["dt"], c["bias"] = (torch.rand(*lead, h, generator=gen) * 0.1).to(dtype), None
    return c


def scan_args(c):
    return [dev(c[k]) for k in ("x", "dt", "A", "B", "C", "D", "bias")]


def flat(c, name):
    t = up(c[name])
    return t.reshape(-1, *t.shape[len(c["lead"]):])


def scan_ref(c, size=False):
    f = (lambda v: None if v is None else v.abs()) if size else (lambda v: v)
    return R.scan(f(flat(c, "x")), flat(c, "dt"), up(c["A"]), f(flat(c, "B")), f(flat(c, "C")), f(up(c["D"])),
                  up(c["bias"]), f(up(c["s"])), c["ranges"], c["softplus"])


def check_scan(c, dtype, y, fin):
    (want, wfin), (size, sfin) = scan_ref(c), scan_ref(c, True)
    steps = max([b - a for a, b in c["ranges"]] + [0]) + 64
    chain = 2.0 ** -20 + steps * 2.0 ** -23
    scores = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    R.close(y.reshape(want.shape), want, R.HALF[dtype] * want.abs() + (scores + chain) * size, "y")
    R.close(fin, wfin, chain * sfin, "final_state")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", SCAN, ids=SCAN_IDS)
def test_selective_scan_forward(case, dtype):
    c = scan_case(case, dtype)
    y, fin = kda.selective_scan_fwd(*scan_args(c), dev(c["s"]), dt_softplus=c["softplus"], cu_seqlens=dev(c["cu"]))
    check_scan(c, dtype, y, fin)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [SCAN[3], SCAN[6]], ids=["regular", "packed"])
def test_selective_scan_strong_decay(case, dtype):
    # exponents far below the smallest float: nothing overflows, old tokens vanish
    c = scan_case(case, dtype, 4, decay=4000.0)
    y, fin = kda.selective_scan_fwd(*scan_args(c), dev(c["s"]), dt_softplus=c["softplus"], cu_seqlens=dev(c["cu"]))
    check_scan(c, dtype, y, fin)


@pytest.mark.parametrize("dtype", DTYPES)
def test_selective_scan_final_state_in_place(dtype):
    for case in (SCAN[3], (9, 300, None, 2, 1, 64, 64, True, True, True), SCAN[6]):
        c = scan_case(case, dtype, 5)
        want = kda.selective_scan_fwd(*scan_args(c), dev(c["s"]), dt_softplus=True, cu_seqlens=dev(c["cu"]))
        s = dev(c["s"]).clone()
        y, fin = kda.selective_scan_fwd(*scan_args(c), s, dt_softplus=True, cu_seqlens=dev(c["cu"]), final_state=s)
        assert fin is s and torch.equal(y, want[0]) and torch.equal(s, want[1])


def test_selective_scan_slices_padding_and_neighbours():
    # x, B, C and dt as slices of one projection; rows behind the last sequence
    # and a poisoned neighbour change nothing
    gen = torch.Generator().manual_seed(6)
    h, g, k, p, lens = 4, 2, 64, 64, [70, 3, 90]
    rows, width = 200, h * p + 2 * g * k + 8
    wide = rnd(gen, rows, width, dtype=torch.bfloat16).to(DEV)
    wide[163:] = float("nan")
    cu = dev(packed(lens))
    A, bias = dev(-torch.rand(h, generator=gen) - 0.1), dev(rnd(gen, h) - 3)

    def parts(t):
        x = t[:, :h * p].view(-1, h, p)
        B = t[:, h * p:h * p + g * k].view(-1, g, k)
        C = t[:, h * p + g * k:h * p + 2 * g * k].view(-1, g, k)
        return x, t[:, width - 8:width - 8 + h], A, B, C, None, bias

    out = torch.full((rows, h, p), 7.0, dtype=torch.bfloat16, device=DEV)
    y, fin = kda.selective_scan_fwd(*parts(wide), dt_softplus=True, cu_seqlens=cu, out=out)
    alone = [v.contiguous() if v is not None else None for v in parts(wide[:163])]
    y2, fin2 = kda.selective_scan_fwd(*alone, dt_softplus=True, cu_seqlens=cu)
    # the longer axis may be cut into other segments: states meet in another order
    assert torch.allclose(y[:163].float(), y2.float(), rtol=2 ** -7, atol=2e-2)
    assert torch.allclose(fin, fin2, rtol=1e-4, atol=1e-4)
    assert (y[163:] == 7.0).all()
    wide[71, :] = float("inf")                     # inside the second sequence
    y3, fin3 = kda.selective_scan_fwd(*parts(wide), dt_softplus=True, cu_seqlens=cu)
    assert torch.equal(y3[:70], y[:70]) and torch.equal(y3[73:163], y[73:163])
    assert torch.equal(fin3[0], fin[0]) and torch.equal(fin3[2], fin[2])
    assert not torch.isfinite(fin3[1]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,h,g,k,p", [(1, 1, 1, 64, 64), (3, 4, 2, 128, 64), (2, 6, 1, 64, 128), (70, 8, 8, 128, 128)])
def test_selective_scan_step(dtype, n, h, g, k, p):
    t = 3
    c = scan_case((n, t, None, h, g, k, p, True, True, True), dtype, 7)
    state = dev(c["s"]).clone()
    ys = []
    x, dt, A, B, C, D, bias = scan_args(c)
    for i in range(t):
        ys.append(kda.selective_scan_step(x[:, i], dt[:, i], A, B[:, i], C[:, i], D, bias, state, dt_softplus=True))
    (want, wfin), (size, sfin) = scan_ref(c), scan_ref(c, True)
    chain = 2.0 ** -20 + (k + t) * 2.0 ** -24
    y = torch.stack(ys, 1).reshape(want.shape)
    R.close(y, want, R.HALF[dtype] * want.abs() + chain * size, "y")
    R.close(state, wfin, chain * sfin, "state")


def scan_grads(c, dy, ds, size=False):
    """Gradients in 64 bits, or (size) the sums of absolute values behind them."""
    f = (lambda v: None if v is None else v.abs()) if size else (lambda v: v)
    x, B, C, D, s = (f(flat(c, "x")), f(flat(c, "B")), f(flat(c, "C")), f(up(c["D"])), f(up(c["s"])))
    if s is None:
        s = torch.zeros(c["n"], *c["ds"].shape[1:], dtype=torch.float64)
    raw = flat(c, "dt") + (up(c["bias"]) if c["bias"] is not None else 0.0)
    delta = torch.nn.functional.softplus(raw) if c["softplus"] else raw
    slope = torch.sigmoid(raw) if c["softplus"] else torch.ones_like(raw)
    la = delta * up(c["A"])                       # log decays: a leaf of their own
    leaves = [v.clone().requires_grad_() for v in (x, B, C, s, delta, la)]
    lx, lB, lC, ls, ldelta, lla = leaves
    if D is not None:
        D = D.clone().requires_grad_()
    # the recurrence with the two uses of delta apart: exp(la) and delta B x^T
    ys, fin = [], []
    H, G = x.shape[1], B.shape[1]
    Bh, Ch = (v.repeat_interleave(H // G, 1) for v in (lB, lC))
    for i, (a, b) in enumerate(c["ranges"]):
        S = ls[i]
        for t in range(a, b):
            S = torch.exp(lla[t])[:, None, None] * S + (ldelta[t][:, None] * Bh[t])[:, :, None] * lx[t][:, None, :]
            y = torch.einsum("hk,hkp->hp", Ch[t], S)
            ys.append(y + D[:, None] * lx[t] if D is not None else y)
        fin.append(S)
    loss = (torch.stack(fin) * ds).sum()
    if ys:
        loss = loss + (torch.stack(ys) * dy).sum()
    got = torch.autograd.grad(loss, leaves + ([D] if D is not None else []), allow_unused=True, materialize_grads=True)
    gx, gB, gC, gs, gdelta, gla = got[:6]
    A = up(c["A"]).abs() if size else up(c["A"])
    gd = (gdelta + A * gla) * slope
    return {"dx": gx, "ddt": gd, "dA": (gla * delta).sum(0), "dB": gB, "dC": gC,
            "dD": got[6] if D is not None else None, "ddt_bias": gd.sum(0) if c["bias"] is not None else None,
            "dstate": gs}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", SCAN, ids=SCAN_IDS)
def test_selective_scan_backward(case, dtype):
    """bf16 outputs: each term goes through at most two roundings to bf16
    (score or its gradient; state), 2 2^-8 of the sum of absolute values.  fp32
    outputs: the chunk's values are fp32 throughout; a sum over m tokens in
    fp64 adds nothing, chains over a sequence 2^-23 a step."""
    c = scan_case(case, dtype, 8)
    got = dict(zip(("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dstate"),
                   kda.selective_scan_bwd(*scan_args(c), dev(c["dy"]), dev(c["s"]), dev(c["ds"]),
                                          dt_softplus=c["softplus"], cu_seqlens=dev(c["cu"]),
                                          want_d_initial_state=True)))
    dy, ds = flat(c, "dy"), up(c["ds"])
    want, size = scan_grads(c, dy, ds), scan_grads(c, dy.abs(), ds.abs(), True)
    steps = max([b - a for a, b in c["ranges"]] + [0]) + 64
    chain = 2.0 ** -19 + steps * 2.0 ** -23
    inner = 2 * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for name in ("dx", "dB", "dC"):
        R.close(got[name].reshape(want[name].shape), want[name],
                R.HALF[dtype] * want[name].abs() + (inner + chain) * size[name], name)
    R.close(got["ddt"].reshape(want["ddt"].shape), want["ddt"],
            R.HALF[dtype] * want["ddt"].abs() + chain * size["ddt"], "ddt")
    for name in ("dA", "dD", "ddt_bias", "dstate"):
        if want[name] is None:
            assert got[name] is None
        else:
            R.close(got[name], want[name], chain * size[name], name)


def test_selective_scan_backward_against_differences():
    # a directional difference of the library's own fp32 forward
    c = scan_case((2, 90, None, 4, 2, 64, 64, True, True, True), torch.float32, 9)
    args, s, dy, ds = scan_args(c), dev(c["s"]), dev(c["dy"]), dev(c["ds"])
    grads = kda.selective_scan_bwd(*args, dy, s, ds, dt_softplus=True)
    gen = torch.Generator().manual_seed(10)
    eps = 1e-2

    def loss(*v):
        y, fin = kda.selective_scan_fwd(*v[:7], v[7], dt_softplus=True)
        return float((y.double() * dy.double()).sum() + (fin.double() * ds.double()).sum())

    order = args[:7] + [s]
    for k, (v, g) in enumerate(zip(order, (grads[0], grads[1], grads[2], grads[3], grads[4], grads[5], grads[6], grads[7]))):
        d = torch.randn(v.shape, generator=gen).to(DEV)
        d = d / d.norm() * (0.1 * v.norm())
        hi, lo = list(order), list(order)
        hi[k], lo[k] = v + eps * d, v - eps * d
        diff = (loss(*hi) - loss(*lo)) / (2 * eps)
        along = float((g.double() * d.double()).sum())
        # third-order term eps^2 / 6 of the direction, and fp32 cancellation in the loss
        scale = float((g.double() * d.double()).abs().sum()) + 1e-3 * abs(loss(*order))
        assert abs(diff - along) < 2e-3 * scale, (k, diff, along)


def test_selective_scan_backward_into_one_buffer_and_padding():
    gen = torch.Generator().manual_seed(11)
    h, g, k, p, lens = 4, 2, 64, 64, [70, 3, 90]
    rows, width = 200, h * p + 2 * g * k
    cu = dev(packed(lens))

    def data(n):
        torch.manual_seed(0)
        return [torch.randn(200, *s, device=DEV).to(torch.bfloat16)[:n].contiguous()
                for s in ((h, p), (h,), (g, k), (g, k), (h, p))]
    A, bias = dev(-torch.rand(h, generator=gen) - 0.1), dev(rnd(gen, h) - 3)
    x, dt, B, C, dy = data(rows)
    for v in (x, dt, B, C, dy):
        v[163:] = float("nan")
    buf = torch.full((rows, width), 7.0, dtype=torch.bfloat16, device=DEV)
    views = [buf[:, :h * p].view(rows, h, p), buf[:, h * p:h * p + g * k].view(rows, g, k),
             buf[:, h * p + g * k:].view(rows, g, k)]
    got = kda.selective_scan_bwd(x, dt, A, B, C, None, bias, dy, dt_softplus=True, cu_seqlens=cu, dx=views[0],
                                 dB=views[1], dC=views[2])
    x, dt, B, C, dy = data(163)
    want = kda.selective_scan_bwd(x, dt, A, B, C, None, bias, dy, dt_softplus=True, cu_seqlens=cu)
    for i in (0, 1, 3, 4):
        a, b = got[i][:163].float(), want[i].float()
        # heads may be summed in other parts: one bf16 step
        assert torch.allclose(a, b, rtol=2 ** -7, atol=2 ** -7 * float(b.abs().max()))
    for i in (2, 6):
        assert torch.allclose(got[i], want[i], rtol=1e-4, atol=1e-4 * float(want[i].abs().max()))
    assert (buf[163:] == 7.0).all()
    with pytest.raises(kda.KDAError):
        kda.selective_scan_bwd(x, dt, A, B, C, None, bias, dy, dt_softplus=True, cu_seqlens=cu,
                               dx=buf[:163, :h * p].view(163, h, p), dB=buf[:163, 64:64 + g * k].view(163, g, k))


# calls of 16, 8 and 66 chunks: segments of one, two and three chunks
SEGMENTS = [(1, 1000, None, 4, 1, 128, 64, True, True, True), (1, 500, None, 16, 2, 64, 128, False, True, True),
            (1, 4200, None, 2, 1, 64, 64, True, True, False), (0, 0, [150, 0, 257, 64, 30], 4, 2, 64, 64, True, True, True)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", SEGMENTS, ids=["one", "two", "three", "packed"])
def test_selective_scan_segments_of_short_calls(case, dtype):
    test_selective_scan_forward(case, dtype)
    test_selective_scan_backward(case, dtype)


def test_selective_scan_step_of_a_long_batch():
    # one token of long sequences: 16.8M elements between the rows of x
    gen = torch.Generator().manual_seed(12)
    n, t, h, g, k, p = 2, 65600, 4, 2, 64, 64
    r = lambda *s: rnd(gen, *s, dtype=torch.bfloat16).to(DEV)
    x = torch.zeros(n, t, h, p, dtype=torch.bfloat16, device=DEV)
    x[:, 7], dt, B, C = r(n, h, p), r(n, h), r(n, g, k), r(n, g, k)
    A, D, bias, s = dev(-torch.rand(h, generator=gen) - 0.1), dev(rnd(gen, h)), dev(rnd(gen, h)), dev(rnd(gen, n, h, k, p))
    s2 = s.clone()
    assert x[:, 7].stride(0) > 2 ** 23
    y = kda.selective_scan_step(x[:, 7], dt, A, B, C, D, bias, s, dt_softplus=True)
    y2 = kda.selective_scan_step(x[:, 7].contiguous(), dt, A, B, C, D, bias, s2, dt_softplus=True)
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_short_conv_backward_of_eight_byte_rows(dtype):
    # the backward's accesses are eight bytes: tensors that start eight bytes
    # behind a multiple of 16 take the same kernel, and so give the same bits
    c = conv_case((2, 700, None, 2304, 4, True, True, "silu"), dtype, 13)
    off = 8 // c["x"].element_size()

    def moved(t):
        buf = torch.empty(t.numel() + off, dtype=t.dtype, device=DEV)
        return buf[off:].view(t.shape).copy_(t)

    w, b = dev(c["w"]), dev(c["b"])
    want = kda.short_conv_bwd(dev(c["x"]), w, b, dev(c["dy"]), dev(c["s"]), dev(c["ds"]))
    dx = moved(torch.zeros_like(c["x"]))
    assert dx.data_ptr() % 16 == 8
    got = kda.short_conv_bwd(moved(c["x"]), w, b, moved(c["dy"]), moved(c["s"]), moved(c["ds"]), dx=dx)
    for i in range(4):
        assert torch.equal(got[i], want[i]), i
    # a width of whole eight bytes, not of 16
    test_short_conv_backward((2, 90, None, 92 if dtype == torch.bfloat16 else 90, 4, True, True, "silu"), dtype)


def test_refused_sizes_report_the_status_of_the_call():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    f = lambda *s: torch.zeros(s, device=DEV)

    def status(fn, *a, **kw):
        with pytest.raises(kda.KDAError) as e:
            fn(*a, **kw)
        return e.value.status
    unsupported, invalid = kda.kda.KDA_ERR_UNSUPPORTED, kda.kda.KDA_ERR_INVALID_ARG
    for k, p, st in ((32, 64, unsupported), (64, 96, unsupported), (64, 64, None)):
        args = (z(2, 5, 4, p), z(2, 5, 4), f(4), z(2, 5, 2, k), z(2, 5, 2, k))
        if st is not None:
            assert status(kda.selective_scan_fwd, *args) == st
            assert status(kda.selective_scan_bwd, *args, None, None, z(2, 5, 4, p)) == st
            assert status(kda.selective_scan_step, z(2, 4, p), z(2, 4), f(4), z(2, 2, k), z(2, 2, k), None, None,
                          f(2, 4, k, p)) == st
    args = (z(2, 5, 3, 64), z(2, 5, 3), f(3), z(2, 5, 2, 64), z(2, 5, 2, 64))       # groups that do not divide heads
    assert status(kda.selective_scan_fwd, *args) == invalid
    assert status(kda.selective_scan_bwd, *args, None, None, z(2, 5, 3, 64)) == invalid
    x = z(2, 5, 8)
    assert status(kda.short_conv_fwd, x, f(8, 5)) == unsupported
    assert status(kda.short_conv_bwd, x, f(8, 5), None, x) == unsupported
    wide = z(2, 32768)
    assert status(kda.group_norm_fwd, wide, 1, f(32768)) == unsupported
    assert status(kda.group_norm_bwd, wide, 1, f(32768), None, None, wide) == unsupported
    assert status(kda.group_norm_bwd, wide, 3, f(32768), None, None, wide) == invalid


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [
    (40, 130, None, 4, 1, 64, 64, True, True, True),        # many sequences a segment, some across two
    (2, 2500, None, 4, 2, 128, 64, True, True, True),       # each across many segments
    (1, 700, None, 3, 1, 64, 128, True, True, False),
    (32, 64, None, 2, 1, 64, 64, True, True, True),         # ends of sequences on ends of segments
    (0, 0, [3, 0, 700, 64, 1, 0, 190, 500, 128], 4, 2, 64, 64, True, True, True),
    (0, 0, [0] * 40 + [900] + [0] * 30, 4, 2, 64, 64, True, True, True),
], ids=["many", "long", "one", "even", "packed", "empty"])
def test_selective_scan_final_states_over_initial_ones(case, dtype):
    c = scan_case(case, dtype, 14)
    s, cu = dev(c["s"]), dev(c["cu"])
    y, fin = kda.selective_scan_fwd(*scan_args(c), s, dt_softplus=True, cu_seqlens=cu)
    both = s.clone()
    ws = torch.full((1 << 24,), 77, dtype=torch.uint8, device=DEV)
    h, p, (g, k) = c["x"].shape[-2], c["x"].shape[-1], c["B"].shape[-2:]
    t = sum(case[2]) if case[2] is not None else case[1]
    need = kda.load_library().kda_selective_scan_fwd_workspace_size(
        c["n"], int(cu is not None), t, h, g, k, p, 1 if dtype == torch.bfloat16 else 0)
    y2, fin2 = kda.selective_scan_fwd(*scan_args(c), both, dt_softplus=True, cu_seqlens=cu, final_state=both,
                                      workspace=ws[:need])
    assert fin2 is both and torch.equal(y, y2) and torch.equal(fin, fin2)
    assert (ws[need:] == 77).all()
    if c["x"].numel() < 100000:
        check_scan(c, dtype, y2, fin2)
