"""The mixer operators on the GPU where a workgroup takes more than one step of
its loops: chunks behind chunks, heads behind heads, rows behind rows; and
decays far beyond a chunk's usual range.  Against 64-bit references."""
import pytest
import torch

import gated_delta_rule_66_amd as kda
import mixer_ref as R
import test_gpu_mixer as G

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = [torch.bfloat16, torch.float32]


def resets(c, seed):
    """Step sizes that clear the state every twenty tokens or so and leave it
    nearly alone between: log decays of -1e6 and of -0.2 to -1."""
    gen = torch.Generator().manual_seed(seed)
    dt = torch.rand(c["dt"].shape, generator=gen) * 0.8e-6 + 0.2e-6
    dt[torch.rand(c["dt"].shape, generator=gen) < 0.05] = 1.0
    c["A"] = torch.full_like(c["A"], -1e6)
    c["dt"] = dt.to(c["dt"].dtype)
    return c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("h,g,k,p", [(2, 1, 64, 64), (4, 2, 128, 64), (3, 1, 64, 128)])
def test_selective_scan_tokens_that_clear_the_state(dtype, h, g, k, p):
    # sums of log decays near -1e7 a chunk, of which differences of a tenth count
    c = resets(G.scan_case((1, 150, None, h, g, k, p, True, False, True), dtype, 20), 21)
    y, fin = kda.selective_scan_fwd(*G.scan_args(c), G.dev(c["s"]))
    G.check_scan(c, dtype, y, fin)


# ---- selective scan: chunks behind chunks, heads behind heads -----------------------------
# (case as in test_gpu_mixer, segments forward, segments backward, parts of a
# group's heads backward).  A workgroup walks three chunks or more of K = 64 and
# 128, of a pair of heads or of one, over boundaries of sequences inside a
# segment, and takes three heads or more of a chunk in the gradient kernel.
DEEP = {
    "pair 128x64": ((3, 500, None, 96, 8, 128, 64, True, True, True), 8, 6, 4),
    "one 128x64": ((3, 500, None, 63, 9, 128, 64, True, True, True), 8, 5, 1),
    "one 128x128": ((3, 500, None, 56, 8, 128, 128, True, True, True), 8, 5, 1),
    "pair 64x64": ((3, 500, None, 96, 8, 64, 64, False, False, True), 8, 6, 4),
    "one 64x128": ((3, 500, None, 48, 8, 64, 128, True, True, False), 8, 6, 1),
    "packed 128x64": ((0, 0, [64, 300, 1, 0, 200, 64, 256, 90, 33, 260, 257], 63, 9, 128, 64, True, True, True), 9, 5, 2),
    "packed 64x128": ((0, 0, [64, 300, 1, 0, 200, 64, 256, 90, 33, 260, 257], 48, 8, 64, 128, True, True, True), 9, 6, 2),
    "alone 128x64": ((2, 200, None, 260, 4, 128, 64, True, True, True), 1, 1, 8),
    "alone 64x128": ((2, 200, None, 260, 4, 64, 128, True, True, True), 1, 1, 8),
}


def check_plan(case, fwd_segs, bwd_segs, parts, dtype):
    """The workspaces are those of the segments and parts the case is here for,
    so that it cannot lose its purpose unseen."""
    n, t, lens, h, g, k, p = case[:7]
    if lens is not None:
        n, t = len(lens), sum(lens)
        m, chunks = t, t // 64 + n
    else:
        m, chunks = n * t, n * -(-t // 64)
    a = lambda v: -(-v // 256) * 256
    off = a(4 * (n + 1)) if lens is not None else 0
    gates, state = a(chunks * h * 5 * 64 * 4), h * k * p * 4
    segs = lambda s: a(s * state) + a(s * h * 4) if s > 1 else 0
    lib, code = kda.load_library(), 1 if dtype == torch.bfloat16 else 0
    sizes = (n, int(lens is not None), t, h, g, k, p, code)
    assert lib.kda_selective_scan_fwd_workspace_size(*sizes) == off + gates + segs(fwd_segs)
    part = a(parts * m * g * k * 4) if parts > 1 else 0
    assert lib.kda_selective_scan_bwd_workspace_size(*sizes) == \
        off + gates + 2 * segs(bwd_segs) + 2 * a(chunks * state) + a(chunks * 3 * h * 4) + 2 * part


def scan_all(c, size=False):
    """Outputs and gradients in 64 bits on the GPU, token by token, or (size) the
    sums of absolute values behind them."""
    f = (lambda v: None if v is None else v.abs()) if size else (lambda v: v)
    get = lambda name: G.flat(c, name).to(DEV)
    par = lambda name: None if c[name] is None else G.up(c[name]).to(DEV)
    x, B, C, dy = f(get("x")), f(get("B")), f(get("C")), f(get("dy"))
    D, s0, ds, A = f(par("D")), f(par("s")), f(par("ds")), par("A")
    raw = get("dt") + (par("bias") if c["bias"] is not None else 0.0)
    delta = torch.nn.functional.softplus(raw) if c["softplus"] else raw
    slope = torch.sigmoid(raw) if c["softplus"] else torch.ones_like(raw)
    a = torch.exp(delta * A)
    M, H, P = x.shape
    g, K = B.shape[1:]
    Bh, Ch = (v.repeat_interleave(H // g, 1) for v in (B, C))
    y, dx, dBh, dCh = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(Bh), torch.zeros_like(Ch)
    ddelta, dla = torch.zeros_like(delta), torch.zeros_like(delta)
    fin, dstate = [], []
    for i, (lo, hi) in enumerate(c["ranges"]):
        S = s0[i] if s0 is not None else x.new_zeros(H, K, P)
        kept = [S]
        for t in range(lo, hi):
            S = a[t][:, None, None] * S + (delta[t][:, None] * Bh[t])[:, :, None] * x[t][:, None, :]
            y[t] = (Ch[t][:, :, None] * S).sum(1)
            kept.append(S)
        fin.append(S)
        carry = ds[i]
        for t in reversed(range(lo, hi)):
            dS = carry + Ch[t][:, :, None] * dy[t][:, None, :]
            u = (Bh[t][:, :, None] * dS).sum(1)
            dx[t] = delta[t][:, None] * u
            dBh[t] = (dS * (delta[t][:, None] * x[t])[:, None, :]).sum(2)
            dCh[t] = (kept[t - lo + 1] * dy[t][:, None, :]).sum(2)
            ddelta[t] = (u * x[t]).sum(1)
            carry = a[t][:, None, None] * dS
            dla[t] = (carry * kept[t - lo]).sum((1, 2))
        dstate.append(carry)
    if D is not None:
        y, dx = y + D[:, None] * x, dx + D[:, None] * dy
    gd = (ddelta + (A.abs() if size else A) * dla) * slope
    heads = lambda v: v.view(M, g, H // g, K).sum(2)
    got = {"y": y, "fin": torch.stack(fin), "dx": dx, "ddt": gd, "dA": (dla * delta).sum(0), "dB": heads(dBh),
           "dC": heads(dCh), "dD": (dy * x).sum((0, 2)) if D is not None else None,
           "ddt_bias": gd.sum(0) if c["bias"] is not None else None, "dstate": torch.stack(dstate)}
    return {k: None if v is None else v.cpu() for k, v in got.items()}


def check_all(c, dtype):
    """Forward and gradients.  Bounds as in test_gpu_mixer, but for bf16 tokens
    each term of an output takes one operand as two bf16 (scores, states or score
    gradients: truncated to 2^-7, the rest of it rounded, 2^-9 of that): 2^-16 of
    the sum of absolute values beside the output's own rounding."""
    want, size = scan_all(c), scan_all(c, True)
    cu, how = G.dev(c["cu"]), dict(dt_softplus=c["softplus"])
    y, fin = kda.selective_scan_fwd(*G.scan_args(c), G.dev(c["s"]), cu_seqlens=cu, **how)
    names = ("dx", "ddt", "dA", "dB", "dC", "dD", "ddt_bias", "dstate")
    got = dict(zip(names, kda.selective_scan_bwd(*G.scan_args(c), G.dev(c["dy"]), G.dev(c["s"]), G.dev(c["ds"]),
                                                 cu_seqlens=cu, want_d_initial_state=True, **how)))
    steps = max([b - a for a, b in c["ranges"]] + [0]) + 64
    half, bf = R.HALF[dtype], dtype == torch.bfloat16
    chain = 2.0 ** -20 + steps * 2.0 ** -23
    R.close(y.reshape(want["y"].shape), want["y"],
            half * want["y"].abs() + ((2.0 ** -16 if bf else 0.0) + chain) * size["y"], "y")
    R.close(fin, want["fin"], chain * size["fin"], "final_state")
    chain = 2.0 ** -19 + steps * 2.0 ** -23
    for name in names:
        if want[name] is None:
            assert got[name] is None
            continue
        inner = 2.0 ** -16 if bf and name in ("dx", "dB", "dC") else 0.0
        outer = half if name in ("dx", "dB", "dC", "ddt") else 0.0
        R.close(got[name].reshape(want[name].shape), want[name],
                outer * want[name].abs() + (inner + chain) * size[name], name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", DEEP)
def test_selective_scan_of_many_chunks_and_heads_a_workgroup(name, dtype):
    case = DEEP[name][0]
    check_plan(*DEEP[name], dtype)
    check_all(G.scan_case(case, dtype, 22), dtype)


@pytest.mark.parametrize("dtype", DTYPES)
def test_selective_scan_gradients_behind_tokens_that_clear_the_state(dtype):
    check_all(resets(G.scan_case((2, 200, None, 6, 2, 64, 64, True, False, True), dtype, 23), 24), dtype)


# ---- group norm: rows behind rows -----------------------------------------------------------
ROWS = [
    # more rows than a launch has teams, forward and backward
    (2600, 2048, 1, "silu", True, True, False, True),       # a block a row
    (2600, 2048, 1, "silu", True, False, True, True),
    (600, 8192, 1, "sigmoid", True, False, True, True),     # 1024 threads; fp32 two accesses a lane
    (60000, 64, 1, "silu", False, False, True, True),       # lanes of a wave
    (20000, 256, 32, "silu", True, False, False, True),     # one lane a group (bf16)
    (700, 1500, 1, "silu", False, False, True, True),       # bf16: one channel an access, two accesses a lane
    (700, 1501, 1, None, False, False, False, True),
    (500, 4001, 1, "sigmoid", True, True, True, True),      # four accesses a lane
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ROWS, ids=["%dx%d" % c[:2] + "-%d" % i for i, c in enumerate(ROWS)])
def test_group_norm_of_many_rows_a_team(case, dtype):
    G.test_group_norm_forward(case, dtype)
    G.test_group_norm_backward(case, dtype)


# ---- short convolution: tiles behind tiles, and the longer ones ------------------------------
def conv_all(c, size=False):
    """y and the gradients of a convolution without states, in 64 bits on the
    GPU, or the sums of absolute values behind them."""
    f = (lambda v: v.abs()) if size else (lambda v: v)
    D, W = c["w"].shape
    x, w, b, dy = (f(c[k].to(DEV).double()) for k in ("x", "w", "b", "dy"))
    x, dy = x.reshape(-1, D), dy.reshape(-1, D)
    pos = torch.cat([torch.arange(hi - lo) for lo, hi in c["ranges"]]).to(DEV)
    left = torch.cat([hi - lo - 1 - torch.arange(hi - lo) for lo, hi in c["ranges"]]).to(DEV)
    lag = lambda v, j: torch.where((pos >= j)[:, None], torch.roll(v, j, 0), 0.0)
    lead = lambda v, j: torch.where((left >= j)[:, None], torch.roll(v, -j, 0), 0.0)
    pre = b + sum(w[:, W - 1 - j] * lag(x, j) for j in range(W))
    if size:
        y, q = pre, dy * (1.1 + pre)
    else:
        s = torch.sigmoid(pre)
        y, q = pre * s, dy * s * (1 + pre * (1 - s))
    dw = torch.stack([(q * lag(x, W - 1 - i)).sum(0) for i in range(W)], 1)
    dx = sum(w[:, W - 1 - j] * lead(q, j) for j in range(W))
    return [v.cpu() for v in (y, dx, dw, q.sum(0))]


def ragged(total, longest, seed):
    gen, lens = torch.Generator().manual_seed(seed), []
    while sum(lens) < total:
        lens.append(min(int(torch.randint(1, longest, (1,), generator=gen)), total - sum(lens)))
    return lens


TILES = {
    "several a thread": (3000, 3, None, 1024, 4),
    "32 rows": (2, 4100, None, 1024, 3),
    "64 rows, packed": (0, 0, ragged(16500, 700, 1), 2048, 4),
    "several of 64 rows, packed, one channel an access": (0, 0, ragged(17000, 900, 2), 4097, 4),
    "forward of 32 rows": (1, 65600, None, 1024, 2),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", TILES)
def test_short_conv_of_many_tiles(name, dtype):
    n, t, lens, d, w = TILES[name]
    if name == "several a thread":
        # blocks of four tiles: as many as the workspace has rows of sums
        code = 1 if dtype == torch.bfloat16 else 0
        need = kda.load_library().kda_short_conv_bwd_workspace_size(n, 0, t, d, w, code)
        assert need // (4 * (w + 1) * d) * 4 < n
    if name.startswith("several of 64"):
        # 64 channels and four tiles a block, 64 blocks along so many channels
        assert 2048 // -(-d // 64) <= 64 and 64 * 4 < -(-sum(lens) // 64)
    c = G.conv_case((n, t, lens, d, w, True, False, "silu"), dtype, 25)
    y, _ = kda.short_conv_fwd(G.dev(c["x"]), G.dev(c["w"]), G.dev(c["b"]), cu_seqlens=G.dev(c["cu"]))
    dx, dw, db, _ = kda.short_conv_bwd(G.dev(c["x"]), G.dev(c["w"]), G.dev(c["b"]), G.dev(c["dy"]),
                                       cu_seqlens=G.dev(c["cu"]))
    want, size = conv_all(c), conv_all(c, True)
    half, m = R.HALF[dtype], want[0].shape[0]
    R.close(y.reshape(m, d), want[0], half * want[0].abs() + 2.0 ** -20 * (size[0] + want[0].abs()), "y")
    R.close(dx.reshape(m, d), want[1], half * want[1].abs() + 2.0 ** -19 * size[1], "dx")
    R.close(dw, want[2], (2.0 ** -19 + m * 2.0 ** -24) * size[2], "dweight")
    R.close(db, want[3], (2.0 ** -19 + m * 2.0 ** -24) * size[3], "dbias")


def test_selective_scan_over_its_own_states_in_a_graph():
    # each replay continues from the states of the one before
    c = G.scan_case((3, 500, None, 8, 2, 64, 64, True, True, True), torch.bfloat16, 26)
    args, s = G.scan_args(c), G.dev(c["s"])
    own, stream = s.clone(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        kda.selective_scan_fwd(*args, s.clone(), dt_softplus=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, _ = kda.selective_scan_fwd(*args, own, dt_softplus=True, final_state=own)
    for _ in range(4):
        want, s = kda.selective_scan_fwd(*args, s, dt_softplus=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(own, s)
