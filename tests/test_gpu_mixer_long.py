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
    """Forward and gradients, with the bounds of test_gpu_mixer."""
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
            half * want["y"].abs() + ((2.0 ** -8 if bf else 0.0) + chain) * size["y"], "y")
    R.close(fin, want["fin"], chain * size["fin"], "final_state")
    chain = 2.0 ** -19 + steps * 2.0 ** -23
    for name in names:
        if want[name] is None:
            assert got[name] is None
            continue
        inner = 2 * 2.0 ** -8 if bf and name in ("dx", "dB", "dC") else 0.0
        outer = half if name in ("dx", "dB", "dC", "ddt") else 0.0
        R.close(got[name].reshape(want[name].shape), want[name],
                outer * want[name].abs() + (inner + chain) * size[name], name)


@pytest.mark.parametrize("dtype", DTYPES)
def test_selective_scan_gradients_behind_tokens_that_clear_the_state(dtype):
    check_all(resets(G.scan_case((2, 200, None, 6, 2, 64, 64, True, False, True), dtype, 23), 24), dtype)
