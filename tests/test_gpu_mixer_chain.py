"""The mixer operators as a model uses them together, on streams, in graphs
and at sizes whose offsets pass 32 bits."""
import pytest
import torch

import gated_delta_rule_66_amd as kda
import mixer_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


def layer(seed, h=4, g=2, k=64, p=64, w=4):
    gen = torch.Generator().manual_seed(seed)
    d = h * p + 2 * g * k
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)
    return {"h": h, "g": g, "k": k, "p": p, "w": w, "d": d, "conv": r(d, w) * 0.5, "cbias": r(d) * 0.1,
            "A": -torch.rand(h, generator=gen).to(DEV) * 4 - 0.5, "D": r(h), "bias": r(h) - 3, "norm": 1 + 0.1 * r(h * p)}


def split(L, xbc):
    h, g, k, p = (L[n] for n in "hgkp")
    lead = xbc.shape[:-1]
    x, B, C = xbc.split([h * p, g * k, g * k], -1)
    return x.view(*lead, h, p), B.view(*lead, g, k), C.view(*lead, g, k)


def prompt(L, proj, conv_state=None, state=None, cu=None):
    """One layer over prompts: conv, scan on its slices, gated norm.  proj:
    [..., d + h p + h] (x B C | gate | dt)."""
    d, hp = L["d"], L["h"] * L["p"]
    u, z, dt = proj[..., :d], proj[..., d:d + hp], proj[..., d + hp:]
    c, cs = kda.short_conv_fwd(u, L["conv"], L["cbias"], conv_state, cu_seqlens=cu)
    x, B, C = split(L, c)
    y, s = kda.selective_scan_fwd(x, dt, L["A"], B, C, L["D"], L["bias"], state, dt_softplus=True, cu_seqlens=cu)
    return kda.group_norm_fwd(y.flatten(-2), L["g"], L["norm"], None, z, gate_first=True), cs, s


def token(L, proj, conv_state, state):
    d, hp = L["d"], L["h"] * L["p"]
    u, z, dt = proj[..., :d], proj[..., d:d + hp], proj[..., d + hp:]
    x, B, C = split(L, kda.short_conv_step(u, L["conv"], L["cbias"], conv_state))
    y = kda.selective_scan_step(x, dt, L["A"], B, C, L["D"], L["bias"], state, dt_softplus=True)
    return kda.group_norm_fwd(y.flatten(-2), L["g"], L["norm"], None, z, gate_first=True)


def gradients(L, proj, d_out, conv_state, state, cu):
    """The layer's backward: norm, scan (dx, dB and dC as columns of one
    buffer), convolution.  Returns d_proj and the parameters' gradients."""
    d, hp = L["d"], L["h"] * L["p"]
    u, z, dt = proj[..., :d], proj[..., d:d + hp], proj[..., d + hp:]
    c, _ = kda.short_conv_fwd(u, L["conv"], L["cbias"], conv_state, cu_seqlens=cu)
    x, B, C = split(L, c)
    y, _ = kda.selective_scan_fwd(x, dt, L["A"], B, C, L["D"], L["bias"], state, dt_softplus=True, cu_seqlens=cu)
    dy, dnorm, _, dz = kda.group_norm_bwd(y.flatten(-2), L["g"], L["norm"], None, z, d_out, gate_first=True)
    dc = torch.empty_like(c)
    vx, vB, vC = split(L, dc)
    _, ddt, dA, _, _, dD, dbias, dstate = kda.selective_scan_bwd(
        x, dt, L["A"], B, C, L["D"], L["bias"], dy.view(y.shape), state, None, dt_softplus=True, cu_seqlens=cu, dx=vx,
        dB=vB, dC=vC)
    du, dw, dcb, dconv = kda.short_conv_bwd(u, L["conv"], L["cbias"], dc, conv_state, None, cu_seqlens=cu)
    return (torch.cat([du, dz, ddt], -1), dw, dcb, dA, dD, dbias, dnorm, dconv, dstate)


def inputs(L, *lead, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(*lead, L["d"] + L["h"] * L["p"] + L["h"], generator=gen).to(dtype).to(DEV)


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 1.2e-2)])
def test_prompt_then_tokens_equals_the_whole_prompt(dtype, tol):
    # bf16: conv, scan and norm each round to half a step (2^-8), the scan's
    # scores and state once more: below 3 2^-8 = 1.2e-2 in all
    L = layer(0)
    n, t, tail = 3, 150, 5
    proj = inputs(L, n, t, dtype=dtype)
    y, cs, s = prompt(L, proj)
    y1, cs1, s1 = prompt(L, proj[:, :t - tail].contiguous())
    got = [y1]
    for i in range(t - tail, t):
        got.append(token(L, proj[:, i], cs1, s1)[:, None])
    assert rel(torch.cat(got, 1), y) < tol
    assert torch.equal(cs1, cs) and rel(s1, s) < 1e-5


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-5), (torch.bfloat16, 1.2e-2)])
def test_packed_prompts_equal_single_ones(dtype, tol):
    L = layer(1)
    lens = [65, 0, 1, 200, 64, 7]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    proj = inputs(L, sum(lens), dtype=dtype)
    y, cs, s = prompt(L, proj, cu=cu)
    at = 0
    for i, m in enumerate(lens):
        if m == 0:
            assert (cs[i] == 0).all() and (s[i] == 0).all()
            continue
        y1, cs1, s1 = prompt(L, proj[None, at:at + m])
        assert rel(y[at:at + m], y1[0]) < tol
        assert torch.equal(cs[i], cs1[0]) and rel(s[i], s1[0]) < 1e-5
        at += m


def layer_reference(L, proj, conv_state, state, ranges):
    d, hp, h, g, k, p = L["d"], L["h"] * L["p"], L["h"], L["g"], L["k"], L["p"]
    u, z, dt = proj[:, :d], proj[:, d:d + hp], proj[:, d + hp:]
    c, _ = R.conv(u, L["conv"], L["cbias"], conv_state, ranges, "silu")
    x, B, C = c[:, :hp].reshape(-1, h, p), c[:, hp:hp + g * k].reshape(-1, g, k), c[:, hp + g * k:].reshape(-1, g, k)
    y, _ = R.scan(x, dt, L["A"], B, C, L["D"], L["bias"], state, ranges, True)
    return R.norm(y.reshape(-1, hp), g, L["norm"], None, z, "silu", True, False, 1e-5)


def layer_leaves(L, proj, conv_state, state):
    D = {n: (v.detach().cpu().double().requires_grad_() if isinstance(v, torch.Tensor) else v) for n, v in L.items()}
    return D, [v.detach().cpu().double().requires_grad_() for v in (proj, conv_state, state)]


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 5e-2)])
def test_layer_gradients_over_packed_prompts(dtype, tol):
    # fp32: three operators, each within 2^-19 of its terms' absolute sums, which
    # pass a gradient's norm by less than 50 here.  bf16: six roundings to half a
    # step on the way back (c, y, dy, dc, d_proj and the scan's operands), 2^-8
    # each in the worst case and at random about a fifth of their sum: 6 2^-8 = 2.3e-2,
    # twice that where they meet the convolution's activation
    L = layer(5)
    lens = [65, 0, 3, 90]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    proj = inputs(L, sum(lens), dtype=dtype)
    gen = torch.Generator().manual_seed(6)
    cs = torch.randn(4, L["w"] - 1, L["d"], generator=gen).to(dtype).to(DEV)
    s = torch.randn(4, L["h"], L["k"], L["p"], generator=gen).to(DEV)
    d_out = torch.randn(sum(lens), L["h"] * L["p"], generator=gen).to(dtype).to(DEV)
    got = gradients(L, proj, d_out, cs, s, cu)
    D, (p64, c64, s64) = layer_leaves(L, proj, cs, s)
    y = layer_reference(D, p64, c64, s64, R.seqs(4, 0, cu.tolist()))
    leaves = [p64, D["conv"], D["cbias"], D["A"], D["D"], D["bias"], D["norm"], c64, s64]
    want = torch.autograd.grad((y * d_out.cpu().double()).sum(), leaves)
    for name, a, b in zip(("proj", "conv", "cbias", "A", "D", "bias", "norm", "conv_state", "state"), got, want):
        assert rel(a.cpu(), b) < tol, (name, rel(a.cpu(), b))


def test_backward_in_a_graph_replayed():
    L = layer(7)
    lens = [130, 70]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(DEV)
    m = sum(lens)
    proj, d_out = inputs(L, m, dtype=torch.bfloat16), inputs(L, m, dtype=torch.bfloat16, seed=1)[:, :L["h"] * L["p"]].contiguous()
    cs = torch.zeros(2, L["w"] - 1, L["d"], dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(2, L["h"], L["k"], L["p"], device=DEV)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        gradients(L, proj, d_out, cs, s, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = gradients(L, proj, d_out, cs, s, cu)
    for i in range(3):
        proj.copy_(inputs(L, m, dtype=torch.bfloat16, seed=40 + i))
        s.copy_(torch.randn(s.shape, device=DEV))
        want = gradients(L, proj, d_out, cs, s, cu)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_kda_layer_with_convolution_and_gated_norm():
    # the convolution before and the gated norm behind the KDA prefill, prompt
    # against token by token
    gen = torch.Generator().manual_seed(3)
    B, T, H, K = 2, 80, 2, 64
    D = H * K
    dt = torch.bfloat16
    r = lambda *s: torch.randn(s, generator=gen).to(DEV)
    qkv, z = r(B, T, 3 * D).to(dt), r(B, T, D).to(dt)
    g, beta = (-r(B, T, H, K).abs()).to(dt), torch.sigmoid(r(B, T, H)).to(dt)
    w, norm = r(3 * D, 4) * 0.3, 1 + 0.1 * r(D)
    c, cs = kda.short_conv_fwd(qkv, w)
    parts = [v.contiguous().view(B, T, H, K) for v in c.split(D, -1)]
    parts[0], parts[1] = (torch.nn.functional.normalize(v.float(), dim=-1).to(dt) for v in parts[:2])
    o, s = kda.chunk_fwd(*parts, g, beta)
    y = kda.group_norm_fwd(o.flatten(-2), H, norm, None, z, activation="sigmoid")
    state, conv = torch.zeros_like(s), torch.zeros_like(cs)
    for t in range(T):
        ct = kda.short_conv_step(qkv[:, t], w, None, conv)
        q, k, v = (a.contiguous().view(B, H, K) for a in ct.split(D, -1))
        q, k = (torch.nn.functional.normalize(a.float(), dim=-1).to(dt) for a in (q, k))
        ot = kda.recurrent_step(q, k, v, g[:, t].contiguous(), beta[:, t].contiguous(), state)
        yt = kda.group_norm_fwd(ot.flatten(-2), H, norm, None, z[:, t], activation="sigmoid")
        # the prefill is held to 2e-2 of the recurrence
        assert rel(yt, y[:, t]) < 3e-2
    assert torch.equal(conv, cs)


def test_calls_in_a_graph_replayed():
    L = layer(2)
    proj = inputs(L, 2, 300, dtype=torch.bfloat16)
    tok = inputs(L, 2, dtype=torch.bfloat16, seed=9)
    _, cs0, s0 = prompt(L, proj)
    stream = torch.cuda.Stream()
    cs, s = cs0.clone(), s0.clone()
    with torch.cuda.stream(stream):
        prompt(L, proj)
        token(L, tok, cs.clone(), s.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y, _, _ = prompt(L, proj)
        yt = token(L, tok, cs, s)
    for i in range(3):
        proj.copy_(inputs(L, 2, 300, dtype=torch.bfloat16, seed=20 + i))
        tok.copy_(inputs(L, 2, dtype=torch.bfloat16, seed=30 + i))
        want, _, _ = prompt(L, proj)
        c1, s1 = cs.clone(), s.clone()
        wt = token(L, tok, c1, s1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(yt, wt)
        assert torch.equal(cs, c1) and torch.equal(s, s1)


def test_two_streams_at_once():
    L = layer(4)
    a, b = (inputs(L, 1, 700, dtype=torch.bfloat16, seed=i) for i in (1, 2))
    want = prompt(L, a), prompt(L, b)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got = []
        for st, v in zip(streams, (a, b)):
            with torch.cuda.stream(st):
                got.append(prompt(L, v))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_offsets_past_32_bits():
    # 2^31 and more elements: the last rows against a call on them alone
    rows, d = 262_200, 8320
    x = torch.randn(4096, d, device=DEV).to(torch.bfloat16).repeat(65, 1)[:rows]
    assert x.numel() > 1 << 31
    w = torch.randn(d, 4, device=DEV)
    y, fin = kda.short_conv_fwd(x[None], w)
    tail = kda.short_conv_fwd(x[None, -64:], w, None, x[None, -67:-64].contiguous())
    assert torch.equal(y[0, -64:], tail[0][0]) and torch.equal(fin, tail[1])
    del y
    n = kda.group_norm_fwd(x, 65, w[:, 0].contiguous(), None, None)
    assert torch.equal(n[-64:], kda.group_norm_fwd(x[-64:].contiguous(), 65, w[:, 0].contiguous(), None, None))
    del n, x
    # a scan over 130 heads of 128 whose state reaches back less than 2048 tokens
    t, h = 131_200, 130
    x = torch.randn(2050, h, 128, device=DEV).to(torch.bfloat16).repeat(64, 1, 1)[None, :t]
    assert x.numel() > 1 << 31
    B = torch.randn(1, t, 1, 64, device=DEV).to(torch.bfloat16)
    C = torch.randn(1, t, 1, 64, device=DEV).to(torch.bfloat16)
    dt = torch.full((1, t, h), 0.05, dtype=torch.bfloat16, device=DEV)
    A = torch.full((h,), -2.0, device=DEV)
    y, fin = kda.selective_scan_fwd(x, dt, A, B, C)
    part = [v[:, -2048:].contiguous() for v in (x, dt, B, C)]
    y1, fin1 = kda.selective_scan_fwd(part[0], part[1], A, part[2], part[3])
    # e^{-0.1 * 1984} of the older state is left at the last 64 tokens
    assert rel(y[:, -64:], y1[:, -64:]) < 1e-2 and rel(fin, fin1) < 1e-5
