"""Plain 64-bit references of the mixer operators, token by token on the CPU,
and the bounds that the tests hold the kernels to (test infrastructure)."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def seqs(n, t, cu):
    if cu is None:
        return [(i * t, (i + 1) * t) for i in range(n)]
    c = [int(v) for v in cu]
    return list(zip(c[:-1], c[1:]))


def act(v, name):
    return v if name is None else v * torch.sigmoid(v) if name == "silu" else torch.sigmoid(v)


def conv(x, weight, bias, state, ranges, activation):
    """(y, final state) of flat rows x [M, D] in float64 (differentiable)."""
    D, W = weight.shape
    y = [None] * len(ranges)
    fin = []
    for i, (a, b) in enumerate(ranges):
        before = state[i] if state is not None else x.new_zeros(W - 1, D)
        full = torch.cat([before, x[a:b]])
        c = torch.zeros(b - a, D, dtype=x.dtype) + (bias if bias is not None else 0.0)
        for w in range(W):
            c = c + weight[:, w] * full[w:w + b - a]
        y[i] = act(c, activation)
        fin.append(full[b - a:])
    return torch.cat(y) if y else x[:0], torch.stack(fin)


def scan(x, dt, A, B, C, D, dt_bias, state, ranges, softplus):
    """(y [M, H, P], final states) token by token (differentiable)."""
    M, H, P = x.shape
    G, K = B.shape[1:]
    raw = dt + dt_bias if dt_bias is not None else dt
    delta = torch.nn.functional.softplus(raw) if softplus else raw
    Bh, Ch = (t.repeat_interleave(H // G, 1) for t in (B, C))
    ys, fin = [], []
    for i, (a, b) in enumerate(ranges):
        S = state[i] if state is not None else x.new_zeros(H, K, P)
        for t in range(a, b):
            S = torch.exp(delta[t] * A)[:, None, None] * S + (delta[t][:, None] * Bh[t])[:, :, None] * x[t][:, None, :]
            y = torch.einsum("hk,hkp->hp", Ch[t], S)
            ys.append(y + D[:, None] * x[t] if D is not None else y)
        fin.append(S)
    return torch.stack(ys) if ys else x[:0], torch.stack(fin)


def norm(x, groups, weight, bias, gate, activation, gate_first, center, eps):
    u = x * act(gate, activation) if gate is not None and gate_first else x
    u = u.reshape(*x.shape[:-1], groups, x.shape[-1] // groups)
    if center:
        u = u - u.mean(-1, keepdim=True)
    n = (u / torch.sqrt(u.square().mean(-1, keepdim=True) + eps)).reshape(x.shape)
    if weight is not None:
        n = n * weight
    if bias is not None:
        n = n + bias
    if gate is None:
        return act(n, activation)
    return n if gate_first else n * act(gate, activation)


def close(got, want, bound, what):
    """|got - want| <= bound everywhere (float64)."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), "%s: over its bound by %.3g at %s (want %.6g)" % (
        what, over.max(), tuple(int(v) for v in torch.unravel_index(over.argmax(), over.shape)),
        want.flatten()[over.argmax()])
