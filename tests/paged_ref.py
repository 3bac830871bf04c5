"""Plain 64-bit references of the paged cache operators on the CPU, and the
bounds that the tests hold the kernels to (test infrastructure)."""
import torch

LARGEST = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def spans(n, t, cu):
    """(first token row, tokens) of each sequence."""
    if cu is None:
        return [(i * t, t) for i in range(n)]
    c = [int(v) for v in cu]
    return [(a, b - a) for a, b in zip(c[:-1], c[1:])]


def quantise(x, kv):
    """(codes as float64, scale bytes) of float64 rows."""
    top = LARGEST[kv]
    most = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    most = torch.where(bad, 0.0, most)
    e = torch.frexp(most / top)[1].to(torch.int64) - 2
    for _ in range(4):          # frexp's exponent is at most one step off
        e = torch.where(torch.ldexp(torch.full_like(most, top), e) < most, e + 1, e)
    e = torch.where(most == 0, -117, e).clamp(min=-117)
    v = torch.ldexp(torch.where(bad[..., None], 0.0, x), -e[..., None])
    if kv == torch.int8:
        code = torch.round(v)
    else:
        step = torch.ldexp(torch.ones_like(v), (torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4).to(torch.int64))
        code = torch.round(v / step) * step
    return code, torch.where(bad, 255, e + 127).to(torch.uint8)


def values(cache, scale):
    """The numbers that a cache stands for, float64."""
    v = cache.cpu().to(torch.float32).double()
    if scale is None:
        return v
    b = scale.cpu().view(torch.uint8).to(torch.int64)
    p = torch.ldexp(torch.ones(b.shape, dtype=torch.float64), b - 127)
    return v * torch.where(b == 255, float("nan"), p)[..., None]


def place(table, positions, page_size, pages, seq, pos):
    """(page, row) of a position or None."""
    length = min(max(int(positions[seq]), 0), table.shape[1] * page_size)
    if pos < 0 or pos >= length:
        return None
    page = int(table[seq, pos // page_size])
    return (page, pos % page_size) if 0 <= page < pages else None


def attn(q, k, v, table, positions, ranges, scale, gate=None):
    """q [M, H, D], k and v [P, Hk, S, D] float64 values.  Returns (o, bound parts): o [M, H, D], the weighted mean of
    |v| of each output, and each (row, head)'s largest scale sum |q_d k_d|."""
    M, H, D = q.shape
    P, Hk, S, _ = k.shape
    table = table.cpu()
    o = torch.zeros(M, H, D, dtype=torch.float64)
    mean = torch.zeros_like(o)
    size = torch.zeros(M, H, 1, dtype=torch.float64)
    for i, (first, n) in enumerate(ranges):
        length = min(max(int(positions[i]), 0), table.shape[1] * S)
        at = torch.arange(length)
        pages = table[i].long()[at // S] if length else at
        there = (pages >= 0) & (pages < P)
        at, pages = at[there], pages[there]
        ki, vi = (c[pages, :, at % S].transpose(0, 1) for c in (k, v))      # [Hk, C, D]
        for t in range(n):
            m = int((at <= length - n + t).sum())
            if m == 0:
                continue
            for h in range(H):
                kk, vv = ki[h * Hk // H, :m], vi[h * Hk // H, :m]
                p = torch.softmax(kk @ q[first + t, h] * scale, 0)
                o[first + t, h] = p @ vv
                mean[first + t, h] = p @ vv.abs()
                size[first + t, h] = (kk.abs() @ q[first + t, h].abs()).amax() * scale
    if gate is not None:
        s = torch.sigmoid(gate)
        o, mean = o * s, mean * s
    return o, mean, size


def attn_wide(q, k, v, table, positions, ranges, scale, gate=None):
    """attn() of whole sequences at a time, on the tensors' own device."""
    M, H, D = q.shape
    P, Hk, S, _ = k.shape
    o, mean, size = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q[..., :1])
    for i, (first, n) in enumerate(ranges):
        if n == 0:
            continue
        length = min(max(int(positions[i]), 0), table.shape[1] * S)
        at = torch.arange(length, device=q.device)
        pages = table[i].long()[at // S]
        there = (pages >= 0) & (pages < P)
        at, pages = at[there], pages[there]
        if len(at) == 0:
            continue
        ki, vi = (c[pages, :, at % S].transpose(0, 1).contiguous() for c in (k, v))         # [Hk, C, D]
        seen = at <= (length - n + torch.arange(n, device=q.device))[:, None]               # [n, C]
        for h in range(Hk):
            rows = slice(h * H // Hk, (h + 1) * H // Hk)
            qq = q[first:first + n, rows].transpose(0, 1)                                   # [G, n, D]
            score = torch.where(seen, (qq.reshape(-1, D) @ ki[h].T).view(len(qq), n, -1) * scale, -torch.inf)
            p = torch.where(seen.any(-1)[:, None], torch.softmax(score, -1), 0.0)
            use = torch.where(seen.any(0)[:, None], vi[h], 0.0)
            clean = torch.nan_to_num(use, nan=0.0, posinf=0.0, neginf=0.0)
            got = (p.reshape(-1, len(at)) @ clean).view(len(qq), n, D)
            bad = use - clean           # NaN and infinities reach the rows that see them
            for j in torch.nonzero(~torch.isfinite(vi[h]).all(-1)).flatten().tolist():
                got = got + torch.where(seen[:, j, None] & ~torch.isfinite(bad[j]), bad[j], 0.0)
            o[first:first + n, rows] = got.transpose(0, 1)
            mean[first:first + n, rows] = (p.reshape(-1, len(at)) @ clean.abs()).view(len(qq), n, D).transpose(0, 1)
            terms = (qq.abs().reshape(-1, D) @ ki[h].abs().T).view(len(qq), n, -1)
            size[first:first + n, rows] = torch.where(seen, terms, 0.0).amax(-1, keepdim=True).transpose(0, 1) * scale
    if gate is not None:
        s = torch.sigmoid(gate)
        o, mean = o * s, mean * s
    return o, mean, size


def attn_bound(o, mean, size, dt, D, positions):
    """The output's own rounding; a weight's rounding to bf16; and in fp32, doubled because a weight stands above and
    below the fraction: scores of D products (each sum's and product's rounding relative to the sum of magnitudes),
    the exponential (its argument's rounding and its own, 2^-21), the sums over the positions, the gate."""
    fp32 = 2 * ((D + 8) * 2.0 ** -24 * size * 1.5 + 2.0 ** -21 + (positions + 64) * 2.0 ** -24) + 2.0 ** -20
    weight = 2.0 ** -8 if dt == torch.bfloat16 else 0.0
    return HALF[dt] * o.abs() + (weight + fp32) * (1 + 2.0 ** -7) * mean + 1e-30


def close(got, want, bound, what):
    """|got - want| <= bound everywhere (float64), NaN where NaN is wanted, the same infinities."""
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN at other places" % what
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), "%s: other infinities" % what
    fine = torch.isfinite(want)
    over = torch.where(fine, (got - torch.where(fine, want, 0.0)).abs() - bound, -1.0)
    if over.numel():
        assert (over <= 0).all(), "%s: over its bound by %.3g at %s (want %.6g, got %.6g)" % (
            what, over.max(), tuple(int(x) for x in torch.unravel_index(over.argmax(), over.shape)),
            want.flatten()[over.argmax()], got.flatten()[over.argmax()])


def attn_bound_two(o, mean, positions):
    """attn_bound() of cancelling(): bf16, weights as two bf16 (2^-16 of each stays out), scores that are exact.  What
    scores of up to 2 lose in fp32 on their way to a weight: the rounding of log2(e), of the maximum times it and of
    the exponent (5 x 2 x 2^-24), the same again for each of four moves of the maximum (6 x 2 x 2^-24 each), five
    exponentials (2^-23 each); then the sum over the positions, and the same of the divisor relative to o."""
    fp32 = (58 + 10 + 2 * (positions + 64)) * 2.0 ** -24
    return (HALF[torch.bfloat16] + 2.0 ** -16 + fp32) * o.abs() + (2.0 ** -16 + fp32) * (1 + 2.0 ** -7) * mean + 1e-30


def cancelling(n, t, length, H, hk, d, kv, seed):
    """n sequences of t tokens at the end of `length` positions whose outputs nearly vanish, so that their own rounding
    hides nothing of their weights': (q [n t, H, d], k and v [n length, hk, d]), exact in bf16.  Scores (scale 1) are
    products of one channel; the first position's value takes back what the others add up to, in each channel for one
    of the rows."""
    g = torch.Generator().manual_seed(seed)
    q = torch.zeros(n * t, H, d)
    q[..., 5] = torch.rand(n * t, H, generator=g) / 2 + 0.5
    q = q.to(torch.bfloat16).double()
    k = (torch.rand(n * length, hk, d, generator=g) * 4 - 2).to(torch.bfloat16).double()
    v = torch.randn(n * length, hk, d, generator=g).to(torch.bfloat16).double()
    held = k if kv not in LARGEST else values(*quantise(k, kv))
    for i in range(n):
        vi = v[i * length:(i + 1) * length]
        for h in range(hk):
            r = 0
            for c in range(d):
                tok, head = r // (H // hk), h * (H // hk) + r % (H // hk)
                m = length - t + tok + 1
                p = torch.exp(held[i * length:i * length + m, h, 5] * q[i * t + tok, head, 5])
                vi[0, h, c] = (-(p[1:] @ vi[1:m, h, c]) / p[0]).to(torch.bfloat16).double()
                r = (r + 1) % (t * (H // hk))
    return q, k, v


TWO_PARTS = [  # n, t, length, H, hk, d, page: up to 16 rows (tokens times heads a cache head) a sequence
    (2, 1, 3, 4, 4, 64, 16), (2, 1, 40, 16, 1, 64, 32), (3, 1, 130, 32, 8, 128, 64), (2, 4, 130, 8, 2, 128, 16),
    (1, 16, 70, 3, 3, 128, 256), (2, 2, 33, 14, 2, 64, 128)]
