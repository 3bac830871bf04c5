"""Paged cache operators on the GPU against 64-bit references: writing, reading
back, attention of new tokens, and a run of them as a layer makes it."""
import pytest
import torch

import gated_delta_rule_66_amd as kda
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4M3, I8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int8


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Cache:
    """A pool with the tables of some sequences, its pages in random order; rows that no sequence holds are NaN."""

    def __init__(self, lens, kv, hk, d, page, seed, spare=2, blocks=None, views=False):
        g = gen(seed)
        self.kv, self.page, self.lens = kv, page, list(lens)
        held = [-(-max(n, 0) // page) for n in lens]
        self.pages = sum(held) + spare
        blocks = max(max(held, default=0), 1) if blocks is None else blocks
        order = torch.randperm(self.pages, generator=g)
        table = torch.full((len(lens), blocks), -1, dtype=torch.int32)
        used = 0
        held = [min(n, blocks) for n in held]
        for i, n in enumerate(held):
            table[i, :n] = order[used:used + n].to(torch.int32)
            used += n
        self.table = table.to(DEV)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        shape = (self.pages, hk, page, d)
        self.k_scale = self.v_scale = None
        pool = [torch.randn(shape, generator=g) for _ in range(2)]
        if kv in ref.LARGEST:
            code, byte = zip(*(ref.quantise(x.double(), kv) for x in pool))
            pool = [c.to(torch.float32) for c in code]
            self.k_scale, self.v_scale = (b.to(DEV).view(torch.float8_e8m0fnu) for b in byte)
        if views:       # views of one buffer of both, with another page's room between
            both = torch.zeros((self.pages, 3, hk, page, d), device=DEV).to(kv)
            self.k_cache, self.v_cache = both[:, 0], both[:, 2]
            self.k_cache.copy_(pool[0].to(kv))
            self.v_cache.copy_(pool[1].to(kv))
        else:
            self.k_cache, self.v_cache = (x.to(kv).to(DEV) for x in pool)
        free = torch.ones(self.pages, page, dtype=torch.bool)
        for i, n in enumerate(lens):
            for b in range(held[i]):
                free[table[i, b], :max(0, min(page, n - b * page))] = False
        self.free = free
        self.spoil(free)

    def spoil(self, where):
        """Rows [pages, page] that must not be read become NaN (int8: their scale)."""
        at = where[:, None, :].expand(-1, self.k_cache.shape[1], -1).to(DEV)
        if self.kv == I8 or self.kv == E4M3:
            for s in (self.k_scale, self.v_scale):
                s.view(torch.uint8)[at] = 255
        else:
            for c in (self.k_cache, self.v_cache):
                c.masked_fill_(at[..., None], float("nan"))

    def args(self):
        return self.k_cache, self.v_cache, self.table, self.seq_lens, self.k_scale, self.v_scale

    def values(self):
        return ref.values(self.k_cache, self.k_scale), ref.values(self.v_cache, self.v_scale)


def cu_of(new):
    return torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).to(DEV)


def check_attn(c, q, new, what, gate=None, scale=None, packed=True, **kw):
    n, t = len(new), max(new, default=0)
    cu = cu_of(new) if packed else None
    got = kda.paged_attn(q, *c.args(), gate=gate, scale=scale, cu_seqlens=cu, **kw)
    torch.cuda.synchronize()
    H, D = q.shape[-2:]
    k, v = c.values()
    flat = lambda x: None if x is None else x.reshape(-1, H, D).cpu().double()
    o, mean, size = ref.attn(flat(q), k, v, c.table, c.lens, ref.spans(n, t, cu), scale or D ** -0.5, flat(gate))
    bound = ref.attn_bound(o, mean, size, q.dtype, D, max(list(c.lens) + [1]))
    ref.close(got.reshape(o.shape), o, torch.nan_to_num(bound), what)
    return got


def rows(dt, n, h, d, seed, std=1.0):
    return (torch.randn((n, h, d), generator=gen(seed)) * std).to(dt).to(DEV)


# ---- writing and reading back ----------------------------------------------------------
KINDS = [(BF, BF), (BF, E4M3), (BF, I8), (F32, F32), (F32, E4M3), (F32, I8)]


def expect_write(c, k, v, new):
    """Caches (values as stored) and scale bytes after a write, on the CPU."""
    table, out = c.table.cpu(), []
    for x, cache, scale in ((k, c.k_cache, c.k_scale), (v, c.v_cache, c.v_scale)):
        want = cache.cpu().to(torch.float32).double()
        byte = None if scale is None else scale.cpu().view(torch.uint8).clone()
        code, b = (x.double().cpu(), None) if scale is None else ref.quantise(x.double().cpu(), c.kv)
        for i, (first, n) in enumerate(ref.spans(len(new), 0, cu_of(new))):
            length = min(max(c.lens[i], 0), table.shape[1] * c.page)
            for t in range(n):
                at = ref.place(table, c.lens, c.page, c.pages, i, length - n + t)
                if at is None:
                    continue
                want[at[0], :, at[1]] = code[first + t]
                if byte is not None:
                    byte[at[0], :, at[1]] = b[first + t]
        out.append((want, byte))
    return out


def check_write(c, k, v, new, packed=True):
    want = expect_write(c, k.reshape(-1, *k.shape[-2:]), v.reshape(-1, *v.shape[-2:]), new)
    kda.kv_cache_write(k, v, *c.args(), cu_seqlens=cu_of(new) if packed else None)
    torch.cuda.synchronize()
    for name, cache, scale, (w, b) in (("k", c.k_cache, c.k_scale, want[0]), ("v", c.v_cache, c.v_scale, want[1])):
        got = cache.cpu().to(torch.float32).double()
        assert torch.equal(torch.nan_to_num(got, nan=-1e9), torch.nan_to_num(w, nan=-1e9)), name
        if b is not None:
            assert torch.equal(scale.cpu().view(torch.uint8), b), name


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("d,hk,page", [(64, 3, 16), (128, 2, 64), (128, 5, 256), (64, 1, 32)])
def test_write_packed(dt, kv, d, hk, page):
    new = [1, 37, 0, page + 3, 5]
    c = Cache([40, 37, 9, page + 3, 2 * page + 1], kv, hk, d, page, seed=1, views=d == 128)
    m = sum(new)
    k, v = rows(dt, m + 3, hk, d, 2), rows(dt, m + 3, hk, d, 3, std=30.0)
    check_write(c, k, v, new)           # three rows behind the last sequence


@pytest.mark.parametrize("dt,kv", KINDS)
def test_write_regular_slices_and_places_that_are_not_there(dt, kv):
    d, hk, page, t = 128, 2, 16, 20
    c = Cache([100, 7, 0, 33, -4], kv, hk, d, page, seed=4, blocks=6)       # 100 > 6 * 16 is clamped
    c.table[3, 1] = -1
    c.table[0, 5] = c.pages
    wide = rows(dt, 5 * t, 3 * hk, d, 5).view(5, t, 3 * hk, d)
    check_write(c, wide[:, :, hk:2 * hk], wide[:, :, 2 * hk:], [t] * 5, packed=False)


@pytest.mark.parametrize("kv", [E4M3, I8])
def test_write_every_bf16_value(kv):
    """Every finite bf16 magnitude, against largest values of some fractions; and rows of zeros, NaN, infinities."""
    d, page = 128, 256
    bits = torch.arange(0x7f00, dtype=torch.int32)      # below 2^127
    x = (bits << 16).view(torch.float32)
    x = torch.where(bits % 3 == 0, -x, x).view(-1, d)
    # rows of neighbouring magnitudes, and the same rows beside a value up to 2^9 times larger
    big = torch.cat([x * f for f in (1.0, 3.0, 100.0)])
    mixed = x.repeat(3, 1)
    mixed[:, 0] = big.abs().amax(-1).clamp(max=1.6e38)
    x = torch.cat([x, mixed, torch.zeros(1, d), torch.full((1, d), float("nan")), torch.full((1, d), float("inf"))]).to(BF)
    special = torch.randn(3, d, generator=gen(6)).to(BF)
    special[0, 5], special[1, 127], special[2, 0] = float("nan"), float("inf"), -float("inf")
    x = torch.cat([x, special])
    m = x.shape[0]
    c = Cache([m], kv, 1, d, page, seed=7)
    x = x.to(DEV).view(m, 1, d)
    check_write(c, x, x.flip(0).contiguous(), [m])
    k, v = kda.kv_cache_read(*c.args(), m, cu_seqlens=cu_of([m]))
    code, byte = ref.quantise(x.double().cpu(), kv)
    want = ref.values(code, byte)
    assert torch.equal(torch.nan_to_num(k.cpu().double(), nan=-1.0), torch.nan_to_num(want, nan=-1.0))
    assert torch.equal(torch.nan_to_num(v.cpu().double(), nan=-1.0), torch.nan_to_num(want.flip(0), nan=-1.0))


@pytest.mark.parametrize("kv", [E4M3, I8])
def test_write_fp32_near_the_borders(kv):
    """fp32 values one step to either side of a border between codes, and of a power of the scale."""
    top, d = ref.LARGEST[kv], 64
    r = torch.randint(0, 127, (400, d), generator=gen(8)).float() + 0.5
    x = torch.cat([r, torch.nextafter(r, torch.zeros(())), torch.nextafter(r, torch.full((), 1e9))])
    x[:, 0] = top
    x[::3, 0] = torch.nextafter(torch.tensor(top), torch.tensor(1e9))
    x[1::3, 0] = torch.nextafter(torch.tensor(top), torch.tensor(0.0))
    x *= torch.ldexp(torch.ones(x.shape[0], 1), torch.randint(-60, 60, (x.shape[0], 1), generator=gen(9)))
    m = x.shape[0]
    c = Cache([m], kv, 1, d, 16, seed=10)
    check_write(c, x.to(DEV).view(m, 1, d), (-x).to(DEV).view(m, 1, d), [m])


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("d,hk,page", [(64, 3, 16), (128, 2, 128)])
def test_read(dt, kv, d, hk, page):
    new = [1, 50, 0, page + 3, 12]
    c = Cache([40, 50, 9, 2 * page + 3, 5], kv, hk, d, page, seed=11, blocks=4 if page == 16 else 3, views=True)
    c.table[3, 1] = c.pages + 5
    cu, m = cu_of(new), sum(new)
    out = [torch.full((m + 2, hk, d), 7.0, dtype=dt, device=DEV) for _ in range(2)]
    k, v = kda.kv_cache_read(*c.args(), m + 2, dtype=dt, cu_seqlens=cu, k=out[0], v=out[1])
    torch.cuda.synchronize()
    assert k is out[0] and v is out[1]
    for got, val in zip((k, v), c.values()):
        want = torch.zeros(m + 2, hk, d, dtype=torch.float64)
        want[m:] = 7.0
        for i, (first, n) in enumerate(ref.spans(5, 0, cu)):
            length = min(c.lens[i], c.table.shape[1] * page)
            for t in range(n):
                at = ref.place(c.table.cpu(), c.lens, page, c.pages, i, length - n + t)
                if at is not None:
                    want[first + t] = val[at[0], :, at[1]]
        assert torch.equal(got.cpu().double(), want)


# ---- attention -------------------------------------------------------------------------
SHAPES = [  # H, Hk, D, page
    (4, 4, 64, 16), (8, 2, 128, 64), (6, 1, 64, 32), (5, 5, 128, 256), (12, 3, 128, 16), (16, 1, 64, 128)]


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("H,hk,d,page", SHAPES)
def test_one_token(dt, kv, H, hk, d, page):
    lens = [1, 2, 31, 32, 33, 64, 129, 300, 0, 17]
    c = Cache(lens, kv, hk, d, page, seed=20, views=page == 64)
    q = rows(dt, len(lens), H, d, 21, std=2.0).view(len(lens), 1, H, d)
    got = check_attn(c, q, [1] * len(lens), "one token", packed=False)
    assert not got[8].any()


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("H,hk,d,page", SHAPES)
@pytest.mark.parametrize("t", [2, 5, 9])
def test_few_tokens(dt, kv, H, hk, d, page, t):
    """Some tokens a sequence; sequences of fewer positions than tokens have rows that see nothing."""
    lens = [t, 40, 3, 0, 161]
    c = Cache(lens, kv, hk, d, page, seed=22)
    q = rows(dt, 5 * t, H, d, 23, std=2.0).view(5, t, H, d)
    z = rows(dt, 5 * t, H, d, 24).view(5, t, H, d)
    check_attn(c, q, [t] * 5, "few tokens", gate=z, packed=False)


@pytest.mark.parametrize("dt,kv", KINDS)
@pytest.mark.parametrize("H,hk,d,page", SHAPES)
def test_packed_prompts(dt, kv, H, hk, d, page):
    """Prompts and single tokens packed, rows behind the last sequence left alone, q and gate slices."""
    new = [70, 1, 0, 33, 129, 2]
    lens = [70, 150, 20, 200, 129, 1]
    c = Cache(lens, kv, hk, d, page, seed=25)
    m = sum(new)
    wide = rows(dt, m + 4, 2 * H, d, 26, std=1.5)
    out = torch.full((m + 4, H, d), 7.0, dtype=dt, device=DEV)
    q, z = wide[:, :H], wide[:, H:]
    cu = cu_of(new)
    got = kda.paged_attn(q, *c.args(), gate=z, cu_seqlens=cu, out=out)
    torch.cuda.synchronize()
    assert got is out and (out[m:] == 7.0).all()
    k, v = c.values()
    o, mean, size = ref.attn(q[:m].double().cpu(), k, v, c.table, lens, ref.spans(6, 0, cu), d ** -0.5,
                             z[:m].double().cpu())
    ref.close(out[:m], o, ref.attn_bound(o, mean, size, dt, d, 200), "packed")


@pytest.mark.parametrize("dt,kv", [(BF, BF), (BF, E4M3), (BF, I8), (F32, F32), (F32, I8)])
@pytest.mark.parametrize("new,length", [([1], 5000), ([3], 4097), ([40], 3000), ([1, 20], 2500), ([150], 150)])
def test_long_contexts_are_split_and_joined(dt, kv, new, length):
    c = Cache([length] * len(new), kv, 2, 64, 32, seed=27, blocks=250)
    q = rows(dt, sum(new), 4, 64, 28, std=2.0)
    check_attn(c, q, new, "split")


@pytest.mark.parametrize("dt,kv", [(BF, BF), (BF, E4M3), (BF, I8), (F32, F32), (F32, E4M3)])
@pytest.mark.parametrize("t", [1, 4, 50])
def test_pages_that_are_not_there(dt, kv, t):
    """Holes in the tables: below zero, behind the pool, and sequences without a page."""
    c = Cache([300, 200, 90, 64], kv, 2, 64, 16, seed=29, blocks=40)
    c.table[0, 3:9] = -1
    c.table[0, 12] = c.pages
    c.table[1, 0] = -7
    c.table[1, -2:] = 2 ** 31 - 1
    c.table[2] = -1
    c.table[3, 3] = -1          # the last tokens' own page
    q = rows(dt, 4 * t, 4, 64, 30, std=2.0)
    got = check_attn(c, q, [t] * 4, "holes")
    assert not got[2 * t:3 * t].any()


@pytest.mark.parametrize("dt,kv", [(BF, BF), (F32, F32), (BF, E4M3), (BF, I8), (F32, I8)])
@pytest.mark.parametrize("t", [3, 6, 70])
def test_nothing_reaches_a_token_from_behind_it(dt, kv, t):
    """NaN and infinities in keys and values of later tokens: earlier tokens stay what they are."""
    c = Cache([t + 45, t], kv, 2, 64, 32, seed=31)
    for i, length in enumerate(c.lens):
        pos = length - t // 2
        page, row = int(c.table[i, pos // 32]), pos % 32
        if kv in ref.LARGEST:
            c.k_scale.view(torch.uint8)[page, 0, row] = 255
            c.v_scale.view(torch.uint8)[page, 1, row] = 255
        else:
            c.k_cache[page, 0, row, 3] = float("nan")
            c.v_cache[page, 1, row, 5] = float("nan")
            c.v_cache[page, 1, row, 6] = float("inf")
            c.v_cache[page, 1, row, 7] = -float("inf")
            c.v_cache[page, 1, row, 8] = float("inf")
            if pos + 1 < length:
                page, row = int(c.table[i, (pos + 1) // 32]), (pos + 1) % 32
                c.v_cache[page, 1, row, 8] = -float("inf")
    q = rows(dt, 2 * t, 4, 64, 32)
    got = check_attn(c, q, [t, t], "later tokens")
    assert torch.isfinite(got[:t - t // 2]).all()


@pytest.mark.parametrize("dt,kv", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("t", [1, 40])
def test_scores_far_apart(dt, kv, t):
    """Scores that rise along the sequence by far more than an exponential holds, and equal ones."""
    c = Cache([200, 130], kv, 2, 64, 16, seed=33)
    ramp = torch.linspace(-300, 300, 224).view(14, 1, 16, 1)
    order = torch.argsort(c.table[0, :13].cpu().long())
    for b in range(13):
        c.k_cache[int(c.table[0, b]), :, :, 0] = ramp[b, 0, :, 0].to(kv).to(DEV)
    q = rows(dt, 2 * t, 4, 64, 34)
    q[..., 0] = 8.0
    q[t:, :, 1:] = 0.0
    assert order.numel() == 13
    check_attn(c, q, [t, t], "far apart", scale=1.0)
    q.zero_()
    check_attn(c, q, [t, t], "equal")


@pytest.mark.parametrize("kv", [BF, E4M3, I8])
@pytest.mark.parametrize("page,hk", [(16, 16), (64, 16), (128, 32)])
def test_prompts_that_fill_the_card(kv, page, hk):
    """Prompts of many rows, with holes in the tables, a NaN behind most tokens, and a gate.  (The widest workgroups.)"""
    new, lens = [1024, 1100], [1024 + 77, 1100]
    c = Cache(lens, kv, hk, 128, page, seed=62)
    c.table[0, 64 // page + 1] = -1
    c.table[1, 5] = c.pages
    page_of, row = int(c.table[1, 900 // page]), 900 % page
    if kv == BF:
        c.v_cache[page_of, 1, row, 5] = float("nan")
        c.v_cache[page_of, 1, row, 70] = float("inf")
        c.k_cache[page_of, 2, row, 7] = float("nan")
    else:
        c.v_scale.view(torch.uint8)[page_of, 1, row] = 255
        c.k_scale.view(torch.uint8)[page_of, 2, row] = 255
    H, m = 4 * hk, sum(new)
    q, z = rows(BF, m, H, 128, 63, std=1.5), rows(BF, m, H, 128, 64)
    cu = cu_of(new)
    got = kda.paged_attn(q, *c.args(), gate=z, cu_seqlens=cu)
    k, v = (x.to(DEV) for x in c.values())
    o, mean, size = ref.attn_wide(q.double(), k, v, c.table, lens, ref.spans(2, 0, cu), 128 ** -0.5, z.double())
    o, mean, size = o.cpu(), mean.cpu(), size.cpu()
    ref.close(got, o, torch.nan_to_num(ref.attn_bound(o, mean, size, BF, 128, 1101), nan=0.0, posinf=0.0), "prompts")
    # tokens before position 900 of the second sequence, and its heads of other cache heads, are numbers
    assert torch.isfinite(got[:1024]).all() and torch.isfinite(got[1024:1924]).all() and torch.isfinite(got[:, :4]).all()
    assert torch.isnan(got[1924:, 4:8, 5]).all() and torch.isnan(got[1924:, 8:12]).all()


@pytest.mark.parametrize("kv", [BF, E4M3, I8])
@pytest.mark.parametrize("page,new,lens,width", [(16, [256, 300], [12000, 3001], 32768), (64, [777, 260], [777, 4096], 16384),
                                                 (128, [500, 0, 1200], [500, 70, 1333], 32768), (64, [1025], [17000], 17024),
                                                 (16, [1100, 1000], [2000, 1200], 16384),
                                                 (64, [1500, 600], [17000, 601], 32768)])
def test_long_contexts_of_narrow_heads(kv, page, new, lens, width):
    """Heads of 64 under wide tables, whose rows end inside workgroups (the widest, where they fill several), with a gate."""
    hk, m = 16, sum(new)
    c = Cache(lens, kv, hk, 64, page, seed=71)
    more = torch.full((len(lens), width // page - c.table.shape[1]), -1, dtype=torch.int32, device=DEV)
    c.table = torch.cat([c.table, more], 1).contiguous()
    c.table[0, 100 // page] = -1
    page_of, row = int(c.table[-1, 600 // page]), 600 % page
    if kv == BF:
        c.v_cache[page_of, 1, row, 5] = float("nan")
    else:
        c.v_scale.view(torch.uint8)[page_of, 1, row] = 255
    q, z = rows(BF, m, 4 * hk, 64, 72, std=1.5), rows(BF, m, 4 * hk, 64, 73)
    cu = cu_of(new)
    got = kda.paged_attn(q, *c.args(), gate=z, cu_seqlens=cu)
    k, v = (x.to(DEV) for x in c.values())
    o, mean, size = ref.attn_wide(q.double(), k, v, c.table, lens, ref.spans(len(new), 0, cu), 64 ** -0.5, z.double())
    o, mean, size = o.cpu(), mean.cpu(), size.cpu()
    ref.close(got, o, torch.nan_to_num(ref.attn_bound(o, mean, size, BF, 64, max(lens)), nan=0.0, posinf=0.0), "narrow")


def test_no_sequences_no_tokens():
    c = Cache([40, 3], BF, 2, 64, 16, seed=35)
    none = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    assert kda.paged_attn(none, *c.args(), cu_seqlens=cu_of([0, 0])).shape == (0, 4, 64)
    before = c.k_cache.clone()
    kda.kv_cache_write(none[:, :2], none[:, :2], *c.args(), cu_seqlens=cu_of([0, 0]))
    k, _ = kda.kv_cache_read(*c.args(), 0)
    assert k.shape == (2, 0, 2, 64) and torch.equal(before.nan_to_num(), c.k_cache.nan_to_num())
    empty = Cache([], BF, 2, 64, 16, seed=36)
    assert kda.paged_attn(none.view(0, 1, 4, 64), *empty.args()).numel() == 0
    nopages = Cache([0, 0], BF, 2, 64, 16, seed=36, spare=0)
    q = rows(BF, 2, 4, 64, 37).view(2, 1, 4, 64)
    assert not kda.paged_attn(q, *nopages.args()).any()


@pytest.mark.parametrize("dt,kv", [(BF, BF), (BF, E4M3), (F32, F32), (F32, I8)])
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("n,t,length", [(70, 9, 40), (64, 12, 30), (65, 1, 50)])
def test_many_sequences(dt, kv, packed, n, t, length):
    """Batches around the number of lanes that order their tiles by length, lengths that tie among them."""
    g = torch.Generator().manual_seed(51)
    lens = [length - 3 * int(torch.randint(0, 4, (1,), generator=g)) for _ in range(n)]
    new = [int(torch.randint(0, t + 1, (1,), generator=g)) for _ in range(n)] if packed else [t] * n
    new[3] = t
    c = Cache(lens, kv, 2, 64, 16, seed=52)
    q = rows(dt, sum(new), 10, 64, 53, std=2.0)
    check_attn(c, q if packed else q.view(n, t, 10, 64), new, "many", packed=packed)


@pytest.mark.parametrize("dt,kv", [(BF, BF), (BF, E4M3), (BF, I8), (F32, F32)])
@pytest.mark.parametrize("H,hk,t", [(20, 1, 1), (40, 1, 2), (64, 1, 5), (33, 3, 7)])
def test_many_heads_of_one_cache_head(dt, kv, H, hk, t):
    c = Cache([t + 70, 5], kv, hk, 128, 32, seed=54)
    q = rows(dt, 2 * t, H, 128, 55).view(2, t, H, 128)
    check_attn(c, q, [t, t], "many heads", packed=False)


@pytest.mark.parametrize("dt,kv", [(BF, E4M3), (BF, I8), (F32, E4M3), (F32, I8)])
def test_scales_of_every_size(dt, kv):
    """Scale bytes from 1 (2^-126) to 253, what a cache written elsewhere may hold, read back exactly; 255 is NaN."""
    c = Cache([256], kv, 1, 64, 16, seed=56)
    codes = torch.arange(256, dtype=torch.int32).repeat(64).view(256, 64).to(torch.uint8)
    if kv == E4M3:      # its NaN codes are tested as such below; 2^8 * 1.75 * 2^120 is the largest that fp32 holds
        codes = torch.where((codes & 127) == 127, 0, codes.int()).to(torch.uint8)
    byte = torch.arange(256).clamp(min=1, max=246)
    byte[255] = 255
    for cache, scale in ((c.k_cache, c.k_scale), (c.v_cache, c.v_scale)):
        for pos in range(256):
            page = int(c.table[0, pos // 16])
            cache.view(torch.uint8)[page, 0, pos % 16] = codes[pos].to(DEV)
            scale.view(torch.uint8)[page, 0, pos % 16] = int(byte[pos])
    k, v = kda.kv_cache_read(*c.args(), 256, dtype=dt)
    want = codes.view(kv).float().double() * torch.ldexp(torch.ones(256, 1, dtype=torch.float64), byte[:, None] - 127)
    want[255] = float("nan")
    # Exact but for subnormal products (below 2^-126, of scales below 2^-117 that no write makes): bf16 holds these in
    # steps of 2^-133, so they are off by half a step, 2^-134, or come as zeros.
    small = want.abs() < 2.0 ** -126
    for got in (k, v):
        got = got.view(256, 64).double().cpu()
        same = (got == want) | (small & ((got == 0) | ((got - want).abs() <= 2.0 ** -134))) | (torch.isnan(got) & torch.isnan(want))
        assert same.all(), torch.nonzero(~same)[:4]
    # a NaN code under an ordinary scale
    if kv == E4M3:
        c.v_cache.view(torch.uint8)[int(c.table[0, 0]), 0, 3, 5] = 0x7f
        c.v_scale.view(torch.uint8).fill_(127)
        c.k_scale.view(torch.uint8).fill_(120)
        c.seq_lens.fill_(6)
        c.lens = [6]
        got = check_attn(c, rows(dt, 5, 2, 64, 57), [5], "a NaN code")
        assert torch.isfinite(got[:2]).all() and torch.isnan(got[2:, :, 5]).all()


@pytest.mark.parametrize("dt,kv,t", [(BF, BF, 1), (BF, BF, 40), (BF, E4M3, 40), (F32, F32, 3)])
def test_pools_beyond_four_gigabytes(dt, kv, t):
    """The same pages at the end of a large pool and in a small one: the same bits."""
    hk, d, page = 8, 128, 256
    c = Cache([700, 300], kv, hk, d, page, seed=58)
    each = hk * d * page * c.k_cache.element_size()
    pages = (5 << 30) // each
    m = 2 * t
    q, k, v = rows(dt, m, 16, d, 59).view(2, t, 16, d), rows(dt, m, hk, d, 60), rows(dt, m, hk, d, 61)
    k, v = k.view(2, t, hk, d), v.view(2, t, hk, d)
    big = [torch.empty((pages, hk, page, d), dtype=kv, device=DEV) for _ in range(2)]
    scales = [None, None]
    for b, cache in zip(big, (c.k_cache, c.v_cache)):
        b[pages - c.pages:].copy_(cache)
    if c.k_scale is not None:
        scales = [torch.full((pages, hk, page), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
        for b, s in zip(scales, (c.k_scale, c.v_scale)):
            b[pages - c.pages:].copy_(s.view(torch.uint8))
        scales = [s.view(torch.float8_e8m0fnu) for s in scales]
    table = torch.where(c.table >= 0, c.table + (pages - c.pages), -1).to(torch.int32)
    there = (big[0], big[1], table, c.seq_lens, *scales)
    kda.kv_cache_write(k, v, *c.args())
    kda.kv_cache_write(k, v, *there)
    assert torch.equal(kda.paged_attn(q, *c.args()), kda.paged_attn(q, *there))
    for a, b in zip(kda.kv_cache_read(*c.args(), t, dtype=dt), kda.kv_cache_read(*there, t, dtype=dt)):
        assert torch.equal(a, b)


# ---- together --------------------------------------------------------------------------
@pytest.mark.parametrize("dt,kv", [(BF, BF), (BF, E4M3), (BF, I8), (F32, F32)])
def test_prompt_chunks_and_steps(dt, kv):
    """A layer's life: a prompt in chunks, then single tokens, each written before it is attended to; the whole equals
    the attention of the values that the cache holds."""
    H, hk, d, page = 4, 2, 64, 16
    lens = [90, 47]
    total = Cache(lens, kv, hk, d, page, seed=40)
    total.spoil(torch.ones(total.pages, page, dtype=torch.bool))
    g = gen(41)
    q, k, v, z = ([torch.randn((n, h, d), generator=g).to(dt).to(DEV) for n in lens] for h in (H, hk, hk, H))
    outs = [[], []]
    done = [0, 0]
    steps = [(40, 16), (30, 20)] + [(1, 1)] * 11 + [(9, 0)]
    for new in steps:
        cu = cu_of(new)
        total.seq_lens = torch.tensor([a + b for a, b in zip(done, new)], dtype=torch.int32, device=DEV)
        part = lambda x: torch.cat([x[i][done[i]:done[i] + new[i]] for i in range(2)])
        kda.kv_cache_write(part(k), part(v), *total.args(), cu_seqlens=cu)
        o = kda.paged_attn(part(q), *total.args(), gate=part(z), cu_seqlens=cu)
        for i in range(2):
            outs[i].append(o[int(cu[i]):int(cu[i + 1])])
            done[i] += new[i]
    assert done == lens
    rk, rv = kda.kv_cache_read(*total.args(), sum(lens), dtype=dt, cu_seqlens=cu_of(lens))
    torch.cuda.synchronize()
    kv_, vv_ = total.values()
    flat = lambda x: torch.cat(x).cpu().double()
    cu = cu_of(lens)
    o, mean, size = ref.attn(flat(q), kv_, vv_, total.table, lens, ref.spans(2, 0, cu), d ** -0.5, flat(z))
    ref.close(torch.cat([torch.cat(x) for x in outs]), o, ref.attn_bound(o, mean, size, dt, d, 90), "steps")
    want = flat(k)
    if kv in ref.LARGEST:
        want = ref.values(*ref.quantise(want, kv))
    assert torch.equal(rk.double().cpu(), want)


@pytest.mark.parametrize("dt,kv,new", [(BF, BF, [1, 1, 1]), (BF, E4M3, [40, 1, 30]), (F32, I8, [9, 1, 2])])
def test_captured_and_replayed(dt, kv, new):
    """Write, attention and read in one graph, replayed with other tokens and lengths, eager work in between."""
    H, hk, d, page = 4, 2, 128, 32
    c = Cache([700, 90, 64], kv, hk, d, page, seed=42)
    c.spoil(torch.zeros(c.pages, page, dtype=torch.bool))
    m = sum(new)
    q, k, v = rows(dt, m, H, d, 43), rows(dt, m, hk, d, 44), rows(dt, m, hk, d, 45)
    cu, out = cu_of(new), torch.empty((m, H, d), dtype=dt, device=DEV)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    rk, rv = (torch.empty((m, hk, d), dtype=dt, device=DEV) for _ in range(2))

    def call():
        kda.kv_cache_write(k, v, *c.args(), cu_seqlens=cu)
        kda.paged_attn(q, *c.args(), cu_seqlens=cu, out=out, workspace=ws)
        kda.kv_cache_read(*c.args(), m, dtype=dt, cu_seqlens=cu, k=rk, v=rv)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(4):
        q.copy_(rows(dt, m, H, d, 50 + step))
        k.copy_(rows(dt, m, hk, d, 60 + step))
        c.seq_lens.copy_(torch.tensor([700 - 100 * step, 90 - step, 64], dtype=torch.int32))
        out.fill_(float("nan"))
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, rk, rv, c.k_cache.to(torch.float32), c.v_cache.to(torch.float32))]
        ws.fill_(127)
        call()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, rk, rv, c.k_cache.to(torch.float32), c.v_cache.to(torch.float32))):
            assert torch.equal(a.nan_to_num(), b.nan_to_num()), step
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("dt,kv,d,t,hk,width", [(BF, BF, 128, 1, 2, 16384), (BF, E4M3, 64, 8, 2, 16384),
                                                (BF, I8, 128, 40, 2, 16384), (BF, BF, 64, 300, 16, 32768),
                                                (BF, E4M3, 64, 1024, 8, 32768), (BF, BF, 128, 200, 4, 16384),
                                                (F32, F32, 64, 9, 2, 16384)])
def test_replays_whose_lengths_cross_ranges(dt, kv, d, t, hk, width):
    """One graph, lengths from none to the table's end in any order: ranges that appear and vanish between replays leave
    nothing of the replay before.  (One token, few, chunks, the widest rows, fp32.)"""
    c = Cache([width, width], kv, hk, d, 64, seed=81)
    q = rows(dt, 2 * t, 4 * hk, d, 82).view(2, t, 4 * hk, d)
    out = torch.empty_like(q)
    call = lambda o: kda.paged_attn(q, *c.args(), out=o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for lens in ([width, 1], [1, 0], [5000, width], [width, width - 1], [0, 0], [700, 9000], [width, 1]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got, eager = out.clone(), call(None)
        assert torch.equal(got, eager), lens
        k, v = (x.to(DEV) for x in c.values())
        flat = q.reshape(-1, 4 * hk, d).double()
        o, mean, size = (x.cpu() for x in ref.attn_wide(flat, k, v, c.table, lens, ref.spans(2, t, None), d ** -0.5))
        ref.close(got.reshape(o.shape), o, ref.attn_bound(o, mean, size, dt, d, width), lens)


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace and an output of its own, equal the same calls in turn."""
    c = Cache([6000, 900], BF, 2, 128, 64, seed=46)
    q = [rows(BF, 2, 8, 128, 47 + i).view(2, 1, 8, 128) for i in range(2)]
    want = [kda.paged_attn(x, *c.args()) for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, x in zip(streams, q):
            with torch.cuda.stream(s):
                got.append(kda.paged_attn(x, *c.args()))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_profile_names():
    c = Cache([6000], E4M3, 2, 128, 64, seed=48)
    q = rows(BF, 1, 8, 128, 49)
    kda.profile_start(8)
    kda.kv_cache_write(q[:, :2], q[:, 2:4], *c.args(), cu_seqlens=cu_of([1]))
    kda.paged_attn(q, *c.args(), cu_seqlens=cu_of([1]))
    kda.kv_cache_read(*c.args(), 1)
    names = [n for n, _ in kda.profile_stop(8)]
    assert names == ["cache_write", "attn_step", "attn_join", "cache_read"]


# kernel -> (tokens, heads, cache heads, head dim, dtypes, width of the table, positions, length of a range)
SPLIT = {"step16": (1, 8, 2, 128, 8192, 2600, 512), "step32": (5, 8, 2, 64, 8192, 2600, 512),
         "chunk": (70, 8, 2, 128, 8192, 4200, 1024), "chunk narrow": (70, 8, 2, 64, 8192, 4200, 1024),
         "chunk wide rows": (64, 32, 2, 64, 262144, 9300, 4096), "fp32": (9, 8, 2, 64, 8192, 2600, 512)}


@pytest.mark.parametrize("poison", [3e4, float("inf"), float("nan")])
@pytest.mark.parametrize("page,at", [(16, -128), (16, -64), (16, 0), (64, -128), (64, -64), (64, 0)])
@pytest.mark.parametrize("kernel,kv", [(k, kv) for k in SPLIT for kv in ((F32, I8) if k == "fp32" else (BF, E4M3, I8))])
def test_holes_where_ranges_meet(kernel, kv, page, at, poison):
    """64 positions without a page in the first, the second last or the last tile of every range.  Page 0, which no
    sequence has, holds keys and values that would drown every other."""
    t, H, hk, d, width, length, span = SPLIT[kernel]
    dt = F32 if kernel == "fp32" else BF
    c = Cache([length], kv, hk, d, page, seed=91, blocks=width // page)
    take = int((~torch.isin(torch.arange(c.pages, dtype=torch.int32), c.table.cpu())).nonzero()[0])
    for cache in (c.k_cache, c.v_cache, c.k_scale, c.v_scale):
        if cache is not None:
            raw = cache if cache.dtype == kv else cache.view(torch.uint8)
            raw[take] = raw[0].clone()
    c.table[c.table == 0] = take
    if kv in ref.LARGEST:       # the codes' largest number, or their NaN
        for cache, scale in ((c.k_cache, c.k_scale), (c.v_cache, c.v_scale)):
            cache[0] = torch.tensor(ref.LARGEST[kv]).to(kv).to(DEV)
            scale.view(torch.uint8)[0] = 133 if poison == 3e4 else 255
    else:
        c.k_cache[0] = 1.0 if poison == float("inf") else poison
        c.k_cache[0, ..., 0] = poison
        c.v_cache[0] = poison
    for b in range(span, length, span):
        first = b + at
        c.table[0, first // page:(first + 64) // page] = -1
    q = rows(dt, t, H, d, 92, std=1.5)
    got = kda.paged_attn(q.view(1, t, H, d), *c.args()).view(t, H, d)
    k, v = (x.to(DEV) for x in c.values())
    o, mean, size = (x.cpu() for x in ref.attn_wide(q.double(), k, v, c.table, [length], [(0, t)], d ** -0.5))
    ref.close(got, o, ref.attn_bound(o, mean, size, dt, d, length), kernel)


@pytest.mark.parametrize("dt,kv", [(BF, BF), (F32, F32)])
@pytest.mark.parametrize("H,hk,d,page", [(8, 2, 128, 64), (16, 1, 64, 16), (4, 4, 64, 32)])
@pytest.mark.parametrize("t", [1, 5, 24, 70])
def test_infinities_that_every_token_sees(dt, kv, H, hk, d, page, t):
    """Infinities and NaN among the values of positions that all rows see whole blocks around: every token's sum has
    them, whatever its weights (a weight's own rounding may leave zero or fall below it)."""
    lens = [300, 700]
    c = Cache(lens, kv, hk, d, page, seed=93)
    inf = float("inf")
    for i, pos in ((0, 5), (0, 40), (1, 5), (1, 130), (1, 513)):
        at = int(c.table[i, pos // page]), slice(None), pos % page
        c.v_cache[at][:, 3] = inf
        c.v_cache[at][:, 20] = -inf
        c.v_cache[at][:, 37] = float("nan")
        c.v_cache[at][:, 50] = inf if pos == 5 else -inf        # both: NaN
    q = rows(dt, 2 * t, H, d, 94).view(2, t, H, d)
    got = check_attn(c, q, [t, t], "infinities", packed=False)
    assert (got[..., 3] == inf).all() and (got[..., 20] == -inf).all()
    assert torch.isnan(got[..., 37]).all() and torch.isnan(got[..., 50]).all()
    got[..., [3, 20, 37, 50]] = 0.0
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("kv", [E4M3, I8])
@pytest.mark.parametrize("t", [1, 5, 24, 70])
def test_codes_beyond_the_largest_number(dt, kv, t):
    """Codes whose values pass 2^128 are infinite or the largest numbers: never NaN, where every token sees them."""
    H, hk, d, page = 8, 2, 64, 16
    c = Cache([300, 700], kv, hk, d, page, seed=95)
    sign = torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0)
    for i, pos in ((0, 5), (1, 130), (1, 513)):
        at = int(c.table[i, pos // page]), slice(None), pos % page
        c.v_cache[at] = (sign * ref.LARGEST[kv]).expand(hk, d).to(kv).to(DEV)
        c.v_scale.view(torch.uint8)[at] = 254
    q = rows(dt, 2 * t, H, d, 96).view(2, t, H, d)
    got = kda.paged_attn(q, *c.args()).float().cpu()
    assert not torch.isnan(got).any()
    assert (got * sign > 2.0 ** 96).all()       # weights here are above 2^-24, the rest of a sum below 2^4


@pytest.mark.parametrize("kv", [BF, E4M3, I8])
@pytest.mark.parametrize("n,t,length,H,hk,d,page", ref.TWO_PARTS)
def test_weights_in_two_parts(kv, n, t, length, H, hk, d, page):
    """Up to 16 rows a sequence: weights are off by 2^-16, not by a rounding to bf16."""
    c = Cache([length] * n, kv, hk, d, page, seed=97)
    q, k, v = (x.to(BF).to(DEV) for x in ref.cancelling(n, t, length, H, hk, d, kv, 98))
    kda.kv_cache_write(k.view(n, length, hk, d), v.view(n, length, hk, d), *c.args())
    got = kda.paged_attn(q.view(n, t, H, d), *c.args(), scale=1.0).view(n * t, H, d)
    o, mean, _ = ref.attn(q.cpu().double(), *c.values(), c.table, c.lens, ref.spans(n, t, None), 1.0)
    ref.close(got, o, ref.attn_bound_two(o, mean, length), "two parts")


@pytest.mark.parametrize("dt,n,t,H,hk,d,page", [(BF, 4, 512, 32, 8, 128, 16), (BF, 4, 512, 32, 8, 64, 64), (BF, 1, 1, 8, 2, 128, 64),
                                                (BF, 8, 4, 16, 2, 128, 16), (F32, 1, 9, 8, 2, 64, 64)])
def test_time_does_not_go_by_what_stands_in_for_missing_pages(dt, n, t, H, hk, d, page):
    """Long sequences whose first pages are gone, and a page 0, no sequence's, of NaN or of zeros: the same bits, and
    no more than twice the time (it was 3 to 37 times)."""
    length = 16384
    blocks = length // page
    pool = [torch.randn((n * blocks + 1, hk, page, d), generator=gen(99 + i)).to(dt).to(DEV) for i in range(2)]
    table = torch.randperm(n * blocks, generator=gen(101)).view(n, blocks) + 1
    table[:, :blocks // 8] = -1
    table, lens = table.to(torch.int32).to(DEV), torch.full((n,), length, dtype=torch.int32, device=DEV)
    q = rows(dt, n * t, H, d, 102).view(n, t, H, d)
    outs, times = [], []
    for fill in (0.0, float("nan")):
        for p in pool:
            p[0] = fill
        out = torch.empty_like(q)
        best = float("inf")
        for _ in range(6):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(3):
                kda.paged_attn(q, *pool, table, lens, out=out)
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end))
        outs.append(out)
        times.append(best)
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()
    assert times[1] < 2 * times[0], times


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("length", [130, 5000])
@pytest.mark.parametrize("t", [1, 5, 24, 70])
def test_scores_of_minus_infinity(dt, t, length):
    """A token whose scores are all -infinity gets zeros, whatever the values; one that sees another position gets that one's."""
    H, hk, d, page = 8, 2, 64, 16
    c = Cache([length, length], dt, hk, d, page, seed=103)
    c.k_cache[..., 0] = -float("inf")
    c.v_cache[int(c.table[0, 1]), :, 3, 7] = float("inf")
    c.v_cache[int(c.table[0, 2]), :, 4, 9] = float("nan")
    at = int(c.table[1, 3]), slice(None), 5
    c.k_cache[at][:, 0] = 1.0
    q = rows(dt, 2 * t, H, d, 104).view(2, t, H, d)
    q[..., 0] = 1.0
    got = kda.paged_attn(q, *c.args())
    assert not got[0].any() and torch.equal(got[1], c.v_cache[at].repeat_interleave(H // hk, 0).expand(t, H, d))
