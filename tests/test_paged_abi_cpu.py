"""Argument checks of the paged cache operators' C ABI and binding (no GPU:
nothing here is launched, addresses are never dereferenced)."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_66_amd as kda
from gated_delta_rule_66_amd import kda as K_
from gated_delta_rule_66_amd import paged

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F32, BF16, E4M3, I8 = 0, 1, 2, 3
M = 1 << 40             # distance between the made-up buffers
BIG = ctypes.c_size_t(-1).value


def lib():
    if not os.path.exists(kda.LIB_PATH):
        kda.build_library()
    return K_.load_library()


def cache(dt=BF16, pages=10, heads=2, page=16, d=64, blocks=4, **kw):
    width = heads * page * d
    c = dict(dt=dt, pages=pages, heads=heads, page_size=page, head_dim=d, blocks=blocks, k=20 * M, v=21 * M,
             k_page_stride=width, v_page_stride=width, k_scale=22 * M if dt >= E4M3 else None,
             v_scale=23 * M if dt >= E4M3 else None, block_table=24 * M, block_table_stride=blocks, seq_lens=25 * M)
    c.update(kw)
    return K_.PagedCache(**c)


def write(n=2, cu=None, t=5, dt=BF16, k=M, ks=None, v=2 * M, vs=None, c=None, **kw):
    c = cache(**kw) if c is None else c
    w = c.heads * c.head_dim
    return lib().kda_kv_cache_write(n, cu, t, dt, k, w if ks is None else ks, v, w if vs is None else vs,
                                    ctypes.byref(c), None)


def read(n=2, cu=None, t=5, dt=BF16, k=M, v=2 * M, **kw):
    return lib().kda_kv_cache_read(n, cu, t, dt, k, v, ctypes.byref(cache(**kw)), None)


def attn(n=2, cu=None, t=5, h=4, dt=BF16, scale=0.125, q=M, qs=None, z=2 * M, zs=None, o=3 * M, ws=4 * M, nbytes=1 << 38,
         **kw):
    c = cache(**kw)
    w = h * c.head_dim
    return lib().kda_paged_attn(n, cu, t, h, dt, scale, q, w if qs is None else qs, z, w if zs is None else zs, o,
                                ctypes.byref(c), ws, nbytes, None)


def need(n, packed, t, h, dt=BF16, **kw):
    return lib().kda_paged_attn_workspace_size(n, packed, t, h, dt, ctypes.byref(cache(**kw)))


CALLS = [write, read, attn]


@pytest.mark.parametrize("call", CALLS)
def test_refused_sizes(call):
    assert call(n=-1) == INVALID
    assert call(t=-1) == INVALID
    assert call(dt=5) == INVALID
    for bad in (dict(heads=0), dict(heads=-2), dict(pages=-1), dict(blocks=-1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(d=96), dict(d=32), dict(d=0), dict(page=8), dict(page=48), dict(page=512), dict(page=0),
                dict(page=-16), dict(heads=65536), dict(blocks=(1 << 26) + 1)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n=1 << 16, t=1 << 16) == UNSUPPORTED
    assert call(n=0) == OK and call(t=0) == OK
    assert call(n=0, k_scale=None, block_table=None, seq_lens=None) == OK


def test_types_that_do_not_go_together():
    null = ctypes.POINTER(K_.PagedCache)()
    assert lib().kda_kv_cache_write(1, None, 1, BF16, M, 128, 2 * M, 128, null, None) == INVALID
    assert lib().kda_kv_cache_read(1, None, 1, BF16, M, 2 * M, null, None) == INVALID
    assert lib().kda_paged_attn(1, None, 1, 2, BF16, 1.0, M, 128, None, 0, 3 * M, null, 4 * M, 1 << 30, None) == INVALID
    assert lib().kda_paged_attn_workspace_size(1, 0, 1, 2, BF16, null) == BIG
    for dt, kv in ((BF16, F32), (F32, BF16)):
        assert write(dt=dt, c=cache(dt=kv)) == UNSUPPORTED
        assert lib().kda_kv_cache_read(2, None, 5, dt, M, 2 * M, ctypes.byref(cache(dt=kv)), None) == UNSUPPORTED
        assert lib().kda_paged_attn_workspace_size(2, 0, 5, 4, dt, ctypes.byref(cache(dt=kv))) == BIG
    for kv in (E4M3, I8):
        assert write(c=cache(dt=kv, k_scale=None)) == INVALID
        assert write(c=cache(dt=kv, v_scale=None)) == INVALID
        assert write(c=cache(dt=kv, v_scale=23 * M + 8)) == INVALID
    assert write(k_scale=22 * M) == INVALID             # scales of a cache without codes
    assert write(v_scale=23 * M) == INVALID
    for kv in (-1, 4):
        assert write(c=cache(dt=kv)) == INVALID


@pytest.mark.parametrize("call", CALLS)
def test_refused_pointers(call):
    for name in ("k", "v") if call is not attn else ("q", "o"):
        assert call(**{name: None}) == INVALID, name
        assert call(**{name: M // 2 + 8}) == INVALID, name
    for bad in (dict(k_page_stride=2047), dict(v_page_stride=2052), dict(seq_lens=None), dict(seq_lens=25 * M + 2),
                dict(block_table=None), dict(block_table=24 * M + 1), dict(block_table_stride=3)):
        assert call(**bad) == INVALID, bad
    assert call(k_page_stride=1 << 41) == UNSUPPORTED
    assert call(cu=6) == INVALID
    if call is attn:
        assert attn(k=None) == INVALID and attn(v=None) == INVALID and attn(k=20 * M + 8) == INVALID


def test_refused_strides_and_overlaps():
    assert write(ks=120) == INVALID and write(vs=132) == INVALID
    assert write(ks=1 << 58) == UNSUPPORTED
    assert write(k=20 * M) == INVALID                   # tokens in the cache
    assert write(c=cache(k=24 * M)) == INVALID          # the cache on the table
    assert read(k=25 * M) == INVALID                    # rows on the lengths
    assert write(c=cache(v=20 * M)) == INVALID          # both caches in one place
    assert write(c=cache(v=20 * M + 4096 * 9)) == INVALID
    assert write(c=cache(dt=E4M3, v_scale=22 * M)) == INVALID
    assert read(v=M) == INVALID
    assert read(k=21 * M) == INVALID
    assert attn(o=M) == INVALID and attn(o=2 * M) == INVALID and attn(o=20 * M) == INVALID
    assert attn(ws=M) == INVALID or need(2, 0, 5, 4) == 0
    assert attn(h=3) == INVALID and attn(h=0) == INVALID
    assert attn(qs=252) == INVALID and attn(zs=260) == INVALID and attn(qs=1 << 58) == UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert attn(scale=scale) == INVALID, scale


def test_attention_sizes_and_workspace():
    assert need(2, 0, 5, 3) == BIG and need(2, 0, 5, 1 << 17) == BIG and need(-1, 0, 5, 4) == BIG
    assert need(0, 0, 5, 4) == 0 and need(2, 0, 0, 4) == 0
    long = dict(blocks=1 << 12, page=256)               # one sequence of up to a million positions is split
    n = need(1, 0, 1, 4, **long)
    assert 0 < n < 1 << 30
    assert attn(n=1, t=1, nbytes=n - 1, **long) == WORKSPACE
    assert attn(n=1, t=1, ws=None, **long) == WORKSPACE
    assert attn(n=1, t=1, ws=4 * M + 8, **long) == INVALID
    assert attn(n=1, t=1, ws=M, **long) == INVALID      # over q
    assert need(1, 0, 1 << 30, 4) == BIG                # rows beyond an int
    assert need(1 << 20, 0, 64, 64, heads=64) == BIG    # grids beyond the launch's threads


def test_binding_refusals():
    cpu = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for call in (lambda: kda.paged_attn(cpu, pool, pool, table, lens),
                 lambda: kda.kv_cache_write(cpu, cpu, pool, pool, table, lens),
                 lambda: kda.kv_cache_read(pool, pool, table, lens, None, None, 1)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    dev = pool.get_device()     # -1: the checks below compare devices only

    def make(k=pool, v=pool, tab=table, ln=lens, ks=None, vs=None):
        return paged._cache(k, v, tab, ln, ks, vs, dev)

    assert make().k_page_stride == 2048
    both = torch.zeros(3, 2, 2, 16, 64, dtype=torch.bfloat16)
    assert make(both[:, 0], both[:, 1]).v_page_stride == 4096
    codes = torch.zeros(3, 2, 16, 64, dtype=torch.int8)
    scale = torch.zeros(3, 2, 16, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    assert make(codes, codes, ks=scale, vs=scale).dt == I8
    for bad in (dict(k=pool[0]), dict(k=pool.half(), v=pool.half()), dict(v=pool.float()), dict(v=pool[:2]),
                dict(k=pool.transpose(1, 2)), dict(ks=scale, vs=scale), dict(k=codes, v=codes),
                dict(k=codes, v=codes, ks=scale, vs=scale.view(torch.uint8)), dict(k=codes, v=codes, ks=scale, vs=scale[:2]),
                dict(tab=table.long()), dict(tab=table[0]), dict(tab=torch.zeros(4, 1, dtype=torch.int32).t().expand(2, 4)),
                dict(ln=lens.long()), dict(ln=torch.ones(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            make(**bad)
    with pytest.raises(ValueError):
        paged._batch((2, 1, 4, 64), lens, None, dev, "q")
    with pytest.raises(ValueError):
        paged._batch((2, 4, 64), lens, None, dev, "q")
    with pytest.raises(ValueError):
        paged._batch((2, 4, 64), lens, torch.zeros(3, dtype=torch.int32), dev, "q")
    assert paged._batch((7, 4, 64), lens, torch.zeros(2, dtype=torch.int32), dev, "q") == (1, 1, 7)
