"""What the paged cache tests' bounds let pass (no GPU): weights in two parts
do, weights of one bf16 do not."""
import pytest
import torch

from tests import paged_ref as ref

BF = torch.bfloat16


@pytest.mark.parametrize("kv", [BF, torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("n,t,length,H,hk,d,page", ref.TWO_PARTS)
def test_bound_of_weights_in_two_parts(kv, n, t, length, H, hk, d, page):
    q, k, v = ref.cancelling(n, t, length, H, hk, d, kv, 98)
    if kv != BF:
        k, v = (ref.values(*ref.quantise(x, kv)) for x in (k, v))
    k, v = (x.view(n, length, hk, d).transpose(1, 2).contiguous() for x in (k, v))      # a page a sequence
    table = torch.arange(n, dtype=torch.int32)[:, None]
    o, mean, _ = ref.attn(q, k, v, table, [length] * n, ref.spans(n, t, None), 1.0)
    bound = ref.attn_bound_two(o, mean, length)
    for parts in (1, 2):
        got = torch.zeros_like(o)
        for i in range(n):
            for j in range(t):
                m = length - t + j + 1
                for h in range(H):
                    kk, vv = k[i, h * hk // H, :m], v[i, h * hk // H, :m]
                    s = kk @ q[i * t + j, h]
                    p = torch.exp(s - s.max())
                    first = p.to(BF).double()
                    use = first + (p - first).to(BF).double() if parts == 2 else first
                    got[i * t + j, h] = (use @ vv) / p.sum()
        got = got.to(BF).double()
        if parts == 2:
            ref.close(got, o, bound, "two parts")
        else:
            with pytest.raises(AssertionError):
                ref.close(got, o, bound, "one part")
            assert ((got - o).abs() > 2 * bound).any()
