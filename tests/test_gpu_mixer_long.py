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
