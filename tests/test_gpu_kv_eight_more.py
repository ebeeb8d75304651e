"""A cache of 8 bits: which codes append leaves in which heads."""
import math

import pytest
import torch

from test_gpu_kv import BF16, F16, i32
from test_gpu_kv_eight import make8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("rot", [0, 64])
def test_codes_of_nan_stand_only_in_heads_that_are_nan(ss, cuda_device, dtype, D, rot):
    """Heads of every size and of the largest numbers, every third with a NaN or an
    infinity somewhere: byte 255 there and nowhere else, and no code of NaN elsewhere."""
    dev, N, H = cuda_device, 64, 9
    g = torch.Generator(device=dev).manual_seed(D)
    size = torch.randint(-30, 17, (1, N, H, 1), generator=g, device=dev)
    x = torch.randn((1, N, H, D), generator=g, device=dev) * torch.exp2(size.float())
    x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
    at = torch.randint(0, D, (N, H), generator=g, device=dev)
    bad = torch.zeros((N, H), dtype=torch.bool, device=dev)
    for value, h in ((math.nan, 0), (math.inf, 3), (-math.inf, 6)):
        x[0, torch.arange(N, device=dev), h, at[:, h]] = value
        bad[:, h] = True
    c, table = make8(ss, dev, [5], [N], 16, H, D, dtype)
    rope = ss.Rope(ss.rope_frequencies(rot)[0].to(dev)) if rot else None
    c.append(0, c.plan(N, H), None, x, x.clone(), rope)
    z = 5 + torch.arange(N, device=dev)
    pg = i32(table[0], dev).long()[z // 16]
    for pool, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        assert torch.equal(scale[0, pg, :, z % 16] == 255, bad)
        nan = (pool.view(torch.uint8)[0, pg, :, z % 16] & 127) == 127
        assert not nan[~bad].any()
    assert ((c.v.view(torch.uint8)[0, pg, :, z % 16] & 127) == 127)[:, 0].any(-1).all()   # a NaN's own code
    for got in c.read(0, None, i32([5], dev), N):
        assert torch.equal(got[0].isnan().all(-1), bad) and torch.equal(got[0].isnan().any(-1), bad)
