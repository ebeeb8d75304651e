"""A cache of 8 bits: which codes append leaves in which heads, and of elements that are not
turned."""
import math

import pytest
import torch

import kv_more_reference as more
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


@pytest.mark.parametrize("layout,rot", [("half", 128), ("interleaved", 128), ("half", 48), ("half", 20), ("interleaved", 64)])
@pytest.mark.parametrize("dtype,m", [(BF16, 1.0), (F16, 1.0), (BF16, 1.25), (F16, 1.1)])
def test_codes_where_some_pairs_are_not_turned(ss, cuda_device, layout, rot, dtype, m):
    """Patches of a grid that counts from 0, and a frequency of 0: elements that are their
    16-bit inputs times m, ties among them, beside others that are turned."""
    dev, N, H, D = cuda_device, 400, 8, 128
    c, _ = make8(ss, dev, [3], [N], 64, H, D, dtype)
    g = torch.Generator(device=dev).manual_seed(rot)
    k = torch.randn((1, N, H, D), generator=g, device=dev).to(dtype)
    k[0, ::7] = (torch.randint(-31, 32, k[0, ::7].shape, generator=g, device=dev) / 16).to(dtype)   # many ties
    f = torch.tensor([10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=torch.float64, device=dev)
    f[3] = 0.0
    axis = torch.arange(rot // 2, device=dev) % 3
    yx = torch.cartesian_prod(torch.arange(20, device=dev), torch.arange(20, device=dev))
    pos = torch.cat((torch.zeros_like(yx[:, :1]), yx), 1)
    c.append(0, c.plan(N, H), None, k, k, ss.Rope(f, layout, m, axis.int()), positions=pos.int()[None].contiguous())
    got = c.read(0, None, i32([3], dev), N)[0][0].double()
    x = k[0].double()
    mm = torch.tensor(m, dtype=torch.float32).double().item()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    t = (pos[:, axis] * f)[:, None]
    u, w, h = (a * t.cos() - b * t.sin()) * mm, (a * t.sin() + b * t.cos()) * mm, torch.hypot(a, b) * mm
    join = (lambda p, q: torch.cat((p, q), -1)) if layout == "half" else (lambda p, q: torch.stack((p, q), -1).flatten(-2))
    y = torch.cat((join(u, w), x[..., rot:]), -1)
    pair = torch.cat((join(h, h), x[..., rot:].abs()), -1)
    still = torch.cat((join(t == 0, t == 0).expand_as(y[..., :rot]), torch.ones_like(y[..., rot:], dtype=torch.bool)), -1)
    want, byte = more.held(y)
    # (as for text: an element of a third of its pair or more, and no subnormal code; of what is not turned, all)
    exact = still & (m in (1.0, 1.25))
    sure = exact | ((y.abs() >= pair / 3) & (y.abs() >= torch.exp2(byte[..., None].double() - 127 - 6)))
    wrong = (got != want.to(dtype).double()) & sure
    assert still.double().mean() > 0.3 and not wrong.any(), int(wrong.sum())
