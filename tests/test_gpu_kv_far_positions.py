"""Rotary append at positions up to the ends of 32 bits, against angles that are reduced
in integers: the codes of a cache of 8 bits tell them apart to the last bits."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import kv_more_reference as more
from test_gpu_kv import BF16, F16, half_step, i32, make
from test_gpu_kv_eight import make8

pytestmark = pytest.mark.gpu
BITS = 200
TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234,
                  10 ** 96)


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


def test_two_pi_is_two_pi():
    # Machin's: pi / 4 = 4 arctan(1 / 5) - arctan(1 / 239)
    def arctan(n):
        t, s, k = (1 << 400) // n, (1 << 400) // n, 1
        while t:
            t //= -n * n
            k += 2
            s += t // k
        return s
    got = Fraction(8 * (4 * arctan(5) - arctan(239)), 1 << 400)
    assert abs(got - TWO_PI) < Fraction(1, 10 ** 95)


def angles(pos, freq):
    """[..., pairs] radians in [0, 2 pi), 64 bits: pos a list of integers."""
    turn = [int(Fraction(f) / TWO_PI * (1 << BITS)) for f in freq]
    mask = (1 << BITS) - 1
    # (off by |pos| 2^-200 turns, and a double's half step)
    return np.array([[float(Fraction((p * t) & mask, 1 << BITS)) for t in turn] for p in pos]) * (2 * np.pi)


def turned(x, t, layout, m):
    """x [n, heads, D] in 64 bits, t [n, D / 2]: and the pairs' magnitudes."""
    D = x.shape[-1]
    a, b = (x[..., :D // 2], x[..., D // 2:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    c, s = (torch.as_tensor(f(t), device=x.device)[:, None] * m for f in (np.cos, np.sin))
    u, w, h = a * c - b * s, a * s + b * c, torch.hypot(a, b) * abs(m)
    if layout == "half":
        return torch.cat((u, w), -1), torch.cat((h, h), -1)
    return torch.stack((u, w), -1).flatten(-2), h.repeat_interleave(2, -1)


def far_positions(rng, N):
    pos = rng.integers(-2 ** 31, 2 ** 31, N)
    pos[:8] = [2 ** 31 - 1, -2 ** 31, 2 ** 30, -2 ** 30, 1, -1, 0, 2 ** 24 + 1]
    return pos


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,D,m", [(BF16, 128, 1.0), (F16, 64, 1.0), (F16, 128, 1.25)])
def test_codes_of_keys_turned_far_are_those_of_exact_ones(ss, cuda_device, layout, dtype, D, m):
    """Frequencies of about one radian and more, where an angle is the hardest to have.  The
    kernel's angles are off by 2^-31 at most, the reference's by 2^-50: none of the 10^6
    elements lies that close to a tie but by a chance of 10^-3 (an element's ties lie 2^-4 of
    it apart, 2^5 * 2^-31 a chance of 2^-26 where it is off by so much)."""
    dev, N, H = cuda_device, 1024, 8
    rng = np.random.default_rng(D)
    c, _ = make8(ss, dev, [3], [N], 64, H, D, dtype)
    g = torch.Generator(device=dev).manual_seed(D)
    k = torch.randn((1, N, H, D), generator=g, device=dev).to(dtype)
    freq = rng.uniform(0.3, 6.0, D // 2)
    freq[:4] = [1.0, 2.0 ** -20 / 3, 1e-4, 123456.789]
    pos = far_positions(rng, N)
    c.append(0, c.plan(N, H), None, k, k, ss.Rope(torch.as_tensor(freq, device=dev), layout, m),
             positions=i32(pos[None], dev))
    got = c.read(0, None, i32([3], dev), N)[0][0]
    y, pair = turned(k[0].double(), angles([int(p) for p in pos], freq), layout, m)
    want, byte = more.held(y)
    sure = (y.abs() >= pair / 3) & (y.abs() >= torch.exp2(byte[..., None].double() - 127 - 6))
    assert sure.double().mean() > 0.7
    wrong = (got.double() != want.to(dtype).double()) & sure
    assert not wrong.any(), int(wrong.sum())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_queries_and_keys_of_16_bits_turned_far(ss, cuda_device, layout):
    """Half a step of fp16, and fp32's 16 / 3 * 2^-24 of a pair."""
    dev, N, H, D = cuda_device, 300, 2, 64
    rng = np.random.default_rng(1)
    c, table = make(ss, dev, [0], [N], 64, H, D, F16)
    g = torch.Generator(device=dev).manual_seed(1)
    q, k = (torch.randn((1, N, h, D), generator=g, device=dev).to(F16) for h in (4, H))
    freq = rng.uniform(0.3, 6.0, D // 2)
    pos = far_positions(rng, N)
    out = c.append(0, c.plan(N, 4), q, k, k, ss.Rope(torch.as_tensor(freq, device=dev), layout), positions=i32(pos[None], dev))
    t = angles([int(p) for p in pos], freq)
    at = torch.arange(N, device=dev)
    keys = c.k[0][i32(table[0], dev).long()[at // 64], :, at % 64]
    for got, x in ((out[0], q[0]), (keys, k[0])):
        y, pair = turned(x.double(), t, layout, 1.0)
        tol = half_step(F16) * y.abs() + 16 / 3 * 2.0 ** -24 * pair * (1 + half_step(F16)) + 2.0 ** -25
        assert ((got.double() - y).abs() <= tol).all(), float(((got.double() - y).abs() / tol).max())
