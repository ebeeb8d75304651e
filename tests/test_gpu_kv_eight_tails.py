"""Attention over a cache of 8 bits where one key has most of a row's weight and the
rest of a long history shares what is left: on both sides of what the kernel for few
rows takes, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import kv_more_reference as more
from test_gpu_kv import BF16, F16, half_step, i32, make, queries
from test_gpu_kv_eight import E4M3, exponents, gathered, make8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


def one_history(ss, dev, n, T, page, D, dtype, seed=0):
    """n sequences of T committed tokens on the same pages, a page of its own for each
    one's new token; codes and scales of nothing yet."""
    P = T // page
    table = i32(np.concatenate((np.tile(np.arange(P), (n, 1)), P + np.arange(n)[:, None]), 1), dev)
    pages = P + n
    refs = i32([n] * P + [1] * n, dev)
    code = lambda: torch.zeros((1, pages, 1, page, D), dtype=torch.uint8, device=dev)  # noqa: E731
    scale = lambda: torch.full((1, pages, 1, page), 127, dtype=torch.uint8, device=dev)  # noqa: E731
    c = ss.KVCache.wrap(code().view(E4M3), code().view(E4M3), table, i32([T] * n, dev), i32([P + 1] * n, dev), refs,
                        torch.zeros((pages + 31) // 32, dtype=torch.int32, device=dev), scale(), scale(), dtype)
    return c, table.cpu().numpy()


def bound(out, mag, v2, T, rows, apart=True):
    """Half a step of the output, and of each weight; then what adds up.

    A weight that the kernel for few rows takes as parts is off besides by a rounding to
    2^-13 of a unit (fp16: 2^-17) in which the row's largest is at least 2^7.5 where one
    key exceeds the others by 2^7.5 (fp16: 2^5.5), else 2^4 (2^2): up or down by where a
    number that runs through all of a step falls, so of mean zero and a standard
    deviation of at most half a step.  Such errors of the keys add up like sqrt(sum v^2) of
    them; 6 of those.  (Another such rounding, to 2^-24 of the unit, is nothing beside it.)

    fp32: scores as they are here (magnitudes up to 2^5, 2 D products of which two are not
    zero) are off by 2^-17, the exponential by 2^-21.  A matrix instruction aligns its
    products to the sum that it adds them to and cuts what is below that one's last place,
    2^-23 of it, each time the same way where values have one sign; each half of the
    blocks has a sum of its own.  Past 32 rows, weights of 16 bits, that may be each of T / 2
    products (as for a cache of 16 bits).  Up to 32 rows products of codes are multiples of
    2^-9 times the 2^-3 that these values are multiples of, and a sum below 2^11 has all of
    those: what is cut is at most each of 32 keys' sum beyond that."""
    u = half_step(out.dtype)
    added = T / 2 / (32 if rows <= 32 else 1)
    step = 2.0 ** -13 / 2.0 ** (7.5 if apart else 4) if out.dtype == BF16 else 2.0 ** -17 / 2.0 ** (5.5 if apart else 2)
    return u * out.double().abs() + (u + 2.0 ** -16 + added * 2.0 ** -23) * mag + 6 * step / 2 * v2 + 2.0 ** -24


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (BF16, 64), (F16, 64), (F16, 128)])
@pytest.mark.parametrize("T,n", [(4096, 152), (32768, 152), (131072, 152), (131072, 3), (1 << 20, 152)])
@pytest.mark.parametrize("at", ["first", "middle", "last", "four"])
def test_one_key_and_a_long_flat_rest(ss, cuda_device, dtype, D, T, n, at):
    """Rows whose other keys have 2^-8 to 2^-26 of the largest weight each, values of
    all ones, ones but for that key, of one sign, and of both; units that one CTA works
    on (152 of them) and such as many share; 1, 16, 32 and 33 rows a unit.  "four": such
    keys among each 32 of the first 128."""
    dev, page = cuda_device, 128
    c, table = one_history(ss, dev, n, T, page, D, dtype)
    g = torch.Generator(device=dev).manual_seed(T)
    peak = {"first": [0], "middle": [T // 2 + 77], "last": [T - 1], "four": [5, 40, 70, 127]}[at]
    z = torch.arange(T, device=dev)
    k = torch.zeros((T, D), dtype=torch.float64, device=dev)
    k[:, 0] = -1.0      # weight 2^(-q0), but for
    k[peak, 0] = 0.0
    k[:, 1] = torch.randint(-8, 9, (T,), generator=g, device=dev).double() / 8
    k[peak, 1] = 0.0
    v = torch.ones((T, D), dtype=torch.float64, device=dev)
    v[peak, 1::4] = 0.0
    rand = torch.randint(8, 16, (T, D), generator=g, device=dev).double() / 8
    v[:, 2::4] = rand[:, 2::4]
    v[:, 3::4] = rand[:, 3::4] * (1 - 2.0 * torch.randint(0, 2, (T, 1), generator=g, device=dev))
    pg, where = i32(table[0], dev).long()[z // page], z % page
    for pool, x in ((c.k, k), (c.v, v)):
        pool.view(torch.uint8)[0, pg, 0, where] = x.float().to(E4M3).view(torch.uint8)
    # new tokens: as the first value, and as keys of the rest
    c.v.view(torch.uint8)[0, T // page:] = c.v.view(torch.uint8)[0, pg[0], 0, where[0]]
    c.k.view(torch.uint8)[0, T // page:, 0, :, 0] = 0xb8
    assert torch.equal(gathered(c, table, 0, n - 1, T)[0][:, 0], k)
    for rows in (1, 16, 32, 33):
        e = torch.linspace(8, 26, rows, device=dev) if rows > 1 else torch.tensor([18.5], device=dev)
        q = torch.zeros((n, 1, rows, D), dtype=dtype, device=dev)
        q[:, 0, :, 0] = (e * 4).round().to(dtype) / 4
        q[:, 0, ::2, 1] = 0.5     # every second row's weights differ by up to 2^0.5 either way
        plan = c.plan(1, rows)
        out = c.attend(0, plan, q, scale=math.log(2.0))
        assert (plan.status == 0).all()
        kk, vv = (x[:, 0] for x in gathered(c, table, 0, 0, T + 1))
        s = q[0, 0].double() @ kk.T     # in powers of two
        p = torch.exp2(s - s.amax(1, keepdim=True))
        p /= p.sum(1, keepdim=True)
        want, mag = p @ vv, p @ vv.abs()
        tol = bound(out[0, 0], mag, (vv * vv).sum(0).sqrt() * p.amax(1, keepdim=True), T, rows, at != "four")
        d = (out[:, 0].double() - want).abs()
        assert torch.isfinite(out).all()
        assert (d <= tol).all(), f"{rows} rows: {float((d / tol).max()):.2f} of the bound, {float(d.max()):.2e} off"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T", [16384, 32768])
@pytest.mark.parametrize("nats", [10.0, 12.0, 14.0])
def test_one_key_and_others_about_one_score_on_both_sides_of_32_rows(ss, cuda_device, dtype, T, nats):
    """A first key so many nats above the others, whose values share a mean: the same
    relative error, as a vector, by either kernel."""
    dev, page, D, n = cuda_device, 64, 64, 152
    c, table = one_history(ss, dev, n, T, page, D, dtype)
    g = torch.Generator(device=dev).manual_seed(int(nats))
    z = torch.arange(T, device=dev)
    k = torch.randn((T, D), generator=g, device=dev) / 8
    k[:, 0] = -1.0
    k[0] = 0.0
    v = 0.75 + torch.randn((T, D), generator=g, device=dev) / 4
    v[0] = torch.randn(D, generator=g, device=dev)
    pg, where = i32(table[0], dev).long()[z // page], z % page
    for pool, x in ((c.k, k), (c.v, v)):
        pool.view(torch.uint8)[0, pg, 0, where] = x.to(E4M3).view(torch.uint8)
    kk, vv = (x[:, 0] for x in gathered(c, table, 0, 0, T + 1))
    for rows in (32, 33):
        q = torch.randn((1, 1, rows, D), generator=g, device=dev).expand(n, 1, rows, D).to(dtype).contiguous()
        q[..., 0] = nats
        out = c.attend(0, c.plan(1, rows), q, scale=1.0)
        p = torch.softmax(q[0, 0].double() @ kk.T, -1)
        want = p @ vv
        # (as above, each row's error as a vector)
        tol = bound(want.to(dtype), p @ vv.abs(), (vv * vv).sum(0).sqrt() * p.amax(1, keepdim=True), T, rows)
        tol = tol.norm(dim=-1)
        d = (out[:, 0].double() - want).norm(dim=-1)
        assert (d <= tol).all(), f"{rows} rows: {float((d / tol).max()):.2f} of the bound"


def test_masked_keys_have_no_weight_whatever_is_added(ss, cuda_device):
    """Values of 448 behind what a token sees, and before its window: not one of their
    weights is anything but zero."""
    dev, N, Q, H, D, lens = cuda_device, 4, 8, 2, 64, [2, 126, 127, 128, 700, 1025]
    for dtype in (BF16, F16):
        for window, sinks in ((None, 0), (50, 2)):
            c, table = make8(ss, dev, lens, [N] * len(lens), 32, H, D, dtype)
            plan = c.plan(N, Q, n_tok=i32([1] * len(lens), dev), window=window, sinks=sinks)
            q = queries(len(lens), N, Q, D, dtype, dev)
            want = c.attend(0, plan, q)
            seen = torch.zeros((c.pages, 32), dtype=torch.bool, device=dev)
            for b, n in enumerate(lens):
                for t in np.nonzero(more.window_sight(n, 1, window, sinks).any(0))[0]:
                    seen[int(table[b, t // 32]), t % 32] = True
            dead = ~seen[None, :, None, :].expand_as(c.v_scale)
            c.v.view(torch.uint8)[dead] = 0x7e
            c.v_scale[dead] = 134
            assert torch.equal(c.attend(0, plan, q), want)


def test_eight_is_what_sixteen_bits_give_with_fewer_tokens_than_planned_for(ss, cuda_device):
    """80 rows a unit of which 12 take part: the kernel for more rows, so the same as a
    16-bit cache of the same values."""
    dev, N, Q, H, D = cuda_device, 20, 8, 2, 128
    lens = [0, 130, 900, 3000]
    for dtype in (BF16, F16):
        c, table = make8(ss, dev, lens, [N] * 4, 64, H, D, dtype)
        wide = [more.values(x.view(torch.uint8), s).to(dtype) for x, s in ((c.k, c.k_scale), (c.v, c.v_scale))]
        w = ss.KVCache.wrap(*wide, c.table, c.lens, c.held, c.refs, c.free)
        q = queries(4, N, Q, D, dtype, dev)
        for window in (None, 200):
            few = c.plan(N, Q, n_tok=i32([3] * 4, dev), window=window)
            out = c.attend(0, few, q)
            assert torch.equal(out, w.attend(0, few, q)) and (out[:, :3] != 0).any()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,Q,H,N", [(128, 8, 2, 4), (64, 8, 1, 4), (128, 8, 1, 8), (64, 64, 2, 1)])
def test_a_sequence_alone_gives_what_it_gives_in_a_batch(ss, cuda_device, dtype, D, Q, H, N):
    """Bit for bit where one CTA has a unit in both, which a history of one block makes
    sure of (no share begins inside a block); by the bound for longer ones."""
    dev, lens = cuda_device, [5, 120, 64, 0, 77, 900]
    c, table = make8(ss, dev, lens, [N] * len(lens), 64, H, D, dtype)
    q = queries(len(lens), N, Q, D, dtype, dev)
    out = c.attend(0, c.plan(N, Q), q)
    for b, n in enumerate(lens):
        one = c.attend(0, c.plan(N, Q, rows=i32([b], dev)), q[b:b + 1].contiguous())
        if n + N <= 128:
            assert torch.equal(one[0], out[b]), b
        for got in (one[0], out[b]):
            k, v = (x.to(dtype) for x in gathered(c, table, 0, b, n + N))
            more.check(got, q[b], k, v, more.window_sight(n, N, None, 0), exponents=exponents(c, table, 0, b, n + N))
