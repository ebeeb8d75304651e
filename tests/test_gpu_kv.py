"""The paged cache on the GPU: bookkeeping against plain integers, the rotary
append and the attention against 64 bits."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def i32(a, dev):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)


def make(ss, dev, lens, n_tok, page=64, H=2, D=128, dtype=BF16, layers=1, shared=None, seed=0, spare=3, fill=None):
    """A cache whose pages lie anywhere in the pool.  shared: (group ids, tokens
    that each group's members share).  fill: what slots that hold no token
    contain (None: other tokens' values)."""
    rng = np.random.default_rng(seed)
    n = len(lens)
    hold = [-(-(a + b) // page) for a, b in zip(lens, n_tok)]
    mp = max(max(hold), 1)
    table = np.full((n, mp), -1, np.int64)
    used = 0
    for b in range(n):
        s = 0
        if shared is not None:
            lead = shared[0].index(shared[0][b])
            if lead < b:
                s = min(shared[1] // page, lens[b] // page, lens[lead] // page)
                table[b, :s] = table[lead, :s]
        table[b, s:hold[b]] = np.arange(used, used + hold[b] - s)
        used += hold[b] - s
    pages = used + spare
    perm = rng.permutation(pages)
    table = np.where(table >= 0, perm[np.clip(table, 0, None)], -1)
    refs = np.bincount(table[table >= 0], minlength=pages)
    g = torch.Generator(device=dev).manual_seed(seed)
    k = torch.randn((layers, pages, H, page, D), generator=g, device=dev).to(dtype)
    v = torch.randn((layers, pages, H, page, D), generator=g, device=dev).to(dtype)
    if fill is not None:
        live = torch.zeros((pages, page), dtype=torch.bool)
        for b in range(n):
            for t in range(lens[b] + n_tok[b]):
                live[table[b, t // page], t % page] = True
        dead = (~live).to(dev)
        k[:, dead.nonzero()[:, 0], :, dead.nonzero()[:, 1]] = fill
        v[:, dead.nonzero()[:, 0], :, dead.nonzero()[:, 1]] = fill
    m = ref.Pages(pages, page, n, mp)
    m.refs = refs
    c = ss.KVCache.wrap(k, v, i32(table, dev), i32(lens, dev), i32(hold, dev), i32(refs, dev), i32(m.free_bits(), dev))
    return c, table


def gathered(c, table, layer, b, T):
    at = torch.arange(T, device=c.device)
    pg = torch.as_tensor(table[b], device=c.device)[at // c.page]
    return c.k[layer][pg, :, at % c.page], c.v[layer][pg, :, at % c.page]


def check_attend(c, table, q, out, lens, n_tok, parent=None, scale=None, layer=0, status=None):
    n, N, Q, D = q.shape
    u = half_step(q.dtype)
    for b in range(n):
        T = n_tok[b]
        assert (out[b, T:] == 0).all(), f"sequence {b}: tokens behind its last are zeros"
        if T == 0:
            continue
        k, v = gathered(c, table, layer, b, lens[b] + T)
        see = np.tril(np.ones((T, T), bool)) if parent is None else ref.sight(parent[b])[0]
        o, mag, e = ref.attend(q[b, :T], k, v, lens[b], see, scale or 1 / math.sqrt(D))
        tol = u * o.abs() + (u + e) * mag + 2.0 ** -24
        d = (out[b, :T].double() - o).abs()
        assert torch.isfinite(out[b, :T]).all(), f"sequence {b}"
        assert (d <= tol).all(), f"sequence {b}: {float((d / tol).max()):.2f} of the bound"


def queries(n, N, Q, D, dtype, dev, seed=1, gain=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn((n, N, Q, D), generator=g, device=dev) * gain).to(dtype)


LENS = [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 255, 256, 300, 517, 1000]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page,D,Q,H", [(16, 128, 8, 2), (64, 64, 4, 4), (32, 64, 15, 3), (128, 128, 16, 1), (64, 128, 7, 1)])
@pytest.mark.parametrize("N", [1, 4, 21])
def test_attend_chains(ss, cuda_device, dtype, page, D, Q, H, N):
    rng = np.random.default_rng(N + D)
    n_tok = [int(x) for x in rng.integers(0, N + 1, len(LENS))]
    n_tok[0], n_tok[3] = N, N
    c, table = make(ss, cuda_device, LENS, n_tok, page, H, D, dtype, seed=N)
    q = queries(len(LENS), N, Q, D, dtype, cuda_device, gain=2.0)
    plan = c.plan(N, Q, n_tok=i32(n_tok, cuda_device))
    out = c.attend(0, plan, q)
    assert (plan.status == 0).all()
    check_attend(c, table, q, out, LENS, n_tok)


@pytest.mark.parametrize("N,Q,H,page,D", [(8, 16, 2, 16, 128), (32, 8, 1, 64, 128), (32, 12, 2, 32, 64), (1, 2, 2, 64, 64),
                                          (13, 5, 1, 128, 128)])
def test_attend_trees(ss, cuda_device, N, Q, H, page, D):
    rng = np.random.default_rng(N)
    n = len(LENS)
    parent = ref.random_parents(rng, n, N)
    fc, ns = ref.links(parent)
    c, table = make(ss, cuda_device, LENS, [N] * n, page, H, D, seed=N)
    q = queries(n, N, Q, D, BF16, cuda_device)
    plan = c.plan(N, Q, tree=(i32(fc, cuda_device), i32(ns, cuda_device)))
    out = c.attend(0, plan, q)
    assert (plan.status == 0).all()
    check_attend(c, table, q, out, LENS, [N] * n, parent)


@pytest.mark.parametrize("seed", range(5))
def test_attend_many_small_shapes(ss, cuda_device, seed):
    """Few blocks, odd head counts and lengths: shares of single blocks, units cut
    in two and three, tiles of whole tokens that leave rows over."""
    rng = np.random.default_rng(seed)
    for _ in range(14):
        n, rep = int(rng.integers(1, 5)), int(rng.choice([1, 2, 3, 5, 7, 8, 20, 43, 48, 64]))
        H, page, D = int(rng.choice([1, 1, 2, 3])), int(rng.choice([16, 32, 64, 128])), int(rng.choice([64, 128]))
        N = int(rng.integers(1, 1 + max(1, 600 // rep)))
        lens = [int(x) for x in rng.integers(0, int(rng.choice([2, 100, 700])), n)]
        n_tok = [int(x) for x in rng.integers(0, N + 1, n)]
        n_tok[0] = N
        c, table = make(ss, cuda_device, lens, n_tok, page, H, D, F16 if rng.random() < 0.5 else BF16, seed=seed)
        q = queries(n, N, H * rep, D, c.dtype, cuda_device, gain=1.5)
        plan = c.plan(N, H * rep, n_tok=i32(n_tok, cuda_device))
        assert (plan.status == 0).all()
        check_attend(c, table, q, c.attend(0, plan, q), lens, n_tok)


def test_a_pool_past_four_gigabytes(ss, cuda_device):
    """Pages at both ends of pools of 5.6 GB and two layers: append, attend, copy on
    write and commit all reach them."""
    dev, page, H, D, N = cuda_device, 128, 8, 128, 5
    pages = 10_700
    c = ss.KVCache(2, pages, page, H, D, 3, 4, device=dev)
    assert c.k.numel() * 2 > 5.6e9
    # every page but the first and the last few is someone else's
    c.refs[2:pages - 6] = 1
    words = torch.zeros(((pages + 31) // 32, 32), dtype=torch.int64)
    free = torch.zeros(pages, dtype=torch.bool)
    free[:2], free[pages - 6:] = True, True
    words.view(-1)[:pages] = free.long()
    w = (words << torch.arange(32)).sum(1)
    c.free.copy_(torch.where(w >= 1 << 31, w - (1 << 32), w).int())
    rows = i32([0], dev)
    lens = 3 * page - 40
    assert c.reserve(rows, lens).tolist() == [0]
    assert c.table[0, :3].tolist() == [0, 1, pages - 6]
    held = c.table[0, :3].long()
    for x in (c.k, c.v):
        x[:, held] = torch.randn((2, 3, H, page, D), generator=torch.Generator(device=dev).manual_seed(1),
                                 device=dev).to(BF16)
    c.commit(rows, i32([lens - 1], dev))
    c.fork(i32([0, 0], dev), i32([1, 2], dev))
    assert c.reserve(None, N).tolist() == [0, 0, 0]
    assert sorted(c.table[:, 2].tolist()) == [pages - 5, pages - 4, pages - 3]
    q, k, v = (queries(3, N, h, D, BF16, dev, seed=s) for s, h in ((1, 16), (2, H), (3, H)))
    parent = np.array([[-1, 0, 0, 1, 3]] * 3)
    fc, ns = ref.links(parent)
    plan = c.plan(N, 16, tree=(i32(fc, dev), i32(ns, dev)), group=i32([0, 0, 0], dev))
    assert (plan.status == 0).all()
    c.append(1, plan, None, k, v)
    table = c.table.cpu().numpy()
    out = c.attend(1, plan, q)
    check_attend(c, table, q, out, [lens] * 3, [N] * 3, parent, layer=1)
    want = torch.cat((gathered(c, table, 1, 2, lens)[1], v[2, [0, 1, 3, 4]]))
    assert c.commit(None, i32([3, 3, 3], dev), i32([[1, 3, 4, -1, -1]] * 3, dev)).tolist() == [0, 0, 0]
    assert torch.equal(gathered(c, c.table.cpu().numpy(), 1, 2, lens + 4)[1], want)


def test_a_plan_used_too_late_stays_inside_the_pool(ss, cuda_device):
    """A plan whose sequence was emptied behind its back: what it gives is undefined,
    but nothing outside the pool is read or written, and nothing of others is."""
    dev = cuda_device
    c, table = make(ss, dev, [70, 70], [4, 4], 16, 1, 64)
    q, k = queries(2, 4, 2, 64, BF16, dev), queries(2, 4, 1, 64, BF16, dev)
    plan = c.plan(4, 2)
    c.truncate(i32([0], dev))
    before = c.k.clone()
    got = c.append(0, plan, q, k, k)
    assert (got[0] == 0).all() and torch.equal(got[1], q[1])
    changed = (before != c.k)[0].flatten(1).any(1).nonzero()[:, 0].tolist()
    assert set(changed) <= {int(x) for x in table[1]}
    c.attend(0, plan, q)
    torch.cuda.synchronize()


@pytest.mark.parametrize("N,Q,H,shared", [(4, 16, 2, 512), (1, 4, 4, 64), (3, 7, 1, 130), (8, 64, 2, 1000)])
@pytest.mark.parametrize("page", [16, 64])
def test_attend_groups(ss, cuda_device, N, Q, H, shared, page):
    rng = np.random.default_rng(shared)
    ids = [5] * 7 + [2] + [9] * 12 + [5] * 3 + [4] * 2
    n = len(ids)
    # the second run of 5s begins again: it shares nothing with the first
    run = [i if i < 20 else i for i in ids]
    lens = [int(shared + x) for x in rng.integers(0, 400, n)]
    lens[-1] = 3    # one member shorter than what the others share
    n_tok = [int(x) for x in rng.integers(0, N + 1, n)]
    n_tok[1] = 0
    n_tok[0] = n_tok[8] = n_tok[20] = n_tok[22] = N
    keys = [0] * 7 + [1] + [2] * 12 + [3] * 3 + [4] * 2
    c, table = make(ss, cuda_device, lens, n_tok, page, H, 128, shared=(keys, shared), seed=shared)
    q = queries(n, N, Q, 128, BF16, cuda_device)
    nt = i32(n_tok, cuda_device)
    for group in (run, [1] * n, list(range(n))):   # any grouping is right: what is shared is found in the tables
        plan = c.plan(N, Q, n_tok=nt, group=i32(group, cuda_device))
        out = c.attend(0, plan, q)
        assert (plan.status == 0).all()
        check_attend(c, table, q, out, lens, n_tok)


@pytest.mark.parametrize("n,N,Q,H,lens", [(3, 300, 8, 2, [0, 77, 700]), (1, 1000, 6, 1, [129]), (2, 513, 4, 4, [64, 5])])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_prompt_chunks(ss, cuda_device, n, N, Q, H, lens, D):
    n_tok = [N] + [N - 11 * b for b in range(1, n)]
    c, table = make(ss, cuda_device, lens, n_tok, 32, H, D, F16, seed=N)
    q = queries(n, N, Q, D, F16, cuda_device)
    plan = c.plan(N, Q, n_tok=i32(n_tok, cuda_device))
    check_attend(c, table, q, c.attend(0, plan, q), lens, n_tok)


def test_attend_long_and_peaked(ss, cuda_device):
    """Scores far apart, rising along the keys (the running maximum moves all the
    way), and a history over many CTAs."""
    lens, n_tok = [20000, 4097], [4, 2]
    c, table = make(ss, cuda_device, lens, n_tok, 64, 1, 128, seed=3)
    ramp = torch.linspace(0.1, 3.0, 20004, device=cuda_device)
    at = torch.arange(20004, device=cuda_device)
    pg = torch.as_tensor(table[0], device=cuda_device)[at // 64]
    c.k[0, pg, 0, at % 64] = (ramp[:, None] * torch.ones(128, device=cuda_device)).to(BF16)
    q = queries(2, 4, 8, 128, BF16, cuda_device).abs()
    plan = c.plan(4, 8, n_tok=i32(n_tok, cuda_device))
    check_attend(c, table, q, c.attend(0, plan, q), lens, n_tok)
    check_attend(c, table, q, c.attend(0, plan, q, scale=0.9), lens, n_tok, scale=0.9)


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("N", [1, 7, 200])
def test_what_no_token_sees_does_not_reach_it(ss, cuda_device, fill, N):
    """Slots without a token, and new tokens outside a token's sight, may hold
    anything."""
    lens = [0, 5, 64, 100, 127, 128, 250]
    n = len(lens)
    n_tok = [max(1, N - b) for b in range(n)]
    c, table = make(ss, cuda_device, lens, n_tok, 64, 2, 128, fill=fill, seed=N)
    q = queries(n, N, 6, 128, BF16, cuda_device)
    plan = c.plan(N, 6, n_tok=i32(n_tok, cuda_device))
    check_attend(c, table, q, c.attend(0, plan, q), lens, n_tok)
    # the last new token of each sequence spoiled: the ones before do not see it, it sees itself
    for b in range(n):
        t = lens[b] + n_tok[b] - 1
        c.v[0, table[b, t // 64], :, t % 64, 3:50] = fill
        c.k[0, table[b, t // 64], :, t % 64] = 0
    out = c.attend(0, plan, q)
    check_attend(c, table, q, torch.where(torch.arange(N, device=cuda_device)[None, :, None, None] <
                                          i32(n_tok, cuda_device)[:, None, None, None] - 1, out, 0.0),
                 lens, [t - 1 for t in n_tok])
    for b in range(n):
        got = out[b, n_tok[b] - 1, :, 3:50].float()
        if math.isnan(fill):
            assert got.isnan().all()
        elif math.isinf(fill):
            assert (got == fill).all()
        assert out[b, n_tok[b] - 1, :, 50:].isfinite().all()


@pytest.mark.parametrize("D,N,lens", [(64, 1, [0, 1, 129]), (128, 5, [700, 5000, 130]), (128, 90, [3, 260, 9])])
@pytest.mark.parametrize("group", [None, [0, 0, 0]])
def test_scores_of_minus_infinity(ss, cuda_device, D, N, lens, group):
    """Keys that score -infinity take no weight, in blocks of nothing else too; a
    query that sees no other gets zeros."""
    dev = cuda_device
    shared = (group, 2 * 64) if group else None
    c, table = make(ss, dev, lens, [N] * 3, 64, 1, D, shared=shared, seed=9)
    q = queries(3, N, 4, D, BF16, dev).abs() + 0.25
    g = i32(group, dev) if group else None
    c.k.abs_()
    c.k[..., 0] = -math.inf
    plan = c.plan(N, 4, group=g)
    assert (c.attend(0, plan, q) == 0).all()
    # the last 3 tokens of each history, and the new ones, are seen by score
    for b in range(3):
        for t in range(max(0, lens[b] - 3), lens[b] + N):
            c.k[0, table[b, t // 64], :, t % 64, 0] = 0.5
    out = c.attend(0, plan, q)
    u = half_step(BF16)
    for b in range(3):
        k, v = gathered(c, table, 0, b, lens[b] + N)
        keep = torch.isfinite(k[:, 0, 0])
        base = int(keep[:lens[b]].sum())
        o, mag, e = ref.attend(q[b], k[keep], v[keep], base, np.tril(np.ones((N, N), bool)), 1 / math.sqrt(D))
        e = e + 2 * (lens[b] + N) * 2.0 ** -23   # (sums over the others' zeros too)
        assert ((out[b].double() - o).abs() <= u * o.abs() + (u + e) * mag + 2.0 ** -24).all()


@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_siblings_do_not_see_each_other(ss, cuda_device, fill):
    rng = np.random.default_rng(4)
    N, lens = 16, [0, 30, 64, 120, 200]
    n = len(lens)
    parent = ref.random_parents(rng, n, N)
    fc, ns = ref.links(parent)
    c, table = make(ss, cuda_device, lens, [N] * n, 32, 1, 64, seed=2)
    bad = 6
    for b in range(n):
        t = lens[b] + bad
        c.k[0, table[b, t // 32], :, t % 32] = fill
        c.v[0, table[b, t // 32], :, t % 32] = fill
    q = queries(n, N, 4, 64, BF16, cuda_device)
    plan = c.plan(N, 4, tree=(i32(fc, cuda_device), i32(ns, cuda_device)))
    out = c.attend(0, plan, q)
    u = half_step(BF16)
    for b in range(n):
        see, _ = ref.sight(parent[b])
        k, v = gathered(c, table, 0, b, lens[b] + N)
        k, v = k.clone(), v.clone()
        k[lens[b] + bad], v[lens[b] + bad] = 0, 0
        o, mag, e = ref.attend(q[b], k, v, lens[b], see & (np.arange(N) != bad)[None], 1 / 8)
        blind = ~torch.as_tensor(see[:, bad], device=cuda_device)
        d = (out[b].double() - o).abs()
        assert (d <= u * o.abs() + (u + e) * mag + 2.0 ** -24)[blind].all()
        assert not out[b][~blind].isfinite().any()


def test_attend_takes_views_buffers_layers_and_other_streams(ss, cuda_device):
    lens, n_tok, N, Q, H, D = [70, 300], [4, 3], 4, 8, 2, 64
    c, table = make(ss, cuda_device, lens, n_tok, 64, H, D, layers=3, seed=5)
    wide = queries(2, N, Q + 2 * H + 1, D, BF16, cuda_device)
    q = wide[:, :, 1:Q + 1]
    nt = i32(n_tok, cuda_device)
    plan = c.plan(N, Q, n_tok=nt)
    buf = torch.full((2, N, Q, D), 7.0, dtype=BF16, device=cuda_device)
    for layer in (2, 0, 1):
        assert c.attend(layer, plan, q, out=buf) is buf
        check_attend(c, table, q, buf, lens, n_tok, layer=layer)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = c.attend(1, c.plan(N, Q, n_tok=nt), q)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, buf)
    # rows in another order, a part of them
    rows = i32([1], cuda_device)
    out1 = c.attend(1, c.plan(N, Q, rows=rows, n_tok=nt[1:].clone()), q[1:])
    check_attend(c, table[1:], q[1:], out1, lens[1:], n_tok[1:], layer=1)


def test_attend_is_the_same_every_time(ss, cuda_device):
    lens, n_tok, N = [3000, 40, 900, 901], [4, 4, 1, 3], 4
    c, _ = make(ss, cuda_device, lens, n_tok, 64, 2, 128, shared=([0] * 4, 32), seed=6)
    q = queries(4, N, 16, 128, BF16, cuda_device)
    nt = i32(n_tok, cuda_device)
    first = c.attend(0, c.plan(N, 16, n_tok=nt), q)
    for _ in range(20):
        assert torch.equal(first, c.attend(0, c.plan(N, 16, n_tok=nt), q))


def test_a_captured_step_follows_the_cache(ss, cuda_device):
    """plan, append, attend and commit captured once, replayed as the cache grows."""
    n, N, Q, H, D = 3, 4, 4, 2, 64
    c = ss.KVCache(1, 40, 16, H, D, n, 12, device=cuda_device)
    e = ss.KVCache(1, 40, 16, H, D, n, 12, device=cuda_device)
    f, m = ss.rope_frequencies(D)
    rope = ss.Rope(f.to(cuda_device), "half", m)
    q, k, v = (queries(n, N, h, D, BF16, cuda_device, seed=s) for s, h in ((1, Q), (2, H), (3, H)))
    acc = i32([0, 1, 3], cuda_device)

    def step(x):
        x.reserve(None, N)
        plan = x.plan(N, Q)
        qr = x.append(0, plan, q, k, v, rope)
        o = x.attend(0, plan, qr)
        x.commit(None, acc)
        return o, plan.status

    warm = ss.KVCache(1, 40, 16, H, D, n, 12, device=cuda_device)
    step(warm)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, status = step(c)
    for r in range(9):
        q.normal_()
        k.normal_()
        g.replay()
        want, _ = step(e)
        assert (status == 0).all()
        assert torch.equal(out, want), r
        for x in ("table", "lens", "held", "refs", "free"):
            assert torch.equal(getattr(c, x), getattr(e, x)), (r, x)


def test_plans_that_are_held_keep_their_memory(ss, cuda_device):
    """A plan's memory is used again only once nothing of it can be read."""
    lens = [100, 300, 17]
    c, table = make(ss, cuda_device, lens, [4] * 3, 64, 2, 64)
    q = queries(3, 4, 8, 64, BF16, cuda_device)
    one, two = c.plan(4, 8), c.plan(4, 8, n_tok=i32([1, 2, 3], cuda_device))
    assert one.ptr != two.ptr
    check_attend(c, table, q, c.attend(0, one, q), lens, [4] * 3)
    check_attend(c, table, q, c.attend(0, two, q), lens, [1, 2, 3])
    ptr, status = one.ptr, one.status
    del one
    three = c.plan(4, 8, n_tok=i32([9, 9, 9], cuda_device))
    assert three.ptr != ptr and status.tolist() == [0, 0, 0]
    ptr = two.ptr
    del two
    four = c.plan(4, 8)
    assert four.ptr == ptr
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert c.plan(4, 8).ptr != ptr
    g = torch.cuda.CUDAGraph()
    ptr = four.ptr
    del four
    with torch.cuda.graph(g):
        plan = c.plan(4, 8)
        out = c.attend(0, plan, q)
        held = plan.ptr
        del plan
    assert held != ptr
    for _ in range(3):
        assert c.plan(4, 8).ptr != held
    g.replay()
    check_attend(c, table, q, out, lens, [4] * 3)


def test_a_bad_sequence_gets_zeros_and_its_status(ss, cuda_device):
    lens, N = [100, 100, 100, 100, 100, 100], 4
    c, table = make(ss, cuda_device, lens, [4] * 6, 64, 2, 64, seed=8)
    nt = i32([4, 4, -1, 5, 4, 4], cuda_device)
    c.table[1, 0] = 10 ** 6
    c.held[4] = 1
    q = queries(7, N, 4, 64, BF16, cuda_device)
    plan = c.plan(N, 4, rows=i32([0, 1, 2, 3, 4, 5], cuda_device), n_tok=nt)
    assert plan.status.tolist() == [0, ref.ST_PAGE, ref.ST_BADDRAFT, ref.ST_BADDRAFT, ref.ST_PAGE, 0]
    out = c.attend(0, plan, q[:6])
    check_attend(c, table, q[:6], out, lens, [4, 0, 0, 0, 0, 4])
    before = c.k.clone()
    k = queries(6, N, 2, 64, BF16, cuda_device, seed=3)
    qr = c.append(0, plan, q[:6].contiguous(), k, k)
    assert (qr[1:5] == 0).all() and torch.equal(qr[0], q[0])
    changed = (before != c.k).flatten(2).any(2).any(0)
    assert set(changed.nonzero()[:, 0].tolist()) <= {int(table[b, 1]) for b in (0, 5)}
    rows = i32([0, 0, 6, -1, 2, 5], cuda_device)
    c.held[4] = 2
    plan = c.plan(N, 4, rows=rows)
    R = ref.ST_ROW
    assert plan.status.tolist() == [R, R, R, R, 0, 0]
    assert (c.attend(0, plan, q[:6])[:4] == 0).all()


def test_a_shared_page_is_not_written_without_a_reserve(ss, cuda_device):
    c = ss.KVCache(1, 8, 16, 1, 64, 3, 4, device=cuda_device)
    c.reserve(i32([0], cuda_device), 20)
    c.commit(i32([0], cuda_device), i32([19], cuda_device))
    c.fork(i32([0], cuda_device), i32([1], cuda_device))
    assert c.plan(2, 1, rows=i32([0, 1], cuda_device)).status.tolist() == [ref.ST_CAPACITY] * 2
    c.reserve(i32([1], cuda_device), 2)
    assert c.plan(2, 1, rows=i32([0, 1], cuda_device)).status.tolist() == [0, 0]


def test_malformed_trees_are_refused(ss, cuda_device):
    N, n = 5, 7
    fc = np.full((n, N), -1, np.int32)
    ns = np.full((n, N), -1, np.int32)
    fc[:, :4] = [1, 2, 3, 4]               # chains
    fc[1, 2] = 1                           # back
    ns[2, 0] = 3                           # the root has a sibling
    ns[3, 1] = 3                           # linked twice
    fc[4, 3] = -1                          # node 4 not linked
    fc[5, 3] = 5                           # outside
    c, table = make(ss, cuda_device, [10] * n, [N] * n, 16, 1, 64)
    plan = c.plan(N, 1, tree=(i32(fc, cuda_device), i32(ns, cuda_device)))
    assert plan.status.tolist() == [0] + [ref.ST_BADDRAFT] * 5 + [0]


# ------------------------------------------------------------------ append ----

def check_rotated(got, x, pos, f, layout, m):
    """Half a step of the type, the angle's error (2^-22 half turns of fp32
    sincospi input and result, times the pair's magnitude) and three roundings of fp32."""
    want = ref.rotate(x, pos, f, layout, m)
    tol = half_step(got.dtype) * want.abs() + 2.0 ** -20 * abs(m) * x.double().abs().amax() * 2 + 2.0 ** -25
    assert ((got.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 2), (64, 30), (64, 64), (64, 48), (128, 126)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_rotates_and_writes(ss, cuda_device, layout, D, rot, dtype):
    lens, n_tok, N, Q, H = [0, 15, 16, 77], [5, 3, 0, 4], 5, 6, 2
    c, table = make(ss, cuda_device, lens, n_tok, 16, H, D, dtype, layers=2, seed=rot)
    f, m = ss.rope_frequencies(rot, scaling="yarn" if rot > 8 else "linear", factor=4.0, original_len=64)
    rope = ss.Rope(f.to(cuda_device), layout, m)
    qkv = queries(4, N, Q + 2 * H, D, dtype, cuda_device)
    q, k, v = qkv[:, :, :Q], qkv[:, :, Q:Q + H], qkv[:, :, Q + H:]
    before = c.k.clone(), c.v.clone()
    plan = c.plan(N, Q, n_tok=i32(n_tok, cuda_device))
    out = c.append(1, plan, q, k, v, rope)
    written = torch.zeros(c.k.shape[1], 16, dtype=torch.bool)
    for b in range(4):
        T = n_tok[b]
        assert (out[b, T:] == 0).all()
        if T == 0:
            continue
        pos = [lens[b] + t for t in range(T)]
        check_rotated(out[b, :T], q[b, :T].cpu(), pos, f.tolist(), layout, m)
        for t in range(T):
            pg, at = table[b, pos[t] // 16], pos[t] % 16
            written[pg, at] = True
            check_rotated(c.k[1, pg, :, at][None], k[b, t].cpu()[None], [pos[t]], f.tolist(), layout, m)
            assert torch.equal(c.v[1, pg, :, at], v[b, t])
    # nothing else is touched
    same = (~written).to(cuda_device)[None, :, None, :, None]
    for x, y in zip((c.k, c.v), before):
        assert torch.equal(x[0], y[0]) and torch.equal(torch.where(same, x, 0)[1], torch.where(same, y, 0)[1])


def test_append_in_place_without_rotation_and_keys_alone(ss, cuda_device):
    lens, N, Q, H, D = [3, 40], 4, 4, 2, 64
    f, m = ss.rope_frequencies(D)
    rope = ss.Rope(f.to(cuda_device), "half", m)
    q, k, v = (queries(2, N, h, D, BF16, cuda_device, seed=s) for s, h in ((1, Q), (2, H), (3, H)))
    c, table = make(ss, cuda_device, lens, [N, N], 16, H, D)
    plan = c.plan(N, Q)
    want = c.append(0, plan, q, k, v, rope)
    turned = c.k.clone()
    mine = q.clone()
    assert c.append(0, plan, mine, k, v, rope, out=mine) is mine
    assert torch.equal(mine, want)
    assert c.append(0, plan, None, k, v, rope) is None
    assert torch.equal(c.k, turned)
    assert torch.equal(c.append(0, plan, q, k, v), q)
    for b in range(2):
        for t in range(N):
            p = lens[b] + t
            assert torch.equal(c.k[0, table[b, p // 16], :, p % 16], k[b, t])


def test_append_follows_tree_depths(ss, cuda_device):
    rng = np.random.default_rng(1)
    N, lens, D = 12, [9, 100], 64
    parent = ref.random_parents(rng, 2, N)
    fc, ns = ref.links(parent)
    c, table = make(ss, cuda_device, lens, [N, N], 32, 1, D)
    f, m = ss.rope_frequencies(D)
    q, k, v = (queries(2, N, 1, D, F16, cuda_device, seed=s).to(BF16) for s in (1, 2, 3))
    plan = c.plan(N, 1, tree=(i32(fc, cuda_device), i32(ns, cuda_device)))
    out = c.append(0, plan, q, k, v, ss.Rope(f.to(cuda_device)))
    for b in range(2):
        depth = ref.sight(parent[b])[1]
        check_rotated(out[b], q[b].cpu(), [lens[b] + int(d) for d in depth], f.tolist(), "half", 1.0)


@pytest.mark.parametrize("pos", [10 ** 5, 10 ** 6 + 7, 15 * 10 ** 6])
def test_append_at_far_positions(ss, cuda_device, pos):
    """Every page but the last one stands for the same slots: only the position matters."""
    page, D = 128, 128
    mp = pos // page + 2
    dev = cuda_device
    k = torch.zeros((1, 33, 1, page, D), dtype=F16, device=dev)
    table = torch.zeros((1, mp), dtype=torch.int32, device=dev)
    hold = (pos + 2 + page - 1) // page
    table[0, pos // page:] = torch.arange(1, 1 + mp - pos // page, dtype=torch.int32, device=dev)
    refs = torch.ones(33, dtype=torch.int32, device=dev)
    c = ss.KVCache.wrap(k, k.clone(), table, i32([pos], dev), i32([hold], dev), refs, i32([0, 0], dev))
    f, m = ss.rope_frequencies(D)
    q, kn, vn = (queries(1, 2, 1, D, F16, dev, seed=s) for s in (1, 2, 3))
    plan = c.plan(2, 1)
    assert plan.status.tolist() == [0]
    out = c.append(0, plan, q, kn, vn, ss.Rope(f.to(dev)))
    check_rotated(out[0], q[0].cpu(), [pos, pos + 1], f.tolist(), "half", m)


# ------------------------------------------------------------------- pages ----

def same_state(c, m):
    assert c.lens.tolist() == m.lens.tolist()
    assert c.held.tolist() == m.held.tolist()
    assert c.refs.tolist() == m.refs.tolist()
    assert np.array_equal(c.table.cpu().numpy(), m.table)
    assert np.array_equal(c.free.cpu().numpy(), m.free_bits())


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("page,D", [(16, 64), (32, 128)])
def test_pages_follow_the_plain_statement(ss, cuda_device, seed, page, D):
    """Random reserves, commits of chains and trees, forks and truncations, in a
    pool that runs out now and then; every table and every value compared."""
    rng = np.random.default_rng(seed)
    S, pages, mp, L, H = 14, 45, 9, 2, 3
    dev = cuda_device
    c = ss.KVCache(L, pages, page, H, D, S, mp, device=dev)
    c.k.normal_(generator=torch.Generator(device=dev).manual_seed(seed))
    c.v.normal_(generator=torch.Generator(device=dev).manual_seed(seed + 100))
    m = ref.Pages(pages, page, S, mp, [c.k.float().cpu().numpy(), c.v.float().cpu().numpy()])
    same_state(c, m)
    pending = {}
    for turn in range(60):
        n = int(rng.integers(1, S + 1))
        rows = [int(x) for x in rng.permutation(S)[:n]]
        if rng.random() < 0.1:
            rows[-1] = S + 3
        dr = i32(rows, dev)
        kind = rng.choice(["reserve", "reserve", "commit", "commit", "fork", "truncate"])
        if kind == "reserve":
            nt = [int(x) for x in rng.integers(0, 40, n)]
            if rng.random() < 0.1:
                nt[0] = -2
            st = c.reserve(dr, i32(nt, dev)).tolist()
            assert st == m.reserve(rows, nt), (turn, rows, nt)
            for r, t, s in zip(rows, nt, st):
                if s == 0:
                    pending[r] = t
        elif kind == "commit":
            if rng.random() < 0.5:
                acc = [int(rng.integers(-1, max(0, pending.get(r, 0)) + 1)) for r in rows]
                assert c.commit(dr, i32(acc, dev)).tolist() == m.commit(rows, acc), (turn, rows, acc)
            else:
                N = int(rng.integers(1, 33))
                acc, path = [], np.full((n, N), -1, np.int64)
                for i in range(n):
                    a = int(rng.integers(0, N))
                    path[i, :a] = np.sort(rng.permutation(np.arange(1, N))[:a])
                    if rng.random() < 0.05 and a > 1:
                        path[i, :2] = path[i, [1, 0]]
                    acc.append(a if rng.random() < 0.9 else -1)
                assert c.commit(dr, i32(acc, dev), i32(path, dev)).tolist() == m.commit(rows, acc, path), turn
        elif kind == "fork":
            empty = [r for r in range(S) if m.held[r] == 0 and m.lens[r] == 0]
            full = [r for r in range(S) if r not in empty]
            if not empty or not full:
                continue
            dst = empty[:int(rng.integers(1, len(empty) + 1))]
            src = [int(rng.choice(full)) for _ in dst]
            if rng.random() < 0.2:
                dst.append(dst[0])
                src.append(src[0])
            assert c.fork(i32(src, dev), i32(dst, dev)).tolist() == m.fork(src, dst), turn
        else:
            new = [int(x) for x in rng.integers(0, 80, n)]
            if rng.random() < 0.3:
                new = [0] * n
                st = c.truncate(dr).tolist()
            else:
                st = c.truncate(dr, i32(new, dev)).tolist()
            assert st == m.truncate(rows, new), turn
        same_state(c, m)
    assert np.array_equal(c.k.float().cpu().numpy(), m.data[0])
    assert np.array_equal(c.v.float().cpu().numpy(), m.data[1])


def test_the_same_row_twice_changes_nothing(ss, cuda_device):
    dev = cuda_device
    c = ss.KVCache(1, 20, 16, 1, 64, 4, 6, device=dev)
    rows = i32([1, 2, 1], dev)
    assert c.reserve(rows, 5).tolist() == [0, 0, ref.ST_ROW]
    assert c.held.tolist() == [0, 1, 1, 0]
    assert c.commit(rows, i32([2, 2, 2], dev)).tolist() == [ref.ST_ROW, 0, ref.ST_ROW]
    assert c.lens.tolist() == [0, 0, 3, 0]
    assert c.truncate(rows).tolist() == [ref.ST_ROW, 0, ref.ST_ROW]
    assert c.held.tolist() == [0, 1, 0, 0]


def test_reserving_more_than_the_table_holds(ss, cuda_device):
    dev = cuda_device
    c = ss.KVCache(1, 20, 16, 1, 64, 3, 6, device=dev)
    for ask in ([96, 97, 5], [3, 10 ** 6, 1 << 30], [1, (1 << 30) + 1, -1]):
        want = [1 if 96 < x <= 1 << 30 else ref.ST_BADDRAFT if not 0 <= x <= 1 << 30 else 0 for x in ask]
        assert c.reserve(None, i32(ask, dev)).tolist() == want
        if max(ask) <= 1 << 30 and min(ask) >= 0:
            assert want == ref.Pages(20, 16, 3, 6).reserve([0, 1, 2], ask)
    assert c.reserve(None, 97).tolist() == [1, 1, 1]
    assert c.held.tolist() == [6, 0, 1]


def test_many_sequences_and_a_large_pool(ss, cuda_device):
    """More sequences than a block of threads, a bitmap of several rounds, pages
    taken behind a long run of others' pages."""
    dev = cuda_device
    S, pages = 2500, 300_001
    c = ss.KVCache(1, pages, 16, 1, 64, S, 4, device=dev)
    m = ref.Pages(pages, 16, S, 4)
    c.refs[:200_000] = 1
    c.free[:200_000 // 32] = 0
    m.refs[:200_000] = 1
    rng = np.random.default_rng(0)
    nt = [int(x) for x in rng.integers(0, 64, S)]
    assert c.reserve(None, i32(nt, dev)).tolist() == m.reserve(list(range(S)), nt)
    same_state(c, m)
    half = list(range(0, S, 2))
    assert c.truncate(i32(half, dev)).tolist() == [0] * len(half)
    m.truncate(half, [0] * len(half))
    same_state(c, m)


@pytest.mark.parametrize("n", [31, 32, 33, 70])
@pytest.mark.parametrize("tree", [False, True])
def test_plans_of_few_and_of_many_sequences(ss, cuda_device, n, tree):
    """Up to 32 sequences are planned in one launch, more in two: the same
    statuses and results."""
    dev, N, Q = cuda_device, 9, 6
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 400, n)]
    n_tok = [N] * n if tree else [int(x) for x in rng.integers(0, N + 1, n)]
    c, table = make(ss, dev, lens, [N] * n, 32, 2, 64, seed=n)
    parent = ref.random_parents(rng, n, N)
    fc, ns = (i32(x, dev) for x in ref.links(parent))
    want = [0] * n
    last = n - 1
    c.held[last] = 0 if lens[last] else -1          # fewer pages than tokens
    c.table[1, lens[1] // 32] = c.pages             # a page outside the pool
    want[last], want[1] = ref.ST_PAGE, ref.ST_PAGE
    if tree:
        fc[n // 2, 0] = N
    else:
        n_tok[n // 2] = N + 1
    want[n // 2] = ref.ST_BADDRAFT
    if not tree:
        n_tok[1] = N
    rows = list(range(n))
    rows[3], want[3] = n, ref.ST_ROW
    rows[5], want[5], want[6] = 6, ref.ST_ROW, ref.ST_ROW
    q = queries(n, N, Q, 64, BF16, dev)
    plan = c.plan(N, Q, rows=i32(rows, dev), n_tok=None if tree else i32(n_tok, dev), tree=(fc, ns) if tree else None)
    out = c.attend(0, plan, q)
    assert plan.status.tolist() == want
    takes = [0 if st else t for st, t in zip(want, n_tok)]
    check_attend(c, table, q, out, lens, takes, parent if tree else None)


@pytest.mark.parametrize("at", [0, 5, 100, 127, 128, 133])
def test_a_group_shares_pages_up_to_the_first_that_differs(ss, cuda_device, at):
    dev, page, N, Q = cuda_device, 16, 2, 4
    lens = [16 * 135 + x for x in (3, 40, 17, 100)]
    n = len(lens)
    c, table = make(ss, dev, lens, [N] * n, page, 1, 128, shared=([0] * n, 16 * 135), seed=at)
    fresh = next(p for p in range(c.pages) if p not in set(table.flatten().tolist()))
    old = int(table[2, at])
    c.k[:, fresh], c.v[:, fresh] = c.k[:, old].neg(), c.v[:, old].neg()   # other keys there, so that a wrong page shows
    table[2, at] = fresh
    c.table[2, at] = fresh
    c.refs[fresh] = 1
    c.refs[old] -= 1
    q = queries(n, N, Q, 128, BF16, dev)
    plan = c.plan(N, Q, group=i32([7] * n, dev))
    out = c.attend(0, plan, q)
    assert (plan.status == 0).all()
    check_attend(c, table, q, out, lens, [N] * n)


@pytest.mark.parametrize("n,N,Q,H", [(8300, 1, 2, 1), (40, 600, 64, 1)])
def test_more_tiles_than_shared_memory_holds(ss, cuda_device, n, N, Q, H):
    """8300 short sequences of a tile each (beyond 8192 the shares are looked up
    in memory), and sequences of many tiles, which several threads plan."""
    dev = cuda_device
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(0, 40, n)]
    n_tok = [int(x) for x in rng.integers(max(1, N - 300), N + 1, n)]
    c, table = make(ss, dev, lens, n_tok, 16, H, 64, seed=n)
    q = queries(n, N, Q, 64, BF16, dev)
    plan = c.plan(N, Q, n_tok=i32(n_tok, dev))
    out = c.attend(0, plan, q)
    assert (plan.status == 0).all() and torch.isfinite(out).all()
    some = [0, 1, n // 2, n - 2, n - 1] + [int(x) for x in rng.integers(0, n, 40 if N == 1 else 3)]
    check_attend(c, table[some], q[some], out[some], [lens[b] for b in some], [n_tok[b] for b in some])
    assert all((out[b, n_tok[b]:] == 0).all() for b in range(0, n, max(1, n // 40)))
