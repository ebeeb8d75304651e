"""kv_attend's bounded waits: with a limit that no wait meets, the kernel gives
up by itself, says which sequences have no result, and leaves the context, the
cache and its own workspace usable."""
import pytest
import torch

from test_gpu_kv import check_attend, i32, make, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


@pytest.mark.parametrize("N,lens,group", [(4, [3000, 100, 700], None), (200, [64, 0, 900], None),
                                          (2, [600, 601, 640], [0, 0, 0])])
@pytest.mark.parametrize("D", [64, 128])
def test_waits_run_out_and_the_next_call_is_right(ss, cuda_device, N, lens, group, D):
    from sam_drafting_verification_gb300 import _binding as bd
    lib = bd.lib()
    dev = cuda_device
    shared = ([0] * 3, 512) if group else None
    c, table = make(ss, dev, lens, [N] * 3, 64, 2, D, shared=shared)
    q = queries(3, N, 8, D, torch.bfloat16, dev)
    g = i32(group, dev) if group else None
    before = lib.kv_set_wait_limit_ns(1)
    try:
        for _ in range(3):
            plan = c.plan(N, 8, group=g)
            c.attend(0, plan, q)
            torch.cuda.synchronize()
            st = plan.status.tolist()
            assert set(st) <= {0, bd.ST_TIMEOUT} and bd.ST_TIMEOUT in st
    finally:
        assert lib.kv_set_wait_limit_ns(before) == 1
    plan = c.plan(N, 8, group=g)
    out = c.attend(0, plan, q)
    assert (plan.status == 0).all()
    check_attend(c, table, q, out, lens, [N] * 3)


def steady(ss, cuda_device, D, N, lens, group=None, H=2, Q=8):
    shared = ([0] * len(lens), 512) if group else None
    c, table = make(ss, cuda_device, lens, [N] * len(lens), 64, H, D, shared=shared, seed=N)
    q = queries(len(lens), N, Q, D, torch.bfloat16, cuda_device)
    g = i32(group, cuda_device) if group else None
    want = c.attend(0, c.plan(N, Q, group=g), q)
    check_attend(c, table, q, want, lens, [N] * len(lens))
    return c, q, g, Q, want


@pytest.mark.parametrize("D", [64, 128])
def test_giving_up_at_any_step_hands_nothing_on(ss, cuda_device, D):
    """Limits from one that no wait meets to some that most meet, over shares of
    many blocks: roles give up in the middle of their rings.  Every sequence that
    keeps its status keeps its result, and the calls after are whole."""
    from sam_drafting_verification_gb300 import _binding as bd
    lib = bd.lib()
    N, lens = 40, [9000, 30, 4000, 700]   # 160 rows a key head: two row tiles
    c, q, g, Q, want = steady(ss, cuda_device, D, N, lens)
    for ns in (1, 300, 700, 1500, 3000, 6000, 12000, 25000):
        before = lib.kv_set_wait_limit_ns(ns)
        try:
            plan = c.plan(N, Q)
            out = c.attend(0, plan, q)
            torch.cuda.synchronize()
        finally:
            lib.kv_set_wait_limit_ns(before)
        for b, st in enumerate(plan.status.tolist()):
            assert st in (0, bd.ST_TIMEOUT)
            if st == 0:
                assert torch.equal(out[b], want[b]), (ns, b)
        assert torch.equal(c.attend(0, c.plan(N, Q), q), want), ns


@pytest.mark.parametrize("D,N,lens,group", [(128, 4, [100, 50, 260], None), (64, 4, [700, 90, 1000], None),
                                            (128, 1, [0, 3, 127], None), (128, 200, [64, 0, 900], None),
                                            (64, 2, [600, 601, 640], [0, 0, 0])])
def test_giving_up_with_everything_asked_for(ss, cuda_device, D, N, lens, group):
    """Shares that fit the ring: the loader has requested all of its tiles, and met
    no wait, before another role gives up.  What is in flight has to land in the
    CTA that asked for it: calls that give up and calls that do not take turns on
    the same SMs, and each of the latter is whole."""
    from sam_drafting_verification_gb300 import _binding as bd
    lib = bd.lib()
    c, q, g, Q, want = steady(ss, cuda_device, D, N, lens, group)
    for turn in range(30):
        before = lib.kv_set_wait_limit_ns(1 + 40 * turn)
        try:
            plan = c.plan(N, Q, group=g)
            c.attend(0, plan, q)
        finally:
            lib.kv_set_wait_limit_ns(before)
        after = c.plan(N, Q, group=g)
        got = c.attend(0, after, q)   # may begin as the one before ends
        assert set(plan.status.tolist()) <= {0, bd.ST_TIMEOUT}
        assert (after.status == 0).all() and torch.equal(got, want), turn
