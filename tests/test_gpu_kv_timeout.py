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
