"""Groups whose first samples take no part: what the others share is read once all
the same."""
import numpy as np
import pytest
import torch

import kv_reference as ref
from test_gpu_kv import BF16, check_attend, i32, make, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


def work_of(plan):
    """What a plan's units cost altogether (the third word behind its statuses), in
    key blocks and what a unit takes besides."""
    at = -(-4 * plan.n // 256) * 256
    return int(plan.buf[at:at + 12].view(torch.int32)[2])


N, Q, H, PAGE, SHARED = 2, 4, 1, 16, 8192


def group_of(ss, dev, n, extra, seed=0):
    lens = [SHARED + x for x in extra]
    c, table = make(ss, dev, lens, [N] * n, PAGE, H, 128, shared=([0] * n, SHARED), seed=seed)
    return c, table, lens, queries(n, N, Q, 128, BF16, dev)


@pytest.mark.parametrize("how", ["no token", "too many tokens", "empty row", "no row", "too few pages", "named twice",
                                 "page outside", "shared tail"])
@pytest.mark.parametrize("dead", [[0], [0, 1, 2], [1], [5], [0, 3, 5], list(range(35))])
def test_sharing_does_not_hang_on_members_that_take_no_part(ss, cuda_device, dead, how):
    dev = cuda_device
    n = 6 if len(dead) < 6 else 38     # (36 and more: looked for in two rounds of a warp)
    extra = [int(x) for x in np.random.default_rng(1).integers(0, 200, n)]
    extra = [x if x % PAGE else x + 1 for x in extra]
    c, table, lens, q = group_of(ss, dev, n, extra)
    live = [b for b in range(n) if b not in dead]
    # the same sequences without the others, and each for itself
    rows = i32(live, dev)
    only = c.plan(N, Q, rows=rows, group=i32([3] * len(live), dev))
    apart = c.plan(N, Q, rows=rows)
    want = c.attend(0, only, q[live].contiguous())
    assert work_of(only) < work_of(apart) / 2

    n_tok, rows = [N] * n, list(range(n))
    for b in dead:
        if how == "no token":
            n_tok[b] = 0
        elif how == "too many tokens":
            n_tok[b] = N + 1
        elif how == "empty row":
            n_tok[b] = c.lens[b] = c.held[b] = 0
        elif how == "no row":
            rows[b] = -1
        elif how == "too few pages":
            c.held[b] = lens[b] // PAGE + 1
            c.lens[b] = (lens[b] // PAGE + 1) * PAGE
        elif how == "named twice":
            rows[b] = dead[0]
            if len(dead) == 1:
                pytest.skip("needs two")
        elif how == "page outside":
            c.table[b, 1] = c.pages
        else:
            c.refs[int(table[b, lens[b] // PAGE])] = 2
    plan = c.plan(N, Q, rows=i32(rows, dev), n_tok=i32(n_tok, dev), group=i32([3] * n, dev))
    st = {"no token": 0, "too many tokens": ref.ST_BADDRAFT, "empty row": 0, "no row": ref.ST_ROW,
          "too few pages": ref.ST_CAPACITY, "named twice": ref.ST_ROW, "page outside": ref.ST_PAGE,
          "shared tail": ref.ST_CAPACITY}[how]
    assert plan.status.tolist() == [st if b in dead else 0 for b in range(n)]
    out = c.attend(0, plan, q)
    took = [N if b in live else 0 for b in range(n)]
    check_attend(c, table, q, out, lens, took)
    if how != "page outside":   # (a table that is no table shares as far as it goes)
        assert work_of(plan) == work_of(only)
        if max(dead) < min(live) or min(dead) > max(live):   # the same rows of the same units
            assert torch.equal(out[live], want)


def test_a_single_member_that_takes_part_reads_for_itself(ss, cuda_device):
    dev = cuda_device
    c, table, lens, q = group_of(ss, dev, 4, [3, 30, 7, 100])
    for alone in range(4):
        n_tok = [N if b == alone else 0 for b in range(4)]
        plan = c.plan(N, Q, n_tok=i32(n_tok, dev), group=i32([0] * 4, dev))
        assert work_of(plan) == work_of(c.plan(N, Q, n_tok=i32(n_tok, dev)))
        check_attend(c, table, q, c.attend(0, plan, q), lens, n_tok)
    plan = c.plan(N, Q, n_tok=i32([0] * 4, dev), group=i32([0] * 4, dev))
    assert work_of(plan) == 0 and (c.attend(0, plan, q) == 0).all()


def test_trees_of_a_group_whose_first_sample_is_refused(ss, cuda_device):
    dev, n, nodes = cuda_device, 4, 7
    rng = np.random.default_rng(3)
    lens = [SHARED + x for x in (5, 60, 33, 2)]
    c, table = make(ss, dev, lens, [nodes] * n, PAGE, H, 64, shared=([0] * n, SHARED), seed=4)
    parent = ref.random_parents(rng, n, nodes)
    fc, ns = ref.links(parent)
    tree = (i32(fc, dev), i32(ns, dev))
    whole = work_of(c.plan(nodes, Q, tree=tree, group=i32([0] * n, dev)))
    fc[0, 0] = nodes
    plan = c.plan(nodes, Q, tree=(i32(fc, dev), tree[1]), group=i32([0] * n, dev))
    assert plan.status.tolist() == [ref.ST_BADDRAFT, 0, 0, 0]
    assert work_of(plan) <= whole
    assert work_of(plan) < work_of(c.plan(nodes, Q, tree=(i32(fc, dev), tree[1]))) / 2
    q = queries(n, nodes, Q, 64, BF16, dev)
    check_attend(c, table, q, c.attend(0, plan, q), lens, [0] + [nodes] * (n - 1), parent)
