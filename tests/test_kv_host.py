"""The paged cache without a GPU: exported symbols, arguments that the C entry
points refuse before any launch (placeholder pointers, never touched), the
binding's own checks, and the frequency tables."""
import ctypes
import math
import os
import re

import pytest
import torch

import sam_drafting_verification_gb300 as ss
from sam_drafting_verification_gb300 import _binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096   # an aligned address


def test_library_exports_every_declared_symbol():
    src = open(os.path.join(ROOT, "include", "samspec_kv.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"\b(kv_[a-z_]+)\s*\(", src)))
    assert names == sorted(bd.KV_EXPORTED)
    lib = bd.lib()
    assert all(hasattr(lib, n) for n in names)


def test_status_words_have_texts():
    lib = bd.lib()
    src = open(os.path.join(ROOT, "include", "samspec_kv.h")).read()
    codes = {m[0]: int(m[1]) for m in re.findall(r"#define\s+(SAMSPEC_ST_[A-Z]+)\s+(\d+)", src)}
    assert codes == {"SAMSPEC_ST_PAGE": bd.ST_PAGE, "SAMSPEC_ST_ROW": bd.ST_ROW}
    texts = [lib.samspec_strerror(v) for v in range(0, 12)]
    assert len(set(texts)) == 12 and b"unknown code" not in texts


def desc(**kw):
    f = dict(k=P, v=P, table=P, lens=P, held=P, refs=P, free_bits=P, dtype=bd.BF16, layers=2, n_pages=100, page=64,
             kv_heads=4, head_dim=128, seqs=8, max_pages=10)
    f.update(kw)
    return ctypes.byref(bd.KvCacheDesc(*f.values()))


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), bd.EINVAL), (dict(table=0), bd.EINVAL), (dict(free_bits=0), bd.EINVAL),
    (dict(dtype=bd.F32), bd.EDTYPE), (dict(dtype=9), bd.EDTYPE),
    (dict(page=8), bd.ESIZE), (dict(page=48), bd.ESIZE), (dict(page=256), bd.ESIZE), (dict(head_dim=96), bd.ESIZE),
    (dict(kv_heads=0), bd.ESIZE), (dict(kv_heads=1025), bd.ESIZE), (dict(layers=0), bd.ESIZE), (dict(seqs=0), bd.ESIZE),
    (dict(max_pages=0), bd.ESIZE), (dict(max_pages=(1 << 20) + 1), bd.ESIZE), (dict(n_pages=1 << 30, layers=2), bd.ESIZE),
    (dict(n_pages=1 << 24, kv_heads=8, page=16), bd.ESIZE), (dict(k=P + 8), bd.EALIGN), (dict(v=P + 4), bd.EALIGN),
])
def test_every_entry_point_refuses_a_bad_cache(kw, code):
    lib, d = bd.lib(), desc(**kw)
    assert lib.kv_reserve(d, None, 2, 4, None, None, P, 1 << 20, None) == code
    assert lib.kv_fork(d, P, P, 2, None, None) == code
    assert lib.kv_commit(d, None, 2, 4, P, None, None, None) == code
    assert lib.kv_truncate(d, None, 2, None, None, None) == code
    assert lib.kv_plan(d, None, 2, 4, 8, None, None, None, None, P, 1 << 30, None) == code
    assert lib.kv_append(d, 0, P, 2, 4, 8, None, 0, None, P, 512, P, 512, None, 0, 0, 1.0, None) == code
    assert lib.kv_attend(d, 0, P, 1 << 30, 2, 4, 8, P, 1024, 0.1, P, None) == code
    assert lib.kv_plan_bytes(d, 2, 4, 8, 0) == 0 and lib.kv_reserve_workspace_bytes(d, 2) == 0


def test_a_null_cache_is_refused():
    lib = bd.lib()
    assert lib.kv_truncate(None, None, 2, None, None, None) == bd.EINVAL
    assert lib.kv_plan_bytes(None, 2, 4, 8, 0) == 0


def test_page_calls_refuse_bad_arguments():
    lib, d = bd.lib(), desc()
    need = lib.kv_reserve_workspace_bytes(d, 3)
    assert need > 0

    def reserve(rows=P, n=3, N=4, ws=P, size=need):
        return lib.kv_reserve(d, rows, n, N, None, None, ws, size, None)

    assert reserve(ws=None) == bd.EINVAL and reserve(n=0) == bd.ESIZE and reserve(N=-1) == bd.ESIZE
    assert reserve(size=need - 1) == bd.ESIZE and reserve(ws=P + 8) == bd.EALIGN
    assert reserve(rows=None, n=9) == bd.ESIZE      # more than the cache has
    assert lib.kv_fork(d, None, P, 2, None, None) == bd.EINVAL and lib.kv_fork(d, P, P, 0, None, None) == bd.ESIZE
    assert lib.kv_commit(d, P, 2, 4, None, None, None, None) == bd.EINVAL
    assert lib.kv_commit(d, P, 2, 33, P, P, P, None) == bd.ESIZE    # paths of 32 nodes at most
    assert lib.kv_commit(d, P, 2, 4, P, P, None, None) == bd.EINVAL  # a path needs the status
    assert lib.kv_commit(d, None, 9, 4, P, None, None, None) == bd.ESIZE
    assert lib.kv_truncate(d, None, 9, None, None, None) == bd.ESIZE
    assert lib.kv_truncate(d, P, 0, None, None, None) == bd.ESIZE


def test_plan_refuses_bad_arguments():
    lib, d = bd.lib(), desc()
    small, large = (lib.kv_plan_bytes(d, 3, 4, 8, g) for g in (0, 1))
    assert 0 < small < large

    def plan(n=3, N=4, q=8, fc=None, ns=None, group=None, buf=P, size=large):
        return lib.kv_plan(d, P, n, N, q, None, fc, ns, group, buf, size, None)

    assert plan(buf=None) == bd.EINVAL and plan(fc=P) == bd.EINVAL and plan(ns=P) == bd.EINVAL
    assert plan(size=small - 1) == bd.ESIZE and plan(group=P, size=small) == bd.ESIZE and plan(buf=P + 16) == bd.EALIGN
    assert plan(N=33, fc=P, ns=P, size=1 << 40) == bd.ESIZE
    for n, N, q in ((0, 4, 8), (3, 0, 8), (3, 4, 0), (3, 4, 6), (3, 4, 4 * 65), (3, (1 << 16) + 1, 8),
                    ((1 << 20) + 1, 1, 4), (1 << 14, 1 << 14, 4)):
        assert lib.kv_plan_bytes(d, n, N, q, 0) == 0 and plan(n=n, N=N, q=q, size=1 << 60) == bd.ESIZE


def test_append_and_attend_refuse_bad_arguments():
    lib, d = bd.lib(), desc()
    size = lib.kv_plan_bytes(d, 3, 4, 8, 0)

    def append(layer=0, plan=P, q=P, qs=1024, qo=P, k=P, ks=512, v=P, vs=512, freq=P, rot=128, layout=0):
        return lib.kv_append(d, layer, plan, 3, 4, 8, q, qs, qo, k, ks, v, vs, freq, rot, layout, 1.0, None)

    assert append(layer=2) == bd.EINVAL and append(layer=-1) == bd.EINVAL and append(plan=None) == bd.EINVAL
    assert append(k=None) == bd.EINVAL and append(v=None) == bd.EINVAL and append(qo=None) == bd.EINVAL
    assert append(q=None) == bd.EINVAL and append(freq=None) == bd.EINVAL and append(layout=2) == bd.EINVAL
    assert append(rot=130) == bd.ESIZE and append(rot=3) == bd.ESIZE and append(rot=-2) == bd.ESIZE
    assert append(ks=504) == bd.EINVAL and append(vs=0) == bd.EINVAL and append(qs=1016) == bd.EINVAL
    assert append(ks=516) == bd.EALIGN and append(qs=1025, qo=P + 16384) == bd.EALIGN and append(k=P + 2) == bd.EALIGN
    assert append(qs=1536) == bd.EINVAL          # in place only where tokens follow one another
    assert append(plan=P + 64) == bd.EALIGN

    def attend(layer=0, plan=P, bytes=size, q=P, qs=1024, scale=0.1, out=P):
        return lib.kv_attend(d, layer, plan, bytes, 3, 4, 8, q, qs, scale, out, None)

    assert attend(layer=2) == bd.EINVAL and attend(plan=None) == bd.EINVAL and attend(q=None) == bd.EINVAL
    assert attend(out=None) == bd.EINVAL
    for s in (0.0, -0.1, math.nan, math.inf):
        assert attend(scale=s) == bd.EINVAL
    assert attend(bytes=size - 1) == bd.ESIZE and attend(qs=1016) == bd.EINVAL and attend(qs=1028) == bd.EALIGN
    assert attend(q=P + 8) == bd.EALIGN and attend(out=P + 16) == bd.EALIGN and attend(plan=P + 128) == bd.EALIGN


# ------------------------------------------------------------- the binding ----

class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_bytes") else 0
        return entry


@pytest.fixture
def cache(monkeypatch):
    rec = _Recorder()
    monkeypatch.setattr(bd, "lib", lambda: rec)
    monkeypatch.setattr(ss, "_is_cuda", lambda t: t.device.type in ("cpu", "meta"))
    monkeypatch.setattr(ss, "_stream", lambda device=None: None)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros((2, 5, 2, 16, 64), dtype=torch.bfloat16)
    c = ss.KVCache.wrap(k, k.clone(), i(4, 3), i(4), i(4), i(5), i(1))
    c.rec = rec
    return c


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def names(c):
    return [n for n, _ in c.rec.calls if not n.endswith("_bytes")]


def test_wrap_checks_every_tensor(cache):
    i = i32
    k = torch.zeros((2, 5, 2, 16, 64), dtype=torch.bfloat16)
    good = [k, k, i(4, 3), i(4), i(4), i(5), i(1)]
    for at, bad, err in ((0, k.float(), TypeError), (0, k[0], ValueError), (1, k.half(), TypeError), (1, k[:1], ValueError),
                         (1, k.transpose(2, 3), ValueError), (2, i(12), ValueError), (2, i(4, 3).long(), TypeError),
                         (3, i(5), ValueError), (4, i(3), ValueError), (5, i(4), ValueError), (6, i(2), ValueError),
                         (3, torch.zeros(4, dtype=torch.int32, device="meta"), ValueError), (0, None, TypeError)):
        args = list(good)
        args[at] = bad
        with pytest.raises(err):
            ss.KVCache.wrap(*args)


def test_page_calls_check_their_tensors(cache):
    c = cache
    assert c.reserve(i32(2), i32(2)).shape == (2,) and c.reserve(None, 7).shape == (4,)
    assert c.truncate(i32(3)).shape == (3,) and c.commit(i32(2), i32(2), i32(2, 8)).shape == (2,)
    assert c.fork(i32(2), i32(2)).shape == (2,)
    assert names(c) == ["kv_reserve"] * 2 + ["kv_truncate", "kv_commit", "kv_fork"]
    c.rec.calls.clear()
    for call in (lambda: c.reserve(i32(2), i32(3)), lambda: c.reserve(i32(2).long(), i32(2)), lambda: c.reserve(i32(2, 1), 1),
                 lambda: c.reserve(i32(4)[::2], i32(2)), lambda: c.reserve(None, i32(9)), lambda: c.reserve([0], 1),
                 lambda: c.commit(i32(2), i32(3)), lambda: c.commit(i32(2), i32(2), i32(3, 8)), lambda: c.commit(i32(2), 3),
                 lambda: c.commit(i32(2), i32(2), i32(2)), lambda: c.fork(i32(2), i32(1)), lambda: c.fork(None, i32(1)),
                 lambda: c.truncate(i32(2), i32(1)), lambda: c.truncate(i32(2), i32(2), out=i32(3)),
                 lambda: c.truncate(i32(2), torch.zeros(2)), lambda: c.truncate(None, i32(6))):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert names(c) == []


def test_passes_check_their_tensors(cache):
    c = cache
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    plan = c.plan(3, 4, rows=i32(2), n_tok=i32(2))
    assert plan.status.shape == (2,)
    wide = bf(2, 3, 8, 64)
    out = c.attend(1, plan, wide[:, :, 2:6])
    assert out.shape == (2, 3, 4, 64) and out.is_contiguous()
    assert c.append(0, plan, wide[:, :, :4], wide[:, :, 4:6], wide[:, :, 6:]).shape == (2, 3, 4, 64)
    assert c.append(0, plan, None, bf(2, 3, 2, 64), bf(2, 3, 2, 64)) is None
    strides = [a for n, a in c.rec.calls if n == "kv_append"][0]
    assert strides[7] == 512 and strides[10] == 512
    assert names(c) == ["kv_plan", "kv_attend", "kv_append", "kv_append"]
    c.rec.calls.clear()
    q, k = bf(2, 3, 4, 64), bf(2, 3, 2, 64)
    for call in (lambda: c.plan(3, 4, rows=i32(2), n_tok=i32(3)), lambda: c.plan(3, 4, tree=(i32(4, 3), i32(4, 2))),
                 lambda: c.plan(3, 4, rows=i32(2), group=i32(4)), lambda: c.plan(2, 4, rows=i32(2), out=plan),
                 lambda: c.plan(3, 4, rows=i32(2), group=i32(2), out=plan),
                 lambda: c.attend(0, plan, q.half()), lambda: c.attend(0, plan, bf(2, 3, 5, 64)), lambda: c.attend(0, plan, None),
                 lambda: c.attend(0, plan, bf(2, 3, 4, 128)[..., ::2]), lambda: c.attend(0, plan, bf(2, 4, 4, 64)[:, :3]),
                 lambda: c.attend(0, plan, bf(2, 4, 3, 64).transpose(1, 2)), lambda: c.attend(0, plan, q, out=bf(2, 3, 4, 32)),
                 lambda: c.append(0, plan, q, bf(2, 3, 4, 64), k), lambda: c.append(0, plan, q, k, k.float()),
                 lambda: c.append(0, plan, q, k, k, ss.Rope(torch.zeros(33, dtype=torch.float64))),
                 lambda: c.append(0, plan, q, k, k, out=q.float())):
        with pytest.raises((TypeError, ValueError)):
            call()
    assert names(c) == []


def test_rope_refuses_what_it_cannot_turn(cache):
    for f, layout, m in ((torch.zeros(4), "half", 1.0), (torch.zeros((2, 2), dtype=torch.float64), "half", 1.0),
                         (torch.zeros(0, dtype=torch.float64), "half", 1.0),
                         (torch.zeros(4, dtype=torch.float64), "quarter", 1.0),
                         (torch.zeros(4, dtype=torch.float64), "half", math.nan)):
        with pytest.raises((TypeError, ValueError)):
            ss.Rope(f, layout, m)


def test_frequencies():
    f, m = ss.rope_frequencies(8, base=100.0)
    assert m == 1.0 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    g, _ = ss.rope_frequencies(8, base=100.0, scaling="linear", factor=4.0)
    assert torch.allclose(g, f / 4)
    n, _ = ss.rope_frequencies(8, base=100.0, scaling="ntk", factor=4.0)
    assert math.isclose(float(n[0]), 1.0) and math.isclose(float(n[-1]), float(f[-1]) / 4)
    y, m = ss.rope_frequencies(64, scaling="yarn", factor=8.0, original_len=2048)
    f, _ = ss.rope_frequencies(64)
    assert math.isclose(m, 0.1 * math.log(8) + 1)
    turns = 2048 * f / (2 * math.pi)
    # pairs that turn often are kept, those that turn less than once are stretched, none is outside
    assert torch.equal(y[turns > 64], f[turns > 64]) and torch.allclose(y[turns < 0.5], f[turns < 0.5] / 8)
    assert ((y <= f) & (y >= f / 8 * (1 - 1e-12))).all()
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, base=-1.0), dict(rot=8, factor=0.0)):
        with pytest.raises(ValueError):
            ss.rope_frequencies(**bad)


def test_plan_memory_is_taken_by_one_thread_alone(cache, monkeypatch):
    """Another thread takes a plan's spare memory while this one looks at it:
    each gets memory of its own, large enough."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ss, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: Memory(n))
    monkeypatch.setattr(cache, "device", torch.device("cuda", 0))
    taken = []

    class Memory:
        def __init__(self, size, meanwhile=None):
            self.size, self.meanwhile = size, meanwhile

        def numel(self):
            if self.meanwhile:
                self.meanwhile()
                self.meanwhile = None
            return self.size

        def data_ptr(self):
            return P

    def other_thread():
        if spare:
            taken.append(spare.pop(0))

    spare = cache._spare[0] = [Memory(4096, other_thread), Memory(1024, other_thread)]
    plan = cache._new_plan(2, 3, 4, False, 4096)
    assert plan.buf.size >= 4096 and all(plan.buf is not t for t in taken)


def test_a_plan_of_another_cache_is_refused(cache):
    """A plan names rows and pages of its own cache, which another may not have."""
    k = torch.zeros((2, 5, 2, 16, 64), dtype=torch.bfloat16)
    other = ss.KVCache.wrap(k, k.clone(), i32(3, 2), i32(3), i32(3), i32(5), i32(1))
    same = ss.KVCache.wrap(k, k.clone(), *(getattr(cache, f) for f in ("table", "lens", "held", "refs", "free")))
    plan = cache.plan(3, 4, rows=i32(2), n_tok=i32(2))
    q, kv = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16)
    cache.rec.calls.clear()
    for call in (lambda c: c.attend(0, plan, q), lambda c: c.append(0, plan, q, kv, kv),
                 lambda c: c.append(0, plan, None, kv, kv), lambda c: c.plan(3, 4, rows=i32(2), out=plan)):
        with pytest.raises(ValueError):
            call(other)
    assert names(cache) == []
    same.attend(0, plan, q)
    same.append(0, plan, q, kv, kv)


def test_reserve_takes_a_number_past_32_bits_as_too_many(cache):
    for ask, got in ((1 << 32, (1 << 31) - 1), ((1 << 32) + 4, (1 << 31) - 1), (-(1 << 32), -1), (7, 7)):
        cache.rec.calls.clear()
        cache.reserve(None, ask)
        assert [a[3] for n, a in cache.rec.calls if n == "kv_reserve"] == [got]


@pytest.mark.parametrize("page,D,max_pages,skew", [(48, 64, 3, 0), (8, 64, 3, 0), (16, 96, 3, 0), (16, 64, (1 << 20) + 1, 0),
                                                   (16, 64, 3, 4)])
def test_a_cache_outside_the_limits_is_refused_when_made(monkeypatch, page, D, max_pages, skew):
    monkeypatch.setattr(ss, "_is_cuda", lambda t: True)
    k = torch.zeros(skew + 2 * page * D, dtype=torch.bfloat16)[skew:].view(1, 2, 1, page, D)
    tensors = (i32(1, max_pages), i32(1), i32(1), i32(2), i32(1))
    with pytest.raises(bd.SamspecError):
        ss.KVCache.wrap(k, k, *tensors)
    good = torch.zeros((1, 2, 1, 16, 64), dtype=torch.bfloat16)
    assert ss.KVCache.wrap(good, good, i32(1, 3), *tensors[1:]).page == 16


def test_kernels_that_begin_early_promise_no_constant_inputs():
    """With programmatic dependent launch a kernel is resident while the one before
    it still writes what this one reads after its wait: `const __restrict__` would
    say that it does not change meanwhile."""
    csrc = os.path.join(ROOT, "sam_drafting_verification_gb300", "csrc")
    for f in ("attend.cu", "cache.cu", "kv.cuh"):
        src = re.sub(r"//.*", "", open(os.path.join(csrc, f)).read())
        assert "wait_for_previous()" in src
        for promise in ("__restrict__", "__ldg(", "ld.global.nc"):
            assert promise not in src, (f, promise)


def test_reserve_judges_a_tensor_as_it_does_a_number(cache):
    """More tokens than the table holds are too many (ST_CAPACITY), not a bad
    number, however they are given."""
    for ask in (i32(2), 5000):
        cache.rec.calls.clear()
        cache.reserve(i32(2), ask)
        assert all(a[3] >= 5000 for n, a in cache.rec.calls if n == "kv_reserve")


class _Block:
    def __init__(self, size):
        self.size = size

    def numel(self):
        return self.size

    def data_ptr(self):
        return P


@pytest.mark.parametrize("current,capturing", [(0, {0}), (1, {0}), (0, {1}), (1, {1}), (1, set())])
def test_capture_is_asked_of_the_caches_own_device(cache, monkeypatch, current, capturing):
    """With another device current, a plan that is captured neither takes spare
    memory nor gives its own back, and one that is not does both."""
    now = [current]

    class Device:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            now.append(self.device.index)

        def __exit__(self, *exc):
            now.pop()

    monkeypatch.setattr(torch.cuda, "device_count", lambda: 2)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[-1] in capturing)
    monkeypatch.setattr(ss, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: _Block(n))
    monkeypatch.setattr(cache, "device", torch.device("cuda", 0))
    old = _Block(4096)
    spare = cache._spare[0] = [old]
    plan = cache._new_plan(2, 3, 4, False, 4096)
    assert now == [current]
    assert (plan.buf is old) == (0 not in capturing)
    mine = plan.buf
    del plan
    assert (mine in spare) == (0 not in capturing)


def test_large_plans_give_their_memory_back_to_torch(cache, monkeypatch):
    """What a cache holds on to for its next plans is bounded, whatever was planned."""
    monkeypatch.setattr(torch.cuda, "device_count", lambda: 1)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(ss, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch, "empty", lambda n, **kw: _Block(n))
    monkeypatch.setattr(cache, "device", torch.device("cuda", 0))
    for need in (4096, 1 << 20, 1 << 30, 64 << 20, 200 << 20, 1 << 34):
        plan = cache._new_plan(2, 3, 4, False, need)
        assert plan.buf.numel() >= need
        del plan
        assert sum(x.numel() for x in cache._spare.get(0, [])) <= 2 * (64 << 20)
    small = cache._new_plan(2, 3, 4, False, 64 << 20)   # (what was kept last, still there)
    assert small.buf.numel() == 64 << 20 and cache._spare[0] == []


@pytest.mark.parametrize("pages,page,heads", [(1 << 14, 64, 8), (1 << 20, 16, 3), (300, 128, 1024)])
@pytest.mark.parametrize("N,rep", [(1, 4), (200, 4), (7, 33)])
def test_the_limit_of_a_plans_work_is_the_one_stated(pages, page, heads, N, rep):
    """units * ((max_pages * page / 128 + 2) * 2 + 5) * kv_heads < 2^31"""
    lib = bd.lib()
    tokens = 2 * (128 // rep)
    each = ((pages * page // 128 + 2) * 2 + 5) * heads
    d = desc(max_pages=pages, page=page, kv_heads=heads, n_pages=64, seqs=1 << 20)
    for grouped in (0, 1):
        units = lambda n: n * -(-N // tokens) + (-(-n * N // tokens) + n if grouped else 0)  # noqa: E731
        n = 1
        while units(n + 1) * each < 1 << 31 and n < 1 << 20:
            n += 1
        most = ((1 << 29 if grouped else 1 << 30) - 1) // (N * rep * heads)
        n = min(n, most)
        assert lib.kv_plan_bytes(d, n, N, rep * heads, grouped) > 0
        assert lib.kv_plan_bytes(d, n + 1, N, rep * heads, grouped) == 0


@pytest.mark.parametrize("n,N,Q", [(8, 4001, 32), (3, 5, 8)])
def test_a_grouped_plan_holds_two_results_of_every_row(n, N, Q):
    lib = bd.lib()
    one, two = (lib.kv_plan_bytes(desc(kv_heads=8), n, N, Q, g) for g in (0, 1))
    results = 2 * n * N * Q * (4 * 128 + 8)
    assert results <= two - one <= 1.02 * results + (64 << 20)
