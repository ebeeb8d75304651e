"""A rollout whose target model reads a paged cache: drafts, verification,
rotary append, attention over shared prompts, commit and release together.  The
model is one attention layer whose queries, keys and values are looked up by
token, so that what every pass should see follows from the text alone; each
pass's attention is compared with 64 bits."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import workloads
from test_gpu_kv import check_rotated, half_step, i32

pytestmark = pytest.mark.gpu


class CachedModel:
    """logits = (attention output of the token) W, W fp32; checks every pass."""

    def __init__(self, ss, cache, V, Q, texts, dev, seed=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        H, D = cache.kv_heads, cache.head_dim
        self.cache, self.Q = cache, Q
        self.q, self.k, self.v = (torch.randn((V, h, D), generator=g, device=dev).to(cache.dtype) for h in (Q, H, H))
        self.w = torch.randn((Q * D, V), generator=g, device=dev)
        f, self.m = ss.rope_frequencies(D)
        self.f = f.tolist()
        self.rope = ss.Rope(f.to(dev), "half", self.m)
        self.texts = texts          # what each cache row should hold, then the tokens of the pass
        self.passes = 0

    def look_up(self, t, plan, tokens):
        return t[tokens.clamp_min(0).long()]

    def prefill(self, rows, tokens, n_tok):
        plan = self.cache.plan(tokens.shape[1], self.Q, rows=rows, n_tok=n_tok)
        assert (plan.status == 0).all()
        self.cache.append(0, plan, None, self.look_up(self.k, plan, tokens), self.look_up(self.v, plan, tokens), self.rope)

    def __call__(self, rows, n_done, tokens, n_tok, plan):
        c = self.cache
        q = c.append(0, plan, self.look_up(self.q, plan, tokens), self.look_up(self.k, plan, tokens),
                     self.look_up(self.v, plan, tokens), self.rope)
        o = c.attend(0, plan, q)
        self.passes += 1
        if self.passes % 4 == 1:
            self.check(rows.tolist(), tokens, n_tok.tolist(), q, o)
        return (o.float().flatten(2) @ self.w).contiguous()

    def check(self, rows, tokens, n_tok, q, o):
        c, u = self.cache, half_step(self.cache.dtype)
        for i in (0, len(rows) // 2, len(rows) - 1):
            row, T = rows[i], n_tok[i]
            base = int(c.lens[row])
            at = torch.arange(base + T, device=c.device)
            pg = c.table[row].long()[at // c.page]
            k, v = c.k[0][pg, :, at % c.page], c.v[0][pg, :, at % c.page]
            text = self.texts(row)[:base + 1]
            assert len(text) == base + 1, "the cache holds the text but for its last token"
            text = torch.tensor(text + tokens[i, 1:T].tolist(), device=c.device)
            assert torch.equal(v, self.v[text])
            check_rotated(k[-8:], self.k[text[-8:]].cpu(), list(range(base + T))[-8:], self.f, "half", self.m)
            want, mag, e = ref.attend(q[i, :T], k, v, base, np.tril(np.ones((T, T), bool)), c.head_dim ** -0.5)
            assert ((o[i, :T].double() - want).abs() <= u * want.abs() + (u + e) * mag + 2.0 ** -24).all()


@pytest.mark.parametrize("K,threshold,temperature", [(3, None, 0.0), (3, 7, 1.0), (0, None, 0.0), (7, None, 0.7)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rollout_with_a_cache(ss, cuda_device, K, threshold, temperature, dtype):
    dev = cuda_device
    rng = np.random.default_rng(K)
    V, Q, H, D, page, prompts, samples = 80, 8, 2, 64, 16, 3, 4
    B = prompts * samples
    plen = [130, 300, 517]
    text = [workloads.make_stream(rng, n, V, 0.5, 4, 32) for n in plen]
    batch = ss.SamBatch(B, 700, V, device=dev)
    hist = np.zeros((B, max(plen)), np.int32)
    for b in range(B):
        hist[b, :plen[b // samples]] = text[b // samples]
    batch.extend(i32(hist, dev), i32([plen[b // samples] for b in range(B)], dev))
    cache = ss.KVCache(1, 220, page, H, D, B, 48, dtype=dtype, device=dev)
    run = {}

    def so_far(row):
        out = run["ro_out"][row] if "ro_out" in run else []
        return text[row // samples].tolist() + out

    model = CachedModel(ss, cache, V, Q, so_far, dev)
    # the first sample of each prompt is filled, the others are forks of it
    first = i32([p * samples for p in range(prompts)], dev)
    n_tok = i32([n - 1 for n in plen], dev)
    assert (cache.reserve(first, n_tok) == 0).all()
    toks = np.zeros((prompts, max(plen) - 1), np.int32)
    for p in range(prompts):
        toks[p, :plen[p] - 1] = text[p][:-1]
    model.prefill(first, i32(toks, dev), n_tok)
    assert (cache.commit(first, n_tok - 1) == 0).all()
    others = [b for b in range(B) if b % samples]
    assert (cache.fork(i32([b - b % samples for b in others], dev), i32(others, dev)) == 0).all()
    used = int((cache.refs > 0).sum())
    assert used == sum(-(-(n - 1) // page) for n in plen), "forks hold no page of their own"

    from sam_drafting_verification_gb300.rollout import Rollout
    ro = Rollout(batch, model, K=K, threshold=threshold, temperature=temperature, seed=5, cache=cache, q_heads=Q,
                 last=i32([text[b // samples][-1] for b in range(B)], dev),
                 group=i32([b // samples for b in range(B)], dev))
    # the rollout's own token lists, as they grow
    import sam_drafting_verification_gb300.rollout as mod
    made = mod.RolloutResult

    def watched(tokens):
        run["ro_out"] = tokens
        return made(tokens=tokens)

    mod.RolloutResult = watched
    try:
        limits = [int(x) for x in rng.integers(5, 60, B)]
        res = ro.run(limits)
    finally:
        mod.RolloutResult = made
    assert [len(t) for t in res.tokens] == limits
    assert model.passes == res.steps
    assert (cache.held == 0).all() and (cache.refs == 0).all(), "every page came back"
    if K == 3 and threshold is None:
        assert res.accepted > 0


def test_rollout_says_when_the_cache_is_full(ss, cuda_device):
    dev = cuda_device
    V = 40
    batch = ss.SamBatch(2, 200, V, device=dev)
    batch.extend(torch.zeros((2, 4), dtype=torch.int32, device=dev), i32([4, 4], dev))
    cache = ss.KVCache(1, 3, 16, 1, 64, 2, 8, device=dev)
    from sam_drafting_verification_gb300.rollout import Rollout

    def model(rows, n_done, tokens, n_tok, plan):
        return torch.zeros((len(rows), tokens.shape[1], V), device=dev)

    ro = Rollout(batch, model, K=0, cache=cache, q_heads=1, last=i32([0, 0], dev))
    with pytest.raises(RuntimeError, match="cache status 1"):
        ro.run([60, 60])
    with pytest.raises(ValueError):
        Rollout(batch, model, cache=cache)


@pytest.fixture(scope="module")
def ss(cuda_device):
    import sam_drafting_verification_gb300 as ss
    return ss


def test_tree_step_keeps_the_accepted_path(ss, cuda_device):
    """spec_verify_tree's path and accept_len go to commit: the cache then holds
    the context, node 0 and the accepted nodes, as if only they had been appended."""
    dev = cuda_device
    rng = np.random.default_rng(8)
    n, N, V, Q, H, D, page = 9, 10, 300, 4, 2, 128, 32
    lens = [int(x) for x in rng.integers(0, 90, n)]
    cache = ss.KVCache(3, 80, page, H, D, n, 6, device=dev)
    assert (cache.reserve(None, i32(lens, dev)) == 0).all()
    cache.commit(None, i32([x - 1 for x in lens], dev))
    cache.k.normal_()
    cache.v.normal_()
    parent = ref.random_parents(rng, n, N)
    fc, ns = (i32(x, dev) for x in ref.links(parent))
    tok = i32(np.stack([rng.permutation(V)[:N] for _ in range(n)]), dev)
    assert (cache.reserve(None, N) == 0).all()
    plan = cache.plan(N, Q, tree=(fc, ns))
    k, v = (torch.randn((3, n, N, H, D), device=dev).to(torch.bfloat16) for _ in range(2))
    for layer in range(3):
        cache.append(layer, plan, None, k[layer], v[layer])
    logits = torch.randn((n, N, V), device=dev)
    for b in range(n):   # some children are their parent's most likely token
        for j in range(1, N):
            if rng.random() < 0.6:
                logits[b, parent[b, j], tok[b, j]] += 9.0
    r = ss.spec_verify_tree(logits, tok, fc, ns, temperature=0.0)
    assert (r["status"] == 0).all() and int(r["accept_len"].max()) > 1
    before = cache.k.clone(), cache.v.clone(), cache.table.clone()
    assert (cache.commit(None, r["accept_len"], r["path"]) == 0).all()
    acc, path = r["accept_len"].tolist(), r["path"].tolist()
    for b in range(n):
        nodes = [0] + path[b][:acc[b]]
        T = lens[b] + len(nodes)
        assert int(cache.lens[b]) == T and int(cache.held[b]) == -(-T // page)
        at = torch.arange(T, device=dev)
        pg = cache.table[b].long()[at // page]
        old = before[2][b].long()[at[:lens[b]] // page]
        for x, y, new in ((cache.k, before[0], k), (cache.v, before[1], v)):
            got = x[:, pg, :, at % page]
            assert torch.equal(got[:lens[b]], y[:, old, :, at[:lens[b]] % page])
            assert torch.equal(got[lens[b]:], new[:, b, nodes].transpose(0, 1))


@pytest.mark.parametrize("K", [0, 3])
def test_a_row_that_the_cache_refused_keeps_its_length(ss, cuda_device, K):
    """Two sequences and no page left: the second one's pass is refused.  Its row then
    holds what it held before, while the first one's has grown."""
    dev, V = cuda_device, 40
    batch = ss.SamBatch(2, 200, V, device=dev)
    batch.extend(torch.zeros((2, 32), dtype=torch.int32, device=dev), i32([32, 32], dev))
    cache = ss.KVCache(1, 4, 16, 1, 64, 2, 8, device=dev)
    first = i32([20, 31], dev)
    assert cache.reserve(None, first).tolist() == [0, 0]
    assert cache.commit(None, first - 1).tolist() == [0, 0]      # two pages each
    from sam_drafting_verification_gb300.rollout import Rollout
    held = []

    def model(rows, n_done, tokens, n_tok, plan):
        held.append((cache.lens.tolist(), plan.status.tolist(), n_tok.tolist()))
        logits = torch.zeros((len(rows), tokens.shape[1], V), device=dev)
        logits[..., 0] = 9.0       # every draft of zeros is accepted
        return logits

    ro = Rollout(batch, model, K=K, cache=cache, q_heads=1, last=i32([0, 0], dev))
    with pytest.raises(RuntimeError, match="sequence 1: cache status 1"):
        ro.run([60, 60])
    lens, status, n_tok = held[-1]
    assert status == [0, 1]
    assert cache.lens.tolist() == [lens[0] + n_tok[0], lens[1]]
    assert (cache.held * 16 >= cache.lens).all()


def test_a_shared_row_that_the_cache_refused_keeps_its_length(ss, cuda_device):
    """Two samples of one prompt and no page left for a copy of the page that they
    share: the slots behind the prompt are neither's, and nothing is committed."""
    dev, V = cuda_device, 40
    batch = ss.SamBatch(2, 200, V, device=dev)
    batch.extend(torch.zeros((2, 9), dtype=torch.int32, device=dev), i32([9, 9], dev))
    cache = ss.KVCache(1, 1, 16, 1, 64, 2, 4, device=dev)
    assert cache.reserve(i32([0], dev), 8).tolist() == [0]
    assert cache.commit(i32([0], dev), i32([7], dev)).tolist() == [0]
    assert cache.fork(i32([0], dev), i32([1], dev)).tolist() == [0]
    from sam_drafting_verification_gb300.rollout import Rollout

    def model(rows, n_done, tokens, n_tok, plan):
        return torch.zeros((len(rows), tokens.shape[1], V), device=dev)

    with pytest.raises(RuntimeError, match="cache status 1"):
        Rollout(batch, model, K=2, cache=cache, q_heads=1, last=i32([0, 0], dev)).run([5, 5])
    assert cache.lens.tolist() == [8, 8] and cache.refs.tolist() == [2]
