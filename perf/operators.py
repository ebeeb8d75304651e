"""Cases for the paged key/value cache: attention of a verification pass, rotary
append, and the pages' bookkeeping (fork, reserve, commit, truncate).

The cache is plain tensors that a program holds: pools k, v [layers, pages,
kv_heads, page, head_dim], a page table [sequences, max_pages], committed
lengths, pages held, references of each page and a bitmap of the free ones
(bit p % 32 of word p // 32).  The plain forms below work on the same tensors
in elementary torch operations, in 32 bits (positions' angles in 64), rounded
once at the end.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases ----

def _case(name=None, **kw):
    c = dict(kind="attend", n=1, N=1, q_heads=32, kv_heads=8, head_dim=128, page=64, layers=1, dtype="bf16",
             len_lo=512, len_hi=512, group=1, shared=0, tree=False, ragged=False, rot=0, layout="half",
             scaling="none", mix=1)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one short request, one token: what a single call costs
        _case("attend_one_token", n=1, N=1, len_lo=700, len_hi=700),
        # a decode step of 64 requests with 4096-token histories and 3 drafts each
        _case("attend_chain_b64", n=64, N=4, len_lo=4096, len_hi=4096),
        # 8-node draft trees over short histories of mixed lengths, 16-token pages
        _case("attend_tree_b256", n=256, N=8, q_heads=16, kv_heads=2, len_lo=60, len_hi=2000, page=16, tree=True),
        # a rollout's groups: 16 samples of each of 16 prompts, the prompts stored once
        _case("attend_group_b256", n=256, N=4, q_heads=64, kv_heads=8, len_lo=8200, len_hi=10000, group=16,
              shared=8192),
        # the long tail of a rollout: few requests, long histories, narrow heads, fp16
        _case("attend_long_b32", n=32, N=4, q_heads=32, kv_heads=4, head_dim=64, len_lo=16384, len_hi=32768,
              dtype="fp16", ragged=True),
        # a prompt taken in chunks of up to 1000 tokens behind what is there already
        _case("attend_chunk_b4", n=4, N=1000, q_heads=32, kv_heads=8, len_lo=0, len_hi=4000, ragged=True),
        # the drafts' queries and keys of a decode step: rotated, keys and values written to their pages
        _case("append_chain_b64", kind="append", n=64, N=4, len_lo=4096, len_hi=4096, rot=128, scaling="yarn"),
        # a prompt's: many tokens, interleaved pairs, half of each head
        _case("append_prompt_b8", kind="append", n=8, N=4001, q_heads=32, kv_heads=8, len_lo=0, len_hi=300, rot=64,
              layout="interleaved", dtype="fp16", ragged=True),
        # one request's single step of bookkeeping
        _case("pages_one", kind="commit", n=1, N=4, len_lo=700, len_hi=700, layers=2),
        # accepted paths of 8-node trees brought to the front of their slots, the rest released
        _case("pages_commit_tree_b256", kind="commit", n=256, N=8, len_lo=100, len_hi=500, layers=4, tree=True),
        # 16 samples forked off each of 16 prompts: shared pages counted, partly filled ones copied
        _case("pages_fork_b256", kind="fork", n=256, N=4, len_lo=600, len_hi=1200, layers=16, group=16),
        # one whole decode step of the cache: reserve, append and attend on two layers, commit
        _case("step_tree_b64", kind="step", n=64, N=8, q_heads=32, kv_heads=8, len_lo=500, len_hi=4000, layers=2,
              tree=True, rot=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "commit", "fork", "step"])
    kv = rng.choice([1, 2, 4, 8])
    rep = rng.choice([1, 2, 3, 4, 5, 7, 8])
    hd = rng.choice([64, 128])
    c = _case(kind=kind, q_heads=kv * rep, kv_heads=kv, head_dim=hd, page=rng.choice([16, 32, 64, 128]),
              dtype=rng.choice(["bf16", "fp16"]), mix=rng.randrange(1, 1 << 30))
    c["tree"] = rng.random() < 0.4
    c["N"] = rng.randrange(1, 33) if c["tree"] or kind != "append" else _log_int(rng, 1, 2000)
    c["ragged"] = not c["tree"] and rng.random() < 0.5
    c["n"] = _log_int(rng, 1, 256 if c["N"] <= 64 else 8)
    top = max(64, min(12000, 600000 // c["n"]))
    c["len_hi"] = _log_int(rng, 16, top)
    c["len_lo"] = rng.randrange(0, c["len_hi"] + 1)
    if kind in ("append", "step") or rng.random() < 0.2:
        c["rot"] = 2 * rng.randrange(1, hd // 2 + 1)
        c["layout"] = rng.choice(["half", "interleaved"])
        c["scaling"] = rng.choice(["none", "linear", "yarn"])
    if kind == "attend" and rng.random() < 0.4 and c["n"] > 1:
        c["group"] = rng.randrange(2, c["n"] + 1)
        c["shared"] = rng.randrange(0, c["len_lo"] + 1)
    if kind in ("commit", "step"):
        c["layers"] = rng.randrange(1, 4)
        c["len_hi"] = min(c["len_hi"], 2000)
        c["len_lo"] = min(c["len_lo"], c["len_hi"])
    if kind == "fork":
        c["layers"], c["group"] = rng.randrange(1, 9), rng.randrange(1, 17)
        c["len_hi"] = min(c["len_hi"], 1500)
        c["len_lo"] = min(c["len_lo"], c["len_hi"])
        c["N"] = min(c["N"], 64)
    if kind == "attend" and not c["tree"] and rng.random() < 0.2:
        c["N"], c["n"] = _log_int(rng, 33, 1000), rng.randrange(1, 4)
        c["group"], c["shared"] = 1, 0
        c["len_hi"] = min(c["len_hi"], 4000)
        c["len_lo"] = min(c["len_lo"], c["len_hi"])
    while not _fits(work(c)) and (c["n"] > 1 or c["layers"] > 1):   # no dearer than the largest listed case
        c["n"], c["layers"] = max(1, c["n"] // 2), max(1, c["layers"] - 1)
        c["group"] = min(c["group"], c["n"])
    return c


def _fits(w):
    return w["bytes"] < 1.4e9 and w["flops"] < 2.9e11


def _shape(c):
    """Lengths, tokens per sequence, groups and trees of a case: the case's alone, whatever the seed."""
    r = np.random.default_rng(c["mix"])
    n, N = c["n"], c["N"]
    if c["kind"] == "fork":   # n samples off ceil(n / group) prompts
        m = -(-n // c["group"])
        lens = r.integers(c["len_lo"], c["len_hi"] + 1, m)
    else:
        lo, hi = max(1, c["len_lo"]), max(1, c["len_hi"])
        lens = np.exp(r.uniform(math.log(lo), math.log(hi), n)).round().astype(np.int64)
        lens = np.clip(lens, c["len_lo"], c["len_hi"])
        if c["len_lo"] == 0 and n > 1:
            lens[0] = 0
    ntok = r.integers(1, N + 1, n) if c["ragged"] else np.full(n, N)
    if c["ragged"]:
        ntok[r.integers(0, n)] = N
    parent = np.zeros((n, N), np.int64)
    for b in range(n if c["tree"] else 0):
        kids = np.zeros(N, np.int64)
        for j in range(1, N):
            p = int(r.integers(max(0, j - 4), j))
            p = p if kids[p] < 3 else j - 1
            parent[b, j] = p
            kids[p] += 1
    path = np.full((n, N), -1, np.int64)
    acc = np.zeros(n, np.int64)
    for b in range(n):        # an accepted path: down the tree as far as a coin goes
        at, t = 0, 0
        while c["tree"] and r.random() < 0.75:
            kids = [j for j in range(at + 1, N) if parent[b, j] == at]
            if not kids:
                break
            at = int(kids[int(r.integers(0, len(kids)))])
            path[b, t] = at
            t += 1
        if not c["tree"]:
            t = int(r.integers(0, int(ntok[b])))
            path[b, :t] = np.arange(1, t + 1)
        acc[b] = t
    return lens, ntok, parent, path, acc


# ----------------------------------------------------------------- inputs ----

def _links(parent):
    n, N = parent.shape
    fc, ns = np.full((n, N), -1, np.int32), np.full((n, N), -1, np.int32)
    for b in range(n):
        last = {}
        for j in range(1, N):
            p = int(parent[b, j])
            if p in last:
                ns[b, last[p]] = j
            else:
                fc[b, p] = j
            last[p] = j
    return fc, ns


def _inv_freq(c):
    """Radians per position of each rotated pair, 64 bits."""
    rot = c["rot"]
    base = 10000.0
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "yarn":
        factor, old = 8.0, 4096
        edge = lambda turns: rot * math.log(old / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(edge(32.0)), 0), min(math.ceil(edge(1.0)), rot - 1)
        ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _bits(refs):
    """The bitmap of the free pages, as int32 words."""
    free = torch.nn.functional.pad((refs == 0).to(torch.int64), (0, -refs.numel() % 32)).view(-1, 32)
    w = (free << torch.arange(32, device=refs.device)).sum(1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    r = np.random.default_rng([seed, 77])
    lens, ntok, parent, path, acc = _shape(c)
    n, N, page, L, H, D = c["n"], c["N"], c["page"], c["layers"], c["kv_heads"], c["head_dim"]
    forks = c["kind"] == "fork"
    reserved = c["kind"] in ("attend", "append")
    m = len(lens)                                   # sequences that hold tokens
    S = m + n if forks else n
    hold = -(-(lens + (ntok if reserved else 0)) // page)
    mp = int(max(-(-(lens.max() + N) // page), hold.max(), 1))
    table = np.full((S, mp), -1, np.int64)
    shared_pages = c["shared"] // page if c["group"] > 1 and not forks else 0
    used = 0
    for b in range(m):
        s = min(shared_pages, int(hold[b])) if b % c["group"] else 0
        if s:
            table[b, :s] = table[b - b % c["group"], :s]
        table[b, s:hold[b]] = np.arange(used, used + hold[b] - s)
        used += int(hold[b]) - s
    spare = 0 if reserved else n * (-(-N // page) + 1)
    pages = used + spare + 5
    perm = r.permutation(pages)                     # a pool in use: pages lie anywhere
    table = np.where(table >= 0, perm[np.clip(table, 0, None)], -1)
    refs = np.bincount(table[table >= 0], minlength=pages)
    i32 = lambda a: torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    dt = DT[c["dtype"]]
    rand = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    pool = lambda: torch.empty((L, pages, H, page, D), dtype=dt, device=dev).normal_(generator=g)  # noqa: E731
    st = dict(case=c, k=pool(), v=pool(), table=i32(table), refs=i32(refs),
              lens=i32(np.concatenate([lens, np.zeros(S - m, np.int64)])),
              held=i32(np.concatenate([hold, np.zeros(S - m, np.int64)])), n_tok=i32(ntok))
    st["free"] = _bits(st["refs"])
    st["base"] = st["lens"].clone()
    st["rows"] = torch.arange(n, dtype=torch.int32, device=dev) + (m if forks else 0)
    if forks:
        st["src"] = torch.arange(n, dtype=torch.int32, device=dev) // c["group"]
        st["zero"] = torch.zeros(n, dtype=torch.int32, device=dev)
        return st
    st["accept"], st["path"] = i32(acc), i32(path)
    if c["tree"]:
        fc, ns = _links(parent)
        st["first_child"], st["next_sibling"] = i32(fc), i32(ns)
    st["group"] = torch.arange(n, dtype=torch.int32, device=dev) // c["group"]
    # one projection's output holds a token's queries, keys and values: they are views of it
    Q = c["q_heads"]
    qkv = rand(L, n, N, (Q + 2 * H) * D)
    qkv[..., :Q * D] *= 2.0
    qkv = qkv.to(dt)
    st["q"] = qkv[..., :Q * D].unflatten(-1, (Q, D))
    st["k_new"] = qkv[..., Q * D:(Q + H) * D].unflatten(-1, (H, D))
    st["v_new"] = qkv[..., (Q + H) * D:].unflatten(-1, (H, D))
    if c["rot"]:
        f, st["mscale"] = _inv_freq(c)
        st["inv_freq"] = torch.as_tensor(f, device=dev)
    return st


# ------------------------------------------------------------ plain forms ----

def _ancestors(st):
    """[n, N, N] truth: node j is i or above it; depth [n, N]."""
    c = st["case"]
    N, dev = c["N"], st["k"].device
    if not c["tree"]:
        d = torch.arange(N, device=dev)
        return (d[None, :] <= d[:, None]).expand(c["n"], N, N), d.expand(c["n"], N)
    at = torch.arange(N, device=dev)
    child = (st["first_child"][..., None] == at).double()
    sib = (st["next_sibling"][..., None] == at).double()
    eye = torch.eye(N, dtype=torch.float64, device=dev).expand(c["n"], N, N)
    par = child @ torch.linalg.solve_triangular(eye - sib, eye, upper=True, unitriangular=True)
    below = torch.linalg.solve_triangular(eye - par, eye, upper=True, unitriangular=True).round()
    return below.transpose(1, 2) > 0.5, below.sum(1).long() - 1


def _attend(st, layer):
    """softmax(q k^T / sqrt(d)) v over a sequence's pages and its new tokens."""
    c = st["case"]
    n, N, Q, H, D, page = c["n"], c["N"], c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    lens, ntok, dev = st["lens"].long(), st["n_tok"].long(), st["k"].device
    pos = torch.arange(st["table"].shape[1] * page, device=dev)
    pg = st["table"].long().clamp_min(0).repeat_interleave(page, 1)
    k = st["k"][layer][pg, :, pos % page].float().permute(0, 2, 3, 1)      # [n, H, D, T]
    v = st["v"][layer][pg, :, pos % page].float().permute(0, 2, 1, 3)      # [n, H, T, D]
    q = st["q"][layer].float().reshape(n, N, H, Q // H, D).permute(0, 2, 1, 3, 4).reshape(n, H, -1, D)
    s = (q @ k * (1.0 / math.sqrt(D))).view(n, H, N, Q // H, -1)
    see, _ = _ancestors(st)
    node = pos[None] - lens[:, None]
    new = (node >= 0) & (node < ntok[:, None])
    ok = (node < 0)[:, None] | new[:, None] & see.gather(2, node.clamp(0, N - 1)[:, None].expand(n, N, -1))
    live = torch.arange(N, device=dev) < ntok[:, None]
    ok = (ok & live[..., None])[:, None, :, None]
    s = s.masked_fill(~ok, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    z = p.sum(-1, keepdim=True)
    o = p.view(n, H, -1, pos.numel()) @ v.masked_fill(~(new | (node < 0))[:, None, :, None], 0.0)
    o = o / z.view(n, H, -1, 1).clamp_min(1e-30)
    return o.view(n, H, N, Q // H, D).permute(0, 2, 1, 3, 4).reshape(n, N, Q, D).to(st["q"].dtype)


def _rotate(x, cos, sin, layout):
    rot = 2 * cos.shape[-1]
    y, rest = x.float()[..., :rot], x.float()[..., rot:]
    a, b = (y[..., :rot // 2], y[..., rot // 2:]) if layout == "half" else (y[..., 0::2], y[..., 1::2])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((y, rest), -1).to(x.dtype)


def _append(st, layers, queries=True):
    """Queries and keys turned to their positions, keys and values put into their slots."""
    c = st["case"]
    N, page, dev = c["N"], c["page"], st["k"].device
    q, k, v = st["q"][layers] if queries else None, st["k_new"][layers], st["v_new"][layers]
    live = torch.arange(N, device=dev) < st["n_tok"][:, None]
    if c["rot"]:
        pos = st["lens"].long()[:, None] + _ancestors(st)[1]
        ang = pos.double()[..., None] * st["inv_freq"]
        cos, sin = (st["mscale"] * ang.cos()).float()[:, :, None], (st["mscale"] * ang.sin()).float()[:, :, None]
        k = _rotate(k, cos, sin, c["layout"])
        q = _rotate(q, cos, sin, c["layout"]) if queries else None
    if queries:
        q = torch.where(live[..., None, None], q, torch.zeros((), dtype=q.dtype, device=dev))
    slot = (st["lens"].long()[:, None] + torch.arange(N, device=dev))
    pg = st["table"].long().gather(1, (slot // page).clamp_max(st["table"].shape[1] - 1))[live]
    at = (slot % page)[live]
    st["k"][layers, pg, :, at] = k[..., live, :, :].movedim(-3, 0) if isinstance(layers, slice) else k[live]
    st["v"][layers, pg, :, at] = v[..., live, :, :].movedim(-3, 0) if isinstance(layers, slice) else v[live]
    return q


def _release(st, rows, new):
    """Lengths cut to `new`, pages behind them given back."""
    page, rows = st["case"]["page"], rows.long()
    col = torch.arange(st["table"].shape[1], device=rows.device)
    need = (new.long() + page - 1) // page
    t = st["table"][rows].long()
    drop = (col >= need[:, None]) & (col < st["held"][rows].long()[:, None])
    st["refs"].index_add_(0, t[drop], torch.full_like(t[drop], -1, dtype=torch.int32))
    st["table"][rows] = torch.where(drop, -1, t).int()
    st["lens"][rows] = new.int()
    st["held"][rows] = need.int()
    st["free"].copy_(_bits(st["refs"]))


def _reserve(st, rows, ntok):
    """Pages for `ntok` more tokens, the lowest free ones first; a partly filled page that others hold too is copied."""
    page, rows = st["case"]["page"], rows.long()
    lens, held, t = st["lens"][rows].long(), st["held"][rows].long(), st["table"][rows].long()
    tail = t.gather(1, (lens // page).clamp_max(t.shape[1] - 1)[:, None])[:, 0]
    copy = (lens % page > 0) & (st["refs"][tail.clamp_min(0)] > 1)
    cow = copy.long()
    more = ((lens + ntok.long() + page - 1) // page - held).clamp_min(0)
    first = torch.cumsum(more + cow, 0) - more - cow
    free = (st["refs"] == 0).nonzero()[:, 0]
    fresh = free[first[copy]]
    st["refs"].index_add_(0, tail[copy], torch.full_like(tail[copy], -1, dtype=torch.int32))
    col = torch.arange(t.shape[1], device=t.device)
    new = (col >= held[:, None]) & (col < (held + more)[:, None])
    t = torch.where(new, free[((first + cow)[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)], t)
    t[copy, (lens // page)[copy]] = fresh
    st["refs"][t[new]] = 1
    st["refs"][fresh] = 1
    st["table"][rows] = t.int()
    st["held"][rows] = (held + more).int()
    st["free"].copy_(_bits(st["refs"]))
    filled = (torch.arange(page, device=t.device) < (lens % page)[copy][:, None])[None, :, None, :, None]
    for x in (st["k"], st["v"]):
        x[:, fresh] = torch.where(filled, x[:, tail[copy]], x[:, fresh])


def _commit(st, rows):
    """Node 0 and the accepted path's nodes become the next tokens, the other slots are given up."""
    c, page = st["case"], st["case"]["page"]
    rows = rows.long()
    lens, t = st["lens"][rows].long(), st["table"][rows].long()
    step = torch.arange(c["N"], device=t.device)
    take = step < st["accept"].long()[:, None]
    b = torch.arange(c["n"], device=t.device)[:, None].expand_as(take)[take]
    src, dst = (lens[:, None] + st["path"].long())[take], (lens[:, None] + 1 + step)[take]
    for x in (st["k"], st["v"]):
        x[:, t[b, dst // page], :, dst % page] = x[:, t[b, src // page], :, src % page]
    _release(st, rows, lens + 1 + st["accept"].long())


def _fork(st, src, dst):
    page, src, dst = st["case"]["page"], src.long(), dst.long()
    need = (st["lens"][src].long() + page - 1) // page
    t = st["table"][src].long()
    keep = torch.arange(t.shape[1], device=t.device) < need[:, None]
    st["refs"].index_add_(0, t[keep], torch.ones_like(t[keep], dtype=torch.int32))
    st["table"][dst] = torch.where(keep, t, -1).int()
    st["lens"][dst] = st["lens"][src]
    st["held"][dst] = need.int()
    st["free"].copy_(_bits(st["refs"]))


def _state(st):
    return {x: st[x] for x in ("k", "v", "table", "lens", "held", "refs", "free")}


def _run_plain(st):
    kind, rows = st["case"]["kind"], st["rows"]
    if kind == "attend":
        return _attend(st, 0)
    if kind == "append":
        return {"q": _append(st, 0), "k": st["k"], "v": st["v"]}
    if kind == "fork":
        _release(st, rows, st["zero"])
        _fork(st, st["src"], rows)
        _reserve(st, rows, st["n_tok"])
        return _state(st)
    _release(st, rows, st["base"])
    _reserve(st, rows, st["n_tok"])
    got = {}
    if kind == "step":
        q = _append(st, slice(None))
        back, st["q"] = st["q"], q
        got["out"] = [_attend(st, layer) for layer in range(st["case"]["layers"])]
        st["q"] = back
    else:
        _append(st, slice(None), queries=False)
    _commit(st, rows)
    return {**_state(st), **got}


# --------------------------------------------------------- the framework's ----

def _run_own(st):
    import sam_drafting_verification_gb300 as ss
    c, rows = st["case"], st["rows"]
    kind = c["kind"]
    if "cache" not in st:   # the handle that a program keeps for its cache and its positions
        st["cache"] = ss.KVCache.wrap(*(st[x] for x in ("k", "v", "table", "lens", "held", "refs", "free")))
        st["rope"] = ss.Rope(st["inv_freq"], c["layout"], st["mscale"]) if "inv_freq" in st else None
    cache, rope = st["cache"], st["rope"]
    if kind == "fork":
        cache.truncate(rows, st["zero"])
        cache.fork(st["src"], rows)
        cache.reserve(rows, st["n_tok"])
        return _state(st)
    tree = (st["first_child"], st["next_sibling"]) if c["tree"] else None
    group = st["group"] if c["group"] > 1 else None
    if kind in ("commit", "step"):
        cache.truncate(rows, st["base"])
        cache.reserve(rows, st["n_tok"])
    plan = cache.plan(c["N"], c["q_heads"], rows=rows, n_tok=st["n_tok"], tree=tree, group=group)
    if kind == "attend":
        return cache.attend(0, plan, st["q"][0])
    if kind == "append":
        return {"q": cache.append(0, plan, st["q"][0], st["k_new"][0], st["v_new"][0], rope), "k": st["k"],
                "v": st["v"]}
    got = {}
    for layer in range(c["layers"]):
        q = cache.append(layer, plan, st["q"][layer] if kind == "step" else None, st["k_new"][layer],
                         st["v_new"][layer], rope)
        if kind == "step":
            got.setdefault("out", []).append(cache.attend(layer, plan, q))
    cache.commit(rows, st["accept"], st["path"] if c["tree"] else None)
    return {**_state(st), **got}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work ----

def work(case):
    c = case
    lens, ntok, parent, path, acc = _shape(c)
    n, N, Q, H, D, L, page = (c[x] for x in ("n", "N", "q_heads", "kv_heads", "head_dim", "layers", "page"))
    tok = 2 * 2 * H * D                      # a token's key and value, bytes
    toks = int(ntok.sum())
    state = 4 * (3 * n + int((-(-lens // page)).sum()))
    if c["kind"] == "fork":
        fill = (lens % page)[np.arange(n) // c["group"]]
        return {"bytes": float(state + 2 * L * tok * int(fill.sum())), "flops": 0.0}
    shared = c["shared"] // page * page if c["group"] > 1 else 0
    keys = sum(int(lens[b] + ntok[b]) - (min(shared, int(lens[b])) if b % c["group"] else 0) for b in range(n))
    if c["tree"]:
        depth = np.zeros((n, N), np.int64)
        for j in range(1, N):
            depth[:, j] = depth[np.arange(n), parent[:, j]] + 1
        seen = int((lens * N).sum() + (depth + 1).sum())
    else:
        seen = int((lens * ntok + ntok * (ntok + 1) // 2).sum())
    attend = {"bytes": keys * tok + 2 * 2 * toks * Q * D + state, "flops": 4 * D * Q * seen}
    append = 2 * tok * toks + (2 * 2 * toks * Q * D if c["kind"] != "commit" else 0)
    moved = int((path[:, :] > np.arange(1, N + 1)).sum())
    if c["kind"] == "attend":
        return {"bytes": float(attend["bytes"]), "flops": float(attend["flops"])}
    if c["kind"] == "append":
        return {"bytes": float(append + state), "flops": 6.0 * toks * (Q + H) * c["rot"] // 2}
    if c["kind"] == "commit":
        return {"bytes": float(L * (append + 2 * moved * tok) + 2 * state), "flops": 0.0}
    return {"bytes": float(L * (append + attend["bytes"] + 2 * moved * tok) + 2 * state),
            "flops": float(L * attend["flops"])}


# ------------------------------------------------------------------ exact ----

def _exact_rotate(x, pos, f, m, layout):
    """x [T, heads, D] in 64 bits turned to pos [T]: each pair as a complex number times exp(i angle)."""
    h = f.numel()
    y = x.clone()
    z = (torch.complex(x[..., :h], x[..., h:2 * h]) if layout == "half"
         else torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()))
    z = z * torch.polar(torch.full_like(f, m).expand(len(pos), h), pos.double()[:, None] * f)[:, None]
    y[..., :2 * h] = torch.cat((z.real, z.imag), -1) if layout == "half" else torch.view_as_real(z).flatten(-2)
    return y


def exact(case, seed):
    c = case
    if c["kind"] == "fork":
        return None
    st = prepare(c, seed)
    lens, ntok, parent, path, acc = _shape(c)
    N, page, Q, H, D, L = (c[x] for x in ("N", "page", "q_heads", "kv_heads", "head_dim", "layers"))
    table = st["table"].long()
    depth = np.tile(np.arange(N), (c["n"], 1))
    for j in range(1, N if c["tree"] else 1):
        depth[:, j] = depth[np.arange(c["n"]), parent[:, j]] + 1
    outs = [torch.zeros((c["n"], N, Q, D), dtype=torch.float64, device=table.device) for _ in range(L)]
    qs = [torch.zeros_like(outs[0]) for _ in range(L)]
    write = c["kind"] != "attend"
    if write and c["kind"] != "append":
        return None if c["kind"] == "commit" else _exact_step(st, lens, ntok, parent, depth, outs)
    for b in range(c["n"]):
        T, base = int(ntok[b]), int(lens[b])
        if c["kind"] == "append":
            pos = torch.as_tensor(base + depth[b, :T], device=table.device)
            x = st["q"][0, b, :T].double()
            qs[0][b, :T] = _exact_rotate(x, pos, st["inv_freq"], st["mscale"], c["layout"]) if c["rot"] else x
            continue
        at = torch.arange(base + T, device=table.device)
        k = st["k"][0][table[b, at // page], :, at % page].double()
        v = st["v"][0][table[b, at // page], :, at % page].double()
        outs[0][b, :T] = _exact_one(c, st["q"][0, b, :T].double(), k, v, base, parent[b])
    if c["kind"] == "append":
        k, v = st["k"].double(), st["v"].double()
        for b in range(c["n"]):
            T, base = int(ntok[b]), int(lens[b])
            at = torch.arange(base, base + T, device=table.device)
            pos = torch.as_tensor(base + depth[b, :T], device=table.device)
            x = st["k_new"][0, b, :T].double()
            x = _exact_rotate(x, pos, st["inv_freq"], st["mscale"], c["layout"]) if c["rot"] else x
            k[0][table[b, at // page], :, at % page] = x
            v[0][table[b, at // page], :, at % page] = st["v_new"][0, b, :T].double()
        return {"q": qs[0], "k": k, "v": v}
    return outs[0]


def _exact_one(c, q, k, v, base, parent):
    """One sequence: q [T, Q, D] over k, v [base + T, H, D], head by head."""
    T, Q, D = q.shape
    rep = Q // c["kv_heads"]
    dev = q.device
    if c["tree"]:
        see = np.eye(T, dtype=bool)
        for j in range(1, T):
            see[j] |= see[parent[j]]
        see = torch.as_tensor(see, device=dev)
    else:
        see = torch.ones((T, T), dtype=torch.bool, device=dev).tril()
    bias = torch.zeros((T, base + T), dtype=torch.float64, device=dev)
    bias[:, base:].masked_fill_(~see, -math.inf)
    o = torch.empty_like(q)
    for h in range(Q):
        w = torch.softmax(q[:, h] @ k[:, h // rep].T / math.sqrt(D) + bias, -1)
        o[:, h] = w @ v[:, h // rep]
    return o


def _exact_step(st, lens, ntok, parent, depth, outs):
    """The attention of a whole step, from the keys before they were rounded to the cache's type."""
    c = st["case"]
    page, dt = c["page"], DT[c["dtype"]]
    table = st["table"].long()
    for layer in range(c["layers"]):
        for b in range(c["n"]):
            T, base = int(ntok[b]), int(lens[b])
            pos = torch.as_tensor(base + depth[b, :T], device=table.device)
            at = torch.arange(base, device=table.device)
            q, k, v = (st[x][layer, b, :T].double() for x in ("q", "k_new", "v_new"))
            if c["rot"]:
                q, k = (_exact_rotate(x, pos, st["inv_freq"], st["mscale"], c["layout"]) for x in (q, k))
                q, k = q.to(dt).double(), k.to(dt).double()   # both are held in the cache's type between the calls
            k = torch.cat((st["k"][layer][table[b, at // page], :, at % page].double(), k))
            v = torch.cat((st["v"][layer][table[b, at // page], :, at % page].double(), v))
            outs[layer][b, :T] = _exact_one(c, q, k, v, base, parent[b])
    return {"k": None, "v": None, "table": None, "lens": None, "held": None, "refs": None, "free": None,
            "out": outs}
