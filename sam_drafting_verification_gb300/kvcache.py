"""The paged key/value cache of the target model and the attention of a
verification pass (include/samspec_kv.h), over torch CUDA tensors.

A decode step of a model with a cache, between drafting and verification:

    cache.reserve(rows, n_tok)                       # slots for the new tokens
    plan = cache.plan(N, q_heads, rows=rows, n_tok=n_tok)      # or tree=(first_child, next_sibling)
    for each layer:
        q = cache.append(layer, plan, q, k, v, rope) # rotate, write keys and values
        o = cache.attend(layer, plan, q)             # [n, N, q_heads, head_dim]
    ... logits, spec_verify / spec_verify_tree ...
    cache.commit(rows, accept_len, path)             # keep what was accepted

A sequence's new tokens are its last emitted token (not in the cache yet) and
the K drafts, so N = K + 1; a draft tree's node 0 is that token.
"""
from __future__ import annotations

import ctypes
import math
import sys

import torch

from . import _binding as _b
from . import _cuda_device, _req

_pkg = sys.modules[__package__]
_DTYPES = {torch.bfloat16: _b.BF16, torch.float16: _b.F16}
# Memory of a plan that is gone is kept for the next one up to this size (two of
# them a stream): it saves some 5 us of host time a plan.  Plans beyond it, of long
# prompts or large groups, work for far longer than that, and their memory returns
# to torch's allocator.
_SPARE_BYTES = 64 << 20


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Radians per position of each of the rot / 2 pairs (fp64, on the host), and
    the factor that queries and keys are scaled by.  scaling:
      "none"    base^(-2j / rot)
      "linear"  positions divided by `factor`
      "ntk"     the base stretched to base * factor^(rot / (rot - 2)): the
                lowest frequency divided by factor, the highest kept
      "yarn"    YaRN (Peng et al. 2023): pairs that turn more than beta_fast
                times over original_len positions kept, those that turn less
                than beta_slow times divided by factor, a linear ramp over the
                pairs between; queries and keys scaled by 0.1 ln(factor) + 1
    """
    rot = int(rot)
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not (base > 0 and factor > 0):
        raise ValueError("base and factor must be positive")
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling in ("none", "ntk"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        raise ValueError(f"unknown scaling {scaling!r}")

    def pair_of(turns):   # the pair that turns so many times over original_len positions
        return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f / factor * ramp + f * (1 - ramp), (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


class Rope:
    """Rotary positions: `inv_freq` fp64 CUDA tensor [rot / 2] (radians per
    position), layout "half" (pairs (j, j + rot / 2)) or "interleaved" (pairs
    (2j, 2j + 1)) of the first rot elements of a head, scaled by mscale."""

    def __init__(self, inv_freq, layout: str = "half", mscale: float = 1.0):
        if layout not in ("half", "interleaved"):
            raise ValueError("layout must be 'half' or 'interleaved'")
        self.inv_freq = _req(inv_freq, torch.float64, "inv_freq")
        if inv_freq.dim() != 1 or inv_freq.numel() < 1:
            raise ValueError("inv_freq must be [rot / 2]")
        self.rot = 2 * inv_freq.numel()
        self.layout = _b.ROPE_HALF if layout == "half" else _b.ROPE_INTERLEAVED
        self.mscale = float(mscale)
        if not math.isfinite(self.mscale):
            raise ValueError("mscale must be finite")


class KVPlan:
    """The plan of one pass (KVCache.plan): `status` int32 [n], one word per
    sequence (0: takes part), and the device memory that kv_append and
    kv_attend read and work in (of the cache that made it, or one of the same
    sizes and table).  It belongs to the stream that it was made on:
    where another one reads it, keep the plan until that one is done, and where a
    graph was captured with it, as long as that is replayed."""

    def __init__(self, n, N, q_heads, grouped, buf, nbytes, sizes, spare=None):
        self.sizes = sizes   # of the cache: what it holds are that one's rows and pages
        self.n, self.N, self.q_heads, self.grouped, self.buf, self.bytes = n, N, q_heads, grouped, buf, nbytes
        self.ptr = buf.data_ptr()
        self._spare = spare

    @property
    def status(self):
        self._spare = None   # the view may outlive the plan
        return self.buf[:4 * self.n].view(torch.int32)

    def __del__(self):
        # the cache's next plan on the stream may take the memory (allocating
        # and freeing it anew takes as long as the rest of a small call)
        spare = getattr(self, "_spare", None)
        if spare is not None and len(spare) < 2:
            spare.append(self.buf)


class KVCache:
    """A paged cache for `seqs` sequences: pools k, v [layers, pages, kv_heads,
    page, head_dim] (bfloat16 or float16), a page table, committed lengths,
    pages held, references and free pages.  The tensors are the caller's to
    read; only the calls below change them."""

    def __init__(self, layers: int, pages: int, page: int, kv_heads: int, head_dim: int, seqs: int,
                 max_pages: int, dtype=torch.bfloat16, device=None):
        dev = _cuda_device(device)
        i32 = lambda *s, fill=0: torch.full(s, fill, dtype=torch.int32, device=dev)  # noqa: E731
        if dtype not in _DTYPES:
            raise TypeError("the cache's dtype must be bfloat16 or float16")
        if min(layers, pages, page, kv_heads, head_dim, seqs, max_pages) < 1:
            raise ValueError("sizes must be positive")
        free = i32((pages + 31) // 32, fill=-1)
        if pages % 32:
            free[-1] = (1 << pages % 32) - 1
        self._set(torch.empty((layers, pages, kv_heads, page, head_dim), dtype=dtype, device=dev),
                  torch.empty((layers, pages, kv_heads, page, head_dim), dtype=dtype, device=dev),
                  i32(seqs, max_pages, fill=-1), i32(seqs), i32(seqs), i32(pages), free)

    @classmethod
    def wrap(cls, k, v, table, lens, held, refs, free):
        """A cache over tensors that the caller holds: k, v [layers, pages,
        kv_heads, page, head_dim], table int32 [seqs, max_pages], lens and held
        int32 [seqs], refs int32 [pages], free int32 [ceil(pages / 32)] (a bit
        for each page, set where refs is 0)."""
        self = cls.__new__(cls)
        self._set(k, v, table, lens, held, refs, free)
        return self

    def _set(self, k, v, table, lens, held, refs, free):
        if not isinstance(k, torch.Tensor) or k.dtype not in _DTYPES:
            raise TypeError("k must be a bfloat16 or float16 tensor")
        if k.dim() != 5:
            raise ValueError("k must be [layers, pages, kv_heads, page, head_dim]")
        dev = k.device
        _req(k, k.dtype, "k")
        _req(v, k.dtype, "v", k.shape, dev)
        _req(table, torch.int32, "table", None, dev)
        if table.dim() != 2:
            raise ValueError("table must be [seqs, max_pages]")
        seqs, max_pages = table.shape
        layers, pages, kv_heads, page, head_dim = k.shape
        _req(lens, torch.int32, "lens", (seqs,), dev)
        _req(held, torch.int32, "held", (seqs,), dev)
        _req(refs, torch.int32, "refs", (pages,), dev)
        _req(free, torch.int32, "free", ((pages + 31) // 32,), dev)
        self.k, self.v, self.table, self.lens, self.held, self.refs, self.free = k, v, table, lens, held, refs, free
        self.device, self.dtype = dev, k.dtype
        self.layers, self.pages, self.kv_heads, self.page, self.head_dim = (int(x) for x in k.shape)
        self.seqs, self.max_pages = int(seqs), int(max_pages)
        self.lib = _b.lib()
        self._desc = _b.KvCacheDesc(*(t.data_ptr() for t in (k, v, table, lens, held, refs, free)),
                                    _DTYPES[k.dtype], *(int(x) for x in (layers, pages, page, kv_heads, head_dim,
                                                                         seqs, max_pages)))
        self._ref = ctypes.byref(self._desc)
        if self.lib.kv_reserve_workspace_bytes(self._ref, 1) == 0:   # what every call would refuse
            raise _b.SamspecError(f"a cache outside the limits: {tuple(k.shape)}, {seqs} x {max_pages} pages, "
                                  "or k and v not 16-byte aligned")
        self._sizes = (dev, self.page, self.kv_heads, self.head_dim, self.seqs, self.max_pages)
        self._bytes = {}   # workspace sizes by call sizes
        self._spare = {}   # by stream: memory of plans that are gone

    # -- helpers ---------------------------------------------------------------
    def _call(self, name, *args):
        """The entry point on the device's current stream, with that device
        current for the launch."""
        index = self.device.index
        if self.device.type != "cuda":
            rc = getattr(self.lib, name)(self._ref, *args, _pkg._stream(self.device))
        elif index == torch.cuda.current_device():
            rc = getattr(self.lib, name)(self._ref, *args, _pkg._raw_stream(index))
        else:
            with torch.cuda.device(self.device):
                rc = getattr(self.lib, name)(self._ref, *args, _pkg._raw_stream(index))
        if rc != _b.OK:
            _b.check(rc, name)

    def _i32(self, t, name, shape):
        # the common case in a few comparisons; _req says what is wrong
        try:
            if t.dtype is torch.int32 and t.shape == shape and t.device == self.device and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            pass
        return _req(t, torch.int32, name, shape, self.device).data_ptr()

    def _rows(self, rows, n=None):
        """(how many sequences a call names, the pointer)"""
        if rows is None:
            n = self.seqs if n is None else n
            if n > self.seqs:
                raise ValueError(f"{n} sequences named, the cache has {self.seqs}")
            return n, None
        if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
            raise ValueError("rows must be an int32 tensor [n]")
        n = rows.shape[0] if n is None else n
        return n, self._i32(rows, "rows", (n,))

    def _status(self, n, out):
        if out is None:
            return torch.empty(n, dtype=torch.int32, device=self.device)
        self._i32(out, "out", (n,))
        return out

    # -- pages -----------------------------------------------------------------
    def reserve(self, rows, n_tok, out=None):
        """Room for n_tok more tokens (int32 [n], or one number) behind the
        committed ones of sequences `rows` (int32 [n], or None for all).  Returns
        the status words int32 [n]: ST_CAPACITY where pages ran out, or the
        sequence would be longer than its table."""
        if isinstance(n_tok, torch.Tensor):
            if n_tok.dim() != 1:
                raise ValueError("n_tok must be [n]")
            n, rp = self._rows(rows, n_tok.shape[0])
            most, np = 1 << 30, self._i32(n_tok, "n_tok", (n,))   # (the call's limit, past any cache's)
        else:
            n, rp = self._rows(rows)
            most, np = max(-1, min(int(n_tok), (1 << 31) - 1)), None   # (the call takes 32 bits)
        st = self._status(n, out)
        need = self._bytes.get(n)
        if need is None:
            need = self._bytes[n] = int(self.lib.kv_reserve_workspace_bytes(self._ref, n))
        ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self._call("kv_reserve", rp, n, most, np, st.data_ptr(), ws.data_ptr(), need)
        return st

    def fork(self, src, dst, out=None):
        """Sequences dst (int32 [n], empty) become copies of src (int32 [n]),
        sharing their pages.  Returns the status words int32 [n]."""
        if src is None or dst is None:
            raise ValueError("src and dst must be int32 tensors [n]")
        n, sp = self._rows(src)
        _, dp = self._rows(dst, n)
        st = self._status(n, out)
        self._call("kv_fork", sp, dp, n, st.data_ptr())
        return st

    def commit(self, rows, accept_len, path=None, out=None):
        """Keeps the last emitted token and the accepted drafts of a pass:
        accept_len int32 [n] (spec_verify, spec_verify_tree; -1 keeps nothing),
        path int32 [n, N] (spec_verify_tree; None for chains).  Returns the
        status words int32 [n]."""
        if not isinstance(accept_len, torch.Tensor) or accept_len.dim() != 1:
            raise ValueError("accept_len must be an int32 tensor [n]")
        n, rp = self._rows(rows, accept_len.shape[0])
        ap, pp, N = self._i32(accept_len, "accept_len", (n,)), None, 1 << 30
        if path is not None:
            if not isinstance(path, torch.Tensor) or path.dim() != 2:
                raise ValueError("path must be an int32 tensor [n, N]")
            N = path.shape[1]
            pp = self._i32(path, "path", (n, N))
        st = self._status(n, out)
        self._call("kv_commit", rp, n, N, ap, pp, st.data_ptr())
        return st

    def truncate(self, rows, new_len=None, out=None):
        """Cuts sequences to at most new_len tokens (int32 [n]; None: empties
        them) and gives back the pages behind, reserved ones too."""
        lp = None
        if new_len is not None:
            if not isinstance(new_len, torch.Tensor) or new_len.dim() != 1:
                raise ValueError("new_len must be an int32 tensor [n]")
            n, rp = self._rows(rows, new_len.shape[0])
            lp = self._i32(new_len, "new_len", (n,))
        else:
            n, rp = self._rows(rows)
        st = self._status(n, out)
        self._call("kv_truncate", rp, n, lp, st.data_ptr())
        return st

    # -- a pass ------------------------------------------------------------------
    def plan(self, N: int, q_heads: int, rows=None, n_tok=None, tree=None, group=None, out=None):
        """Plans a pass of up to N new tokens for each of the sequences `rows`
        (int32 [n], or None for all): n_tok int32 [n] of them, a chain (None: N),
        or tree=(first_child, next_sibling) int32 [n, N] as for spec_verify_tree.
        group int32 [n]: consecutive sequences of one number read the pages
        that they share once (those without tokens, or with a status, count for
        nothing).  out: the plan of an earlier call with the same
        sizes, written again in place."""
        N, q_heads = int(N), int(q_heads)
        n, rp = self._rows(rows)
        np = fp = sp = gp = None
        if tree is not None:    # every node takes part
            fp = self._i32(tree[0], "first_child", (n, N))
            sp = self._i32(tree[1], "next_sibling", (n, N))
        elif n_tok is not None:
            np = self._i32(n_tok, "n_tok", (n,))
        if group is not None:
            gp = self._i32(group, "group", (n,))
        if out is None:
            key = (n, N, q_heads, gp is not None)
            need = self._bytes.get(key)
            if need is None:
                need = self._bytes[key] = int(self.lib.kv_plan_bytes(self._ref, n, N, q_heads, gp is not None))
            if need == 0:
                raise _b.SamspecError(f"sizes outside the limits: n={n}, N={N}, q_heads={q_heads}")
            out = self._new_plan(n, N, q_heads, gp is not None, need)
        elif (out.n, out.N, out.q_heads) != (n, N, q_heads) or out.sizes != self._sizes or \
                (gp is not None and not out.grouped):
            raise ValueError("out: a plan of other sizes")
        self._call("kv_plan", rp, n, N, q_heads, np, fp, sp, gp, out.ptr, out.bytes)
        return out

    def _capturing(self):
        """Is the stream that the calls go to (the cache's device's, which need not
        be the current one) being captured in a graph?"""
        if torch.cuda.device_count() > 1 and torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                return torch.cuda.is_current_stream_capturing()
        return torch.cuda.is_current_stream_capturing()

    def _new_plan(self, n, N, q_heads, grouped, need):
        # memory of a plan that is gone, if one of about this size was used on
        # this stream (and is small enough to be kept); not inside a graph capture,
        # whose graph keeps its own
        spare = buf = None
        if need <= _SPARE_BYTES and self.device.type == "cuda" and not self._capturing():
            spare = self._spare.setdefault(_pkg._raw_stream(self.device.index), [])
            try:
                for _ in range(2):   # taken out before it is looked at: another thread may do the same
                    x = spare.pop(0)
                    if need <= x.numel() <= 4 * need:
                        buf = x
                        break
                    spare.append(x)
            except IndexError:
                pass
        if buf is None:
            if spare:
                spare.clear()
            buf = torch.empty(need, dtype=torch.uint8, device=self.device)
        return KVPlan(n, N, q_heads, grouped, buf, need, self._sizes, spare)

    def _tokens(self, t, name, plan, heads):
        """t [n, N, heads, head_dim] of the cache's dtype, checked; its token
        stride in elements.  A view into a wider projection output will do."""
        if plan.sizes is not self._sizes and plan.sizes != self._sizes:
            raise ValueError("the plan is one of a cache of other sizes")
        shape = (plan.n, plan.N, heads, self.head_dim)
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a CUDA tensor")
        if t.dtype is not self.dtype:
            raise TypeError(f"{name} must be {self.dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        s, row = t.stride(), heads * self.head_dim
        step = s[1] if plan.N > 1 else s[0] if plan.n > 1 else row
        if s[3] != 1 or (heads > 1 and s[2] != self.head_dim) or (plan.n > 1 and s[0] != plan.N * step) or step < row:
            raise ValueError(f"{name}: tokens must follow one another at one stride, heads and elements without gaps")
        return step

    def _output(self, out, plan):
        shape = (plan.n, plan.N, plan.q_heads, self.head_dim)
        if out is None:
            return torch.empty(shape, dtype=self.dtype, device=self.device)
        return _req(out, self.dtype, "out", shape, self.device)

    def append(self, layer: int, plan: KVPlan, q, k, v, rope: Rope | None = None, out=None):
        """Writes the new tokens' keys and values k, v [n, N, kv_heads, head_dim]
        into their slots of `layer`, keys turned to their positions, and returns
        the turned queries (q [n, N, q_heads, head_dim]; out may be q itself
        where that is contiguous; None: keys and values only)."""
        qs, qp, op = 0, None, None
        if q is not None:
            qs = self._tokens(q, "q", plan, plan.q_heads)
            out = self._output(out, plan)
            qp, op = q.data_ptr(), out.data_ptr()
        else:
            out = None
        ks, vs = self._tokens(k, "k", plan, self.kv_heads), self._tokens(v, "v", plan, self.kv_heads)
        rot, layout, mscale, freq = 0, 0, 1.0, None
        if rope is not None:
            if rope.rot > self.head_dim:
                raise ValueError("rope: more pairs than the head has")
            if rope.inv_freq.device != self.device:
                raise ValueError(f"rope must be on {self.device}, got {rope.inv_freq.device}")
            rot, layout, mscale, freq = rope.rot, rope.layout, rope.mscale, rope.inv_freq.data_ptr()
        self._call("kv_append", int(layer), plan.ptr, plan.n, plan.N, plan.q_heads, qp, qs, op, k.data_ptr(), ks,
                   v.data_ptr(), vs, freq, rot, layout, mscale)
        return out

    def attend(self, layer: int, plan: KVPlan, q, scale: float | None = None, out=None):
        """softmax(scale q k^T) v of each new token over what it sees (scale:
        1 / sqrt(head_dim) unless given).  Returns [n, N, q_heads, head_dim];
        tokens that take no part get zeros."""
        qs = self._tokens(q, "q", plan, plan.q_heads)
        out = self._output(out, plan)
        self._call("kv_attend", int(layer), plan.ptr, plan.bytes, plan.n, plan.N, plan.q_heads, q.data_ptr(), qs,
                   self.head_dim ** -0.5 if scale is None else float(scale), out.data_ptr())
        return out
