"""A plain statement of the paged cache for the tests: its bookkeeping in Python
integers and numpy, its rotary append and attention in 64 bits."""
import math

import numpy as np
import torch

ST_OK, ST_CAPACITY, ST_BADDRAFT, ST_PAGE, ST_ROW = 0, 1, 6, 10, 11


class Pages:
    """The bookkeeping.  `data` [layers, pages, kv_heads, page, head_dim] stands
    for both pools (None: counts only)."""

    def __init__(self, pages, page, seqs, max_pages, data=None):
        self.page, self.max_pages = page, max_pages
        self.table = np.full((seqs, max_pages), -1, np.int64)
        self.lens = np.zeros(seqs, np.int64)
        self.held = np.zeros(seqs, np.int64)
        self.refs = np.zeros(pages, np.int64)
        self.data = data

    def free_bits(self):
        n = self.refs.size
        w = np.zeros((n + 31) // 32, np.uint32)
        for p in range(n):
            if self.refs[p] == 0:
                w[p // 32] |= np.uint32(1 << (p % 32))
        return w.view(np.int32)

    def pages_of(self, tokens):
        return -(-int(tokens) // self.page)

    def reserve(self, rows, n_tok):
        st, free, at, shared = [], [p for p in range(self.refs.size) if self.refs[p] == 0], 0, self.refs.copy()
        for i, row in enumerate(rows):
            nt = int(n_tok[i])
            if not 0 <= row < len(self.lens) or row in rows[:i]:
                st.append(ST_ROW)
                continue
            if nt < 0:
                st.append(ST_BADDRAFT)
                continue
            n = int(self.lens[row])
            want = self.pages_of(n + nt)
            if want > self.max_pages:
                st.append(ST_CAPACITY)
                continue
            more = max(0, want - int(self.held[row]))
            cow = n % self.page != 0 and shared[self.table[row, n // self.page]] > 1
            if more + cow and at + more + cow > len(free):
                st.append(ST_CAPACITY)
                at = len(free) if at + more + cow > len(free) else at
                continue
            got = free[at:at + more + cow]
            at += more + cow
            if cow:
                old, new = self.table[row, n // self.page], got.pop(0)
                self.table[row, n // self.page] = new
                self.refs[old] -= 1
                self.refs[new] = 1
                if self.data is not None:
                    for d in self.data:
                        d[:, new, :, :n % self.page] = d[:, old, :, :n % self.page]
            for p in got:
                self.table[row, self.held[row]] = p
                self.held[row] += 1
                self.refs[p] = 1
            st.append(ST_OK)
        return st

    def fork(self, src, dst):
        st = []
        ok = [0 <= s < len(self.lens) and 0 <= d < len(self.lens) and dst.count(d) == 1 and d not in src and s not in dst
              and self.lens[d] == 0 and self.held[d] == 0 for s, d in zip(src, dst)]
        for s, d, good in zip(src, dst, ok):
            if good:
                k = self.pages_of(self.lens[s])
                self.table[d] = -1
                self.table[d, :k] = self.table[s, :k]
                self.refs[self.table[s, :k]] += 1
                self.lens[d], self.held[d] = self.lens[s], k
            st.append(ST_OK if good else ST_ROW)
        return st

    def set_len(self, row, n):
        k = self.pages_of(n)
        for x in range(k, int(self.held[row])):
            self.refs[self.table[row, x]] -= 1
            self.table[row, x] = -1
        self.lens[row], self.held[row] = n, min(k, int(self.held[row]))

    def truncate(self, rows, new_len):
        st = []
        for i, row in enumerate(rows):
            if not 0 <= row < len(self.lens) or rows.count(row) > 1:
                st.append(ST_ROW)
            elif new_len[i] < 0:
                st.append(ST_BADDRAFT)
            else:
                self.set_len(row, min(int(self.lens[row]), int(new_len[i])))
                st.append(ST_OK)
        return st

    def commit(self, rows, accept, path=None):
        st, refs = [], self.refs.copy()
        for i, row in enumerate(rows):
            a = int(accept[i])
            if not 0 <= row < len(self.lens) or rows.count(row) > 1:
                st.append(ST_ROW)
                continue
            N = 1 << 30 if path is None else path.shape[1]
            nodes = list(range(1, a + 1)) if path is None else [int(x) for x in path[i, :max(a, 0)]]
            if not -1 <= a < N or any(not 0 < x < N for x in nodes) or any(x >= y for x, y in zip(nodes, nodes[1:])):
                st.append(ST_BADDRAFT)
                continue
            n = int(self.lens[row])
            if n + (nodes[-1] if nodes else a) + 1 > self.held[row] * self.page:
                st.append(ST_CAPACITY)
                continue
            if path is not None and any(refs[self.table[row, x]] > 1
                                        for x in range(n // self.page, self.pages_of(n + 1 + a))):
                st.append(ST_CAPACITY)
                continue
            if self.data is not None:
                for d in self.data:
                    for t, x in enumerate(nodes):
                        s, e = n + x, n + 1 + t
                        d[:, self.table[row, e // self.page], :, e % self.page] = \
                            d[:, self.table[row, s // self.page], :, s % self.page]
            self.set_len(row, n + 1 + a)
            st.append(ST_OK)
        return st


def random_parents(rng, n, N, reach=6, width=3):
    parent = np.full((n, N), -1, np.int64)
    for b in range(n):
        kids = np.zeros(N, int)
        for j in range(1, N):
            cand = [p for p in range(max(0, j - reach), j) if kids[p] < width]
            parent[b, j] = cand[int(rng.integers(0, len(cand)))]
            kids[parent[b, j]] += 1
    return parent


def links(parent):
    """(first_child, next_sibling) int32 of parents [n, N]."""
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


def sight(parent):
    """Of one tree: see [N, N] (node j sees node i) and depths."""
    N = len(parent)
    see, depth = np.eye(N, dtype=bool), np.zeros(N, np.int64)
    for j in range(1, N):
        see[j] |= see[parent[j]]
        depth[j] = depth[parent[j]] + 1
    return see, depth


def attend(q, k, v, base, see, scale):
    """One sequence in 64 bits: q [T, Q, D], k, v [base + T, H, D], see [T, T].
    Returns the output and the bound of its error in a 16-bit type of half step
    u: |out - exact| <= u |exact| + (u + e) * sum p |v|, e the fp32 part: scores
    of D products each (their sum's error at most D 2^-23 of the sum of
    magnitudes, twice for numerator and denominator), exponentials to 2^-20, and
    sums over the keys (2^-23 a key).  Per element: (exact, sum p |v|, e)."""
    T, Q, D = q.shape
    rep = Q // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, mag, err = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(T, Q, 1, dtype=torch.float64, device=q.device)
    ok = torch.ones((T, base + T), dtype=torch.bool, device=q.device)
    ok[:, base:] = torch.as_tensor(see, device=q.device)
    for h in range(Q):
        s = (q[:, h] @ k[:, h // rep].T * scale).masked_fill(~ok, -math.inf)
        a = (q[:, h].abs() @ k[:, h // rep].abs().T * abs(scale)).masked_fill(~ok, 0).amax(1, keepdim=True)
        p = torch.softmax(s, -1)
        out[:, h] = p @ v[:, h // rep]
        mag[:, h] = p @ v[:, h // rep].abs()
        err[:, h] = 2 * D * 2.0 ** -23 * a + 2.0 ** -19 + 2 * (base + T) * 2.0 ** -23
    return out, mag, err


def rotate(x, pos, inv_freq, layout, mscale):
    """x [T, heads, D] to positions pos [T] (Python integers), 64 bits; angles
    reduced in exact integers first."""
    rot = 2 * len(inv_freq)
    y = x.double().clone()
    for t, p in enumerate(pos):
        for j, f in enumerate(inv_freq):
            a = math.fmod(int(p) * float(f), 2 * math.pi) if int(p) < 1 << 20 else _far(int(p), float(f))
            c, s = math.cos(a) * mscale, math.sin(a) * mscale
            i0, i1 = (j, j + rot // 2) if layout == "half" else (2 * j, 2 * j + 1)
            u, w = y[t, :, i0].clone(), y[t, :, i1].clone()
            y[t, :, i0], y[t, :, i1] = u * c - w * s, u * s + w * c
    return y


def _far(p, f):
    from fractions import Fraction
    two_pi = Fraction(31415926535897932384626433832795028841971, 5 * 10 ** 39)
    a = Fraction(f) * p
    return float(a - (a // two_pi) * two_pi)
