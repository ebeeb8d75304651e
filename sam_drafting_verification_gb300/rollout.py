"""Host loop of a speculative rollout over the library's decode step.

Each step drafts with the sequences' suffix automata and verifies the drafts
against the target model's logits in one `sam_spec_step` call ("SAM投机推理：
长序列强化学习训练加速利器" §1.1).  Whether a step speculates follows the
adaptive switch of the same article, §3.1.1: drafting is on only while the
number of active requests is at most a threshold (late in a rollout, when a
few long requests are left).

The loop keeps the active set on the host (it reads each step's emitted
tokens back to detect finished sequences); everything per token runs in the
library's kernels.  The target model is a callable:

    model(rows, n_done, draft, draft_len) -> logits [n, K+1, V]

with rows (int32 [n], the automata / sequences of this step), n_done (int64
[n], tokens each has generated so far), draft (int32 [n, K]) and draft_len
(int32 [n]); row j of a sequence's logits scores the token after its first j
drafts.

With a KVCache the loop also keeps the cache: it reserves each step's slots,
plans the pass, commits what was accepted and frees finished sequences.  The
model then gets what such a pass works on:

    model(rows, n_done, tokens, n_tok, plan) -> logits [n, K+1, V]

with tokens (int32 [n, K+1]: the last token, which the cache does not hold yet,
and the drafts, -1 behind them), n_tok (int32 [n], 1 + draft_len) and the plan
for cache.append and cache.attend.
"""
from __future__ import annotations

from dataclasses import dataclass, field

import torch

from . import KVCache, SamBatch, verify_workspace


def speculation_k(n_active: int, threshold: int | None, K: int) -> int:
    """Draft length for a step with n_active requests: K while n_active is at
    most the threshold (no threshold: always), else 0 (plain decoding)."""
    if threshold is None or n_active <= threshold:
        return int(K)
    return 0


@dataclass
class RolloutResult:
    tokens: list                      # generated tokens per sequence (python ints)
    steps: int = 0                    # decode steps run
    k_per_step: list = field(default_factory=list)       # draft length used by each step
    active_per_step: list = field(default_factory=list)  # active sequences at each step
    accepted: int = 0                 # drafts accepted over the rollout


class Rollout:
    def __init__(self, batch: SamBatch, model, K: int = 3, threshold: int | None = None,
                 temperature: float = 0.0, seed: int = 0, eos: int | None = None,
                 cache: KVCache | None = None, q_heads: int | None = None, last=None, group=None):
        """cache: row b holds sequence b's prompt but for its last token, which
        is last[b] (int32 [B], on the device).  q_heads: the model's query
        heads.  group (int32 [B], optional): sequences of one number that
        follow one another share pages (KVCache.plan)."""
        self.batch, self.model, self.K = batch, model, int(K)
        self.threshold, self.temperature, self.seed, self.eos = threshold, float(temperature), int(seed), eos
        self.cache, self.q_heads, self.last, self.group = cache, q_heads, last, group
        if cache is not None:
            if q_heads is None or last is None:
                raise ValueError("a cache needs q_heads and last")
            if cache.seqs < batch.B:
                raise ValueError(f"the cache has {cache.seqs} sequences, the batch {batch.B}")

    def run(self, max_new_tokens) -> RolloutResult:
        """Generates up to max_new_tokens[b] tokens per sequence (or until eos)
        from the automata's current texts (prompts already extended).

        The step that finishes a sequence extends its automaton by every token
        that step emitted, so the automaton may hold up to K tokens beyond the
        ones returned for it (those after its eos or past its limit).  A
        finished sequence's automaton is not used again by this rollout; a
        caller that goes on with it should reset and rebuild it from the
        returned text.  With a cache, a finished sequence's row is emptied and
        its pages are given back (one whose limit is 0 takes no part: its row
        stays as it is).  Where run raises for a sequence that the cache had no
        room for, every row of that step stands for what it holds: the refused
        ones as before the step, the others with the step's accepted tokens."""
        dev = self.batch.device
        B = self.batch.B
        limit = [int(x) for x in max_new_tokens]
        out = [[] for _ in range(B)]
        active = [b for b in range(B) if limit[b] > 0]
        res = RolloutResult(tokens=out)
        if not active:
            return res
        rows = torch.tensor(active, dtype=torch.int32, device=dev)
        k = speculation_k(len(active), self.threshold, self.K)
        empty = torch.zeros((len(active), 0), dtype=torch.int32, device=dev)
        zero = torch.zeros(len(active), dtype=torch.int32, device=dev)
        # the first drafts: an empty extension that drafts k tokens
        draft, dlen, _, _ = self.batch.step_rows(rows, empty, zero, k)
        # one workspace for the whole rollout, and one buffer for the per-step
        # outputs the host reads (emit, emit_len, status, accept_len), so that
        # a step costs one device-to-host copy
        ws = verify_workspace(len(active), self.K, 1, dev)
        hostbuf = torch.empty(len(active) * (self.K + 5), dtype=torch.int32, device=dev)
        cache, plan_status = self.cache, None
        if cache is not None:
            last = self.last[rows.long()]
            group = self.group[rows.long()] if self.group is not None else None
        step = 0
        while active:
            n = len(active)
            n_done = torch.tensor([len(out[b]) for b in active], dtype=torch.int64, device=dev)
            if cache is None:
                logits = self.model(rows, n_done, draft, dlen)
            else:
                n_tok = dlen + 1
                cache.reserve(rows, n_tok)   # what it refuses, the plan refuses
                plan = cache.plan(int(draft.shape[1]) + 1, self.q_heads, rows=rows, n_tok=n_tok, group=group)
                logits = self.model(rows, n_done, torch.cat((last[:, None], draft), 1), n_tok, plan)
            k_next = speculation_k(n, self.threshold, self.K)
            K1 = int(draft.shape[1]) + 1
            o = {"emit": hostbuf[:n * K1].view(n, K1), "emit_len": hostbuf[n * K1:n * K1 + n],
                 "status": hostbuf[n * K1 + n:n * K1 + 2 * n],
                 "accept_len": hostbuf[n * K1 + 2 * n:n * K1 + 3 * n]}
            r = self.batch.spec_step(logits, draft, dlen, K_next=k_next, rows=rows,
                                     temperature=self.temperature, seed=self.seed, step=step,
                                     workspace=ws, out=o)
            res.k_per_step.append(int(draft.shape[1]))
            res.active_per_step.append(n)
            read = n * K1 + 3 * n
            if cache is not None:
                last = r["out_token"]
                # of a sequence that the plan refused, or whose attention gave up,
                # the slots hold no keys and values: nothing is kept
                refused = plan.status
                cache.commit(rows, torch.where(refused == 0, r["accept_len"], -1))
                hostbuf[read:read + n] = refused
                read += n
            h = hostbuf[:read].cpu()
            if cache is not None:
                plan_status = h[n * K1 + 3 * n:].tolist()
            emit = h[:n * K1].view(n, K1).tolist()
            elen = h[n * K1:n * K1 + n].tolist()
            st = h[n * K1 + n:n * K1 + 2 * n].tolist()
            acc = h[n * K1 + 2 * n:n * K1 + 3 * n].tolist()
            keep = []
            for i, b in enumerate(active):
                if plan_status is not None and plan_status[i] != 0:
                    raise RuntimeError(f"sequence {b}: cache status {plan_status[i]}")
                if st[i] != 0:
                    raise RuntimeError(f"sequence {b}: verification status {st[i]}")
                res.accepted += acc[i]
                toks = emit[i][:elen[i]]
                room = limit[b] - len(out[b])
                stop = False
                for t in toks[:room]:
                    out[b].append(t)
                    if self.eos is not None and t == self.eos:
                        stop = True
                        break
                if not stop and len(out[b]) < limit[b]:
                    keep.append(i)
            step += 1
            res.steps = step
            if len(keep) != n:
                idx = torch.tensor(keep, dtype=torch.int64, device=dev)
                if cache is not None:
                    kept = set(keep)
                    cache.truncate(torch.tensor([b for i, b in enumerate(active) if i not in kept],
                                                dtype=torch.int32, device=dev))
                    last = last[idx].contiguous()
                    group = group[idx].contiguous() if group is not None else None
                active = [active[i] for i in keep]
                rows = rows[idx].contiguous()
                draft = r["next_draft"][idx].contiguous()
                dlen = r["next_draft_len"][idx].contiguous()
            else:
                draft, dlen = r["next_draft"], r["next_draft_len"]
        return res
