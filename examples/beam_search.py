"""Beam search over a paged cache, every operator around it together.

The prompts of a batch go into the cache in chunks; then each sequence has
several beams, which share the pages of what they have in common:

    table, lengths, counts, copies = spec_pages_fork(table, lengths, parents, counts)
    spec_pages_copy(caches, copies)
    each layer:  lengths = spec_chunk_append(k, v, caches, rows, lengths, table)
                 plan = spec_chunk_plan(rows, lengths, q, caches, table)    once
                 out = spec_chunk_attention(q, caches, plan, table)
    logits = spec_process_logits(logits, history, penalties, masks)
    tokens, beams, scores = spec_beam_select(logits, scores, ended beams, lengths' powers)
    history, ... = spec_beam_reorder(history, beams)

and, when the best beam of each is left, spec_pages_compact gives the end of the
pool back.  Run it with ``python examples/beam_search.py`` on a GPU with the
library built.
"""
from __future__ import annotations

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
for path in (HERE, os.path.dirname(HERE)):
    if path not in sys.path:
        sys.path.insert(0, path)

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tree_step import Model  # noqa: E402


class Search:
    """A batch's beams: rows b K .. b K + K - 1 of the table are sequence b's (before the first
    selection, and after keep_best, one row each)."""

    def __init__(self, model, prompts, beams=4, page=16, most=128, chunk=24, end_token=0, alpha=0.7,
                 frequency=0.0, allowed=None):
        self.model, self.B, self.K, self.page = model, len(prompts), beams, page
        self.end_token, self.alpha, self.frequency, self.allowed = end_token, alpha, frequency, allowed
        B, dev, L = self.B, "cuda", len(model.layers)
        i32 = dict(dtype=torch.int32, device=dev)
        pages = -(-most // page)
        shape = (L, B * beams * pages, page, model.kv_heads, model.head_dim)
        self.k_cache = torch.empty(shape, dtype=model.embed.dtype, device=dev)
        self.v_cache = torch.empty_like(self.k_cache)
        self.ref = torch.zeros(shape[1], **i32)            # references to a page
        self.table = torch.empty((0, pages), **i32)
        self.length = torch.empty(0, **i32)                # tokens of a row in the cache
        # a row of pages for each prompt, which goes in chunk by chunk
        size = torch.tensor([len(p) for p in prompts], **i32)
        self.fork(torch.full((B,), -1, **i32), size)
        last = [None] * B
        for at in range(0, max(len(p) for p in prompts), chunk):
            parts = [p[at:at + chunk] for p in prompts]
            count = torch.tensor([len(p) for p in parts], **i32)
            logits = self.feed(torch.tensor(sum(parts, []), device=dev), count)
            for b, end in enumerate(torch.cumsum(count, 0).tolist()):
                if parts[b]:
                    last[b] = logits[end - 1]
        # the beams' texts, their numbers of new tokens, and what they have come to
        self.history = torch.zeros((B, 1, most), **i32)
        for b, p in enumerate(prompts):
            self.history[b, 0, :len(p)] = torch.tensor(p, **i32)
        self.prompt_len = size
        self.new = torch.zeros((B, 1), **i32)
        self.ended = torch.zeros((B, 1), **i32)
        self.scores = torch.zeros((B, 1), device=dev)
        self.choose(torch.stack(last).view(B, 1, -1), beams)

    def fork(self, parent, reserve):
        self.table, self.length, self.ref, copies = sv.spec_pages_fork(
            self.table, self.length, parent, self.ref, self.page, reserve=reserve)
        sv.spec_pages_copy(self.k_cache, self.v_cache, copies)

    def feed(self, tokens, count):
        """The model over new tokens, count[r] of row r one behind the other: their logits."""
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        start = torch.cat([zero, torch.cumsum(count, 0, dtype=torch.int32)])
        n = int(start[-1])
        row = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count.long())
        place = self.length[row] + torch.arange(n, device="cuda") - start[row]
        step = {}

        def attend(i, q, k, v):
            step["length"] = sv.spec_chunk_append(k, v, self.k_cache[i], self.v_cache[i], start,
                                                  self.length, self.table)
            if i == 0:
                step["plan"] = sv.spec_chunk_plan(start, step["length"], q, self.k_cache[0],
                                                  self.table)
            return sv.spec_chunk_attention(q, self.k_cache[i], self.v_cache[i], step["plan"],
                                           self.table)
        logits = self.model.forward(tokens.long(), place.long(), attend)
        self.length = step["length"]
        return logits

    def choose(self, logits, n):
        """The n best continuations of each sequence, and the beams made so."""
        B, K, V = logits.shape
        text = self.prompt_len[:, None] + self.new
        logits = sv.spec_process_logits(
            logits.reshape(B * K, 1, V), history=self.history.flatten(0, 1),
            history_len=text.flatten(), prompt_len=self.prompt_len.repeat_interleave(K),
            frequency=torch.full((B * K,), self.frequency, device="cuda"),
            allowed=self.allowed).view(B, K, V)
        norm = (self.new + 1 - self.ended).clamp(min=1).float() ** self.alpha
        self.tokens, self.beams, self.scores = sv.spec_beam_select(
            logits, self.scores, n, finished=self.ended, norm=norm, end_token=self.end_token)
        self.history = sv.spec_beam_reorder(self.history, self.beams)
        self.new = sv.spec_beam_reorder(self.new, self.beams)
        was = sv.spec_beam_reorder(self.ended, self.beams)
        # a beam that does not exist (none was left to choose) has ended, too
        alive = (was == 0) & (self.beams >= 0)
        at = (self.prompt_len[:, None] + self.new).long()
        b, j = alive.nonzero(as_tuple=True)
        self.history[b, j, at[b, j]] = self.tokens[b, j]
        self.new = self.new + alive
        self.ended = (~alive | (self.tokens == self.end_token)).to(torch.int32)
        first = torch.arange(B, dtype=torch.int32, device="cuda")[:, None] * K
        parent = torch.where(self.beams >= 0, first + self.beams, -1)
        self.fork(parent.flatten(), (1 - self.ended).flatten())

    def step(self):
        """One more token of every beam that has not ended; False when there is none."""
        live = self.ended.flatten() == 0
        if not bool(live.any()):
            return False
        B, K = self.ended.shape
        logits = torch.empty((B * K, self.model.vocab), device="cuda")  # (of ended beams: not read)
        logits[live] = self.feed(self.tokens.flatten()[live], live.to(torch.int32))
        self.choose(logits.view(B, K, -1), self.K)
        return True

    def keep_best(self):
        """The best beam of each sequence is left, its pages at the front of the pool, with
        room for one more token; returns the number of pages in use."""
        B, K = self.ended.shape
        one = torch.ones(B, dtype=torch.int32, device="cuda")
        self.fork(torch.arange(0, B * K, K, dtype=torch.int32, device="cuda"), one)
        for name in ("history", "new", "ended", "scores", "tokens"):
            setattr(self, name, getattr(self, name)[:, :1].contiguous())
        self.table, self.ref, copies, used = sv.spec_pages_compact(self.table, self.ref, self.page)
        sv.spec_pages_copy(self.k_cache, self.v_cache, copies)
        return int(used)


def main():
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(1, 97, (n,), generator=gen).tolist() for n in (70, 1, 33, 12)]
    search = Search(Model(), prompts)
    steps = 1
    while steps < 40 and search.step():
        steps += 1
    if int(search.length.min()) < 0:
        raise RuntimeError(f"sequence error: {search.length.tolist()}")
    shared = int((search.ref > 1).sum())
    held = int((search.ref > 0).sum())
    print(f"{steps} steps; {held} pages in use, {shared} of them shared between beams; "
          f"{search.keep_best()} for the best beams")
    for b, p in enumerate(prompts):
        n = int(search.new[b, 0])
        print(b, f"{float(search.scores[b, 0]):.3f}",
              search.history[b, 0, len(p):len(p) + n].tolist())


if __name__ == "__main__":
    main()
