"""Decoding with trees of drafted tokens, every operator of a serving step together.

A small transformer with random weights generates text for a batch of
sequences.  Each step drafts a tree below every sequence's last token, runs
the model once over all of its nodes, and keeps the part that the target
agrees with:

    plan = spec_tree_plan(parents, counts, lengths, cache, table)      once
    each layer:  out = spec_tree_attention(q, k, v, caches, plan, table)
    logits = spec_process_logits(logits, history, drafts, penalties, masks)
    tokens, nodes, accepted = spec_verify_tree(logits, draft logits, ...)
    lengths = spec_tree_commit(k, v, caches, lengths, accepted, nodes, table)

Run it with ``python examples/tree_step.py`` on a GPU with the library built.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402

# the root, its 3 drafts, 2 below each of them, 1 below each of those
PARENT = [-1, 0, 0, 0, 1, 1, 2, 2, 3, 3, 4, 5, 6, 7, 8, 9]


class Model:
    """Random weights: `layers` of attention and a feed-forward, learned positions."""

    def __init__(self, vocab=97, width=128, layers=2, heads=8, kv_heads=2, most=512, seed=0,
                 dtype=torch.float16, device="cuda"):
        gen = torch.Generator().manual_seed(seed)

        def w(*shape, scale):
            return (torch.randn(shape, generator=gen) * scale).to(dtype).to(device)
        self.vocab, self.heads, self.kv_heads, self.head_dim = vocab, heads, kv_heads, 64
        self.embed = w(vocab, width, scale=1.0)
        self.place = w(most, width, scale=0.5)
        hd = self.head_dim
        self.layers = [dict(qkv=w((heads + 2 * kv_heads) * hd, width, scale=width ** -0.5),
                            o=w(width, heads * hd, scale=(heads * hd) ** -0.5),
                            up=w(2 * width, width, scale=width ** -0.5),
                            down=w(width, 2 * width, scale=(2 * width) ** -0.5))
                       for _ in range(layers)]
        self.head = w(vocab, width, scale=2 * width ** -0.5)
        # the draft: what follows a token most of the time, guessed from the token alone
        self.draft_head = (self.head.float() + 0.02 * w(vocab, width, scale=1.0).float()).to(dtype)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, tokens, positions, attend):
        """Logits of tokens [.., n]; attend(layer, q, k, v) is the attention."""
        h, kv, hd = self.heads, self.kv_heads, self.head_dim
        x = self.embed[tokens] + self.place[positions]
        for i, layer in enumerate(self.layers):
            qkv = (self.norm(x) @ layer["qkv"].T).unflatten(-1, (h + 2 * kv, hd))
            out = attend(i, qkv[..., :h, :], qkv[..., h:h + kv, :], qkv[..., h + kv:, :])
            x = x + out.flatten(-2) @ layer["o"].T
            x = x + torch.relu(self.norm(x) @ layer["up"].T) @ layer["down"].T
        return self.norm(x).float() @ self.head.float().T

    def draft_logits(self, tokens):
        return self.norm(self.embed[tokens]).float() @ self.draft_head.float().T


class Decoder:
    """The state of a batch: paged caches of every layer, lengths, text so far."""

    def __init__(self, model, prompts, page=16, most=256, seed=0):
        self.model, self.B = model, len(prompts)
        B, dev, L = self.B, "cuda", len(model.layers)
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        pages = -(-most // page)
        shape = (L, B * pages, page, model.kv_heads, model.head_dim)
        self.k_cache = torch.empty(shape, dtype=model.embed.dtype, device=dev)
        self.v_cache = torch.empty_like(self.k_cache)
        order = torch.randperm(B * pages, generator=self.gen, device=dev)
        self.table = order.to(torch.int32).view(B, pages)
        self.length = torch.zeros(B, dtype=torch.int32, device=dev)   # tokens in the cache
        self.history = torch.zeros((B, most), dtype=torch.int32, device=dev)
        self.text_len = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=dev)
        self.prompt_len = self.text_len.clone()
        for b, p in enumerate(prompts):
            self.history[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        # the prompts go through the model as chains: all but the last token into the cache
        n = max(len(p) for p in prompts) - 1
        if n > 0:
            chain = torch.arange(-1, n - 1, dtype=torch.int32, device=dev).repeat(B, 1)
            count = self.text_len - 1
            _, k, v, plan = self.run(self.history[:, :n].contiguous(), chain, count)
            some = (count - 1).clamp(min=-1)          # nothing to commit: -1, the length stays
            new = sv.spec_tree_commit(k, v, self.k_cache, self.v_cache, self.length, some,
                                      page_table=self.table)
            self.length = torch.where(count > 0, new, self.length)

    def run(self, tokens, parent, count):
        """The model over trees of tokens [B, N]: (logits, new keys and values, plan)."""
        plan = sv.spec_tree_plan(parent, count, self.length, self.k_cache[0],
                                 page_table=self.table)
        keys, values = [], []

        def attend(i, q, k, v):
            keys.append(k)
            values.append(v)
            return sv.spec_tree_attention(q, k, v, self.k_cache[i], self.v_cache[i], plan,
                                          page_table=self.table)
        logits = self.model.forward(tokens.long().clamp(min=0), plan.positions.long().clamp(min=0),
                                    attend)
        return logits, torch.stack(keys), torch.stack(values), plan

    def step(self, parent=PARENT, temperature=0.0, repetition=1.0, frequency=0.0, allowed=None):
        """Draft, score, verify and commit one tree per sequence.  Returns the
        tokens [B, N] that the step adds (then -1) and their number [B]."""
        B, N, dev = self.B, len(parent), "cuda"
        V = self.model.vocab
        full = lambda x: torch.full((B,), x, device=dev)  # noqa: E731
        rand = lambda *s: torch.rand(s, generator=self.gen, device=dev)  # noqa: E731
        par = torch.tensor(parent, dtype=torch.int32, device=dev).repeat(B, 1)
        count = torch.full((B,), N, dtype=torch.int32, device=dev)
        last = self.history.gather(1, (self.text_len - 1).long()[:, None])[:, 0]
        # the tree: children of a node are drawn from the draft there
        tokens = torch.empty((B, N), dtype=torch.int32, device=dev)
        tokens[:, 0] = last
        draft = torch.empty((B, N, V), device=dev)
        for n in range(N):
            if n > 0:
                if temperature > 0:
                    p = torch.softmax(draft[:, parent[n]] / temperature, -1)
                    tokens[:, n] = torch.multinomial(p, 1, generator=self.gen)[:, 0]
                else:  # the best, second best, ... of the draft
                    rank = sum(q == parent[n] for q in parent[1:n])
                    tokens[:, n] = draft[:, parent[n]].topk(rank + 1)[1][:, rank]
            draft[:, n] = self.model.draft_logits(tokens[:, n].long())
        logits, k, v, _ = self.run(tokens, par, count)
        logits = sv.spec_process_logits(
            logits.contiguous(), history=self.history, history_len=self.text_len,
            prompt_len=self.prompt_len, draft_tokens=tokens, parent=par,
            repetition=full(repetition), frequency=full(frequency), allowed=allowed)
        out, nodes, accepted = sv.spec_verify_tree(logits, draft, par, tokens, count, rand(B, N),
                                                   rand(B), full(temperature))
        self.length = sv.spec_tree_commit(k, v, self.k_cache, self.v_cache, self.length, accepted,
                                          out_nodes=nodes, page_table=self.table)
        # the text: accepted path, then the drawn token (the next step's root)
        at = self.text_len[:, None] + torch.arange(N, device=dev)
        keep = out >= 0
        b, i = keep.nonzero(as_tuple=True)
        self.history[b, at[b, i].long()] = out[b, i]
        self.text_len = self.text_len + keep.sum(1).to(torch.int32)
        return out, accepted + 1


def main():
    model = Model()
    dec = Decoder(model, [[5, 17, 3, 40], [9], [1, 2, 3, 4, 5, 6, 7], [60, 61]])
    total = steps = 0
    while int(dec.text_len.max()) < 120:
        _, n = dec.step(repetition=1.1, frequency=0.2)
        if int(n.min()) < 1:
            raise RuntimeError(f"sequence error: {n.tolist()}")
        total += int(n.sum())
        steps += 1
    print(f"{total} tokens for {dec.B} sequences in {steps} steps: "
          f"{total / steps / dec.B:.2f} tokens a step")
    for b in range(dec.B):
        print(b, dec.history[b, :int(dec.text_len[b])].tolist()[:24], "...")


if __name__ == "__main__":
    main()
