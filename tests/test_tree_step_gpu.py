"""The example of a serving step (examples/tree_step.py): all operators together.

In greedy mode every token that the trees commit must be the target's own
choice: at each position the plain model over the whole text, in 64 bits and
without any cache or tree, gives the token the highest logit, up to the
rounding of the half-precision run."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.conftest import ROOT  # noqa: E402

sys.path.insert(0, os.path.join(ROOT, "examples"))
import tree_step as ts  # noqa: E402

PROMPTS = [[5, 17, 3, 40], [9], [1, 2, 3, 4, 5, 6, 7], [60, 61]]


def plain_logits(model, text):
    """The model over one text in 64 bits, on the CPU."""
    text = text.cpu()
    wide = ts.Model.__new__(ts.Model)
    wide.__dict__.update(model.__dict__)
    for name in ("embed", "place", "head"):
        setattr(wide, name, getattr(model, name).cpu().double())
    wide.layers = [{k: v.cpu().double() for k, v in layer.items()} for layer in model.layers]
    wide.norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = len(text)
    G = model.heads // model.kv_heads
    mask = torch.ones((n, n), dtype=torch.bool).triu(1)

    def attend(i, q, k, v):
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) / model.head_dim ** 0.5
        p = torch.softmax(s.masked_fill(mask, float("-inf")), -1)
        return torch.einsum("hij,jhd->ihd", p, v)
    x = wide.embed[text] + wide.place[torch.arange(n)]
    for i, layer in enumerate(wide.layers):
        qkv = (wide.norm(x) @ layer["qkv"].T).unflatten(-1, (model.heads + 2 * model.kv_heads, 64))
        h, kv = model.heads, model.kv_heads
        out = attend(i, qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:])
        x = x + out.flatten(-2) @ layer["o"].T
        x = x + torch.relu(wide.norm(x) @ layer["up"].T) @ layer["down"].T
    return wide.norm(x) @ wide.head.T


@pytest.mark.parametrize("parent", [[-1], [-1, 0, 1, 2], ts.PARENT])
def test_greedy_trees_emit_the_targets_own_tokens(parent):
    model = ts.Model()
    dec = ts.Decoder(model, PROMPTS)
    for _ in range(12):
        out, n = dec.step(parent)
        assert int(n.min()) >= 1
    assert torch.equal(dec.length, dec.text_len - 1)
    for b, prompt in enumerate(PROMPTS):
        text = dec.history[b, :int(dec.text_len[b])].long().cpu()
        logits = plain_logits(model, text)
        for i in range(len(prompt), len(text)):
            row = logits[i - 1]
            # logits of size 2 from a run whose every activation has 11 bits, a few dozen of them
            assert float(row.max() - row[text[i]]) < 0.05, (b, i)
    if len(parent) == 1:
        assert bool((dec.text_len - dec.prompt_len == 12).all())


def test_sampled_steps_under_a_mask_and_penalties():
    """Only tokens that the mask allows come out, and no sequence fails."""
    model = ts.Model(seed=3)
    dec = ts.Decoder(model, PROMPTS, seed=4)
    words = torch.tensor([0b1010, 0, -1, 0], dtype=torch.int32, device="cuda").view(1, 1, 4)
    ok = {1, 3} | set(range(64, 96))
    for _ in range(6):
        out, n = dec.step(temperature=0.9, repetition=1.3, frequency=0.5, allowed=words)
        assert int(n.min()) >= 1
        assert {int(x) for x in out[out >= 0]} <= ok
