"""The example of a beam search (examples/beam_search.py): prompts in chunks, forks, copies,
chunk attention, selection, reordering and compaction together.

The plain model over whole texts in 64 bits, without a cache, says what every candidate of
a step is worth; the beams that a step keeps must be the best of them, up to the
rounding of the half-precision run."""
import os
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from tests.conftest import ROOT  # noqa: E402

sys.path.insert(0, os.path.join(ROOT, "examples"))
import beam_search as bs  # noqa: E402
from tests.test_tree_step_gpu import plain_logits  # noqa: E402

# A step's logits are off by 0.05 between two of a row (test_tree_step_gpu), so a token's
# log-probability, the difference of a logit and a mean over the row's, by no more.
STEP = 0.05


def prompts(seed=1):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(1, 97, (n,), generator=gen).tolist() for n in (70, 1, 33, 12)]


def counts_of(table, pages):
    held = table[table >= 0].long()
    return torch.bincount(held, minlength=pages).int()


def check_pages(s):
    """Counts are the tables' own, a row has pages for its next token, and no row's page in use
    that is written next is another row's."""
    assert torch.equal(counts_of(s.table, len(s.ref)), s.ref)
    live = s.ended.flatten() == 0
    assert int(s.length.min()) >= 0
    for r in range(len(s.table)):
        n, held = int(s.length[r]), int((s.table[r] >= 0).sum())
        assert held == -(-(n + int(live[r])) // s.page)
        if live[r]:
            assert int(s.ref[s.table[r, n // s.page]]) == 1


def texts(s, given):
    """A sequence's beams: (text, new tokens, ended, score, norm of its candidates)."""
    out = []
    for b, p in enumerate(given):
        new, ended = s.new[b].tolist(), s.ended[b].tolist()
        out.append([(s.history[b, k, :len(p) + new[k]].tolist(), new[k], ended[k],
                     float(s.scores[b, k])) for k in range(len(new))])
    return out


@pytest.mark.parametrize("beams,alpha,end_token,chunk", [(4, 0.7, 0, 24), (3, 0.0, 96, 7),
                                                         (6, 1.0, 40, 128)])
def test_every_step_keeps_the_best(beams, alpha, end_token, chunk):
    model, given = bs.Model(vocab=97), prompts()
    s = bs.Search(model, given, beams=beams, alpha=alpha, end_token=end_token, chunk=chunk, page=8)
    before = [[(list(p), 0, 0, 0.0)] for p in given]
    for _ in range(8):
        check_pages(s)
        after = texts(s, given)
        for b in range(len(given)):
            worth = {}  # text -> (compared, score)
            for text, new, ended, score in before[b]:
                if ended:
                    worth[tuple(text)] = score / max(1, new) ** alpha, score
                    continue
                logp = torch.log_softmax(plain_logits(model, torch.tensor(text))[-1], 0).numpy()
                for x in np.argsort(-logp)[:2 * beams]:
                    worth[(*text, int(x))] = ((score + logp[x]) / (new + 1) ** alpha,
                                              score + logp[x])
            best = sorted((w for w, _ in worth.values()), reverse=True)
            kept = [tuple(text) for text, *_ in after[b]]
            assert len(set(kept)) == beams
            for text, _, _, score in after[b]:
                # (the scores before are the run's own, so only this step's logits are off)
                assert abs(worth[tuple(text)][1] - score) < STEP
                assert worth[tuple(text)][0] > best[beams - 1] - STEP
        before = after
        if not s.step():
            break
    # what is left after the others are given up reads as before from its new pages
    used = s.keep_best()
    assert used == int((s.ref > 0).sum()) and int((s.ref[used:] > 0).sum()) == 0
    assert torch.equal(counts_of(s.table, len(s.ref)), s.ref)
    live = (s.ended[:, 0] == 0).nonzero()[:, 0].tolist()
    if live:
        count = (1 - s.ended[:, 0]).to(torch.int32)
        got = s.feed(s.tokens[live, 0], count).double().cpu()
        for row, b in zip(got, live):
            text = s.history[b, 0, :len(given[b]) + int(s.new[b, 0])].cpu()
            assert float((row - plain_logits(model, text)[-1]).abs().max()) < STEP


def test_masked_and_penalised_searches_run():
    """Fewer tokens allowed than beams: beams that do not exist stay out, and come in later."""
    words = torch.tensor([0b1010, 0, 0, 0], dtype=torch.int32, device="cuda").view(1, 1, 4)
    s = bs.Search(bs.Model(seed=3), prompts(2), beams=5, frequency=0.5, allowed=words, page=16)
    assert (s.beams >= 0).sum(1).tolist() == [2] * 4
    for _ in range(6):
        check_pages(s)
        assert s.step()
    assert (s.beams >= 0).all() and set(s.tokens.flatten().tolist()) <= {1, 3}


def test_example_runs(capsys):
    bs.main()
    assert "shared between beams" in capsys.readouterr().out
