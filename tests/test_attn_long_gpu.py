"""Attention over long caches on inputs that show a lost or misplaced tile, row
tiles in pairs, small weights in fp16, and what a wait that gives up leaves
(tests/attn_ref.py has the 64-bit form and its bound)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import attn_ref as ar  # noqa: E402
from tests import serve_util as su  # noqa: E402
from tests.test_attn_gpu import BF16, FP16, dev, make, run  # noqa: E402

gpu = pytest.mark.gpu


def check(c, scale=None):
    out, lse = run(c, scale=scale)
    r = ar.attention(c, scale)
    err, tol = (out - r["out"]).abs(), ar.tolerance(c, r)
    assert bool((err <= tol).all()), float((err / tol).max())
    seen = torch.isfinite(r["lse"])
    assert torch.equal(seen, torch.isfinite(lse)) and bool((lse[~seen] == -math.inf).all())
    assert bool(((lse - r["lse"]).abs() <= ar.lse_tolerance(c, r))[seen].all())


# B, N, Hkv, G, D, page size (0: contiguous), positions, dtype: one row tile and pairs of them
LONG = [(1, 29, 1, 4, 128, 64, 39999, BF16), (1, 29, 2, 4, 64, 16, 30001, FP16),
        (2, 5, 1, 7, 64, 128, 20000, BF16), (1, 1, 1, 1, 64, 0, 30001, FP16),
        (1, 40, 1, 8, 128, 128, 20000, BF16), (1, 40, 1, 8, 128, 0, 20011, FP16),
        (2, 9, 2, 16, 64, 32, 25000, BF16), (1, 33, 2, 5, 80, 8, 15000, FP16)]


def long_case(B, N, H, G, D, S, L, dtype, ends):
    c = make(B, N, H, G, D, S, L, dtype, seed=L, lens=[L, L - 1111], nodes=[N])
    return ar.directed(c, ends, seed=L + 1)


@gpu
@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_every_tile_of_a_long_cache_counts(shape, ends):
    check(long_case(*shape, ends), scale=1.0)


@pytest.mark.parametrize("ends", [False, True])
@pytest.mark.parametrize("shape", LONG, ids=str)
def test_a_lost_tile_would_show(shape, ends):
    """In the inputs above, the values of any tile that a row is directed at make more of some
    output than the bound allows; with as many rows as D that is every tile."""
    c = long_case(*shape, ends)
    r = ar.attention(c, 1.0)
    tol = ar.tolerance(c, r)
    D, rows = shape[4], min(shape[4], shape[1] * shape[3])
    for b in range(shape[0]):
        parts = ar.parts_of_tiles(c, b)
        shows = (parts.abs() > 2 * tol[b]).flatten(1).any(1)
        want = torch.arange(len(parts)) % D < rows
        assert bool(shows[want].all()) and int(want.sum()) >= 4


# ------------------------------------------------------------ pairs of row tiles

@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 80, 96, 128])
def test_pairs_over_many_tiles(D, dtype):
    """Three row tiles of 25 nodes, shares of a dozen whole tiles, counts of nodes that leave
    a tile of the pair, or the second pair, empty."""
    check(make(8, 60, 4, 5, D, 32, 4000, dtype, seed=D, lens=[4000, 3905, 128, 2047],
               nodes=[60, 7, 33, 26, 51]))


@gpu
@pytest.mark.parametrize("B", [33, 40, 200])
def test_pairs_of_many_sequences(B):
    lens = [0, 3, 128, 300, 1, 64, 0, 129, 257, 17]
    check(make(B, 20, 2, 8, 128, 16, 300, BF16, seed=B, lens=lens, nodes=[20, 1, 16, 17]))
    check(make(B, 9, 1, 16, 64, 0, 300, FP16, seed=B + 1, lens=lens, nodes=[9, 8, 0, 3]))


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N,G", [(60, 5), (20, 5)])
def test_scores_that_grow_inside_a_share(N, G, dtype):
    """Scores rising, then falling, along the sequence, in pairs and in single row tiles: sums
    are rescaled in the middle of a share of many whole tiles."""
    c = make(8, N, 4, G, 128, 0, 4000, dtype, seed=N, lens=[4000, 3333], nodes=[N])
    ramp = torch.linspace(0.0, 6.0, 4000).view(1, -1, 1, 1)
    c["k_cache"] = (c["k_cache"].float() * ramp).to(dtype)
    check(c, scale=0.25)
    c["k_cache"] = c["k_cache"].flip(1)
    check(c, scale=0.25)


@gpu
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_nonfinite_new_values_in_pairs(dtype):
    """As in one row tile: a NaN or an infinity of a drafted node's value, in either half of the
    head, reaches the node's descendants and nobody else."""
    N = 140
    c = make(2, N, 2, 2, 128, 16, 700, dtype, seed=10, lens=[677, 128], nodes=[N, 135])
    clean, _ = run(c)
    want = clean.clone()
    c["v_new"] = c["v_new"].clone()
    for b, x, h, d, value in ((0, 1, 0, 5, math.nan), (0, 1, 0, 70, math.inf),
                              (0, 130, 1, 127, -math.inf), (1, 64, 1, 0, math.inf),
                              (1, 128, 0, 63, math.nan), (1, 128, 0, 64, -math.inf)):
        c["v_new"][b, x, h, d] = value
        rows = [n for n in range(int(c["n_nodes"][b])) if x in su.ancestors(c["parent"][b], n)]
        want[b, rows, 2 * h:2 * h + 2, d] = value
    out, _ = run(c)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(0.0, 1e30, -1e30), want.nan_to_num(0.0, 1e30, -1e30))


@gpu
@pytest.mark.parametrize("length", [0, 500])
def test_chain_of_a_thousand_nodes(length):
    check(make(1, 1024, 1, 2, 128, 64, 600, BF16, seed=3, kind="chain", lens=[length], nodes=[1024]))


@gpu
def test_captured_step_with_its_commit():
    """Plan, attention of row tiles in pairs and the commit in one graph, replayed over its own
    results: each replay's lengths are those that the one before left."""
    c = make(3, 40, 1, 4, 64, 16, 700, BF16, seed=14, kind="chain", lens=[100, 7, 0], nodes=[40])
    d = {k: dev(v) for k, v in c.items()}
    accepted = torch.tensor([39, 0, 11], dtype=torch.int32, device="cuda")
    length = d["cache_len"].clone()

    def step():
        plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], length, d["k_cache"],
                                 page_table=d["table"])
        out = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                     plan, page_table=d["table"])
        new = sv.spec_tree_commit(d["k_new"], d["v_new"], d["k_cache"], d["v_cache"], length,
                                  accepted, page_table=d["table"])
        length.copy_(new)
        return out
    step()
    torch.cuda.synchronize()
    length.copy_(d["cache_len"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    lens = c["cache_len"]
    kc, vc = c["k_cache"][None], c["v_cache"][None]
    for _ in range(3):
        g.replay()
        now = dict(c, cache_len=lens, k_cache=kc[0], v_cache=vc[0])
        r = ar.attention(now)
        assert bool(((out.cpu().double() - r["out"]).abs() <= ar.tolerance(now, r)).all())
        kc, vc, lens = su.commit_ref(c["k_new"][None], c["v_new"][None], kc, vc, lens,
                                     accepted.cpu().numpy(), None, c["table"])
        lens = lens.astype(np.int32)
        assert length.cpu().tolist() == lens.tolist()
        # (the eager call before the capture wrote the same rows at the first lengths)
        assert torch.equal(d["k_cache"].cpu(), kc[0]) and torch.equal(d["v_cache"].cpu(), vc[0])


@gpu
@pytest.mark.parametrize("N,G", [(1, 4), (40, 4)])
@pytest.mark.parametrize("at", [0, 77, 127])
def test_small_weights_of_fp16_count(N, G, at):
    """One key of each tile has nearly all of the weight and a value of 0; the output is what
    20000 keys with weights of 2^-23 to 2^-26 of theirs give together."""
    L, D = 20000, 64
    c = make(1, N, 1, G, D, 0, L, FP16, seed=at, kind="star", lens=[L], nodes=[N])
    gen = torch.Generator().manual_seed(at)
    for name in ("q", "k_cache", "k_new"):
        c[name] = torch.zeros_like(c[name])
    c["q"][..., 0] = 1.0
    c["k_cache"][..., 0] = -torch.randint(16, 19, (1, L, 1), generator=gen).to(FP16)
    c["k_new"][..., 0] = -30.0
    c["v_cache"] = (64 + 64 * torch.rand(c["v_cache"].shape, generator=gen)).to(FP16)
    c["k_cache"][0, at::ar.KT], c["v_cache"][0, at::ar.KT] = 0.0, 0.0
    check(c, scale=1.0)


class Losing:
    """The library, its tree attention with a CTA whose wait gives up (include/spec_bench.h)."""

    def __init__(self, lib, cta, after):
        self.lib, self.lose = lib, (cta, after)

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def spec_tree_attention(self, args, ws, size, stream):
        return self.lib.spec_selftest_attention_timeout(args, ws, size, *self.lose, stream)


def giving_up(monkeypatch, c, cta, after):
    """(results without and with the lost wait, plan, results of a new plan afterwards)"""
    d = {k: dev(v) for k, v in c.items()}

    def call():
        plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                                 page_table=d["table"])
        got = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                     plan, page_table=d["table"], want_lse=True)
        torch.cuda.synchronize()
        return got, plan
    want, plan = call()
    assert plan.read_status() == sv.SPEC_DEV_OK
    with monkeypatch.context() as m:
        m.setattr(sv, "_lib", Losing(sv.library(), cta, after))
        got, lost = call()
    again, plan = call()
    assert plan.read_status() == sv.SPEC_DEV_OK
    return want, got, lost, again


# 6 sequences of 1 or 2 row groups over up to 235 tiles and 2 heads: shares of a dozen tiles and more
LOSING = dict(B=6, Hkv=2, G=5, S=16, cap=30000, dtype=BF16, lens=[30000, 22222, 0, 27777])


@gpu
@pytest.mark.parametrize("N,D", [(5, 64), (60, 64), (60, 128)])
@pytest.mark.parametrize("cta,after", [(0, 0), (7, 0), (0, 1), (9, 1)])
def test_a_wait_that_gives_up_is_reported(monkeypatch, N, D, cta, after):
    """The status is read, the GPU answers, and the next step is right again, whether the CTA has
    nothing in flight (after 0) or loads and products of its first piece (after 1)."""
    c = make(N=N, D=D, seed=N, nodes=[N, 3, 0], **LOSING)
    want, _, lost, again = giving_up(monkeypatch, c, cta, after)
    assert lost.read_status() == sv.SPEC_DEV_WAIT_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(again, want))


# shares of several whole items, idle ones among them
SHORT = dict(B=200, Hkv=2, G=5, S=16, cap=300, dtype=BF16,
             lens=[0, 3, 128, 300, 1, 64, 0, 129, 257, 17])


@gpu
@pytest.mark.parametrize("N,D", [(5, 64), (60, 64), (60, 128)])
@pytest.mark.parametrize("shape,cta,after", [(LOSING, 0, 0), (LOSING, 9, 1), (LOSING, 30, 1),
                                             (SHORT, 0, 0), (SHORT, 70, 1), (SHORT, 101, 2)])
def test_rows_of_a_wait_that_gives_up_are_nan(monkeypatch, N, D, shape, cta, after):
    """A row is what it is without the lost wait, or NaN throughout with its log-sum-exp;
    none is left unwritten or joined from an earlier call's sums."""
    c = make(N=N, D=D, seed=N, nodes=[N, 3, 0], **shape)
    (want, want_lse), (out, lse), lost, _ = giving_up(monkeypatch, c, cta, after)
    assert lost.read_status() == sv.SPEC_DEV_WAIT_TIMEOUT
    nan = torch.isnan(out)
    assert torch.equal(nan.all(-1), nan.any(-1)) and torch.equal(nan.all(-1), torch.isnan(lse))
    assert bool(nan.any()) and not bool(nan.all())
    keep = ~nan.all(-1)
    assert torch.equal(out[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])
