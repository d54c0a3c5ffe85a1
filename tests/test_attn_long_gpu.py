"""Attention over long caches against its 64-bit form and bound (tests/attn_ref.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import attn_ref as ar  # noqa: E402
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
