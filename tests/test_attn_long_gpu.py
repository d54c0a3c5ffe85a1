"""Attention over long caches against its 64-bit form and bound (tests/attn_ref.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import attn_ref as ar  # noqa: E402
from tests.test_attn_gpu import FP16, make, run  # noqa: E402

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
