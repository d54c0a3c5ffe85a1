"""Offsets past 32 bits, in elements and bytes: caches, rows, states and logits of several GB, of
which a few places at the far end are looked at."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402
from tests.test_chunk_gpu import attend, check  # noqa: E402

BF16, I32 = torch.bfloat16, dict(dtype=torch.int32, device="cuda")


def test_pages_at_the_end_of_a_long_cache():
    """Append, attention and page copies among pages that start 2.6e9 elements on."""
    P, S, H, D = 20001, 128, 8, 128
    small = pu.make_chunk(1, [150, 3], [250, 500], H, 4, D, S, BF16)
    far = torch.arange(P - small["k_cache"].shape[0], P, device="cuda")
    st = dict(small)
    for name in ("k_cache", "v_cache"):
        st[name] = torch.empty((P, S, H, D), dtype=BF16, device="cuda")
        st[name][far] = small[name]
    st["table"] = (small["table"] + int(far[0])).int()
    out, lse, _ = attend(st)
    again, lse2, _ = attend(small)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    check(small, out, lse)
    # the same new tokens, appended to a cache that has the old positions only
    k, v = (torch.cat([c[pu.positions(small, b, int(small["length"][b]))][past:]
                       for b, past in enumerate((250, 500))])
            for c in (small["k_cache"], small["v_cache"]))
    for c in (st["k_cache"], st["v_cache"]):
        for b, past in enumerate((250, 500)):
            pages, slots = pu.positions(st, b, int(st["length"][b]))
            c[pages[past:], slots[past:]] = 0
    new = sv.spec_chunk_append(k, v, st["k_cache"], st["v_cache"], st["start"],
                               torch.tensor([250, 500], **I32), st["table"])
    assert torch.equal(new, st["length"])
    assert torch.equal(attend(st)[0], out)
    copies = torch.tensor([[P - 1, 5, -1], [2, P - 2, -1], [S, 100, 0]], **I32)
    st["k_cache"][[2, 5]], st["v_cache"][[2, 5]] = 1.0, 2.0
    want = st["k_cache"][P - 1].clone(), st["v_cache"][P - 1].clone()
    sv.spec_pages_copy(st["k_cache"], st["v_cache"], copies)
    for c, w, one in ((st["k_cache"], want[0], 1.0), (st["v_cache"], want[1], 2.0)):
        assert torch.equal(c[2], w) and torch.equal(c[P - 1], w)
        assert bool((c[P - 2, :100] == one).all())


def test_rows_at_the_end_of_many():
    """Queries and outputs that start 2.3e9 elements on: rows before the first sequence's are none's."""
    T, n = 70000, 33
    small = pu.make_chunk(2, [n], [70], 64, 4, 128, 16, BF16)
    q = torch.empty((T, 256, 128), dtype=BF16, device="cuda")
    q[T - n:] = small["q"]
    out, lse, _ = attend(dict(small, q=q, start=small["start"] + T - n))
    want, want_lse, _ = attend(small)
    assert torch.equal(out[T - n:], want) and torch.equal(lse[T - n:], want_lse)


def test_a_state_of_several_gb():
    state = torch.zeros((2, 1, 2, 1_500_000_016), dtype=torch.uint8, device="cuda")
    for l in range(2):
        for k in range(2):
            state[l, 0, k, :16] = 10 * l + k
            state[l, 0, k, -17:] = 100 + 10 * l + k
    got = sv.spec_beam_reorder(state, torch.tensor([[1, 0]], **I32), dim=1)
    for l in range(2):
        for k in range(2):
            assert bool((got[l, 0, k, :16] == 10 * l + 1 - k).all())
            assert bool((got[l, 0, k, -17:] == 100 + 10 * l + 1 - k).all())


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_logits_of_many_sequences(dtype):
    """Rows that start 2.2e9 elements on."""
    B, V = 17001, 128257
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty((B, 1, V), dtype=dtype, device="cuda")
    x[:-9] = 0.5  # every logit equal: the first ones win
    x[-9:] = torch.randn((9, 1, V), generator=gen, device="cuda").to(dtype)
    s = torch.full((B, 1), -1.0, device="cuda")
    tokens, beams, best = sv.spec_beam_select(x, s, 2)
    assert tokens[:-9].eq(torch.tensor([0, 1], device="cuda")).all() and beams.eq(0).all()
    want = pu.beam_ref(x[-9:].float().cpu(), s[-9:].cpu(), 2)
    assert tokens[-9:].tolist() == want[0].tolist()
    off = (best[-9:].double().cpu() - torch.from_numpy(want[2])).abs()
    assert float(off.max()) <= 13 * 2.0 ** -24 + 5e-6
