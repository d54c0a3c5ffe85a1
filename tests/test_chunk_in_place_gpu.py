"""Chunk attention whose output takes the place of its queries, on a GPU: the bits of one with room of
its own, items that lie in one CTA's share and split ones among them."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,past,Hkv,G,D,S", [
    ([1], [300], 2, 4, 128, 16), ([70, 5, 0, 200], [9000, 3000, 50, 0], 2, 5, 128, 64),
    ([600, 3, 300], [0, 129, 1000], 4, 3, 64, 0), ([1] * 300, [40] * 300, 2, 8, 80, 16)])
def test_in_place(dtype, new, past, Hkv, G, D, S):
    st = pu.make_chunk(3, new, past, Hkv, G, D, S, dtype)
    plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"], st["table"])
    a = (st["k_cache"], st["v_cache"], plan, st["table"])
    want, lse = sv.spec_chunk_attention(st["q"], *a, want_lse=True)
    for _ in range(3):
        q = st["q"].clone()
        got, lse2 = sv.spec_chunk_attention(q, *a, want_lse=True, out=q)
        assert got is q and torch.equal(q, want) and torch.equal(lse2, lse)


def test_partly_in_place_is_refused():
    st = pu.make_chunk(4, [9], [30], 2, 4, 64, 16, torch.bfloat16)
    plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"], st["table"])
    room = torch.zeros((10, 8, 64), dtype=torch.bfloat16, device="cuda")
    for out in (room[1:], st["k_cache"].view(-1)[:9 * 8 * 64].view(9, 8, 64)):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_chunk_attention(room[:9], st["k_cache"], st["v_cache"], plan, st["table"], out=out)
