"""Chunk attention, its plan and append where rows belong to no sequence, on a GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402


@pytest.mark.parametrize("at", [0, 3, 10])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_padded_rows_of_empty_sequences(at, dtype):
    """A step whose rows are all padding: nothing is written, and no sequence is in error."""
    st = pu.make_chunk(1, [10], [30], 2, 4, 64, 16, dtype)
    start = torch.full((4,), at, dtype=torch.int32, device="cuda")
    length = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")
    table = st["table"].expand(3, -1).contiguous()
    for q in (st["q"], torch.full_like(st["q"], float("nan"))):
        plan = sv.spec_chunk_plan(start, length, q, st["k_cache"], page_table=table)
        out = torch.full_like(q, 7.0)
        out, lse = sv.spec_chunk_attention(q, st["k_cache"], st["v_cache"], plan, page_table=table,
                                           out=out, want_lse=True)
        assert bool((out == 7).all())
        assert plan.status.tolist() == [0, 0, 0] and plan.read_status() == sv.SPEC_DEV_OK
    kept = st["k_cache"].clone(), st["v_cache"].clone()
    new = torch.randn(10, 2, 64, device="cuda").to(dtype)
    got = sv.spec_chunk_append(new, new, st["k_cache"], st["v_cache"], start, length, table)
    assert torch.equal(got, length)
    assert torch.equal(st["k_cache"], kept[0]) and torch.equal(st["v_cache"], kept[1])
