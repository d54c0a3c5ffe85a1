"""Beams' states of complex numbers whose view conjugates or negates what memory holds, on a GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402


@pytest.mark.parametrize("dtype", [torch.complex64, torch.complex128])
@pytest.mark.parametrize("first", ["plain", "view"])
def test_views_of_complex_states(dtype, first):
    """Whichever of the two the binding has seen before, with the same sizes and strides."""
    gen = torch.Generator().manual_seed(int(first == "plain") + dtype.itemsize)
    shape = (3, 4, 5 + int(first == "plain"))
    plain = torch.randn(shape, generator=gen, dtype=dtype).cuda()
    beams = torch.randint(0, 4, (3, 2), generator=gen).int().cuda()
    at = torch.arange(3, device="cuda")[:, None], beams.long()
    for state in ([plain, plain.conj()] if first == "plain" else [plain.conj(), plain]) * 2:
        assert torch.equal(sv.spec_beam_reorder(state, beams), state[at])
    out = torch.empty((3, 2, shape[2]), dtype=dtype, device="cuda")
    assert torch.equal(sv.spec_beam_reorder(plain.conj(), beams, out=out), plain.conj()[at])
    with pytest.raises(ValueError, match="view"):
        sv.spec_beam_reorder(plain, beams, out=out.conj())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_beam_reorder(plain.conj(), beams, stream=side)
    side.synchronize()
    assert torch.equal(got, plain.conj()[at])
