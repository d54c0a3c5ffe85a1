"""The beam selection refuses outputs that lie over its inputs or over one another, on the CPU: every
call here returns before any CUDA runtime call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from speculative_decoding_verification_65_gb300 import build as sv_build  # noqa: E402
from tests.test_serving_checks import _set  # noqa: E402

M = 1 << 20
B, K, V, N = 2, 4, 100, 3


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.library()


def select(lib, **kw):
    a = _set(sv._BeamArgs(), logits=M, scores=2 * M, norm=3 * M, finished=4 * M, out_tokens=5 * M,
             out_beams=6 * M, out_scores=7 * M, B=B, K=K, V=V, n=N, end_token=3, dtype=sv.SPEC_F32)
    _set(a, **kw)
    need = lib.spec_beam_workspace_size(a.B, a.K, a.V, a.n, a.dtype)
    return lib.spec_beam_select(ctypes.byref(a), ctypes.c_void_p(8 * M), need, None)


@pytest.mark.parametrize("name", ["out_tokens", "out_beams", "out_scores"])
@pytest.mark.parametrize("at,size", [
    (M, B * K * V * 4), (2 * M, B * K * 4), (3 * M, B * K * 4), (4 * M, B * K * 4)])
def test_outputs_over_inputs(lib, name, at, size):
    for over in (at, at + size - 4, at - B * N * 4 + 4):
        assert select(lib, **{name: over}) == sv.SPEC_EINVAL, hex(over)


@pytest.mark.parametrize("name,other", [("out_tokens", 6 * M), ("out_beams", 7 * M),
                                        ("out_scores", 5 * M)])
def test_outputs_over_one_another(lib, name, other):
    for over in (other, other + B * N * 4 - 4, other - B * N * 4 + 4):
        assert select(lib, **{name: over}) == sv.SPEC_EINVAL, hex(over)


def test_scores_in_place(lib):
    """The update that suggests itself where as many are taken as there are beams."""
    assert select(lib, n=K, out_scores=2 * M) == sv.SPEC_EINVAL
