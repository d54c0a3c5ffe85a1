"""The chunk attention refuses outputs that lie over its inputs or over one another, on the CPU: every
call here returns before any CUDA runtime call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from speculative_decoding_verification_65_gb300 import build as sv_build  # noqa: E402
from tests.test_serving_checks import _set  # noqa: E402

M = 1 << 20
B, ROWS, HQ, HKV, D, S, PAGES = 2, 9, 8, 2, 64, 16, 9
OUT = ROWS * HQ * D * 2


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.library()


def attend(lib, **kw):
    a = _set(sv._ChunkArgs(), q=M, k_cache=2 * M, v_cache=3 * M, page_table=4 * M, plan=5 * M, out=6 * M,
             out_lse=7 * M, scale=0.1, B=B, rows=ROWS, Hq=HQ, Hkv=HKV, D=D, page_size=S,
             pages_per_seq=4, num_pages=PAGES, dtype=sv.SPEC_BF16, q_stride=(HQ * D, D),
             k_cache_stride=(S * HKV * D, HKV * D, D), v_cache_stride=(S * HKV * D, HKV * D, D))
    need = lib.spec_chunk_attention_workspace_size(HQ, HKV, D)
    return lib.spec_chunk_attention(ctypes.byref(_set(a, **kw)), ctypes.c_void_p(8 * M), need, None)


@pytest.mark.parametrize("at,size", [
    (M, OUT), (2 * M, PAGES * S * HKV * D * 2), (3 * M, PAGES * S * HKV * D * 2), (4 * M, B * 4 * 4),
    (5 * M, 256)])  # (a plan's header)
def test_outputs_over_inputs(lib, at, size):
    for over in (at - OUT + 16, at + size - 16):
        assert attend(lib, out=over) == sv.SPEC_EINVAL, hex(over)
    for over in (at - ROWS * HQ * 4 + 4, at, at + size - 4):
        assert attend(lib, out_lse=over) == sv.SPEC_EINVAL, hex(over)


def test_outputs_over_one_another(lib):
    for over in (6 * M, 6 * M + OUT - 4, 6 * M - ROWS * HQ * 4 + 4):
        assert attend(lib, out_lse=over) == sv.SPEC_EINVAL


def test_in_the_place_of_strided_queries(lib):
    """Rows of q with room between them, or its heads the other way round: not what out is."""
    assert attend(lib, out=M, q_stride=(2 * HQ * D, D)) == sv.SPEC_EINVAL
    assert attend(lib, out=M, q_stride=(D, ROWS * D)) == sv.SPEC_EINVAL
