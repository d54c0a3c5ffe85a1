"""Refusals of the operators around prefill and beam search (chunk append, plan and
attention, beam selection and reordering, pages forked, compacted and copied), in
the library and in the binding, on the CPU: every call here returns before any
CUDA runtime call.  And their restatements on worked examples."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from speculative_decoding_verification_65_gb300 import build as sv_build  # noqa: E402
from tests import prefill_util as pu  # noqa: E402
from tests.test_serving_checks import _by_threads, _Fake, _FakeTorch, _set, A, BF16, F32, I32  # noqa: E402

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.library()


# ------------------------------------------------------------------ chunks

def append(lib, **kw):
    a = _set(sv._AppendArgs(), k_new=A, v_new=A, k_cache=A, v_cache=A, row_start=4 * A,
             cache_len=5 * A, page_table=7 * A, out_len=2 * A, layers=1, B=2, rows=9, Hkv=2, D=64,
             page_size=16, pages_per_seq=4, num_pages=9, elem_size=2)
    return lib.spec_chunk_append(ctypes.byref(_set(a, **kw)), None)


@pytest.mark.parametrize("bad", [
    dict(k_new=0), dict(v_new=0), dict(k_cache=0), dict(v_cache=0), dict(row_start=0),
    dict(cache_len=0), dict(out_len=0), dict(k_new=A + 1), dict(v_cache=A + 1),
    dict(elem_size=4, k_new=A + 2), dict(row_start=A + 2), dict(cache_len=A + 1),
    dict(out_len=A + 2), dict(page_table=A + 2), dict(layers=-1), dict(B=-1), dict(B=65536),
    dict(rows=-1), dict(rows=(1 << 24) + 1), dict(Hkv=0), dict(D=0), dict(page_size=0),
    dict(pages_per_seq=0), dict(num_pages=-1), dict(elem_size=1), dict(elem_size=8),
    dict(Hkv=1 << 13, D=1 << 12), dict(page_size=1 << 20, pages_per_seq=1 << 12),
    dict(page_table=0), dict(page_table=0, pages_per_seq=1, num_pages=1),
    dict(Hkv=1 << 21, D=8, k_new_stride=(0, 1 << 26, 16)),
    dict(out_len=4 * A), dict(out_len=4 * A + 8), dict(out_len=4 * A - 4), dict(out_len=5 * A + 4),
    dict(out_len=7 * A + 28), dict(out_len=7 * A - 4)])
def test_append_refusals(lib, bad):
    assert append(lib, **bad) == sv.SPEC_EINVAL


def test_append_of_nothing(lib):
    assert append(lib, B=0, row_start=0, k_new=0) == sv.SPEC_OK
    assert lib.spec_chunk_append(None, None) == sv.SPEC_EINVAL


def test_plan_refusals(lib):
    def call(start=A, length=A, table=A, B=2, T=9, G=4, S=16, M=4, P=9, plan=A, bytes_=1 << 20):
        return lib.spec_chunk_plan(vp(start), vp(length), vp(table), B, T, G, S, M, P, vp(plan),
                                   bytes_, None)
    for bad in (dict(start=0), dict(length=0), dict(plan=0), dict(start=A + 2), dict(length=A + 1),
                dict(table=A + 2), dict(plan=A + 128), dict(B=-1), dict(B=65536), dict(T=-1),
                dict(T=(1 << 24) + 1), dict(G=0), dict(G=129), dict(S=0), dict(M=0), dict(P=-1),
                dict(S=1 << 20, M=1 << 12), dict(table=0), dict(table=0, M=1, P=1)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    need = lib.spec_chunk_plan_size(2, 9, 4)
    assert call(bytes_=need - 1) == sv.SPEC_ENOSPACE
    assert call(B=0, start=0, plan=0) == sv.SPEC_OK
    for bad in ((-1, 9, 4), (65536, 9, 4), (2, -1, 4), (2, 9, 0), (2, 9, 129), (2, 1 << 25, 4)):
        assert lib.spec_chunk_plan_size(*bad) == lib.spec_chunk_plan_status(*bad) == 0


@pytest.mark.parametrize("B,T,G", [(1, 1, 1), (3, 700, 128), (65535, 70000, 7), (2, 0, 8)])
def test_plan_holds_every_row_group(lib, B, T, G):
    """32 bytes for each group and 8 for each sum, however the rows are dealt to the sequences."""
    tokens = 2 * (128 // G)
    worst = min(B, T)  # as many single tokens as can be, the rest in one sequence
    groups = worst - 1 + -(-(T - worst + 1) // tokens) if worst else 0
    at, size = lib.spec_chunk_plan_status(B, T, G), lib.spec_chunk_plan_size(B, T, G)
    assert at >= 256 and at % 4 == 0 and size % 256 == 0
    assert size >= at + 4 * B + 32 * groups + 8 * (groups + 1)


def attend(lib, ws=A, ws_bytes=None, **kw):
    a = _set(sv._ChunkArgs(), q=A, k_cache=A, v_cache=A, page_table=A, plan=A, out=A, scale=0.1, B=2,
             rows=9, Hq=8, Hkv=2, D=64, page_size=16, pages_per_seq=4, num_pages=9,
             dtype=sv.SPEC_BF16, q_stride=(512, 64), k_cache_stride=(2048, 128, 64),
             v_cache_stride=(2048, 128, 64))
    need = lib.spec_chunk_attention_workspace_size(8, 2, 64)
    return lib.spec_chunk_attention(ctypes.byref(_set(a, **kw)), vp(ws),
                                    need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k_cache=0), dict(v_cache=0), dict(plan=0), dict(out=0), dict(q=A + 8),
    dict(k_cache=A + 2), dict(out=A + 4), dict(plan=A + 16), dict(page_table=A + 2),
    dict(out_lse=A + 2), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
    dict(scale=math.nan), dict(B=-1), dict(B=65536), dict(rows=-1), dict(rows=(1 << 24) + 1),
    dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(Hq=258, Hkv=2), dict(D=0), dict(D=4), dict(D=100),
    dict(D=136), dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=192),
    dict(pages_per_seq=0), dict(num_pages=-1), dict(dtype=sv.SPEC_F32), dict(dtype=3),
    dict(page_size=1 << 20, pages_per_seq=1 << 12), dict(page_table=0),
    dict(q_stride=(512, 4)), dict(q_stride=(-512, 64)), dict(k_cache_stride=(2048, -128, 64)),
    dict(q_stride=(0, 64)), dict(q_stride=(512, 0)), dict(k_cache_stride=(0, 128, 64)),
    dict(v_cache_stride=(2048, 0, 64)), dict(v_cache_stride=(2048, 128, 0)),
    dict(page_table=0, pages_per_seq=1, num_pages=1), dict(ws=0), dict(ws=A + 64)])
def test_attention_refusals(lib, bad):
    assert attend(lib, **bad) == sv.SPEC_EINVAL


def test_attention_workspace(lib):
    need = lib.spec_chunk_attention_workspace_size(8, 2, 64)
    assert need >= 256 and need % 256 == 0
    assert attend(lib, ws_bytes=need - 1) == sv.SPEC_ENOSPACE
    assert attend(lib, B=0, q=0, plan=0) == sv.SPEC_OK
    assert attend(lib, rows=0, q=0, plan=0) == sv.SPEC_OK
    assert lib.spec_chunk_attention(None, vp(A), need, None) == sv.SPEC_EINVAL
    for bad in ((8, 3, 64), (8, 2, 65), (8, 2, 256), (258, 2, 64), (0, 0, 64), (1 << 17, 1 << 16, 8)):
        assert lib.spec_chunk_attention_workspace_size(*bad) == 0


def test_selftest_refusals(lib):
    need = lib.spec_chunk_attention_workspace_size(8, 2, 64)
    a = _set(sv._ChunkArgs(), q=0, k_cache=A, v_cache=A, page_table=A, plan=A, out=A, scale=0.1, B=2,
             rows=9, Hq=8, Hkv=2, D=64, page_size=16, pages_per_seq=4, num_pages=9,
             dtype=sv.SPEC_BF16)
    for cta, after in ((-1, 0), (0, -1), (0, 0)):
        assert lib.spec_selftest_chunk_timeout(ctypes.byref(a), vp(A), need, cta, after,
                                               None) == sv.SPEC_EINVAL


# ------------------------------------------------------------------- beams

def select(lib, ws=A, ws_bytes=None, **kw):
    a = _set(sv._BeamArgs(), logits=A, scores=A, norm=A, finished=A, out_tokens=A, out_beams=A,
             out_scores=A, B=2, K=4, V=100, n=4, end_token=3, dtype=sv.SPEC_F32)
    need = lib.spec_beam_workspace_size(2, 4, 100, 4, sv.SPEC_F32)
    return lib.spec_beam_select(ctypes.byref(_set(a, **kw)), vp(ws),
                                need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(logits=0), dict(scores=0), dict(out_tokens=0), dict(out_beams=0), dict(out_scores=0),
    dict(logits=A + 8), dict(scores=A + 2), dict(norm=A + 2), dict(finished=A + 1),
    dict(out_tokens=A + 2), dict(out_beams=A + 2), dict(out_scores=A + 2), dict(B=-1),
    dict(B=65536), dict(K=0), dict(K=65), dict(n=0), dict(n=65), dict(V=1), dict(V=(1 << 20) + 1),
    dict(end_token=-1), dict(end_token=100), dict(dtype=2), dict(ws=0), dict(ws=A + 64)])
def test_select_refusals(lib, bad):
    assert select(lib, **bad) == sv.SPEC_EINVAL


def test_select_workspace(lib):
    need = lib.spec_beam_workspace_size(2, 4, 100, 4, sv.SPEC_F32)
    assert need % 256 == 0
    assert select(lib, ws_bytes=need - 1) == sv.SPEC_ENOSPACE
    assert select(lib, B=0, logits=0) == sv.SPEC_OK
    assert lib.spec_beam_select(None, vp(A), need, None) == sv.SPEC_EINVAL
    for bad in ((-1, 4, 100, 4, 0), (2, 0, 100, 4, 0), (2, 65, 100, 4, 0), (2, 4, 1, 4, 0),
                (2, 4, 100, 65, 0), (2, 4, 100, 4, 2)):
        assert lib.spec_beam_workspace_size(*bad) == 0


def test_reorder_refusals(lib):
    def call(src=A, beams=A, out=8 * A, lead=1, B=2, K=4, n=4, bytes_=64):
        return lib.spec_beam_reorder(vp(src), vp(beams), vp(out), lead, B, K, n, bytes_, None)
    for bad in (dict(src=0), dict(beams=0), dict(out=0), dict(beams=A + 2), dict(lead=-1),
                dict(B=-1), dict(K=-1), dict(n=-1), dict(bytes_=-1), dict(out=A),
                dict(out=A + 2 * 4 * 64 - 1), dict(out=A - 2 * 4 * 64 + 1),
                dict(lead=1 << 16, B=1 << 10, n=1 << 10), dict(bytes_=(1 << 40) + 1)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    for none in (dict(lead=0), dict(B=0), dict(n=0), dict(bytes_=0)):
        assert call(src=0, out=0, **none) == sv.SPEC_OK


# ------------------------------------------------------------------- pages

def fork(lib, ws=A, ws_bytes=None, **kw):
    a = _set(sv._ForkArgs(), table_in=A, length_in=2 * A, parent=3 * A, reserve=4 * A, ref_in=5 * A,
             table_out=6 * A, length_out=7 * A, ref_out=8 * A, copies=9 * A, rows_in=2, rows_out=3,
             pages_per_seq=4, page_size=16, num_pages=9)
    need = lib.spec_pages_workspace_size(3, 9)
    return lib.spec_pages_fork(ctypes.byref(_set(a, **kw)), vp(ws),
                               need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(table_in=0), dict(length_in=0), dict(parent=0), dict(ref_in=0), dict(table_out=0),
    dict(length_out=0), dict(ref_out=0), dict(copies=0), dict(table_in=A + 2), dict(parent=A + 1),
    dict(reserve=A + 2), dict(copies=A + 2), dict(rows_in=-1), dict(rows_out=-1),
    dict(rows_in=65536), dict(rows_out=65536), dict(pages_per_seq=0), dict(page_size=0),
    dict(num_pages=-1), dict(num_pages=(1 << 24) + 1), dict(pages_per_seq=1 << 16, page_size=1 << 15),
    dict(ws=0), dict(ws=A + 64),
    # outputs over inputs, and over one another
    dict(table_out=A), dict(table_out=A + 28), dict(length_out=2 * A), dict(ref_out=5 * A),
    dict(ref_out=5 * A - 32), dict(copies=3 * A + 8), dict(copies=4 * A), dict(length_out=6 * A + 44),
    dict(copies=8 * A)])
def test_fork_refusals(lib, bad):
    assert fork(lib, **bad) == sv.SPEC_EINVAL


def compact(lib, ws=A, ws_bytes=None, **kw):
    a = _set(sv._CompactArgs(), table_in=A, ref_in=2 * A, table_out=3 * A, ref_out=4 * A,
             copies=5 * A, used=6 * A, rows=2, pages_per_seq=4, page_size=16, num_pages=9)
    need = lib.spec_pages_workspace_size(2, 9)
    return lib.spec_pages_compact(ctypes.byref(_set(a, **kw)), vp(ws),
                                  need if ws_bytes is None else ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(table_in=0), dict(ref_in=0), dict(table_out=0), dict(ref_out=0), dict(copies=0),
    dict(used=0), dict(ref_in=A + 2), dict(used=A + 2), dict(rows=-1), dict(rows=65536),
    dict(pages_per_seq=0), dict(page_size=0), dict(num_pages=0), dict(num_pages=(1 << 24) + 1),
    dict(ws=0), dict(ws=A + 64), dict(table_out=A), dict(ref_out=2 * A + 32), dict(used=4 * A),
    dict(copies=4 * A - 44), dict(used=2 * A + 4)])
def test_compact_refusals(lib, bad):
    assert compact(lib, **bad) == sv.SPEC_EINVAL


def test_pages_workspace(lib):
    assert fork(lib, ws_bytes=lib.spec_pages_workspace_size(3, 9) - 1) == sv.SPEC_ENOSPACE
    assert compact(lib, ws_bytes=lib.spec_pages_workspace_size(2, 9) - 1) == sv.SPEC_ENOSPACE
    assert fork(lib, rows_in=0, rows_out=0, num_pages=0, table_in=0, table_out=0) == sv.SPEC_OK
    assert lib.spec_pages_fork(None, vp(A), 1 << 20, None) == sv.SPEC_EINVAL
    assert lib.spec_pages_compact(None, vp(A), 1 << 20, None) == sv.SPEC_EINVAL
    for bad in ((-1, 9), (65536, 9), (3, -1), (3, (1 << 24) + 1)):
        assert lib.spec_pages_workspace_size(*bad) == 0


def test_copy_refusals(lib):
    def call(**kw):
        a = _set(sv._CopyArgs(), k_cache=A, v_cache=A, copies=A, n=3, layers=2, Hkv=2, D=64,
                 page_size=16, num_pages=9, elem_size=2)
        return lib.spec_pages_copy(ctypes.byref(_set(a, **kw)), None)
    for bad in (dict(k_cache=0), dict(v_cache=0), dict(copies=0), dict(k_cache=A + 1),
                dict(copies=A + 2), dict(elem_size=4, v_cache=A + 2), dict(n=-1),
                dict(n=(1 << 24) + 1), dict(layers=-1), dict(Hkv=0), dict(D=0), dict(page_size=0),
                dict(num_pages=-1), dict(elem_size=1), dict(elem_size=8),
                dict(page_size=1 << 20, Hkv=64, D=128)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    for none in (dict(n=0), dict(layers=0), dict(num_pages=0)):
        assert call(k_cache=0, copies=0, **none) == sv.SPEC_OK
    assert lib.spec_pages_copy(None, None) == sv.SPEC_EINVAL


# ----------------------------------------------------------------- binding

def _refuses(call, good, bad, error=ValueError):
    with pytest.raises(error):
        call(**{**good, **bad})


def _row_args():
    return dict(k_new=_Fake((3, 9, 2, 64), BF16), v_new=_Fake((3, 9, 2, 64), BF16),
                k_cache=_Fake((3, 9, 16, 2, 64), BF16), v_cache=_Fake((3, 9, 16, 2, 64), BF16),
                row_start=_Fake((3,), I32), cache_len=_Fake((2,), I32), page_table=_Fake((2, 4), I32))


@pytest.mark.parametrize("bad,error", [
    (dict(k_cache=_Fake((9, 16, 2, 64), BF16)), ValueError),
    (dict(k_cache=_Fake((2, 9, 16, 2, 64), BF16)), ValueError),
    (dict(v_new=_Fake((3, 8, 2, 64), BF16)), ValueError),
    (dict(v_cache=_Fake((3, 9, 16, 2, 32), BF16)), ValueError),
    (dict(k_new=_Fake((3, 9, 2, 64), I32), v_new=_Fake((3, 9, 2, 64), I32)), TypeError),
    (dict(v_new=_Fake((3, 9, 2, 64), F32)), TypeError),
    (dict(v_cache=_Fake((3, 9, 16, 2, 64), F32)), TypeError),
    (dict(row_start=_Fake((2,), I32)), ValueError), (dict(row_start=_Fake((3,), F32)), ValueError),
    (dict(cache_len=_Fake((2, 1), I32)), ValueError),
    (dict(cache_len=_Fake((2,), I32, "cuda:1")), ValueError),
    (dict(page_table=_Fake((3, 4), I32)), ValueError), (dict(page_table=None), ValueError),
    (dict(k_new=_Fake((3, 9, 2, 64), BF16, strides=(1, 2, 3, 4))), ValueError),
    (dict(v_new=_Fake((3, 9, 2, 64), BF16, "cuda:1")), ValueError),
    (dict(out_len=_Fake((3,), I32)), ValueError),
    (dict(out_len=_Fake((2,), torch.int64)), ValueError)])
def test_append_binding_refuses(bad, error):
    good = _row_args()
    if bad == dict(page_table=None):
        good.update({k: _Fake((3, 1, 16, 2, 64), BF16) for k in ("k_cache", "v_cache")})
    _refuses(sv.spec_chunk_append, good, bad, error)


@pytest.mark.parametrize("bad", [
    dict(row_start=_Fake((2,), I32)), dict(row_start=_Fake((3,), torch.int64)),
    dict(kv_len=_Fake((2, 1), I32)), dict(kv_len=_Fake((2,), F32)), dict(q=_Fake((9, 8), BF16)),
    dict(q=_Fake((9, 7, 64), BF16)), dict(q=_Fake((9, 300, 64), BF16)),
    dict(k_cache=_Fake((9, 16, 2), BF16)), dict(k_cache=_Fake((9, 16, 0, 64), BF16)),
    dict(page_table=_Fake((2,), I32)), dict(page_table=_Fake((2, 4), I32, contiguous=False)),
    dict(page_table=_Fake((2, 4), I32, "cuda:1"))])
def test_chunk_plan_binding_refuses(lib, bad):
    _refuses(sv.spec_chunk_plan, dict(
        row_start=_Fake((3,), I32), kv_len=_Fake((2,), I32), q=_Fake((9, 8, 64), BF16),
        k_cache=_Fake((9, 16, 2, 64), BF16), page_table=_Fake((2, 4), I32)), bad)


def test_chunk_plan_refuses_another_ones_plan(lib):
    for B, rows, G, dev in ((3, 9, 4, "cuda:0"), (2, 8, 4, "cuda:0"), (2, 9, 2, "cuda:0"),
                            (2, 9, 4, "cuda:1")):
        plan = sv.ChunkPlan(B, rows, G, (16, 4, 9), _Fake((4096,), I32, dev))
        with pytest.raises(ValueError, match="plan is for"):
            sv.spec_chunk_plan(_Fake((3,), I32), _Fake((2,), I32), _Fake((9, 8, 64), BF16),
                               _Fake((9, 16, 2, 64), BF16), _Fake((2, 4), I32), plan=plan)


def _chunk_args(S=16):
    return dict(q=_Fake((9, 8, 64), BF16), k_cache=_Fake((9, S, 2, 64), BF16),
                v_cache=_Fake((9, S, 2, 64), BF16),
                plan=sv.ChunkPlan(2, 9, 4, (S, 4, 9), _Fake((4096,), I32)),
                page_table=_Fake((2, 4), I32))


@pytest.mark.parametrize("bad,error", [
    (dict(q=_Fake((9, 8), BF16)), ValueError), (dict(q=_Fake((8, 8, 64), BF16)), ValueError),
    (dict(q=_Fake((9, 8, 64), F32)), TypeError), (dict(q=_Fake((9, 4, 64), BF16)), ValueError),
    (dict(q=_Fake((9, 8, 60), BF16)), ValueError),
    (dict(q=_Fake((9, 8, 64), BF16, "cuda:1")), ValueError),
    (dict(q=_Fake((9, 8, 64), BF16, strides=(516, 64, 1))), ValueError),
    (dict(k_cache=_Fake((9, 16, 2, 64), BF16, strides=(2048, 128, 1, 2))), ValueError),
    (dict(v_cache=_Fake((9, 16, 2, 64), torch.float16)), TypeError),
    (dict(v_cache=_Fake((9, 16, 2, 32), BF16)), ValueError),
    (dict(k_cache=_Fake((9, 16, 4, 64), BF16)), ValueError), (dict(page_table=None), ValueError),
    (dict(page_table=_Fake((2, 5), I32)), ValueError), (dict(scale=0.0), ValueError),
    (dict(scale=math.nan), ValueError), (dict(scale=-math.inf), ValueError),
    (dict(out=_Fake((9, 8, 64), F32)), ValueError), (dict(out=_Fake((9, 8, 32), BF16)), ValueError)])
def test_chunk_attention_binding_refuses(lib, bad, error):
    _refuses(sv.spec_chunk_attention, _chunk_args(), bad, error)


@pytest.mark.parametrize("S", [1, 4, 24, 192])
def test_page_sizes_that_the_chunk_attention_refuses(lib, S):
    with pytest.raises(ValueError, match="page size"):
        sv.spec_chunk_attention(**_chunk_args(S))


@pytest.mark.parametrize("bad,error", [
    (dict(logits=_Fake((2, 400), F32)), ValueError),
    (dict(logits=_Fake((2, 4, 100), torch.float16)), TypeError),
    (dict(logits=_Fake((2, 4, 100), F32, contiguous=False)), ValueError),
    (dict(logits=_Fake((2, 65, 100), F32)), ValueError), (dict(n=0), ValueError),
    (dict(n=65), ValueError), (dict(end_token=100), ValueError), (dict(end_token=-1), ValueError),
    (dict(scores=_Fake((2, 3), F32)), ValueError),
    (dict(scores=_Fake((2, 4), torch.float64)), ValueError),
    (dict(finished=_Fake((2, 4), torch.bool)), ValueError),
    (dict(norm=_Fake((2,), F32)), ValueError),
    (dict(norm=_Fake((2, 4), F32, "cuda:1")), ValueError)])
def test_select_binding_refuses(lib, bad, error):
    _refuses(sv.spec_beam_select,
             dict(logits=_Fake((2, 4, 100), F32), scores=_Fake((2, 4), F32), n=4), bad, error)


@pytest.mark.parametrize("bad", [
    dict(state=_Fake((2,), I32)), dict(state=_Fake((2, 5, 9), I32, contiguous=False)),
    dict(beams=_Fake((2,), I32)), dict(beams=_Fake((3, 4), I32)), dict(dim=-1), dict(dim=2),
    dict(beams=_Fake((2, 4), torch.int64)), dict(beams=_Fake((2, 4), I32, "cuda:1")),
    dict(out=_Fake((2, 5, 9), I32)), dict(out=_Fake((2, 4, 9), F32))])
def test_reorder_binding_refuses(bad):
    _refuses(sv.spec_beam_reorder, dict(state=_Fake((2, 5, 9), I32), beams=_Fake((2, 4), I32)), bad)


@pytest.mark.parametrize("bad", [
    dict(table=_Fake((2,), I32)), dict(table=_Fake((2, 4), torch.int64)),
    dict(length=_Fake((3,), I32)), dict(parent=_Fake((3, 1), I32)), dict(parent=_Fake((3,), F32)),
    dict(ref_count=_Fake((9,), torch.int64)), dict(ref_count=_Fake((9,), I32, "cuda:1")),
    dict(reserve=_Fake((2,), I32)), dict(out=[_Fake((3, 4), I32)]),
    dict(out=[_Fake((3, 4), I32), _Fake((3,), I32), _Fake((9,), I32), _Fake((3, 2), I32)]),
    dict(ref_count=_Fake(((1 << 24) + 1,), I32))])
def test_fork_binding_refuses(lib, bad):
    _refuses(sv.spec_pages_fork, dict(
        table=_Fake((2, 4), I32), length=_Fake((2,), I32), parent=_Fake((3,), I32),
        ref_count=_Fake((9,), I32), page_size=16), bad)


@pytest.mark.parametrize("bad", [
    dict(table=_Fake((2,), I32)), dict(table=_Fake((2, 4), I32, contiguous=False)),
    dict(ref_count=_Fake((9, 1), I32)), dict(ref_count=_Fake((9,), F32)),
    dict(out=[_Fake((2, 4), I32), _Fake((9,), I32), _Fake((3, 5), I32), _Fake((1,), I32)])])
def test_compact_binding_refuses(lib, bad):
    _refuses(sv.spec_pages_compact,
             dict(table=_Fake((2, 4), I32), ref_count=_Fake((9,), I32), page_size=16), bad)


@pytest.mark.parametrize("bad,error", [
    (dict(k_cache=_Fake((9, 16, 2), BF16)), ValueError),
    (dict(v_cache=_Fake((8, 16, 2, 64), BF16)), ValueError),
    (dict(v_cache=_Fake((9, 16, 2, 64), torch.float16)), TypeError),
    (dict(k_cache=_Fake((9, 16, 2, 64), torch.uint8), v_cache=_Fake((9, 16, 2, 64), torch.uint8)),
     TypeError),
    (dict(copies=_Fake((2, 3), I32)), ValueError), (dict(copies=_Fake((3,), I32)), ValueError),
    (dict(copies=_Fake((3, 3), torch.int64)), ValueError),
    (dict(copies=_Fake((3, 3), I32, contiguous=False)), ValueError),
    (dict(v_cache=_Fake((9, 16, 2, 64), BF16, "cuda:1")), ValueError),
    (dict(v_cache=_Fake((9, 16, 2, 64), BF16, strides=(2048, 128, 1, 2))), ValueError)])
def test_copy_binding_refuses(bad, error):
    _refuses(sv.spec_pages_copy, dict(k_cache=_Fake((9, 16, 2, 64), BF16),
                                      v_cache=_Fake((9, 16, 2, 64), BF16),
                                      copies=_Fake((3, 3), I32)), bad, error)


def test_a_failed_check_is_not_kept(lib):
    """The checks are kept by what they depend on: a call that was refused is refused again, and
    one that differs in a dtype, a device or a stride is looked at anew."""
    for _ in range(2):
        for bad in (dict(v_new=_Fake((3, 9, 2, 64), F32)),
                    dict(row_start=_Fake((3,), I32, "cuda:1")),
                    dict(v_new=_Fake((3, 9, 2, 64), BF16, strides=(1, 2, 3, 4)))):
            with pytest.raises((TypeError, ValueError)):
                sv.spec_chunk_append(**{**_row_args(), **bad})


@pytest.mark.parametrize("which", ["_chunk_ws", "_beam_ws", "_pages_ws"])
def test_workspaces_belong_to_one_thread(monkeypatch, which):
    monkeypatch.setattr(sv, "_torch", lambda: _FakeTorch)
    cache, dev = getattr(sv, which), torch.device("cuda:0")
    (a, b), (c, d) = _by_threads(lambda: sv._scratch(cache, 512, dev, 7, None))
    assert a is b and c is d and a is not c
    assert sv._scratch(cache, 512, dev, 8, None) is not a
    assert sv._scratch(cache, 512, torch.device("cuda:1"), 7, None) is not a
    assert sv._scratch(cache, 1024, dev, 7, None).numel() == 1024


def _calls(dev):
    """A call of every entry point with tensors on `dev`."""
    f = lambda shape, dtype: _Fake(shape, dtype, dev)  # noqa: E731
    ws = f((1 << 20,), torch.uint8)
    cache = f((9, 16, 2, 64), BF16)
    table, start, length = f((2, 4), I32), f((3,), I32), f((2,), I32)
    q, new = f((9, 8, 64), BF16), f((9, 2, 64), BF16)
    plan = sv.ChunkPlan(2, 9, 4, (16, 4, 9), f((4096,), I32))
    parent, ref = f((3,), I32), f((9,), I32)
    yield lambda: sv.spec_chunk_append(new, new, cache, cache, start, length, table)
    yield lambda: sv.spec_chunk_plan(start, length, q, cache, table, plan=plan)
    yield lambda: sv.spec_chunk_attention(q, cache, cache, plan, table, ws=ws)
    yield lambda: sv.spec_beam_select(f((2, 4, 100), F32), f((2, 4), F32), 4, ws=ws)
    yield lambda: sv.spec_beam_reorder(f((2, 4, 9), I32), f((2, 4), I32))
    yield lambda: sv.spec_pages_fork(table, length, parent, ref, 16, ws=ws)
    yield lambda: sv.spec_pages_compact(table, ref, 16, ws=ws)
    yield lambda: sv.spec_pages_copy(cache, cache, f((3, 5), I32))


def test_library_calls_run_with_the_tensors_device_current(lib, monkeypatch):
    """With cuda:0 current, a call on cuda:1 tensors enters that device around the library's call,
    and one on cuda:0 tensors enters none."""
    seen = []

    class Device:
        def __init__(self, dev):
            self.dev = str(dev)

        def __enter__(self):
            seen.append(self.dev)

        def __exit__(self, *exc):
            seen.append("out")

    class Lib:
        def __getattr__(self, name):
            if name.endswith(("_size", "_status")):
                return getattr(lib, name)
            return lambda *args: seen.append(name) or sv.SPEC_OK
    monkeypatch.setattr(sv, "_lib", Lib())
    monkeypatch.setattr(sv, "_on", Device)
    monkeypatch.setattr(sv, "_raw_getters", (lambda i: 7, lambda: 0))
    monkeypatch.setattr(sv, "_empty_on", lambda s, shape, dtype, dev: _Fake(shape, dtype, dev))
    monkeypatch.setattr(sv, "_plain_empty", lambda shape, st, dtype: _Fake(shape, dtype))
    names = ("spec_chunk_append", "spec_chunk_plan", "spec_chunk_attention", "spec_beam_select",
             "spec_beam_reorder", "spec_pages_fork", "spec_pages_compact", "spec_pages_copy")
    for dev in ("cuda:1", "cuda:0"):
        for name, call in zip(names, _calls(dev)):
            call()
            assert seen == (["cuda:1", name, "out"] if dev == "cuda:1" else [name])
            seen.clear()


def test_status_of_an_empty_batch():
    assert sv.ChunkPlan(0, 5, 4, (16, 4, 9), None).read_status() == sv.SPEC_DEV_OK


# ------------------------------------------------- the restatements themselves

def test_beams_by_hand():
    x = torch.tensor([[[0.0, math.log(3)], [0.0, 0.0]]])
    tokens, beams, best = pu.beam_ref(x, torch.tensor([[-1.0, -1.0]]), 3)
    assert tokens.tolist() == [[1, 0, 1]] and beams.tolist() == [[0, 1, 1]]
    np.testing.assert_allclose(best[0], -1 + np.log([0.75, 0.5, 0.5]), atol=1e-7)
    tokens, beams, best = pu.beam_ref(x, torch.tensor([[-1.0, -0.1]]), 5, end_token=1,
                                      finished=torch.tensor([[0, 1]]))
    assert tokens.tolist() == [[1, 1, 0, -1, -1]] and beams.tolist() == [[1, 0, 0, -1, -1]]


def test_forks_by_hand():
    """Two children of a row of 5 tokens in pages of 4: the first keeps the page in use, the
    second has a copy of its one token; an old row that nobody takes over gives its pages up."""
    table = np.array([[3, 1, -1], [0, -1, -1]], np.int32)
    ref = np.array([1, 1, 0, 1, 0], np.int32)
    new, length, count, copies = pu.fork_ref(table, np.array([5, 2], np.int32),
                                             np.array([0, 0, -1]), ref, 4)
    assert new.tolist() == [[3, 1, -1], [3, 2, -1], [-1, -1, -1]]
    assert length.tolist() == [5, 5, 0] and count.tolist() == [0, 1, 1, 2, 0]
    assert copies.tolist() == [[-1, 1, -1], [-1, 2, -1], [0, 1, 0]]


def test_compaction_by_hand():
    new, count, copies, used = pu.compact_ref(np.array([[4, 1], [5, -1]], np.int32),
                                              np.array([0, 2, 0, 0, 1, 1], np.int32), 8)
    assert used == 3 and new.tolist() == [[0, 1], [2, -1]] and count.tolist() == [1, 2, 1, 0, 0, 0]
    assert copies.tolist() == [[4, 5, -1], [0, 2, -1], [8, 8, 0]]
