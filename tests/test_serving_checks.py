"""Refusals of the serving operators (tree attention, its plan, the cache
commit, logits processing), in the library and in the binding, on the CPU:
every call here returns before any CUDA runtime call."""
import contextlib
import ctypes
import math
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from speculative_decoding_verification_65_gb300 import build as sv_build  # noqa: E402
from tests import serve_util as su  # noqa: E402
from tests.test_binding_checks import _FakeCuda  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    sv_build.build()
    return sv.library()


A = 0x10000  # stands for any aligned device address


def _set(args, **kw):
    for k, v in kw.items():
        if k.endswith("_stride"):
            getattr(args, k)[:] = v
        else:
            setattr(args, k, v)
    return args


def attention(**kw):
    a = _set(sv._AttentionArgs(), q=A, k_new=A, v_new=A, k_cache=A, v_cache=A, page_table=A, plan=A,
             out=A, scale=0.1, B=2, N=4, Hq=8, Hkv=2, D=64, page_size=16, pages_per_seq=4,
             num_pages=9, dtype=sv.SPEC_BF16, q_stride=(2048, 512, 64), k_new_stride=(512, 128, 64),
             v_new_stride=(512, 128, 64), k_cache_stride=(2048, 128, 64),
             v_cache_stride=(2048, 128, 64))
    return _set(a, **kw)


def attend(lib, a, ws=A, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.spec_tree_attention_workspace_size(4, 8, 2, 64)
    return lib.spec_tree_attention(ctypes.byref(a), ctypes.c_void_p(ws), ws_bytes, None)


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k_new=0), dict(v_new=0), dict(k_cache=0), dict(v_cache=0), dict(plan=0),
    dict(out=0), dict(q=A + 8), dict(k_cache=A + 2), dict(out=A + 4), dict(plan=A + 16),
    dict(page_table=A + 2), dict(out_lse=A + 2), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=math.inf), dict(scale=math.nan), dict(B=-1), dict(B=65536), dict(N=0), dict(N=1025),
    dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(Hq=258, Hkv=2), dict(D=0), dict(D=4), dict(D=100),
    dict(D=136), dict(page_size=0), dict(page_size=4), dict(page_size=24), dict(page_size=192),
    dict(pages_per_seq=0), dict(num_pages=-1), dict(dtype=sv.SPEC_F32), dict(dtype=3),
    dict(page_size=1 << 20, pages_per_seq=1 << 12), dict(page_table=0),
    dict(q_stride=(2048, 512, 4)), dict(k_cache_stride=(2048, -128, 64)),
    dict(page_table=0, pages_per_seq=1, num_pages=1)])
def test_attention_refusals(lib, bad):
    assert attend(lib, attention(**bad)) == sv.SPEC_EINVAL


def test_attention_workspace(lib):
    assert attend(lib, attention(), ws=0) == sv.SPEC_EINVAL
    assert attend(lib, attention(), ws=A + 64) == sv.SPEC_EINVAL
    need = lib.spec_tree_attention_workspace_size(4, 8, 2, 64)
    assert need >= 256 and need % 256 == 0
    assert attend(lib, attention(), ws_bytes=need - 1) == sv.SPEC_ENOSPACE
    assert attend(lib, attention(B=0, q=0, plan=0)) == sv.SPEC_OK
    assert lib.spec_tree_attention(None, ctypes.c_void_p(A), need, None) == sv.SPEC_EINVAL
    for bad in ((0, 8, 2, 64), (4, 8, 3, 64), (4, 8, 2, 65), (4, 8, 2, 256), (1025, 8, 2, 64)):
        assert lib.spec_tree_attention_workspace_size(*bad) == 0


def test_plan_refusals(lib):
    def call(parent=A, n=A, length=A, table=A, B=2, N=5, S=16, M=4, P=9, plan=A, bytes_=1 << 20):
        vp = ctypes.c_void_p
        return lib.spec_tree_plan(vp(parent), vp(n), vp(length), vp(table), B, N, S, M, P,
                                  vp(plan), bytes_, None)
    for bad in (dict(parent=0), dict(n=0), dict(length=0), dict(plan=0), dict(parent=A + 2),
                dict(n=A + 1), dict(length=A + 2), dict(table=A + 2), dict(plan=A + 128),
                dict(B=-1), dict(B=65536), dict(N=0), dict(N=1025), dict(S=0), dict(M=0),
                dict(P=-1), dict(S=1 << 20, M=1 << 12), dict(table=0),
                dict(table=0, M=1, P=1)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    need = lib.spec_tree_plan_size(2, 5)
    assert call(bytes_=need - 1) == sv.SPEC_ENOSPACE
    assert call(B=0, parent=0, plan=0) == sv.SPEC_OK
    assert lib.spec_tree_plan_size(-1, 4) == 0 and lib.spec_tree_plan_size(1, 1025) == 0
    at = [lib.spec_tree_plan_offset(7, 130, i) for i in range(4)]
    assert at[3] == 0 and len(set(at[:3])) == 3 and all(x % 256 == 0 and x > 0 for x in at[:3])
    assert max(at[0] + 7 * 130 * 4, at[1] + 28, at[2] + 7 * 130 * 8 * 4) <= \
        lib.spec_tree_plan_size(7, 130)


def test_commit_refusals(lib):
    def call(**kw):
        a = _set(sv._CommitArgs(), k_new=A, v_new=A, k_cache=A, v_cache=A, cache_len=A,
                 out_num_accepted=A, out_nodes=A, page_table=A, out_len=2 * A, layers=1, B=2, N=4,
                 Hkv=2, D=64, page_size=16, pages_per_seq=4, num_pages=9, elem_size=2)
        return lib.spec_tree_commit(ctypes.byref(_set(a, **kw)), None)
    for bad in (dict(k_new=0), dict(v_new=0), dict(k_cache=0), dict(v_cache=0), dict(cache_len=0),
                dict(out_num_accepted=0), dict(out_len=0), dict(out_len=A), dict(k_new=A + 1),
                dict(cache_len=A + 2), dict(out_nodes=A + 2), dict(page_table=A + 2), dict(layers=-1),
                dict(B=-1), dict(N=0), dict(N=1025), dict(Hkv=0), dict(D=0), dict(page_size=0),
                dict(pages_per_seq=0), dict(num_pages=-1), dict(elem_size=8), dict(elem_size=1),
                dict(elem_size=4, k_new=A + 2), dict(page_table=0),
                dict(page_table=0, pages_per_seq=1, num_pages=1)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    assert call(B=0, k_new=0) == sv.SPEC_OK
    assert lib.spec_tree_commit(None, None) == sv.SPEC_EINVAL


def test_logits_refusals(lib):
    def call(**kw):
        a = _set(sv._LogitsArgs(), logits=A, out=A, history=A, history_len=A, prompt_len=A,
                 draft_tokens=A, B=2, R=4, V=100, H=7, draft_cols=3, dtype=sv.SPEC_F32)
        return lib.spec_process_logits(ctypes.byref(_set(a, **kw)), None)
    for bad in (dict(logits=0), dict(out=0), dict(logits=A + 8), dict(out=A + 4), dict(history=0),
                dict(history_len=0), dict(prompt_len=0), dict(draft_tokens=0), dict(draft_cols=2),
                dict(draft_cols=5), dict(parent=A), dict(parent=A + 2, draft_cols=4), dict(B=-1),
                dict(B=65536), dict(R=0), dict(R=1025, draft_cols=1024), dict(V=1),
                dict(V=(1 << 20) + 1), dict(H=-1), dict(H=(1 << 24) + 1), dict(dtype=2),
                dict(bias_cols=3), dict(bias_cols=-1), dict(bias_cols=3, bias_tokens=A),
                dict(bias_cols=4097, bias_tokens=A, bias_values=A), dict(allowed=A + 2),
                dict(allowed=A, allowed_stride_r=-4), dict(repetition=A + 2), dict(n_nodes=A + 1)):
        assert call(**bad) == sv.SPEC_EINVAL, bad
    assert call(B=0, logits=0) == sv.SPEC_OK
    assert lib.spec_process_logits(None, None) == sv.SPEC_EINVAL


# ----------------------------------------------------------------- binding

class _Fake(_FakeCuda):
    """_FakeCuda with strides."""

    def __init__(self, shape, dtype, device="cuda:0", contiguous=True, strides=None):
        super().__init__(shape, dtype, device, contiguous)
        st, n = [], 1
        for x in reversed(shape):
            st.insert(0, n)
            n *= x
        self._strides = tuple(strides or st)

    def stride(self, i=None):
        return self._strides if i is None else self._strides[i]

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()


I32, BF16, F32 = torch.int32, torch.bfloat16, torch.float32


def _plan_args(**kw):
    d = dict(parent=_Fake((2, 5), I32), n_nodes=_Fake((2,), I32), cache_len=_Fake((2,), I32),
             k_cache=_Fake((9, 16, 2, 64), BF16), page_table=_Fake((2, 4), I32))
    d.update(kw)
    return d


@pytest.mark.parametrize("bad", [
    dict(parent=_Fake((2,), I32)), dict(parent=_Fake((2, 5), torch.int64)),
    dict(n_nodes=_Fake((3,), I32)), dict(cache_len=_Fake((2,), F32)),
    dict(cache_len=_Fake((2,), I32, "cuda:1")), dict(k_cache=_Fake((9, 16, 2), BF16)),
    dict(page_table=_Fake((3, 4), I32)), dict(page_table=_Fake((2,), I32)),
    dict(page_table=_Fake((2, 4), I32, contiguous=False)),
    dict(page_table=None, k_cache=_Fake((1, 16, 2, 64), BF16))])
def test_plan_binding_refuses(lib, bad):
    with pytest.raises(ValueError):
        sv.spec_tree_plan(**_plan_args(**bad))


def _attention_args(**kw):
    d = dict(q=_Fake((2, 5, 8, 64), BF16), k_new=_Fake((2, 5, 2, 64), BF16),
             v_new=_Fake((2, 5, 2, 64), BF16), k_cache=_Fake((9, 16, 2, 64), BF16),
             v_cache=_Fake((9, 16, 2, 64), BF16),
             plan=sv.TreePlan(2, 5, (16, 4, 9), torch.zeros(sv.library().spec_tree_plan_size(2, 5),
                                                           dtype=torch.uint8)),
             page_table=_Fake((2, 4), I32))
    d["plan"].data = _Fake((4096,), torch.uint8)
    d.update(kw)
    return d


@pytest.mark.parametrize("bad,error", [
    (dict(q=_Fake((2, 5, 8), BF16)), ValueError), (dict(k_new=_Fake((2, 4, 2, 64), BF16)), ValueError),
    (dict(v_new=_Fake((2, 5, 2, 32), BF16)), ValueError),
    (dict(v_cache=_Fake((9, 16, 2, 32), BF16)), ValueError),
    (dict(k_cache=_Fake((9, 16, 4, 64), BF16)), ValueError),
    (dict(q=_Fake((2, 5, 8, 64), F32)), TypeError),
    (dict(v_cache=_Fake((9, 16, 2, 64), torch.float16)), TypeError),
    (dict(q=_Fake((2, 5, 8, 64), BF16, strides=(2560, 512, 1, 8))), ValueError),
    (dict(q=_Fake((2, 5, 8, 64), BF16, strides=(2600, 513, 64, 1))), ValueError),
    (dict(k_new=_Fake((2, 5, 2, 64), BF16, "cuda:1")), ValueError),
    (dict(page_table=None), ValueError), (dict(page_table=_Fake((2, 5), I32)), ValueError),
    (dict(scale=0.0), ValueError), (dict(scale=math.nan), ValueError)])
def test_attention_binding_refuses(lib, bad, error):
    with pytest.raises(error):
        sv.spec_tree_attention(**_attention_args(**bad))


def test_page_sizes_that_the_attention_refuses(lib):
    for S in (1, 4, 24, 192):
        a = _attention_args(k_cache=_Fake((9, S, 2, 64), BF16), v_cache=_Fake((9, S, 2, 64), BF16))
        a["plan"].geometry = (S, 4, 9)
        with pytest.raises(ValueError, match="page size"):
            sv.spec_tree_attention(**a)


@pytest.mark.parametrize("bad,error", [
    (dict(k_cache=_Fake((9, 16, 2, 64), BF16)), ValueError),
    (dict(v_new=_Fake((3, 2, 5, 2, 32), BF16)), ValueError),
    (dict(k_cache=_Fake((2, 9, 16, 2, 64), BF16)), ValueError),
    (dict(k_new=_Fake((3, 2, 5, 2, 64), I32), v_new=_Fake((3, 2, 5, 2, 64), I32)), TypeError),
    (dict(v_cache=_Fake((3, 9, 16, 2, 64), F32)), TypeError),
    (dict(out_num_accepted=_Fake((2,), torch.int64)), ValueError),
    (dict(out_nodes=_Fake((2, 4), I32)), ValueError),
    (dict(k_new=_Fake((3, 2, 5, 2, 64), BF16, strides=(1, 2, 3, 4, 5))), ValueError)])
def test_commit_binding_refuses(lib, bad, error):
    d = dict(k_new=_Fake((3, 2, 5, 2, 64), BF16), v_new=_Fake((3, 2, 5, 2, 64), BF16),
             k_cache=_Fake((3, 9, 16, 2, 64), BF16), v_cache=_Fake((3, 9, 16, 2, 64), BF16),
             cache_len=_Fake((2,), I32), out_num_accepted=_Fake((2,), I32),
             out_nodes=_Fake((2, 5), I32), page_table=_Fake((2, 4), I32))
    d.update(bad)
    with pytest.raises(error):
        sv.spec_tree_commit(**d)


@pytest.mark.parametrize("bad", [
    dict(logits=_Fake((2, 100), F32)), dict(logits=_Fake((2, 4, 100), F32, contiguous=False)),
    dict(history=_Fake((2, 9), I32)), dict(history_len=_Fake((2,), I32)),
    dict(draft_tokens=_Fake((2, 5), I32)), dict(draft_tokens=_Fake((2, 2), I32)),
    dict(parent=_Fake((2, 4), I32)),
    dict(parent=_Fake((2, 4), I32), draft_tokens=_Fake((2, 3), I32)),
    dict(n_nodes=_Fake((3,), I32)), dict(repetition=_Fake((2,), torch.float64)),
    dict(bias_tokens=_Fake((2, 3), I32)), dict(bias_values=_Fake((2, 3), F32)),
    dict(bias_tokens=_Fake((2, 5000), I32), bias_values=_Fake((2, 5000), F32)),
    dict(allowed=_Fake((2, 4, 3), I32)), dict(allowed=_Fake((2, 3, 4), I32)),
    dict(allowed=_Fake((2, 4, 4), torch.int64)),
    dict(allowed=_Fake((2, 4, 4), I32, strides=(32, 8, 2)))])
def test_logits_binding_refuses(bad):
    with pytest.raises(ValueError):
        sv.spec_process_logits(**{"logits": _Fake((2, 4, 100), F32), **bad})
    with pytest.raises(TypeError):
        sv.spec_process_logits(_Fake((2, 4, 100), torch.float16))


# ------------------------------------------------- the restatements themselves

def test_restatements_on_worked_examples():
    """Two keys of equal score average their values; a sibling is not seen; a
    penalty of each kind by hand."""
    q = torch.ones((1, 3, 1, 8))
    kn, vn = torch.zeros((1, 3, 1, 8)), torch.arange(24.0).view(1, 3, 1, 8)
    kc = torch.zeros((1, 4, 1, 8))
    vc = torch.full((1, 4, 1, 8), 100.0)
    parent = np.array([[-1, 0, 0]], np.int32)
    out, lse, _, _ = su.attention_ref(q, kn, vn, kc, vc, parent, [3], [1])
    assert out[0, 0, 0, 0] == (100 + 0) / 2 and abs(out[0, 2, 0, 1] - (100 + 1 + 17) / 3) < 1e-12
    assert abs(lse[0, 1, 0] - math.log(3)) < 1e-12
    x = np.array([[[2.0, -2.0, 1.0, 0.5], [2.0, -2.0, 1.0, 0.5]]])
    y, written, _ = su.logits_ref(
        x, history=np.array([[0, 1, 1]]), history_len=np.array([3]), prompt_len=np.array([1]),
        draft_tokens=np.array([[3]]), repetition=[2.0], frequency=[0.25], presence=[1.0],
        bias_tokens=np.array([[2, -1, 2]]), bias_values=np.array([[1.0, 9.0, 0.5]]),
        allowed=np.array([[[0b1111], [0b1011]]], np.uint32))
    np.testing.assert_array_equal(y[0, 0], [1.0, -4 - 0.5 - 1, 2.5, 0.5])
    np.testing.assert_array_equal(y[0, 1], [1.0, -5.5, -math.inf, 0.25 - 0.25 - 1])
    assert written.all()
    pos, status, mask = su.plan_ref(np.array([[-1, 0, 0, 1], [-1, 1, 0, 0]]), [4, 2], [10, 0], 20)
    assert pos.tolist() == [[10, 11, 11, 12], [-1] * 4] and status.tolist() == [0, -1]
    assert mask[0, :, 0].tolist() == [1, 3, 5, 11]


# ------------------------------------------- workspaces, lengths, empty plans

class _FakeTorch:
    """What the workspace caches use of torch, without a GPU."""
    uint8 = torch.uint8

    class cuda:
        @staticmethod
        def is_current_stream_capturing():
            return False

        @staticmethod
        def stream(s):
            return contextlib.nullcontext()

    @staticmethod
    def empty(n, dtype, device):
        return torch.empty(n, dtype=dtype)

    zeros = empty


def _by_threads(call):
    """call() twice in this thread and twice in another one."""
    other = []
    t = threading.Thread(target=lambda: other.extend([call(), call()]))
    t.start()
    t.join()
    return [call(), call()], other


def test_attention_workspace_belongs_to_one_thread(lib, monkeypatch):
    """A call's two kernels hand partial sums over in it, and another thread's call on the same
    stream may come between them."""
    monkeypatch.setattr(sv, "_torch", lambda: _FakeTorch)
    dev = torch.device("cuda:0")
    (a, b), (c, d) = _by_threads(lambda: sv._attention_workspace(4, 8, 2, 64, dev, 7, None))
    assert a is b and c is d and a is not c
    assert sv._attention_workspace(4, 8, 2, 64, dev, 8, None) is not a
    assert sv._attention_workspace(4, 8, 2, 64, dev, 7, None) is a


def test_verification_workspace_belongs_to_one_thread(lib, monkeypatch):
    monkeypatch.setattr(sv, "_torch", lambda: _FakeTorch)
    dev, stream = torch.device("cuda:0"), type("Stream", (), {"cuda_stream": 7})()
    (a, b), (c, d) = _by_threads(lambda: sv._cached_workspace(1000, dev, stream))
    assert a is b and c is d and a is not c


def test_attention_selftest_refusals(lib):
    ws = lib.spec_tree_attention_workspace_size(4, 8, 2, 64)
    vp = ctypes.c_void_p
    for cta, after, a in ((-1, 0, attention()), (0, -1, attention()), (0, 0, attention(q=0))):
        assert lib.spec_selftest_attention_timeout(ctypes.byref(a), vp(A), ws, cta, after,
                                                   None) == sv.SPEC_EINVAL


def test_commit_refuses_lengths_over_its_inputs(lib):
    """CTAs of a sequence read its inputs while one of them writes its length."""
    def call(**kw):
        a = _set(sv._CommitArgs(), k_new=A, v_new=A, k_cache=A, v_cache=A, cache_len=4 * A,
                 out_num_accepted=5 * A, out_nodes=6 * A, page_table=7 * A, out_len=2 * A, layers=1,
                 B=2, N=4, Hkv=2, D=64, page_size=16, pages_per_seq=4, num_pages=9, elem_size=2)
        return lib.spec_tree_commit(ctypes.byref(_set(a, **kw)), None)
    for at in (4 * A, 4 * A + 4, 4 * A - 4, 5 * A, 5 * A + 4, 6 * A - 4, 6 * A + 28, 7 * A + 28,
               7 * A - 4):
        assert call(out_len=at) == sv.SPEC_EINVAL, hex(at)


def test_status_of_an_empty_batch(lib):
    """Nothing ran, and nothing was written to read."""
    assert sv.TreePlan(0, 5, (16, 4, 9), None).read_status() == sv.SPEC_DEV_OK


def test_commit_refuses_more_runs_than_it_counts(lib):
    """A path's runs of strided heads are counted in 32 bits."""
    a = _set(sv._CommitArgs(), k_new=A, v_new=A, k_cache=A, v_cache=A, cache_len=4 * A,
             out_num_accepted=5 * A, page_table=7 * A, out_len=2 * A, layers=1, B=2, N=1024,
             Hkv=1 << 21, D=8, page_size=16, pages_per_seq=400, num_pages=900, elem_size=2,
             k_new_stride=(0, 0, 1 << 25, 16), v_new_stride=(0, 0, 1 << 25, 16),
             k_cache_stride=(0, 1 << 29, 1 << 25, 16), v_cache_stride=(0, 1 << 29, 1 << 25, 16))
    assert lib.spec_tree_commit(ctypes.byref(a), None) == sv.SPEC_EINVAL
