"""Logits processing against its plain 64-bit restatement (tests/serve_util.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import serve_util as su  # noqa: E402

F32, BF16 = torch.float32, torch.bfloat16


def make(B, R, V, seed=0, hist=50, chain=True, cols=None, bias=0, mask=None, words=None):
    rng = np.random.default_rng(seed)
    words = words or V
    c = {}
    if hist is not None:
        c["history"] = rng.integers(0, words, (B, hist)).astype(np.int32)
        c["history_len"] = rng.integers(0, hist + 1, B).astype(np.int32)
        c["prompt_len"] = (rng.random(B) * (c["history_len"] + 1)).astype(np.int32)
    cols = (R - 1 if chain else R) if cols is None else cols
    c["draft_tokens"] = rng.integers(0, words, (B, cols)).astype(np.int32)
    if not chain:
        c["parent"] = np.stack([su.random_tree(rng, R, "tree") for _ in range(B)])
        c["draft_tokens"][:, 0] = -5
    c["repetition"] = rng.uniform(0.7, 1.6, B).astype(np.float32)
    c["frequency"] = rng.uniform(-0.5, 1, B).astype(np.float32)
    c["presence"] = rng.uniform(-0.5, 1, B).astype(np.float32)
    if bias:
        c["bias_tokens"] = rng.integers(-1, words, (B, bias)).astype(np.int32)  # repeats too
        c["bias_values"] = rng.normal(0, 3, (B, bias)).astype(np.float32)
    if mask is not None:
        shape = {"row": (B, R), "sequence": (B, 1), "one": (1, 1)}[mask]
        c["allowed"] = rng.integers(0, 2 ** 32, (*shape, -(-V // 32)), dtype=np.uint32)
        c["allowed"][0, 0, :] = 0  # a row that may be nothing
    return c


def inputs(B, R, V, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((B, R, V), generator=gen) * 4).to(dtype)


def dev(c):
    return {k: torch.from_numpy(v.view(np.int32) if v.dtype == np.uint32 else v).cuda()
            for k, v in c.items()}


def check(x, c, in_place=False):
    out = torch.full_like(x, 77.0).cuda()
    src = x.cuda()
    if in_place:
        out = src
    got = sv.spec_process_logits(src, out=out, **dev(c))
    assert got is out
    got = out.cpu()
    want, written, mag = su.logits_ref(x.double().numpy(), **c)
    keep = torch.from_numpy(written)
    rest = x if in_place else torch.full_like(x, 77.0)
    assert torch.equal(got[~keep], rest[~keep])  # rows past n_nodes are left alone
    got, want, mag = got[keep].double().numpy(), want[written], mag[written]
    for kind in (np.isnan, np.isposinf, np.isneginf):
        np.testing.assert_array_equal(kind(got), kind(want))
    fine = np.isfinite(want)
    # up to six fp32 operations on terms of these magnitudes, each off by half a step, and the
    # result's own rounding
    half = torch.finfo(x.dtype).eps / 2
    tol = 8 * 2.0 ** -24 * mag[fine] + half * np.abs(want[fine])
    assert np.all(np.abs(got[fine] - want[fine]) <= tol * 1.001)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,R,V", [(1, 1, 2), (3, 5, 31), (2, 4, 33), (4, 9, 1000), (2, 3, 4099),
                                   (3, 2, 8192), (1, 7, 100003), (40, 3, 5001), (2, 6, 128256)])
def test_sizes(B, R, V, dtype):
    """Rows that start anywhere, in one tile or many; every kind of change."""
    for mask in (None, "row"):
        check(inputs(B, R, V, dtype), make(B, R, V, seed=V, bias=20, mask=mask))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_words_repeat_often(dtype):
    """Many occurrences of the same tokens in the prompt, the history and the drafts."""
    check(inputs(3, 9, 700, dtype), make(3, 9, 700, seed=1, hist=3000, words=7, bias=300))
    check(inputs(3, 40, 700, dtype), make(3, 40, 700, seed=2, hist=100, chain=False, words=4))


@pytest.mark.parametrize("R", [1, 2, 29, 200, 1024])
def test_trees(R):
    c = make(2, R, 501, seed=R, chain=False, mask="row", bias=3)
    check(inputs(2, R, 501, BF16), c)
    c["n_nodes"] = np.array([R, max(1, R // 2)], np.int32)
    c["draft_tokens"][1, max(1, R // 2):] = -9     # past the count: ignored
    c["parent"][1, max(1, R // 2):] = 10 ** 6
    check(inputs(2, R, 501, BF16), c)


def test_draft_rows_and_count_of_rows():
    """Chains with as many tokens as rows (the draft's own rows), and rows past n_nodes."""
    c = make(3, 6, 301, seed=3, cols=6)
    c["draft_tokens"][:, 5] = 10 ** 6              # no row follows the last token
    check(inputs(3, 6, 301, F32), c)
    c["n_nodes"] = np.array([1, 6, 3], np.int32)
    c["draft_tokens"][0] = -3
    check(inputs(3, 6, 301, F32), c)


@pytest.mark.parametrize("mask", ["row", "sequence", "one"])
def test_shared_masks_and_in_place(mask):
    check(inputs(4, 5, 777, BF16), make(4, 5, 777, seed=4, mask=mask), in_place=True)
    check(inputs(4, 5, 4096, F32), make(4, 5, 4096, seed=5, mask=mask, bias=9), in_place=True)


def test_parts_alone():
    B, R, V = 3, 4, 2049
    full = make(B, R, V, seed=6, bias=5, mask="row")
    for names in ((), ("repetition",), ("allowed",), ("bias_tokens", "bias_values"),
                  ("draft_tokens", "presence"), ("history", "history_len", "prompt_len", "frequency"),
                  ("history", "history_len", "prompt_len", "repetition")):
        check(inputs(B, R, V, F32, seed=7), {k: full[k] for k in names})


def test_nonfinite_logits():
    """NaN and infinities go through untouched places bit by bit, and masked places are -inf."""
    x = inputs(2, 2, 999, F32, seed=8)
    x[0, 0, 5], x[0, 1, 6], x[1, 0, 7], x[1, 1, :] = math.nan, math.inf, -math.inf, -math.inf
    c = make(2, 2, 999, seed=9, words=20, bias=5)
    check(x, c)
    c["allowed"] = np.full((2, 2, 32), 0xffffffff, np.uint32)
    c["allowed"][0, 0, 0] &= ~np.uint32(1 << 5)
    check(x, c)
    nan = torch.full((1, 1, 64), 0x7fc12345, dtype=torch.int32).view(F32)
    got = sv.spec_process_logits(nan.cuda())
    assert torch.equal(got.view(torch.int32).cpu(), nan.view(torch.int32))


def test_bad_sequences_are_nan():
    """Each kind of bad value fills its own sequence's rows and no other's."""
    B, R, V = 14, 4, 3000
    c = make(B, R, V, seed=10, bias=4, chain=False)
    c["n_nodes"] = np.full(B, R, np.int32)
    c["history_len"][:] = 50
    c["prompt_len"][:] = 20
    c["repetition"][1], c["repetition"][2], c["repetition"][3] = 0.0, math.nan, math.inf
    c["frequency"][4] = math.inf
    c["presence"][5] = math.nan
    c["history_len"][6] = 51
    c["prompt_len"][7] = 51
    c["history"][8, 49] = V
    c["history"][9, 0] = -1
    c["draft_tokens"][10, 3] = V
    c["parent"][11, 2] = 2
    c["bias_tokens"][12, 0] = -2
    c["n_nodes"][13] = 0
    check(inputs(B, R, V, BF16), c)


def test_long_history_and_large_counts():
    c = make(1, 2, 40, seed=11, hist=200000, words=3)
    c["history_len"][:], c["prompt_len"][:] = 200000, 5
    check(inputs(1, 2, 40, F32), c)


def test_step_masked_then_verified():
    """Masked and penalised rows go straight into the verification: an accepted or drawn
    token is always one that its row's mask allows."""
    rng = np.random.default_rng(12)
    B, k, V = 64, 4, 1000
    x = inputs(B, k + 1, V, F32, seed=13).cuda()
    d = inputs(B, k, V, F32, seed=14).cuda()
    c = make(B, k + 1, V, seed=15, mask="row")
    c["allowed"][0, 0, 0] = 6
    c["draft_tokens"] = rng.integers(0, V, (B, k)).astype(np.int32)
    a = dev(c)
    t = sv.spec_process_logits(x, **a)
    tok, n = sv.spec_verify(t, d, a["draft_tokens"],
                            torch.from_numpy(rng.random((B, k), np.float32)).cuda(),
                            torch.from_numpy(rng.random(B, np.float32)).cuda(),
                            torch.full((B,), 0.8, device="cuda"))
    tok, n = tok.cpu().numpy(), n.cpu().numpy()
    assert (n >= 0).all()
    for b in range(B):
        for i in range(n[b] + 1):
            x = int(tok[b, i])
            assert (int(c["allowed"][b, i, x // 32]) >> (x % 32)) & 1


def test_many_sequences_on_another_stream():
    x = inputs(5, 3, 900, BF16, seed=16).cuda()
    c = dev(make(5, 3, 900, seed=17))
    want = sv.spec_process_logits(x, **c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sv.spec_process_logits(x, stream=s, **c)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("V", [64, 61])
def test_columns_of_other_rows_keep_their_bits(V, dtype):
    """A token drafted on another row's path only, and no bias for it: -0 and the bits of a NaN
    stay, beside columns that do change."""
    word, ints = {F32: (torch.int32, (-2 ** 31, 0x7fc12345)),
                  BF16: (torch.int16, (-2 ** 15, 0x7fc5))}[dtype]
    for value in ints:
        x = inputs(1, 4, V, dtype, seed=18)
        for token in (5, 9, 60):
            x[0, :, token] = torch.tensor(value, dtype=word).view(dtype)
        i32 = lambda *a: torch.tensor([a], dtype=torch.int32, device="cuda")  # noqa: E731
        one = lambda v: torch.tensor([v], device="cuda")  # noqa: E731
        got = sv.spec_process_logits(
            x.cuda(), draft_tokens=i32(-1, 5, 9, 60), parent=i32(-1, 0, 0, 2), repetition=one(1.5),
            frequency=one(0.25), presence=one(0.5), bias_tokens=i32(7, -1), bias_values=i32(1, 1).float())
        bits, was = got.cpu().view(word)[0], x.view(word)[0]
        path = [[], [5], [9], [9, 60]]
        for r in range(4):
            keep = [t for t in range(V) if t != 7 and t not in path[r]]
            assert torch.equal(bits[r, keep], was[r, keep]), (value, r)
            assert not torch.equal(got.cpu()[0, r, 7], x[0, r, 7])
