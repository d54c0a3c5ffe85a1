"""Beam selection and reordering on a GPU against a sort of all candidates in 64
bits (prefill_util.beam_ref): tokens and beams equal, scores to fp32's last bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402


def check(logits, scores, n, **kw):
    want = pu.beam_ref(logits, scores, n, **kw)
    cuda = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    tokens, beams, best = (x.cpu().numpy() for x in
                           sv.spec_beam_select(logits.cuda(), scores.cuda(), n, **cuda))
    assert np.array_equal(tokens, want[0]), np.argwhere(tokens != want[0])[:4]
    assert np.array_equal(beams, want[1])
    gone = ~np.isfinite(want[2])
    assert np.array_equal(best[gone], want[2][gone], equal_nan=True)
    # half a step of the result, and the logarithm of the total: 5e-6 by the kernel's account
    off = np.abs(best[~gone] - want[2][~gone])
    assert (off <= np.abs(want[2][~gone]) * 2.0 ** -24 + 5e-6).all(), off.max()
    return tokens, beams


def rows(seed, B, K, V, dtype, spread=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, K, V, generator=gen) * spread).to(dtype)
    return x, -10 * torch.rand(B, K, generator=gen)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V,n", [
    (1, 1, 2, 1), (2, 3, 7, 9), (1, 4, 32000, 4), (3, 5, 1003, 10), (2, 4, 9001, 64),
    (1, 64, 517, 64), (1, 2, 151937, 17), (5, 8, 20011, 16), (40, 1, 4099, 1), (1, 1, 70001, 33)])
def test_against_a_sort(dtype, B, K, V, n):
    check(*rows(B * V + n, B, K, V, dtype), n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ended_beams_and_lengths(dtype):
    x, s = rows(1, 6, 4, 5003, dtype)
    gen = torch.Generator().manual_seed(2)
    fin = (torch.rand(6, 4, generator=gen) < 0.4).int()
    fin[0] = 1
    norm = (1 + 30 * torch.rand(6, 4, generator=gen)) ** 0.7
    check(x, s, 6, finished=fin, norm=norm, end_token=17)
    check(x, s, 3, finished=fin, end_token=5002)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(dtype):
    x, s = rows(3, 3, 4, 12345, dtype)
    x[0] = 1.5                       # every logit equal: a segment has more ties than it keeps
    x[1] = torch.round(x[1])         # many ties at the cut
    x[2] = x[2, :1]                  # four equal beams, equal scores
    s[:] = -2.0
    check(x, s, 8)


@pytest.mark.parametrize("order", [1, -1])
def test_sorted_rows(order):
    """Rising logits: every tile beats all that came before."""
    x = torch.linspace(-30, 30, 50021)[::order].repeat(1, 2, 1).contiguous() if order > 0 else \
        torch.linspace(-30, 30, 50021).flip(0).repeat(1, 2, 1).contiguous()
    check(x, torch.tensor([[-1.0, -1.25]]), 20)
    check(x.to(torch.bfloat16), torch.tensor([[-1.0, -1.2]]), 64)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orders_that_fp32_leaves_open(dtype):
    """Beams whose rows are the same up to one far, light element each: scores of different beams
    differ by 1e-7 or so, below what fp32 statistics tell."""
    B, K, V = 20, 6, 30011
    x, s = rows(4, B, 1, V, dtype, 2.0)
    x = x.expand(B, K, V).clone()
    gen = torch.Generator().manual_seed(5)
    for b in range(B):
        for k in range(K):
            x[b, k, int(torch.randint(V, (1,), generator=gen))] = -2.0 - k % 3
    check(x, torch.full((B, K), -3.0), 12)


@pytest.mark.parametrize("n", [1, 2, 3])
@pytest.mark.parametrize("lengths", [False, True])
def test_the_last_place_left_open(n, lengths):
    """The best of one beam against the n-th of another to fp32's last bits, so that fp32 statistics
    may put the wrong one out, and equal logits behind the n-th."""
    B, V = 64, 6001
    x, s = rows(8, B, 2, V, torch.float32)
    x[:, 0] = torch.where(x[:, 0] > 8, 8.0, x[:, 0])  # many at the top of beam 0, all equal
    norm = torch.ones(B, 2)
    if lengths:
        norm = 1 + torch.arange(2 * B).reshape(B, 2) % 7
    rank = x.double().amax(2) - torch.logsumexp(x.double(), 2)
    s[:, 0] = -5.0
    s[:, 1] = ((s[:, 0] + rank[:, 0]) / norm[:, 0] * norm[:, 1] - rank[:, 1]).float()
    check(x, s, n, norm=norm.float())


def test_equal_ends_and_extreme_norms():
    """Ended beams whose score / norm is the same number in 64 bits; norms near fp32's ends."""
    x, s = rows(10, 5, 4, 2003, torch.float32)
    norm = torch.tensor([3.0, 2, 7, 1]).repeat(5, 1)
    s[:] = -norm
    fin = torch.ones(5, 4, dtype=torch.int32)
    norm[2], norm[3] = 1e-40, 3e38
    s[3] = -torch.tensor([3e38, 2e38, 1e-3, 1e38])
    norm[4, :2], s[4] = 1e-44, -1.0
    fin[4] = 0
    check(x, s, 3, finished=fin, norm=norm)
    check(x, s, 9, finished=fin * 0, norm=norm)


def test_hidden_logits_and_dead_beams():
    x, s = rows(6, 5, 3, 3001, torch.float32)
    ninf = -math.inf
    x[0, 0] = ninf                       # a mask that leaves nothing
    x[1] = ninf                          # in all beams
    x[2, :, 5:] = ninf                   # fewer candidates than wanted
    s[3, 1] = ninf                       # a beam that does not exist, of any logits
    x[3, 1] = math.nan
    s[4] = ninf
    tokens, _ = check(x, s, 16)
    assert (tokens[1] == -1).all() and (tokens[4] == -1).all()
    assert (tokens[2] >= 0).sum() == 15


def test_errors_mark_their_sequence_only():
    x, s = rows(7, 8, 3, 3001, torch.bfloat16)
    norm = torch.ones(8, 3)
    x[1, 2, 3000] = math.nan
    x[2, 0, 0] = math.inf
    s[3, 1] = math.nan
    s[4, 0] = math.inf
    norm[5, 2] = 0
    norm[6, 1] = math.nan
    tokens, _ = check(x, s, 5, norm=norm)
    assert (tokens[[0, 7]] >= 0).all() and (tokens[1:7] == -1).all()


def test_calls_of_several_sizes_share_a_workspace():
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    for seed, (B, K, V, n) in enumerate([(1, 4, 5000, 4), (64, 2, 700, 5), (3, 8, 40000, 16),
                                         (300, 1, 100, 3), (1, 4, 5000, 4)]):
        x, s = rows(seed, B, K, V, torch.float32)
        x[:, 1:] = x[:, :1]
        s[:] = -1
        want = pu.beam_ref(x, s, n)
        got = sv.spec_beam_select(x.cuda(), s.cuda(), n, ws=ws)
        assert np.array_equal(got[0].cpu().numpy(), want[0])
        assert np.array_equal(got[1].cpu().numpy(), want[1])


def test_captured_and_on_another_stream():
    x, s = rows(9, 3, 4, 20000, torch.bfloat16)
    want = pu.beam_ref(x, s, 8)
    x, s = x.cuda(), s.cuda()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.spec_beam_select(x, s, 8)
    for _ in range(3):
        got[0].zero_()
        g.replay()
        assert np.array_equal(got[0].cpu().numpy(), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = sv.spec_beam_select(x, s, 8, stream=side)
    side.synchronize()
    assert np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype,rest", [(torch.int32, (300,)), (torch.bfloat16, (7, 3)),
                                        (torch.uint8, (13,)), (torch.float64, (2,)),
                                        (torch.float16, (5000, 4)), (torch.int32, ())])
@pytest.mark.parametrize("lead", [(), (3,)])
def test_reorder(dtype, rest, lead):
    gen = torch.Generator().manual_seed(1)
    state = torch.randint(0, 100, (*lead, 4, 5, *rest), generator=gen).to(dtype).cuda()
    beams = torch.randint(-1, 5, (4, 7), generator=gen).int().cuda()
    beams[0, 0] = 9
    got = sv.spec_beam_reorder(state, beams, dim=len(lead))
    flat = state.view(-1, 4, 5, *rest)
    for b in range(4):
        for j in range(7):
            k = int(beams[b, j])
            want = flat[:, b, k] if 0 <= k < 5 else torch.zeros_like(flat[:, b, 0])
            assert torch.equal(got.view(-1, 4, 7, *rest)[:, b, j], want)
