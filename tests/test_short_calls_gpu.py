"""The binding's short way (csrc/calls.cpp) of calls that it has seen: the results, refusals and
workspaces of the long one."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402

BF16, I32 = torch.bfloat16, dict(dtype=torch.int32, device="cuda")


@pytest.fixture(autouse=True)
def loaded():
    assert sv._load_calls() and sv._run


def case(seed, paged=True):
    """Every call on inputs of one form; the seed gives what they hold."""
    st = pu.make_chunk(seed, [40, 3, 90], [50, 500, 0], 2, 4, 64, 16 if paged else 0, BF16)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = [torch.randn(133, 2, 64, generator=gen, device="cuda").to(BF16) for _ in range(2)]
    before = torch.tensor([50, 500, 0], **I32)
    x = torch.randn(3, 4, 5003, generator=gen, device="cuda").to(BF16)
    s = -torch.rand(3, 4, generator=gen, device="cuda")
    fin = (torch.rand(3, 4, generator=gen, device="cuda") < 0.3).int()
    table = torch.randperm(99, generator=gen, device="cuda")[:60].int().view(6, 10)
    ref = torch.zeros(99, **I32)
    ref[table.flatten().long()] = 1
    size = torch.randint(0, 100, (6,), generator=gen, **I32)
    parent = torch.randint(-1, 6, (9,), generator=gen, **I32)
    kv = [torch.randn(2, 99, 10, 2, 16, generator=gen, device="cuda") for _ in range(2)]

    def every():
        kc, vc = st["k_cache"].clone(), st["v_cache"].clone()
        length = sv.spec_chunk_append(*new, kc, vc, st["start"], before, st["table"])
        plan = sv.spec_chunk_plan(st["start"], length, st["q"], kc, st["table"])
        out = sv.spec_chunk_attention(st["q"], kc, vc, plan, st["table"])
        picked = sv.spec_beam_select(x, s, 5, finished=fin, end_token=7)
        state = sv.spec_beam_reorder(x, picked[1])
        forked = sv.spec_pages_fork(table, size, parent, ref, 10)
        a, b = kv[0].clone(), kv[1].clone()
        sv.spec_pages_copy(a, b, forked[3])
        moved = sv.spec_pages_compact(forked[0], forked[2], 10)
        sv.spec_pages_copy(a, b, moved[2])
        assert plan.status.tolist() == [0, 0, 0] and plan.geometry == (
            st["k_cache"].shape[1], st["table"].shape[1] if paged else 1, st["k_cache"].shape[0])
        return [kc, vc, length, out, *picked, state, *forked, *moved, a, b]
    return every


def same(a, b):
    return all(x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype
               and torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(a, b))


def counted(monkeypatch):
    """How many calls went the short way."""
    took, run = [], sv._run

    def wrapped(*a):
        got = run(*a)
        took.append(got is not None)
        return got
    monkeypatch.setattr(sv, "_run", wrapped)
    return took


@pytest.mark.parametrize("paged", [True, False])
def test_both_ways_agree(monkeypatch, paged):
    calls = [case(seed, paged) for seed in range(3)]
    with monkeypatch.context() as m:
        m.setattr(sv, "_run", None)
        want = [call() for call in calls]
    took = counted(monkeypatch)
    assert all(same(call(), w) for call, w in zip(calls, want))
    assert sum(took) == len(took) == 3 * 9


def test_what_a_call_depends_on_is_looked_at(monkeypatch):
    """A call that differs in a dtype, a stride, a number or a missing tensor goes the long way first,
    and one that is refused there is refused again."""
    x, s = torch.randn(2, 3, 999, device="cuda"), torch.zeros(2, 3, device="cuda")
    fin = torch.zeros(2, 3, **I32)
    sv.spec_beam_select(x, s, 3)
    took = counted(monkeypatch)
    sv.spec_beam_select(x, s, 3)
    for again in range(2):
        sv.spec_beam_select(x, s, 2)
        sv.spec_beam_select(x, s, 3, end_token=5)
        sv.spec_beam_select(x, s, 3, finished=fin)
        sv.spec_beam_select(x.bfloat16(), s, 3)
        sv.spec_beam_select(x[:1], s[:1], 3)
    assert took == [True] + [False] * 5 + [True] * 5
    for bad in (dict(scores=s.double()), dict(scores=s.t().contiguous().t()), dict(n=65),
                dict(logits=x[..., :500]), dict(logits=x.cpu())):
        for _ in range(2):
            with pytest.raises(ValueError):
                sv.spec_beam_select(**{**dict(logits=x, scores=s, n=3), **bad})


def test_addresses_are_looked_at_in_every_call():
    """Shapes and strides of a call that is known, an address that the library refuses."""
    st = pu.make_chunk(1, [5], [20], 1, 4, 64, 16, BF16)
    plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"], st["table"])
    for _ in range(2):
        sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan, st["table"])
    room = torch.zeros(st["q"].numel() + 1, dtype=BF16, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        sv.spec_chunk_attention(room[1:].view(st["q"].shape), st["k_cache"], st["v_cache"], plan,
                                st["table"])


def test_plans_are_told_apart():
    """A plan of the same bytes for another cache's geometry is refused, whatever calls were seen."""
    a, b = (pu.make_chunk(1, [5], [20], 1, 4, 64, 16, BF16, cap=c) for c in (32, 64))
    for st in (a, b):
        plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"], st["table"])
        sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan, st["table"])
    plan = sv.spec_chunk_plan(a["start"], a["length"], a["q"], a["k_cache"], a["table"])
    with pytest.raises(ValueError, match="plan is for"):
        sv.spec_chunk_attention(b["q"], b["k_cache"], b["v_cache"], plan, b["table"])
    again = sv.spec_chunk_plan(b["start"], b["length"], b["q"], b["k_cache"], b["table"], plan=plan)
    assert again is plan
    got = sv.spec_chunk_attention(b["q"], b["k_cache"], b["v_cache"], plan, b["table"])
    want = sv.spec_chunk_attention(b["q"], b["k_cache"], b["v_cache"],
                                   sv.spec_chunk_plan(b["start"], b["length"], b["q"], b["k_cache"],
                                                      b["table"]), b["table"])
    assert torch.equal(got, want)


def test_threads_streams_and_graphs(monkeypatch):
    """A thread or stream without a workspace of its own goes the long way once; a captured call with a
    workspace always does, since it needs one that is the graph's."""
    call = case(5)
    want = call()
    took = counted(monkeypatch)
    assert same(call(), want) and all(took)
    took.clear()
    others = []
    t = threading.Thread(target=lambda: others.extend([call(), call()]))
    t.start()
    t.join()
    assert took.count(False) == 3 and all(took[9:]) and all(same(o, want) for o in others)
    took.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert same(call(), want) and same(call(), want)
    assert took.count(False) == 3 and all(took[9:])
    x, s = torch.randn(2, 3, 999, device="cuda"), torch.zeros(2, 3, device="cuda")
    ref = sv.spec_beam_select(x, s, 3)
    state = sv.spec_beam_reorder(x, ref[1])
    took.clear()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.spec_beam_select(x, s, 3)
        moved = sv.spec_beam_reorder(x, got[1])
    assert took == [False, True]
    g.replay()
    assert same(got, ref) and torch.equal(moved, state)
