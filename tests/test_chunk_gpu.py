"""Chunk attention, its plan and the append on a GPU against 64-bit restatements
(prefill_util.py), with serve_util's derived tolerance."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402
from tests import serve_util as su  # noqa: E402


def attend(st, **kw):
    plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"],
                              page_table=st["table"])
    out, lse = sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan,
                                       page_table=st["table"], want_lse=True, **kw)
    assert plan.read_status() == sv.SPEC_DEV_OK
    return out, lse, plan


def check(st, out, lse, scale=None, rows=slice(None)):
    ref, rlse, mag, big = pu.chunk_ref(st, scale)
    D, keys = ref.shape[2], int(st["length"].max())
    tol = su.attention_tolerance(ref, mag, big, st["q"].dtype, D, keys)
    off = (out.double() - ref).abs()[rows]
    assert not bool(torch.isnan(out[rows]).any())
    worst = float((off / tol[rows]).max())
    assert worst <= 1, worst
    # the logarithm: its scores' rounding, the total's (fp32 sums) and its own
    ltol = (D + 4) * 2.0 ** -23 * big + 2.0 ** -16 + rlse.abs() * 2.0 ** -22
    assert bool(((lse.double() - rlse).abs() <= ltol)[rows].all())


CASES = [
    # new, past, Hkv, G, D, S, dtype
    ([1], [0], 1, 1, 64, 0, torch.bfloat16),
    ([1], [127], 2, 4, 128, 16, torch.bfloat16),
    ([1, 1, 1], [128, 129, 0], 2, 4, 128, 8, torch.float16),
    ([2, 0, 130], [5, 9, 300], 2, 3, 64, 32, torch.bfloat16),
    ([127, 128, 129], [0, 0, 0], 2, 1, 128, 64, torch.bfloat16),
    ([256, 257], [1, 255], 1, 1, 40, 128, torch.float16),
    ([40, 3, 0, 77], [200, 513, 64, 0], 3, 5, 72, 16, torch.bfloat16),
    ([65, 64, 63], [63, 64, 65], 2, 4, 128, 256, torch.float16),
    ([33], [1000], 2, 7, 96, 64, torch.bfloat16),
    ([19, 6], [31, 400], 1, 16, 128, 8, torch.bfloat16),
    ([5], [260], 1, 128, 64, 64, torch.float16),
    ([3, 2], [130, 7], 1, 65, 8, 16, torch.bfloat16),
    ([600], [0], 1, 2, 128, 0, torch.bfloat16),
    ([300, 17], [0, 700], 4, 8, 64, 0, torch.float16),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_64_bits(i):
    new, past, Hkv, G, D, S, dtype = CASES[i]
    st = pu.make_chunk(i, new, past, Hkv, G, D, S, dtype)
    out, lse, plan = attend(st)
    assert plan.status.tolist() == [0] * len(new)
    check(st, out, lse)
    again = attend(st)[0]
    assert torch.equal(out, again)


@pytest.mark.parametrize("new,past,Hkv,G,S,dtype", [
    ([1024, 700, 1], [2048, 100, 3000], 2, 4, 64, torch.bfloat16),
    ([512], [20000], 2, 5, 256, torch.bfloat16),
    ([7] * 40, list(range(0, 4000, 100)), 2, 4, 16, torch.float16),
    ([3000], [0], 2, 8, 0, torch.bfloat16),
])
def test_longer_ones(new, past, Hkv, G, S, dtype):
    st = pu.make_chunk(3, new, past, Hkv, G, 128, S, dtype)
    out, lse, _ = attend(st)
    check(st, out, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.02, 1.0, 3.0])
def test_scores_that_grow_along_the_keys(dtype, scale):
    """The maximum rises from tile to tile, so the sums are rescaled again and again."""
    st = pu.make_chunk(5, [70, 200], [900, 0], 2, 4, 64, 16, dtype)
    st["q"][:] = 0.25
    for b, n in enumerate(st["length"].tolist()):
        pages, slots = pu.positions(st, b, n)
        ramp = torch.linspace(-1, 1, n, device="cuda")[:, None, None].expand(n, 2, 64)
        st["k_cache"][pages, slots] = ramp.to(dtype)
    out, lse, _ = attend(st, scale=scale)
    check(st, out, lse, scale)


def test_strided_inputs():
    """Queries as a slice of a projection, heads before slots, layers between pages."""
    st = pu.make_chunk(6, [50, 20], [100, 30], 2, 4, 64, 16, torch.bfloat16)
    plain, lse, _ = attend(st)
    q = torch.zeros(70, 12, 64, dtype=torch.bfloat16, device="cuda")
    q[:, 2:10] = st["q"]
    wide = dict(st, q=q[:, 2:10])
    for name in ("k_cache", "v_cache"):
        x = st[name]
        y = torch.full((x.shape[0], 3, 2, 16, 72), float("nan"), dtype=x.dtype, device="cuda")
        y[:, 1, :, :, :64] = x.transpose(1, 2)
        wide[name] = y[:, 1, :, :, :64].transpose(1, 2)
    out, lse2, _ = attend(wide)
    assert torch.equal(out, plain) and torch.equal(lse, lse2)


@pytest.mark.parametrize("poison", [math.nan, math.inf, -math.inf])
def test_what_lies_behind_a_length_has_no_effect(poison):
    st = pu.make_chunk(7, [37, 5, 1], [100, 0, 127], 2, 4, 128, 16, torch.bfloat16, cap=400)
    want, wl, _ = attend(st)
    keep = torch.zeros(st["k_cache"].shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(st["length"].tolist()):
        keep[pu.positions(st, b, n)] = True
        st["table"][b, -(-n // 16):] = torch.tensor(-7 if b else 1 << 30, dtype=torch.int32)
    for name in ("k_cache", "v_cache"):
        st[name][~keep] = poison
    got, gl, plan = attend(st)
    assert plan.status.tolist() == [0, 0, 0]
    assert torch.equal(got, want) and torch.equal(gl, wl)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("at", [(0, 3), (0, 40), (1, 0), (1, 19), (2, 0)])
def test_a_value_affects_only_rows_that_see_it(D, value, at):
    """A non-finite element of a new token's value: earlier rows keep their bits, later
    ones have it in that column and nowhere else."""
    b, i = at
    st = pu.make_chunk(8, [60, 20, 1], [50, 128, 7], 2, 2, D, 16, torch.bfloat16)
    start, pasts = st["start"].tolist(), [50, 128, 7]
    want, _, _ = attend(st)
    S, pos = 16, pasts[b] + i
    page = int(st["table"][b, pos // S])
    st["v_cache"][page, pos % S, 1, 5] = value
    zeroed = dict(st, v_cache=st["v_cache"].clone())
    zeroed["v_cache"][page, pos % S, 1, 5] = 0
    clean, _, _ = attend(zeroed)
    got, _, _ = attend(st)
    row = start[b] + i
    late = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    late[row:start[b + 1], 2:4, 5] = True
    if math.isnan(value):
        assert bool(torch.isnan(got[late]).all())
    else:
        assert bool((got[late] == value).all())
    assert torch.equal(got[~late], clean[~late])
    early = torch.ones_like(late)
    early[row:start[b + 1], 2:4] = False
    assert torch.equal(got[early], want[early])


def test_a_key_affects_only_rows_that_see_it():
    st = pu.make_chunk(9, [60], [70], 1, 4, 64, 16, torch.float16)
    want, _, _ = attend(st)
    for i in (0, 31, 57):
        bad = dict(st, k_cache=st["k_cache"].clone())
        page, slot = pu.positions(st, 0, 130)
        bad["k_cache"][page[70 + i], slot[70 + i], 0, 0] = math.nan
        got, _, _ = attend(bad)
        assert torch.equal(got[:i], want[:i])
        assert bool(torch.isnan(got[i:]).all())


def test_errors_mark_their_sequence_only():
    st = pu.make_chunk(10, [9, 30, 4, 50, 6], [20, 10, 0, 300, 40], 2, 4, 64, 16, torch.bfloat16)
    want, wl, _ = attend(st)
    st["table"][1, 2] = -1                      # a page that a position needs
    st["table"][3, 5] = st["k_cache"].shape[0]
    st["length"][4] = 5                          # fewer positions than rows
    out, lse, plan = attend(st)
    assert plan.status.tolist() == [0, -1, 0, -1, -1]
    start = st["start"].tolist()
    for b in range(5):
        rows = slice(start[b], start[b + 1])
        if b in (0, 2):
            assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wl[rows])
        else:
            assert bool(torch.isnan(out[rows]).all()) and bool(torch.isnan(lse[rows]).all())


@pytest.mark.parametrize("start", [[0, 9, 5, 20], [-1, 5, 9, 20], [0, 5, 9, 21]])
def test_rows_that_are_no_runs_fail_every_sequence(start):
    st = pu.make_chunk(11, [5, 4, 11], [20, 10, 0], 2, 4, 64, 16, torch.bfloat16)
    st["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    out, lse, plan = attend(st)
    assert plan.status.tolist() == [-1, -1, -1]
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


def test_rows_of_no_sequence_are_left_alone():
    st = pu.make_chunk(12, [5, 40], [20, 100], 2, 4, 128, 16, torch.bfloat16)
    want, _, _ = attend(st)
    q = torch.full((60, 8, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    q[4:49] = st["q"]
    moved = dict(st, q=q, start=st["start"] + 4)
    out = torch.full_like(q, 7.0)
    plan = sv.spec_chunk_plan(moved["start"], moved["length"], q, st["k_cache"],
                              page_table=st["table"])
    got = sv.spec_chunk_attention(q, st["k_cache"], st["v_cache"], plan, page_table=st["table"],
                                  out=out)
    assert torch.equal(got[4:49], want)
    assert bool((got[:4] == 7).all()) and bool((got[49:] == 7).all())


def test_no_rows_and_no_sequences():
    st = pu.make_chunk(13, [0, 0], [20, 0], 2, 4, 64, 16, torch.bfloat16)
    out, _, plan = attend(st)
    assert out.shape == (0, 8, 64) and plan.status.tolist() == [0, 0]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    q = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    plan = sv.spec_chunk_plan(none.new_zeros(1), none, q, st["k_cache"],
                              page_table=st["table"][:0].contiguous())
    assert sv.spec_chunk_attention(q, st["k_cache"], st["v_cache"], plan,
                                   page_table=st["table"][:0].contiguous()).numel() == 0


def test_many_sequences():
    rng = np.random.default_rng(4)
    new, past = rng.integers(0, 4, 600), rng.integers(0, 90, 600)
    st = pu.make_chunk(14, new, past, 1, 4, 64, 16, torch.bfloat16)
    out, lse, _ = attend(st)
    check(st, out, lse)


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("S,D,dtype", [(16, 64, torch.bfloat16), (5, 24, torch.float32),
                                       (0, 7, torch.float16), (1, 128, torch.bfloat16)])
def test_append(layers, S, D, dtype):
    new, past = [4, 0, 33, 1], [7, 20, 0, 15]
    st = pu.make_chunk(15, new, past, 2, 1, D, S, dtype, cap=40)
    L = layers or 1
    shape = (L, *st["k_cache"].shape)
    gen = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2))
    kn, vn = (torch.randn((L, 40, 2, D), generator=gen).to(dtype).cuda() for _ in range(2))
    start = torch.tensor([1, 5, 5, 38, 39], dtype=torch.int32, device="cuda")
    lens = torch.tensor(past, dtype=torch.int32, device="cuda")
    wk, wv = kc.clone(), vc.clone()
    full = torch.tensor(new) + torch.tensor(past)
    for b in range(4):
        pages, slots = pu.positions(st, b, int(full[b]))
        rows = slice(int(start[b]), int(start[b + 1]))
        wk[:, pages[past[b]:], slots[past[b]:]] = kn[:, rows]
        wv[:, pages[past[b]:], slots[past[b]:]] = vn[:, rows]
    a = (kn, vn, kc, vc) if layers else (kn[0], vn[0], kc[0], vc[0])
    got = sv.spec_chunk_append(*a, start, lens, page_table=st["table"])
    assert got.tolist() == full.tolist()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_errors_leave_the_sequence_alone():
    st = pu.make_chunk(16, [4, 5, 6, 2], [20, 20, 20, 20], 2, 1, 64, 16, torch.bfloat16)
    kn, vn = torch.randn(2, 17, 2, 64, device="cuda").to(torch.bfloat16)
    lens = torch.tensor([20, 20, 30, -1], dtype=torch.int32, device="cuda")
    st["table"][1, 1] = st["k_cache"].shape[0]
    before = st["k_cache"].clone(), st["v_cache"].clone()
    got = sv.spec_chunk_append(kn, vn, st["k_cache"], st["v_cache"], st["start"], lens,
                               page_table=st["table"])
    assert got.tolist() == [24, -1, -1, -1]
    pages, slots = pu.positions(st, 0, 24)
    for x, y, new in zip((st["k_cache"], st["v_cache"]), before, (kn, vn)):
        y[pages[20:], slots[20:]] = new[:4]
        assert torch.equal(x, y)
    bad = torch.tensor([0, 4, 3, 15, 17], dtype=torch.int32, device="cuda")
    got = sv.spec_chunk_append(kn, vn, st["k_cache"], st["v_cache"], bad, lens,
                               page_table=st["table"])
    assert got.tolist() == [-1] * 4 and torch.equal(st["k_cache"], before[0])


def test_other_streams_and_captured_graphs():
    """Two graphs of the same thread, replayed on two streams at once, and eager calls."""
    cases = [pu.make_chunk(20 + i, [300, 40], [500, 9], 2, 4, 128, 16, torch.bfloat16)
             for i in range(2)]
    want = [attend(st)[0] for st in cases]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cases], [], []
    for st, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"],
                                      page_table=st["table"])
            outs.append(sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan,
                                                page_table=st["table"]))
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = attend(cases[0])[0]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0])
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = sv.spec_chunk_plan(cases[1]["start"], cases[1]["length"], cases[1]["q"],
                              cases[1]["k_cache"], page_table=cases[1]["table"], stream=side)
    got = sv.spec_chunk_attention(cases[1]["q"], cases[1]["k_cache"], cases[1]["v_cache"], plan,
                                  page_table=cases[1]["table"], stream=side)
    side.synchronize()
    assert torch.equal(got, want[1])


class Losing:
    """The library, its chunk attention with a CTA whose wait gives up (include/spec_bench.h)."""

    def __init__(self, lib, cta, after):
        self.lib, self.lose = lib, (cta, after)

    def __getattr__(self, name):
        return getattr(self.lib, name)

    def spec_chunk_attention(self, args, ws, size, stream):
        return self.lib.spec_selftest_chunk_timeout(args, ws, size, *self.lose, stream)


# shares inside long items, and of several whole ones with idle ones among them
LONG = ([70, 5, 0, 200], [20000, 9000, 50, 30000], 2, 5)
SHORT = ([3, 0, 40, 1] * 50, [0, 9, 100, 128] * 50, 2, 5)


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("shape,cta,after", [(LONG, 0, 0), (LONG, 7, 0), (LONG, 0, 1), (LONG, 30, 1),
                                             (SHORT, 0, 0), (SHORT, 70, 1), (SHORT, 101, 2)])
def test_a_wait_that_gives_up(monkeypatch, D, dtype, shape, cta, after):
    """The status is read, a row is what it is without the lost wait or NaN throughout, none is left
    unwritten or joined from an earlier call's sums, and the next step is right, whether the CTA has
    nothing in flight (after 0) or loads and products of its pieces."""
    new, past, Hkv, G = shape
    st = pu.make_chunk(8, new, past, Hkv, G, D, 16, dtype)
    if len(new) > 4:
        st["length"][2] = -1  # a sequence in error: its item is idle

    def call():
        plan = sv.spec_chunk_plan(st["start"], st["length"], st["q"], st["k_cache"],
                                  page_table=st["table"])
        got = sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan,
                                      page_table=st["table"], want_lse=True)
        return *got, plan.read_status()
    want, want_lse, status = call()
    assert status == sv.SPEC_DEV_OK
    with monkeypatch.context() as m:
        m.setattr(sv, "_lib", Losing(sv.library(), cta, after))
        out, lse, status = call()
    assert status == sv.SPEC_DEV_WAIT_TIMEOUT
    rows = st["start"][-1]
    bad = torch.isnan(want[:rows]).all(-1)
    nan = torch.isnan(out[:rows])
    assert torch.equal(nan.all(-1), nan.any(-1))
    assert torch.equal(nan.all(-1), torch.isnan(lse[:rows]))
    assert bool((nan.all(-1) & ~bad).any()) and not bool(nan.all())
    keep = ~nan.all(-1)
    assert torch.equal(out[:rows][keep], want[:rows][keep])
    assert torch.equal(lse[:rows][keep], want_lse[:rows][keep])
    again, lse, status = call()
    assert status == sv.SPEC_DEV_OK
    assert torch.equal(torch.isnan(again), torch.isnan(want))
    assert torch.equal(again.nan_to_num(), want.nan_to_num())
