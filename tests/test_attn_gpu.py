"""Tree attention, its plan and the cache commit against plain 64-bit
restatements (tests/serve_util.py)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import serve_util as su  # noqa: E402

BF16, FP16 = torch.bfloat16, torch.float16


def make(B, N, Hkv, G, D, S, cap, dtype, seed=0, kind="tree", lens=None, nodes=None, fill=None):
    """One call's inputs on the CPU.  S = 0: a contiguous cache.  Slots past a
    sequence's length, unowned pages and rows past n_nodes hold `fill`."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    parent = np.stack([su.random_tree(rng, N, kind) for _ in range(B)])
    nodes = rng.integers(1, N + 1, B) if nodes is None else np.resize(nodes, B)
    nodes = nodes.astype(np.int32)
    if S == 0:
        table, P, S, M = None, B, cap, 1
    else:
        M = -(-cap // S)
        P = B * M + 2
        table = rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32)
    lens = rng.integers(0, cap + 1, B) if lens is None else np.minimum(np.resize(lens, B), cap)
    lens = lens.astype(np.int32)
    r = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    c = dict(q=r(B, N, Hkv * G, D), k_new=r(B, N, Hkv, D), v_new=r(B, N, Hkv, D),
             k_cache=r(P, S, Hkv, D), v_cache=r(P, S, Hkv, D), parent=parent, n_nodes=nodes,
             cache_len=lens, table=table)
    if fill is not None:
        used = torch.zeros((P, S), dtype=torch.bool)
        for b in range(B):
            for t in range(int(lens[b])):
                used[b if table is None else int(table[b, t // S]), t % S] = True
        for name in ("k_cache", "v_cache"):
            c[name][~used] = fill
        for b in range(B):
            for name in ("q", "k_new", "v_new"):
                c[name][b, int(nodes[b]):] = fill
        if table is not None:  # pages that no position needs
            for b in range(B):
                table[b, -(-int(lens[b]) // S):] = 2 ** 31 - 1 if b % 2 else -1
    return c


def dev(a):
    return None if a is None else (a if torch.is_tensor(a) else torch.from_numpy(a)).cuda()


def run(c, **kw):
    d = {k: dev(v) for k, v in c.items()}
    plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                             page_table=d["table"])
    out, lse = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                      plan, page_table=d["table"], want_lse=True, **kw)
    torch.cuda.synchronize()
    assert plan.status.cpu().tolist() == [0] * c["q"].shape[0]
    return out.cpu().double(), lse.cpu().double()


def check(c, scale=None):
    out, lse = run(c, scale=scale)
    ref, rlse, mag, big = su.attention_ref(
        c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["parent"], c["n_nodes"],
        c["cache_len"], c["table"], scale)
    D, keys = c["q"].shape[3], int(c["cache_len"].max()) + c["q"].shape[1]
    tol = su.attention_tolerance(ref, mag, big, c["q"].dtype, D, keys)
    err = (out - ref).abs()
    assert bool((err <= tol).all()), (err / tol).max()
    # the total of up to `keys` weights in fp32, exponentials to 2^-21, scores as above
    ltol = (D + 4) * 2.0 ** -23 * big + 2.0 ** -18 + 2.0 ** -22 * rlse.abs().nan_to_num(0, 0, 0)
    seen = torch.isfinite(rlse)
    assert torch.equal(seen, torch.isfinite(lse)) and bool((lse[~seen] == -math.inf).all())
    assert bool(((lse - rlse).abs()[seen] <= ltol[seen]).all())
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [8, 40, 64, 80, 96, 128])
def test_head_sizes(D, dtype):
    check(make(3, 7, 2, 3, D, 16, 300, dtype, seed=D))


@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 1), (1, 128), (2, 7), (8, 5), (1, 71), (2, 16)])
def test_groups_of_heads(Hkv, G):
    check(make(2, 9, Hkv, G, 64, 32, 200, BF16, seed=Hkv * G))


@pytest.mark.parametrize("length", [0, 1, 2, 127, 128, 129, 255, 256, 257, 383, 1000])
@pytest.mark.parametrize("S", [0, 8, 128])
def test_lengths(length, S):
    """One token and a few nodes, over lengths at and around the tiles' ends."""
    check(make(2, 1, 2, 4, 64, S, 1000, BF16, seed=length, lens=[length], nodes=[1]))
    check(make(2, 6, 2, 4, 128, S, 1000, BF16, seed=length + 1, lens=[length, 5], nodes=[6, 3]))


@pytest.mark.parametrize("S", [8, 16, 32, 64, 128, 256, 384])
def test_page_sizes_with_anything_in_unused_places(S):
    """NaN and infinities past the lengths, in pages of nobody, in rows past n_nodes, and
    page numbers out of range where no position needs a page."""
    for fill in (math.nan, math.inf, -math.inf):
        c = make(4, 11, 2, 4, 64, S, 900, BF16, seed=S, fill=fill)
        clean = make(4, 11, 2, 4, 64, S, 900, BF16, seed=S, fill=0.0)
        out, lse = run(c)
        out2, lse2 = check(clean)
        assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("N,kind", [(1, "tree"), (2, "chain"), (31, "tree"), (32, "star"),
                                    (33, "chain"), (100, "tree"), (127, "star"), (128, "chain"),
                                    (129, "tree"), (300, "tree"), (520, "chain")])
def test_trees(N, kind):
    check(make(2, N, 1, 4, 64, 32, 260, BF16, seed=N, kind=kind, nodes=[N, max(1, N // 3)]))


def test_many_ragged_sequences():
    """More sequences than CTAs, zero lengths among them, and one long one."""
    lens = [0, 3, 128, 700, 1, 64, 0, 129, 5000, 17]
    check(make(203, 3, 1, 2, 64, 16, 5000, BF16, seed=5, lens=lens, nodes=[1, 3, 2]))


def test_one_long_sequence_is_split():
    check(make(1, 5, 2, 4, 128, 64, 40000, BF16, seed=6, lens=[39999], nodes=[5]))
    check(make(1, 1, 1, 1, 64, 0, 30001, FP16, seed=7, lens=[30001], nodes=[1]))


def test_sharp_and_growing_scores():
    """Scores far apart, rising along the sequence: the running maximum moves on
    every tile, and one key takes nearly all of the weight."""
    c = make(2, 4, 1, 4, 64, 32, 1500, BF16, seed=8, lens=[1500, 1111], nodes=[4])
    ramp = torch.linspace(0.0, 6.0, c["k_cache"].shape[0] * c["k_cache"].shape[1])
    c["k_cache"] = (c["k_cache"].float() * ramp.view(*c["k_cache"].shape[:2], 1, 1)).to(BF16)
    check(c, scale=1.0)
    c["k_cache"] = c["k_cache"].flip(0)
    check(c, scale=0.5)


def test_scores_of_minus_infinity_and_nan_rows():
    """A -inf key element gives weight 0 to the key; a NaN query makes its own row NaN only."""
    c = make(1, 3, 1, 2, 64, 16, 200, BF16, seed=9, lens=[200], nodes=[3])
    c["q"] = c["q"].abs() + 0.1
    clean = dict(c, k_cache=c["k_cache"].clone(), q=c["q"].clone())
    c["q"][0, 1, 0, 3] = math.nan
    out, _ = run(c)
    ref, _ = run(clean)
    assert torch.isnan(out[0, 1, 0]).all()
    out[0, 1, 0] = ref[0, 1, 0]
    assert torch.equal(out, ref)
    # every key in the cache at -inf: what is left are the new keys
    c = dict(clean, k_cache=torch.full_like(clean["k_cache"], -math.inf))
    out, lse = run(c)
    empty = dict(clean, cache_len=np.zeros(1, np.int32))
    ref, rlse = run(empty)
    torch.testing.assert_close(out, ref, rtol=2.0 ** -7, atol=2.0 ** -8)
    torch.testing.assert_close(lse, rlse, rtol=1e-5, atol=1e-5)


def test_nonfinite_new_values_reach_only_the_rows_that_see_them():
    """The value of one drafted node holds NaN and infinities: the node and its
    descendants get them, element by element; the others are as without."""
    N = 140
    c = make(1, N, 2, 2, 64, 16, 100, BF16, seed=10, lens=[77], nodes=[N], kind="tree")
    clean, _ = run(c)
    seen = {x: [n for n in range(N) if x in su.ancestors(c["parent"][0], n)] for x in (1, 130)}
    c["v_new"] = c["v_new"].clone()
    c["v_new"][0, 1, 0, 5] = math.nan
    c["v_new"][0, 1, 0, 6] = math.inf
    c["v_new"][0, 130, 1, 63] = -math.inf
    out, _ = run(c)
    want = clean.clone()
    want[0, seen[1], 0:2, 5] = math.nan
    want[0, seen[1], 0:2, 6] = math.inf
    want[0, seen[130], 2:4, 63] = -math.inf
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(0.0, 1e30, -1e30), want.nan_to_num(0.0, 1e30, -1e30))
    assert 1 < len(seen[1]) < N


def test_strided_views_and_layouts():
    """q, k and v as slices of one projection, a cache stored heads first, keys
    and values side by side in one tensor: bit-equal to contiguous copies."""
    c = make(3, 5, 4, 3, 64, 32, 300, BF16, seed=11)
    d = {k: dev(v) for k, v in c.items()}
    plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                             page_table=d["table"])
    want = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"], plan,
                                  page_table=d["table"])
    qkv = torch.cat([d["q"], d["k_new"], d["v_new"]], 2)
    q, k, v = qkv[:, :, :12], qkv[:, :, 12:16], qkv[:, :, 16:]
    heads_first = d["k_cache"].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
    both = torch.stack([d["k_cache"], d["v_cache"]], 1)
    for kc, vc in ((heads_first, d["v_cache"]), (both[:, 0], both[:, 1])):
        got = sv.spec_tree_attention(q, k, v, kc, vc, plan, page_table=d["table"])
        assert torch.equal(got, want)


def test_idle_and_bad_sequences():
    c = make(5, 6, 2, 2, 64, 16, 200, BF16, seed=12, lens=[100], nodes=[6, 0, 6, 6, 4])
    c["parent"][2, 3] = 3            # not below itself
    c["table"][3, 2] = 10 ** 6       # a page that does not exist
    d = {k: dev(v) for k, v in c.items()}
    plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                             page_table=d["table"])
    out, lse = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                      plan, page_table=d["table"], want_lse=True)
    assert plan.status.cpu().tolist() == [0, 0, -1, -1, 0]
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all())
    assert bool(torch.isnan(out[2:4]).all()) and bool(torch.isnan(lse[2:4]).all())
    keep = [0, 4]
    c2 = {k: (None if v is None else v[keep]) if k not in ("k_cache", "v_cache") else v
          for k, v in c.items()}
    want, _ = run(c2)
    torch.testing.assert_close(out.cpu().double()[keep], want, rtol=2.0 ** -6, atol=2.0 ** -8)


def test_repeats_are_bit_equal_and_other_streams_work():
    c = make(7, 9, 2, 4, 128, 64, 3000, BF16, seed=13)
    d = {k: dev(v) for k, v in c.items()}

    def once(stream=None):
        plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                                 page_table=d["table"], stream=stream)
        out = sv.spec_tree_attention(d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                     plan, page_table=d["table"], stream=stream)
        assert plan.read_status(stream) == sv.SPEC_DEV_OK
        return out
    want = once()
    for _ in range(5):
        assert torch.equal(once(), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = once(s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_graph_capture_follows_new_lengths():
    """A captured plan + attention + commit replays with the lengths of the moment."""
    c = make(4, 5, 2, 2, 64, 16, 400, BF16, seed=14, lens=[100, 7, 0, 300], nodes=[5])
    d = {k: dev(v) for k, v in c.items()}
    call = lambda: sv.spec_tree_attention(  # noqa: E731
        d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
        sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                          page_table=d["table"]), page_table=d["table"])
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for lens in ([100, 7, 0, 300], [1, 250, 128, 0]):
        d["cache_len"].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        got = out.clone()
        assert torch.equal(got, call())


# ------------------------------------------------------------------- plan

@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 64, 127, 128, 129, 255, 256, 1000, 1024])
@pytest.mark.parametrize("kind", ["tree", "chain", "star"])
def test_plan(N, kind):
    rng = np.random.default_rng(N)
    B, S, M, P = 6, 16, 20, 50
    parent = np.stack([su.random_tree(rng, N, kind) for _ in range(B)])
    nodes = rng.integers(0, N + 1, B).astype(np.int32)
    nodes[0] = N
    lens = rng.integers(0, M * S + 1, B).astype(np.int32)
    table = rng.integers(0, P, (B, M)).astype(np.int32)
    if N > 3:
        parent[1, 3], nodes[1] = 5, N       # an error
        nodes[2], parent[2, 3:] = 3, -9     # past the count: ignored
    nodes[3] = N + 1 if N % 2 else -1
    lens[4] = M * S + 1 if N % 2 else -5
    table[5, 0] = P
    got = sv.spec_tree_plan(dev(parent), dev(nodes), dev(lens),
                            torch.empty((P, S, 1, 8), dtype=BF16, device="cuda"),
                            page_table=dev(table))
    pos, status, mask = su.plan_ref(parent, nodes, lens, M * S, table, S, P)
    np.testing.assert_array_equal(got.status.cpu().numpy(), status)
    np.testing.assert_array_equal(got.positions.cpu().numpy(), pos)
    np.testing.assert_array_equal(got.mask.cpu().numpy().view(np.uint32), mask)


def test_plan_refill_and_empty_batch():
    c = make(3, 5, 1, 1, 64, 0, 100, BF16)
    d = {k: dev(v) for k, v in c.items()}
    plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"])
    d["cache_len"].zero_()
    same = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"], plan=plan)
    assert same is plan and int(plan.positions[:, 0].max()) == 0
    e = {k: (v[:0] if k not in ("k_cache", "v_cache") else v) for k, v in d.items()
         if v is not None}
    plan = sv.spec_tree_plan(e["parent"], e["n_nodes"], e["cache_len"], e["k_cache"])
    out = sv.spec_tree_attention(e["q"], e["k_new"], e["v_new"], e["k_cache"], e["v_cache"], plan)
    assert out.shape[0] == 0


# ----------------------------------------------------------------- commit

@pytest.mark.parametrize("dtype", [BF16, FP16, torch.float32])
@pytest.mark.parametrize("layers,B,N,H,D,S,tree", [
    (1, 1, 1, 1, 1, 0, False), (2, 5, 9, 3, 64, 16, True), (3, 4, 7, 2, 7, 5, True),
    (1, 3, 200, 1, 128, 32, False), (4, 2, 33, 2, 80, 1, True), (1, 40, 4, 8, 128, 64, True)])
def test_commit(dtype, layers, B, N, H, D, S, tree):
    rng = np.random.default_rng(N)
    gen = torch.Generator().manual_seed(N)
    cap = 4 * N + 7
    if S == 0:
        table, P, S = None, B + 1, cap
    else:
        M = -(-cap // S)
        P = B * M + 1
        table = rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32)
        cap = M * S
    r = lambda *s: torch.randn(s, generator=gen).to(dtype)  # noqa: E731
    kn, vn = r(layers, B, N, H, D), r(layers, B, N, H, D)
    kc, vc = r(layers, P, S, H, D), r(layers, P, S, H, D)
    lens = rng.integers(0, cap - N, B).astype(np.int32)
    acc = rng.integers(0, N, B).astype(np.int32)
    nodes = rng.integers(0, N, (B, N)).astype(np.int32) if tree else None
    if B >= 4:
        acc[0] = -1                        # an error of the verification
        lens[1], acc[1] = cap - 1, N - 1   # past the end
        if table is not None:
            table[2, lens[2] // S] = P     # no such page
        if tree:
            acc[3], nodes[3, 0] = max(1, N // 2), N
    wk, wv, wl = su.commit_ref(kn, vn, kc, vc, lens, acc, nodes, table)
    dk, dv = kc.cuda(), vc.cuda()
    got = sv.spec_tree_commit(kn.cuda(), vn.cuda(), dk, dv, dev(lens), dev(acc),
                              out_nodes=dev(nodes), page_table=dev(table))
    np.testing.assert_array_equal(got.cpu().numpy(), wl)
    assert torch.equal(dk.cpu(), wk) and torch.equal(dv.cpu(), wv)
    # one layer, from and to strided views
    if layers > 1:
        both = torch.cat([kc, vc], -1).cuda()
        new = torch.cat([vn, kn], -1).cuda()
        got = sv.spec_tree_commit(new[1, ..., D:], new[1, ..., :D], both[1, ..., :D],
                                  both[1, ..., D:], dev(lens), dev(acc), out_nodes=dev(nodes),
                                  page_table=dev(table))
        assert torch.equal(both[1, ..., :D].cpu(), wk[1])
        assert torch.equal(both[1, ..., D:].cpu(), wv[1])
        assert torch.equal(both[0].cpu(), torch.cat([kc, vc], -1)[0])


def test_commit_then_attention_equals_attention_over_the_tree():
    """A chain committed to the cache and one more node on it see what a chain of one more
    node sees before the commit."""
    c = make(3, 6, 2, 2, 64, 16, 300, BF16, seed=20, kind="chain", lens=[100, 15, 0], nodes=[6])
    whole, _ = run(c)
    d = {k: dev(v) for k, v in c.items()}
    acc = torch.full((3,), 4, dtype=torch.int32, device="cuda")
    length = sv.spec_tree_commit(d["k_new"], d["v_new"], d["k_cache"], d["v_cache"],
                                 d["cache_len"], acc, page_table=d["table"])
    assert length.cpu().tolist() == [105, 20, 5]
    one = lambda t: t[:, 5:6]  # noqa: E731
    root = torch.full((3, 1), -1, dtype=torch.int32, device="cuda")
    plan = sv.spec_tree_plan(root, torch.ones(3, dtype=torch.int32, device="cuda"), length,
                             d["k_cache"], page_table=d["table"])
    got = sv.spec_tree_attention(one(d["q"]), one(d["k_new"]), one(d["v_new"]), d["k_cache"],
                                 d["v_cache"], plan, page_table=d["table"])
    # the same weights in another order of tiles: a rounding each
    torch.testing.assert_close(got.cpu().double(), whole[:, 5:6], rtol=2.0 ** -6, atol=2.0 ** -7)
