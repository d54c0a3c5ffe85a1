"""Forks, copies and compaction of a cache's pages on a GPU against row-by-row
restatements (prefill_util.py).  Everything is whole numbers and copies: equal."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import prefill_util as pu  # noqa: E402


def cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def fork(table, length, parent, ref, S, reserve=None, **kw):
    got = sv.spec_pages_fork(cuda(table), cuda(length), cuda(parent), cuda(ref), S,
                             reserve=None if reserve is None else cuda(reserve), **kw)
    return [x.cpu().numpy() for x in got]


def check_fork(*a):
    want = pu.fork_ref(*a)
    got = fork(*a)
    for name, x, y in zip(("table", "length", "ref", "copies"), got, want):
        assert np.array_equal(x, y), (name, x, y)
    return got


def pool(seed, R, M, S, P, others=0.1):
    """Random rows over a pool, prefixes shared by neighbours, and other owners' pages."""
    rng = np.random.default_rng(seed)
    free = list(rng.permutation(P))
    ref = np.zeros(P, np.int32)
    table, length = np.full((R, M), -1, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        held = int(rng.integers(0, M + 1))
        both = int(rng.integers(0, held + 1)) if r and rng.random() < 0.7 else 0
        both = min(both, int((table[r - 1] >= 0).sum()))
        row = list(table[r - 1, :both])
        while len(row) < held and len(free) > P // 3:
            row.append(free.pop())
        table[r, :len(row)] = row
        ref[row] += 1
        length[r] = rng.integers(0, len(row) * S + 1)
    for p in free[:int(others * P)]:
        ref[p] = 1 + p % 3
    return table, length, ref, rng


@pytest.mark.parametrize("R,M,S,P", [(1, 1, 1, 3), (4, 6, 16, 60), (9, 40, 8, 900), (30, 33, 5, 5000),
                                     (200, 20, 64, 9000), (3, 100, 1, 400)])
@pytest.mark.parametrize("seed", range(3))
def test_fork(R, M, S, P, seed):
    table, length, ref, rng = pool(seed, R, M, S, P)
    for R1 in (R, 1, 2 * R + 3):
        parent = rng.integers(-1, R, R1)
        reserve = rng.integers(0, 2 * S + 2, R1)
        check_fork(table, length, parent, ref, S, reserve)
    check_fork(table, length, rng.integers(-1, R, R), ref, S)


def test_identity_keeps_everything_that_is_not_shared():
    table, length, ref, _ = pool(5, 6, 8, 16, 100)
    table[3] = -1
    ref[:] = 0
    for e in table[table >= 0]:
        ref[e] += 1
    got = check_fork(table, length, np.arange(6), ref, 16)
    for r in range(6):
        n = int(length[r]) // 16
        assert np.array_equal(got[0][r, :n], table[r, :n])


def test_dropping_all_frees_all():
    table, length, ref, _ = pool(6, 12, 10, 16, 200, others=0)
    got = check_fork(table, length, np.full(4, -1), ref, 16)
    assert (got[2] == 0).all() and (got[1] == 0).all()
    got = fork(table, length, np.zeros(0), ref, 16)
    assert (got[2] == 0).all()


def test_not_enough_pages_changes_nothing():
    table, length, ref, _ = pool(7, 5, 10, 16, 60)
    ref[ref == 0] = 1
    want = ref.copy()
    got = check_fork(table, length, np.arange(5), ref, 16, np.full(5, 40))
    assert np.array_equal(got[2], want) and (got[1] == -1).all() and (got[0] == -1).all()


def test_errors():
    table, length, ref, _ = pool(8, 8, 10, 16, 300)
    length[:] = np.minimum(length, 60)
    table[2, 0], length[2] = 300, 5              # no such page
    length[3] = 161                              # longer than a row
    length[4] = (table[4] >= 0).sum() * 16 + 1   # longer than its pages
    parent = np.array([0, 8, -2, 2, 3, 4, 1, 1, 0, 5, -1])
    reserve = np.array([0, 0, 0, 0, 0, 0, 101, -1, 160, 3, 9])
    got = check_fork(table, length, parent, ref, 16, reserve)
    assert list(got[1][1:6]) == [-1] * 5 and got[1][7] == -1 and got[1][10] == 0


def test_a_pool_of_many_blocks():
    """The free pages lie at the end of a pool of a million, few at a time."""
    P = 1 << 20
    ref = np.ones(P, np.int32)
    free = np.sort(np.random.default_rng(1).permutation(P)[:50])
    ref[free] = 0
    table = np.full((3, 64), -1, np.int32)
    got = fork(table, np.zeros(3), np.arange(3), ref, 16, np.array([160, 320, 240]))
    assert np.array_equal(got[0][got[0] >= 0], free[:45])
    assert int(got[2].sum()) == P - 5


@pytest.mark.parametrize("R,M,S,P", [(1, 1, 1, 1), (4, 6, 16, 61), (30, 33, 5, 5000),
                                     (200, 20, 64, 9000), (3, 10, 8, 4096), (0, 5, 8, 100)])
@pytest.mark.parametrize("seed", range(2))
def test_compact(R, M, S, P, seed):
    table, _, ref, _ = pool(seed, R, M, S, P)
    want = pu.compact_ref(table, ref, S)
    got = sv.spec_pages_compact(cuda(table), cuda(ref), S)
    for x, y in zip(got[:3], want[:3]):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(got[3]) == want[3]


@pytest.mark.parametrize("value", [0, 1])
def test_compact_of_an_empty_or_a_full_pool(value):
    ref = np.full(8192, value, np.int32)
    table = np.arange(8192).reshape(64, 128) if value else np.full((64, 128), -1)
    got = sv.spec_pages_compact(cuda(table), cuda(ref), 16)
    assert np.array_equal(got[0].cpu().numpy(), table) and np.array_equal(got[1].cpu().numpy(), ref)
    assert bool((got[2][:2] == -1).all()) and int(got[3]) == 8192 * value


@pytest.mark.parametrize("layers,S,H,D,dtype", [
    (None, 16, 2, 64, torch.bfloat16), (3, 5, 3, 7, torch.float16), (2, 1, 1, 1, torch.float32),
    (2, 256, 8, 128, torch.bfloat16), (4, 33, 2, 10, torch.float32)])
@pytest.mark.parametrize("strided", [False, True])
def test_copy(layers, S, H, D, dtype, strided):
    gen = torch.Generator().manual_seed(2)
    shape = (layers or 1, 40, S, H, D)
    if strided:
        k, v = (torch.randn((shape[0], 40, H, S, D + 2), generator=gen).to(dtype).cuda()
                .transpose(2, 3)[..., :D] for _ in range(2))
    else:
        k, v = (torch.randn(shape, generator=gen).to(dtype).cuda() for _ in range(2))
    copies = torch.tensor([[3, -1, 7, 3, 0, 5, 40, 8], [11, 12, 13, 14, -1, 40, 15, 16],
                           [S, S, 1, S - 1, S, S, S, S + 1]], dtype=torch.int32, device="cuda")
    wk, wv = k.clone(), v.clone()
    for w in (wk, wv):
        w[:, 11, :S] = w[:, 3, :S]
        w[:, 13, :1] = w[:, 7, :1]
        w[:, 14, :S - 1] = w[:, 3, :S - 1]
    sv.spec_pages_copy(*((k, v) if layers else (k[0], v[0])), copies)
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_copy_of_a_long_list():
    """Most entries copy nothing; the others lie anywhere in the list."""
    P, n = 3000, 20000
    rng = np.random.default_rng(3)
    pages = rng.permutation(P)
    copies = np.full((3, n), -1, np.int32)
    copies[2] = 0
    at = np.sort(rng.permutation(n)[:1000])
    copies[0, at], copies[1, at], copies[2, at] = pages[:1000], pages[1000:2000], 8
    k = torch.randn(2, P, 8, 1, 32, device="cuda")
    v = torch.randn(2, P, 8, 1, 32, device="cuda")
    wk, wv = k.clone(), v.clone()
    src, dst = cuda(pages[:1000]).long(), cuda(pages[1000:2000]).long()
    wk[:, dst], wv[:, dst] = wk[:, src], wv[:, src]
    sv.spec_pages_copy(k, v, cuda(copies))
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_a_life_of_a_pool():
    """Rows grow, fork, die and are compacted; what the rows hold never changes, each page has
    as many references as table entries, and nothing is lost."""
    S, M, P, R = 4, 12, 200, 8
    rng = np.random.default_rng(9)
    table = torch.full((R, M), -1, dtype=torch.int32, device="cuda")
    length = torch.zeros(R, dtype=torch.int32, device="cuda")
    ref = torch.zeros(P, dtype=torch.int32, device="cuda")
    k = torch.zeros(1, P, S, 1, 2, device="cuda")
    v = torch.zeros_like(k)
    texts, stamp = [[] for _ in range(R)], 0.0
    for step in range(40):
        parent = rng.integers(0, R, R)
        parent[rng.random(R) < 0.15] = -1
        grow = rng.integers(0, 4, R)
        texts = [list(texts[p]) if p >= 0 else [] for p in parent]
        grow = np.array([g if len(t) + g <= S * M else 0 for g, t in zip(grow, texts)])
        if max(map(len, texts)) > S * (M - 1):
            parent[:], grow[:], texts = -1, 0, [[] for _ in range(R)]
        table, length, ref, copies = sv.spec_pages_fork(table, length, cuda(parent), ref, S,
                                                        reserve=cuda(grow))
        sv.spec_pages_copy(k, v, copies)
        assert length.tolist() == [len(t) for t in texts]
        start = np.concatenate([[0], np.cumsum(grow)])
        new = torch.arange(start[-1], device="cuda").float() + stamp + 1
        stamp += float(start[-1])
        rows = torch.stack([new, -new], 1)[:, None, :].contiguous()
        for r in range(R):
            texts[r] += new[start[r]:start[r + 1]].tolist()
        if start[-1]:
            length = sv.spec_chunk_append(rows, 2 * rows, k[0], v[0], cuda(start), length,
                                          page_table=table)
        if step % 7 == 6:
            table, ref, copies, used = sv.spec_pages_compact(table, ref, S)
            sv.spec_pages_copy(k, v, copies)
            assert bool((ref[:int(used)] > 0).all()) and int(ref[int(used):].sum()) == 0
        t = table.cpu().numpy()
        assert np.array_equal(np.bincount(t[t >= 0], minlength=P), ref.cpu().numpy())
        for r in range(R):
            n = len(texts[r])
            at = torch.arange(n, device="cuda")
            got = k[0, table[r].long()[at // S], at % S, 0]
            assert got[:, 0].tolist() == texts[r] and got[:, 1].tolist() == [-x for x in texts[r]]
            assert v[0, table[r].long()[at // S], at % S, 0, 0].tolist() == [2 * x for x in texts[r]]


@pytest.mark.parametrize("P", [300, 4096, 4097])
@pytest.mark.parametrize("R0,R1", [(16, 16), (17, 16), (16, 17), (2, 16)])
def test_fork_by_one_cta_or_several(R0, R1, P):
    """Around the sizes up to which one CTA does it all."""
    table, length, ref, rng = pool(R0 + R1, R0, 9, 8, P)
    for _ in range(3):
        check_fork(table, length, rng.integers(-1, R0, R1), ref, 8, rng.integers(0, 17, R1))


@pytest.mark.parametrize("R,M", [(64, 64), (241, 17)])
@pytest.mark.parametrize("P", [4096, 4097])
def test_compact_by_one_cta_or_several(R, M, P):
    table, _, ref, _ = pool(R, R, M, 4, P)
    want = pu.compact_ref(table, ref, 4)
    got = sv.spec_pages_compact(cuda(table), cuda(ref), 4)
    for x, y in zip(got[:3], want[:3]):
        assert np.array_equal(x.cpu().numpy(), y)
    assert int(got[3]) == want[3]


def test_fork_without_pages():
    """A pool of no pages has rows of no tokens only."""
    none = np.zeros(0, np.int32)
    got = fork(np.zeros((0, 3)), none, [-1, -1], none, 4)
    assert (got[0] == -1).all() and got[1].tolist() == [0, 0] and got[3].tolist() == [[-1] * 2] * 2 + [[0] * 2]
    got = fork(np.zeros((0, 3)), none, [-1, -1], none, 4, reserve=np.array([1, 0]))
    assert (got[0] == -1).all() and got[1].tolist() == [-1, -1]
