"""The operators around prefill and beam search from several host threads on one stream, and in
graphs that run at once, with the default workspaces."""
import sys
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402

I32 = dict(dtype=torch.int32, device="cuda")


def chunk_job(seed, split=True):
    """One sequence whose keys several CTAs share out: what they leave is joined by a second kernel."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T, H, n = 40, 4, 9000 if split else 200
    q = torch.randn(T, 4 * H, 64, generator=gen, device="cuda").bfloat16()
    k, v = (torch.randn(1, n, H, 64, generator=gen, device="cuda").bfloat16() for _ in range(2))
    start, length = torch.tensor([0, T], **I32), torch.tensor([n - seed], **I32)

    def call(stream=None):
        plan = sv.spec_chunk_plan(start, length, q, k, stream=stream)
        return (sv.spec_chunk_attention(q, k, v, plan, stream=stream),)
    return call


def beam_job(seed):
    """Beams of equal rows: every order is open, so both kernels work."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(3, 1, 9001, generator=gen, device="cuda").expand(3, 5, 9001).contiguous()
    x[:, 1:, seed] -= 1e-3
    s = torch.full((3, 5), -1.0, device="cuda")
    return lambda stream=None: sv.spec_beam_select(x, s, 7, stream=stream)


def pages_job(seed):
    gen = torch.Generator().manual_seed(seed)
    table = torch.randperm(300, generator=gen)[:100].int().view(10, 10).cuda()
    length = torch.randint(60, 150, (10,), generator=gen).int().cuda()
    ref = torch.zeros(300, **I32)
    ref[table.flatten().long()] = 1
    parent = torch.randint(0, 10, (30,), generator=gen).int().cuda()

    def call(stream=None):
        forked = sv.spec_pages_fork(table, length, parent, ref, 16, stream=stream)
        return (*forked, *sv.spec_pages_compact(forked[0], forked[2], 16, stream=stream))
    return call


@pytest.mark.parametrize("job", [chunk_job, beam_job, pages_job])
def test_threads_on_one_stream(job):
    jobs = [(call, call()) for call in map(job, range(4))]
    torch.cuda.synchronize()
    gate, wrong = threading.Barrier(len(jobs)), []

    def work(call, want):
        gate.wait()
        outs = [call() for _ in range(400)]
        wrong.append(sum(not torch.equal(a, b) for out in outs for a, b in zip(out, want)))
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    assert wrong == [0] * len(jobs)


@pytest.mark.parametrize("job", [chunk_job, beam_job, pages_job])
def test_two_graphs_at_once(job):
    """Graphs captured on one stream have workspaces of their own: replayed on two streams, they
    run side by side, and beside eager calls."""
    calls = [job(seed) for seed in range(3)]
    want = [call() for call in calls]
    graphs, outs = [], []
    for call in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(20):
        for out in outs:
            for x in out:
                x.fill_(77)
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            eager = calls[2]()
        torch.cuda.synchronize()
        for got, ref in zip([*outs, eager], want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("job", [chunk_job, beam_job, pages_job])
def test_a_stream_that_is_not_the_current_one(job):
    call = job(1)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [call(stream=side) for _ in range(3)]
    side.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_small_and_large_calls_take_turns():
    """One thread's workspaces grow and are used again by smaller calls."""
    calls = [chunk_job(1), chunk_job(2, split=False), beam_job(3), pages_job(4), chunk_job(5)]
    want = [call() for call in calls]
    for _ in range(10):
        for call, ref in zip(reversed(calls), reversed(want)):
            assert all(np.array_equal(a.float().cpu().numpy(), b.float().cpu().numpy())
                       for a, b in zip(call(), ref))
