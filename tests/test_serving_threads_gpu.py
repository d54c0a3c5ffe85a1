"""Host threads that plan and attend at once, on one stream, with the default workspaces."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import speculative_decoding_verification_65_gb300 as sv  # noqa: E402
from tests import serve_util as su  # noqa: E402
from tests.test_attn_gpu import BF16, dev, make  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# The first calls of a process: chains of some size, made by one or two threads at once.
CHILD = r"""
import sys, threading
import torch
import speculative_decoding_verification_65_gb300 as sv

def plan(N, stream=None):
    i32 = dict(dtype=torch.int32, device="cuda")
    with torch.cuda.stream(stream or torch.cuda.current_stream()):
        parent = torch.arange(-1, N - 1, **i32).view(1, N)
        made = sv.spec_tree_plan(parent, torch.full((1,), N, **i32), torch.zeros(1, **i32),
                                 torch.empty((1, 8, 1, 8), dtype=torch.bfloat16, device="cuda"))
        return made.positions.cpu()[0].tolist() == list(range(N)) and not int(made.status)

sizes, repeats = [int(n) for n in sys.argv[1].split(",")], int(sys.argv[2])
sv.library()
wrong = []
gate = threading.Barrier(len(sizes))
def work(N):
    stream = torch.cuda.Stream()
    gate.wait()
    for _ in range(repeats):
        try:
            if not plan(N, stream):
                wrong.append(N)
        except BaseException as e:
            wrong.append(repr(e))
threads = [threading.Thread(target=work, args=(n,)) for n in sizes]
for t in threads: t.start()
for t in threads: t.join()
print(wrong[:3])
sys.exit(1 if wrong else 0)
"""


@pytest.mark.parametrize("sizes,repeats", [("611", 1), ("612", 1), ("614", 1), ("620", 1),
                                           ("1024,700,640,1024", 1500)])
def test_plans_of_any_size_in_a_fresh_process(sizes, repeats):
    """Sizes at which the plan's shared memory passes 48 KB, and threads with several of them."""
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    run = subprocess.run([sys.executable, "-c", CHILD, sizes, str(repeats)], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout[-1000:] + run.stderr[-2000:]


def test_attention_from_threads_on_one_stream():
    """Threads, each with its own inputs, call on the same stream; what a call's first kernel
    leaves for its second is not the other thread's."""
    jobs = []
    for seed in range(4):
        c = make(2, 5, 2, 4, 64, 16, 4000, BF16, seed=seed, lens=[4000, 3000], nodes=[5])
        d = {k: dev(v) for k, v in c.items()}
        plan = sv.spec_tree_plan(d["parent"], d["n_nodes"], d["cache_len"], d["k_cache"],
                                 page_table=d["table"])
        args = (d["q"], d["k_new"], d["v_new"], d["k_cache"], d["v_cache"], plan, d["table"])
        jobs.append((args, sv.spec_tree_attention(*args)))
    torch.cuda.synchronize()
    gate, wrong = threading.Barrier(len(jobs)), []

    def work(i):
        args, want = jobs[i]
        gate.wait()
        outs = [sv.spec_tree_attention(*args) for _ in range(2000)]
        wrong.append(sum(not torch.equal(out, want) for out in outs))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
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
