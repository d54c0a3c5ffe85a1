"""The serving operators around speculative verification, with plain forms.

A decoding step with drafted tokens runs, for each batch of sequences:

  plan     ancestors and positions of every sequence's tree of drafted tokens
  attn     (each layer) attention of all tree nodes over a paged or contiguous
           key/value cache and over their ancestors among the new tokens; the
           plan is part of the pass, as in a step's first layer
  logits   penalties for repeated tokens, biases and grammar masks on the rows
           that the verification reads next
  commit   keys and values of the accepted path appended to the cache

A node's parent has a lower index, node 0 is the root (the last committed
token, not in the cache yet), and a chain of k drafts is the tree
parent[n] = n - 1 with k + 1 nodes.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one small batch of 11-node trees: what a short step pays for its plan
        dict(name="plan B8 N11", op="plan", B=8, N=11, shape="tree", L=4096, S=16),
        # a full serving batch of wide trees
        dict(name="plan B512 N256", op="plan", B=512, N=256, shape="tree", L=8192, S=64),
        # plain decoding of one sequence, one token, no drafts: latency counts
        dict(name="attn B1 N1 L4096", op="attn", B=1, N=1, shape="chain", Hkv=8, G=4, D=128,
             L=4096, S=16, dtype="bf16"),
        # chains of 4 drafts with a group size that divides no tile
        dict(name="attn B32 N5 L2048 D64", op="attn", B=32, N=5, shape="chain", Hkv=4, G=7, D=64,
             L=2048, S=64, dtype="fp16"),
        # 29-node trees over an ordinary context: a serving batch
        dict(name="attn B64 N29 L8192", op="attn", B=64, N=29, shape="tree", Hkv=8, G=4, D=128,
             L=8192, S=64, dtype="bf16"),
        # wide trees for few sequences over one contiguous cache: product-bound
        dict(name="attn B4 N256 L16384", op="attn", B=4, N=256, shape="tree", Hkv=8, G=8, D=128,
             L=16384, S=0, dtype="bf16"),
        # chains of 8 drafts over very long contexts
        dict(name="attn B8 N9 L131072", op="attn", B=8, N=9, shape="chain", Hkv=8, G=5, D=128,
             L=131072, S=256, dtype="bf16"),
        # one sequence constrained by a grammar, 4 drafts
        dict(name="logits B1 R5 V32000", op="logits", B=1, R=5, V=32000, dtype="bf16", hist=1000,
             shape="chain", bias=16, mask=True),
        # the fp32 verification batch with 8 drafts, long histories
        dict(name="logits B256 R9 V151936", op="logits", B=256, R=9, V=151936, dtype="f32",
             hist=8192, shape="chain", bias=0, mask=False),
        # trees under a grammar mask for every node
        dict(name="logits B64 N29 V128256", op="logits", B=64, R=29, V=128256, dtype="bf16",
             hist=2048, shape="tree", bias=64, mask=True),
        # one layer's cache after a tree was verified
        dict(name="commit 1 layer B64 N29", op="commit", layers=1, B=64, N=29, shape="tree",
             Hkv=8, D=128, L=4096, S=64, dtype="bf16"),
        # every layer's cache at the end of a step
        dict(name="commit 32 layers B32 N29", op="commit", layers=32, B=32, N=29, shape="tree",
             Hkv=8, D=128, L=512, S=32, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "attn", "attn", "attn", "logits", "logits", "commit"])
    shape = rng.choice(["tree", "chain"])
    S = rng.choice([0, 8, 16, 32, 64, 128, 256])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 512), N=_log(rng, 1, 256), shape=shape,
                    L=_log(rng, 256, 16384), S=S)
    if op == "attn":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        D = rng.choice([64, 64, 80, 96, 128, 128, 128])
        N, L = _log(rng, 1, 256), _log(rng, 64, 131072)
        most = min(256, (1 << 30) // (L * Hkv * D), int(5.5e11 / (4.0 * Hkv * G * N * L * D)))
        return dict(op=op, B=_log(rng, 1, max(1, most)), N=N, shape=shape, Hkv=Hkv, G=G, D=D, L=L,
                    S=S, dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "logits":
        V, R, dtype = _log(rng, 1000, 160000), _log(rng, 1, 40), rng.choice(["bf16", "f32"])
        most = min(512, int(1.4e9 / (V * R * SIZE[dtype])))
        return dict(op=op, B=_log(rng, 1, max(1, most)), R=R, V=V, dtype=dtype,
                    hist=_log(rng, 1, 8192), shape=shape, bias=rng.choice([0, 5, 64, 300]),
                    mask=rng.random() < 0.5)
    layers, Hkv, D = _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 80, 96, 128])
    L = _log(rng, 64, 4096)
    most = min(256, (1 << 29) // (layers * L * Hkv * D))
    return dict(op=op, layers=layers, B=_log(rng, 1, max(1, most)), N=_log(rng, 1, 64),
                shape=shape, Hkv=Hkv, D=D, L=L, S=S, dtype=rng.choice(["bf16", "fp16", "f32"]))


# ------------------------------------------------------------------ inputs

def _trees(B, N, shape, rng):
    """Parents [B, N] and node counts [B]: chains, or trees whose node n hangs
    below a random earlier node; entries past a sequence's count are -1."""
    n = np.arange(N)
    if shape == "chain":
        parent = np.tile(n - 1, (B, 1))
    else:
        parent = np.floor(rng.random((B, N)) * n).astype(np.int64)
    parent[:, 0] = -1
    count = rng.integers((N + 1) // 2, N + 1, size=B)
    parent[n[None, :] >= count[:, None]] = -1
    return parent.astype(np.int32), count.astype(np.int32)


def _pages(B, L, S, rng):
    """A page table over shuffled pages with a few that no sequence owns, the
    number of pages, and the page size. S = 0: one contiguous run per sequence."""
    if S == 0:
        return None, B, L
    M = -(-L // S)
    P = B * M + 3
    return rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32), P, S


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=dtype) * scale
            if scale != 1.0 else torch.randn(shape, generator=gen, device="cuda", dtype=dtype))


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": c}
    if c["op"] in ("plan", "attn", "commit"):
        B, N, L = c["B"], c["N"], c["L"]
        parent, count = _trees(B, N, c["shape"], rng)
        table, P, S = _pages(B, L, c["S"], rng)
        cap = L if table is None else table.shape[1] * S
        high = max(0, cap - N)
        cache_len = rng.integers(high // 2, high + 1, size=B).astype(np.int32)
        st.update(parent=_dev(parent), n_nodes=_dev(count), cache_len=_dev(cache_len),
                  table=_dev(table))
    if c["op"] == "plan":
        # the cache is only asked for its geometry here
        st["k_cache"] = torch.empty((P, S, 1, 8), dtype=torch.bfloat16, device="cuda")
    elif c["op"] == "attn":
        dt, H, G, D = DTYPES[c["dtype"]], c["Hkv"], c["G"], c["D"]
        # queries, new keys and new values as slices of one projection
        qkv = _normal(gen, (B, N, (G + 2) * H, D), dt)
        st["q"], st["k_new"], st["v_new"] = (qkv[:, :, :G * H], qkv[:, :, G * H:(G + 1) * H],
                                             qkv[:, :, (G + 1) * H:])
        st["k_cache"] = _normal(gen, (P, S, H, D), dt)
        st["v_cache"] = _normal(gen, (P, S, H, D), dt)
    elif c["op"] == "commit":
        dt, H, D, layers = DTYPES[c["dtype"]], c["Hkv"], c["D"], c["layers"]
        st["k_new"] = _normal(gen, (layers, B, N, H, D), dt)
        st["v_new"] = _normal(gen, (layers, B, N, H, D), dt)
        st["k_cache"] = _normal(gen, (layers, P, S, H, D), dt)
        st["v_cache"] = _normal(gen, (layers, P, S, H, D), dt)
        # the verification's answer: a path from the root to some node
        nodes = np.full((B, N), -1, np.int32)
        accepted = np.zeros(B, np.int32)
        for b in range(B):
            path, n = [], int(rng.integers(0, count[b]))
            while n > 0:
                path.append(n)
                n = int(parent[b, n])
            accepted[b] = len(path)
            nodes[b, :len(path)] = path[::-1]
        st["accepted"] = _dev(accepted)
        st["nodes"] = _dev(nodes) if c["shape"] == "tree" else None
    elif c["op"] == "logits":
        B, R, V, hist = c["B"], c["R"], c["V"], c["hist"]
        st["logits"] = _normal(gen, (B, R, V), DTYPES[c["dtype"]], 3.0)
        # frequent tokens repeat, as in text
        word = lambda *shape: np.minimum(V - 1, V ** rng.random(shape) - 1).astype(np.int32)  # noqa: E731
        length = rng.integers(0, hist + 1, size=B).astype(np.int32)
        st.update(history=_dev(word(B, hist)), history_len=_dev(length),
                  prompt_len=_dev((rng.random(B) * (length + 1)).astype(np.int32)))
        if c["shape"] == "tree":
            parent, count = _trees(B, R, "tree", rng)
            parent = np.where(parent < 0, 0, parent)  # every row of this batch is a node
            tokens = word(B, R)
            tokens[:, 0] = -1
            st.update(parent=_dev(parent.astype(np.int32)), tokens=_dev(tokens))
        else:
            st.update(parent=None, tokens=_dev(word(B, R - 1)))
        some = rng.random((3, B)).astype(np.float32) * (rng.random((3, B)) < 0.8)
        st.update(repetition=_dev((1 + 0.3 * some[0]).astype(np.float32)),
                  frequency=_dev((0.5 * some[1]).astype(np.float32)),
                  presence=_dev((0.5 * some[2]).astype(np.float32)))
        st["bias_tokens"] = st["bias_values"] = st["allowed"] = None
        if c["bias"]:
            M = c["bias"]
            step = V // M
            bt = (np.arange(M) * step + rng.integers(0, step, size=(B, M))).astype(np.int32)
            bt[rng.random((B, M)) < 0.1] = -1  # unused entries
            st["bias_tokens"] = _dev(bt)
            st["bias_values"] = _dev(rng.normal(0, 4, size=(B, M)).astype(np.float32))
        if c["mask"]:
            W = -(-V // 32)
            words = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=gen, device="cuda",
                                  dtype=torch.int64).to(torch.int32)
            # half of the positions are free text
            free = torch.rand((B, R, 1), generator=gen, device="cuda") < 0.5
            st["allowed"] = torch.where(free, torch.full_like(words, -1), words)
    return st


# ------------------------------------------------------------- plain forms

def _reach(parent, n_nodes):
    """[B, N, N] bool: node j is node n or one of its ancestors; no row or
    column past a sequence's count."""
    B, N = parent.shape
    n = torch.arange(N, device=parent.device)
    live = n < n_nodes[:, None]
    edge = (parent.clamp(min=0)[:, :, None] == n) & (n > 0)[:, None] & live[:, :, None]
    r = (edge | torch.eye(N, dtype=torch.bool, device=parent.device)).float()
    for _ in range(max(1, N - 1).bit_length()):  # paths of up to 1, 2, 4, ... edges
        r = ((r @ r) > 0).float()
    return (r > 0) & live[:, :, None] & live[:, None, :]


def _bits(b):
    """Booleans [..., n] as int32 words, bit j of word w for entry 32 w + j."""
    w = b.reshape(*b.shape[:-1], -1, 32).to(torch.int64)
    return (w << torch.arange(32, device=b.device)).sum(-1).to(torch.int32)


def _plan_plain(st):
    reach = _reach(st["parent"], st["n_nodes"])
    N = reach.shape[1]
    live = torch.arange(N, device=reach.device) < st["n_nodes"][:, None]
    depth = reach.sum(-1).to(torch.int32) - 1
    positions = torch.where(live, st["cache_len"][:, None] + depth, -1).to(torch.int32)
    mask = _bits(torch.nn.functional.pad(reach, (0, -N % 128)))
    return {"positions": positions, "mask": mask, "status": torch.zeros_like(st["n_nodes"])}


def _run_of(cache, table, kind):
    """[B, H, L, D] of a sequence's cache slots in order."""
    rows = cache if table is None else cache[table.long()].flatten(1, 2)
    return rows.transpose(1, 2).to(kind)


def _attn_plain(st, kind=torch.float32):
    q, c = st["q"], st["case"]
    B, N, Hq, D = q.shape
    H, G = c["Hkv"], c["G"]
    k = torch.cat([_run_of(st["k_cache"], st["table"], kind),
                   st["k_new"].transpose(1, 2).to(kind)], 2)
    s = q.to(kind).reshape(B, N, H, G, D).transpose(1, 2).reshape(B, H, N * G, D)
    s = (s @ k.transpose(2, 3)) * D ** -0.5
    del k
    L = s.shape[3] - N
    past = torch.arange(L, device=q.device) < st["cache_len"][:, None]
    seen = torch.cat([past[:, None, :].expand(B, N, L), _reach(st["parent"], st["n_nodes"])], 2)
    seen = seen[:, None, :, None, :].expand(B, H, N, G, L + N).reshape(B, H, N * G, L + N)
    s = s.masked_fill(~seen, -math.inf)
    del seen
    m = s.amax(-1, keepdim=True)
    p = (s - m.masked_fill(m == -math.inf, 0.0)).exp()
    del s
    total = p.sum(-1, keepdim=True)
    v = torch.cat([_run_of(st["v_cache"], st["table"], kind),
                   st["v_new"].transpose(1, 2).to(kind)], 2)
    o = (p @ v) / total.clamp(min=1e-30)
    o = o.reshape(B, H, N, G, D).transpose(1, 2).reshape(B, N, Hq, D)
    live = torch.arange(N, device=q.device) < st["n_nodes"][:, None]
    return o.masked_fill(~live[:, :, None, None], 0.0).to(q.dtype)


def _logits_plain(st):
    x = st["logits"].float()
    B, R, V = x.shape
    dev = x.device
    i = torch.arange(st["history"].shape[1], device=dev)
    inside = i < st["history_len"][:, None]
    written = inside & (i >= st["prompt_len"][:, None])
    where = st["history"].long()
    any_ = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, where, inside.int())
    out = torch.zeros((B, V), dtype=torch.int32, device=dev).scatter_add_(1, where, written.int())
    if st["parent"] is None:
        path = torch.arange(R - 1, device=dev) < torch.arange(R, device=dev)[:, None]
        path = path.expand(B, R, R - 1)
    else:
        path = _reach(st["parent"], torch.full((B,), R, device=dev))
        path = path & (torch.arange(R, device=dev) > 0)
    tokens = st["tokens"].clamp(min=0).long()[:, None, :].expand(path.shape)
    drafted = torch.zeros((B, R, V), dtype=torch.int32, device=dev)
    drafted.scatter_add_(2, tokens, path.int())
    count = drafted + out[:, None, :]
    seen = (drafted + any_[:, None, :]) > 0
    per = lambda name: st[name][:, None, None]  # noqa: E731
    x = torch.where(seen, torch.where(x > 0, x / per("repetition"), x * per("repetition")), x)
    x = x - per("frequency") * count - per("presence") * (count > 0)
    if st["bias_tokens"] is not None:
        bt = st["bias_tokens"]
        add = torch.zeros((B, V), device=dev)
        add.scatter_add_(1, bt.clamp(min=0).long(), st["bias_values"] * (bt >= 0))
        x = x + add[:, None, :]
    if st["allowed"] is not None:
        j = torch.arange(V, device=dev)
        bit = (st["allowed"][:, :, j // 32] >> (j % 32).int()) & 1
        x = x.masked_fill(bit == 0, -math.inf)
    return x.to(st["logits"].dtype)


def _commit_plain(st):
    N = st["k_new"].shape[2]
    n = torch.arange(N, device="cuda")
    take = n <= st["accepted"][:, None]
    b, i = take.nonzero(as_tuple=True)
    node = i if st["nodes"] is None else torch.where(i == 0, 0, st["nodes"][b, (i - 1).clamp(min=0)].long())
    at = st["cache_len"][b].long() + i
    S = st["k_cache"].shape[2]
    page = b if st["table"] is None else st["table"][b, at // S].long()
    st["k_cache"][:, page, at % S] = st["k_new"][:, b, node]
    st["v_cache"][:, page, at % S] = st["v_new"][:, b, node]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"],
            "cache_len": st["cache_len"] + st["accepted"] + 1}


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import speculative_decoding_verification_65_gb300 as sv
        if op == "plan":
            plan = sv.spec_tree_plan(st["parent"], st["n_nodes"], st["cache_len"], st["k_cache"],
                                     page_table=st["table"])
            return {"positions": plan.positions, "mask": plan.mask, "status": plan.status}
        if op == "attn":
            plan = sv.spec_tree_plan(st["parent"], st["n_nodes"], st["cache_len"], st["k_cache"],
                                     page_table=st["table"])
            return sv.spec_tree_attention(st["q"], st["k_new"], st["v_new"], st["k_cache"],
                                          st["v_cache"], plan, page_table=st["table"])
        if op == "logits":
            return sv.spec_process_logits(
                st["logits"], history=st["history"], history_len=st["history_len"],
                prompt_len=st["prompt_len"], draft_tokens=st["tokens"], parent=st["parent"],
                repetition=st["repetition"], frequency=st["frequency"], presence=st["presence"],
                bias_tokens=st["bias_tokens"], bias_values=st["bias_values"],
                allowed=st["allowed"])
        length = sv.spec_tree_commit(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                                     st["cache_len"], st["accepted"], out_nodes=st["nodes"],
                                     page_table=st["table"])
        return {"k_cache": st["k_cache"], "v_cache": st["v_cache"], "cache_len": length}
    if op == "plan":
        return _plan_plain(st)
    if op == "attn":
        return _attn_plain(st)
    if op == "logits":
        return _logits_plain(st)
    return _commit_plain(st)


# ------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass at the mean of its ragged sizes."""
    c = case
    B = c["B"]
    if c["op"] == "plan":
        N = c["N"]
        M = -(-c["L"] // c["S"]) * 3 // 4 if c["S"] else 0
        return {"bytes": B * (8.0 + 4 * N * 2 + 16 * N * -(-N // 128) + 4 * M + 4), "flops": 0.0}
    if c["op"] == "attn":
        cap = c["L"] if not c["S"] else -(-c["L"] // c["S"]) * c["S"]
        past = max(0, cap - c["N"]) * 0.75
        nodes = (c["N"] + (c["N"] + 1) // 2) / 2
        size, H, G, D = SIZE[c["dtype"]], c["Hkv"], c["G"], c["D"]
        moved = B * H * D * size * (2 * past + nodes * (2 + G) + c["N"] * G)
        return {"bytes": moved, "flops": 4.0 * B * H * G * D * nodes * (past + nodes / 2)}
    if c["op"] == "logits":
        cells = float(B) * c["R"] * c["V"]
        moved = 2 * cells * SIZE[c["dtype"]] + (cells / 8 if c["mask"] else 0)
        return {"bytes": moved + B * (2.0 * c["hist"] + 4 * c["R"] + 8 * c["bias"] + 20),
                "flops": 3 * cells}
    # a path to a random node: about the logarithm of the tree, half of a chain
    nodes = (c["N"] + (c["N"] + 1) // 2) / 2
    path = 1 + (math.log(max(1.0, nodes)) if c["shape"] == "tree" else nodes / 2)
    return {"bytes": 4.0 * c["layers"] * B * path * c["Hkv"] * c["D"] * SIZE[c["dtype"]] + 12 * B,
            "flops": 0.0}


# ------------------------------------------------- definitions in 64 bits

def _path_nodes(parent, n):
    path = []
    while n >= 0:
        path.append(n)
        n = int(parent[n]) if n > 0 else -1
    return path


def _attn_exact(st):
    """softmax(q k^T / sqrt(D)) v over the keys that a node sees, one sequence
    and one head of keys at a time."""
    q, c = st["q"], st["case"]
    B, N, Hq, D = q.shape
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64, device=q.device)
    parent, count = st["parent"].cpu().numpy(), st["n_nodes"].tolist()
    for b in range(B):
        n, length = count[b], int(st["cache_len"][b])
        hidden = torch.ones((n, length + n), dtype=torch.bool)
        hidden[:, :length] = False
        for i in range(n):
            hidden[i, [length + j for j in _path_nodes(parent[b], i)]] = False
        hidden = hidden.cuda()
        if st["table"] is None:
            pages = torch.full((length,), b, device=q.device)
            slots = torch.arange(length, device=q.device)
        else:
            S = st["k_cache"].shape[1]
            t = torch.arange(length, device=q.device)
            pages, slots = st["table"][b][t // S].long(), t % S
        for h in range(c["Hkv"]):
            k = torch.cat([st["k_cache"][pages, slots, h], st["k_new"][b, :n, h]]).double()
            v = torch.cat([st["v_cache"][pages, slots, h], st["v_new"][b, :n, h]]).double()
            for g in range(c["G"]):
                head = h * c["G"] + g
                s = q[b, :n, head].double() @ k.T / math.sqrt(D)
                s[hidden] = -math.inf
                out[b, :n, head] = torch.softmax(s, 1) @ v
    return out


def _logits_exact(st):
    x = st["logits"].double()
    B, R, V = x.shape
    history, length, prompt = (st[n].cpu().numpy() for n in ("history", "history_len", "prompt_len"))
    tokens = st["tokens"].cpu().numpy()
    parent = None if st["parent"] is None else st["parent"].cpu().numpy()
    rep, freq, pres = (st[n].double().tolist() for n in ("repetition", "frequency", "presence"))
    for b in range(B):
        old = np.bincount(history[b, :prompt[b]], minlength=V)
        new = np.bincount(history[b, prompt[b]:length[b]], minlength=V)
        old, new = torch.from_numpy(old).cuda(), torch.from_numpy(new).cuda()
        for r in range(R):
            if parent is None:
                path = [int(t) for t in tokens[b, :r]]
            else:
                path = [int(tokens[b, j]) for j in _path_nodes(parent[b], r) if j > 0]
            c = new.clone()
            if path:
                c += torch.bincount(torch.tensor(path), minlength=V).cuda()
            y = x[b, r]
            known = (c + old) > 0
            y = torch.where(known & (y > 0), y / rep[b], torch.where(known, y * rep[b], y))
            x[b, r] = y - freq[b] * c - pres[b] * (c > 0)
        if st["bias_tokens"] is not None:
            used = st["bias_tokens"][b] >= 0
            x[b, :, st["bias_tokens"][b][used].long()] += st["bias_values"][b][used].double()
    if st["allowed"] is not None:
        shift = torch.arange(32, device=x.device, dtype=torch.int32)
        bit = (st["allowed"].unsqueeze(-1) >> shift) & 1
        x[bit.flatten(2)[:, :, :V] == 0] = -math.inf
    return x


def exact(case, seed):
    if case["op"] not in ("attn", "logits"):
        return None  # whole numbers and copies
    w = work(case)
    if w["flops"] > 8e11 or case["B"] * case.get("Hkv", 1) > 4096:
        return None
    st = prepare(case, seed)
    return _attn_exact(st) if case["op"] == "attn" else _logits_exact(st)


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(one.get("name", "drawn"), {k: "%.3g" % v for k, v in work(one).items()}, one)
