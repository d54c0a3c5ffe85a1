"""The operators around a prompt's prefill and beam search, with plain forms.

  chunk    (each layer) the keys and values of a chunk of new tokens appended to
           a paged or contiguous cache, and the causal attention of the chunk's
           queries over all of the cache; the plan is part of the pass, as in a
           step's first layer.  Sequences lie one behind the other, each with a
           number of new tokens of its own.
  beam     beam search's selection over beams and vocabulary, and the beams'
           token histories in the order of the selected
  fork     the page tables of the selected beams: whole pages are shared, the
           others' last pages copied in every layer, dropped beams' pages freed
           and pages for the next tokens taken
  compact  the pages in use moved to the front of the pool

A page is free when no table refers to it (reference count 0), and pages are
taken in ascending order.
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
        # the last tokens of one prompt: latency counts
        dict(name="chunk B1 n40 past600", op="chunk", B=1, n=40, past=600, Hkv=8, G=4, D=128, S=16,
             dtype="bf16"),
        # short prompts from their first token on, a group size that divides no tile
        dict(name="chunk B8 n301 D64", op="chunk", B=8, n=301, past=0, Hkv=4, G=7, D=64, S=64,
             dtype="fp16"),
        # an ordinary prefill batch: ragged chunks behind cached parts
        dict(name="chunk B8 n1024 past4096", op="chunk", B=8, n=1024, past=4096, Hkv=8, G=4, D=128,
             S=64, dtype="bf16"),
        # a chunk far inside a long document
        dict(name="chunk B1 n512 past131072", op="chunk", B=1, n=512, past=131072, Hkv=8, G=5,
             D=128, S=256, dtype="bf16"),
        # whole long prompts over one contiguous cache
        dict(name="chunk B2 n8192", op="chunk", B=2, n=8192, past=0, Hkv=8, G=8, D=128, S=0,
             dtype="bf16"),
        # one sentence with four beams
        dict(name="beam B1 K4 V32000", op="beam", B=1, K=4, V=32000, n=4, H=256, dtype="bf16"),
        # a batch with twice as many candidates as beams
        dict(name="beam B64 K8 V128256", op="beam", B=64, K=8, V=128256, n=16, H=2048,
             dtype="bf16"),
        # fp32 logits
        dict(name="beam B32 K5 V151936", op="beam", B=32, K=5, V=151936, n=10, H=1024,
             dtype="f32"),
        # one sentence's four beams
        dict(name="fork 4 beams", op="fork", B=1, K=4, L=600, S=16, layers=4, Hkv=8, D=128,
             most=1, dtype="bf16"),
        # a batch of beams after a step, every layer's pages
        dict(name="fork 512 beams", op="fork", B=64, K=8, L=1500, S=16, layers=8, Hkv=2, D=128,
             most=8, dtype="bf16"),
        # a small pool with holes
        dict(name="compact P512", op="compact", B=16, K=1, L=600, S=32, layers=4, Hkv=8, D=128,
             dtype="bf16"),
        # a large one
        dict(name="compact P16384", op="compact", B=128, K=2, L=1500, S=16, layers=8, Hkv=4,
             D=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "beam", "beam", "fork", "fork", "compact"])
    if op == "chunk":
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8])
        D = rng.choice([64, 64, 80, 96, 128, 128, 128])
        past = rng.choice([0, _log(rng, 16, 131072), _log(rng, 16, 131072)])
        n = _log(rng, 1, 8192)
        S = rng.choice([0, 8, 16, 32, 64, 128, 256])
        while Hkv * G * n * max(64 * (past + n), D * (past + n / 2)) > 2e11:  # the largest's work
            n = n // 2
        cost = Hkv * G * n * max(64 * (past + n), D * (past + n / 2))
        most = min(256, (1 << 29) // ((past + n) * Hkv * D), int(2e11 / cost))
        return dict(op=op, B=_log(rng, 1, max(1, most)), n=n, past=past, Hkv=Hkv, G=G, D=D, S=S,
                    dtype=rng.choice(["bf16", "bf16", "fp16"]))
    if op == "beam":
        V, K, dtype = _log(rng, 1000, 160000), rng.choice([1, 2, 3, 4, 5, 8, 16]), \
            rng.choice(["bf16", "f32"])
        most = min(128, int(6.5e7 / (V * K)))
        return dict(op=op, B=_log(rng, 1, max(1, most)), K=K, V=V, n=rng.choice([K, 2 * K, K + 1]),
                    H=_log(rng, 16, 2048), dtype=dtype)
    B, K, S = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 8, 16, 32, 64])
    Hkv, D, dtype = rng.choice([1, 2, 8]), rng.choice([64, 80, 128]), rng.choice(["bf16", "f32"])
    layers, L = _log(rng, 1, 32), _log(rng, max(4, S), 1500)
    while 4 * B * K * L * Hkv * D * layers * SIZE[dtype] > 5e9:  # a pool of a few GB
        L, B, layers = max(4, L // 2), max(1, B - B // 4), max(1, layers - layers // 4)
    c = dict(op=op, B=B, K=K, L=L, S=S, layers=layers, Hkv=Hkv, D=D, dtype=dtype)
    if op == "fork":
        c["most"] = rng.choice([1, 1, 8, 40])
    return c


# ------------------------------------------------------------------ inputs

def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _beams(c, rng):
    """A pool of pages and the tables of B sequences with K beams each: a prompt's
    whole pages are shared by its beams, the others their own.  Pages of other
    requests lie between.  (table [B K, M], lengths, reference counts)"""
    B, K, L, S = c["B"], c["K"], c["L"], c["S"]
    M = -(-(L + 48) // S)
    ragged = np.random.default_rng(L)  # a case's sizes, whose order and pages the seed gives
    size = ragged.integers((L + 1) // 2, L + 1, size=B)
    prompt = (size * ragged.uniform(0.3, 0.95, B)).astype(np.int64)
    order = rng.permutation(B)
    length, shared = np.repeat(size[order], K), np.repeat(prompt[order], K) // S
    held = -(-length // S)
    table = np.full((B * K, M), -1, np.int64)
    names, count = 0, []
    for r in range(B * K):
        if r % K == 0:
            prompt = np.arange(names, names + shared[r])
            names += shared[r]
            count += [K] * int(shared[r])
        table[r, :shared[r]] = prompt
        mine = int(held[r] - shared[r])
        table[r, shared[r]:held[r]] = np.arange(names, names + mine)
        names += mine
        count += [1] * mine
    other = names // 4 + 3                                   # pages of other requests
    count += list(rng.integers(1, 4, size=other))
    free = names // 3 + 2 * B * K + (48 // S + 2) * B * K    # pages of none
    total = names + other + free
    place = rng.permutation(total)
    ref = np.zeros(total, np.int64)
    ref[place[:names + other]] = count
    table = np.where(table >= 0, place[table.clip(min=0)], -1)
    return table.astype(np.int32), length.astype(np.int32), ref.astype(np.int32)


def prepare(case, seed):
    c = dict(case)
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": c}
    if c["op"] == "chunk":
        B, n, past, H, G, D, S = (c[x] for x in ("B", "n", "past", "Hkv", "G", "D", "S"))
        dt = DTYPES[c["dtype"]]
        new = np.random.default_rng(n).integers((n + 1) // 2, n + 1, size=B)
        new[0] = n  # a case's sizes, whose order the seed gives
        start = np.concatenate([[0], np.cumsum(rng.permutation(new))])
        before = rng.integers((past + 1) // 2, past + 1, size=B)
        cap = past + n
        if S == 0:
            st["table"], P, S = None, B, cap
        else:
            M = -(-cap // S)
            P = B * M + 3
            st["table"] = _dev(rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32))
        st.update(start=_dev(start.astype(np.int32)), before=_dev(before.astype(np.int32)))
        # queries, keys and values as slices of one projection
        qkv = _normal(gen, (int(start[-1]), (G + 2) * H, D), dt)
        st["q"], st["k_new"], st["v_new"] = (qkv[:, :G * H], qkv[:, G * H:(G + 1) * H],
                                             qkv[:, (G + 1) * H:])
        st["k_cache"] = _normal(gen, (P, S, H, D), dt)
        st["v_cache"] = _normal(gen, (P, S, H, D), dt)
    elif c["op"] == "beam":
        B, K, V, H = c["B"], c["K"], c["V"], c["H"]
        x = torch.randn((B, K, V), generator=gen, device="cuda") * 2.0
        # a few continuations stand out, more clearly in some places than in others
        few = _dev(rng.integers(0, V, size=(B, K, 12)))
        x.scatter_add_(2, few, _dev(rng.uniform(2, 12, size=(B, K, 12)).astype(np.float32)))
        st["logits"] = x.to(DTYPES[c["dtype"]])
        # log-probabilities of the beams so far, some of them ended, divided by a power of
        # their length as they are compared
        length = rng.integers(1, H, size=(B, K))
        ended = rng.random((B, K)) < 0.15
        scores = -rng.uniform(0.2, 0.4, size=(B, 1)) * length.mean(1, keepdims=True) \
            - rng.exponential(2.0, size=(B, K))
        st["scores"] = _dev(scores.astype(np.float32))
        st["finished"] = _dev(ended.astype(np.int32))
        st["norm"] = _dev(((length + ~ended) ** 0.6).astype(np.float32))
        st["history"] = _dev(rng.integers(0, V, size=(B, K, H)).astype(np.int32))
    else:
        table, length, ref = _beams(c, rng)
        R, B, K = len(length), c["B"], c["K"]
        if c["op"] == "fork":
            # each beam's place is taken by a beam of the same sequence; some sequences end
            first = np.repeat(np.arange(B) * K, K)
            parent = first + np.minimum(K - 1, rng.exponential(K / 4, size=R).astype(np.int64))
            parent[np.repeat(rng.random(B) < 0.08, K)] = -1
            st["parent"] = _dev(parent.astype(np.int32))
            reserve = rng.integers(1, c["most"] + 1, size=R) * (parent >= 0)
            st["reserve"] = _dev(reserve.astype(np.int32))
        st.update(table=_dev(table), length=_dev(length), ref=_dev(ref))
        shape = (c["layers"], len(ref), c["S"], c["Hkv"], c["D"])
        st["k_cache"] = _normal(gen, shape, DTYPES[c["dtype"]])
        st["v_cache"] = _normal(gen, shape, DTYPES[c["dtype"]])
    return st


# ------------------------------------------------------------- plain forms

def _run_of(cache, table):
    """[B, H, L, D] of a sequence's cache slots in order, in 32 bits."""
    rows = cache if table is None else cache[table.long()].flatten(1, 2)
    return rows.transpose(1, 2).float()


def _chunk_plain(st):
    q, c = st["q"], st["case"]
    T, Hq, D = q.shape
    B, n, H, G, S = c["B"], c["n"], c["Hkv"], c["G"], st["k_cache"].shape[1]
    start, before, dev = st["start"].long(), st["before"].long(), q.device
    # append
    row = torch.arange(T, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), row, right=True)
    i = row - start[b]
    at = before[b] + i
    page = b if st["table"] is None else st["table"][b, at // S].long()
    st["k_cache"][page, at % S] = st["k_new"]
    st["v_cache"][page, at % S] = st["v_new"]
    # every sequence's rows, up to the longest chunk's number
    rows = (start[:-1, None] + torch.arange(n, device=dev)).clamp(max=T - 1)
    last = before[:, None] + torch.arange(n, device=dev)
    s = q[rows].float().view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    s = (s @ _run_of(st["k_cache"], st["table"]).transpose(2, 3)) * D ** -0.5
    L = s.shape[3]
    hidden = torch.arange(L, device=dev) > last[:, :, None]
    s = s.view(B, H, G, n, L).masked_fill_(hidden[:, None, None], -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = s.view(B, H, G * n, L) @ _run_of(st["v_cache"], st["table"])
    o = (o.view(B, H, G, n, D) / total).permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D)
    return {"out": o[b, i].to(q.dtype), "k_cache": st["k_cache"], "v_cache": st["v_cache"],
            "length": (before + start[1:] - start[:-1]).to(torch.int32)}


def _beam_plain(st):
    c = st["case"]
    B, K, V, n = c["B"], c["K"], c["V"], c["n"]
    x = st["logits"].double()
    m = x.amax(-1, keepdim=True)
    x = x - (m + (x - m).exp().sum(-1, keepdim=True).log())
    s = st["scores"].double()[:, :, None] + x
    # a beam that has ended goes on by one token (0) at no cost
    end = st["finished"][:, :, None] != 0
    s = torch.where(end, -math.inf, s)
    s[:, :, 0] = torch.where(end[:, :, 0], st["scores"].double(), s[:, :, 0])
    rank = (s / st["norm"].double()[:, :, None]).flatten(1)
    at = torch.sort(rank, dim=1, descending=True, stable=True)[1][:, :n]
    beam, token = at // V, at % V
    score = s.flatten(1).gather(1, at)
    none = score == -math.inf
    beam, token = beam.masked_fill(none, -1), token.masked_fill(none, -1)
    H = st["history"].shape[2]
    text = st["history"].gather(1, beam.clamp(min=0)[:, :, None].expand(B, n, H))
    return {"tokens": token.to(torch.int32), "beams": beam.to(torch.int32), "scores": score.float(),
            "history": text.masked_fill(none[:, :, None], 0)}


def _copy_plain(st, copies):
    src, dst, slots = copies
    e, i = (torch.arange(st["case"]["S"], device=src.device) < slots[:, None]).nonzero(as_tuple=True)
    src, dst = src[e], dst[e]
    st["k_cache"][:, dst, i] = st["k_cache"][:, src, i]
    st["v_cache"][:, dst, i] = st["v_cache"][:, src, i]


def _listed_pages(which, number, most):
    """The pages p with which[p], in order, as a list of `most` entries (then -1)."""
    P = len(which)
    rank = torch.cumsum(which, 0) - 1
    to = torch.where(which & (rank < most), rank, most)
    out = torch.full((most + 1,), -1, dtype=torch.int64, device=which.device)
    out.scatter_(0, to, torch.arange(P, device=which.device))
    out[most] = -1
    return out


def _fork_plain(st):
    table, ref, S = st["table"].long(), st["ref"], st["case"]["S"]
    parent, reserve = st["parent"].long(), st["reserve"].long()
    R0, M = table.shape
    R, P, dev = len(parent), len(ref), ref.device
    r, i = torch.arange(R, device=dev), torch.arange(M, device=dev)
    live, pa = parent >= 0, parent.clamp(min=0)
    length = torch.where(live, st["length"][pa].long(), 0)
    rows = table[pa]
    eldest = torch.full((R0 + 1,), R, device=dev).scatter_reduce_(
        0, torch.where(live, parent, R0), r, "amin")
    first = live & (eldest[pa] == r)
    private = i >= (length // S)[:, None]
    single = ref[rows.clamp(min=0)] == 1
    need = i < ((length + reserve + S - 1) // S)[:, None]
    keep = need & live[:, None] & (rows >= 0) & (~private | (first[:, None] & single))
    fresh = need & ~keep
    free = _listed_pages(ref == 0, P, P)
    take = free[(torch.cumsum(fresh.flatten(), 0) - 1).clamp(min=0)].view(R, M)
    new = torch.where(keep, rows, torch.where(fresh, take, -1))
    tail = length % S
    here = (length // S).clamp(max=M - 1)[:, None]
    copied = live & (tail > 0) & fresh.gather(1, here)[:, 0]
    copies = torch.stack([torch.where(copied, rows.gather(1, here)[:, 0], -1),
                          torch.where(copied, new.gather(1, here)[:, 0], -1),
                          torch.where(copied, tail, 0)])
    count = torch.cat([ref.long(), ref.new_zeros(1, dtype=torch.int64)])
    one = torch.ones((), dtype=torch.int64, device=dev)
    count.scatter_add_(0, torch.where(table >= 0, table, P).flatten(), -one.expand(R0 * M))
    count.scatter_add_(0, torch.where(new >= 0, new, P).flatten(), one.expand(R * M))
    _copy_plain(st, copies)
    return {"table": new.to(torch.int32), "length": length.to(torch.int32),
            "ref": count[:P].to(torch.int32), "copies": copies.to(torch.int32),
            "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _compact_plain(st):
    table, ref = st["table"].long(), st["ref"]
    P, dev = len(ref), ref.device
    used = ref > 0
    n, p = used.sum(), torch.arange(P, device=dev)
    moved = used & (p >= n)
    most = P // 2
    src, dst = _listed_pages(moved, n, most), _listed_pages(~used & (p < n), n, most)
    dst = torch.where(src >= 0, dst, -1)
    to = torch.where(moved, dst[(torch.cumsum(moved, 0) - 1).clamp(min=0)], p)
    new = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    count = torch.zeros(P + 1, dtype=torch.int32, device=dev)
    count.scatter_(0, torch.where(used, to, P), ref)
    copies = torch.stack([src, dst, torch.where(src >= 0, st["case"]["S"], 0)])[:, :most]
    _copy_plain(st, copies)
    return {"table": new.to(torch.int32), "ref": count[:P], "copies": copies.to(torch.int32),
            "used": n.to(torch.int32).view(1), "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import speculative_decoding_verification_65_gb300 as sv
        if op == "chunk":
            length = sv.spec_chunk_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                                          st["start"], st["before"], page_table=st["table"])
            plan = sv.spec_chunk_plan(st["start"], length, st["q"], st["k_cache"],
                                      page_table=st["table"])
            out = sv.spec_chunk_attention(st["q"], st["k_cache"], st["v_cache"], plan,
                                          page_table=st["table"])
            return {"out": out, "k_cache": st["k_cache"], "v_cache": st["v_cache"],
                    "length": length}
        if op == "beam":
            tokens, beams, scores = sv.spec_beam_select(
                st["logits"], st["scores"], st["case"]["n"], finished=st["finished"],
                norm=st["norm"], end_token=0)
            return {"tokens": tokens, "beams": beams, "scores": scores,
                    "history": sv.spec_beam_reorder(st["history"], beams)}
        if op == "fork":
            table, length, ref, copies = sv.spec_pages_fork(
                st["table"], st["length"], st["parent"], st["ref"], st["case"]["S"],
                reserve=st["reserve"])
            sv.spec_pages_copy(st["k_cache"], st["v_cache"], copies)
            return {"table": table, "length": length, "ref": ref, "copies": copies,
                    "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        table, ref, copies, used = sv.spec_pages_compact(st["table"], st["ref"], st["case"]["S"])
        sv.spec_pages_copy(st["k_cache"], st["v_cache"], copies)
        return {"table": table, "ref": ref, "copies": copies, "used": used,
                "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return {"chunk": _chunk_plain, "beam": _beam_plain, "fork": _fork_plain,
            "compact": _compact_plain}[op](st)


# ------------------------------------------------------------------- work

def work(case):
    """Bytes and operations of one pass at the mean of its ragged sizes."""
    c = case
    B = c["B"]
    size = SIZE[c["dtype"]]
    if c["op"] == "chunk":
        H, G, D = c["Hkv"], c["G"], c["D"]
        n = (c["n"] + (c["n"] + 1) // 2) / 2
        past = (c["past"] + (c["past"] + 1) // 2) / 2
        # new keys and values read and written, queries and outputs, the cached keys and values
        moved = B * H * D * size * (4 * n + 2 * G * n + 2 * past)
        return {"bytes": moved + 12.0 * B, "flops": 4.0 * B * H * G * D * n * (past + (n + 1) / 2)}
    if c["op"] == "beam":
        cells = float(B) * c["K"] * c["V"] * 0.85
        return {"bytes": cells * size + 8.0 * B * c["n"] * c["H"] + 12.0 * B * (c["K"] + c["n"]),
                "flops": 3 * cells}
    R, S = B * c["K"], c["S"]
    length = 0.75 * c["L"]
    pages = B * (length * 0.62 + c["K"] * (length * 0.38 + S)) / S
    pool = pages * 1.6 + R * (4 + 48 // S)
    M = -(-(c["L"] + 48) // S)
    tables = 8.0 * R * M + 8.0 * pool
    page = 2.0 * c["layers"] * c["Hkv"] * c["D"] * size
    if c["op"] == "fork":
        return {"bytes": tables + 20.0 * R + 2 * page * 0.4 * R * (S - 1) / 2, "flops": 0.0}
    used = 1.25 * pages
    return {"bytes": tables + 2 * page * S * used * (1 - used / pool), "flops": 0.0}


# ------------------------------------------------- definitions in 64 bits

def _chunk_exact(st):
    """softmax(q k^T / sqrt(D)) v over the positions up to a token's own, one sequence and one
    head of keys at a time, some rows at a time."""
    q, c = st["q"], st["case"]
    T, Hq, D = q.shape
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    start, before = st["start"].cpu().numpy(), st["before"].cpu().numpy()
    S = st["k_cache"].shape[1]
    for b in range(c["B"]):
        n, past = int(start[b + 1] - start[b]), int(before[b])
        t = torch.arange(past, device=q.device)
        pages = torch.full_like(t, b) if st["table"] is None else st["table"][b][t // S].long()
        mine = slice(int(start[b]), int(start[b + 1]))
        for h in range(c["Hkv"]):
            k = torch.cat([st["k_cache"][pages, t % S, h], st["k_new"][mine, h]]).double()
            v = torch.cat([st["v_cache"][pages, t % S, h], st["v_new"][mine, h]]).double()
            for i0 in range(0, n, 256):
                i1 = min(n, i0 + 256)
                last = past + torch.arange(i0, i1, device=q.device)
                hidden = torch.arange(past + i1, device=q.device)[None, :] > last[:, None]
                for g in range(c["G"]):
                    head = h * c["G"] + g
                    rows = slice(int(start[b]) + i0, int(start[b]) + i1)
                    s = q[rows, head].double() @ k[:past + i1].T / math.sqrt(D)
                    s[hidden] = -math.inf
                    out[rows, head] = torch.softmax(s, 1) @ v[:past + i1]
    return out


def _beam_exact(st):
    """The n largest log-probabilities of each sequence as they are compared."""
    c = st["case"]
    best = torch.empty((c["B"], c["n"]), dtype=torch.float64)
    for b in range(c["B"]):
        every = []
        for k in range(c["K"]):
            so_far, norm = float(st["scores"][b, k]), float(st["norm"][b, k])
            if int(st["finished"][b, k]):
                every.append(torch.tensor([[so_far / norm, so_far]], dtype=torch.float64))
                continue
            row = st["logits"][b, k].double()
            top = torch.topk(row - torch.logsumexp(row, 0), min(c["n"], c["V"])).values.cpu()
            every.append(torch.stack([(so_far + top) / norm, so_far + top], 1))
        every = torch.cat(every)
        order = torch.argsort(every[:, 0], descending=True)[:c["n"]]
        best[b] = -math.inf
        best[b, :len(order)] = every[order, 1]
    return best


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None  # whole numbers and copies
    if case["op"] == "chunk":
        if work(case)["flops"] > 4e11 or case["B"] * case["Hkv"] * case["G"] > 4096:
            return None
        return {"out": _chunk_exact(prepare(case, seed)), "k_cache": None, "v_cache": None,
                "length": None}
    return {"tokens": None, "beams": None, "scores": _beam_exact(prepare(case, seed)),
            "history": None}


if __name__ == "__main__":
    for one in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(one.get("name", "drawn"), {k: "%.3g" % v for k, v in work(one).items()}, one)
