"""Plain restatements of chunk attention and append, beam selection and the page
operators (include/spec_chunk.h, include/spec_beam.h, include/spec_pages.h): 64
bits, one element at a time where that is affordable.  No code shared with the
library."""
import math

import numpy as np
import torch


# ------------------------------------------------------------------ chunks

def make_chunk(seed, new, past, Hkv, G, D, S, dtype, device="cuda", cap=None):
    """Inputs of a step: caches that hold `past` positions of each sequence and
    `new` more, page table, row starts.  S = 0: one contiguous run per sequence."""
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    new, past = np.asarray(new), np.asarray(past)
    B, T = len(new), int(new.sum())
    most = int(cap or max(1, (new + past).max()))
    if S:
        M = -(-most // S)
        P = B * M + 2
        table = torch.from_numpy(rng.permutation(P)[:B * M].reshape(B, M).astype(np.int32))
    else:
        S, P, table = most, B, None
    def rnd(*s):
        return torch.randn(s, generator=gen).to(dtype).to(device)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    return dict(q=rnd(T, G * Hkv, D), k_cache=rnd(P, S, Hkv, D), v_cache=rnd(P, S, Hkv, D),
                start=start.to(device),
                length=torch.from_numpy((new + past).astype(np.int32)).to(device),
                table=None if table is None else table.to(device))


def positions(st, b, n):
    """(pages, slots) of sequence b's first n positions."""
    S = st["k_cache"].shape[1]
    t = torch.arange(n, device=st["k_cache"].device)
    if st["table"] is None:
        return torch.full_like(t, b), t
    return st["table"][b].long()[t // S], t % S


def chunk_ref(st, scale=None):
    """(out, lse, mag, big) in 64 bits: mag is sum_j w_j |v_jd|, big the largest
    sum_d |q_d k_d| * scale of a row (serve_util.attention_tolerance)."""
    q = st["q"].double()
    T, Hq, D = q.shape
    Hkv = st["k_cache"].shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    out, mag = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    big = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    start, length = st["start"].tolist(), st["length"].tolist()
    for b in range(len(length)):
        n = start[b + 1] - start[b]
        if n == 0:
            continue
        pages, slots = positions(st, b, length[b])
        rows = slice(start[b], start[b + 1])
        hidden = (torch.arange(length[b], device=q.device)[None, :]
                  > length[b] - n + torch.arange(n, device=q.device)[:, None])
        for h in range(Hkv):
            k, v = st["k_cache"][pages, slots, h].double(), st["v_cache"][pages, slots, h].double()
            for g in range(h * G, (h + 1) * G):
                s = (q[rows, g] @ k.T) * scale
                s[hidden] = -math.inf
                m = s.amax(1, keepdim=True)
                p = torch.exp(s - m)
                total = p.sum(1, keepdim=True)
                out[rows, g] = (p @ v) / total
                mag[rows, g] = (p @ v.abs()) / total
                lse[rows, g] = (m + total.log())[:, 0]
                big[rows, g] = ((q[rows, g].abs() @ k.abs().T) * scale).amax(1)
    return out, lse, mag, big


# ------------------------------------------------------------------- beams

def beam_ref(logits, scores, n, finished=None, norm=None, end_token=0):
    """(tokens, beams, scores) by sorting every candidate; exact ties go to the
    lower k V + x.  Sums of exponentials by math.fsum, so equal rows in any order give
    equal totals."""
    B, K, V = logits.shape
    x = logits.double().numpy()
    tokens, beams = np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32)
    best = np.full((B, n), -math.inf)
    for b in range(B):
        got, bad = [], False
        for k in range(K):
            s = float(scores[b, k])
            c = 1.0 if norm is None else float(norm[b, k])
            if math.isnan(s) or s == math.inf:
                bad = True
                continue
            if s == -math.inf:
                continue
            if not c > 0 or math.isinf(c):
                bad = True
                continue
            if finished is not None and int(finished[b, k]):
                got.append((-(s / c), k * V + end_token, s))
                continue
            row = x[b, k]
            if np.isnan(row).any() or (row == math.inf).any():
                bad = True
                continue
            m = row.max()
            if m == -math.inf:
                continue
            lse = m + math.log(math.fsum(np.exp(row - m)))
            at = np.argsort(-row, kind="stable")[:n]
            got += [(-((s + (row[i] - lse)) / c), k * V + int(i), s + (row[i] - lse))
                    for i in at if row[i] > -math.inf]
        if bad:
            best[b] = math.nan
            continue
        for i, (_, f, s) in enumerate(sorted(got, key=lambda g: g[:2])[:n]):
            tokens[b, i], beams[b, i], best[b, i] = f % V, f // V, s
    return tokens, beams, best


# ------------------------------------------------------------------- pages

def old_row(table, length, P, S):
    """The pages of a row, or None for a row in error."""
    held = []
    for e in table:
        if e < 0:
            break
        held.append(int(e))
    if any(e >= P for e in held) or length < 0 or length > len(held) * S:
        return None
    return held


def fork_ref(table, length, parent, ref, S, reserve=None):
    """(table, length, ref, copies) as include/spec_pages.h says, row by row."""
    R0, M = table.shape
    R, P = len(parent), len(ref)
    new, out = np.full((R, M), -1, np.int32), np.full(R, -1, np.int32)
    count, copies = ref.copy(), np.full((3, R), -1, np.int32)
    copies[2] = 0
    free = [p for p in range(P) if ref[p] == 0]
    olds = [old_row(table[o], int(length[o]), P, S) for o in range(R0)]
    taken = set()
    for r in range(R):
        o, more = int(parent[r]), 0 if reserve is None else int(reserve[r])
        if not -1 <= o < R0 or more < 0 or (o >= 0 and olds[o] is None):
            continue
        held, n = ([], 0) if o < 0 else (olds[o], int(length[o]))
        pages = -(-(n + more) // S)
        if pages > M:
            continue
        first = o not in taken
        taken.add(o)
        row = []
        for i in range(pages):
            e = held[i] if i < len(held) else -1
            if e >= 0 and (i < n // S or (first and ref[e] == 1)):
                row.append(e)
                continue
            if not free:
                return (np.full((R, M), -1, np.int32), np.full(R, -1, np.int32), ref.copy(),
                        np.stack([np.full(R, -1), np.full(R, -1), np.zeros(R)]).astype(np.int32))
            row.append(free.pop(0))
            if i == n // S and n % S:
                copies[:, r] = e, row[-1], n % S
        new[r, :len(row)] = row
        out[r] = n
        for e in row:
            count[e] += 1
    for row in (h for h in olds if h is not None):
        for e in row:
            count[e] -= 1
    return new, out, count, copies


def compact_ref(table, ref, S):
    P = len(ref)
    used = int((ref > 0).sum())
    holes = [p for p in range(used) if ref[p] <= 0]
    movers = [p for p in range(used, P) if ref[p] > 0]
    to = dict(zip(movers, holes))
    copies = np.full((3, P // 2), -1, np.int32)
    copies[2] = 0
    count = np.zeros_like(ref)
    for p in range(P):
        if ref[p] > 0:
            count[to.get(p, p)] = ref[p]
    for i, (a, b) in enumerate(zip(movers, holes)):
        copies[:, i] = a, b, S
    new = np.vectorize(lambda e: to.get(int(e), int(e)), otypes=[np.int32])(table) \
        if table.size else table.copy()
    return new, count, copies, used
