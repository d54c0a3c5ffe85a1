"""Plain 64-bit restatements of tree attention, its plan, the cache commit and
logits processing (include/spec_attn.h, include/spec_logits.h), one element at
a time where that is affordable, and random inputs for them.  CPU only; no
code shared with the library."""
import math

import numpy as np
import torch


def ancestors(parent, n):
    """Node n and its ancestors, n first."""
    path = [n]
    while n > 0:
        n = int(parent[n])
        path.append(n)
    return path


def random_tree(rng, N, kind):
    if kind == "chain":
        p = np.arange(N) - 1
    elif kind == "star":
        p = np.zeros(N, np.int64)
    else:
        p = np.floor(rng.random(N) * np.arange(N)).astype(np.int64)
    p[0] = -1
    return p.astype(np.int32)


def plan_ref(parent, n_nodes, cache_len, cap, table=None, page_size=1, num_pages=1):
    """(positions [B,N], status [B], mask [B,N,W]) by following parents."""
    B, N = parent.shape
    W = 4 * -(-N // 128)
    pos = np.full((B, N), -1, np.int32)
    status = np.zeros(B, np.int32)
    mask = np.zeros((B, N, W), np.uint32)
    for b in range(B):
        n, length = int(n_nodes[b]), int(cache_len[b])
        ok = 0 <= n <= N and 0 <= length <= cap
        ok = ok and all(0 <= parent[b, i] < i for i in range(1, n))
        if ok and n > 0 and table is not None:
            ok = all(0 <= table[b, i] < num_pages for i in range(-(-length // page_size)))
        if not ok:
            status[b] = -1
            continue
        for i in range(n):
            path = ancestors(parent[b], i)
            pos[b, i] = length + len(path) - 1
            for j in path:
                mask[b, i, j >> 5] |= np.uint32(1 << (j & 31))
    return pos, status, mask


def attention_ref(q, k_new, v_new, k_cache, v_cache, parent, n_nodes, cache_len, table=None,
                  scale=None):
    """(out, lse, bound) in float64 from CPU tensors.  bound[b,n,h,d] is
    sum_j w_j |v_jd|, what relative errors of the weights are measured by, and
    with it comes the largest sum_d |q_d k_d| * scale of the row, what the
    rounding of its scores is measured by."""
    B, N, Hq, D = q.shape
    Hkv = k_new.shape[2]
    G = Hq // Hkv
    scale = D ** -0.5 if scale is None else scale
    S = k_cache.shape[1]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    lse = torch.full((B, N, Hq), -math.inf, dtype=torch.float64)
    mag = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    big = torch.zeros((B, N, Hq), dtype=torch.float64)
    for b in range(B):
        L = int(cache_len[b])
        t = np.arange(L)
        page = torch.full((L,), b) if table is None else torch.from_numpy(
            table[b][t // S].astype(np.int64))
        slot = torch.from_numpy(t % S)
        for n in range(int(n_nodes[b])):
            sel = torch.tensor(sorted(ancestors(parent[b], n)))
            for h in range(Hkv):
                k = torch.cat([k_cache[page, slot, h], k_new[b, sel, h]]).double()
                v = torch.cat([v_cache[page, slot, h], v_new[b, sel, h]]).double()
                for g in range(G):
                    x = q[b, n, h * G + g].double()
                    s = (k @ x) * scale
                    m = s.max()
                    p = torch.exp(s - m)
                    out[b, n, h * G + g] = (p[:, None] * v).sum(0) / p.sum()
                    mag[b, n, h * G + g] = (p[:, None] * v.abs()).sum(0) / p.sum()
                    big[b, n, h * G + g] = ((k.abs() @ x.abs()) * scale).max()
                    lse[b, n, h * G + g] = m + torch.log(p.sum())
    return out, lse, mag, big


def attention_tolerance(out, mag, big, dtype, D, keys):
    """How far an output may be off: each weight is rounded to the dtype once
    (at most half a step of its value: eps / 2), the result once more; the
    scores are sums of D products in fp32 (each partial sum off by at most
    2^-23 of the largest magnitude, tensor cores truncating), and a score off
    by e scales a weight by 1 +- e, in the sum and in the total (2 e); the
    sums over keys and the exponentials add less than 2^-16.  A half weight
    below its smallest subnormal loses at most 2^-25 of the largest weight."""
    half = torch.finfo(dtype).eps / 2
    e = (D + 4) * 2.0 ** -23 * big[..., None]
    tol = half * out.abs() + (half * (1 + half) + 2 * e + 2.0 ** -16) * mag
    if dtype == torch.float16:
        tol = tol + keys * 2.0 ** -25 * 8.0
    return tol * 1.001 + 1e-30


def commit_ref(k_new, v_new, k_cache, v_cache, cache_len, accepted, nodes=None, table=None):
    """Copies of the caches [layers, P, S, H, D] with the paths appended, and the lengths."""
    kc, vc = k_cache.clone(), v_cache.clone()
    B, N = k_new.shape[1:3]
    P, S = k_cache.shape[1:3]
    cap = S if table is None else table.shape[1] * S
    out = np.full(B, -1, np.int32)
    for b in range(B):
        a, length = int(accepted[b]), int(cache_len[b])
        if not 0 <= a < N or length < 0 or length + a + 1 > cap:
            continue
        moves = []
        for i in range(a + 1):
            node = i if i == 0 or nodes is None else int(nodes[b, i - 1])
            at = length + i
            page = b if table is None else int(table[b, at // S])
            moves.append((node, page, at % S))
        if any(not (0 <= n < N and 0 <= p < P) for n, p, _ in moves):
            continue
        for n, p, s in moves:
            kc[:, p, s] = k_new[:, b, n]
            vc[:, p, s] = v_new[:, b, n]
        out[b] = length + a + 1
    return kc, vc, out


def logits_ref(x, history=None, history_len=None, prompt_len=None, draft_tokens=None, parent=None,
               n_nodes=None, repetition=None, frequency=None, presence=None, bias_tokens=None,
               bias_values=None, allowed=None):
    """(values [B, R, V] in float64 from numpy arrays, written [B, R]: False for the
    rows past n_nodes, and the summed magnitudes of each value's terms)."""
    B, R, V = x.shape
    y = x.copy()
    mag = np.abs(x)
    written = np.ones((B, R), bool)
    for b in range(B):
        nn = R if n_nodes is None else int(n_nodes[b])
        rep = 1.0 if repetition is None else float(repetition[b])
        freq = 0.0 if frequency is None else float(frequency[b])
        pres = 0.0 if presence is None else float(presence[b])
        hist = [] if history is None else list(history[b, :max(0, history_len[b])])
        prompt = 0 if history is None else int(prompt_len[b])
        used = [] if draft_tokens is None else (
            [int(draft_tokens[b, i]) for i in range(1, nn)] if parent is not None
            else [int(t) for t in draft_tokens[b, :max(0, nn - 1)]])
        bias = [] if bias_tokens is None else list(zip(bias_tokens[b], bias_values[b]))
        ok = (0 < rep < math.inf and math.isfinite(freq) and math.isfinite(pres)
              and 1 <= nn <= R and all(0 <= t < V for t in hist + used)
              and all(-1 <= t < V for t, _ in bias))
        if history is not None:
            ok = ok and 0 <= prompt <= history_len[b] <= history.shape[1]
        if ok and parent is not None:
            ok = all(0 <= parent[b, i] < i for i in range(1, nn))
        if not ok:
            y[b, :nn if 1 <= nn <= R else R] = math.nan
            if 1 <= nn <= R:
                written[b, nn:] = False
            continue
        written[b, nn:] = False
        old = np.bincount(np.array(hist[:prompt], np.int64), minlength=V)
        new = np.bincount(np.array(hist[prompt:], np.int64), minlength=V)
        add, size = np.zeros(V), np.zeros(V)
        for t, v in bias:
            if t >= 0:
                add[t] += float(v)
                size[t] += abs(float(v))
        for r in range(nn):
            if draft_tokens is None:
                path = []
            elif parent is None:
                path = [int(t) for t in draft_tokens[b, :r]]
            else:
                path = [int(draft_tokens[b, i]) for i in ancestors(parent[b], r) if i > 0]
            c = new + np.bincount(np.array(path, np.int64), minlength=V)
            seen = (c + old) > 0
            z = x[b, r]
            z = np.where(seen, np.where(z > 0, z / rep, z * rep), z)
            z = z - freq * c - pres * (c > 0) + add
            if allowed is not None:
                w = allowed[min(b, allowed.shape[0] - 1), min(r, allowed.shape[1] - 1)]
                bit = (w[np.arange(V) // 32].astype(np.int64) >> (np.arange(V) % 32)) & 1
                z = np.where(bit == 1, z, -math.inf)
            y[b, r] = z
            mag[b, r] = (np.abs(x[b, r]) * max(rep, 1 / rep) + abs(freq) * c
                         + abs(pres) * (c > 0) + size)
    return y, written, mag
