"""Tree attention in 64 bits, a sequence and a key head at a time, with the bound of its
outputs, and inputs whose every tile of keys some row depends on.  CPU only; no
code shared with the library."""
import math

import numpy as np
import torch

KT = 128  # keys of a tile


def attention(c, scale=None):
    """Outputs of the inputs `c` (tests/test_attn_gpu.py's make): a dict of out, lse, mag =
    sum_j w_j |v_j|, top = the row's largest w_j and big = its largest sum_d |q_d k_d| * scale,
    in float64."""
    q = c["q"]
    B, N, Hq, D = q.shape
    H, S = c["k_new"].shape[2], c["k_cache"].shape[1]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    r = dict(out=torch.zeros((B, N, Hq, D), dtype=torch.float64),
             mag=torch.zeros((B, N, Hq, D), dtype=torch.float64),
             lse=torch.full((B, N, Hq), -math.inf, dtype=torch.float64),
             top=torch.zeros((B, N, Hq), dtype=torch.float64),
             big=torch.zeros((B, N, Hq), dtype=torch.float64))
    for b in range(B):
        n, L = int(c["n_nodes"][b]), int(c["cache_len"][b])
        if n == 0:
            continue
        t = np.arange(L)
        page = torch.full((L,), b) if c["table"] is None else torch.from_numpy(
            c["table"][b][t // S].astype(np.int64))
        slot = torch.from_numpy(t % S)
        sees = torch.zeros((n, L + n), dtype=torch.bool)
        sees[:, :L] = True
        for i in range(n):  # (a parent comes before its node)
            if i > 0:
                sees[i, L:] = sees[int(c["parent"][b, i]), L:]
            sees[i, L + i] = True
        sees = sees.repeat_interleave(G, 0)
        for h in range(H):
            k = torch.cat([c["k_cache"][page, slot, h], c["k_new"][b, :n, h]]).double()
            v = torch.cat([c["v_cache"][page, slot, h], c["v_new"][b, :n, h]]).double()
            x = q[b, :n, h * G:(h + 1) * G].reshape(n * G, D).double()
            s = (x @ k.T * scale).masked_fill(~sees, -math.inf)
            m = s.amax(1, keepdim=True)
            p = (s - m).exp()
            total = p.sum(1, keepdim=True)
            heads = slice(h * G, (h + 1) * G)
            r["out"][b, :n, heads] = ((p @ v) / total).view(n, G, D)
            r["mag"][b, :n, heads] = ((p @ v.abs()) / total).view(n, G, D)
            r["lse"][b, :n, heads] = (m + total.log()).view(n, G)
            r["top"][b, :n, heads] = (1 / total).view(n, G)
            size = (x.abs() @ k.abs().T * scale).masked_fill(~sees, 0.0)
            r["big"][b, :n, heads] = size.amax(1).view(n, G)
    return r


def tolerance(c, r):
    """How far an output may be off: the result is rounded once (half a step, eps / 2) and so
    is each weight; a score is a sum of D products in fp32 (each partial sum off by at most
    2^-23 of the largest magnitude, tensor cores truncating, and as much again a few times
    in the exponent's arithmetic), and a score off by e scales a weight by 1 +- e in the sum
    and in the total; a step of 16 keys truncates the weighted sum once more (2^-23), and
    the total is a sum of fp32 numbers, 128 and one a tile (2^-24 each); the exponential
    itself is good to 2^-21.  In fp16 a weight is held in units of 2^-11 of the row's largest, and
    what lies below the smallest normal number, weight or result, is off by at most 2^-25."""
    dtype, D = c["q"].dtype, c["q"].shape[3]
    keys = int(np.max(c["cache_len"])) + c["q"].shape[1]
    half = torch.finfo(dtype).eps / 2
    e = (D + 8) * 2.0 ** -23 * r["big"][..., None]
    sums = keys / 16 * 2.0 ** -23 + (KT + keys / KT) * 2.0 ** -24 + 2.0 ** -21
    tol = half * r["out"].abs() + (half * (1 + half) + 2 * e + sums) * r["mag"]
    if dtype == torch.float16:
        most = max(float(c[n].double().nan_to_num(0, 0, 0).abs().max()) for n in ("v_cache", "v_new"))
        tol = tol + keys * 2.0 ** -36 * most * r["top"][..., None] + 2.0 ** -25
    return tol * 1.001 + 1e-30


def lse_tolerance(c, r):
    """The errors above of a score and of a total."""
    keys = int(np.max(c["cache_len"])) + c["q"].shape[1]
    return ((c["q"].shape[3] + 8) * 2.0 ** -23 * r["big"] + (KT + keys / KT) * 2.0 ** -24
            + 2.0 ** -20 + 2.0 ** -22 * r["lse"].abs().nan_to_num(0, 0, 0))


SHARP = 18.0


def directed(c, ends, seed=0):
    """Sets q, k and v of `c` so that row y (node and head of the group) has score SHARP (use scale
    1) with the keys of every D-th tile, from tile y % D on, and 0 with all others: each
    tile carries a large part of some row.  With `ends` only the first and the last key of
    a tile, of a page and of the sequence count.  A tile's values share a sign in each column."""
    gen = torch.Generator().manual_seed(seed)
    B, N, Hq, D = c["q"].shape
    H, S = c["k_new"].shape[2], c["k_cache"].shape[1]
    G, dt = Hq // H, c["q"].dtype
    rows = (torch.arange(N)[:, None] * G + torch.arange(Hq)[None, :] % G) % D
    c["q"] = (torch.nn.functional.one_hot(rows, D) * SHARP).to(dt).repeat(B, 1, 1, 1)
    for name in ("k_cache", "k_new"):
        c[name] = torch.zeros_like(c[name])
    c["v_new"] = torch.randn(c["v_new"].shape, generator=gen).to(dt)
    for b in range(B):
        L = int(c["cache_len"][b])
        t = torch.arange(L)
        page = torch.full((L,), b) if c["table"] is None else torch.from_numpy(
            c["table"][b][t.numpy() // S].astype(np.int64))
        on = torch.ones(L, dtype=torch.bool)
        if ends:
            on = (t % KT == 0) | (t % KT == KT - 1) | (t == L - 1)
            if c["table"] is not None and S >= 64:
                on |= (t % S == 0) | (t % S == S - 1)
        k = torch.nn.functional.one_hot(t // KT % D, D) * on[:, None]
        sign = torch.randint(0, 2, (L // KT + 1, H, D), generator=gen) * 2 - 1
        v = sign[t // KT] * (0.75 + 0.5 * torch.rand((L, H, D), generator=gen))
        c["k_cache"][page, t % S] = k[:, None, :].to(dt).expand(L, H, D)
        c["v_cache"][page, t % S] = v.to(dt)
    return c


def parts_of_tiles(c, b, scale=1.0):
    """What each tile of sequence b's cache gives each output: [tiles, N, Hq, D]."""
    N, Hq, D = c["q"].shape[1:]
    H, S, L = c["k_new"].shape[2], c["k_cache"].shape[1], int(c["cache_len"][b])
    lse = attention(c, scale)["lse"]
    t = np.arange(L)
    page = torch.full((L,), b) if c["table"] is None else torch.from_numpy(
        c["table"][b][t // S].astype(np.int64))
    tiles = -(-L // KT)
    out = torch.zeros((tiles, N, Hq, D), dtype=torch.float64)
    G, n = Hq // H, int(c["n_nodes"][b])
    for h in range(H):
        k = c["k_cache"][page, t % S, h].double()
        v = c["v_cache"][page, t % S, h].double()
        for x in range(tiles):
            of = slice(x * KT, min(L, (x + 1) * KT))
            heads = slice(h * G, (h + 1) * G)
            s = c["q"][b, :n, heads].double() @ k[of].T * scale
            out[x, :n, heads] = torch.exp(s - lse[b, :n, heads, None]) @ v[of]
    return out
