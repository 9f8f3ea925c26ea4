"""Attention with capped, biased and windowed scores in 64 bits, and inputs for its tests.

s_j = u_j + slope (j - pos), u_j = softcap tanh(scale <q, K_j> / softcap) or scale <q, K_j>; key j takes part
where j < prefix or j <= pos and (window = 0 or j > pos - window).
"""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # a rounding, relative


def make(seed, lens, Hq, Hkv, D, BS, dtype, chunks=None, q_size=1.5, spare=3, width=None):
    """Sequences in a pool whose every other slot is NaN: slots past the ends, blocks that no table names."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, lens = len(lens), np.asarray(lens, np.int64)
    blocks = -(-lens // BS)
    NB = int(blocks.sum()) + spare
    perm = rng.permutation(NB).astype(np.int32)
    bt = np.full((B, max(1, int(blocks.max())) if width is None else width), -1, np.int32)
    at = 0
    for b in range(B):
        bt[b, :blocks[b]] = perm[at:at + blocks[b]]
        at += blocks[b]
    x = dict(lens=lens.tolist(), BS=BS)
    T = B if chunks is None else int(sum(chunks))
    x["start"] = list(range(B + 1)) if chunks is None else [0] + np.cumsum(chunks).tolist()
    x["q"] = (q_size * torch.randn((T, Hq, D), generator=g, device="cuda")).to(dtype)
    for name in ("k_cache", "v_cache"):
        pool = torch.full((NB, Hkv, BS, D), float("nan"), device="cuda", dtype=dtype)
        for b in range(B):
            for i in range(int(blocks[b])):
                n = min(BS, int(lens[b]) - i * BS)
                pool[int(bt[b, i]), :, :n] = torch.randn((Hkv, n, D), generator=g, device="cuda").to(dtype)
        x[name] = pool
    x["block_tables"] = torch.from_numpy(bt).cuda()
    x["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    x["q_start"] = torch.tensor(x["start"], dtype=torch.int32, device="cuda")
    return x


def slopes(Hq, seed=0):
    """Slopes of both signs and of many sizes, zero among them."""
    r = np.random.default_rng(seed)
    s = 2.0 ** r.uniform(-8, 0, Hq) * np.where(r.random(Hq) < 0.25, -0.02, 1.0)
    s[0] = 0.0
    return torch.from_numpy(s.astype(np.float32)).cuda()


def positions(L, n, window, prefix):
    """Keys that some of the last n queries see, ascending."""
    first = max(0, L - n - window + 1) if window > 0 else 0
    p = min(max(prefix, 0), L)
    return sorted(set(range(min(p, first))) | set(range(first, L)))


def hide(x, window=0, prefix=None):
    """NaN in every position that no query of its sequence sees."""
    for b, L in enumerate(x["lens"]):
        n = x["start"][b + 1] - x["start"][b]
        seen = set(positions(L, n, window, 0 if prefix is None else int(prefix[b])))
        for j in range(L):
            if j not in seen:
                blk = int(x["block_tables"][b, j // x["BS"]])
                x["k_cache"][blk, :, j % x["BS"]] = float("nan")
                x["v_cache"][blk, :, j % x["BS"]] = float("nan")


def reference(x, softcap=0.0, slopes=None, window=0, prefix=None, scale=0.0):
    """(out, tolerance) in float64, [T, Hq, D].

    The tolerance, per element, with A = sum_j softmax_j |V_j|, h the half step of the type, e = 2^-24:
    the final rounding h |out|; each weight rounded to the type h A (bf16 only: float32 weights are not);
    scores off by d, which moves numerator and denominator by d each, 2 d A, where d is D e max(sum |q k| scale) for
    the product's sum, 4 e max|t| for its scalings, 2^-21 softcap for the tanh (2^-23 of the cap, twice, and the
    division), 4 e max|bias|; sums over n keys, at most n / 16 + 64 roundings in a row of 2 e (the tensor core
    truncates) on numerator and denominator."""
    q, BS = x["q"], x["BS"]
    T, Hq, D = q.shape
    Hkv = x["k_cache"].shape[1]
    G = Hq // Hkv
    dt, f64 = q.dtype, torch.float64
    e = 2.0 ** -24
    sc = scale if scale > 0 else D ** -0.5
    out = torch.zeros((T, Hq, D), dtype=f64, device=q.device)
    tol = torch.zeros_like(out)
    for b, L in enumerate(x["lens"]):
        t0, t1 = x["start"][b], x["start"][b + 1]
        n = t1 - t0
        p = 0 if prefix is None else int(prefix[b])
        keys = positions(L, n, window, p)
        if not keys or n == 0:
            continue
        at = torch.tensor(keys, device=q.device)
        blk, slot = x["block_tables"][b].long()[at // BS], at % BS
        pos = torch.arange(L - n, L, device=q.device, dtype=f64).view(n, 1, 1)
        j = at.to(f64).view(1, 1, -1)
        hidden = j > pos
        if window > 0:
            hidden = hidden | (j <= pos - window)
        hidden = hidden & (j >= min(max(p, 0), L))
        for h in range(Hkv):
            k, v = x["k_cache"][blk, h, slot].to(f64), x["v_cache"][blk, h, slot].to(f64)
            qq = q[t0:t1, h * G:(h + 1) * G].to(f64)
            t = torch.einsum("ngd,jd->ngj", qq, k) * sc
            size = torch.einsum("ngd,jd->ngj", qq.abs(), k.abs()) * sc
            d = D * e * size.amax() + 4 * e * t.abs().amax()
            if softcap > 0:
                t = softcap * torch.tanh(t / softcap)
                d = d + 2.0 ** -21 * softcap
            if slopes is not None:
                bias = slopes[h * G:(h + 1) * G].to(f64).view(1, G, 1) * (j - pos)
                t = t + bias
                d = d + 4 * e * torch.where(hidden, 0.0, bias.abs()).amax()
            w = torch.softmax(t.masked_fill(hidden, -math.inf), -1)
            o, A = torch.einsum("ngj,jd->ngd", w, v), torch.einsum("ngj,jd->ngd", w, v.abs())
            rounded = HALF[dt] if dt == torch.bfloat16 else 0.0
            sums = 2 * 2 * e * (len(keys) / 16 + 64)
            out[t0:t1, h * G:(h + 1) * G] = o
            tol[t0:t1, h * G:(h + 1) * G] = HALF[dt] * o.abs() + (rounded + 2 * d + sums) * A * 1.01
    return out, tol


def check(got, ref, tol, rows=None):
    got = got.double()
    if rows is not None:
        got, ref, tol = got[rows], ref[rows], tol[rows]
    assert torch.isfinite(got).all()
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} out of tolerance, by up to {over.max():.3e}"
