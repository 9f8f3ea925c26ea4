"""Plain implementations of the 8-bit cache operators for the tests.

`store` follows the format's float32 formula operation by operation (its result
is compared bit for bit); everything else is float64 on the CPU.
"""
import math

import numpy as np
import torch

DT = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
QMAX = {"e4m3": 448.0, "i8": 127.0}
U24 = 2.0 ** -24  # half a float32 step, relative


def store(x, fmt):
    """x [..., D] (any float type) -> (values in the 8-bit type, float32 scales), on the CPU."""
    x = x.detach().cpu().float()
    inv_q = np.float32(1.0) / np.float32(QMAX[fmt])
    scale = (x.abs().amax(-1) * torch.tensor(inv_q)).clamp_min(2.0 ** -64)
    y = x * (1.0 / scale)[..., None]
    if fmt == "i8":
        vals = y.round().clamp(-127, 127).to(torch.int8)
    else:
        vals = y.clamp(-448, 448).to(torch.float8_e4m3fn)
    bad = ~torch.isfinite(x).all(-1)
    vals.view(torch.uint8)[bad] = 0
    scale[bad] = math.nan
    return vals, scale


def half_step(x, scale, fmt):
    """How far one rounding to the 8-bit type moves x (float64) at most."""
    s = scale[..., None]
    if fmt == "i8":
        return (s / 2).expand_as(x)
    return torch.maximum(x.abs() / 16, s * 2.0 ** -10)


def numbers(vals, scale):
    """What the cache stands for, float64."""
    return vals.detach().cpu().float().double() * scale.detach().cpu().double()[..., None]


def random_cache(nb, Hkv, BS, D, fmt, gen):
    """Two pools and their scales with uneven channels and rows, on the CPU."""
    out = []
    for _ in range(2):
        x = torch.randn(nb, Hkv, BS, D, generator=gen) * torch.exp(0.5 * torch.randn(Hkv, 1, D, generator=gen))
        x *= torch.exp(0.7 * torch.randn(nb, Hkv, BS, 1, generator=gen))
        out.append(store(x, fmt))
    (k, ks), (v, vs) = out
    return k, v, ks, vs


def tables(lens, BS, gen, spare=3, width=None):
    need = [-(-int(L) // BS) for L in lens]
    nb = max(1, sum(need) + spare)
    perm = torch.randperm(nb, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), width or max(1, max(need, default=1))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    return bt, nb


def attention(q, k, v, ks, vs, bt, lens, scale=None, dtype="f32"):
    """(out, tolerance) in float64 for decode attention over the cache (all on the CPU).

    The tolerance adds up, per output element, with W = sum_j p_j |v_j| and
    S = max_j scale * sum_i |q_i k_ij|:
      scores      D + 8 float32 roundings of terms whose magnitudes sum to S move
                  a score by at most (D + 8) 2^-24 S, hence a weight (and the
                  normaliser) by that much relatively: 2 (D + 8) 2^-24 S W;
      exponentials and scales  16 roundings, and an exponent shifted by a V scale's
                  logarithm (up to 64) is rounded at that size, in the weight and in
                  the normaliser: 144 * 2^-24 W;
      sums        L terms and the normaliser's L terms: 2 L 2^-24 W;
      weights     a float16 weight is off by 2^-11 of itself where it is normal
                  (bf16 outputs only; float32 outputs carry a second float16 with
                  the remainder, 2^-22), and below that by at most 2^-25 of the
                  largest weight, which multiplies sum_j |v numbers|;
      output      one rounding: 2^-8 |out| (bf16) or 2^-24 |out| (float32).
    """
    q = q.detach().cpu().double()
    B, Hq, D = q.shape
    Hkv, BS = k.shape[1], k.shape[2]
    G = Hq // Hkv
    scale = scale or D ** -0.5
    k, v = k.float(), v.float()
    out, tol = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        ids = bt[b, :-(-L // BS)].long()
        for h in range(Hkv):
            kk = numbers(k[ids, h].reshape(-1, D)[:L], ks[ids, h].reshape(-1)[:L])
            vn = v[ids, h].double().reshape(-1, D)[:L]
            vsc = vs[ids, h].double().reshape(-1)[:L]
            vv = vn * vsc[:, None]
            qq = q[b, h * G:(h + 1) * G]
            s = scale * qq @ kk.T
            p = torch.softmax(s, -1)
            o = p @ vv
            S = scale * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True)
            W = p @ vv.abs()
            rel = (2 * (D + 8) * S + 144 + 2 * L) * U24 + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22)
            tiny = 2.0 ** -25 * (p * vsc).amax(-1, keepdim=True) * vn.abs().sum(0)
            out[b, h * G:(h + 1) * G] = o
            tol[b, h * G:(h + 1) * G] = rel * W + tiny + (2.0 ** -8 if dtype == "bf16" else U24) * o.abs() + 1e-37
    return out, tol


def norm_rope(x, w, eps, pos, inv_freq, interleaved):
    """(y, reach): x [T, H, D] normalised and rotated in float64, and the sum of
    the magnitudes that were added into each element."""
    x = x.detach().cpu().double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.detach().cpu().double()
    y, reach = x.clone(), x.abs()
    half = len(inv_freq)
    if half == 0:
        return y, reach
    # whole turns taken off with integers, so that far positions stay exact
    ang = torch.tensor([[2 * math.pi * math.fmod(p * (f / (2 * math.pi)), 1.0) for f in inv_freq] for p in pos],
                       dtype=torch.float64)[:, None, :]
    cos, sin = torch.cos(ang), torch.sin(ang)
    ia = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    ic = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, c = x[..., ia], x[..., ic]
    y[..., ia], y[..., ic] = a * cos - c * sin, c * cos + a * sin
    reach = reach.clone()
    reach[..., ia] = reach[..., ic] = a.abs() + c.abs()
    return y, reach
