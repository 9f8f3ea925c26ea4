"""Cases of decode attention over shared prefixes and of attention with capped, biased and windowed scores.

Operators: decode attention of sequences that share the leading blocks of their
tables ("shared"), decode attention with changed scores ("decode") and
chunked-prefill attention with changed scores ("prefill").  Each case is a dict of
plain values; `run` is one pass, in elementary torch operations where `own` is
false and through the library's entry points where it is true; `exact` evaluates
the definitions in 64 bits.

The score of key j for a query at position pos, t_j = D^-1/2 <q, K_j>:
u_j = softcap tanh(t_j / softcap) where softcap > 0, else t_j;
s_j = u_j + slopes[head] (j - pos) where there are slopes, else u_j.
Key j takes part where j < prefix, or j <= pos and (window = 0 or j > pos - window).
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # 64 requests behind one system prompt of 8192 tokens, their own turns of 64-1024
        dict(name="shared-prompt", kind="shared", groups=1, members=64, prefix=8192, lo=64, hi=1024, Hq=32, Hkv=8,
             D=128, BS=16, softcap=0.0, slopes=False),
        # 16 prompts of 1024-4096 tokens, each sampled 4 times in parallel: many small groups
        dict(name="shared-forks", kind="shared", groups=16, members=4, prefix=4096, lo=1, hi=512, Hq=32, Hkv=8, D=128,
             BS=16, softcap=0.0, slopes=False),
        # 32 questions to one document of 65536 tokens, capped scores and a distance bias
        dict(name="shared-document", kind="shared", groups=1, members=32, prefix=65536, lo=16, hi=1024, Hq=64, Hkv=8,
             D=128, BS=16, softcap=30.0, slopes=True),
        # two requests forked in three, a shard with two KV heads, short prompts: latency
        dict(name="shared-few", kind="shared", groups=2, members=3, prefix=256, lo=1, hi=100, Hq=8, Hkv=2, D=64, BS=16,
             softcap=0.0, slopes=False),
        # a serving batch of 64 requests, every score capped
        dict(name="decode-cap", kind="decode", dtype="bf16", B=64, Hq=32, Hkv=8, D=128, BS=16, lo=512, hi=4096,
             softcap=50.0, slopes=False, window=0, prefix=0),
        # few long documents with a distance bias
        dict(name="decode-slopes", kind="decode", dtype="bf16", B=8, Hq=64, Hkv=8, D=128, BS=16, lo=32768, hi=131072,
             softcap=0.0, slopes=True, window=0, prefix=0),
        # 512 requests in a layer with a sliding window that keeps each request's first tokens in sight
        dict(name="decode-window", kind="decode", dtype="bf16", B=512, Hq=32, Hkv=8, D=128, BS=16, lo=128, hi=4096,
             softcap=0.0, slopes=False, window=512, prefix=4),
        # one interactive request on a shard with two KV heads: latency
        dict(name="decode-one", kind="decode", dtype="bf16", B=1, Hq=8, Hkv=2, D=64, BS=16, lo=100, hi=300,
             softcap=50.0, slopes=True, window=0, prefix=0),
        # ragged lengths (empty ones too), odd heads and head size, float32
        dict(name="decode-odd", kind="decode", dtype="f32", B=37, Hq=21, Hkv=3, D=80, BS=32, lo=0, hi=1500,
             softcap=20.0, slopes=True, window=300, prefix=7),
        # prefill chunks of 16 requests, every score capped
        dict(name="prefill-cap", kind="prefill", B=16, n=512, Hq=32, Hkv=8, D=128, BS=16, lo=512, hi=4096,
             softcap=50.0, slopes=False, window=0, prefix=0),
        # chunks far into long documents in a layer with a sliding window, the first tokens in sight
        dict(name="prefill-window", kind="prefill", B=4, n=2048, Hq=64, Hkv=8, D=128, BS=16, lo=16384, hi=32768,
             softcap=0.0, slopes=True, window=1024, prefix=100),
        # one request's short first chunk, which sees all of itself
        dict(name="prefill-few", kind="prefill", B=1, n=37, Hq=8, Hkv=2, D=128, BS=16, lo=37, hi=60, softcap=30.0,
             slopes=False, window=0, prefix=60),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "decode", "decode", "prefill"])
    c = dict(kind=kind, Hkv=rng.randint(1, 12), BS=rng.choice([16, 16, 32, 48, 64]),
             softcap=rng.choice([0.0, 0.0, round(rng.uniform(5.0, 60.0), 1)]), slopes=rng.random() < 0.4)
    if kind == "shared":
        c["D"] = rng.choice([64, 128, 128])
        c["Hq"] = c["Hkv"] * rng.randint(1, 16)
        c["groups"] = _log(rng, 1, 64)
        c["members"] = _log(rng, 1, max(2, 256 // c["groups"]))
        B, row = c["groups"] * c["members"], c["Hkv"] * c["D"]
        # the prefixes' and the rest's cache, and every query's work
        most = min(65536, int(1.5e8 / (c["groups"] * row)), int(2.5e8 / (B * c["Hq"] * c["D"] / 16)))
        c["prefix"] = max(c["BS"], _log(rng, c["BS"], max(c["BS"] + 1, most)))
        c["hi"] = _log(rng, 1, max(2, min(4096, int(5e7 / (B * row)))))
        c["lo"] = rng.randint(1, c["hi"])
        return c
    c["window"] = rng.choice([0, 0, _log(rng, 1, 4096)])
    c["prefix"] = rng.choice([0, 0, _log(rng, 1, 512)])
    c["B"] = _log(rng, 1, 256 if kind == "decode" else 32)
    if kind == "decode":
        c["dtype"] = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        c["D"] = rng.choice([64, 128, 128, 16 * rng.randint(1, 8)])
        c["Hq"] = c["Hkv"] * rng.randint(1, 16)
        most = min(131072, int((1.5e8 if c["dtype"] == "bf16" else 3e7) / (c["B"] * c["Hkv"] * c["D"])))
        c["hi"] = max(1, _log(rng, 1, max(2, most)))
        c["lo"] = rng.randint(0, c["hi"])
        return c
    c["D"] = 128
    c["Hq"] = c["Hkv"] * rng.randint(1, 8)
    c["n"] = _log(rng, 1, max(2, min(2048, int(3e7 / (c["B"] * c["Hq"] * c["D"])))))
    most = min(32768, int(2e10 / (c["B"] * c["n"] * c["Hq"] * c["D"])), int(1e8 / (c["B"] * c["Hkv"] * c["D"])))
    c["lo"] = _log(rng, c["n"], max(c["n"] + 1, most))
    c["hi"] = rng.randint(c["lo"], max(c["lo"], most))
    return c


# ------------------------------------------------------------------ inputs
def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _pool(nb, c, g, dt):
    """One pool [nb, Hkv, BS, D]: normal, with a spread of channel sizes, made in pieces."""
    ch = torch.exp(0.4 * torch.randn((c["Hkv"], 1, c["D"]), generator=g, device="cuda"))
    pool = torch.empty((nb, c["Hkv"], c["BS"], c["D"]), dtype=dt, device="cuda")
    step = max(1, (1 << 28) // (c["Hkv"] * c["BS"] * c["D"]))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        pool[i:i + n] = torch.randn((n, c["Hkv"], c["BS"], c["D"]), generator=g, device="cuda") * ch
    return pool


def _slopes(Hq, r):
    """A geometric row of slopes, one per query head, a little off for each seed."""
    s = 2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq) * r.uniform(0.8, 1.2, Hq)
    return _cuda(s.astype(np.float32))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    BS = c["BS"]
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    dt = _DT[c.get("dtype", "bf16")]
    q_size = 5.0 if c["softcap"] else 1.5  # capped scores are large ones
    if c["kind"] == "shared":
        N, M = c["groups"], c["members"]
        # the prompts' lengths: the longest, and others from a quarter of it on, in whole blocks
        pre = np.maximum(1, r.randint(max(1, c["prefix"] // 4), c["prefix"] + 1, N) // BS)
        pre[0] = max(1, c["prefix"] // BS)
        tail = r.randint(c["lo"], c["hi"] + 1, N * M)
        lens = np.repeat(pre, M) * BS + tail
        own_blocks = -(-tail // BS)
        total = int(pre.sum() + own_blocks.sum())
        nb = total + total // 16 + 1
        perm = r.permutation(nb).astype(np.int32)
        bt = np.full((N * M, int((-(-lens // BS)).max())), -1, np.int32)
        at = 0
        for i in range(N):
            shared = perm[at:at + pre[i]]
            at += pre[i]
            for b in range(i * M, (i + 1) * M):
                bt[b, :pre[i]] = shared
                bt[b, pre[i]:pre[i] + own_blocks[b]] = perm[at:at + own_blocks[b]]
                at += own_blocks[b]
        s["group_start"] = _cuda((np.arange(N + 1) * M).astype(np.int32))
        s["shared_lens"] = _cuda((pre * BS).astype(np.int32))
        s["pre"] = (pre * BS).tolist()
        B = T = N * M
    else:
        B = T = c["B"]
        lens = r.randint(c["lo"], c["hi"] + 1, B)
        if c["kind"] == "prefill":  # the ragged chunks belong to the case: outputs of two seeds have one shape
            rc = np.random.RandomState(B * 131 + c["n"])
            n = rc.randint((c["n"] + 1) // 2, c["n"] + 1, B)
            lens = np.maximum(lens, n)
            s["q_start"] = _cuda(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
            T = int(n.sum())
            s["n"] = n.tolist()
        blocks = -(-lens // BS)
        total = int(blocks.sum())
        nb = total + total // 16 + 1
        bt = np.full((B, max(1, -(-max(c["hi"], int(lens.max())) // BS))), -1, np.int32)
        perm = r.permutation(nb).astype(np.int32)
        at = np.concatenate([[0], np.cumsum(blocks)])
        for b in range(B):
            bt[b, :blocks[b]] = perm[at[b]:at[b + 1]]
        s["prefix_lens"] = _cuda(r.randint(0, c["prefix"] + 1, B).astype(np.int32)) if c["prefix"] else None
    s["lens"] = lens.tolist()
    s["seq_lens"], s["block_tables"] = _cuda(lens.astype(np.int32)), _cuda(bt)
    s["slopes"] = _slopes(c["Hq"], r) if c["slopes"] else None
    s["q"] = (q_size * torch.randn((T, c["Hq"], c["D"]), generator=g, device="cuda")).to(dt)
    s["k_cache"], s["v_cache"] = _pool(nb, c, g, dt), _pool(nb, c, g, dt)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    return {"shared": _shared, "decode": _decode, "prefill": _prefill}[kind](state)


def _own(kind, s):
    import paged_kv_decode_table_gb300 as pkv
    c = s["case"]
    base = (s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"])
    if kind == "shared":
        return pkv.paged_decode_attention_shared(*base, s["group_start"], s["shared_lens"], softcap=c["softcap"],
                                                 slopes=s["slopes"], status=s["status"])
    more = dict(softcap=c["softcap"], slopes=s["slopes"], window=c["window"], prefix_lens=s["prefix_lens"],
                status=s["status"])
    if kind == "decode":
        return pkv.paged_decode_attention_scored(*base, **more)
    return pkv.paged_prefill_attention_scored(*base, s["q_start"], **more)


def _gather(pool, ids):
    """Blocks ids [.., n] of a pool in float32, as [.., Hkv, n * BS, D]."""
    x = pool[ids].to(torch.float32).transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _score(t, c, slopes, key, pos):
    """Products <q, K> [.., Hkv, G, .., keys] to scores; slopes [Hkv, G, 1, ..]; key and pos broadcast to t."""
    t.mul_(c["D"] ** -0.5)
    if c["softcap"]:
        t.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    if slopes is not None:
        t.add_(slopes * (key - pos).to(torch.float32))
    return t


def _seen(c, key, pos, prefix):
    m = key <= pos
    if c["window"]:
        m = m & (key > pos - c["window"])
    return m if prefix is None else m | (key < prefix)


def _softmax_(w):
    """exp(w - max) in place and its sum; a row without keys gives zeros."""
    m = w.amax(-1, keepdim=True)
    w.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    return w, w.sum(-1, keepdim=True)


def _decode(s):
    c, q, lens = s["case"], s["q"], s["seq_lens"].long()
    B, Hq, D = q.shape
    Hkv = c["Hkv"]
    ids = s["block_tables"].long().clamp_min(0)
    w = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), _gather(s["k_cache"], ids).transpose(-1, -2))
    key = torch.arange(w.shape[-1], device=q.device)[None, :]
    pos = lens[:, None] - 1
    prefix = None if s["prefix_lens"] is None else torch.minimum(s["prefix_lens"].long(), lens)[:, None]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hkv, -1, 1)
    _score(w, c, slopes, key[:, None, None], pos[:, None, None])
    w.masked_fill_(~_seen(c, key, pos, prefix)[:, None, None], -math.inf)
    w, total = _softmax_(w)
    o = torch.matmul(w, _gather(s["v_cache"], ids))
    return torch.where(total > 0, o / total, 0.0).view(B, Hq, D).to(q.dtype)


def _prefill(s):
    c, q = s["case"], s["q"]
    Hkv, G, D = c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hkv, G, 1, 1)
    out = torch.empty_like(q)
    t0 = 0
    for b, (n, L) in enumerate(zip(s["n"], s["lens"])):
        ids = s["block_tables"][b, :-(-L // c["BS"])].long()
        key, pos = torch.arange(L, device=q.device)[None, :], torch.arange(L - n, L, device=q.device)[:, None]
        mask = ~_seen(c, key, pos, None if s["prefix_lens"] is None else s["prefix_lens"][b])
        x = q[t0:t0 + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)
        K, V = _gather(s["k_cache"], ids)[:, None, :L], _gather(s["v_cache"], ids)[:, None, :L]
        w, total = _softmax_(_score(torch.matmul(x, K.transpose(-1, -2)), c, slopes, key, pos).masked_fill_(mask, -math.inf))
        out[t0:t0 + n] = (torch.matmul(w, V) / total).permute(2, 0, 1, 3).reshape(n, -1, D).to(q.dtype)
        t0 += n
    return out


def _shared(s):
    c, q = s["case"], s["q"]
    Hkv, G, D, M, BS = c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["members"], c["BS"]
    slopes = None if s["slopes"] is None else s["slopes"].view(Hkv, G, 1)
    out = torch.empty_like(q)
    for i, P in enumerate(s["pre"]):
        b0, longest = i * M, max(s["lens"][i * M:(i + 1) * M])
        lens = s["seq_lens"][b0:b0 + M].long()[:, None, None, None]
        x = q[b0:b0 + M].float().view(M, Hkv, G, D)
        # the prefix, once for all members: [Hkv, members * G, D] x [Hkv, P, D]
        ids = s["block_tables"][b0, :P // BS].long()
        w0 = torch.matmul(x.transpose(0, 1).reshape(Hkv, M * G, D), _gather(s["k_cache"], ids).transpose(-1, -2))
        w0 = w0.view(Hkv, M, G, P).transpose(0, 1)
        w0 = _score(w0, c, slopes, torch.arange(P, device=q.device), lens - 1)
        # what each member has of its own
        ids1 = s["block_tables"][b0:b0 + M, P // BS:-(-longest // BS)].long().clamp_min(0)
        w1 = torch.matmul(x, _gather(s["k_cache"], ids1).transpose(-1, -2))
        key = P + torch.arange(w1.shape[-1], device=q.device)
        w1 = _score(w1, c, slopes, key, lens - 1).masked_fill_(key >= lens, -math.inf)
        m = torch.maximum(w0.amax(-1, keepdim=True), w1.amax(-1, keepdim=True))
        w0, w1 = w0.sub_(m).exp_(), w1.sub_(m).exp_()
        o = torch.matmul(w0.transpose(0, 1).reshape(Hkv, M * G, P), _gather(s["v_cache"], ids))
        o = o.view(Hkv, M, G, D).transpose(0, 1) + torch.matmul(w1, _gather(s["v_cache"], ids1))
        total = w0.sum(-1, keepdim=True) + w1.sum(-1, keepdim=True)
        out[b0:b0 + M] = (o / total).reshape(M, -1, D).to(q.dtype)
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    es = 4 if c.get("dtype") == "f32" else 2
    row, mid = 2 * c["Hkv"] * c["D"] * es, (c["lo"] + c["hi"]) / 2  # one position's K and V; a length
    if c["kind"] == "shared":
        B = c["groups"] * c["members"]
        pre = c["prefix"] * (1 + (c["groups"] - 1) * 0.625)  # of all groups
        return dict(bytes=pre * row + B * mid * row + 2 * B * c["Hq"] * c["D"] * es + (pre + B * mid) / c["BS"] * 4,
                    flops=4 * c["Hq"] * c["D"] * (pre * c["members"] + B * mid))
    pf = c["prefix"] / 2
    if c["kind"] == "decode":
        seen = mid if not c["window"] else sum(
            min(x, c["window"] + min(pf, max(0, x - c["window"])))
            for x in (c["lo"] + (c["hi"] - c["lo"]) * (i + 0.5) / 16 for i in range(16))) / 16
        return dict(bytes=c["B"] * (seen * row + seen / c["BS"] * 4 + 2 * c["Hq"] * c["D"] * es),
                    flops=4 * c["B"] * seen * c["Hq"] * c["D"])
    n = 0.75 * c["n"] if c["n"] > 1 else 1.0
    mid = max(mid, n)
    read = mid if not c["window"] else min(mid, c["window"] + n + pf)
    if c["window"]:
        seen = min(mid - n / 2, c["window"]) + min(pf, max(0.0, mid - n / 2 - c["window"]))
    else:
        seen = max(mid - n / 2, min(pf, mid))
    return dict(bytes=c["B"] * (read * row + 2 * n * c["Hq"] * c["D"] * es + read / c["BS"] * 4),
                flops=4 * c["B"] * n * seen * c["Hq"] * c["D"])


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    c = case
    if c["kind"] == "prefill" and 4.0 * c["B"] * c["n"] * c["hi"] * c["Hq"] * c["D"] > 6e12:
        return None
    s = prepare(c, seed)
    f64 = torch.float64
    G, BS = c["Hq"] // c["Hkv"], c["BS"]
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    start = s["q_start"].tolist() if "q_start" in s else list(range(len(s["lens"]) + 1))
    pre = s.get("prefix_lens")
    pre = [0] * len(s["lens"]) if pre is None else pre.tolist()
    window = c.get("window", 0)
    for b, L in enumerate(s["lens"]):
        if L == 0:
            continue
        rows = slice(start[b], start[b + 1])
        n = start[b + 1] - start[b]
        pos = torch.arange(L - n, L, device="cuda", dtype=f64).view(n, 1, 1)
        if window:  # the positions that some row may see
            first = max(0, L - n - window + 1)
            p = min(pre[b], L, first)
            at = torch.cat([torch.arange(p, device="cuda"), torch.arange(first, L, device="cuda")])
        else:
            at = torch.arange(L, device="cuda")
        blk, slot = s["block_tables"][b].long()[at // BS], at % BS
        j = at.to(f64).view(1, 1, -1)
        hidden = j > pos
        if window:
            hidden = hidden | (j <= pos - window)
        if pre[b]:
            hidden = hidden & (j >= pre[b])
        for h in range(c["Hkv"]):
            heads = slice(h * G, (h + 1) * G)
            k, v = s["k_cache"][blk, h, slot].to(f64), s["v_cache"][blk, h, slot].to(f64)
            z = torch.einsum("ngd,jd->ngj", s["q"][rows, heads].to(f64), k) / math.sqrt(c["D"])
            if c["softcap"]:
                z = c["softcap"] * torch.tanh(z / c["softcap"])
            if s["slopes"] is not None:
                z = z + s["slopes"][heads].to(f64).view(1, G, 1) * (j - pos)
            z = torch.softmax(z.masked_fill(hidden, -math.inf), dim=-1)
            out[rows, heads] = torch.einsum("ngj,jd->ngd", z, v)
    return out
