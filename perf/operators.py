"""Cases of the 8-bit KV cache operators and of the fused query/key preparation.

Operators: decode attention over an 8-bit paged cache ("attention"), the append
that quantises ("append"), the append followed by reading the written blocks
back ("store"), reading blocks back ("read"), and the pass that normalises and
rotates queries and keys and appends keys and values ("prepare").  Each case is
a dict of plain values; `run` is one pass, in elementary torch operations where
`own` is false and through the library's entry points where it is true;
`exact` evaluates the definitions in 64 bits.

8-bit rows: one float32 scale per (token, KV head) row of D values,
scale = max(amax * (1 / Q), 2^-64) with Q = 448 (e4m3) or 127 (int8), and
value = round-to-nearest-even(x * (1 / scale)) in that type, each operation in
float32.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_FMT = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}
_QMAX = {"e4m3": 448.0, "i8": 127.0}
_MIN_SCALE = 2.0 ** -64
_EPS = 1e-6


def listed():
    return [
        # a serving batch of 64 requests with grouped heads, the cache in e4m3
        dict(name="attention-b64", kind="attention", fmt="e4m3", dtype="bf16", B=64, Hq=32, Hkv=8, D=128, BS=16,
             lo=512, hi=4096),
        # few requests with long documents: the cache split over every SM
        dict(name="attention-long", kind="attention", fmt="i8", dtype="bf16", B=8, Hq=64, Hkv=8, D=128, BS=16,
             lo=32768, hi=131072),
        # one interactive request on a shard with two KV heads: latency
        dict(name="attention-one", kind="attention", fmt="e4m3", dtype="bf16", B=1, Hq=8, Hkv=2, D=64, BS=16,
             lo=100, hi=300),
        # ragged lengths (empty ones too), odd heads and head size, float32
        dict(name="attention-odd", kind="attention", fmt="i8", dtype="f32", B=37, Hq=21, Hkv=3, D=80, BS=32,
             lo=0, hi=1500),
        # one decode step of a batch of 64: norm, rotation, quantising append
        dict(name="prepare-decode", kind="prepare", fmt="e4m3", dtype="bf16", B=64, n=1, Hq=32, Hkv=8, D=128, BS=16,
             lo=512, hi=4096, rot=128, interleaved=False),
        # prefill chunks of 16 requests into an unquantised cache
        dict(name="prepare-chunk", kind="prepare", fmt="none", dtype="bf16", B=16, n=512, Hq=32, Hkv=8, D=128, BS=16,
             lo=512, hi=4096, rot=128, interleaved=False),
        # one request at a far position, half of each head rotated, pairs interleaved
        dict(name="prepare-one", kind="prepare", fmt="e4m3", dtype="f32", B=1, n=1, Hq=8, Hkv=2, D=64, BS=16,
             lo=100000, hi=131072, rot=32, interleaved=True),
        # the append of a batch of 512 decode steps
        dict(name="append-decode", kind="append", fmt="e4m3", dtype="bf16", B=512, n=1, Hkv=8, D=128, BS=16,
             lo=128, hi=1024),
        # prefill chunks of 16 requests stored in int8 and read back for their attention
        dict(name="store-chunk", kind="store", fmt="i8", dtype="bf16", B=16, n=512, Hkv=8, D=128, BS=16,
             lo=512, hi=4096),
        # a few new tokens of one request stored and read back
        dict(name="store-few", kind="store", fmt="e4m3", dtype="bf16", B=1, n=5, Hkv=2, D=80, BS=32, lo=5, hi=300),
        # the cached prefixes of a batch of 64 read back
        dict(name="read-b64", kind="read", fmt="e4m3", dtype="bf16", blocks=9216, Hkv=8, D=128, BS=16),
        # one short prefix read back in float32
        dict(name="read-few", kind="read", fmt="i8", dtype="f32", blocks=37, Hkv=3, D=80, BS=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "prepare", "prepare", "append", "store", "read"])
    c = dict(kind=kind, fmt=rng.choice(["e4m3", "i8"]), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
             Hkv=rng.randint(1, 12), D=16 * rng.randint(1, 8), BS=rng.choice([16, 16, 32, 48, 64]))
    if kind == "attention":
        c["Hq"] = c["Hkv"] * rng.randint(1, 16)
        c["B"] = _log(rng, 1, 256)
        most = min(131072, int(2e8 / (c["B"] * c["Hkv"] * c["D"])))
        c["hi"] = max(1, _log(rng, 1, max(2, most)))
        c["lo"] = rng.randint(0, c["hi"])
        return c
    if kind == "read":
        c["blocks"] = _log(rng, 1, max(2, int(1.2e8 / (c["Hkv"] * c["D"] * c["BS"]))))
        return c
    c["B"] = _log(rng, 1, 512)
    c["n"] = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, min(2048, int(8e6 / (c["B"] * c["Hkv"] * c["D"])))))
    c["lo"] = _log(rng, c["n"], 131072)
    c["hi"] = rng.randint(c["lo"], 131072)
    if kind == "prepare":
        c["fmt"] = rng.choice(["e4m3", "none"])
        c["Hq"] = c["Hkv"] * rng.randint(1, 8)
        c["rot"] = 2 * rng.randint(1, c["D"] // 2)
        c["interleaved"] = rng.random() < 0.5
    elif kind == "append":
        c["fmt"] = "e4m3"
    else:
        c["dtype"] = "bf16"
    return c


# ------------------------------------------------------------------ inputs
def _quantise(x, fmt):
    """Rows of x (float32, last dimension) in 8 bits: (values, scales)."""
    scale = (x.abs().amax(-1) * (1.0 / _QMAX[fmt])).clamp_min(_MIN_SCALE)
    y = x * (1.0 / scale)[..., None]
    if fmt == "i8":
        return y.round().clamp(-127.0, 127.0).to(torch.int8), scale
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _rows(shape, g, channels):
    """Keys or values of a cache: normal, with a wide spread of channel sizes and of row sizes."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= channels
    return x * torch.exp(0.4 * torch.randn(shape[:-1], generator=g, device="cuda", dtype=torch.float32))[..., None]


def _pool(nb, c, g):
    """One 8-bit pool [nb, Hkv, BS, D] and its scales, made in pieces."""
    ch = torch.exp(0.5 * torch.randn((c["Hkv"], 1, c["D"]), generator=g, device="cuda", dtype=torch.float32))
    vals = torch.empty((nb, c["Hkv"], c["BS"], c["D"]), dtype=_FMT[c["fmt"]], device="cuda")
    scales = torch.empty((nb, c["Hkv"], c["BS"]), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (c["Hkv"] * c["BS"] * c["D"]))
    for i in range(0, nb, step):
        n = min(step, nb - i)
        vals[i:i + n], scales[i:i + n] = _quantise(_rows((n, c["Hkv"], c["BS"], c["D"]), g, ch), c["fmt"])
    return vals, scales


def _lens(c, seed):
    r = np.random.RandomState(seed % (1 << 32))
    lens = r.randint(c["lo"], c["hi"] + 1, c["B"]).astype(np.int64)
    return lens, r


def _chunks(c, lens):
    """New tokens of each sequence and its length after them.  The ragged counts, and where in a block each
    sequence's first new token falls, belong to the case, so that the outputs of two seeds have one shape."""
    r = np.random.RandomState(c["B"] * 131 + c["n"])
    n = r.randint((c["n"] + 1) // 2, c["n"] + 1, c["B"]) if c["n"] > 1 else np.ones_like(lens)
    full = n + r.randint(0, c["BS"], c["B"])
    return n, np.maximum(full, lens - (lens - full) % c["BS"])


def _tables(first, last, r, BS, hi, spare):
    """Block tables that hold logical blocks first[b] .. last[b] - 1 of each sequence, in random order
    over a pool with `spare` unused blocks; the other entries are -1."""
    total = int((last - first).sum())
    nb = max(1, total + spare)
    perm = r.permutation(nb)[:total].astype(np.int32)
    width = max(1, -(-hi // BS))
    bt = np.full((len(first), width), -1, np.int32)
    j = np.arange(width)[None, :]
    bt[(j >= first[:, None]) & (j < last[:, None])] = perm
    return bt, nb, perm


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = _DT[c["dtype"]]
    s = dict(case=c, status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["kind"] == "read":
        nb = c["blocks"] + c["blocks"] // 8
        s["k_cache"], s["k_scale"] = _pool(nb, c, g)
        s["v_cache"], s["v_scale"] = _pool(nb, c, g)
        s["blocks"] = _cuda(np.random.RandomState(seed % (1 << 32)).permutation(nb)[:c["blocks"]].astype(np.int32))
        return s
    lens, r = _lens(c, seed)
    BS = c["BS"]
    if c["kind"] == "attention":
        bt, nb, _ = _tables(np.zeros_like(lens), -(-lens // BS), r, BS, c["hi"], c["B"])
        s["q"] = (1.5 * torch.randn((c["B"], c["Hq"], c["D"]), generator=g, device="cuda")).to(dt)
    else:  # only the blocks that the new tokens fall into are in the pool
        n, lens = _chunks(c, lens)
        bt, nb, perm = _tables((lens - n) // BS, -(-lens // BS), r, BS, max(c["hi"], c["n"] + BS), c["B"] // 4)
        T = int(n.sum())
        if c["n"] > 1:
            s["q_start"] = _cuda(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
        ch = torch.exp(0.5 * torch.randn((c["Hkv"], c["D"]), generator=g, device="cuda", dtype=torch.float32))
        s["blocks"] = _cuda(perm)
        if c["kind"] == "prepare":
            # what the projection leaves: queries, keys and values of a token in one row
            Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
            x = _rows((T, Hq + 2 * Hkv, D), g, 1.0)
            x[:, Hq:Hq + Hkv] *= ch
            x = x.to(dt)
            s["q"], s["k_new"], s["v_new"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            s["q_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
            s["k_weight"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt)
            s["freqs"] = _cuda(_turns(c["rot"]))
        else:
            s["k_new"] = _rows((T, c["Hkv"], c["D"]), g, ch).to(dt)
            s["v_new"] = _rows((T, c["Hkv"], c["D"]), g, 1.0).to(dt)
    s["block_tables"], s["seq_lens"] = _cuda(bt), _cuda(lens.astype(np.int32))
    if c["fmt"] == "none":
        s["k_cache"] = torch.randn((nb, c["Hkv"], BS, c["D"]), generator=g, device="cuda").to(dt)
        s["v_cache"] = torch.randn((nb, c["Hkv"], BS, c["D"]), generator=g, device="cuda").to(dt)
    else:
        s["k_cache"], s["k_scale"] = _pool(nb, c, g)
        s["v_cache"], s["v_scale"] = _pool(nb, c, g)
    return s


def _turns(rot):
    """The rotation plan: turns per position of each pair, in units of 2^-64 (base 10000)."""
    t = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) / (2.0 * math.pi)
    return np.array([int(v * 2.0 ** 64) for v in t], dtype=np.uint64).view(np.int64)


# ------------------------------------------------------------------ one pass
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(kind, state)
    if kind == "attention":
        return _attention(state)
    if kind == "read":
        return _read(state)
    return _write(kind, state)


def _own(kind, s):
    import paged_kv_decode_table_gb300 as pkv
    if kind == "attention":
        return pkv.paged_decode_attention_q8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                             s["block_tables"], s["seq_lens"], status=s["status"])
    if kind == "read":
        return pkv.kv_read_blocks_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["blocks"],
                                     dtype=_DT[s["case"]["dtype"]], status=s["status"])
    if kind == "prepare":
        q = pkv.qk_norm_rope_append(s["q"], s["k_new"], s["v_new"], s["q_weight"], s["k_weight"], _EPS, s["freqs"],
                                    s["k_cache"], s["v_cache"], s["block_tables"], s["seq_lens"],
                                    q_start=s.get("q_start"), k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                                    interleaved=s["case"]["interleaved"], status=s["status"])
        return _caches(s) + (q,)
    if "q_start" in s:
        pkv.kv_append_chunk_q8(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                               s["block_tables"], s["seq_lens"], s["q_start"], status=s["status"])
    else:
        pkv.kv_append_q8(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                         s["block_tables"], s["seq_lens"], status=s["status"])
    if kind == "append":
        return _caches(s)
    return pkv.kv_read_blocks_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["blocks"],
                                 dtype=_DT[s["case"]["dtype"]], status=s["status"])


def _caches(s):
    if "k_scale" in s:
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    return s["k_cache"], s["v_cache"]


def _gather(pool, scale, ids):
    """Blocks `ids` of an 8-bit pool in float32."""
    x = pool.view(torch.uint8)[ids].view(pool.dtype).to(torch.float32)
    return x.mul_(scale[ids][..., None])


def _attention(s):
    q, lens = s["q"], s["seq_lens"].long()
    B, Hq, D = q.shape
    Hkv, BS = s["k_cache"].shape[1], s["k_cache"].shape[2]
    ids = s["block_tables"].long().clamp_min(0)
    K = _gather(s["k_cache"], s["k_scale"], ids).transpose(1, 2).reshape(B, Hkv, -1, D)
    w = torch.matmul(q.float().view(B, Hkv, Hq // Hkv, D), K.transpose(-1, -2)).mul_(D ** -0.5)
    del K
    past = torch.arange(w.shape[-1], device=q.device)[None, :] >= lens[:, None]
    w.masked_fill_(past[:, None, None, :], -math.inf)
    m = w.amax(-1, keepdim=True)
    w.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = w.sum(-1, keepdim=True)
    V = _gather(s["v_cache"], s["v_scale"], ids).transpose(1, 2).reshape(B, Hkv, -1, D)
    o = torch.matmul(w, V)
    return torch.where(total > 0, o / total, 0.0).view(B, Hq, D).to(q.dtype)


def _read(s):
    dt, ids = _DT[s["case"]["dtype"]], s["blocks"].long()
    return _gather(s["k_cache"], s["k_scale"], ids).to(dt), _gather(s["v_cache"], s["v_scale"], ids).to(dt)


def _places(s):
    """(position, block, slot) of every new token."""
    lens, BS = s["seq_lens"].long(), s["k_cache"].shape[2]
    if "q_start" in s:
        start = s["q_start"].long()
        t = torch.arange(s["k_new"].shape[0], device=lens.device)
        b = torch.searchsorted(start[1:], t, right=True)
        pos = lens[b] - start[b + 1] + t
    else:
        b = torch.arange(lens.shape[0], device=lens.device)
        pos = lens - 1
    return pos, s["block_tables"][b, pos // BS].long(), pos % BS


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS) * w.float()


def _rotate(x, pos, freqs, interleaved):
    half = freqs.shape[0]
    angle = (pos[:, None] * freqs[None, :]).double() * (2.0 * math.pi * 2.0 ** -64)  # whole turns wrap away
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y


def _write(kind, s):
    c = s["case"]
    pos, blk, slot = _places(s)
    k, v, q = s["k_new"].float(), s["v_new"].float(), None
    if kind == "prepare":
        q = _rotate(_norm(s["q"], s["q_weight"]), pos, s["freqs"], c["interleaved"]).to(s["q"].dtype)
        k = _rotate(_norm(k, s["k_weight"]), pos, s["freqs"], c["interleaved"])
    for pool, scale, x in ((s["k_cache"], s.get("k_scale"), k), (s["v_cache"], s.get("v_scale"), v)):
        if scale is None:
            pool[blk, :, slot] = x.to(pool.dtype)
        else:
            vals, sc = _quantise(x, c["fmt"])
            pool.view(torch.uint8)[blk, :, slot] = vals.view(torch.uint8)
            scale[blk, :, slot] = sc
    if kind == "store":
        return _read(s)
    return _caches(s) if q is None else _caches(s) + (q,)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    es = {"bf16": 2, "f32": 4}[c["dtype"]]
    row = c["D"] + 4 if c["fmt"] != "none" else c["D"] * es  # a cached K or V row
    if c["kind"] == "attention":
        tokens = c["B"] * (c["lo"] + c["hi"]) / 2
        return dict(bytes=tokens * c["Hkv"] * 2 * row + 2 * c["B"] * c["Hq"] * c["D"] * es + tokens / c["BS"] * 4
                    + 4 * c["B"], flops=4 * tokens * c["Hq"] * c["D"])
    if c["kind"] == "read":
        rows = 2 * c["blocks"] * c["Hkv"] * c["BS"]
        return dict(bytes=rows * (row + c["D"] * es) + 4 * c["blocks"], flops=rows * c["D"])
    T = c["B"] * c["n"] * (0.75 if c["n"] > 1 else 1.0)
    rows = 2 * T * c["Hkv"]
    out = dict(bytes=rows * (c["D"] * es + row) + 8 * c["B"], flops=rows * c["D"] * 3)
    if c["kind"] == "prepare":
        out["bytes"] += 2 * T * c["Hq"] * c["D"] * es
        out["flops"] += T * (c["Hq"] + c["Hkv"]) * c["D"] * 8
    elif c["kind"] == "store":
        back = T * c["Hkv"] * 2
        out["bytes"] += back * (row + c["D"] * es)
    return out


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_quantise(x, fmt):
    """Rows of x (float64) as (numbers in the 8-bit type, scales)."""
    scale = torch.clamp(x.abs().max(dim=-1).values / _QMAX[fmt], min=_MIN_SCALE)
    y = x / scale.unsqueeze(-1)
    if fmt == "i8":
        return torch.round(y), scale
    _, e = torch.frexp(y)  # |y| = f * 2^e with f in [1/2, 1): 3 bits after the leading one, subnormals from 2^-6
    step = torch.ldexp(torch.ones_like(y), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(y / step) * step, -448.0, 448.0), scale


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    f64 = torch.float64
    if c["kind"] == "attention":
        out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
        G = c["Hq"] // c["Hkv"]
        for b, L in enumerate(s["seq_lens"].tolist()):
            if L == 0:
                continue
            ids = s["block_tables"][b, :-(-L // c["BS"])].long()
            for h in range(c["Hkv"]):
                k, v = (x.view(torch.uint8)[ids, h].view(x.dtype).float().double().reshape(-1, c["D"])[:L]
                        * z[ids, h].double().reshape(-1, 1)[:L]
                        for x, z in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
                logits = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(c["D"])
                out[b, h * G:(h + 1) * G] = torch.softmax(logits, dim=-1) @ v
        return out
    if c["kind"] == "read":
        ids = s["blocks"].long()
        return tuple(p.view(torch.uint8)[ids].view(p.dtype).float().double() * z[ids].double()[..., None]
                     for p, z in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
    # every token's sequence and position, one sequence after the other
    lens, B = s["seq_lens"].tolist(), c["B"]
    start = s["q_start"].tolist() if "q_start" in s else list(range(B + 1))
    seq = np.repeat(np.arange(B), np.diff(start))
    pos = np.concatenate([np.arange(lens[b] - (start[b + 1] - start[b]), lens[b]) for b in range(B)])
    bt = s["block_tables"].cpu().numpy()
    blk, slot = _cuda(bt[seq, pos // c["BS"]].astype(np.int64)), _cuda(pos % c["BS"])
    k, v, q = s["k_new"].to(f64), s["v_new"].to(f64), None
    if c["kind"] == "prepare":
        i = np.arange(c["rot"] // 2)
        angle = pos[:, None].astype(np.float64) * (10000.0 ** (-2.0 * i / c["rot"]))[None, :]
        turn = _cuda(np.exp(1j * angle))[:, None, :]

        def prepared(x, w):
            x = x.to(f64)
            x = x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / c["D"] + _EPS) * w.to(f64)
            r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
            if c["interleaved"]:
                z = torch.view_as_complex(r.reshape(*r.shape[:-1], -1, 2).contiguous()) * turn
                r = torch.view_as_real(z).reshape(r.shape)
            else:
                a, b = r.chunk(2, dim=-1)
                z = torch.complex(a, b) * turn
                r = torch.cat([z.real, z.imag], dim=-1)
            return torch.cat([r, rest], dim=-1)

        q, k = prepared(s["q"], s["q_weight"]), prepared(k, s["k_weight"])
    pools, scales = [], []
    for name, x in (("k", k), ("v", v)):
        pool = s[name + "_cache"].float().double()
        if c["fmt"] == "none":
            pool[blk, :, slot] = x
        else:
            scale = s[name + "_scale"].double()
            pool[blk, :, slot], scale[blk, :, slot] = _exact_quantise(x, c["fmt"])
            scales.append(scale)
        pools.append(pool)
    if c["kind"] == "store":
        ids = s["blocks"].long()
        return tuple(p[ids] * z[ids].unsqueeze(-1) for p, z in zip(pools, scales))
    return tuple(pools + scales + ([] if q is None else [q]))
