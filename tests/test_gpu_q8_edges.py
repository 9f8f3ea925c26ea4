"""The 8-bit cache's calls at the edges of what they are documented for."""
import ctypes
import math
import threading

import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
from tests import q8_ref as R

pytestmark = pytest.mark.gpu
FMTS = ["e4m3", "i8"]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
U24 = 2.0 ** -24  # half a float32 step, relative


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


def cuda(*ts):
    return [t.cuda() for t in ts]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------ block ids
IDS = {  # sequences, their lengths, width of the table, (Hq, Hkv, D)
    "direct": (14, lambda b: 200 + 30 * b, 48, (8, 2, 64)),
    "split": (14, lambda b: 1500 + 130 * b, None, (8, 8, 128)),
    "cuts": (200, lambda b: 40 + (b * 37) % 300, None, (32, 8, 128)),
}


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("path", list(IDS))
def test_any_id_outside_the_pool_gives_zeros_and_a_status(path, fmt):
    """-1, -2, the lowest integer and one past the pool, in the first, a middle and the
    last block; the other sequences are not touched by it."""
    B, length, width, (Hq, Hkv, D) = IDS[path]
    BS = 16
    lens = [length(b) for b in range(B)]
    g = torch.Generator().manual_seed(11)
    bt, nb = R.tables(lens, BS, g, width=width)
    bad = {}
    for n, (i, at) in enumerate((i, at) for i in (-1, -2, -2 ** 31, nb) for at in (0, 1, 2)):
        b = 1 + n
        last = (lens[b] - 1) // BS
        bad[b] = i
        bt[b, (0, last // 2, last)[at]] = i
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, fmt, g)
    q = torch.randn(B, Hq, D, generator=g).to(torch.bfloat16)
    good = [b for b in range(B) if b not in bad]
    want, tol = R.attention(q[good], k, v, ks, vs, bt[good], [lens[b] for b in good], dtype="bf16")
    gq, gk, gv, gks, gvs, gbt, gl = cuda(q, k, v, ks, vs, bt, i32(lens))
    for _ in range(2):  # the second call finds the first one's leavings in shared memory
        st = pkv.new_status()
        out = pkv.paged_decode_attention_q8(gq, gk, gv, gks, gvs, gbt, gl, status=st).cpu().double()
        assert pkv.check_status(st) == 4
        assert all(torch.equal(out[b], torch.zeros_like(out[b])) for b in bad), \
            [(b, bad[b]) for b in bad if not torch.equal(out[b], torch.zeros_like(out[b]))]
        assert ((out[good] - want).abs() <= tol).all()


@pytest.mark.parametrize("path", list(IDS))
def test_one_bad_id_alone_is_reported(path):
    """One sequence holds -2 in one block, and nothing else is wrong."""
    B, length, width, (Hq, Hkv, D) = IDS[path]
    lens = [length(b) for b in range(B)]
    g = torch.Generator().manual_seed(12)
    bt, nb = R.tables(lens, 16, g, width=width)
    bt[3, (lens[3] - 1) // 16] = -2
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, "i8", g)
    q = torch.randn(B, Hq, D, generator=g)
    st = pkv.new_status()
    out = pkv.paged_decode_attention_q8(*cuda(q, k, v, ks, vs, bt, i32(lens)), status=st).cpu()
    assert pkv.check_status(st) == 4
    assert torch.equal(out[3], torch.zeros_like(out[3])) and (out[2] != 0).any()


# ------------------------------------------------------------------ peaked rows
def peaked_cache(L, D, BS, Hkv, fmt, gap, gen):
    """One sequence, the same in every KV head: the key at position 5 scores `gap` nats above a
    flat tail for q [D]; V has mean 1.  Returns q, the pools and the table, and the rows in float64."""
    q = torch.randn(D, generator=gen)
    u = q / q.norm()
    kk = 0.1 * torch.randn(L, D, generator=gen)
    kk -= (kk @ u)[:, None] * u  # the tail scores about 0
    kk[5] = u * (gap * D ** 0.5 / q.norm())
    vv = 1 + 0.2 * torch.randn(L, D, generator=gen)
    vv[5, 0] = 4  # a larger scale, hence a larger contribution, than the tail's rows
    bt, nb = R.tables([L], BS, gen, spare=0)
    at = bt[0, torch.arange(L) // BS].long() * BS + torch.arange(L) % BS
    pools, rows = [], []
    for x in (kk, vv):
        vals, sc = R.store(x, fmt)
        pool, scale = torch.zeros(nb * BS, D, dtype=torch.uint8), torch.zeros(nb * BS)
        pool[at], scale[at] = vals.view(torch.uint8), sc
        pools += [pool.view(nb, 1, BS, D).expand(nb, Hkv, BS, D).contiguous().view(R.DT[fmt]),
                  scale.view(nb, 1, BS).expand(nb, Hkv, BS).contiguous()]
        rows.append((vals.float().double(), sc.double()))
    return q, pools[0], pools[2], pools[1], pools[3], bt, rows


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype,many,L,D,gap", [("f32", True, 32768, 16, 17.0), ("f32", True, 8192, 128, 17.0),
                                                ("f32", False, 32768, 16, 17.0), ("bf16", True, 1 << 20, 16, 17.0)])
def test_a_long_flat_tail_behind_one_large_weight(dtype, many, L, D, gap, fmt):
    """A first token that takes nearly all of the weight, and a tail whose single contributions
    are below 2^-25 of it but whose sum matters.  As many sequences as SMs, over the same
    blocks, so that a warp meets a whole sequence; and five, which the SMs share.

    Tolerance, per element, with p the weights, out the result, W = sum p |v|,
    C = sum p |v - out| and S = max scale sum |q k|:
      scores   2 D truncated additions, 24 more roundings of S, 160 of the exponents' size:
               d = ((2 D + 24) S + 160) 2^-24 in every weight, numerator and sum alike: 2 d C;
      sums     of n = L / 32 or L / 64 steps in the numerator and in the sum, and 700 additions within a
               step, between warps and between ranges, a rounding each: (2 n + 700) 2^-24 W; bf16
               adds tiles of 16 positions instead, each truncated: 2^-23 W L / 16 more;
      weights  a float16 rounding, 2^-11 W (bf16), or two, 2^-22 W (float32), and for weights near
               float16's smallest number half of it: 2^-34 of the largest weight (bf16), 2^-45
               with the second float16 (float32), times sum |v numbers|;
      output   2^-8 or 2^-24 of itself.
    """
    g = torch.Generator().manual_seed(21)
    Hkv, G = 8, 2
    B = torch.cuda.get_device_properties(0).multi_processor_count if many else 5
    q, k, v, ks, vs, bt, ((kn, ksc), (vn, vsc)) = peaked_cache(L, D, 16, Hkv, fmt, gap, g)
    qq = torch.stack([q, 1.02 * q]).to(DTYPES[dtype])
    kk, vv = kn * ksc[:, None], vn * vsc[:, None]
    p = torch.softmax(D ** -0.5 * qq.double() @ kk.T, -1)
    want = p @ vv
    S = D ** -0.5 * (qq.double().abs() @ kk.abs().T).amax(-1, keepdim=True)
    W = p @ vv.abs()
    C = torch.stack([p[h] @ (vv - want[h]).abs() for h in range(G)])
    n = L / (64 if D <= 64 else 32)
    if dtype == "bf16":
        rel, floor, last = 2.0 ** -11 + 2.0 ** -23 * L / 16, 2.0 ** -34, 2.0 ** -8
    else:
        rel, floor, last = 2.0 ** -22, 2.0 ** -45, U24
    tol = (2 * ((2 * D + 24) * S + 160) * U24 * C + ((2 * n + 700) * U24 + rel) * W
           + floor * (p * vsc).amax(-1, keepdim=True) * vn.abs().sum(0) + last * want.abs())
    # the tail adds more than that, in contributions that are each below 2^-25 of the largest
    assert p[:, 6:].sum(-1).min() > 2 * (tol / want.abs()).max()
    w = p * vsc
    assert (w[:, 6:] < 2.0 ** -25 * w[:, 5:6]).all()
    gq = qq.repeat(Hkv, 1).expand(B, Hkv * G, D).contiguous().cuda()
    out = pkv.paged_decode_attention_q8(gq, *cuda(k, v, ks, vs, bt.expand(B, -1).contiguous(), i32([L] * B)))
    err = (out.cpu().double().view(B, Hkv, G, D) - want).abs()
    assert (err <= tol).all(), (err / want.abs()).max().item()


@pytest.mark.parametrize("dtype,Hq,Hkv,D,L", [("bf16", 16, 8, 64, 21000), ("bf16", 128, 8, 128, 18000),
                                              ("bf16", 8, 1, 64, 140000), ("bf16", 10, 5, 80, 18000), ("f32", 16, 8, 64, 9000)])
def test_long_ranges_with_late_maxima(dtype, Hq, Hkv, D, L):
    """Ranges of whole long sequences (as many as SMs, over the same blocks) whose scores grow along
    the cache, so that the maximum is renewed after parts of the sums were set aside."""
    g = torch.Generator().manual_seed(61)
    B = torch.cuda.get_device_properties(0).multi_processor_count
    bt, nb = R.tables([L], 16, g, spare=0)
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, "e4m3", g)
    grow = torch.zeros(nb, 16)
    grow[bt[0].long()] = (torch.arange(nb * 16) / L).view(nb, 16)
    ks *= 0.2 + 1.8 * grow[:, None, :]
    q = torch.randn(1, Hq, D, generator=g).to(DTYPES[dtype])
    want, tol = R.attention(q, k, v, ks, vs, bt, [L], dtype=dtype)
    out = pkv.paged_decode_attention_q8(q.expand(B, -1, -1).contiguous().cuda(), *cuda(k, v, ks, vs),
                                        bt.expand(B, -1).contiguous().cuda(), i32([L] * B).cuda()).cpu().double()
    assert ((out - want).abs() <= tol).all(), ((out - want).norm() / (B ** 0.5 * want.norm())).item()


# ------------------------------------------------------------------ V scales far apart
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([700], 4, 1, 128), ([600, 90], 8, 2, 64), ([9000, 4000], 8, 8, 128),
                                           ([5000], 16, 1, 80)])
def test_zero_rows_keep_their_weight_beside_huge_ones(lens, Hq, Hkv, D, fmt, dtype):
    """Rows of V that are zero (scale 2^-64) in one part of a sequence and about 1e36 in another:
    the zero rows take their share of the weight."""
    BS = 16
    g = torch.Generator().manual_seed(31)
    for zeros_first in (True, False):
        bt, nb = R.tables(lens, BS, g)
        k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, fmt, g)
        x = torch.randn(nb, Hkv, BS, D, generator=g) * 1e36
        for b, L in enumerate(lens):
            blocks = bt[b, :-(-L // BS)].long()
            half = len(blocks) // 2
            x[blocks[:half] if zeros_first else blocks[half:]] = 0
        v, vs = R.store(x, fmt)
        q = torch.randn(len(lens), Hq, D, generator=g).to(DTYPES[dtype])
        want, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype=dtype)
        out = pkv.paged_decode_attention_q8(*cuda(q, k, v, ks, vs, bt, i32(lens))).cpu().double()
        assert ((out - want).abs() <= tol).all(), ((out - want).norm() / want.norm()).item()


# ------------------------------------------------------------------ threads
def raw_q8(lib, q, k, v, ks, vs, bt, lens, out, ws, stream):
    B, Hq, D = q.shape
    NB, Hkv, BS, _ = k.shape
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    args = (p(out), p(q), p(k), p(v), p(ks), p(vs), p(bt), bt.shape[1], p(lens), B, Hq, Hkv, D, BS, NB,
            ctypes.c_float(0.0), 1, 2, p(ws), ws.numel(), None, ctypes.c_void_p(stream.cuda_stream))
    return lambda: lib.pkv_paged_decode_attention_q8(*args)


def in_threads(calls, rounds):
    """Every call `rounds` times, each in a thread of its own; the status codes that came back."""
    codes = [set() for _ in calls]
    start = threading.Barrier(len(calls))

    def work(i):
        start.wait()
        for _ in range(rounds):
            codes[i].add(int(calls[i]()))
    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    return codes


def test_threads_with_shapes_of_one_kernel():
    """Head sizes 80 and 96 and 1, 3 and 8 KV heads share a kernel and need different amounts of shared
    memory; ctypes lets the threads run at the same time."""
    lib = pkv.load_library()
    calls, keep = [], []
    for n, (Hq, Hkv, D) in enumerate([(8, 8, 80), (8, 8, 96), (8, 1, 80), (6, 3, 96)]):
        g = torch.Generator().manual_seed(n)
        lens = [900, 1500]
        bt, nb = R.tables(lens, 16, g)
        k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, "e4m3", g)
        q = torch.randn(2, Hq, D, generator=g).to(torch.bfloat16)
        t = cuda(q, k, v, ks, vs, bt, i32(lens))
        want = pkv.paged_decode_attention_q8(*t)
        out = torch.zeros_like(want)
        ws = torch.empty(max(16, pkv.decode_q8_workspace_bytes(2, Hq, Hkv, D)), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        keep.append((t, want, out, ws, s))
        calls.append(raw_q8(lib, *t, out, ws, s))
    torch.cuda.synchronize()
    assert in_threads(calls, 4000) == [{0}] * len(calls)
    torch.cuda.synchronize()
    for _, want, out, _, _ in keep:
        assert torch.equal(want, out)


# ------------------------------------------------------------------ calls one behind the other
@pytest.mark.parametrize("fmt", FMTS)
def test_calls_that_start_before_their_predecessor_ends(fmt):
    """Appends, read-backs and attention over the same few blocks, back to back: every call sees all
    that the one before it wrote."""
    Hq, Hkv, D, BS, B, rounds = 8, 8, 128, 16, 24, 30
    g = torch.Generator().manual_seed(71)
    bt, nb = R.tables([64] * B, BS, g)
    k, v, ks, vs = cuda(*R.random_cache(nb, Hkv, BS, D, fmt, g))
    bt, ids = bt.cuda(), torch.arange(nb, dtype=torch.int32).cuda()
    kn, vn = (torch.randn(rounds, B, Hkv, D, generator=g).cuda() for _ in range(2))
    q = torch.randn(rounds, B, Hq, D, generator=g).cuda()
    lens = [i32([1 + (7 * r) % 64] * B).cuda() for r in range(rounds)]

    def chain(sync):
        pools = [t.clone() for t in (k, v, ks, vs)]
        res = []
        for r in range(rounds):
            for call in (lambda: pkv.kv_append_q8(kn[r], vn[r], *pools, bt, lens[r]),
                         lambda: pkv.kv_read_blocks_q8(*pools, ids),
                         lambda: pkv.paged_decode_attention_q8(q[r], *pools, bt, lens[r])):
                x = call()
                res += [] if x is None else list(x) if type(x) is tuple else [x]
                if sync:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        return res + pools

    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ rotation
@pytest.mark.parametrize("D,interleaved,at", [(128, False, 0), (128, True, 0), (20, False, 0), (64, False, 1)])
def test_cosines_and_sines_at_any_angle(D, interleaved, at):
    """Rows (1, 0) per pair give the cosine and the sine themselves.  The angle, a 64-bit
    fraction of a turn, is rounded once to float32 within an eighth of a turn of a whole
    quarter: at most 2^-27 half-turns, pi * 2^-27 < 0.4 * 2^-24 in the result; sincospif adds at
    most 1 ulp of the result, which is at most 2^-23 of it."""
    g = torch.Generator().manual_seed(41)
    T, half = 64, D // 2
    hi, lo = (torch.randint(0, 2 ** 32, (half,), generator=g) for _ in range(2))
    freqs = ((hi - 2 ** 31) << 32) | lo  # any 64-bit integer
    lens = [1 + int(x) for x in torch.randint(0, 64, (T,), generator=g)]
    bt, nb = R.tables(lens, 16, g)
    row = torch.zeros(D)
    row[0::2 if interleaved else 1][:half] = 1
    buf = torch.zeros(T * D + at)
    x = row.repeat(T, 1, 1)
    gq = buf.cuda()[at:].view(T, 1, D)  # at: an address that is not 16-byte aligned
    gq.copy_(x)
    kc, vc = (torch.zeros(nb, 1, 16, D, device="cuda") for _ in range(2))
    out = pkv.qk_norm_rope_append(gq, gq.clone(), gq.clone(), None, None, 0.0, freqs.cuda(), kc, vc, *cuda(bt, i32(lens)),
                                  interleaved=interleaved).cpu().double()[:, 0]
    ang = torch.tensor([[2 * math.pi * (((L - 1) * int(f)) % 2 ** 64 / 2 ** 64) for f in freqs] for L in lens],
                       dtype=torch.float64)
    cos, sin = (out[:, 0::2], out[:, 1::2]) if interleaved else (out[:, :half], out[:, half:])
    for got, want in ((cos, torch.cos(ang)), (sin, torch.sin(ang))):
        # 2^-50: the float64 angle's own rounding, at most 2 pi 2^-53
        tol = 0.4 * U24 + 2.0 ** -23 * want.abs() + 2.0 ** -50
        assert ((got - want).abs() <= tol).all(), (((got - want).abs() - tol).max() / U24).item()


# ------------------------------------------------------------------ graphs
@pytest.mark.parametrize("fmt", FMTS)
def test_a_prompt_and_a_decode_step_captured_and_replayed(fmt):
    """Preparation, append, read-back and attention in one graph, replayed on new inputs and
    lengths: the bytes and numbers of the same calls made one by one."""
    Hq, Hkv, D, BS, B = 8, 2, 64, 16, 4
    g = torch.Generator().manual_seed(51)
    bt, nb = R.tables([200] * B, BS, g)
    table, freqs = bt.cuda(), pkv.rope_freqs(D)
    w = torch.rand(D, generator=g).to(torch.bfloat16).cuda() + 0.5
    qs = i32([0, 20, 20, 53, 60]).cuda()

    def buffers():
        pools = cuda(*R.random_cache(nb, Hkv, BS, D, fmt, torch.Generator().manual_seed(52)))
        q, kv, q1, kv1 = (torch.zeros(n, h, D, dtype=torch.bfloat16, device="cuda")
                          for n, h in ((60, Hq), (60, 2 * Hkv), (B, Hq), (B, 2 * Hkv)))
        return (*pools, q, kv, q1, kv1, torch.zeros(2, B, dtype=torch.int32, device="cuda"), pkv.new_status())

    def calls(k, v, ks, vs, q, kv, q1, kv1, lens, st):
        kn, vn = kv[:, :Hkv], kv[:, Hkv:]
        qo = pkv.qk_norm_rope_append(q, kn, vn, w, w, 1e-6, freqs, k, v, table, lens[0], qs, ks, vs, status=st)
        pkv.kv_append_q8(kv1[:, :Hkv].contiguous(), kv1[:, Hkv:].contiguous(), k, v, ks, vs, table, lens[1],
                         status=st)
        rk, rv = pkv.kv_read_blocks_q8(k, v, ks, vs, table[2], status=st)
        a = pkv.paged_decode_attention_q8(q1, k, v, ks, vs, table, lens[1], status=st)
        return qo, rk, rv, a

    cap, plain = buffers(), buffers()

    def fill(bufs, seed):
        gen = torch.Generator().manual_seed(seed)
        for t in bufs[4:8]:
            t.copy_(torch.randn(t.shape, generator=gen))
        lens = [40 + int(x) for x in torch.randint(0, 100, (B,), generator=gen)]
        bufs[8].copy_(i32([lens, [n + 1 for n in lens]]))

    fill(cap, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(*cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(*cap)
    for t, fresh in zip(cap[:4], buffers()[:4]):
        t.copy_(fresh)
    for seed in (2, 3, 4):
        fill(cap, seed)
        fill(plain, seed)
        graph.replay()
        want = calls(*plain)
        torch.cuda.synchronize()
        for a, b in zip((*got, *cap[:4]), (*want, *plain[:4])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert pkv.check_status(cap[9]) == 0 and pkv.check_status(plain[9]) == 0
