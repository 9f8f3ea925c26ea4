"""The 8-bit KV cache on the GPU: stored bytes against the format's formula bit for
bit, everything else against float64 with the tolerances of q8_ref."""
import math

import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
from tests import q8_ref as R

pytestmark = pytest.mark.gpu
FMTS = ["e4m3", "i8"]
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


def cpu_equal(a, b):
    """Bitwise equality of an 8-bit or float tensor on the GPU with one on the CPU."""
    a = a.detach().cpu()
    if a.element_size() == 1:
        return torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    return torch.equal(a.view(torch.int32), b.view(torch.int32)) if a.dtype == torch.float32 else torch.equal(a, b)


def cuda(*ts):
    return [t.cuda() for t in ts]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


# ------------------------------------------------------------------ append
def place(lens, counts, bt, BS):
    """(block, slot) of every new token, and its sequence and position."""
    seq = [b for b, n in enumerate(counts) for _ in range(n)]
    pos = [lens[b] - n + i for b, n in enumerate(counts) for i in range(n)]
    blk = [int(bt[b, p // BS]) for b, p in zip(seq, pos)]
    return blk, [p % BS for p in pos], pos


APPENDS = [  # (Hkv, D, BS, lens, counts or None for one token each)
    (8, 128, 16, [1, 16, 17, 900, 33], None),
    (2, 64, 16, [5, 40, 7, 64], [5, 33, 0, 1]),
    (3, 80, 32, [70, 1, 200], [64, 1, 130]),
    (1, 4, 4, [9, 13], None),
    (5, 100, 8, [50, 3], [50, 2]),
    (1, 1, 1, [3, 2], [2, 2]),
    (2, 256, 48, [100, 49], [60, 49]),
    (12, 16, 64, [64, 65], None),
    (3, 36, 16, [30, 20], [7, 20]),
    # many tokens: several of them a CTA
    (2, 64, 16, [700, 31], [700, 0]),
    (3, 128, 32, [900, 40, 77], [650, 33, 77]),
]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", range(len(APPENDS)))
def test_append_stores_the_format_bit_for_bit(case, dtype, fmt):
    Hkv, D, BS, lens, counts = APPENDS[case]
    g = torch.Generator().manual_seed(100 + case)
    bt, nb = R.tables(lens, BS, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, fmt, g)
    n = counts or [1] * len(lens)
    T = sum(n)
    kn, vn = ((torch.randn(T, Hkv, D, generator=g) * 3).to(DTYPES[dtype]) for _ in range(2))
    kn[0] = 0  # an all-zero row
    gk, gv, gks, gvs, gkn, gvn, gbt = cuda(k, v, ks, vs, kn, vn, bt)
    st = pkv.new_status()
    if counts is None:
        pkv.kv_append_q8(gkn, gvn, gk, gv, gks, gvs, gbt, i32(lens).cuda(), status=st)
    else:
        qs = torch.zeros(len(lens) + 1, dtype=torch.int32)
        qs[1:] = torch.cumsum(i32(counts), 0)
        pkv.kv_append_chunk_q8(gkn, gvn, gk, gv, gks, gvs, gbt, i32(lens).cuda(), qs.cuda(), status=st)
    assert pkv.check_status(st) == 0
    blk, slot, _ = place(lens, n, bt, BS)
    for pool, scale, new in ((k, ks, kn), (v, vs, vn)):
        vals, sc = R.store(new, fmt)
        pool.view(torch.uint8)[blk, :, slot] = vals.view(torch.uint8)
        scale[blk, :, slot] = sc
    for a, b in ((gk, k), (gv, v), (gks, ks), (gvs, vs)):  # whole pools: nothing else was touched
        assert cpu_equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_extreme_rows(fmt):
    """Tiny, huge, subnormal and tied values, and rows with NaN or infinities."""
    D, BS = 64, 16
    rows = torch.zeros(8, 1, D)
    rows[0] = torch.linspace(-1, 1, D) * 3e38
    rows[1] = torch.linspace(-1, 1, D) * 1e-38
    rows[2, 0, 3] = 1e-45
    rows[3] = 1.75 * torch.arange(D) / 256  # amax / Q exact in e4m3's steps: ties
    rows[4] = torch.arange(D) - 31.5
    rows[5, 0, 7] = math.nan
    rows[6, 0, 9] = -math.inf
    rows[7] = 2.0 ** -60
    B = rows.shape[0]
    bt, nb = R.tables([1] * B, BS, torch.Generator().manual_seed(0))
    k, v, ks, vs = R.random_cache(nb, 1, BS, D, fmt, torch.Generator().manual_seed(1))
    gk, gv, gks, gvs, gr, gbt = cuda(k, v, ks, vs, rows, bt)
    st = pkv.new_status()
    pkv.kv_append_q8(gr, gr.flip(0).contiguous(), gk, gv, gks, gvs, gbt, i32([1] * B).cuda(), status=st)
    assert pkv.check_status(st) == 6
    blk = bt[:, 0].long()
    for gp, gs, new in ((gk, gks, rows), (gv, gvs, rows.flip(0))):
        vals, sc = R.store(new, fmt)
        assert cpu_equal(gp.view(torch.uint8)[blk.cuda(), :, 0], vals.view(torch.uint8))
        got = gs[blk.cuda(), :, 0].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(sc))
        ok = ~torch.isnan(sc)
        assert torch.equal(got[ok], sc[ok])


def test_append_skips_what_it_cannot_place():
    Hkv, D, BS = 2, 64, 16
    lens = [20, 0, 33, 10, 40]
    g = torch.Generator().manual_seed(3)
    bt, nb = R.tables([20, 16, 48, 16, 48], BS, g, width=3)
    bt[3, 0] = nb       # one past the pool
    bt[4, 2] = -5
    lens[2] = 3 * BS + 1  # beyond the table
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, "i8", g)
    kn, vn = (torch.randn(5, Hkv, D, generator=g) for _ in range(2))
    gk, gv, gks, gvs, gkn, gvn, gbt = cuda(k, v, ks, vs, kn, vn, bt)
    st = pkv.new_status()
    pkv.kv_append_q8(gkn, gvn, gk, gv, gks, gvs, gbt, i32(lens).cuda(), status=st)
    assert pkv.check_status(st) == 4
    for pool, scale, new in ((k, ks, kn), (v, vs, vn)):
        vals, sc = R.store(new[:1], "i8")
        pool[int(bt[0, 1]), :, 3] = vals[0]
        scale[int(bt[0, 1]), :, 3] = sc[0]
    for a, b in ((gk, k), (gv, v), (gks, ks), (gvs, vs)):
        assert cpu_equal(a, b)


# ------------------------------------------------------------------ read back
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("Hkv,D,BS", [(8, 128, 16), (3, 80, 32), (1, 4, 4), (5, 100, 8), (2, 256, 16), (1, 1, 1),
                                      (7, 24, 5), (2, 36, 16), (8, 128, 32), (3, 64, 48)])
def test_read_blocks_bit_for_bit(Hkv, D, BS, dtype, fmt):
    g = torch.Generator().manual_seed(7)
    k, v, ks, vs = R.random_cache(11, Hkv, BS, D, fmt, g)
    ids = [4, 4, 0, 10, 7]
    st = pkv.new_status()
    gk, gv, gks, gvs = cuda(k, v, ks, vs)
    ko, vo = pkv.kv_read_blocks_q8(gk, gv, gks, gvs, i32(ids).cuda(), dtype=DTYPES[dtype], status=st)
    assert pkv.check_status(st) == 0
    for got, pool, scale in ((ko, k, ks), (vo, v, vs)):
        want = (pool.float() * scale[..., None])[ids].to(DTYPES[dtype])
        assert got.dtype == DTYPES[dtype] and torch.equal(got.cpu(), want)


def test_read_bad_ids_give_zero_blocks_and_unaligned_outputs_work():
    g = torch.Generator().manual_seed(8)
    k, v, ks, vs = R.random_cache(5, 2, 16, 64, "e4m3", g)
    gk, gv, gks, gvs = cuda(k, v, ks, vs)
    ids = i32([2, 5, -1, 0])
    st = pkv.new_status()
    n = 4 * 2 * 16 * 64
    flat = torch.full((2, n + 1), 9.0, device="cuda")
    ko, vo = (flat[i, 1:].view(4, 2, 16, 64) for i in range(2))  # 4-byte aligned only
    pkv.kv_read_blocks_q8(gk, gv, gks, gvs, ids.cuda(), k_out=ko, v_out=vo, status=st)
    assert pkv.check_status(st) == 4
    for got, pool, scale in ((ko, k, ks), (vo, v, vs)):
        want = pool.float() * scale[..., None]
        assert torch.equal(got[0].cpu(), want[2]) and torch.equal(got[3].cpu(), want[0])
        assert bool((got[1:3] == 0).all())
    assert bool((flat[:, 0] == 9).all())


@pytest.mark.parametrize("Hkv,D,BS", [(1, 5, 3), (3, 80, 32), (2, 24, 1)])
@pytest.mark.parametrize("fmt", FMTS)
def test_copy_blocks_of_an_8_bit_cache(Hkv, D, BS, fmt):
    g = torch.Generator().manual_seed(31)
    pools = R.random_cache(9, Hkv, BS, D, fmt, g)
    k, v, ks, vs = cuda(*(p.clone() for p in pools))
    st = pkv.new_status()
    src, dst = [0, 0, 7, 9], [3, 5, 8, 1]  # one source twice; the last id is out of range
    pkv.copy_blocks(k, v, i32(src).cuda(), i32(dst).cuda(), status=st, k_scale=ks, v_scale=vs)
    assert pkv.check_status(st) == 4
    for got, want in zip((k, v, ks, vs), pools):
        want = want.clone()
        raw = want.view(torch.uint8) if want.dtype != torch.float32 else want
        for a, b in zip(src[:3], dst[:3]):
            raw[b] = raw[a]
        assert torch.equal(got.cpu().view(raw.dtype), raw)


# ------------------------------------------------------------------ attention
ATTENTION = [  # (Hq, Hkv, D, BS, lens)
    (32, 8, 128, 16, [1, 0, 16, 17, 255, 700, 31, 15]),
    (8, 8, 128, 16, [100, 333, 64]),
    (64, 8, 128, 16, [2500, 1]),
    (48, 4, 128, 16, [100, 500]),            # 12 query heads a group
    (16, 1, 128, 16, [129, 2000]),
    (34, 2, 128, 16, [129, 40]),             # 17 query heads a group
    (64, 2, 64, 16, [77, 300]),
    (8, 2, 64, 16, [1, 200]),
    (21, 3, 80, 32, [0, 33, 700, 64]),
    (5, 5, 96, 48, [150, 47]),
    (12, 12, 16, 64, [63, 64, 65, 500]),
    (44, 11, 32, 16, [333, 90]),
    (16, 16, 112, 16, [90, 16]),
    (32, 32, 64, 256, [700, 255, 3]),
    (6, 3, 100, 16, [70, 1]),
    (2, 2, 4, 4, [9, 13]),
    (4, 2, 128, 8, [65, 7]),
    (4, 2, 64, 24, [65, 100]),
    (4, 2, 256, 16, [130, 0, 40]),
    (10, 5, 192, 32, [65]),
    (3, 1, 1, 1, [5, 2]),
    (130, 1, 64, 16, [40, 300]),
    (32, 8, 128, 16, [(13 * b) % 90 for b in range(40)]),  # 3 + 3 + 2 KV heads a CTA
    (10, 5, 64, 32, [(5 * b) % 64 for b in range(150)]),
    (9, 9, 128, 16, [1000, 33]),                           # two groups, the second smaller, split
    (60, 5, 112, 16, [1000, 170, 0, 33]),
]


def run_attention(Hq, Hkv, D, BS, lens, fmt, dtype, seed=11, poison=True, **kw):
    g = torch.Generator().manual_seed(seed)
    bt, nb = R.tables(lens, BS, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, fmt, g)
    q = (1.5 * torch.randn(len(lens), Hq, D, generator=g)).to(DTYPES[dtype])
    gk, gv, gks, gvs = cuda(k.clone(), v.clone(), ks.clone(), vs.clone())
    if poison:  # slots behind the end: NaN values (in e4m3) and NaN, infinite and lowest scales
        for b, L in enumerate(lens):
            if L % BS:
                blk = int(bt[b, L // BS])
                for p, s in ((gk, gks), (gv, gvs)):
                    p.view(torch.uint8)[blk, :, L % BS:] = 0x7f
                    s[blk, :, L % BS:] = math.nan
                    s[blk, :, -1] = math.inf if b % 2 else torch.finfo(torch.float32).min
    st = pkv.new_status()
    out = pkv.paged_decode_attention_q8(q.cuda(), gk, gv, gks, gvs, bt.cuda(), i32(lens).cuda(), status=st, **kw)
    assert pkv.check_status(st) == 0
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, scale=kw.get("scale"), dtype=dtype)
    err = (out.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), f"{int((err > tol).sum())} off, worst {float((err / tol).max()):.3g} of the bound"
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", range(len(ATTENTION)))
def test_attention(case, dtype, fmt):
    run_attention(*ATTENTION[case], fmt, dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("Hq,Hkv,D,lens", [(32, 8, 128, [40000]), (4, 1, 128, [30000, 5]), (16, 2, 64, [9000] * 3),
                                           (8, 8, 128, list(range(1, 400, 7))), (7, 7, 80, [3] * 500)])
def test_attention_split_over_many_ranges(Hq, Hkv, D, lens, fmt):
    run_attention(Hq, Hkv, D, 16, lens, fmt, "bf16", seed=12)
    run_attention(Hq, Hkv, D, 16, lens, fmt, "f32", seed=13, scale=0.37)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 64), (36, 9, 80), (20, 2, 128)])
def test_attention_of_more_sequences_than_sms(Hq, Hkv, D):
    """More (sequence, head group) pairs than ranges: joined where a range cuts one; empty
    sequences, bad lengths and bad blocks between them."""
    lens = [(0, 5, 90, 0, 333, 17)[b % 6] for b in range(400)]
    lens[57] = 3000
    for dtype in DTYPES:
        out = run_attention(Hq, Hkv, D, 16, lens, "e4m3", dtype, seed=15)
        assert bool((out[::6] == 0).all())
    g = torch.Generator().manual_seed(16)
    bt, nb = R.tables(lens, 16, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, "i8", g)
    q = torch.randn(400, Hq, D, generator=g).bfloat16()
    bad_bt, bad_lens = bt.clone(), list(lens)
    bad_lens[1], bad_lens[399], bad_bt[57, 100], bad_bt[4, 3] = -1, bt.shape[1] * 16 + 1, nb, -7
    bad = [1, 399, 57, 4]
    good = [b for b in range(400) if b not in bad]
    st = pkv.new_status()
    out = pkv.paged_decode_attention_q8(*cuda(q, k, v, ks, vs, bad_bt, i32(bad_lens)), status=st)
    assert pkv.check_status(st) == 4
    assert bool((out[bad] == 0).all())
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    assert bool(((out.cpu().double() - ref).abs() <= tol)[good].all())


@pytest.mark.parametrize("fmt", FMTS)
def test_attention_wide_scales(fmt):
    """V scales and scores spread over many orders of magnitude: the weights are
    normalised by the largest contribution, not by the largest score."""
    Hq, Hkv, D, BS, lens = 8, 2, 64, 16, [300, 17]
    for spread in (1e-12, 1e-6, 1e6):
        g = torch.Generator().manual_seed(21)
        bt, nb = R.tables(lens, BS, g)
        k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, fmt, g)
        vs[:, :, ::3] *= spread
        vs[:, 1, 5] = 2.0 ** -64
        q = 4 * torch.randn(2, Hq, D, generator=g)
        for dtype in DTYPES:
            qq = q.to(DTYPES[dtype])
            out = pkv.paged_decode_attention_q8(*cuda(qq, k, v, ks, vs, bt, i32(lens)))
            ref, tol = R.attention(qq, k, v, ks, vs, bt, lens, dtype=dtype)
            assert bool(((out.cpu().double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("Hq,Hkv,D,lens", [(8, 2, 64, [300, 17]), (8, 2, 128, [2000]), (4, 2, 100, [300, 40])])
@pytest.mark.parametrize("fmt", FMTS)
def test_attention_over_values_near_the_largest_float(Hq, Hkv, D, lens, fmt):
    """V scales up to 2^119.  Exponents are then shifted by up to 119 instead of 64, which
    enters the bound's 144 * 2^-24 as 2 * 119 + 16: less than twice the bound."""
    g = torch.Generator().manual_seed(22)
    bt, nb = R.tables(lens, 16, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, fmt, g)
    vs = 2.0 ** 119 * (0.5 + 0.5 * torch.rand(vs.shape, generator=g))
    q = torch.randn(len(lens), Hq, D, generator=g)
    for dtype in DTYPES:
        qq = q.to(DTYPES[dtype])
        out = pkv.paged_decode_attention_q8(*cuda(qq, k, v, ks, vs, bt, i32(lens)))
        ref, tol = R.attention(qq, k, v, ks, vs, bt, lens, dtype=dtype)
        assert bool(((out.cpu().double() - ref).abs() <= 2 * tol).all())


@pytest.mark.parametrize("Hq,Hkv,D,BS", [(32, 8, 128, 16), (4, 2, 100, 16), (8, 1, 64, 32)])
def test_attention_bad_rows_are_zero_and_reported(Hq, Hkv, D, BS):
    lens = [200, 90, 64, 0, 75]
    g = torch.Generator().manual_seed(5)
    bt, nb = R.tables(lens, BS, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, "e4m3", g)
    q = torch.randn(5, Hq, D, generator=g).bfloat16()
    bad_bt, bad_lens = bt.clone(), list(lens)
    bad_bt[0, 1] = nb
    bad_bt[1, 0] = -3
    bad_lens[2] = bt.shape[1] * BS + 1
    st = pkv.new_status()
    out = pkv.paged_decode_attention_q8(*cuda(q, k, v, ks, vs, bad_bt, i32(bad_lens)), status=st)
    assert pkv.check_status(st) == 4
    assert bool((out[:4] == 0).all())
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    assert bool(((out.cpu().double() - ref).abs() <= tol)[4].all())


def test_attention_over_a_row_with_nan_is_nan():
    g = torch.Generator().manual_seed(6)
    bt, nb = R.tables([40, 40], 16, g)
    k, v, ks, vs = R.random_cache(nb, 2, 16, 64, "i8", g)
    ks[int(bt[0, 1]), 0, 3] = math.nan
    vs[int(bt[0, 2]), 1, 1] = math.nan
    q = torch.randn(2, 4, 64, generator=g).bfloat16()
    out = pkv.paged_decode_attention_q8(*cuda(q, k, v, ks, vs, bt, i32([40, 40])))
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (24, 2)])
def test_a_head_of_q_is_alone_with_its_infinities_and_its_size(Hq, Hkv):
    """Heads of one group share a warp: one with an infinity, one with NaN and one of
    1e30 leave the others' results as they are."""
    lens = [300, 40]
    g = torch.Generator().manual_seed(61)
    bt, nb = R.tables(lens, 16, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, 64, "i8", g)
    q = torch.randn(2, Hq, 64, generator=g).bfloat16()
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    bad = q.clone()
    bad[0, 1, 5], bad[0, 3, 7], bad[1, 2] = math.inf, math.nan, 1e30
    out = pkv.paged_decode_attention_q8(*cuda(bad, k, v, ks, vs, bt, i32(lens))).cpu().double()
    hit = torch.zeros(2, Hq, dtype=torch.bool)
    hit[0, 1] = hit[0, 3] = hit[1, 2] = True
    assert bool(((out - ref).abs() <= tol)[~hit].all())
    assert bool(torch.isnan(out[0, 1]).all()) and bool(torch.isnan(out[0, 3]).all())


def test_addresses_that_are_not_16_byte_aligned():
    """Every call on tensors that begin one element into their storage."""
    def shifted(t):
        flat = torch.zeros(t.numel() + 1, dtype=torch.uint8 if t.element_size() == 1 else t.dtype, device="cuda")
        out = flat[1:].view(t.dtype).view(t.shape)
        out.copy_(t.cuda())
        assert out.is_contiguous() and out.data_ptr() % 16
        return out

    Hq, Hkv, D, BS, lens = 8, 2, 64, 16, [70, 33, 1]
    g = torch.Generator().manual_seed(62)
    bt, nb = R.tables(lens, BS, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, "e4m3", g)
    q, kn, vn = (torch.randn(3, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    odd = [shifted(t) for t in (q, k, v, ks, vs)]
    gbt, sl = bt.cuda(), i32(lens).cuda()
    out = pkv.paged_decode_attention_q8(*odd, gbt, sl, out=shifted(torch.zeros_like(q)))
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    w = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16()
    even = cuda(k.clone(), v.clone(), ks.clone(), vs.clone())
    freqs = pkv.rope_freqs(D)
    q1 = pkv.qk_norm_rope_append(shifted(q), shifted(kn), shifted(vn), shifted(w), shifted(w), 1e-6, freqs, *odd[1:3],
                                 gbt, sl, k_scale=odd[3], v_scale=odd[4])
    q2 = pkv.qk_norm_rope_append(*cuda(q, kn, vn, w, w), 1e-6, freqs, *even[:2], gbt, sl, k_scale=even[2],
                                 v_scale=even[3])
    # two kernels whose sums are grouped differently: a bf16 step, a float32 half-step of the scale
    assert bool(((q1.float() - q2.float()).abs() <= 2.0 ** -7 * q2.float().abs() + 1e-6).all())
    assert torch.equal(odd[2].view(torch.uint8), even[1].view(torch.uint8)) and torch.equal(odd[4], even[3])
    assert bool(((odd[3] - even[2]).abs() <= 2.0 ** -20 * even[2]).all())


def test_attention_beyond_32_bit_offsets():
    """Pools of more than 2^31 bytes, read at their far end, and an append there."""
    Hkv, D, BS, lens = 8, 128, 16, [50, 33]
    nb = (1 << 31) // (Hkv * D * BS) + 10
    g = torch.Generator().manual_seed(9)
    bt, small = R.tables(lens, BS, g, spare=0)
    k, v, ks, vs = R.random_cache(small, Hkv, BS, D, "i8", g)
    gk = torch.zeros(nb, Hkv, BS, D, dtype=torch.int8, device="cuda")
    gv, gks = torch.zeros_like(gk), torch.ones(nb, Hkv, BS, device="cuda")
    gvs = torch.ones_like(gks)
    for big, part in ((gk, k), (gv, v), (gks, ks), (gvs, vs)):
        big[nb - small:] = part.cuda()
    far = bt + (nb - small)
    q = torch.randn(2, 32, D, generator=g).bfloat16()
    new = torch.randn(2, Hkv, D, generator=g)
    sl = i32(lens).cuda()
    pkv.kv_append_q8(new.cuda(), new.cuda(), gk, gv, gks, gvs, far.cuda(), sl)
    blk, slot, _ = place(lens, [1, 1], bt, BS)
    vals, sc = R.store(new, "i8")
    for p, s in ((k, ks), (v, vs)):
        p[blk, :, slot], s[blk, :, slot] = vals, sc
    out = pkv.paged_decode_attention_q8(q.cuda(), gk, gv, gks, gvs, far.cuda(), sl)
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
    ko, _ = pkv.kv_read_blocks_q8(gk, gv, gks, gvs, i32([nb - 1]).cuda(), dtype=torch.float32)
    assert torch.equal(ko.cpu()[0], k[-1].float() * ks[-1][..., None])


# ------------------------------------------------------------------ norm, rotation, append
PREPARE = [  # (Hq, Hkv, D, BS, rot, interleaved, norms, lens, counts)
    (32, 8, 128, 16, 128, False, True, [1, 700, 131072, 40], None),
    (8, 2, 64, 16, 32, True, True, [100000, 5], None),
    (4, 1, 128, 16, 64, False, False, [60, 90], [60, 31]),
    (6, 3, 80, 32, 80, True, True, [70, 33, 9], [64, 0, 9]),
    (5, 5, 100, 8, 50, False, True, [50, 2000000000], [20, 3]),
    (2, 1, 256, 16, 256, False, True, [30, 31], [30, 1]),
    (3, 1, 36, 16, 10, True, True, [30], None),
    (2, 2, 96, 16, 0, False, True, [17, 18], None),
    (7, 1, 24, 16, 24, False, True, [40], [33]),
    (2, 1, 5, 3, 4, True, True, [7, 8], None),
    (1, 1, 2, 1, 2, False, True, [3], [3]),
    (16, 4, 112, 16, 26, False, True, [300, 1], [150, 1]),
    # many tokens: several of them a CTA
    (8, 2, 64, 16, 64, False, True, [800, 300], [640, 77]),
    (3, 1, 128, 16, 128, True, True, [700], [700]),
    (6, 3, 128, 32, 40, False, False, [650, 90, 5], [650, 33, 5]),
    (2, 2, 64, 16, 0, False, True, [100620, 44], [620, 2]),
    (5, 5, 64, 16, 22, True, True, [700, 9], [610, 9]),
    # more: two warps a token, then one
    (4, 1, 128, 16, 128, False, True, [1500, 90], [1400, 7]),
    (3, 1, 64, 16, 26, False, True, [2700, 40], [2600, 30]),
    (4, 2, 64, 16, 48, True, True, [2700], [2600]),
    (2, 1, 128, 16, 0, False, True, [2100, 3], [2000, 0]),
    (6, 2, 80, 32, 80, False, False, [7000], [6900]),
]


@pytest.mark.parametrize("cache", ["plain", "e4m3", "i8"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("case", range(len(PREPARE)))
def test_norm_rope_append(case, dtype, cache):
    """Tolerances: up to 32 float32 half-steps of what is added into an element
    (norm: 13 additions on the longest path, the division, eps and rsqrt enter
    with half their error, two products; rotation: two products, one sum, the
    angle's rounding of pi 2^-24 and 2 units of sincospi), then the output's
    own rounding.  In 8 bits the row's scale moves by the same amount relative to
    its largest element."""
    Hq, Hkv, D, BS, rot, inter, norms, lens, counts = PREPARE[case]
    g = torch.Generator().manual_seed(300 + case)
    n = counts or [1] * len(lens)
    T, dt = sum(n), DTYPES[dtype]
    width = -(-max(lens) // BS)
    wide = width > 1 << 20  # a far position: the table is long, its early blocks not in the pool
    first = [(L - m) // BS for L, m in zip(lens, n)]
    last = [-(-L // BS) for L in lens]
    need = sum(b - a for a, b in zip(first, last))
    nb = need + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b in range(len(lens)):
        bt[b, first[b]:last[b]] = perm[at:at + last[b] - first[b]]
        at += last[b] - first[b]
    x = (2 * torch.randn(T, Hq + 2 * Hkv, D, generator=g)).to(dt)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(dt) if norms else None for _ in range(2))
    inv_freq = [10000.0 ** (-2 * j / rot) for j in range(rot // 2)] if rot else []
    freqs = pkv.rope_freqs(rot) if rot else None
    if cache == "plain":
        k, v = (torch.randn(nb, Hkv, BS, D, generator=g).to(dt) for _ in range(2))
        ks = vs = None
    else:
        k, v, ks, vs = R.random_cache(nb, Hkv, BS, D, cache, g)
    gx, gk, gv = cuda(x, k, v)
    gks, gvs = (None, None) if ks is None else cuda(ks, vs)
    qs = None
    if counts is not None:
        qs = torch.zeros(len(lens) + 1, dtype=torch.int32)
        qs[1:] = torch.cumsum(i32(counts), 0)
        qs = qs.cuda()
    st = pkv.new_status()
    qo = pkv.qk_norm_rope_append(gx[:, :Hq], gx[:, Hq:Hq + Hkv], gx[:, Hq + Hkv:], None if qw is None else qw.cuda(),
                                 None if kw is None else kw.cuda(), 1e-6, freqs, gk, gv, bt.cuda(), i32(lens).cuda(),
                                 q_start=qs, k_scale=gks, v_scale=gvs, interleaved=inter, status=st)
    assert pkv.check_status(st) == 0
    del wide
    blk, slot, pos = place(lens, n, bt, BS)
    eps_out = 2.0 ** -8 if dtype == "bf16" else R.U24
    ref, reach = R.norm_rope(x[:, :Hq], qw, 1e-6, pos, inv_freq, inter)
    assert bool(((qo.cpu().double() - ref).abs() <= eps_out * ref.abs() + 32 * R.U24 * reach).all())
    kref, reach = R.norm_rope(x[:, Hq:Hq + Hkv], kw, 1e-6, pos, inv_freq, inter)
    vnew = x[:, Hq + Hkv:]
    if cache == "plain":
        got = gk.cpu()[blk, :, slot].double()
        assert bool(((got - kref).abs() <= eps_out * kref.abs() + 32 * R.U24 * reach).all())
        gk[blk, :, slot] = 0
        k[blk, :, slot] = 0
        v[blk, :, slot] = vnew
        assert cpu_equal(gk, k) and cpu_equal(gv, v)
        return
    sc = gks.cpu()[blk, :, slot].double()
    amax = kref.abs().amax(-1)
    slack = 32 * R.U24 * reach.amax(-1)  # how far the row's largest element may be off
    assert bool(((sc - (amax / R.QMAX[cache]).clamp_min(2.0 ** -64)).abs() <= (slack + 4 * R.U24 * amax) / R.QMAX[cache]).all())
    got = R.numbers(gk.cpu().view(torch.uint8)[blk, :, slot].contiguous().view(R.DT[cache]), sc.float())
    tol = R.half_step(kref, sc, cache) * (1 + 2.0 ** -10) + 2 * slack[..., None] + 4 * R.U24 * amax[..., None]
    assert bool(((got - kref).abs() <= tol).all())
    vals, vsc = R.store(vnew, cache)
    v.view(torch.uint8)[blk, :, slot], vs[blk, :, slot] = vals.view(torch.uint8), vsc
    assert cpu_equal(gv, v) and cpu_equal(gvs, vs)
    gk.view(torch.uint8)[blk, :, slot] = 0
    k.view(torch.uint8)[blk, :, slot] = 0
    gks[blk, :, slot] = 0
    ks[blk, :, slot] = 0
    assert cpu_equal(gk, k) and cpu_equal(gks, ks)


def test_norm_rope_append_in_place_and_rows_behind_the_last_sequence():
    Hq, Hkv, D, BS = 4, 2, 64, 16
    g = torch.Generator().manual_seed(31)
    lens, counts = [20, 9], [7, 2]
    bt, nb = R.tables(lens, BS, g)
    T = 12  # three rows more than the sequences use
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    pool = torch.zeros(nb, Hkv, BS, D).bfloat16()
    qs = i32([0, 7, 9]).cuda()
    w = torch.ones(D).bfloat16().cuda()
    args = (w, w, 1e-6, pkv.rope_freqs(D))
    gq, gk, gv, k1, v1, k2, v2 = cuda(q, k, v, pool, pool, pool, pool)
    want = torch.full_like(gq, 5.0)
    pkv.qk_norm_rope_append(gq, gk, gv, *args, k1, v1, bt.cuda(), i32(lens).cuda(), q_start=qs, q_out=want)
    assert bool((want[9:] == 5).all())
    same = pkv.qk_norm_rope_append(gq, gk, gv, *args, k2, v2, bt.cuda(), i32(lens).cuda(), q_start=qs, q_out=gq)
    assert same is gq and torch.equal(gq[:9], want[:9]) and torch.equal(gq[9:].cpu(), q[9:])
    assert torch.equal(k1, k2) and torch.equal(v1, v2)


def test_many_tokens_in_place_with_rows_behind_and_bad_sequences():
    """Several tokens a CTA: 40 sequences, some of them bad, and rows that belong to none."""
    Hq, Hkv, D, BS = 4, 2, 128, 16
    g = torch.Generator().manual_seed(33)
    counts = [(7 * b) % 41 for b in range(40)]
    lens = [n + 3 * b for b, n in enumerate(counts)]
    bt, nb = R.tables(lens, BS, g)
    T = sum(counts) + 5
    assert T > 700
    bad_len, bad_blk = 11, 23
    lens[bad_len] = counts[bad_len] - 1
    bt[bad_blk, (lens[bad_blk] - 1) // BS] = nb
    qs = torch.zeros(41, dtype=torch.int32)
    qs[1:] = torch.cumsum(i32(counts), 0)
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16() for h in (Hq, Hkv, Hkv))
    pool = torch.zeros(nb, Hkv, BS, D).bfloat16()
    gq, gk, gv, kc, vc = cuda(q, k, v, pool, pool)
    st = pkv.new_status()
    out = pkv.qk_norm_rope_append(gq, gk, gv, None, None, 0.0, None, kc, vc, bt.cuda(), i32(lens).cuda(),
                                  q_start=qs.cuda(), q_out=gq, status=st)
    assert pkv.check_status(st) == 4 and out is gq
    want = q.clone()
    want[qs[bad_len]:qs[bad_len + 1]] = 0
    assert torch.equal(gq.cpu(), want)
    wk, wv = pool.clone(), pool.clone()
    for b, n in enumerate(counts):
        for i in range(n):
            pos, t = lens[b] - n + i, int(qs[b]) + i
            if b != bad_len and int(bt[b, pos // BS]) < nb:
                wk[int(bt[b, pos // BS]), :, pos % BS], wv[int(bt[b, pos // BS]), :, pos % BS] = k[t], v[t]
    assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 26, False), (80, 48, True), (128, 0, False)])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n", [1, 30, 300, 700])
def test_in_place_is_the_same_bits(D, rot, inter, dtype, n):
    """q_out is q, with rows copied ahead of their use; one sequence of five cannot be placed."""
    Hq, Hkv, BS, B = 8, 2, 16, 5
    g = torch.Generator().manual_seed(34)
    lens = [n + 11 * b for b in range(B)]
    bt, nb = R.tables(lens, BS, g)
    lens[3] = n - 1  # shorter than its chunk
    qs = i32([n * b for b in range(B + 1)]).cuda()
    q, k, v = (torch.randn(n * B, h, D, generator=g).to(DTYPES[dtype]).cuda() for h in (Hq, Hkv, Hkv))
    w = torch.rand(D, generator=g).to(DTYPES[dtype]).cuda()
    args = (1e-6, pkv.rope_freqs(rot) if rot else None)
    runs = []
    for own in (True, False):
        qq = q.clone()
        pools = [torch.zeros(nb, Hkv, BS, D, dtype=DTYPES[dtype], device="cuda") for _ in range(2)]
        st = pkv.new_status()
        out = pkv.qk_norm_rope_append(qq, k, v, w, w, *args, *pools, bt.cuda(), i32(lens).cuda(), q_start=qs,
                                      interleaved=inter, q_out=qq if own else None, status=st)
        assert pkv.check_status(st) == 4 and bool((out[3 * n:4 * n] == 0).all())
        runs.append((out, *pools))
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_norm_rope_append_bad_sequences():
    Hq, Hkv, D, BS = 4, 2, 64, 16
    g = torch.Generator().manual_seed(32)
    lens = [20, 3, 9, 17]
    counts = [2, 4, 2, 3]        # sequence 1: more new tokens than its length
    bt, nb = R.tables([20, 16, 9, 17], BS, g)
    bt[3, 1] = nb + 4            # sequence 3: its last token has no block
    T = sum(counts)
    q, k, v = (torch.randn(T, h, D, generator=g) for h in (Hq, Hkv, Hkv))
    pool = torch.zeros(nb, Hkv, BS, D)
    gq, gk, gv, kc, vc = cuda(q, k, v, pool, pool)
    st = pkv.new_status()
    qo = pkv.qk_norm_rope_append(gq, gk, gv, None, None, 0.0, None, kc, vc, bt.cuda(), i32(lens).cuda(),
                                 q_start=i32([0, 2, 6, 8, 11]).cuda(), status=st)
    assert pkv.check_status(st) == 4
    want = q.clone()
    want[2:6] = 0
    assert torch.equal(qo.cpu(), want)
    ok = [0, 1, 6, 7, 8, 9]
    blk = [int(bt[b, p // BS]) for b, p in ((0, 18), (0, 19), (2, 7), (2, 8), (3, 14), (3, 15))]
    slot = [18 % BS, 19 % BS, 7, 8, 14, 15]
    wk, wv = pool.clone(), pool.clone()
    wk[blk, :, slot], wv[blk, :, slot] = k[ok], v[ok]
    assert torch.equal(kc.cpu(), wk) and torch.equal(vc.cpu(), wv)


def test_python_refusals_on_the_gpu():
    k = torch.zeros(2, 2, 16, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(2, 2, 16, device="cuda")
    bt, sl = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    row = torch.zeros(1, 2, 64, device="cuda")
    half = torch.zeros(1, 2, 64, device="cuda", dtype=torch.float16)
    bad = [
        (TypeError, lambda: pkv.kv_append_q8(half, half, k, k, s, s, bt, sl)),
        (TypeError, lambda: pkv.kv_append_q8(row, row.bfloat16(), k, k, s, s, bt, sl)),
        (ValueError, lambda: pkv.kv_append_q8(row[:, :1], row[:, :1], k, k, s, s, bt, sl)),
        (TypeError, lambda: pkv.kv_append_q8(row, row, k, k.view(torch.float8_e4m3fn), s, s, bt, sl)),
        (ValueError, lambda: pkv.kv_append_q8(row, row, k, k, s[:1], s, bt, sl)),
        (TypeError, lambda: pkv.kv_append_q8(row, row, k, k, s.double(), s, bt, sl)),
        (TypeError, lambda: pkv.kv_append_q8(row, row, k, k, s, s, bt.long(), sl)),
        (ValueError, lambda: pkv.kv_append_q8(row, row, k, k, s, s, bt[0], sl)),
        (ValueError, lambda: pkv.kv_append_q8(row, row, k, k, s, s, bt.cpu(), sl)),
        (ValueError, lambda: pkv.kv_append_q8(row.transpose(1, 2), row, k, k, s, s, bt, sl)),
        (ValueError, lambda: pkv.paged_decode_attention_q8(row[..., :32].contiguous(), k, k, s, s, bt, sl)),
        (pkv.PkvError, lambda: pkv.paged_decode_attention_q8(row, k, k, s, s, bt, sl,
                                                             workspace=torch.zeros(16, dtype=torch.uint8,
                                                                                   device="cuda"))),
        (pkv.PkvError, lambda: pkv.paged_decode_attention_q8(torch.zeros(1, 3, 64, device="cuda"), k, k, s, s, bt, sl)),
        (TypeError, lambda: pkv.kv_read_blocks_q8(k, k, s, s, sl, dtype=torch.float16)),
        (TypeError, lambda: pkv.kv_read_blocks_q8(k, k, s, s, sl.long())),
        (ValueError, lambda: pkv.qk_norm_rope_append(torch.cat([row, row]), row, row, None, None, 1e-6, None, k, k,
                                                     bt, sl, k_scale=s, v_scale=s)),
        (ValueError, lambda: pkv.qk_norm_rope_append(row.transpose(1, 2).contiguous().transpose(1, 2), row, row, None,
                                                     None, 1e-6, None, k, k, bt, sl, k_scale=s, v_scale=s)),
        (TypeError, lambda: pkv.qk_norm_rope_append(row, row, row, None, None, 1e-6, None, k, k, bt, sl)),
        (pkv.PkvError, lambda: pkv.qk_norm_rope_append(row, row, row, None, None, 1e-6, pkv.rope_freqs(66), k, k, bt,
                                                       sl, k_scale=s, v_scale=s)),
        (TypeError, lambda: pkv.copy_blocks(k.float(), k.float(), sl, sl, k_scale=s, v_scale=s)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt", FMTS)
def test_a_prompt_and_decode_steps_together(fmt):
    """A prompt chunk prepared and stored, its blocks read back for prefill
    attention, a fork with copy-on-write, then decode steps over the 8-bit cache, one
    of them as a captured graph: every stage against float64 from the cache's
    own numbers."""
    Hq, Hkv, D, BS = 16, 4, 128, 16
    g = torch.Generator().manual_seed(77)
    prompt = [37, 64]
    pool = pkv.BlockPool(40, BS, 10)
    for i, L in enumerate(prompt):
        pool.add(i, L)
    bt, sl = pool.tables([0, 1])
    k, v = (torch.zeros(40, Hkv, BS, D, dtype=R.DT[fmt], device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(40, Hkv, BS, device="cuda") for _ in range(2))
    w = (1 + 0.1 * torch.randn(D, generator=g)).bfloat16().cuda()
    freqs = pkv.rope_freqs(D)
    st = pkv.new_status()

    def prepare(T, bt, sl, qs=None):
        x = torch.randn(T, Hq + 2 * Hkv, D, generator=g).bfloat16().cuda()
        return pkv.qk_norm_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], w, w, 1e-6, freqs, k, v, bt, sl,
                                       q_start=qs, k_scale=ks, v_scale=vs, status=st)

    qs = i32([0, 37, 101]).cuda()
    q = prepare(101, bt.cuda(), sl.cuda(), qs)
    # prefill attention over the blocks read back (their rounding to bf16 is prefill's own input)
    used = [int(b) for row, L in zip(bt, prompt) for b in row[:-(-L // BS)]]
    kb, vb = pkv.kv_read_blocks_q8(k, v, ks, vs, i32(used).cuda(), status=st)
    rt = torch.full_like(bt, -1)
    rt[0, :3], rt[1, :4] = torch.arange(3), torch.arange(3, 7)
    pre = pkv.paged_prefill_attention(q, kb, vb, rt.cuda(), sl.cuda(), qs, status=st)
    for b, (t0, L) in enumerate(((0, 37), (37, 64))):  # the last chunk row sees the whole prompt
        ids = rt[b, :-(-L // BS)].long()
        kk = kb.cpu()[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double().repeat_interleave(Hq // Hkv, 0)
        vv = vb.cpu()[ids].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double().repeat_interleave(Hq // Hkv, 0)
        s = torch.einsum("hd,hld->hl", q[t0 + L - 1].cpu().double(), kk) / math.sqrt(D)
        want = torch.einsum("hl,hld->hd", torch.softmax(s, -1), vv)
        # bf16 weights and a bf16 output: 2^-8 of what is added up each
        W = torch.einsum("hl,hld->hd", torch.softmax(s, -1), vv.abs())
        assert bool(((pre[t0 + L - 1].cpu().double() - want).abs() <= 2 * 2.0 ** -8 * W + 1e-5).all())
    # a fork of sequence 0 writes its own copy of the shared tail block
    pool.fork(0, 2)
    pairs = [p for p in (pool.append(i) for i in (2, 0, 1)) if p]
    assert len(pairs) == 1
    pkv.copy_blocks(k, v, i32([pairs[0][0]]).cuda(), i32([pairs[0][1]]).cuda(), status=st, k_scale=ks, v_scale=vs)
    for p in (k, v):
        assert torch.equal(p[pairs[0][0]].view(torch.uint8), p[pairs[0][1]].view(torch.uint8))
    assert torch.equal(ks[pairs[0][0]], ks[pairs[0][1]]) and torch.equal(vs[pairs[0][0]], vs[pairs[0][1]])
    for step in range(3):
        if step:
            for i in (0, 1, 2):
                pool.append(i)
        bt, sl = pool.tables([0, 1, 2])
        q = prepare(3, bt.cuda(), sl.cuda())
        out = pkv.paged_decode_attention_q8(q, k, v, ks, vs, bt.cuda(), sl.cuda(), status=st)
        assert pkv.check_status(st) == 0
        ref, tol = R.attention(q, k.cpu(), v.cpu(), ks.cpu(), vs.cpu(), bt, sl.tolist(), dtype="bf16")
        assert bool(((out.cpu().double() - ref).abs() <= tol).all())


def test_decode_step_object_on_an_8_bit_cache():
    """DecodeStep with k_scale / v_scale runs the append, the attention and the
    sampler of the separate calls."""
    Hq, Hkv, D, BS, V = 8, 2, 64, 16, 1000
    g = torch.Generator().manual_seed(41)
    lens = [30, 1, 64]
    bt, nb = R.tables(lens, BS, g)
    caches = cuda(*R.random_cache(nb, Hkv, BS, D, "e4m3", g))
    other = [t.clone() for t in caches]
    q = torch.randn(3, Hq, D, generator=g).bfloat16().cuda()
    kn, vn = (torch.randn(3, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    gbt, sl = bt.cuda(), i32(lens).cuda()
    logits = torch.randn(3, V, generator=g).cuda()
    samp = (torch.full((3,), 0.8, device="cuda"), i32([5] * 3).cuda(), torch.full((3,), 0.9, device="cuda"),
            torch.arange(3, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda"))
    step = pkv.DecodeStep(q, kn, vn, *caches[:2], gbt, sl, logits, *samp, k_scale=caches[2], v_scale=caches[3])
    tok = step.run().clone()
    pkv.kv_append_q8(kn, vn, *other, gbt, sl)
    out = pkv.paged_decode_attention_q8(q, *other, gbt, sl)
    assert torch.equal(step.out, out) and torch.equal(tok, pkv.sample_tokens(logits, *samp))
    for a, b in zip(caches, other):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_and_two_graphs_at_once():
    """The same calls on two streams and as two captured graphs give what one
    stream gives: no workspace is shared."""
    Hq, Hkv, D, BS = 32, 8, 128, 16
    sets = []
    for seed in (51, 52):
        g = torch.Generator().manual_seed(seed)
        lens = [900 + 37 * seed, 40, 333]
        bt, nb = R.tables(lens, BS, g)
        sets.append((torch.randn(3, Hq, D, generator=g).bfloat16().cuda(),
                     *cuda(*R.random_cache(nb, Hkv, BS, D, "i8", g)), bt.cuda(), i32(lens).cuda()))
    want = [pkv.paged_decode_attention_q8(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    graphs, outs = [], []
    for s, a in zip(streams, sets):
        with torch.cuda.stream(s):
            pkv.paged_decode_attention_q8(*a)  # warm
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            outs.append(pkv.paged_decode_attention_q8(*a))
        graphs.append(gr)
    for _ in range(5):
        direct = []
        for s, a, gr in zip(streams, sets, graphs):
            with torch.cuda.stream(s):
                gr.replay()
                direct.append(pkv.paged_decode_attention_q8(*a))
        torch.cuda.synchronize()
        for w, d, o in zip(want, direct, outs):
            assert torch.equal(w, d) and torch.equal(w, o)
