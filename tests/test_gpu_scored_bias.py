"""Biases over long distances: a few keys far away (or next to the query) whose products make up for their biases exactly,
so that they share the weight.  A bias measured from the other end would be millions, between whose float32 neighbours
lies the whole weight."""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
STEEP = 16.0
MORE = (0.0, 0.125, 0.25, 0.5)  # what the products have on top of that: less than float32 keeps of millions
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


def make(L, first, n, Hq, Hkv, D, dtype, BS=16):
    """A sequence of L, whose last n tokens are the queries.  Head qh has slope -16 (even) or 16 (odd); its query picks dimension
    0 or 1.  There K is 16 i + MORE[i] at first + i, and at L - 1 - i, i < 4: with slope -16 and distances from `first`
    all four are MORE[i], and as much with 16 and distances from L - 1.  All other products are 0."""
    g = torch.Generator(device="cuda")
    g.manual_seed(L + D)
    NB = -(-L // BS)
    k = torch.zeros((NB, Hkv, BS, D), device="cuda", dtype=dtype)
    v = torch.randn((NB, Hkv, BS, D), generator=g, device="cuda").to(dtype)
    for i in range(4):
        a, b = first + i, L - 1 - i
        k[a // BS, :, a % BS, 0] = STEEP * i + MORE[i]
        k[b // BS, :, b % BS, 1] = STEEP * i + MORE[i]
    q = torch.zeros((n, Hq, D), device="cuda", dtype=dtype)
    q[:, 0::2, 0] = 1.0
    q[:, 1::2, 1] = 1.0
    slopes = torch.full((Hq,), STEEP, device="cuda")
    slopes[0::2] = -STEEP
    return dict(q=q, k_cache=k, v_cache=v, block_tables=torch.arange(NB, dtype=torch.int32, device="cuda").view(1, -1),
                seq_lens=torch.tensor([L], dtype=torch.int32, device="cuda"), slopes=slopes)


def expected(x, L, first, n, window=0, prefix=0, spread=None):
    """(out, tolerance) over the keys around both ends of what each row sees (spread: how far apart the rows' ends lie, n by
    default): all others are e^-64 or less of the weight, 2^-70 with their number.

    Scores of up to 3 * 16 log2(e) = 70 and a maximum of as much are rounded at most 6 times each (scale, slope, their
    products, the sum, the exponent), which moves a weight by 12 * 70 e, numerator and denominator; weights (1 / 4 .. 1)
    are rounded to 16 bits at most once, the output once."""
    dt, BS = x["q"].dtype, x["k_cache"].shape[2]
    Hq, Hkv = x["q"].shape[1], x["k_cache"].shape[1]
    m = 64 + (n if spread is None else spread)
    j = torch.tensor(sorted(set(range(min(64, L))) | set(range(first, min(L, first + m))) | set(range(max(0, L - m), L))), device="cuda")
    k, v = (x[c][j // BS, :, j % BS].double().repeat_interleave(Hq // Hkv, 1) for c in ("k_cache", "v_cache"))
    pos = torch.arange(L - n, L, device="cuda").view(n, 1, 1)
    s = torch.einsum("nhd,jhd->nhj", x["q"].double(), k) + x["slopes"].double().view(1, -1, 1) * (j.view(1, 1, -1) - pos)
    hidden = (j > pos) | ((j <= pos - window) if window > 0 else torch.zeros_like(j > pos))
    w = torch.softmax(s.masked_fill(hidden & (j >= prefix), float("-inf")), -1)
    out, size = torch.einsum("nhj,jhd->nhd", w, v), torch.einsum("nhj,jhd->nhd", w, v.abs())
    half = 2.0 ** -8 if dt == BF else E
    return out, half * out.abs() + (2 * 12 * 70 * E + (half if dt == BF else 0.0) + 64 * E) * size


def check(got, ref, tol):
    over = (got.double() - ref).abs() - tol
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()} out of tolerance, by up to {over.max():.3e}"


MASKS = [(0, 0), (150000, 0), (70001, 5)]  # window, prefix


@pytest.mark.parametrize("window,prefix", MASKS)
@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(F32, 4, 2, 64), (F32, 2, 1, 30), (BF, 4, 2, 128), (BF, 2, 1, 64), (BF, 24, 2, 128),
                                            (BF, 2, 1, 200)])
def test_decode(dtype, Hq, Hkv, D, window, prefix):
    L = 300007
    first = 0 if prefix or not window else L - window
    x = make(L, first, 1, Hq, Hkv, D, dtype)
    pl = torch.tensor([prefix], dtype=torch.int32, device="cuda") if prefix else None
    st = pkv.new_status()
    got = pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                            slopes=x["slopes"], window=window, prefix_lens=pl, scale=1.0, status=st)
    assert pkv.check_status(st) == 0
    check(got, *expected(x, L, first, 1, window, prefix))


@pytest.mark.parametrize("Hq,Hkv,D,members", [(4, 2, 128, 2), (4, 2, 64, 3), (16, 2, 128, 40)])
def test_shared(Hq, Hkv, D, members):
    """All of a group have the same tokens up to the end of the prefix, and here behind it."""
    L = 300007
    x = make(L, 0, 1, Hq, Hkv, D, BF)
    st = pkv.new_status()
    got = pkv.paged_decode_attention_shared(x["q"].repeat(members, 1, 1), x["k_cache"], x["v_cache"],
                                            x["block_tables"].repeat(members, 1), x["seq_lens"].repeat(members),
                                            torch.tensor([0, members], dtype=torch.int32, device="cuda"),
                                            torch.tensor([L - 70], dtype=torch.int32, device="cuda"), slopes=x["slopes"],
                                            scale=1.0, status=st)
    assert pkv.check_status(st) == 0
    ref, tol = expected(x, L, 0, 1)
    check(got, ref.expand_as(got), tol.expand_as(got))


@pytest.mark.parametrize("window,prefix", MASKS)
@pytest.mark.parametrize("n", [1, 3, 200])
def test_prefill(n, window, prefix):
    L = 300007
    first = 0 if prefix or not window else L - n - window + 1
    x = make(L, first, n, 4, 2, 128, BF)
    pl = torch.tensor([prefix], dtype=torch.int32, device="cuda") if prefix else None
    st = pkv.new_status()
    got = pkv.paged_prefill_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), slopes=x["slopes"],
                                             window=window, prefix_lens=pl, scale=1.0, status=st)
    assert pkv.check_status(st) == 0
    ref, tol = expected(x, L, first, n, window, prefix)
    check(got, ref, tol)


def test_prefill_keys_behind_the_query():
    """A prefix that attends in both directions: with a positive slope the last key of the prefix is the one that the bias
    favours, for rows in front of it too."""
    n = L = 20000
    x = make(L, 0, n, 2, 1, 128, BF)
    st = pkv.new_status()
    got = pkv.paged_prefill_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), slopes=x["slopes"],
                                             prefix_lens=x["seq_lens"], scale=1.0, status=st)
    assert pkv.check_status(st) == 0
    ref, tol = expected(x, L, 0, n, 0, L, spread=0)
    check(got, ref, tol)
