"""The 8-bit cache's calls at the edges of what they are documented for."""
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
