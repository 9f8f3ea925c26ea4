"""Calls whose waits may run out everywhere: the loaders do issue their copies, but the limit of polls is so short that
consumers give up on cold data.  Whatever a call then gives, it reports, and the next call is as before."""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
import scored_ref as R
from tests import q8_ref

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()
    yield
    torch.cuda.synchronize()
    pkv.test_set_wait_limit()


def short(call, repeat=20):
    """call(status) -> out: with short limits it reports what happened, and afterwards gives what it gave before."""
    want = call(None)
    cold = torch.empty(192 << 20, dtype=torch.uint8, device="cuda")  # larger than the L2 cache
    seen = set()
    try:
        for i in range(repeat):
            pkv.test_set_wait_limit(1 + i % 3, -1)
            cold.fill_(i)
            st = pkv.new_status()
            call(st)
            seen.add(pkv.check_status(st))
    finally:
        torch.cuda.synchronize()
        pkv.test_set_wait_limit()
    assert seen <= {0, 5}
    st = pkv.new_status()
    assert torch.equal(call(st), want)
    assert pkv.check_status(st) == 0


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([30, 20], 8, 2, 64), ([90, 7, 60], 32, 8, 128),  # a CTA a sequence
                                           ([1500 + 10 * i for i in range(6)], 16, 4, 128), ([700] * 40, 32, 2, 64)])
def test_decode_with_changed_scores(lens, Hq, Hkv, D):
    x = R.make(5, lens, Hq, Hkv, D, 16, BF)
    short(lambda st: pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                                       softcap=9.0, status=st))


@pytest.mark.parametrize("lens,Hq,Hkv", [([30, 20], 8, 2), ([1500 + 10 * i for i in range(6)], 32, 8)])
def test_plain_decode(lens, Hq, Hkv):
    x = R.make(5, lens, Hq, Hkv, 128, 16, BF)
    short(lambda st: pkv.paged_decode_attention(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                                status=st))


@pytest.mark.parametrize("lens", [[30, 20], [1500 + 10 * i for i in range(6)]])
def test_decode_of_the_8_bit_cache(lens):
    g = torch.Generator().manual_seed(3)
    bt, nb = q8_ref.tables(lens, 16, g)
    k, v, ks, vs = q8_ref.random_cache(nb, 8, 16, 128, "i8", g)
    q = torch.randn(len(lens), 32, 128, generator=g).bfloat16()
    args = [t.cuda() for t in (q, k, v, ks, vs, bt, torch.tensor(lens, dtype=torch.int32))]
    short(lambda st: pkv.paged_decode_attention_q8(*args, status=st))


@pytest.mark.parametrize("D,members", [(128, 5), (128, 70), (64, 5)])
def test_shared_prefixes(D, members):
    x = R.make(5, [1000 + 10 * i for i in range(members)], 16, 4, D, 16, BF)
    bt = x["block_tables"]
    bt[:, :60] = bt[0, :60]
    more = max(0, (48 << 20) // (4 * members * 16 * 4 * D) + 1 - bt.shape[1])  # so that the prefix is read once
    bt = torch.cat([bt, torch.full((members, more), -1, dtype=torch.int32, device="cuda")], 1)
    groups = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, members], [960])]
    short(lambda st: pkv.paged_decode_attention_shared(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"], *groups,
                                                       softcap=9.0, status=st), 4)


@pytest.mark.parametrize("chunks,before", [([40], 3000), ([3], 3000), ([500, 70, 130] * 16, 600)])
@pytest.mark.parametrize("kw", [None, dict(softcap=9.0)])
def test_prefill(chunks, before, kw):
    x = R.make(6, [n + before for n in chunks], 16, 4, 128, 16, BF, chunks=chunks)
    a = [x[k] for k in ("q", "k_cache", "v_cache", "block_tables", "seq_lens", "q_start")]
    call = pkv.paged_prefill_attention if kw is None else pkv.paged_prefill_attention_scored
    short(lambda st: call(*a, status=st, **(kw or {})), 4)
