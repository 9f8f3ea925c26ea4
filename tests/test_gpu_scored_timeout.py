"""A CTA of the split decode kernel whose loader issues no copy: its consumers give up after the poll budget, the call
reports it, and the next call is as before."""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
import scored_ref as R

pytestmark = pytest.mark.gpu


def _reset():
    torch.cuda.synchronize()
    pkv.test_set_wait_limit()


@pytest.mark.parametrize("shared", [False, True])
def test_silent_loader(shared):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()
    x = R.make(3, [1500 + 10 * i for i in range(6)], 16, 4, 128, 16, torch.bfloat16)
    bt = x["block_tables"]
    bt[:, :60] = bt[0, :60]  # 960 positions of one sequence in front of all
    if shared:  # a wide table, so that the prefix is read once
        bt = torch.cat([bt, torch.full((6, 500), -1, dtype=torch.int32, device="cuda")], 1)
        more = (torch.tensor([0, 6], dtype=torch.int32, device="cuda"), torch.tensor([960], dtype=torch.int32, device="cuda"))
        call = lambda st=None: pkv.paged_decode_attention_shared(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"],
                                                                 *more, softcap=9.0, status=st)
    else:
        call = lambda st=None: pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"],
                                                                 softcap=9.0, status=st)
    ref, tol = R.reference(x, softcap=9.0)
    want = call()
    R.check(want, ref, tol)
    try:
        pkv.test_set_wait_limit(2000, 1)
        st = pkv.new_status()
        call(st)
        assert pkv.check_status(st) == 5
    finally:
        _reset()
    st = pkv.new_status()
    assert torch.equal(call(st), want)
    assert pkv.check_status(st) == 0


def _gives_up(call, cta, out=None):
    """With a silent CTA the call reports it, and every row is what it would be or zeros; the next call is as before."""
    want = call(None, None)
    torch.cuda.synchronize()
    try:
        pkv.test_set_wait_limit(2000, cta)
        st = pkv.new_status()
        got = call(st, out)
        assert pkv.check_status(st) == 5
    finally:
        _reset()
    same, zero = (got == want).all(-1), (got == 0).all(-1)
    assert (same | zero).all()
    assert not same.all()
    st = pkv.new_status()
    assert torch.equal(call(st, None), want)
    assert pkv.check_status(st) == 0


def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


@pytest.mark.parametrize("cta", [0, 1])
@pytest.mark.parametrize("lens,Hq,Hkv,D", [([40000], 16, 4, 128), ([700] * 300 + [0, 5, 30000], 16, 4, 128),  # pieces, whole ones
                                           ([300 + i for i in range(200)], 48, 2, 64), ([50] * 400, 22, 11, 128),
                                           ([60, 30], 16, 4, 128)])  # a CTA for each
def test_silent_loader_of_decode(lens, Hq, Hkv, D, cta):
    _lib()
    x = R.make(3, lens, Hq, Hkv, D, 16, torch.bfloat16)
    _gives_up(lambda st, out: pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"],
                                                                x["seq_lens"], softcap=9.0, out=out, status=st), cta,
              torch.full_like(x["q"], float("nan")))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cta", [0, 3, 20])
@pytest.mark.parametrize("members", [6, 70])  # few rows are held by both query tiles, which take key tiles in turn
def test_silent_loader_of_a_prefix(D, cta, members):
    _lib()
    x = R.make(4, [1000 + 10 * i for i in range(members)], 16, 4, D, 16, torch.bfloat16)
    bt = x["block_tables"]
    bt[:, :60] = bt[0, :60]
    more = max(0, (48 << 20) // (4 * members * 16 * 4 * D) + 1 - bt.shape[1])  # so that the prefix is read once
    bt = torch.cat([bt, torch.full((members, more), -1, dtype=torch.int32, device="cuda")], 1)
    groups = (torch.tensor([0, members], dtype=torch.int32, device="cuda"),
              torch.tensor([960], dtype=torch.int32, device="cuda"))
    _gives_up(lambda st, out: pkv.paged_decode_attention_shared(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"],
                                                                *groups, softcap=9.0, status=st), cta)


@pytest.mark.parametrize("kw", [None, {}, dict(softcap=9.0)])  # None: the plain call
@pytest.mark.parametrize("chunks,before", [([40], 3000), ([3], 3000), ([500, 70, 130] * 16, 600)])  # shared keys, both query tiles, neither
def test_silent_loader_of_prefill(kw, chunks, before):
    _lib()
    x = R.make(6, [n + before for n in chunks], 16, 4, 128, 16, torch.bfloat16, chunks=chunks)
    a = [x[k] for k in ("q", "k_cache", "v_cache", "block_tables", "seq_lens", "q_start")]

    def call(st, out):
        if kw is None:
            return pkv.paged_prefill_attention(*a, out=out, status=st)
        return pkv.paged_prefill_attention_scored(*a, out=out, status=st, **kw)

    _gives_up(call, 0, torch.full_like(x["q"], float("nan")))
    _gives_up(call, 1, torch.full_like(x["q"], float("nan")))
