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
