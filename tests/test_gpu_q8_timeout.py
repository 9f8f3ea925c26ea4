"""The 8-bit attention's bounded waits: a loader that issues no copy makes the
consumers give up with PKV_ERR_TIMEOUT, and the next call computes normally."""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
from tests import q8_ref as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 1, 64), (24, 2, 80)])
def test_a_silent_loader_times_out_and_the_context_stays_usable(Hq, Hkv, D):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    lens = [700, 90]
    g = torch.Generator().manual_seed(3)
    bt, nb = R.tables(lens, 16, g)
    k, v, ks, vs = R.random_cache(nb, Hkv, 16, D, "i8", g)
    q = torch.randn(2, Hq, D, generator=g).bfloat16()
    args = [t.cuda() for t in (q, k, v, ks, vs, bt, torch.tensor(lens, dtype=torch.int32))]
    st = pkv.new_status()
    pkv.test_set_wait_limit(2000, 0)
    try:
        pkv.paged_decode_attention_q8(*args, status=st)
        assert pkv.check_status(st) == 5
    finally:
        pkv.test_set_wait_limit()
    st.zero_()
    out = pkv.paged_decode_attention_q8(*args, status=st)
    assert pkv.check_status(st) == 0
    ref, tol = R.attention(q, k, v, ks, vs, bt, lens, dtype="bf16")
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
