"""8-bit cache operators without a GPU: exported symbols, refusals that return
before a launch, workspace sizing, the rotation's frequencies, and the plain
implementations the GPU tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import q8_ref as R


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_table_gb300 import build as B
    B.build()
    import paged_kv_decode_table_gb300 as pkv
    return pkv.load_library()


P = ctypes.c_void_p
X = P(64)  # never dereferenced: every call below returns before a launch


def append(lib, k=X, v=X, kc=X, vc=X, ks=X, vs=X, bt=X, mb=1, sl=X, qs=None, B=2, T=2, Hkv=2, D=64, BS=16, NB=4, dt=1,
           ct=2):
    return lib.pkv_kv_append_q8(k, v, kc, vc, ks, vs, bt, mb, sl, qs, B, T, Hkv, D, BS, NB, dt, ct, None, None)


def test_append_refusals(lib):
    assert append(lib, B=0, T=0) == 0
    assert append(lib, T=0, qs=X) == 0
    for bad in (dict(B=-1), dict(T=-1), dict(Hkv=0), dict(D=0), dict(D=257), dict(BS=0), dict(NB=0), dict(mb=0),
                dict(dt=2), dict(dt=3), dict(dt=9), dict(ct=0), dict(ct=1), dict(ct=4), dict(T=3), dict(k=None),
                dict(v=None), dict(kc=None), dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None),
                dict(sl=None)):
        assert append(lib, **bad) == 1, bad


def read(lib, ko=X, vo=X, kc=X, vc=X, ks=X, vs=X, ids=X, n=2, Hkv=2, D=64, BS=16, NB=4, ot=1, ct=2):
    return lib.pkv_kv_read_blocks_q8(ko, vo, kc, vc, ks, vs, ids, n, Hkv, D, BS, NB, ot, ct, None, None)


def test_read_refusals(lib):
    assert read(lib, n=0) == 0
    for bad in (dict(n=-1), dict(Hkv=0), dict(D=0), dict(D=257), dict(BS=0), dict(NB=0), dict(ot=2), dict(ot=3),
                dict(ct=0), dict(ct=1), dict(ct=5), dict(ko=None), dict(vo=None), dict(kc=None), dict(vc=None),
                dict(ks=None), dict(vs=None), dict(ids=None)):
        assert read(lib, **bad) == 1, bad


def attend(lib, o=X, q=X, kc=X, vc=X, ks=X, vs=X, bt=X, mb=1, sl=X, B=2, Hq=4, Hkv=2, D=64, BS=16, NB=4, dt=1, ct=2,
           ws=X, wb=1 << 40):
    return lib.pkv_paged_decode_attention_q8(o, q, kc, vc, ks, vs, bt, mb, sl, B, Hq, Hkv, D, BS, NB, 0.0, dt, ct, ws,
                                             wb, None, None)


def test_attention_refusals(lib):
    assert attend(lib, B=0) == 0
    for bad in (dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3), dict(D=0), dict(D=257), dict(BS=0), dict(NB=0),
                dict(mb=0), dict(dt=2), dict(ct=0), dict(ct=1), dict(o=None), dict(q=None), dict(kc=None),
                dict(vc=None), dict(ks=None), dict(vs=None), dict(bt=None), dict(sl=None), dict(ws=None),
                dict(ws=P(8))):
        assert attend(lib, **bad) == 1, bad


def prepare(lib, qo=X, q=X, qst=256, k=X, kst=128, v=X, vst=128, qw=X, kw=X, eps=1e-6, fr=X, rot=64, kc=X, vc=X, ks=X,
            vs=X, bt=X, mb=1, sl=X, qs=None, B=2, T=2, Hq=4, Hkv=2, D=64, BS=16, NB=4, dt=1, ct=2):
    return lib.pkv_qk_norm_rope_append(qo, q, qst, k, kst, v, vst, qw, kw, eps, fr, rot, 0, kc, vc, ks, vs, bt, mb, sl,
                                       qs, B, T, Hq, Hkv, D, BS, NB, dt, ct, None, None)


def test_prepare_refusals(lib):
    assert prepare(lib, B=0, T=0) == 0
    for bad in (dict(B=-1), dict(T=3), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(D=257), dict(BS=0), dict(NB=0),
                dict(mb=0), dict(dt=2), dict(ct=0), dict(ct=7), dict(rot=63), dict(rot=66), dict(rot=-2),
                dict(fr=None), dict(eps=-1.0), dict(eps=math.nan), dict(qst=255), dict(kst=127), dict(vst=127),
                dict(ks=None), dict(vs=None), dict(qo=None), dict(q=None), dict(k=None), dict(v=None), dict(kc=None),
                dict(vc=None), dict(bt=None), dict(sl=None)):
        assert prepare(lib, **bad) == 1, bad


def test_other_calls_refuse_the_8_bit_types(lib):
    for code in (2, 3):
        assert lib.pkv_kv_append(X, X, X, X, X, 1, X, 2, 2, 64, 16, 4, code, None, None) == 1
        assert lib.pkv_kv_append_chunk(X, X, X, X, X, 1, X, X, 2, 4, 2, 64, 16, 4, code, None, None) == 1
        assert lib.pkv_paged_decode_attention(X, X, X, X, X, 1, X, 2, 4, 2, 64, 16, 4, 0.0, code, X, 1 << 40, None,
                                              None) == 1
        assert lib.pkv_copy_blocks(X, X, X, X, 0, 2, 64, 16, 4, code, None, None) == 0
    assert lib.pkv_copy_blocks(X, X, X, X, 0, 2, 64, 16, 4, 4, None, None) == 1


def test_workspace_is_host_arithmetic(lib):
    import paged_kv_decode_table_gb300 as pkv
    for args in ((64, 32, 8, 128), (1, 8, 1, 64), (3, 7, 7, 100), (512, 192, 12, 80), (0, 8, 8, 128)):
        n = pkv.decode_q8_workspace_bytes(*args, num_sms=152)
        assert n > 0 and n % 256 == 0
    for args in ((-1, 8, 8, 128), (2, 0, 1, 128), (2, 8, 3, 128), (2, 8, 8, 0)):
        assert pkv.decode_q8_workspace_bytes(*args, num_sms=152) == 0


def test_python_refuses_host_tensors_and_wrong_types():
    import paged_kv_decode_table_gb300 as pkv
    k = torch.zeros(2, 1, 16, 64, dtype=torch.int8)
    s = torch.zeros(2, 1, 16)
    bt, sl = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    row = torch.zeros(1, 1, 64)
    with pytest.raises(ValueError):
        pkv.kv_append_q8(row, row, k, k, s, s, bt, sl)
    with pytest.raises(TypeError):
        pkv.kv_append_q8(row, row, k.float(), k.float(), s, s, bt, sl)
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_q8(row, k, k, s, s, bt, sl)
    with pytest.raises(ValueError):
        pkv.kv_read_blocks_q8(k, k, s, s, sl)
    with pytest.raises(ValueError):
        pkv.qk_norm_rope_append(row, row, row, None, None, 1e-6, None, k.float(), k.float(), bt, sl)
    with pytest.raises(TypeError):
        pkv.kv_append_chunk_q8(row, row, k, k, s, s, bt, sl, None)


def test_rope_freqs():
    import paged_kv_decode_table_gb300 as pkv
    f = pkv.rope_freqs(8, 10000.0, device="cpu").numpy().view(np.uint64)
    want = [10000.0 ** (-2 * j / 8) / (2 * math.pi) for j in range(4)]
    np.testing.assert_allclose(f.astype(np.float64) / 2.0 ** 64, want, rtol=2 ** -50)
    # angles per position of half a turn and more come out modulo a turn
    g = pkv.rope_freqs(6, inv_freq=[math.pi, 1.5 * math.pi, 2.5 * math.pi], device="cpu").numpy().view(np.uint64)
    np.testing.assert_allclose(g.astype(np.float64) / 2.0 ** 64, [0.5, 0.75, 0.25], rtol=2 ** -50)
    assert pkv.rope_freqs(0, device="cpu").numel() == 0
    for bad in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=4, inv_freq=[1.0])):
        with pytest.raises(ValueError):
            pkv.rope_freqs(**bad, device="cpu")


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_the_plain_store_keeps_its_own_bound(fmt):
    """The format's documented error: half a step of its scale, as the GPU tests assume."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(400, 80, generator=g) * torch.exp(2 * torch.randn(400, 1, generator=g))
    x[0] = 0
    vals, scale = R.store(x, fmt)
    off = (R.numbers(vals, scale) - x.double()).abs()
    # the float32 product x * (1 / scale) is off by 1.5 half-steps of float32, relative to x
    assert bool((off <= R.half_step(x.double(), scale.double(), fmt) + 2 * R.U24 * x.double().abs().amax(-1, keepdim=True)).all())
    assert bool(R.numbers(vals, scale)[0].eq(0).all()) and bool(R.numbers(vals, scale).isfinite().all())
    assert float(scale[0]) == 2.0 ** -64


def test_plain_attention_against_a_worked_row():
    """Two positions with scores 0 and ln 3: weights 1/4 and 3/4."""
    k = torch.zeros(1, 1, 16, 2, dtype=torch.int8)
    k[0, 0, 1, 0] = 1
    v = torch.zeros(1, 1, 16, 2, dtype=torch.int8)
    v[0, 0, 0], v[0, 0, 1] = torch.tensor([4, 8]), torch.tensor([-4, 16])
    ks = torch.full((1, 1, 16), math.log(3.0))
    vs = torch.full((1, 1, 16), 0.5)
    out, _ = R.attention(torch.tensor([[[1.0, 5.0]]]), k, v, ks, vs, torch.zeros(1, 1, dtype=torch.int32), [2], scale=1.0)
    np.testing.assert_allclose(out[0, 0].numpy(), [0.25 * 2 - 0.75 * 2, 0.25 * 4 + 0.75 * 8], rtol=1e-6)


def test_plain_rotation_keeps_pair_lengths_and_wraps():
    x = torch.randn(3, 2, 8, generator=torch.Generator().manual_seed(2))
    y, _ = R.norm_rope(x, None, 0.0, [0, 7, 123456], [1.0, 0.01], True)
    assert torch.equal(y[0], x[0].double()) and torch.equal(y[..., 4:], x[..., 4:].double())
    np.testing.assert_allclose((y[..., :4] ** 2).reshape(3, 2, 2, 2).sum(-1).numpy(),
                               (x[..., :4].double() ** 2).reshape(3, 2, 2, 2).sum(-1).numpy(), rtol=1e-12)
    z, _ = R.norm_rope(x, None, 0.0, [4, 4, 4], [math.pi / 2], False)  # four quarter turns
    np.testing.assert_allclose(z.numpy(), x.double().numpy(), atol=1e-12)
