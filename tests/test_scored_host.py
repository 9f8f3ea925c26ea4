"""Attention with changed scores and over shared prefixes without a GPU: refusals that return before a launch,
workspace sizing, and the grouping of sequences that share blocks."""
import ctypes

import pytest

P = ctypes.c_void_p
X = P(64)  # never dereferenced: every call below returns before a launch


@pytest.fixture(scope="module")
def lib():
    from paged_kv_decode_table_gb300 import build as B
    B.build()
    import paged_kv_decode_table_gb300 as pkv
    return pkv.load_library()


def decode(lib, o=X, q=X, k=X, v=X, bt=X, mb=4, sl=X, pre=None, B=2, Hq=4, Hkv=2, D=64, BS=16, NB=4, scale=0.0, cap=0.0,
           slopes=None, window=0, dt=1, ws=X, wb=1 << 40):
    return lib.pkv_paged_decode_attention_scored(o, q, k, v, bt, mb, sl, pre, B, Hq, Hkv, D, BS, NB, scale, cap, slopes,
                                                 window, dt, ws, wb, None, None)


def shared(lib, o=X, q=X, k=X, v=X, bt=X, mb=4, sl=X, gs=X, sh=X, N=1, B=2, Hq=4, Hkv=2, D=64, BS=16, NB=4, scale=0.0,
           cap=0.0, slopes=None, dt=1, ws=X, wb=1 << 40):
    return lib.pkv_paged_decode_attention_shared(o, q, k, v, bt, mb, sl, gs, sh, N, B, Hq, Hkv, D, BS, NB, scale, cap,
                                                 slopes, dt, ws, wb, None, None)


def prefill(lib, o=X, q=X, k=X, v=X, bt=X, mb=4, sl=X, qs=X, pre=None, B=2, T=4, Hq=4, Hkv=2, D=128, BS=16, NB=4,
            scale=0.0, cap=0.0, slopes=None, window=0, dt=1, ws=X, wb=1 << 40):
    return lib.pkv_paged_prefill_attention_scored(o, q, k, v, bt, mb, sl, qs, pre, B, T, Hq, Hkv, D, BS, NB, scale, cap,
                                                  slopes, window, dt, ws, wb, None, None)


SHAPES = [dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(BS=0), dict(NB=0), dict(mb=0), dict(dt=2),
          dict(dt=3), dict(dt=9)]
NUMBERS = [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-40), dict(cap=3e38),
           dict(cap=1e-30, scale=1e20), dict(scale=float("inf")), dict(scale=3e38)]
POINTERS = [dict(o=None), dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(sl=None)]


def test_decode_refusals(lib):
    assert decode(lib, B=0) == 0
    for bad in SHAPES + NUMBERS + POINTERS + [dict(D=257), dict(ws=None), dict(ws=P(72)), dict(wb=0)]:
        assert decode(lib, **bad) == 1, bad


def test_prefill_refusals(lib):
    assert prefill(lib, B=0) == 0 and prefill(lib, T=0) == 0
    for bad in SHAPES + NUMBERS + POINTERS + [dict(T=-1), dict(qs=None)]:
        assert prefill(lib, **bad) == 1, bad
    for bad in (dict(dt=0), dict(D=64), dict(BS=24), dict(Hq=18), dict(q=P(72)), dict(o=P(72)), dict(k=P(72)), dict(v=P(72))):
        assert prefill(lib, **bad) == 2, bad


def test_shared_refusals(lib):
    assert shared(lib, B=0, N=0) == 0
    for bad in SHAPES + NUMBERS + POINTERS + [dict(D=257), dict(ws=None), dict(ws=P(72)), dict(gs=None), dict(sh=None),
                                              dict(N=-1), dict(N=3)]:
        assert shared(lib, **bad) == 1, bad
    for bad in (dict(dt=0), dict(D=80), dict(D=256), dict(BS=24), dict(Hq=260), dict(q=P(72)), dict(k=P(72)),
                dict(NB=1 << 27), dict(mb=(1 << 31) - 1, BS=64)):
        assert shared(lib, **bad) == 2, bad


def test_out_over_q_and_too_wide_tables(lib):
    """Rows of out are written while other rows of q are read; positions are 32-bit numbers."""
    for call, rows in ((decode, 2), (shared, 2), (prefill, 4)):
        D = 128
        for away in (0, 16, -16, rows * 4 * D * 2 - 16):
            assert call(lib, D=D, q=P(1 << 20), o=P((1 << 20) + away)) == 1, (call, away)
        assert call(lib, D=D, q=P(1 << 20), mb=0x7fff, BS=1 << 16, wb=0) != 2  # (refused for its workspace)
        assert call(lib, D=D, q=P(1 << 20), mb=(0x7fff << 12) + 1, BS=16) == 2
    assert decode(lib, dt=0, q=P(1 << 20), o=P((1 << 20) + 2 * 4 * 64 * 4 - 16)) == 1


def test_workspaces_are_host_arithmetic(lib):
    import paged_kv_decode_table_gb300 as pkv
    for f in (pkv.decode_scored_workspace_bytes, pkv.decode_shared_workspace_bytes):
        a, b = f(64, 32, 8, 128, num_sms=152), f(64, 32, 8, 128, num_sms=76)
        assert a > b > 0 and a % 256 == 0
        # two partial results per SM of (max, sum) and 128 floats for 32 rows
        assert a >= 2 * 152 * 32 * 130 * 4
        assert f(64, 32, 5, 128, num_sms=152) == 0 and f(-1, 32, 8, 128, num_sms=152) == 0
        assert f(0, 32, 8, 128, num_sms=152) > 0 and f(3, 6, 2, 33, num_sms=152) > 0
    f = pkv.prefill_scored_workspace_bytes
    assert f(16, 8192, 32, 8, 128, num_sms=152) == 0  # 1152 pairs of query tiles
    assert f(1, 64, 32, 8, 128, num_sms=152) >= 64 * 32 * 9 * 130 * 4  # 16 of them: 9 shares
    assert f(1, 64, 33, 8, 128, num_sms=152) == 0 and f(1, 64, 32, 8, 64, num_sms=152) == 0
    # and 256 rows of one KV head per SM, twice, behind them
    assert pkv.decode_shared_workspace_bytes(64, 32, 8, 128, num_sms=152) >= 2 * 152 * (32 + 256) * 130 * 4


def test_shared_groups(lib):
    import paged_kv_decode_table_gb300 as pkv
    pool = pkv.BlockPool(200, 4, 40)
    pool.add(0, 23)  # 5 whole blocks and 3 tokens
    for c in (1, 2):
        pool.fork(0, c)
    pool.add(3, 9)
    pool.add(4, 40)
    pool.fork(4, 5)
    groups = lambda *a, **k: tuple(t.tolist() for t in pool.shared_groups(*a, **k))
    assert groups([]) == ([0], [])
    assert groups([0]) == ([0, 1], [0])
    # the tail block is shared until one of them writes, but it is not whole
    assert groups([0, 1, 2]) == ([0, 3], [20])
    assert groups([0, 1, 3, 2]) == ([0, 2, 3, 4], [20, 0, 0])
    assert groups([3, 0, 2, 4, 5]) == ([0, 1, 3, 5], [0, 20, 40])
    assert groups([0, 1, 2], min_blocks=5) == ([0, 3], [20])
    assert groups([0, 1, 2], min_blocks=6) == ([0, 1, 2, 3], [0, 0, 0])
    # one more token fills 0's copy of the tail; the others' tail block is another
    assert pool.append(0) is not None
    assert groups([0, 1, 2]) == ([0, 3], [20])
    with pytest.raises(pkv.PkvError):
        groups([0, 77])
    with pytest.raises(pkv.PkvError):
        groups([0], min_blocks=0)


def test_shared_groups_keeps_long_prefixes(lib):
    """A neighbour that shares little starts a group of its own where joining would cost the run its prefix."""
    import paged_kv_decode_table_gb300 as pkv
    pool = pkv.BlockPool(400, 4, 100)
    pool.add(0, 4)                       # a system prompt of one block
    for s, n in ((1, 160), (4, 160)):    # two long conversations behind it
        pool.fork(0, s)
        for _ in range(n):
            pool.append(s)
    pool.fork(1, 2)
    pool.fork(1, 3)
    pool.fork(4, 5)
    start, shared_lens = (t.tolist() for t in pool.shared_groups([1, 2, 3, 4, 5]))
    assert start == [0, 3, 5] and shared_lens == [164, 164]
    # short ones behind it share it all
    pool.fork(0, 6)
    pool.fork(0, 7)
    pool.append(6)
    start, shared_lens = (t.tolist() for t in pool.shared_groups([0, 6, 7]))
    assert start == [0, 3] and shared_lens == [4]


def test_cap_and_scale_in_the_range_of_normal_numbers(lib):
    """scale / cap in float32 is what products are multiplied by: subnormal it loses digits, and 0 makes all scores equal."""
    for call in (decode, shared, prefill):
        more = dict(N=0) if call is shared else {}
        for bad in (dict(cap=1e38, scale=1e-8), dict(cap=1e35, scale=1e-6), dict(cap=2e38)):  # (the default scale is below 1)
            assert call(lib, B=0, **more, **bad) == 1, bad
        for good in (dict(cap=1e30), dict(cap=1e30, scale=1e-7), dict(cap=2e38, scale=3.0), dict(scale=1e-40)):
            assert call(lib, B=0, **more, **good) == 0, good
