"""Decode and chunked-prefill attention with capped, biased and windowed scores against float64 formulas.

Every slot that no query may see (past the ends, outside windows, blocks of no table) holds NaN.
"""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
import scored_ref as R

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()
    pkv.load_library()


def _prefix(kind, lens, seed=5):
    if kind is None:
        return None
    g = torch.Generator().manual_seed(seed)
    # negative, zero, past the end and in between
    p = [(-3, 0, L + 9, int(torch.randint(0, kind + 1, (1,), generator=g)))[i % 4] for i, L in enumerate(lens)]
    return torch.tensor(p, dtype=torch.int32, device="cuda")


def _decode(x, status=None, **kw):
    return pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                             status=status, **kw)


RAGGED = [1, 0, 15, 16, 17, 33, 64, 100, 257, 31, 0, 5]
MASKS = [dict(), dict(softcap=8.0), dict(slopes=True), dict(window=1), dict(window=20, prefix=4),
         dict(softcap=30.0, slopes=True, window=50, prefix=40), dict(window=16), dict(window=48, prefix=16)]


@pytest.mark.parametrize("mask", range(len(MASKS)))
@pytest.mark.parametrize("dtype,Hq,Hkv,D,BS", [
    (BF, 8, 2, 64, 16), (BF, 32, 8, 128, 16), (BF, 21, 3, 128, 32), (BF, 12, 12, 80, 48), (BF, 32, 2, 128, 16),
    (BF, 40, 1, 96, 16), (BF, 6, 3, 20, 8), (F32, 21, 3, 80, 32), (F32, 2, 2, 4, 4), (F32, 4, 1, 256, 16),
    (BF, 4, 2, 200, 16), (F32, 9, 9, 33, 5)])
def test_decode_ragged(dtype, Hq, Hkv, D, BS, mask):
    m = dict(MASKS[mask])
    x = R.make(mask + D, RAGGED, Hq, Hkv, D, BS, dtype, q_size=5.0 if "softcap" in m else 1.5)
    sl = R.slopes(Hq) if m.pop("slopes", False) else None
    pre = _prefix(m.pop("prefix", None), RAGGED)
    R.hide(x, m.get("window", 0), pre)
    st = pkv.new_status()
    got = _decode(x, st, slopes=sl, prefix_lens=pre, **m)
    ref, tol = R.reference(x, slopes=sl, prefix=pre, **m)
    assert pkv.check_status(st) == 0
    R.check(got, ref, tol)
    assert (got[1] == 0).all() and (got[10] == 0).all()


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,BS,lens", [
    (BF, 1, 64, 8, 128, 16, [20000]), (BF, 3, 32, 8, 128, 16, [9000, 1, 4097]), (BF, 2, 16, 16, 64, 32, [7000, 3000]),
    (F32, 1, 8, 2, 80, 16, [5000]), (BF, 1, 4, 1, 128, 16, [16]), (BF, 2, 36, 3, 112, 64, [3001, 2999])])
@pytest.mark.parametrize("window", [0, 3000])
def test_decode_long(dtype, B, Hq, Hkv, D, BS, lens, window):
    x = R.make(B + Hq, lens, Hq, Hkv, D, BS, dtype)
    sl = R.slopes(Hq, 3)
    pre = torch.tensor([70] * B, dtype=torch.int32, device="cuda")
    R.hide(x, window, pre)
    got = _decode(x, slopes=sl, prefix_lens=pre, window=window, softcap=20.0)
    R.check(got, *R.reference(x, slopes=sl, prefix=pre, window=window, softcap=20.0))


def test_decode_many_short():
    lens = [(7 * i) % 61 for i in range(700)]
    x = R.make(11, lens, 8, 4, 64, 16, BF)
    got = _decode(x, window=30, softcap=10.0)
    R.check(got, *R.reference(x, window=30, softcap=10.0))


@pytest.mark.parametrize("D", [8, 16, 24, 56, 72, 88, 120])
def test_decode_head_sizes(D):
    lens = [300, 7, 0, 64]
    x = R.make(D, lens, 12, 3, D, 16, BF)
    sl = R.slopes(12)
    R.check(_decode(x, slopes=sl, window=100), *R.reference(x, slopes=sl, window=100))


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64), (BF, 64)])
def test_decode_bad_block_in_a_split_sequence(dtype, D):
    lens = [9000, 5000, 20, 7000]
    x = R.make(13, lens, 8, 2, D, 16, dtype)
    ref, tol = R.reference(x)
    x["block_tables"][1, 150] = -1
    x["block_tables"][3, 0] = 1 << 30
    st = pkv.new_status()
    got = _decode(x, st)
    assert pkv.check_status(st) == 4
    assert (got[1] == 0).all() and (got[3] == 0).all()
    R.check(got, ref, tol, [0, 2])


@pytest.mark.parametrize("name", ["q", "k_cache", "v_cache", "out"])
def test_decode_addresses_off_16_bytes(name):
    x = R.make(14, [200, 33], 8, 2, 128, 16, BF)
    ref, tol = R.reference(x, softcap=9.0)
    def off(t):
        y = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return y.copy_(t)
    kw = {}
    if name == "out":
        kw["out"] = off(torch.empty_like(x["q"]))
    else:
        x[name] = off(x[name])
    R.check(_decode(x, softcap=9.0, **kw), ref, tol)


def test_without_changes_is_plain_attention():
    x = R.make(2, [300, 17, 900], 32, 8, 128, 16, BF)
    plain = pkv.paged_decode_attention(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"])
    ref, tol = R.reference(x)
    R.check(plain, ref, tol)
    R.check(_decode(x), ref, tol)


def test_scale_and_huge_cap():
    # a cap far above every score changes them by less than the tolerance, which holds t^3 / (3 cap^2)
    x = R.make(4, [200, 50], 8, 2, 128, 16, BF)
    ref, tol = R.reference(x, scale=0.3)
    R.check(_decode(x, scale=0.3), ref, tol)
    R.check(_decode(x, scale=0.3, softcap=3.0e5), ref, tol * 1.01)


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 80), (BF, 72)])
def test_decode_bad_tables_and_lengths(dtype, D):
    lens = [40, 40, 40, 40]
    x = R.make(7, lens, 4, 2, D, 16, dtype)
    ref, tol = R.reference(x, window=20)
    for b, value, code in ((1, -5, 4), (2, 10 ** 6, 4)):
        st = pkv.new_status()
        bt = x["block_tables"].clone()
        bt[b, 1] = value
        got = pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"], window=20, status=st)
        assert pkv.check_status(st) == code
        assert (got[b] == 0).all()
        R.check(got, ref, tol, [i for i in range(4) if i != b])
    for value in (-1, 49):
        st = pkv.new_status()
        sl = x["seq_lens"].clone()
        sl[3] = value
        got = pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], sl, window=20, status=st)
        assert pkv.check_status(st) == 4
        assert (got[3] == 0).all()
        R.check(got, ref, tol, [0, 1, 2])
    # a bad id outside the window is never read
    bt = x["block_tables"].clone()
    bt[:, 0] = -7
    st = pkv.new_status()
    got = pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], bt, x["seq_lens"], window=20, status=st)
    assert pkv.check_status(st) == 0
    R.check(got, ref, tol)


def test_decode_nonfinite_scores_stay_with_their_heads():
    x = R.make(9, [50, 50], 4, 2, 128, 16, BF)
    ref, tol = R.reference(x)
    x["q"][0, 0, 5] = float("inf")
    got = _decode(x)
    assert not torch.isfinite(got[0, 0].float()).all()
    R.check(got.view(8, 128), ref.view(8, 128), tol.view(8, 128), list(range(1, 8)))


# ------------------------------------------------------------------ prefill
def _prefill(x, status=None, **kw):
    return pkv.paged_prefill_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                              x["q_start"], status=status, **kw)


@pytest.mark.parametrize("mask", range(len(MASKS)))
@pytest.mark.parametrize("Hq,Hkv,BS,chunks,before", [
    (32, 8, 16, [70, 1, 0, 130, 33], [0, 40, 20, 75, 500]), (8, 8, 32, [300, 5], [10, 300]),
    (6, 2, 48, [1, 2, 90, 64], [0, 0, 700, 64]), (16, 2, 16, [37], [0]), (5, 1, 64, [260, 64], [190, 0])])
def test_prefill_ragged(Hq, Hkv, BS, chunks, before, mask):
    m = dict(MASKS[mask])
    lens = [a + b for a, b in zip(chunks, before)]
    x = R.make(mask + Hq, lens, Hq, Hkv, 128, BS, BF, chunks=chunks, q_size=5.0 if "softcap" in m else 1.5)
    sl = R.slopes(Hq) if m.pop("slopes", False) else None
    pre = _prefix(m.pop("prefix", None), lens)
    R.hide(x, m.get("window", 0), pre)
    st = pkv.new_status()
    got = _prefill(x, st, slopes=sl, prefix_lens=pre, **m)
    ref, tol = R.reference(x, slopes=sl, prefix=pre, **m)
    assert pkv.check_status(st) == 0
    R.check(got, ref, tol)


@pytest.mark.parametrize("Hq,Hkv,BS,chunks,before", [
    (8, 1, 16, [3], [5000]), (16, 2, 16, [40, 1, 0], [3000, 900, 100]), (4, 4, 48, [200], [100]), (5, 5, 32, [70], [9000])])
@pytest.mark.parametrize("mask", range(len(MASKS)))
def test_prefill_few_rows_over_long_ranges(Hq, Hkv, BS, chunks, before, mask):
    m = dict(MASKS[mask])
    lens = [a + b for a, b in zip(chunks, before)]
    x = R.make(mask + Hq, lens, Hq, Hkv, 128, BS, BF, chunks=chunks, q_size=5.0 if "softcap" in m else 1.5)
    sl = R.slopes(Hq) if m.pop("slopes", False) else None
    pre = _prefix(m.pop("prefix", None), lens)
    R.hide(x, m.get("window", 0), pre)
    assert pkv.prefill_scored_workspace_bytes(len(lens), sum(chunks), Hq, Hkv, 128) > 0  # the keys are split
    st = pkv.new_status()
    got = _prefill(x, st, slopes=sl, prefix_lens=pre, **m)
    assert pkv.check_status(st) == 0
    R.check(got, *R.reference(x, slopes=sl, prefix=pre, **m))


@pytest.mark.parametrize("Hq,Hkv", [(32, 4), (6, 6), (28, 4)])
@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0, window=100), dict(window=70, prefix=True), dict(softcap=5.0, slopes=True)])
@pytest.mark.parametrize("many", [1, 12])
def test_prefill_chunks_about_one_query_tile(Hq, Hkv, kw, many):
    """Chunks whose rows fit into one query tile, or just do not, over one key tile and more; `many`: with key ranges
    that are not split."""
    TQ = 128 // (Hq // Hkv)
    chunks = [1, TQ, TQ + 1, 3, TQ - 1, 2 * TQ, 2, 1, 5] * many
    lens = [n + k for n, k in zip(chunks, [0, 0, 64, 61, 62, 640, 126, 1000, 130] * many)]
    x = R.make(many, lens, Hq, Hkv, 128, 16, BF, chunks=chunks)
    kw = dict(kw)
    if kw.pop("slopes", False):
        kw["slopes"] = R.slopes(Hq)
    if kw.pop("prefix", False):
        pre = [0, 9, 3, 64, 200, 100, 1, 5, 0] * many
        got = _prefill(x, prefix_lens=torch.tensor(pre, dtype=torch.int32, device="cuda"), **kw)
        R.check(got, *R.reference(x, prefix=pre, **kw))
    else:
        R.check(_prefill(x, **kw), *R.reference(x, **kw))


def test_prefill_prefix_seen_by_all_rows():
    # the whole chunk attends in both directions, in tiles behind the first one too
    x = R.make(3, [600], 8, 1, 128, 16, BF, chunks=[600])
    pre = torch.tensor([600], dtype=torch.int32, device="cuda")
    R.check(_prefill(x, prefix_lens=pre), *R.reference(x, prefix=pre))
    R.check(_prefill(x, prefix_lens=pre, window=7), *R.reference(x, prefix=pre, window=7))


def test_prefill_bad_tables_and_rows_behind_the_last():
    chunks, lens = [40, 40, 40], [100, 100, 100]
    x = R.make(5, lens, 8, 2, 128, 16, BF, chunks=chunks)
    ref, tol = R.reference(x, window=30)
    bt = x["block_tables"].clone()
    bt[1, 5] = 10 ** 7
    bt[0, 0] = -4  # outside every window
    sl = x["seq_lens"].clone()
    sl[2] = 39
    st = pkv.new_status()
    out = torch.full((125, 8, 128), 7.0, dtype=BF, device="cuda")
    q = torch.cat([x["q"], x["q"][:5]])
    got = pkv.paged_prefill_attention_scored(q, x["k_cache"], x["v_cache"], bt, sl, x["q_start"], window=30, status=st,
                                             out=out)
    assert pkv.check_status(st) == 4 and got.data_ptr() == out.data_ptr()
    R.check(got[:120], ref, tol, list(range(40)))
    assert (got[80:120] == 0).all() and (got[120:] == 7).all()


@pytest.mark.parametrize("before", [0, 10, 40])
def test_plain_prefill_reads_no_other_block(before):
    """Tiles end behind the last position that their CTA needs; block 0, which no sequence holds, is NaN."""
    x = R.make(8, [before + 300], 32, 8, 128, 16, BF, chunks=[300])
    for name in ("k_cache", "v_cache"):
        x[name] = torch.cat([torch.full_like(x[name][:1], float("nan")), x[name]])
    x["block_tables"] += 1
    got = pkv.paged_prefill_attention(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"], x["q_start"])
    R.check(got, *R.reference(x))


# ------------------------------------------------------------------ as a program uses them
def test_prefill_split_bad_lengths_and_rows_behind_the_last():
    chunks, lens = [10, 30, 20], [2000, 2500, 1800]
    x = R.make(15, lens, 8, 2, 128, 16, BF, chunks=chunks)
    ref, tol = R.reference(x)
    bt, sl = x["block_tables"].clone(), x["seq_lens"].clone()
    bt[1, 100] = -3
    sl[2] = 16 * bt.shape[1] + 1
    st = pkv.new_status()
    q = torch.cat([x["q"], x["q"][:7]])
    out = torch.full_like(q, 7.0)
    pkv.paged_prefill_attention_scored(q, x["k_cache"], x["v_cache"], bt, sl, x["q_start"], out=out, status=st)
    assert pkv.check_status(st) == 4
    assert pkv.prefill_scored_workspace_bytes(3, 67, 8, 2, 128) > 0
    R.check(out[:60], ref, tol, list(range(10)))
    assert (out[10:60] == 0).all() and (out[60:] == 7).all()


def test_prefill_workspace():
    x = R.make(6, [900], 8, 2, 128, 16, BF, chunks=[20])
    need = pkv.prefill_scored_workspace_bytes(1, 20, 8, 2, 128)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    ref, tol = R.reference(x, softcap=9.0)
    R.check(_prefill(x, softcap=9.0, workspace=ws), ref, tol)
    with pytest.raises(pkv.PkvError):
        _prefill(x, workspace=ws[:need - 256])


def test_streams_and_graphs():
    xs = [R.make(20 + i, [500 + 900 * i, 40, 3000], 32, 8, 128, 16, BF) for i in range(2)]
    refs = [R.reference(x, softcap=15.0, window=600) for x in xs]
    want = [_decode(x, softcap=15.0, window=600) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(_decode(x, softcap=15.0, window=600))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    for o, (ref, tol) in zip(want, refs):
        R.check(o, ref, tol)
    # captured, each graph with the workspace of its own calls; replayed on new queries, in turn
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_decode(x, softcap=15.0, window=600))
        graphs.append(g)
    for x in xs:
        x["q"].copy_(-x["q"])
    want = [_decode(x, softcap=15.0, window=600) for x in xs]
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_split_prefill_on_streams_and_in_graphs():
    xs = [R.make(40 + i, [2000 + 700 * i, 90], 16, 2, 128, 16, BF, chunks=[20, 9]) for i in range(2)]
    assert pkv.prefill_scored_workspace_bytes(2, 29, 16, 2, 128) > 0
    want = [_prefill(x, softcap=15.0) for x in xs]
    for o, x in zip(want, xs):
        R.check(o, *R.reference(x, softcap=15.0))
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(_prefill(x, softcap=15.0))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_prefill(x, softcap=15.0))
        graphs.append(g)
    for x in xs:
        x["q"].copy_(-x["q"])
    want = [_prefill(x, softcap=15.0) for x in xs]
    for g in (graphs[0], graphs[1], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_threads():
    """Calls of different sizes from several threads at once, each on a stream of its own."""
    import threading
    calls = []
    for i in range(3):
        x = R.make(50 + i, [1200 * (i + 1), 33], 8, 2, (128, 64, 72)[i], 16, BF)
        calls.append(lambda x=x: _decode(x, softcap=9.0))
        y = R.make(60 + i, [900 * (i + 1), 40], 8, 2, 128, 16, BF, chunks=[5 + i, 40])
        calls.append(lambda y=y: _prefill(y, window=200))
    z = R.make(70, [70, 900], 6, 2, 40, 16, F32)
    calls.append(lambda: _decode(z, slopes=R.slopes(6)))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [calls[i]() for _ in range(30)]
        s.synchronize()
        wrong.extend(i for o in got if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_empty_batches_and_padding():
    x = R.make(1, [70, 0], 8, 2, 128, 16, BF)
    e = torch.empty(0, 8, 128, dtype=BF, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert pkv.paged_decode_attention_scored(e, x["k_cache"], x["v_cache"], x["block_tables"][:0], none).shape == e.shape
    assert pkv.paged_decode_attention_shared(e, x["k_cache"], x["v_cache"], x["block_tables"][:0], none, none.new_zeros(1),
                                             none).shape == e.shape
    qs = torch.zeros(3, dtype=torch.int32, device="cuda")
    args = (x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"])
    assert pkv.paged_prefill_attention_scored(e, *args, qs).shape == e.shape
    st = pkv.new_status()
    for rows in (5, 700):  # rows behind the last sequence, of which none has any
        q = torch.ones(rows, 8, 128, dtype=BF, device="cuda")
        out = torch.full_like(q, 3.0)
        pkv.paged_prefill_attention_scored(q, *args, qs, out=out, status=st)
        assert (out == 3).all()
    # a padded batch: sequences of length zero, whose table rows are anything
    x = R.make(2, [300, 0, 0, 17, 0], 8, 2, 64, 16, BF)
    for b in (1, 2, 4):
        x["block_tables"][b] = -7
    got = _decode(x, st, slopes=R.slopes(8))
    R.check(got, *R.reference(x, slopes=R.slopes(8)))
    assert pkv.check_status(st) == 0 and (got[[1, 2, 4]] == 0).all()


def test_out_over_q_is_refused():
    x = R.make(1, [70, 80], 8, 2, 128, 16, BF, chunks=[1, 1])
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (lambda: _decode(x, out=x["q"]), lambda: _prefill(x, out=x["q"]),
                 lambda: pkv.paged_decode_attention_shared(*[x[n] for n in ("q", "k_cache", "v_cache", "block_tables", "seq_lens")],
                                                           none, none[:0], out=x["q"])):
        with pytest.raises(pkv.PkvError):
            call()


def test_given_out_and_workspace():
    x = R.make(1, [700, 80], 32, 8, 128, 16, BF)
    ws = torch.full((pkv.decode_scored_workspace_bytes(2, 32, 8, 128),), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x["q"], float("nan"))
    got = _decode(x, out=out, workspace=ws)
    assert got.data_ptr() == out.data_ptr()
    R.check(got, *R.reference(x))
    with pytest.raises(pkv.PkvError):
        _decode(x, workspace=ws[:16])


def test_refusals():
    x = R.make(1, [70, 80], 8, 2, 128, 16, BF)
    for kw, err in ((dict(softcap=-1.0), pkv.PkvError), (dict(softcap=float("nan")), pkv.PkvError),
                    (dict(softcap=1e-39), pkv.PkvError),  # subnormal
                    (dict(softcap="x"), TypeError), (dict(window=1.5), TypeError),
                    (dict(slopes=torch.ones(7, device="cuda")), ValueError), (dict(slopes=torch.ones(8)), ValueError),
                    (dict(slopes=torch.ones(8, device="cuda", dtype=torch.float64)), TypeError),
                    (dict(prefix_lens=torch.ones(2, device="cuda", dtype=torch.int64)), TypeError),
                    (dict(prefix_lens=torch.ones(3, device="cuda", dtype=torch.int32)), ValueError),
                    (dict(out=torch.empty(2, 8, 128, device="cuda")), TypeError),
                    (dict(status=torch.zeros(1, device="cuda")), TypeError)):
        with pytest.raises(err):
            _decode(x, **kw)
    y = R.make(1, [70], 4, 2, 64, 16, BF, chunks=[3])
    with pytest.raises(pkv.PkvError):
        _prefill(y)  # D = 64
    x["q"] = x["q"].transpose(0, 1)
    with pytest.raises(ValueError):
        _decode(x)
