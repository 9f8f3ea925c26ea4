"""Decode attention over shared prefixes against float64 formulas, and in a step with the other calls."""
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


def _cu(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def make(seed, groups, Hq, Hkv, D, BS, dtype, q_size=1.5, loose=(), wide=True):
    """groups: (shared tokens, lengths) of each; loose: lengths of sequences behind the last group; wide: a table so
    wide that the call does not take the batch for a small one, whose prefixes it reads per sequence."""
    lens = [L for _, ls in groups for L in ls] + list(loose)
    x = R.make(seed, lens, Hq, Hkv, D, BS, dtype, q_size=q_size)
    start, at = [0], 0
    for shared, ls in groups:
        whole = shared // BS
        for b in range(at + 1, at + len(ls)):
            if ls[b - at] >= whole * BS:
                x["block_tables"][b, :whole] = x["block_tables"][at, :whole]
        at += len(ls)
        start.append(at)
    x["group_start"], x["shared_lens"] = _cu(start), _cu([s for s, _ in groups])
    if wide:
        B, width = x["block_tables"].shape
        more = max(0, (48 << 20) // (4 * B * BS * Hkv * D) + 1 - width)
        x["block_tables"] = torch.cat([x["block_tables"], torch.full((B, more), -1, dtype=torch.int32, device="cuda")], 1)
    return x


def call(x, **kw):
    return pkv.paged_decode_attention_shared(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"],
                                             x["group_start"], x["shared_lens"], **kw)


GROUPS = [
    [(64, [64, 65, 100, 80])],
    [(160, [170, 300, 160]), (0, [40]), (33, [50, 33, 900]), (48, [48])],
    [(1000, [1000 + i for i in range(40)])],
    [(2048, [2050, 2049]), (2048, [2048, 2100]), (16, [16, 17])],
    [(0, [5, 0, 70])],
    [(15, [15, 16])],
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("groups", range(len(GROUPS)))
@pytest.mark.parametrize("dtype,Hq,Hkv,D,BS", [
    (BF, 32, 8, 128, 16), (BF, 8, 2, 64, 16), (BF, 21, 3, 128, 32), (BF, 12, 12, 64, 48), (BF, 32, 2, 128, 64),
    (BF, 40, 1, 64, 16), (BF, 1, 1, 128, 16), (BF, 120, 1, 128, 16), (BF, 200, 2, 64, 16)])
def test_groups(dtype, Hq, Hkv, D, BS, groups, wide):
    x = make(groups, GROUPS[groups], Hq, Hkv, D, BS, dtype, loose=(20, 0), wide=wide)
    st = pkv.new_status()
    got = call(x, status=st)
    ref, tol = R.reference(x)
    assert pkv.check_status(st) == 0
    R.check(got, ref, tol)


@pytest.mark.parametrize("D,softcap,slopes", [(128, 9.0, False), (128, 0.0, True), (64, 20.0, True)])
def test_scores(D, softcap, slopes):
    x = make(3, [(700, [700 + 3 * i for i in range(20)]), (96, [100, 200])], 24, 4, D, 16, BF, q_size=4.0)
    sl = R.slopes(24) if slopes else None
    got = call(x, softcap=softcap, slopes=sl)
    R.check(got, *R.reference(x, softcap=softcap, slopes=sl))


@pytest.mark.parametrize("D,softcap,slopes", [(128, 0.0, False), (128, 12.0, True), (64, 0.0, True)])
def test_much_behind_the_prefix(D, softcap, slopes):
    """Prefixes and the sequences' own positions both large: the two kernels share the SMs out."""
    x = make(19, [(2048, [2348 + 43 * i for i in range(24)]), (700, [1500, 700, 0, 2900])], 16, 4, D, 16, BF, loose=(1200, 5))
    sl = R.slopes(16) if slopes else None
    want = call(x, softcap=softcap, slopes=sl)
    R.check(want, *R.reference(x, softcap=softcap, slopes=sl))
    for _ in range(20):
        assert torch.equal(call(x, softcap=softcap, slopes=sl), want)


def test_long_prefix_many_rows():
    x = make(5, [(12000, [12000 + 7 * i for i in range(48)])], 32, 4, 128, 16, BF)
    R.check(call(x), *R.reference(x))


def test_many_groups():
    x = make(6, [(48, [48 + i % 9, 60, 49 + i]) for i in range(90)], 8, 4, 128, 16, BF)
    R.check(call(x), *R.reference(x))


def test_more_groups_and_sequences_than_threads():
    x = make(16, [(32, [33 + i % 5, 40, 32][:2 + i % 2]) for i in range(600)], 8, 4, 64, 16, BF, loose=(9,))
    st = pkv.new_status()
    got = call(x, status=st)
    assert pkv.check_status(st) == 0
    R.check(got, *R.reference(x))


def test_bad_blocks_in_many_short_prefixes():
    """Several prefixes per CTA, every third of which holds a block that is none: its members are zeros, and no others."""
    n = 900
    x = make(17, [(64, [64 + i % 40, 80]) for i in range(n)], 8, 8, 128, 16, BF)
    ref, tol = R.reference(x)
    bad = [g for g in range(n) if g % 3 == 1]
    for g in bad:
        x["block_tables"][2 * g:2 * g + 2, g % 4] = -1
    st = pkv.new_status()
    got = call(x, status=st)
    assert pkv.check_status(st) == 4
    rows = [2 * g + i for g in bad for i in range(2)]
    assert (got[rows] == 0).all()
    R.check(got, ref, tol, [b for b in range(2 * n) if b // 2 % 3 != 1])


@pytest.mark.parametrize("wide", [True, False])
def test_the_same_sequence_twice(wide):
    """A sequence that is in the batch twice shares all its whole blocks with itself."""
    x = make(18, [(96, [96, 96, 96]), (80, [90, 90])], 8, 2, 128, 16, BF, wide=wide)
    for b, a in ((1, 0), (2, 0), (4, 3)):
        x["block_tables"][b] = x["block_tables"][a]
    x["q"][1] = x["q"][0]
    got = call(x, softcap=8.0)
    R.check(got, *R.reference(x, softcap=8.0))


def test_threads():
    """Calls of different sizes from several threads at once, each on a stream of its own."""
    import threading
    xs = [make(40 + i, [(320 * (i + 1), [700 + i] * (4 + 30 * i)), (48, [50, 60])], 16, 4, (128, 64)[i % 2], 16, BF, wide=i != 2)
          for i in range(4)]
    xs += [make(44 + i, [(320 * i, [1000 - i] * (3 + 40 * i))], 16, 4, 128, 16, BF) for i in (1, 2)]
    want = [call(x) for x in xs]
    for x, w in zip(xs, want):
        # the large prefixes of 960 and 1280 are longer than their sequences of 702 and 703, which are zeros
        short = x["seq_lens"] < x["shared_lens"][torch.bucketize(torch.arange(len(w), device="cuda"), x["group_start"][1:], right=True)]
        assert (w[short] == 0).all()
        R.check(w, *R.reference(x), ~short)
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = [call(xs[i]) for _ in range(30)]
        s.synchronize()
        wrong.extend(i for o in got if not torch.equal(o, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_no_groups():
    x = make(7, [], 8, 2, 128, 16, BF, loose=(100, 3000, 1))
    R.check(call(x), *R.reference(x))


@pytest.mark.parametrize("wide", [True, False])
def test_bad_members_tables_and_groups(wide):
    groups = [(64, [64, 30, 100, 0]), (32, [60, 60])]
    x = make(8, groups, 8, 2, 128, 16, BF, wide=wide)
    ref, tol = R.reference(x)
    st = pkv.new_status()
    got = call(x, status=st)  # sequence 1 is shorter than its group's prefix; the empty one is no error
    assert pkv.check_status(st) == 4
    assert (got[1] == 0).all() and (got[3] == 0).all()
    R.check(got, ref, tol, [0, 2, 3, 4, 5])
    x["seq_lens"][1] = 0
    # a block of a prefix (in the tables of all its members), of one sequence
    for members, entry, bad in (([0, 1, 2, 3], 1, [0, 2]), ([2], 5, [2]), ([4, 5], 0, [4, 5])):
        y = dict(x, block_tables=x["block_tables"].clone())
        y["block_tables"][members, entry] = 10 ** 6
        st = pkv.new_status()
        got = call(y, status=st)
        assert pkv.check_status(st) == 4
        assert (got[bad] == 0).all()
        R.check(got, ref, tol, [i for i in range(6) if i not in bad and i != 1])
    for start in ([0, 5, 4], [1, 4, 6], [0, 4, 7], [0, -1, 6]):
        st = pkv.new_status()
        got = call(dict(x, group_start=_cu(start)), status=st)
        assert pkv.check_status(st) == 4, start
        assert (got == 0).all(), start
    for shared in ([-16, 32], [64, 2 ** 31 - 1]):
        st = pkv.new_status()
        got = call(dict(x, shared_lens=_cu(shared)), status=st)
        assert pkv.check_status(st) == 4
        good, bad = ([4, 5], [0, 2]) if shared[0] < 0 else ([0, 2], [4, 5])
        assert (got[bad] == 0).all()
        R.check(got, ref, tol, good)


def test_streams_and_graphs():
    xs = [make(30 + i, [(1600, [1600 + 50 * j for j in range(9)]), (320, [400, 500 + i])], 32, 8, 128, 16, BF)
          for i in range(2)]
    want = [call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(call(x))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for x in xs:
        x["q"].copy_(-x["q"])
    want = [call(x) for x in xs]
    for x, w in zip(xs, want):
        R.check(w, *R.reference(x))
    for g in (graphs[0], graphs[1], graphs[0], graphs[0]):
        g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_prompt_forks_and_decodes():
    """A prompt prefilled in two chunks with changed scores, forked, and decoded step by step behind its shared blocks."""
    Hq, Hkv, D, BS, cap = 16, 4, 128, 16, 12.0
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF)
    pool = pkv.BlockPool(64, BS, 16)
    k, v = (torch.full((64, Hkv, BS, D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    pool.add(0, 150)
    keys, values = rand(150, Hkv, D), rand(150, Hkv, D)
    for lo, hi in ((0, 100), (100, 150)):
        bt, _ = pool.tables([0])
        bt, sl, qs = bt.cuda(), _cu([hi]), _cu([0, hi - lo])
        pkv.kv_append_chunk(keys[lo:hi].contiguous(), values[lo:hi].contiguous(), k, v, bt, sl, qs)
        x = dict(q=rand(hi - lo, Hq, D), k_cache=k, v_cache=v, block_tables=bt, seq_lens=sl, q_start=qs, lens=[hi],
                 start=[0, hi - lo], BS=BS)
        got = pkv.paged_prefill_attention_scored(x["q"], k, v, bt, sl, qs, softcap=cap, window=60)
        R.check(got, *R.reference(x, softcap=cap, window=60))
    for child in (1, 2):
        pool.fork(0, child)
    seqs = [0, 1, 2]
    for step in range(12):
        pairs = [p for p in (pool.append(s) for s in seqs) if p]
        if pairs:
            pkv.copy_blocks(k, v, _cu([a for a, _ in pairs]), _cu([b for _, b in pairs]))
        bt, sl = pool.tables(seqs)
        start, shared = pool.shared_groups(seqs)
        assert start.tolist() == [0, 3] and shared.tolist() == [144]
        bt, sl = bt.cuda(), sl.cuda()
        pkv.kv_append(rand(3, Hkv, D), rand(3, Hkv, D), k, v, bt, sl)
        x = dict(q=rand(3, Hq, D), k_cache=k, v_cache=v, block_tables=bt, seq_lens=sl, lens=sl.tolist(),
                 start=[0, 1, 2, 3], BS=BS)
        got = pkv.paged_decode_attention_shared(x["q"], k, v, bt, sl, start.cuda(), shared.cuda(), softcap=cap)
        R.check(got, *R.reference(x, softcap=cap))
        got = pkv.paged_decode_attention_scored(x["q"], k, v, bt, sl, softcap=cap, window=60)
        R.check(got, *R.reference(x, softcap=cap, window=60))


def test_refusals():
    x = make(1, [(32, [40, 50])], 8, 2, 128, 16, BF)
    for kw, err in ((dict(group_start=_cu([0])), ValueError), (dict(shared_lens=_cu([[32]])), ValueError),
                    (dict(group_start=torch.tensor([0, 2], device="cuda")), TypeError),
                    (dict(group_start=None), TypeError), (dict(shared_lens=None), TypeError),
                    # more groups than sequences
                    (dict(group_start=_cu([0, 1, 2, 2]), shared_lens=_cu([0, 0, 0])), pkv.PkvError)):
        with pytest.raises(err):
            call(dict(x, **kw))
    with pytest.raises(pkv.PkvError):
        call(x, softcap=-2.0)
    for y in (make(1, [(32, [40, 50])], 8, 2, 80, 16, BF), make(1, [(32, [40, 50])], 8, 2, 128, 16, F32)):
        with pytest.raises(pkv.PkvError):
            call(y)
    with pytest.raises(pkv.PkvError):
        call(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_groups_that_begin_with_members_without_the_prefix(D, wide):
    """The prefix is read by a member that has it: rows in front of it may be padding, with anything in their tables."""
    x = make(12, [(64, [70, 64, 100]), (160, [200] * 40 + [300, 170]), (48, [50, 49])], 8, 2, D, 16, BF, wide=wide)
    empty = [0] + list(range(3, 3 + 36)) + [45, 46]
    for b in empty:
        x["lens"][b] = 0
    x["seq_lens"] = _cu(x["lens"])
    ref, tol = R.reference(x)
    for junk in (-1, 10 ** 6, int(x["block_tables"][1, 0])):
        y = dict(x, block_tables=x["block_tables"].clone())
        y["block_tables"][empty] = junk
        st = pkv.new_status()
        got = call(y, status=st)
        assert pkv.check_status(st) == 0
        assert (got[empty] == 0).all()
        R.check(got, ref, tol)
    # members that are refused: one shorter than the prefix, one with a length outside the table
    y = dict(x, block_tables=x["block_tables"].clone(), seq_lens=x["seq_lens"].clone())
    y["block_tables"][empty] = 10 ** 6
    y["seq_lens"][0], y["seq_lens"][3] = 30, 2 ** 31 - 1
    st = pkv.new_status()
    got = call(y, status=st)
    assert pkv.check_status(st) == 4
    assert (got[empty] == 0).all()
    R.check(got, ref, tol)
