"""A cap far above most scores beside a few beyond it: a small score keeps its accuracy whatever shares its tile, and keys
that do not take part change nothing."""
import pytest
import torch

import paged_kv_decode_table_gb300 as pkv
import scored_ref as R

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
CAP = 1e6
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


def small_rows(x, small, got, prefix=0):
    """The rows of `small` (bool [T, Hq]) against float64.  As in scored_ref, but a score is off by D e sum |q k| scale for its
    products' sum and by 2^-20 of itself for the cap's polynomial (2^-20.7) and all scalings (4 e)."""
    q, BS = x["q"], x["BS"]
    T, Hq, D = q.shape
    G = Hq // x["k_cache"].shape[1]
    for b, L in enumerate(x["lens"]):
        t0, t1 = x["start"][b], x["start"][b + 1]
        n = t1 - t0
        at = torch.arange(L, device="cuda")
        blk, slot = x["block_tables"][b].long()[at // BS], at % BS
        pos = torch.arange(L - n, L, device="cuda").view(n, 1)
        for qh in range(Hq):
            k, v = x["k_cache"][blk, qh // G, slot].double(), x["v_cache"][blk, qh // G, slot].double()
            qq = q[t0:t1, qh].double()
            t, size = qq @ k.T * D ** -0.5, qq.abs() @ k.abs().T * D ** -0.5
            w = torch.softmax((CAP * torch.tanh(t / CAP)).masked_fill(at > pos, float("-inf")), -1)
            o, a = w @ v, w @ v.abs()
            d = (D * E * size.amax(1) + (4 * E + 2.0 ** -20) * t.abs().amax(1)).view(n, 1)
            tol = 2.0 ** -8 * o.abs() + 1.01 * (2.0 ** -8 + 2 * d + 4 * E * (L / 16 + 64)) * a
            over = ((got[t0:t1, qh].double() - o).abs() - tol)[small[t0:t1, qh]]
            assert (over <= 0).all(), f"row {b}, head {qh}: out by up to {over.max():.3e}"


def mixed(x, every):
    """Every `every`-th row of q (over tokens and heads) becomes so large that its scores pass the cap."""
    T, Hq, _ = x["q"].shape
    large = (torch.arange(T * Hq, device="cuda") % every == 0).view(T, Hq)
    x["q"] = torch.where(large[..., None], (x["q"].float() * 2.0 ** 20), x["q"].float()).to(BF)
    return ~large


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 1, 128), (16, 2, 64), (24, 2, 128), (8, 2, 72)])
def test_decode_heads(Hq, Hkv, D):
    x = R.make(21, [900, 40, 333], Hq, Hkv, D, 16, BF)
    small = mixed(x, 3)
    got = pkv.paged_decode_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"], softcap=CAP)
    small_rows(x, small, got)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("members", [5, 50])
def test_shared_members(D, members):
    x = R.make(22, [1000] * members, 16, 2, D, 16, BF)
    bt = x["block_tables"]
    bt[:, :60] = bt[0, :60]
    small = mixed(x, 5)
    more = max(0, (48 << 20) // (4 * members * 16 * 2 * D) + 1 - bt.shape[1])  # so that the prefix is read once
    wide = torch.cat([bt, torch.full((members, more), -1, dtype=torch.int32, device="cuda")], 1)
    got = pkv.paged_decode_attention_shared(x["q"], x["k_cache"], x["v_cache"], wide, x["seq_lens"],
                                            torch.tensor([0, members], dtype=torch.int32, device="cuda"),
                                            torch.tensor([960], dtype=torch.int32, device="cuda"), softcap=CAP)
    small_rows(x, small, got)


@pytest.mark.parametrize("chunks,before", [([3], 700), ([150, 40], 300)])
def test_prefill_rows(chunks, before):
    x = R.make(23, [n + before for n in chunks], 8, 2, 128, 16, BF, chunks=chunks)
    small = mixed(x, 7)
    got = pkv.paged_prefill_attention_scored(x["q"], x["k_cache"], x["v_cache"], x["block_tables"], x["seq_lens"], x["q_start"],
                                             softcap=CAP)
    small_rows(x, small, got)


@pytest.mark.parametrize("call", ["decode", "prefill", "shared"])
@pytest.mark.parametrize("window", [0, 50])
def test_hidden_keys_change_nothing(call, window):
    """K in positions that no query sees, in blocks that are read: zeros, or products far beyond the cap."""
    if call == "shared" and window:
        pytest.skip("no window there")
    lens = [203, 90, 330, 207]
    x = R.make(24, lens, 8, 2, 128, 16, BF, chunks=[3, 1, 2, 5] if call == "prefill" else None)
    if call == "shared":  # a prefix that ends inside a tile of 64 keys, of blocks that hold no more
        x["block_tables"][:, :5] = x["block_tables"][0, :5]
    outs = []
    for fill in (0.0, 2.0 ** 40):
        k = x["k_cache"].clone()
        k[torch.isnan(k)] = fill  # behind the ends, and blocks that no table names
        for b, L in enumerate(lens):
            n = x["start"][b + 1] - x["start"][b]
            for j in range(max(0, L - n - window + 1) if window else 0):
                k[int(x["block_tables"][b, j // 16]), :, j % 16] = fill
        a = [x["q"], k, x["v_cache"].nan_to_num(0.0), x["block_tables"], x["seq_lens"]]
        if call == "decode":
            outs.append(pkv.paged_decode_attention_scored(*a, softcap=CAP, window=window))
        elif call == "prefill":
            outs.append(pkv.paged_prefill_attention_scored(*a, x["q_start"], softcap=CAP, window=window))
        else:
            a[3] = torch.cat([a[3], torch.full((4, 4000), -1, dtype=torch.int32, device="cuda")], 1)
            outs.append(pkv.paged_decode_attention_shared(*a, torch.tensor([0, 4], dtype=torch.int32, device="cuda"),
                                                          torch.tensor([80], dtype=torch.int32, device="cuda"), softcap=CAP))
    assert torch.isfinite(outs[0]).all()
    assert torch.equal(outs[0], outs[1])
