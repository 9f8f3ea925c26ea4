"""Calls of one kernel with different sizes from several threads at once."""
import ctypes
import threading

import pytest
import torch

import paged_kv_decode_table_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from paged_kv_decode_table_gb300 import build
    build.build()


def ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def in_threads(calls, rounds):
    """Every call `rounds` times, each in a thread of its own; the status codes that came back."""
    codes = [set() for _ in calls]
    start = threading.Barrier(len(calls))

    def work(i):
        start.wait()
        for _ in range(rounds):
            codes[i].add(int(calls[i]()))
    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    return codes


def tables(lens, BS, g):
    need = [-(-n // BS) for n in lens]
    perm = torch.randperm(sum(need), generator=g).to(torch.int32)
    bt = torch.zeros(len(lens), max(need), dtype=torch.int32)
    for b, part in enumerate(perm.split(need)):
        bt[b, :len(part)] = part
    return bt.cuda(), sum(need)


def run(cases, rounds=4000):
    """cases: (call, result of the call made alone, its output buffer, what has to stay alive)."""
    torch.cuda.synchronize()
    assert in_threads([c[0] for c in cases], rounds) == [{0}] * len(cases)
    torch.cuda.synchronize()
    for _, want, out, *_ in cases:
        assert torch.equal(want, out)


def test_decode_attention():
    lib, cases = pkv.load_library(), []
    for n, (Hq, Hkv) in enumerate([(8, 8), (8, 1), (12, 3), (10, 5)]):
        g = torch.Generator().manual_seed(n)
        lens = [900, 1500]
        bt, nb = tables(lens, 16, g)
        k, v = (torch.randn(nb, Hkv, 16, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = torch.randn(2, Hq, 128, generator=g).to(torch.bfloat16).cuda()
        sl = torch.tensor(lens, dtype=torch.int32).cuda()
        want = pkv.paged_decode_attention(q, k, v, bt, sl)
        out = torch.zeros_like(want)
        ws = torch.empty(pkv.decode_workspace_bytes(2, Hq, 128), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        a = (ptr(out), ptr(q), ptr(k), ptr(v), ptr(bt), bt.shape[1], ptr(sl), 2, Hq, Hkv, 128, 16, nb,
             ctypes.c_float(0.0), 1, ptr(ws), ws.numel(), None, ctypes.c_void_p(s.cuda_stream))
        cases.append((lambda a=a: lib.pkv_paged_decode_attention(*a), want, out, q, k, v, bt, sl, ws, s))
    run(cases)


def test_sampler():
    lib, cases = pkv.load_library(), []
    for n, (B, V) in enumerate([(3, 9000), (2, 152064), (5, 50000), (2, 21000)]):
        g = torch.Generator().manual_seed(n)
        logits = torch.randn(B, V, generator=g).cuda()
        temp, top_p = torch.full((B,), 0.8).cuda(), torch.full((B,), 0.9).cuda()
        top_k = torch.full((B,), 50, dtype=torch.int32).cuda()
        seeds, offs = (torch.arange(B).cuda() + i for i in range(2))
        want = pkv.sample_tokens(logits, temp, top_k, top_p, seeds, offs)
        out = torch.zeros_like(want)
        s = torch.cuda.Stream()
        a = (ptr(out), ptr(logits), B, V, ptr(temp), ptr(top_k), ptr(top_p), ptr(seeds), ptr(offs), None, 0, None,
             ctypes.c_void_p(s.cuda_stream))
        cases.append((lambda a=a: lib.pkv_sample_tokens(*a), want, out, logits, temp, top_k, top_p, seeds, offs, s))
    run(cases)


def test_prefill_attention():
    """Queries at a 4-byte address take the kernel whose CTA depends on the query heads of a KV head."""
    lib, cases = pkv.load_library(), []
    for n, (Hq, Hkv) in enumerate([(5, 1), (8, 1), (2, 2), (4, 1)]):
        g = torch.Generator().manual_seed(n)
        lens, qs = [150, 70], [0, 40, 60]
        bt, nb = tables(lens, 16, g)
        k, v = (torch.randn(nb, Hkv, 16, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = torch.randn(60 * Hq * 128 + 2, generator=g).to(torch.bfloat16).cuda()[2:].view(60, Hq, 128)
        sl, st = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, qs))
        want = pkv.paged_prefill_attention(q, k, v, bt, sl, st)
        out = torch.zeros_like(want)
        s = torch.cuda.Stream()
        a = (ptr(out), ptr(q), ptr(k), ptr(v), ptr(bt), bt.shape[1], ptr(sl), ptr(st), 2, 60, Hq, Hkv, 128, 16, nb,
             ctypes.c_float(0.0), 1, None, ctypes.c_void_p(s.cuda_stream))
        cases.append((lambda a=a: lib.pkv_paged_prefill_attention(*a), want, out, q, k, v, bt, sl, st, s))
    run(cases, 2000)
