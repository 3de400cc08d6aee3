"""Decode with a sliding window and sinks: GPU parity with the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from decode_attention_packed_b200.workloads import Workload, make_inputs
from tests.test_gpu_append import split_off_new_tokens
from tests.tolerance import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def draw(lengths, q_len=1, Hq=16, Hkv=4, D=128, dtype="bf16", page_size=16, seed=900):
    return make_inputs(Workload(name="window", B=len(lengths), q_len=q_len, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype,
                                page_size=page_size, causal=True, lengths="list:" + ",".join(map(str, lengths)), seed=seed))


def on_gpu(inp):
    bt = None if inp.block_table is None else inp.block_table.cuda()
    return inp.q.cuda(), inp.k_cache.cuda(), inp.v_cache.cuda(), bt, inp.cache_seqlens.cuda()


def run(inp, window, sinks, num_splits=0, **kw):
    out, lse = mxa.decode(*on_gpu(inp), scale=inp.w.scale, causal=True, window=window, sinks=sinks, num_splits=num_splits,
                          max_seqlen_k=inp.max_seqlen_k, **kw)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    return out.cpu(), lse.cpu()


def check(inp, out, lse, window, sinks):
    w = inp.w
    ro, rl = oracle.decode(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens, Hkv=w.Hkv,
                           page_size=inp.page_size, dtype=w.dtype, scale=w.scale, causal=True, window=window, sinks=sinks)
    assert_out_close(out, ro, w.dtype)
    assert_lse_close(lse, rl)


LENGTHS = [0, 1, 2, 63, 64, 65, 127, 200, 700, 1025, 3000, 4096]


@pytest.mark.parametrize("D,dtype,page_size", [(128, "bf16", 16), (64, "f16", 8), (256, "bf16", 64), (128, "f16", 0),
                                               (64, "bf16", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (33, 4), (64, 64), (300, 0), (257, 130), (5000, 7)])
def test_matches_oracle(D, dtype, page_size, window, sinks):
    inp = draw(LENGTHS, D=D, dtype=dtype, page_size=page_size)
    for num_splits in (0, 1, 5):
        check(inp, *run(inp, window, sinks, num_splits), window, sinks)


@pytest.mark.parametrize("q_len,Hq,Hkv", [(2, 8, 8), (4, 32, 8), (8, 24, 4), (3, 5, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 3), (100, 5), (1000, 64)])
def test_draft_tokens_and_groups(q_len, Hq, Hkv, window, sinks):
    # several queries a row, each with its own window; rows with fewer keys than queries
    inp = draw([0, 1, 5, 90, 129, 1500, 4000], q_len=q_len, Hq=Hq, Hkv=Hkv, page_size=32)
    for num_splits in (0, 3):
        check(inp, *run(inp, window, sinks, num_splits), window, sinks)


@pytest.mark.parametrize("page_size", [16, 0])
def test_hidden_keys_may_hold_anything(page_size):
    # NaN and infinities between the sinks and the window, and in the slots
    # past the row; the hidden pages' table entries point outside the pool
    window, sinks, L = 300, 20, 2100
    inp = draw([L, 40, L], page_size=page_size)
    clean = run(inp, window, sinks)
    low = L - window
    for b in (0, 2):
        for j in list(range(sinks, low)):
            page, slot = (b, j) if page_size == 0 else (int(inp.block_table[b, j // page_size]), j % page_size)
            inp.k_cache[page, slot] = float("nan")
            inp.v_cache[page, slot] = float("inf") if j % 2 else float("nan")
    again = run(inp, window, sinks)
    assert torch.equal(again[0].view(torch.int16), clean[0].view(torch.int16)) and torch.equal(again[1], clean[1])
    if page_size:
        hidden = torch.tensor([sinks <= p * 16 and (p + 1) * 16 <= low for p in range(inp.block_table.shape[1])])
        for b in (0, 2):
            inp.block_table[b, hidden] = 10**6 if b else -1
        again = run(inp, window, sinks)
        assert torch.equal(again[0].view(torch.int16), clean[0].view(torch.int16)) and torch.equal(again[1], clean[1])


@pytest.mark.parametrize("q_len,page_size", [(1, 16), (4, 64), (2, 0)])
def test_append_then_window(q_len, page_size):
    inp = draw([q_len, 70, 600, 2049, 4096], q_len=q_len, page_size=page_size, seed=930)
    k_blank, v_blank, k_new, v_new, before = split_off_new_tokens(inp, q_len)
    k, v = k_blank.cuda(), v_blank.cuda()
    bt = None if inp.block_table is None else inp.block_table.cuda()
    out, lse = mxa.decode(inp.q.cuda(), k, v, bt, before.cuda(), scale=inp.w.scale, causal=True, window=130, sinks=4,
                          max_seqlen_k=inp.max_seqlen_k, k_new=k_new.cuda(), v_new=v_new.cuda())
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert torch.equal(k.cpu().view(torch.int16), inp.k_cache.view(torch.int16))
    assert torch.equal(v.cpu().view(torch.int16), inp.v_cache.view(torch.int16))
    check(inp, out.cpu(), lse.cpu(), 130, 4)


def test_refusals():
    inp = draw([40])
    q, k, v, bt, sl = on_gpu(inp)
    for kw in (dict(window=-1, causal=True), dict(window=4, causal=False), dict(sinks=3, causal=True),
               dict(window=4, causal=True, out_dtype=torch.float32)):
        with pytest.raises(ValueError):
            mxa.decode(q, k, v, bt, sl, **kw)


def test_captured_and_replayed_with_new_lengths():
    # one graph, replayed after the lengths and the queries changed in place
    inp = draw([900, 2000, 64, 1])
    q, k, v, bt, sl = on_gpu(inp)
    prep = mxa.prepare(q, k, bt, max_seqlen_k=inp.max_seqlen_k, window=200, sinks=4)
    out, lse = mxa.decode(q, k, v, bt, sl, causal=True, window=200, sinks=4, prepared=prep)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxa.decode(q, k, v, bt, sl, causal=True, window=200, sinks=4, prepared=prep, out=out, lse=lse)
    inp.cache_seqlens.copy_(torch.tensor([333, 1999, 0, 1], dtype=torch.int32))
    inp.q.copy_(inp.q.flip(0))
    sl.copy_(inp.cache_seqlens)
    q.copy_(inp.q)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    check(inp, out.cpu(), lse.cpu(), 200, 4)
