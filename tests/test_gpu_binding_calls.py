"""Calls of the binding around their preparation, on the GPU; what is handed to
the library is tested without one in test_binding_calls.py."""
import pytest
import torch

from tests.test_gpu_prefill import check, draw

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_chunk_longer_than_it_was_prepared_for(D):
    inp, q, cu = draw([200, 1, 60], [2000, 3000, 60], D=D, seed=2300)
    qd, cd, k, v, table, lens = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    prep = mxa.prepare_prefill(qd, cd, k, table, max_seqlen_q=4, max_seqlen_k=2500)
    out, lse = mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=200, max_seqlen_k=3000, prepared=prep)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    check(inp, q, cu, out.cpu(), lse.cpu())


def test_a_preparation_too_small_is_refused():
    # one block of keys and one token make a grid of few ranges
    inp, q, cu = draw([200, 1, 60], [2000, 3000, 60], seed=2310)
    qd, cd, k, v, table, lens = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    prep = mxa.prepare_prefill(qd[:1], cd[:2], k, table[:1], max_seqlen_q=1, max_seqlen_k=64)
    short = mxa.Prepared(mxa.prepare_prefill(qd, cd, k, table, max_seqlen_q=200).params, None, prep.workspace)
    with pytest.raises(mxa.MxaError):
        mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=200, prepared=short)


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4)])
@pytest.mark.parametrize("num_splits", [0, 3])
def test_a_row_longer_than_the_decode_was_prepared_for(window, sinks, num_splits):
    inp, q, cu = draw([1, 1, 1], [2000, 3000, 60], seed=2320)
    qd, k, v, table, lens = [x.cuda() for x in (q, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    rows = qd.view(3, 1, *q.shape[1:])
    prep = mxa.prepare(rows, k, table, max_seqlen_k=500, num_splits=num_splits, window=window, sinks=sinks)
    out, lse = mxa.decode(rows, k, v, table, lens, causal=True, window=window, sinks=sinks, max_seqlen_k=3000, prepared=prep)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    check(inp, q, cu, out.cpu().view(q.shape), lse.cpu().view(3, -1).t(), window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(2**40 + 5, 0), (2**31 - 1, 2**40), (3, 2**32 + 1)])
def test_windows_past_32_bits_hide_nothing(window, sinks):
    inp, q, cu = draw([1, 1, 1], [2000, 3000, 60], seed=2330)
    qd, cd, k, v, table, lens = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    rows = qd.view(3, 1, *q.shape[1:])
    out, lse = mxa.decode(rows, k, v, table, lens, causal=True, window=window, sinks=sinks)
    chunk = mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=1, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    check(inp, q, cu, out.cpu().view(q.shape), lse.cpu().view(3, -1).t())
    check(inp, q, cu, chunk[0].cpu(), chunk[1].cpu())


def test_a_step_without_new_tokens():
    inp, q, cu = draw([4, 2], [40, 9])
    qd, k, v, table, lens = [x.cuda() for x in (q, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = mxa.prefill(qd[:0], none, k, v, table, lens, max_seqlen_q=0)
    assert out.shape == (0, 8, 128) and lse.shape == (8, 0)
    keep_out, keep_lse = torch.full_like(qd, 7.0), torch.full((8, 6), 7.0, device="cuda")
    mxa.prefill(qd, none, k, v, table, lens, max_seqlen_q=0, out=keep_out, lse=keep_lse)  # padding alone
    no_rows = mxa.prefill(qd[:0], none[:1], k, v, table[:0], lens[:0], max_seqlen_q=0)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert (keep_out == 7).all() and (keep_lse == 7).all() and no_rows[0].shape == (0, 8, 128)
