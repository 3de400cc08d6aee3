"""Attention of chunks of new tokens over the cache: GPU parity with the fp64
oracle.

Tolerance of an output: a weight is rounded to the input type once, off by at
most u = eps / 2 of it, so the sum is off by at most u * A with A = sum_j p_j
|v_j| (the oracle's output for |V|); the output's own rounding adds u * (|O| +
u A); scores, exponentials and sums are float32 (a score of a few units is off
by less than 5e-5, an exponential by 2^-21 of it, the products and sums by
less than 5e-5): 2e-4 * A covers them.
"""
import numpy as np
import pytest
import torch

import oracle
from decode_attention_packed_b200.workloads import Workload, make_inputs, make_varlen_queries
from tests.tolerance import assert_lse_close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def draw(q_lens, lengths, Hq=8, Hkv=2, D=128, dtype="bf16", page_size=16, seed=1000, k_scale=1.0):
    w = Workload(name="prefill", B=len(q_lens), q_len=1, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, page_size=page_size,
                 causal=True, lengths="list:" + ",".join(map(str, lengths)), seed=seed, k_scale=k_scale)
    inp = make_inputs(w)
    q, cu = make_varlen_queries(q_lens, Hq, D, dtype, seed + 1)
    return inp, q, cu


def run(inp, q, cu, **kw):
    bt = None if inp.block_table is None else inp.block_table.cuda()
    max_q = max(1, int((cu[1:] - cu[:-1]).max()))
    out, lse = mxa.prefill(q.cuda(), cu.cuda(), inp.k_cache.cuda(), inp.v_cache.cuda(), bt, inp.cache_seqlens.cuda(),
                           max_seqlen_q=max_q, max_seqlen_k=inp.max_seqlen_k, **kw)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    return out.cpu(), lse.cpu()


def check(inp, q, cu, out, lse, causal=True, window=0, sinks=0, scale=None):
    w = inp.w
    args = dict(Hkv=w.Hkv, page_size=inp.page_size, dtype=w.dtype, scale=w.scale if scale is None else scale,
                causal=causal, window=window, sinks=sinks)
    ro, rl = oracle.decode_varlen(q, cu.numpy(), inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens, **args)
    ra, _ = oracle.decode_varlen(q, cu.numpy(), inp.k_cache, inp.v_cache.abs(), inp.block_table, inp.cache_seqlens, **args)
    u = torch.finfo(q.dtype).eps / 2
    err = np.abs(out.double().numpy() - ro)
    bound = u * ra + u * (np.abs(ro) + u * ra) + 2e-4 * ra
    assert np.isfinite(err).all()
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (f"{(err > bound).sum()} of {err.size} off; worst at {worst}: {err[worst]:.3e} against "
                                  f"{bound[worst]:.3e}")
    assert_lse_close(lse, rl)


Q_LENS = [1, 0, 33, 200, 128, 5, 300]
LENGTHS = [700, 50, 33, 1000, 129, 3, 1025]  # the sixth row has more queries than keys


@pytest.mark.parametrize("D,dtype,page_size", [(128, "bf16", 16), (64, "f16", 8), (256, "bf16", 64), (128, "f16", 0),
                                               (64, "bf16", 24), (256, "f16", 128), (128, "bf16", 192), (64, "f16", 0)])
@pytest.mark.parametrize("causal,window,sinks", [(True, 0, 0), (False, 0, 0), (True, 1, 0), (True, 100, 4),
                                                 (True, 257, 130), (True, 64, 64), (True, 5000, 9)])
def test_matches_oracle(D, dtype, page_size, causal, window, sinks):
    inp, q, cu = draw(Q_LENS, LENGTHS, D=D, dtype=dtype, page_size=page_size)
    check(inp, q, cu, *run(inp, q, cu, causal=causal, window=window, sinks=sinks), causal, window, sinks)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (6, 2), (10, 2), (7, 1), (32, 2), (128, 1), (66, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_groups(Hq, Hkv, D):
    inp, q, cu = draw([70, 1, 0, 3], [200, 90, 10, 3], Hq=Hq, Hkv=Hkv, D=D, seed=1100)
    check(inp, q, cu, *run(inp, q, cu))


@pytest.mark.parametrize("q_lens,lengths", [([1], [1]), ([1], [0]), ([3], [1]), ([1], [9000]), ([257], [257]),
                                            ([16], [6000]), ([0, 0, 1], [5, 0, 128]), ([2] * 150, list(range(2, 302, 2)))])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_small_and_single(q_lens, lengths, D):
    # one token to a few, over nothing and over thousands of keys (cut into
    # many pieces), and many short rows
    inp, q, cu = draw(q_lens, lengths, D=D, seed=1200)
    for causal in (True, False):
        check(inp, q, cu, *run(inp, q, cu, causal=causal), causal)


@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "f16"), (256, "bf16")])
@pytest.mark.parametrize("longest", [1024, 1029])
def test_contiguous_rows_at_any_place(D, dtype, longest):
    # the rows of a contiguous cache start at multiples of 8 tokens, or not
    inp, q, cu = draw([130, 1, 40], [700, 200, longest], D=D, dtype=dtype, page_size=0, seed=1250)
    for window, sinks in ((0, 0), (150, 9)):
        check(inp, q, cu, *run(inp, q, cu, window=window, sinks=sinks), True, window, sinks)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_peaked_scores_rescale_the_accumulator(D):
    # keys times 12, and rising along the row: the running maximum grows many times
    inp, q, cu = draw([150], [1500], D=D, seed=1300, k_scale=4.0)
    ramp = torch.linspace(0.2, 3.0, 1500)
    for j in range(1500):
        page, slot = int(inp.block_table[0, j // 16]), j % 16
        inp.k_cache[page, slot] = (inp.k_cache[page, slot].float() * ramp[j]).to(inp.k_cache.dtype)
    out, lse = run(inp, q, cu)
    w = inp.w
    ro, rl = oracle.decode_varlen(q, cu.numpy(), inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens, Hkv=w.Hkv,
                                  page_size=16, dtype=w.dtype, scale=w.scale, causal=True)
    ra, _ = oracle.decode_varlen(q, cu.numpy(), inp.k_cache, inp.v_cache.abs(), inp.block_table, inp.cache_seqlens,
                                 Hkv=w.Hkv, page_size=16, dtype=w.dtype, scale=w.scale, causal=True)
    # scores reach |s| ~ 50: a float32 score is off by up to D * 2^-24 * sum |q k| * scale < 1e-3,
    # and so is its exponential, relatively
    u = torch.finfo(q.dtype).eps / 2
    err = np.abs(out.double().numpy() - ro)
    assert (err <= u * ra + u * (np.abs(ro) + u * ra) + 2e-3 * ra).all()
    assert np.abs(lse.double().numpy() - rl).max() <= 1e-3


@pytest.mark.parametrize("scale", [0.0, -0.09, 0.5])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scales(scale, D):
    inp, q, cu = draw([40, 3], [300, 70], D=D, seed=1400)
    check(inp, q, cu, *run(inp, q, cu, scale=scale), scale=scale)


@pytest.mark.parametrize("page_size", [16, 0])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_hidden_keys_may_hold_anything(D, page_size):
    # NaN and infinities past the rows' ends and between the sinks and the
    # window; hidden pages' table entries point outside the pool
    window, sinks, L, n = 200, 20, 1500, 60
    inp, q, cu = draw([n, 1], [L, 40], D=D, page_size=page_size, seed=1500)
    clean = run(inp, q, cu, window=window, sinks=sinks)
    low = L - n + 1 - window
    where = lambda b, j: (b, j) if page_size == 0 else (int(inp.block_table[b, j // 16]), j % 16)  # noqa: E731
    spoiled = [(0, j) for j in range(sinks, low)]
    spoiled += [(1, j) for j in (range(40, 48) if page_size else range(40, inp.page_size))]
    if page_size:
        spoiled += [(0, j) for j in range(L, -(-L // 16) * 16)]
    for b, j in spoiled:
        page, slot = where(b, j)
        inp.k_cache[page, slot] = float("nan")
        inp.v_cache[page, slot] = float("inf") if j % 2 else float("nan")
    again = run(inp, q, cu, window=window, sinks=sinks)
    assert torch.equal(again[0].view(torch.int16), clean[0].view(torch.int16)) and torch.equal(again[1], clean[1])
    if page_size:
        for p in range(inp.block_table.shape[1]):
            if p * 16 >= sinks and (p + 1) * 16 <= low:
                inp.block_table[0, p] = 10**6 if p % 2 else -1
        again = run(inp, q, cu, window=window, sinks=sinks)
        assert torch.equal(again[0].view(torch.int16), clean[0].view(torch.int16)) and torch.equal(again[1], clean[1])


def test_bad_pages_read_as_zeros_and_are_reported():
    inp, q, cu = draw([20], [300], seed=1600)
    for entry in (10**6, -5):
        inp.block_table[0, 3] = entry
        bt = inp.block_table.cuda()
        out, _ = mxa.prefill(q.cuda(), cu.cuda(), inp.k_cache.cuda(), inp.v_cache.cuda(), bt, inp.cache_seqlens.cuda(),
                             max_seqlen_q=20, max_seqlen_k=inp.max_seqlen_k)
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_ERR_INVALID_ARG
        assert torch.isfinite(out.float()).all()


def test_broken_offsets_and_lengths_stay_in_bounds():
    inp, q, _ = draw([30, 30, 30], [300, 40, 100], seed=1700)
    total, pad = 90, 64
    w = inp.w
    out_buf = torch.full((total + 2 * pad, w.Hq, w.D), 7.0, dtype=q.dtype, device="cuda")
    lse_buf = torch.full((w.Hq * total + 2 * pad,), 7.0, dtype=torch.float32, device="cuda")
    args = [x.cuda() for x in (inp.k_cache, inp.v_cache, inp.block_table)]
    for cu, lens in (([0, 50, 20, 400], [300, 40, 100]), ([-9, 10, 20, 30], [300, 40, 100]),
                     ([0, 30, 60, 90], [-4, 10**6, 2**31 - 1]), ([5, 40, 60, 90], [0, 0, 0])):
        mxa.prefill(q.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"), *args,
                    torch.tensor(lens, dtype=torch.int32, device="cuda"), max_seqlen_q=30, max_seqlen_k=inp.max_seqlen_k,
                    out=out_buf[pad:-pad], lse=lse_buf[pad:-pad].view(w.Hq, total))
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_ERR_INVALID_ARG
        assert (out_buf[:pad] == 7).all() and (out_buf[-pad:] == 7).all()
        assert (lse_buf[:pad] == 7).all() and (lse_buf[-pad:] == 7).all()


def test_calls_repeat_bit_for_bit_and_in_a_graph():
    # a garbage workspace, many calls, and a graph replayed after its inputs changed
    inp, q, cu = draw([200, 1, 60], [2000, 3000, 60], seed=1800)
    first = run(inp, q, cu)
    args = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    prep = mxa.prepare_prefill(args[0], args[1], args[2], args[4], max_seqlen_q=200, max_seqlen_k=inp.max_seqlen_k)
    prep.workspace.random_(0, 255)
    out, lse = torch.empty_like(args[0]), torch.empty((8, 261), device="cuda")
    for _ in range(20):
        mxa.prefill(*args, max_seqlen_q=200, prepared=prep, out=out, lse=lse)
        assert torch.equal(out.cpu().view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse.cpu(), first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxa.prefill(*args, max_seqlen_q=200, prepared=prep, out=out, lse=lse)
    cu = torch.tensor([0, 61, 62, 261], dtype=torch.int32)
    inp.cache_seqlens.copy_(torch.tensor([1999, 7, 60], dtype=torch.int32))
    args[1].copy_(cu)
    args[5].copy_(inp.cache_seqlens)
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    check(inp, q, cu, out.cpu(), lse.cpu())


def test_two_calls_on_two_streams():
    inp, q, cu = draw([200, 1, 60], [2000, 3000, 60], seed=1900)
    first = run(inp, q, cu)
    args = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    torch.cuda.synchronize()
    results = []
    for _ in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            results.append([mxa.prefill(*args, max_seqlen_q=200, max_seqlen_k=inp.max_seqlen_k) for _ in range(5)])
    torch.cuda.synchronize()
    for out, lse in results[0] + results[1]:
        assert torch.equal(out.cpu().view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse.cpu(), first[1])


def test_no_queries_and_refusals():
    inp, q, cu = draw([4, 2], [40, 9])
    args = [x.cuda() for x in (inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = mxa.prefill(q[:0].cuda(), none, *args, max_seqlen_q=1)
    assert out.shape == (0, 8, 128) and lse.shape == (8, 0)
    qd, cd = q.cuda(), cu.cuda()
    for kw in (dict(causal=False, window=5), dict(sinks=4), dict(window=-1), dict(scale=float("inf"))):
        with pytest.raises(mxa.MxaError):
            mxa.prefill(qd, cd, *args, max_seqlen_q=4, **kw)
    with pytest.raises(ValueError):
        mxa.prefill(qd.transpose(0, 1), cd, *args, max_seqlen_q=4)
    with pytest.raises(ValueError):
        mxa.prefill(qd, cd[:2], *args, max_seqlen_q=4, prepared=mxa.prepare_prefill(qd, cd, args[0], args[2], max_seqlen_q=4))
    with pytest.raises(TypeError):
        mxa.prefill(qd, cd, args[0].half(), *args[1:], max_seqlen_q=4)


@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_most_of_them_idle(D):
    # thousands of rows; long runs without queries, single tokens, one long chunk
    B = 3000
    q_lens = [0] * B
    for b in (0, 7, 700, 701, 702, 1999, 2998):
        q_lens[b] = 1 + b % 3
    q_lens[1500] = 900
    lengths = [5] * B
    for b in range(B):
        if q_lens[b]:
            lengths[b] = q_lens[b] + b % 50
    inp, q, cu = draw(q_lens, lengths, Hq=2, Hkv=1, D=D, seed=1650)
    check(inp, q, cu, *run(inp, q, cu))


def test_padding_behind_the_last_row_stays_as_it_was():
    # one captured call with room for 8 rows and 96 tokens, replayed for smaller batches
    inp, q, cu = draw([30, 0, 1, 40, 1, 0, 2, 22], [300, 9, 77, 40, 1000, 5, 2, 500], seed=1750)
    total = 96
    args = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    prep = mxa.prepare_prefill(args[0], args[1], args[2], args[4], max_seqlen_q=40, max_seqlen_k=inp.max_seqlen_k)
    out, lse = torch.empty_like(args[0]), torch.empty((8, total), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mxa.prefill(*args, max_seqlen_q=40, prepared=prep, out=out, lse=lse)
    for rows in (8, 5, 4, 1, 0):
        end = int(cu[rows])
        part = cu.clamp_max(end)
        args[1].copy_(part)
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_OK
        assert (out[end:] == 7).all() and (lse[:, end:] == 7).all()
        if end:
            check(inp, q[:end], part, out[:end].cpu(), lse[:, :end].cpu())


def test_overlapping_rows_are_reported():
    # offsets that fall back make thousands of rows out of the same tokens:
    # more work than the call was laid out for, none of which is run
    B, T, Hq, Hkv, D, page, width = 12000, 4096, 64, 8, 64, 1024, 128
    k, v = (torch.zeros(4, page, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2))
    q = torch.zeros(T, Hq, D, dtype=torch.float16, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), page * width, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=T, causal=False, out=out)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_ERR_INVALID_ARG
    assert (out == 7).all()


def test_a_prepared_call_refuses_other_shapes():
    inp, q, cu = draw([4, 2], [40, 9])
    qd, cd, k, v, table, lens = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    prep = mxa.prepare_prefill(qd, cd, k, table, max_seqlen_q=4)
    mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=4, prepared=prep)
    for args in ((qd[:, :4].contiguous(), cd, k, v, table, lens), (qd, cd, k[:-1], v[:-1], table, lens),
                 (qd, cd, k, v, table[:, :-1].contiguous(), lens)):
        with pytest.raises(ValueError):
            mxa.prefill(*args, max_seqlen_q=4, prepared=prep)
    with pytest.raises(TypeError):
        mxa.prefill(qd.half(), cd, k.half(), v.half(), table, lens, max_seqlen_q=4, prepared=prep)
    with pytest.raises(ValueError):
        host = mxa.Prepared(prep.params, None, prep.workspace.cpu())
        mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=4, prepared=host)
    with pytest.raises(mxa.MxaError):  # more tokens than it was prepared for
        small = mxa.Prepared(prep.params, None, prep.workspace[:256])
        mxa.prefill(qd, cd, k, v, table, lens, max_seqlen_q=4, prepared=small)


def test_a_stream_given_by_hand():
    inp, q, cu = draw([200, 1, 60], [2000, 3000, 60], seed=1900)
    first = run(inp, q, cu)
    args = [x.cuda() for x in (q, cu, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens)]
    out, lse = torch.empty_like(args[0]), torch.empty((8, 261), device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out.zero_()
        torch.cuda.synchronize()
        mxa.prefill(*args, max_seqlen_q=200, max_seqlen_k=inp.max_seqlen_k, out=out, lse=lse, stream=stream)
        torch.empty(64 << 20, dtype=torch.uint8, device="cuda").fill_(255)  # what the current stream allocates meanwhile
        torch.cuda.synchronize()
        assert torch.equal(out.cpu().view(torch.int16), first[0].view(torch.int16)) and torch.equal(lse.cpu(), first[1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_output_at_a_multiple_of_16_bytes(D):
    inp, q, cu = draw([130, 1, 40], [700, 200, 2000], D=D, seed=1960)
    out = torch.empty(q.numel() + 8, dtype=q.dtype, device="cuda")[8:].view(q.shape)
    assert out.data_ptr() % 32 == 16
    check(inp, q, cu, *run(inp, q, cu, out=out))


@pytest.mark.parametrize("q_lens,lengths", [([300, 2], [3000, 900]), ([1], [9000])])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_nan_in_seen_places_stays(q_lens, lengths, D):
    # also through the merge of units cut in few and in many pieces
    inp, q, cu = draw(q_lens, lengths, D=D, seed=1970)
    keep = inp.v_cache.clone()
    inp.v_cache.fill_(float("nan"))
    out, lse = run(inp, q, cu)
    assert out.isnan().all() and lse.isfinite().all()
    inp.v_cache.copy_(keep)
    inp.k_cache.fill_(float("nan"))
    out, lse = run(inp, q, cu)
    assert out.isnan().all() and lse.isnan().all()
