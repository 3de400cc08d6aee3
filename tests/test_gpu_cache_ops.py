"""Block tables, slot maps and the cache write on the GPU, against the oracle's
tables and a token-by-token copy: equal in every value."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def problem(ctx, new, page, spare=5, width=None, num_free=None, seed=1):
    """A table whose rows hold the pages of their ctx keys, and a free list for the new tokens."""
    r = np.random.default_rng(seed)
    ctx, new = np.asarray(ctx, dtype=np.int64), np.asarray(new, dtype=np.int64)
    have, need = -(-ctx // page), -(-(ctx + new) // page)
    pages = int(need.sum()) + spare
    perm = r.permutation(pages)
    w = max(1, int(need.max(initial=0))) if width is None else width
    table = np.full((ctx.size, w), -7)
    at = 0
    for b in range(ctx.size):
        table[b, :have[b]] = perm[at:at + have[b]]
        at += have[b]
    free = perm[at:] if num_free is None else perm[at:at + num_free]
    cu = np.concatenate([[0], np.cumsum(new)])
    return table, ctx, cu, free, pages


def check(table, ctx, cu, free, pages, page, expect=None):
    t = ints(table)
    slots, lens, used = mxa.extend_tables(t, ints(ctx), ints(cu), ints(free), page_size=page, num_pages=pages,
                                          total_q=int(cu[-1]))
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == (mxa.MXA_OK if expect is None else expect)
    bt, sl, nl, us = oracle.extend_tables(table, ctx, cu, free, page_size=page, num_pages=pages)
    assert np.array_equal(t.cpu().numpy(), bt)
    assert np.array_equal(slots.cpu().numpy(), sl)
    assert np.array_equal(lens.cpu().numpy(), nl)
    assert used.tolist() == [us]


@pytest.mark.parametrize("page", [1, 8, 16, 24, 128])
@pytest.mark.parametrize("B,new_hi", [(1, 1), (1, 700), (7, 1), (130, 40), (1023, 3), (1025, 9), (5000, 2), (2500, 30)])
def test_tables_match_oracle(page, B, new_hi):
    r = np.random.default_rng(B + page)
    ctx = r.integers(0, 300, B)
    new = r.integers(0, new_hi + 1, B)
    ctx[r.integers(0, B, B // 3)] = 0
    check(*problem(ctx, new, page, seed=B), page)


def test_tables_with_empty_rows_and_full_pages():
    check(*problem([0, 0, 16, 16, 32, 31, 0], [0, 16, 0, 16, 1, 1, 0], 16), 16)
    check(*problem([0, 0, 0], [0, 0, 0], 16), 16)
    check(*problem([], [], 16), 16)


@pytest.mark.parametrize("num_free", [0, 1, 3, 40])
def test_tables_when_the_free_list_runs_out(num_free):
    r = np.random.default_rng(num_free)
    ctx, new = r.integers(0, 60, 1500), r.integers(0, 5, 1500)
    check(*problem(ctx, new, 16, num_free=num_free), 16)


def test_tables_when_a_row_is_too_narrow():
    check(*problem([10, 40, 64, 0], [10, 40, 1, 9], 16, width=4), 16)


def test_tables_give_padding_no_slot():
    table, ctx, cu, free, pages = problem([20, 3, 0], [20, 3, 9], 16)
    for total in (32, 33, 5000):
        t = ints(table)
        slots, lens, used = mxa.extend_tables(t, ints(ctx), ints(cu), ints(free), page_size=16, num_pages=pages, total_q=total)
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_OK
        bt, sl, nl, us = oracle.extend_tables(table, ctx, cu, free, page_size=16, num_pages=pages, total_q=total)
        assert np.array_equal(t.cpu().numpy(), bt) and np.array_equal(slots.cpu().numpy(), sl)
        assert np.array_equal(lens.cpu().numpy(), nl) and used.tolist() == [us]


def test_tables_report_a_bad_page():
    table, ctx, cu, free, pages = problem([20, 3], [20, 3], 16)
    free = free.copy()
    free[0] = pages + 3
    check(table, ctx, cu, free, pages, 16, mxa.MXA_ERR_INVALID_ARG)


def test_tables_stay_in_bounds_for_broken_inputs():
    # lengths and offsets that break their rules: clamped and reported; what
    # lies around the outputs stays
    B, width, total = 4, 6, 30
    for lens, cu in (([-5, 10**9, 3, 2**31 - 1], [0, 4, 9, 20, 30]), ([1, 2, 3, 4], [0, 25, 3, 90, -7]),
                     ([1, 2, 3, 4], [5, 6, 7, 8, 9])):
        table_buf = torch.full((B + 2, width), -9, dtype=torch.int32, device="cuda")
        slot_buf = torch.full((total + 128,), -9, dtype=torch.int32, device="cuda")
        len_buf = torch.full((B + 128,), -9, dtype=torch.int32, device="cuda")
        mxa.extend_tables(table_buf[1:-1], ints(lens), ints(cu), torch.arange(40, dtype=torch.int32, device="cuda"),
                          page_size=16, num_pages=64, total_q=total, slots=slot_buf[64:-64], new_seqlens=len_buf[64:-64])
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_ERR_INVALID_ARG
        for buf, pad in ((table_buf, 1), (slot_buf, 64), (len_buf, 64)):
            assert (buf[:pad] == -9).all() and (buf[-pad:] == -9).all()
        assert (slot_buf < 64 * 16).all()


@pytest.mark.parametrize("Hkv,D,dtype", [(8, 128, "bf16"), (1, 64, "f16"), (5, 64, "bf16"), (3, 8, "f16"), (16, 256, "bf16")])
@pytest.mark.parametrize("total", [1, 2, 33, 1000])
def test_write_matches_copy(Hkv, D, dtype, total):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator().manual_seed(total)
    pages, page = 80, 16
    k_cache, v_cache, k_new, v_new = (torch.randn(s, generator=g).to(dt) for s in
                                      ((pages, page, Hkv, D),) * 2 + ((total, Hkv, D),) * 2)
    slots = torch.randperm(pages * page, generator=g)[:total].to(torch.int32)
    if total > 2:
        slots[[1, total - 1]] = -1
    k, v = k_cache.cuda(), v_cache.cuda()
    mxa.write_cache(k_new.cuda(), v_new.cuda(), k, v, slots.cuda())
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            k_cache.view(-1, Hkv, D)[s] = k_new[t]
            v_cache.view(-1, Hkv, D)[s] = v_new[t]
    assert torch.equal(k.cpu().view(torch.int16), k_cache.view(torch.int16))
    assert torch.equal(v.cpu().view(torch.int16), v_cache.view(torch.int16))


def test_write_takes_slices_of_a_fused_projection():
    Hq, Hkv, D, total = 4, 2, 64, 50
    fused = torch.randn(total, (Hq + 2 * Hkv) * D, device="cuda").bfloat16()
    k_new = fused[:, Hq * D:(Hq + Hkv) * D].view(total, Hkv, D)
    v_new = fused[:, (Hq + Hkv) * D:].view(total, Hkv, D)
    k, v = (torch.zeros(8, 16, Hkv, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slots = torch.randperm(128, device="cuda")[:total].int()
    mxa.write_cache(k_new, v_new, k, v, slots)
    assert torch.equal(k.view(-1, Hkv, D)[slots.long()], k_new) and torch.equal(v.view(-1, Hkv, D)[slots.long()], v_new)


def test_write_skips_and_reports_slots_outside_the_pool():
    k, v = (torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    new = torch.ones(4, 2, 64, device="cuda", dtype=torch.float16)
    mxa.write_cache(new, new, k, v, ints([3, -2, 64, 2**31 - 1]))
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_ERR_INVALID_ARG
    want = torch.zeros_like(k)
    want.view(-1, 2, 64)[3] = 1
    assert torch.equal(k, want) and torch.equal(v, want)


def test_argument_checks():
    k = torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.float16)
    new = torch.ones(4, 2, 64, device="cuda", dtype=torch.float16)
    slots = ints([0, 1, 2, 3])
    for bad in ((new.bfloat16(), new, k, k, slots), (new.float(), new.float(), k.float(), k.float(), slots)):
        with pytest.raises(TypeError):
            mxa.write_cache(*bad)
    for bad in ((new, new[:3], k, k, slots), (new, new.transpose(0, 1), k, k, slots), (new, new, k, k[:2], slots),
                (new, new, k, k, slots[:3]), (new, new, k.cpu(), k.cpu(), slots), (new, new.transpose(1, 2).contiguous().transpose(1, 2), k, k, slots)):
        with pytest.raises(ValueError):
            mxa.write_cache(*bad)
    table, lens = torch.zeros(2, 3, device="cuda", dtype=torch.int32), ints([0, 0])
    args = dict(page_size=16, num_pages=4, total_q=2)
    for bad in ((table.t(), lens, ints([0, 1, 2]), ints([0])), (table, ints([0]), ints([0, 1, 2]), ints([0])),
                (table, lens, ints([0, 1]), ints([0])), (table, lens, ints([0, 1, 2]), ints([0]).cpu())):
        with pytest.raises(ValueError):
            mxa.extend_tables(*bad, **args)
    with pytest.raises(ValueError):
        mxa.extend_tables(table, lens, ints([0, 1, 2]), ints([0]), new_seqlens=lens, **args)
    with pytest.raises(TypeError):
        mxa.extend_tables(table.long(), lens, ints([0, 1, 2]), ints([0]), **args)
