"""Pins of the oracle's sliding window and of its table arithmetic: closed
forms, special cases and a brute force that shares nothing with them."""
import math

import numpy as np
import pytest
import torch

import oracle
from decode_attention_packed_b200.workloads import Workload, make_inputs
from tests.brute import brute_attention


def draw(lengths, q_len=1, Hq=4, Hkv=2, D=8, page_size=4, seed=5):
    return make_inputs(Workload(name="window_pin", B=len(lengths), q_len=q_len, Hq=Hq, Hkv=Hkv, D=D, dtype="bf16",
                                page_size=page_size, causal=True, lengths="list:" + ",".join(map(str, lengths)), seed=seed))


def run(inp, window, sinks, scale=None):
    w = inp.w
    return oracle.decode(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens, Hkv=w.Hkv,
                         page_size=inp.page_size, dtype=w.dtype, scale=w.scale if scale is None else scale, causal=True,
                         window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (4, 0), (5, 2), (7, 20), (100, 0)])
def test_visible_keys_are_counted_by_the_lse_at_scale_zero(window, sinks):
    # with scale 0 every visible key weighs the same: LSE = ln(visible keys)
    lengths, q_len = [1, 3, 9, 26], 3
    inp = draw(lengths, q_len)
    _, lse = run(inp, window, sinks, scale=0.0)
    for b, L in enumerate(lengths):
        for t in range(q_len):
            p = L - q_len + t
            n = sum(1 for j in range(max(0, p + 1)) if j > p - window or j < sinks)
            want = math.log(n) if n else -math.inf
            assert np.allclose(lse[b, :, t], want, atol=1e-12) if n else np.isneginf(lse[b, :, t]).all()


def test_a_window_over_everything_is_causal_attention():
    inp = draw([1, 7, 30], 2)
    w = inp.w
    ref = brute_attention(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.cache_seqlens.numpy(), Hkv=w.Hkv,
                          page_size=inp.page_size, scale=w.scale, causal=True)
    for window, sinks in ((30, 0), (1, 30), (29, 1)):
        out, lse = run(inp, window, sinks)
        assert np.allclose(out, ref[0], atol=1e-10) and np.allclose(lse, ref[1], atol=1e-10)


def test_a_window_is_attention_over_the_kept_keys():
    # one query: its window and sinks, gathered into a cache of their own
    inp = draw([29], 1)
    w, window, sinks = inp.w, 6, 3
    out, lse = run(inp, window, sinks)
    kept = list(range(sinks)) + list(range(29 - window, 29))
    at = [int(inp.block_table[0, j // 4]) * 4 + j % 4 for j in kept]
    k, v = (c.reshape(-1, w.Hkv, w.D)[at].unsqueeze(0) for c in (inp.k_cache, inp.v_cache))
    ref = brute_attention(inp.q, k, v, None, np.array([len(kept)]), Hkv=w.Hkv, page_size=len(kept), scale=w.scale,
                          causal=False)
    assert np.allclose(out, ref[0], atol=1e-10) and np.allclose(lse, ref[1], atol=1e-10)


def test_hidden_values_do_not_matter():
    inp = draw([29], 1)
    out, _ = run(inp, 6, 3)
    for j in range(3, 23):
        page, slot = int(inp.block_table[0, j // 4]), j % 4
        inp.k_cache[page, slot] = float("nan")
        inp.v_cache[page, slot] = float("inf")
    again, _ = run(inp, 6, 3)
    assert np.array_equal(out, again)


def test_tables_by_hand():
    # pages of 4; row 0 holds 3 keys and gets 2 (one page more), row 1 holds
    # none and gets 5 (two pages), row 2 holds 4 and gets none
    table = np.array([[9, -1, -1], [-1, -1, -1], [7, -1, -1]])
    bt, slots, new, used = oracle.extend_tables(table, [3, 0, 4], [0, 2, 7, 7], [5, 6, 8, 2], page_size=4, num_pages=10)
    assert bt.tolist() == [[9, 5, -1], [6, 8, -1], [7, -1, -1]]
    assert slots.tolist() == [9 * 4 + 3, 5 * 4, 6 * 4, 6 * 4 + 1, 6 * 4 + 2, 6 * 4 + 3, 8 * 4]
    assert new.tolist() == [5, 5, 4] and used == 3


def test_tables_when_the_pages_run_out():
    # row 0 takes the one free page; row 1 wants one and gets none; row 2 fits
    # the page it holds; row 3 wants more pages than its table has columns
    table = np.array([[-1, -1], [0, -1], [1, -1], [2, -1]])
    bt, slots, new, used = oracle.extend_tables(table, [0, 4, 2, 1], [0, 1, 2, 3, 12], [3], page_size=4, num_pages=4)
    assert bt.tolist() == [[3, -1], [0, -1], [1, -1], [2, -1]]
    assert slots.tolist() == [12, -1, 4 + 2] + [-1] * 9
    assert new.tolist() == [1, 4, 3, 1] and used == 1
