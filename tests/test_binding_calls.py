"""What the binding hands to the library, and what it refuses before it: on the
CPU, with the library's run entry points replaced by a record of their
arguments and host tensors in the place of the device's."""
import ctypes

import pytest
import torch

from decode_attention_packed_b200 import mxa

RUNS = ("mxa_decode_fwd_with_plan", "mxa_decode_fwd_window", "mxa_decode_fwd_f32out", "mxa_decode_fwd_varlen",
        "mxa_decode_fwd_append", "mxa_prefill_fwd", "mxa_extend_tables", "mxa_cache_write")
B, HQ, HKV, D, PAGE, WIDTH = 3, 8, 2, 64, 16, 64


@pytest.fixture
def ran(monkeypatch):
    """The run calls so far: (entry point, its arguments, its params or None)."""
    calls = []
    monkeypatch.setattr(mxa, "_current_device", lambda: -1)  # where host tensors say they are
    monkeypatch.setattr(mxa, "_raw_stream", lambda device: 0)
    plan, plan_window = mxa.mxa_plan, mxa.mxa_plan_window
    monkeypatch.setattr(mxa, "mxa_plan", lambda p, splits=0: plan(p, splits, 148))
    monkeypatch.setattr(mxa, "mxa_plan_window", lambda p, w, s, splits=0: plan_window(p, w, s, splits, 148))
    monkeypatch.setattr(mxa._lib, "mxa_prefill_workspace_size", lambda *args: 4096)

    def entry(name):
        def run(*args):
            p = [a._obj for a in args if isinstance(getattr(a, "_obj", None), mxa.mxa_decode_params_t)]
            shape = mxa.mxa_decode_params_t.from_buffer_copy(p[0]) if p else None
            calls.append((name, args, shape))
            return mxa.MXA_OK
        return run

    for name in RUNS:
        monkeypatch.setattr(mxa._lib, name, entry(name))
    return calls


def tensors(q_tokens=B):
    return dict(q=torch.zeros(q_tokens, HQ, D, dtype=torch.float16),
                k=torch.zeros(B * WIDTH, PAGE, HKV, D, dtype=torch.float16),
                v=torch.zeros(B * WIDTH, PAGE, HKV, D, dtype=torch.float16),
                table=torch.arange(B * WIDTH, dtype=torch.int32).view(B, WIDTH),
                lens=torch.full((B,), 500, dtype=torch.int32), cu=torch.arange(B + 1, dtype=torch.int32))


def bounds_call(which, t, prepared_q, prepared_k):
    """A call of `which` whose preparation had the given bounds, and that takes its own as keywords."""
    row_q = t["q"].view(B, 1, HQ, D)
    if which == "prefill":
        prep = mxa.prepare_prefill(t["q"], t["cu"], t["k"], t["table"], max_seqlen_q=prepared_q, max_seqlen_k=prepared_k)
        return lambda **kw: mxa.prefill(t["q"], t["cu"], t["k"], t["v"], t["table"], t["lens"], prepared=prep, **kw)
    if which == "varlen":
        wide = torch.empty(B, prepared_q, HQ, D, dtype=torch.float16, device="meta")
        prep = mxa.prepare(wide, t["k"], t["table"], max_seqlen_k=prepared_k, device="cpu")
        return lambda **kw: mxa.decode_varlen(t["q"], t["cu"], t["k"], t["v"], t["table"], t["lens"], prepared=prep, **kw)
    more = dict(window=dict(window=256), float32=dict(out_dtype=torch.float32),
                append=dict(k_new=torch.zeros(B, 1, HKV, D, dtype=torch.float16), v_new=torch.zeros(B, 1, HKV, D, dtype=torch.float16)),
                decode={})[which]
    prep = mxa.prepare(row_q, t["k"], t["table"], max_seqlen_k=prepared_k, window=more.get("window", 0))
    return lambda **kw: mxa.decode(row_q, t["k"], t["v"], t["table"], t["lens"], causal=True, prepared=prep, **more, **kw)


@pytest.mark.parametrize("which", ["prefill", "varlen", "decode", "window", "float32", "append"])
def test_a_call_may_go_past_the_keys_it_was_prepared_for(ran, which):
    call = bounds_call(which, tensors(), 4, 128)
    q = dict(max_seqlen_q=4) if which in ("prefill", "varlen") else {}
    for stated, want in ((None, 128), (64, 128), (128, 128), (700, 700), (1 << 20, WIDTH * PAGE)):
        call(max_seqlen_k=stated, **q)
        assert ran[-1][2].max_seqlen_k == want
    call(**q)
    assert ran[-1][2].max_seqlen_k == 128  # the preparation is as it was


@pytest.mark.parametrize("which", ["prefill", "varlen"])
def test_a_call_may_go_past_the_queries_it_was_prepared_for(ran, which):
    call = bounds_call(which, tensors(), 4, 128)
    for stated, want in ((1, 4), (4, 4), (200, 200), (4, 4)):
        call(max_seqlen_q=stated)
        assert (ran[-1][2].q_len, ran[-1][2].max_seqlen_k) == (want, 128)


def test_a_wider_call_is_checked_against_its_plan():
    # the library sizes the workspace anew from the widened shape
    p = mxa.mxa_decode_params_t(4, 1, 32, 8, 128, 512, 16, 1024, 4096, mxa.MXA_BF16)
    plan = mxa.mxa_plan(p, 0, 148)
    wide = mxa._widened(p, 16, None)
    assert (wide.q_len, p.q_len) == (16, 1)
    fake = ctypes.c_void_p(4096)  # not used: the call is refused first
    call = [fake, fake, 64, fake, fake, fake, fake, ctypes.byref(wide), 1.0, 0, ctypes.byref(plan), fake,
            plan.workspace_bytes, fake, None, None]
    assert mxa._lib.mxa_decode_fwd_varlen(*call) == mxa.MXA_ERR_WORKSPACE


def windowed(t, **kw):
    """A windowed decode on `t` with replacements `kw`, prepared for the shapes of tensors()."""
    good = tensors()
    prep = mxa.prepare(good["q"].view(B, 1, HQ, D), good["k"], good["table"], window=256)
    args = dict(t, **{n: kw.pop(n) for n in list(kw) if n in t})
    return mxa.decode(args["q"], args["k"], args["v"], args["table"], args["lens"], causal=True, window=256, prepared=prep, **kw)


def test_windowed_decode_takes_the_documented_tensors(ran):
    t = tensors()
    t["q"] = t["q"].view(B, 1, HQ, D)
    fresh = torch.zeros(B, 1, HKV, D, dtype=torch.float16)
    windowed(t)
    windowed(t, k_new=fresh, v_new=fresh)
    windowed(t, out=torch.zeros_like(t["q"]), lse=torch.zeros(B, HQ, 1))
    windowed(t, q=torch.zeros(4, B, 1, HQ, D, dtype=torch.float16)[2])  # a dense part of a larger tensor
    assert [c[0] for c in ran] == ["mxa_decode_fwd_window"] * 4


BAD = {
    "q of another type": (TypeError, lambda t: dict(q=t["q"].bfloat16())),
    "q strided": (ValueError, lambda t: dict(q=torch.zeros(B, 1, 2 * HQ, D, dtype=torch.float16)[:, :, ::2])),
    "q of more rows": (ValueError, lambda t: dict(q=torch.zeros(B + 1, 1, HQ, D, dtype=torch.float16))),
    "q of more tokens": (ValueError, lambda t: dict(q=torch.zeros(B, 2, HQ, D, dtype=torch.float16))),
    "another cache": (ValueError, lambda t: dict(k=t["k"][:-1], v=t["v"][:-1])),
    "a cache of another type": (TypeError, lambda t: dict(k=t["k"].bfloat16())),
    "values of another shape": (ValueError, lambda t: dict(v=t["v"][:-1])),
    "a strided cache": (ValueError, lambda t: dict(k=torch.zeros(B * WIDTH, PAGE, 2 * HKV, D, dtype=torch.float16)[:, :, :HKV])),
    "a table of another width": (ValueError, lambda t: dict(table=t["table"][:, :-1].contiguous())),
    "a strided table": (ValueError, lambda t: dict(table=t["table"].t().contiguous().t())),
    "a table of 64 bits": (TypeError, lambda t: dict(table=t["table"].long())),
    "lengths of 64 bits": (TypeError, lambda t: dict(lens=t["lens"].long())),
    "lengths of fewer rows": (ValueError, lambda t: dict(lens=t["lens"][:-1])),
    "new keys out of a fused projection": (ValueError, lambda t: dict(k_new=fused(), v_new=fused())),
    "new values out of a fused projection": (ValueError, lambda t: dict(k_new=fused().contiguous(), v_new=fused())),
    "new keys of another type": (TypeError, lambda t: dict(k_new=fused().bfloat16(), v_new=fused().contiguous())),
    "new keys of another shape": (ValueError, lambda t: dict(k_new=fused()[:1].contiguous(), v_new=fused().contiguous())),
    "new keys alone": (ValueError, lambda t: dict(k_new=fused().contiguous())),
    "out of another type": (TypeError, lambda t: dict(out=torch.zeros(B, 1, HQ, D, dtype=torch.bfloat16))),
    "out of another shape": (ValueError, lambda t: dict(out=torch.zeros(B, 1, HQ + 1, D, dtype=torch.float16))),
    "a strided out": (ValueError, lambda t: dict(out=torch.zeros(B, 1, 2 * HQ, D, dtype=torch.float16)[:, :, ::2])),
    "an lse of 16 bits": (TypeError, lambda t: dict(lse=torch.zeros(B, HQ, 1, dtype=torch.float16))),
    "an lse of another shape": (ValueError, lambda t: dict(lse=torch.zeros(B, HQ, 2))),
}


def fused():
    return torch.zeros(B, 1, (HQ + 2 * HKV) * D, dtype=torch.float16)[:, :, HQ * D:(HQ + HKV) * D].view(B, 1, HKV, D)


@pytest.mark.parametrize("what", sorted(BAD))
def test_windowed_decode_refuses(ran, what):
    error, change = BAD[what]
    t = tensors()
    t["q"] = t["q"].view(B, 1, HQ, D)
    with pytest.raises(error):
        windowed(t, **change(t))
    assert ran == []


def test_windowed_decode_refuses_another_device(ran, monkeypatch):
    t = tensors()
    t["q"] = t["q"].view(B, 1, HQ, D)
    monkeypatch.setattr(mxa, "_current_device", lambda: 0)
    with pytest.raises(ValueError):
        windowed(t)
    assert ran == []


def test_append_refuses_strided_tokens(ran):
    # read as dense they would be other tokens' values
    t = tensors()
    q = t["q"].view(B, 1, HQ, D)
    for k_new, v_new in ((fused(), fused()), (fused().contiguous(), fused()), (fused(), fused().contiguous())):
        with pytest.raises(ValueError):
            mxa.decode(q, t["k"], t["v"], t["table"], t["lens"], k_new=k_new, v_new=v_new)
    assert ran == []
    mxa.decode(q, t["k"], t["v"], t["table"], t["lens"], k_new=fused().contiguous(), v_new=fused().contiguous())
    assert [c[0] for c in ran] == ["mxa_decode_fwd_append"]


@pytest.mark.parametrize("given,want", [(2**31 - 1, 2**31 - 1), (2**31, 2**31 - 1), (2**32, 2**31 - 1), (2**32 + 5, 2**31 - 1),
                                        (2**63 - 1, 2**31 - 1), (7, 7)])
def test_windows_past_32_bits_hide_nothing(ran, given, want):
    # as many keys as no row has: not what 32 bits leave of the number
    t = tensors()
    q = t["q"].view(B, 1, HQ, D)
    mxa.decode(q, t["k"], t["v"], t["table"], t["lens"], causal=True, window=given, sinks=given)
    mxa.prefill(t["q"], t["cu"], t["k"], t["v"], t["table"], t["lens"], max_seqlen_q=1, window=given, sinks=given)
    assert ran[0][1][9:11] == (want, want) and ran[1][1][10:12] == (want, want)
    p = mxa.mxa_decode_params_t(B, 1, HQ, HKV, D, B * WIDTH, PAGE, WIDTH, WIDTH * PAGE, mxa.MXA_F16)
    assert mxa.mxa_plan_window(p, given, given).as_dict() == mxa.mxa_plan_window(p, want, want).as_dict()


@pytest.mark.parametrize("given", [-1, -2**31, -2**32 + 5])
def test_negative_windows_stay_negative(ran, given):
    t = tensors()
    q = t["q"].view(B, 1, HQ, D)
    for kw in (dict(window=given), dict(window=5, sinks=given)):
        with pytest.raises(ValueError):
            mxa.decode(q, t["k"], t["v"], t["table"], t["lens"], causal=True, **kw)
        mxa.prefill(t["q"], t["cu"], t["k"], t["v"], t["table"], t["lens"], max_seqlen_q=1, **kw)
        assert min(ran[-1][1][10:12]) == -1  # which the library refuses


def test_a_step_without_new_tokens(ran):
    # every row idle: the largest count is 0, with padding tokens or none
    t = tensors()
    for tokens in (0, 3):
        mxa.prefill(t["q"][:tokens], torch.zeros_like(t["cu"]), t["k"], t["v"], t["table"], t["lens"], max_seqlen_q=0)
        assert ran[-1][2].q_len == 1
    prep = mxa.prepare_prefill(t["q"], t["cu"], t["k"], t["table"], max_seqlen_q=0)
    mxa.prefill(t["q"], t["cu"], t["k"], t["v"], t["table"], t["lens"], max_seqlen_q=0, prepared=prep)
    assert ran[-1][2].q_len == 1
    shape = mxa.prepare_prefill(t["q"], t["cu"], t["k"], t["table"], max_seqlen_q=-1).params
    assert shape.q_len == -1  # which the library refuses


def test_a_step_without_rows():
    # an empty block table has no address
    p = mxa.mxa_decode_params_t(0, 1, HQ, HKV, D, B * WIDTH, PAGE, WIDTH, WIDTH * PAGE, mxa.MXA_F16)
    fake = ctypes.c_void_p(4096)  # not used: there is nothing to do
    for table in (None, fake):
        call = [fake, fake, 0, fake, fake, table, fake, ctypes.byref(p), 1.0, 1, 0, 0, None, 0, fake, None, None]
        assert mxa._lib.mxa_prefill_fwd(*call) == mxa.MXA_OK


@pytest.mark.parametrize("rows,width,code", [(2**15 + 1, 2**15, mxa.MXA_ERR_UNSUPPORTED), (2**16 - 1, 2**15, mxa.MXA_ERR_UNSUPPORTED),
                                             (2**15, 2**15, mxa.MXA_ERR_UNSUPPORTED), (2**15 - 1, 2**15, mxa.MXA_ERR_INVALID_ARG)])
def test_tables_stay_within_32_bits(rows, width, code):
    # The kernel walks the pages taken, up to rows * width of them, in strides
    # of its grid: with 2^31 - 1 pages the step past the last one would not fit
    # 32 bits.  (The one that is small enough fails for its missing pointers.)
    assert rows * width < 2**31
    fake = ctypes.c_void_p(4096)  # not used: the call is refused
    assert mxa._lib.mxa_extend_tables(None, fake, fake, fake, rows, 9, 5, 1, 64, width, fake, fake, fake, None) == code


def test_a_decode_without_rows():
    p = mxa.mxa_decode_params_t(0, 1, HQ, HKV, D, B * WIDTH, PAGE, WIDTH, WIDTH * PAGE, mxa.MXA_F16)
    plan = mxa.mxa_plan(p, 0, 148)
    fake = ctypes.c_void_p(4096)  # not used: there is nothing to do
    for table in (None, fake):
        plain = [None, fake, fake, table, None, ctypes.byref(p), 1.0, 1, ctypes.byref(plan), None, 0, None, None, None]
        assert mxa._lib.mxa_decode_fwd_with_plan(*plain) == mxa.MXA_OK
        window = [None, fake, fake, None, None, table, None, ctypes.byref(p), 1.0, 5, 0, ctypes.byref(plan), None, 0, None, None, None]
        assert mxa._lib.mxa_decode_fwd_window(*window) == mxa.MXA_OK
