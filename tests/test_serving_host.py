"""The paged-serving entry points on the host: plans and workspace sizes, and
the refusal of bad arguments before anything is launched."""
import ctypes

import pytest

from decode_attention_packed_b200 import mxa
from decode_attention_packed_b200.mxa import MXA_ERR_INVALID_ARG, MXA_ERR_UNSUPPORTED, MXA_ERR_WORKSPACE, MXA_OK

FAKE = ctypes.c_void_p(4096)  # never dereferenced: every call below is refused first
ODD = ctypes.c_void_p(4098)


def params(**kw):
    base = dict(B=4, q_len=1, Hq=32, Hkv=8, D=128, num_pages=512, page_size=16, max_pages_per_seq=1024,
                max_seqlen_k=16384, dtype=mxa.MXA_BF16)
    base.update(kw)
    return mxa.mxa_decode_params_t(*[base[f] for f, _ in mxa.mxa_decode_params_t._fields_])


def test_window_plan_is_sized_by_the_keys_a_window_leaves():
    p = params(B=1, Hq=8)
    full, windowed = mxa.mxa_plan(p, 0, sm_count=148), mxa.mxa_plan_window(p, 512, 4, sm_count=148)
    # 8 units of 256 blocks fill the wave; a window of 512 keys leaves
    # (512 + 0 + 4 + 3 * 64) / 64 = 12 blocks (rounded up), pieces of 2
    assert full.grid == 296 and windowed.grid == 8 * 12 // 2
    # a window as long as the rows plans like none
    assert mxa.mxa_plan_window(p, 16384, 0, sm_count=148).as_dict() == full.as_dict()
    assert mxa.mxa_plan_window(p, 2**31 - 1, 2**31 - 1, sm_count=148).as_dict() == full.as_dict()
    assert mxa.mxa_plan_window(p, 512, 4, num_splits=3, sm_count=148).num_splits == 3


@pytest.mark.parametrize("window,sinks", [(0, 0), (-1, 0), (5, -1)])
def test_window_refusals(window, sinks):
    plan = mxa.mxa_plan_t()
    p = params()
    assert mxa._lib.mxa_plan_window(ctypes.byref(p), window, sinks, 0, 148, ctypes.byref(plan)) == MXA_ERR_INVALID_ARG
    good = mxa.mxa_plan(p, 1, sm_count=148)
    call = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE, ctypes.byref(p), 1.0, window, sinks, ctypes.byref(good), None, 0,
            FAKE, None, None]
    assert mxa._lib.mxa_decode_fwd_window(*call) == MXA_ERR_INVALID_ARG


@pytest.mark.parametrize("at,value,code", [
    (0, None, MXA_ERR_INVALID_ARG), (1, None, MXA_ERR_INVALID_ARG), (2, ODD, MXA_ERR_INVALID_ARG),
    (3, FAKE, MXA_ERR_INVALID_ARG),   # new keys without new values
    (4, FAKE, MXA_ERR_INVALID_ARG),   # and the other way round
    (6, None, MXA_ERR_INVALID_ARG), (14, None, MXA_ERR_INVALID_ARG), (11, None, MXA_ERR_INVALID_ARG),
    (8, float("nan"), MXA_ERR_INVALID_ARG),
    (12, None, MXA_ERR_WORKSPACE),    # the plan splits
])
def test_window_decode_refusals(at, value, code):
    p = params()
    plan = mxa.mxa_plan_window(p, 512, 4, sm_count=148)
    assert plan.workspace_bytes > 0
    call = [FAKE, FAKE, FAKE, None, None, FAKE, FAKE, ctypes.byref(p), 1.0, 512, 4, ctypes.byref(plan), FAKE,
            plan.workspace_bytes, FAKE, None, None]
    call[at] = value
    assert mxa._lib.mxa_decode_fwd_window(*call) == code


@pytest.mark.parametrize("at,value,code", [
    (0, None, MXA_ERR_INVALID_ARG), (1, None, MXA_ERR_INVALID_ARG), (2, None, MXA_ERR_INVALID_ARG),
    (3, None, MXA_ERR_INVALID_ARG), (4, -1, MXA_ERR_INVALID_ARG), (4, 0, MXA_ERR_INVALID_ARG),
    (5, -1, MXA_ERR_INVALID_ARG), (6, -1, MXA_ERR_INVALID_ARG), (7, 0, MXA_ERR_INVALID_ARG),
    (8, 0, MXA_ERR_INVALID_ARG), (9, 0, MXA_ERR_INVALID_ARG), (10, None, MXA_ERR_INVALID_ARG),
    (11, None, MXA_ERR_INVALID_ARG), (12, None, MXA_ERR_INVALID_ARG), (10, ODD, MXA_ERR_INVALID_ARG),
    (11, ctypes.c_void_p(8192), MXA_ERR_INVALID_ARG),  # the old lengths' own buffer
    (8, 2**28, MXA_ERR_UNSUPPORTED), (9, 2**28, MXA_ERR_UNSUPPORTED),
])
def test_extend_tables_refusals(at, value, code):
    call = [FAKE, ctypes.c_void_p(8192), FAKE, FAKE, 4, 9, 5, 16, 64, 8, FAKE, FAKE, FAKE, None]
    call[at] = value
    if at == 10 and value is ODD:
        call[at] = ctypes.c_void_p(4097)
    assert mxa._lib.mxa_extend_tables(*call) == code


@pytest.mark.parametrize("at,value,code", [
    (0, None, MXA_ERR_INVALID_ARG), (1, ODD, MXA_ERR_INVALID_ARG), (2, 1016, MXA_ERR_INVALID_ARG),
    (3, 1028, MXA_ERR_UNSUPPORTED), (4, None, MXA_ERR_INVALID_ARG), (5, -1, MXA_ERR_INVALID_ARG),
    (6, 0, MXA_ERR_INVALID_ARG), (7, 0, MXA_ERR_INVALID_ARG), (8, 0, MXA_ERR_INVALID_ARG), (9, 0, MXA_ERR_INVALID_ARG),
    (10, 5, MXA_ERR_INVALID_ARG), (11, None, MXA_ERR_INVALID_ARG), (12, None, MXA_ERR_INVALID_ARG),
    (8, 2**28, MXA_ERR_UNSUPPORTED),
])
def test_cache_write_refusals(at, value, code):
    call = [FAKE, FAKE, 1024, 1024, FAKE, 3, 8, 128, 64, 16, mxa.MXA_BF16, FAKE, FAKE, None]
    call[at] = value
    assert mxa._lib.mxa_cache_write(*call) == code


def test_cache_write_wants_16_byte_tokens_and_takes_none():
    call = [FAKE, FAKE, 12, 12, FAKE, 3, 3, 4, 64, 16, mxa.MXA_BF16, FAKE, FAKE, None]
    assert mxa._lib.mxa_cache_write(*call) == MXA_ERR_UNSUPPORTED
    call = [None, None, 1024, 1024, None, 0, 8, 128, 64, 16, mxa.MXA_BF16, None, None, None]
    assert mxa._lib.mxa_cache_write(*call) == MXA_OK  # no token: nothing to do


PREFILL = ["q", "cu", "total_q", "k", "v", "table", "lens", "params", "scale", "causal", "window", "sinks", "ws", "ws_bytes",
           "out", "lse", "stream"]


def prefill_status(p, **kw):
    call = dict(q=FAKE, cu=FAKE, total_q=9, k=FAKE, v=FAKE, table=FAKE, lens=FAKE, params=ctypes.byref(p), scale=1.0,
                causal=1, window=0, sinks=0, ws=FAKE, ws_bytes=1 << 40, out=FAKE, lse=None, stream=None)
    call.update(kw)
    return mxa._lib.mxa_prefill_fwd(*[call[n] for n in PREFILL])


@pytest.mark.parametrize("shape,code", [
    (dict(B=-1), MXA_ERR_INVALID_ARG), (dict(q_len=0), MXA_ERR_INVALID_ARG), (dict(Hq=0), MXA_ERR_INVALID_ARG),
    (dict(Hq=30), MXA_ERR_INVALID_ARG), (dict(dtype=2), MXA_ERR_INVALID_ARG), (dict(page_size=0), MXA_ERR_INVALID_ARG),
    (dict(num_pages=0), MXA_ERR_INVALID_ARG), (dict(max_seqlen_k=-1), MXA_ERR_INVALID_ARG), (dict(B=0), MXA_ERR_INVALID_ARG),
    (dict(D=96), MXA_ERR_UNSUPPORTED), (dict(Hq=129, Hkv=1), MXA_ERR_UNSUPPORTED), (dict(B=12289), MXA_ERR_UNSUPPORTED),
    (dict(num_pages=2**28), MXA_ERR_UNSUPPORTED), (dict(max_seqlen_k=2**30), MXA_ERR_UNSUPPORTED),
])
def test_prefill_shape_refusals(shape, code):
    p = params(**shape)
    assert prefill_status(p) == code
    assert mxa.mxa_prefill_workspace_size(p, 9) == mxa.SIZE_MAX


@pytest.mark.parametrize("kw,code", [
    (dict(total_q=-1), MXA_ERR_INVALID_ARG), (dict(total_q=2**27), MXA_ERR_UNSUPPORTED),
    (dict(causal=2), MXA_ERR_INVALID_ARG), (dict(window=-1), MXA_ERR_INVALID_ARG), (dict(sinks=-1), MXA_ERR_INVALID_ARG),
    (dict(causal=0, window=5), MXA_ERR_INVALID_ARG), (dict(sinks=4), MXA_ERR_INVALID_ARG),
    (dict(scale=float("nan")), MXA_ERR_INVALID_ARG), (dict(scale=float("inf")), MXA_ERR_INVALID_ARG),
    (dict(table=None), MXA_ERR_INVALID_ARG),  # a contiguous cache has a row per request
    (dict(q=None), MXA_ERR_INVALID_ARG), (dict(cu=None), MXA_ERR_INVALID_ARG), (dict(k=None), MXA_ERR_INVALID_ARG),
    (dict(v=None), MXA_ERR_INVALID_ARG), (dict(lens=None), MXA_ERR_INVALID_ARG), (dict(out=None), MXA_ERR_INVALID_ARG),
    (dict(q=ODD), MXA_ERR_INVALID_ARG), (dict(k=ODD), MXA_ERR_INVALID_ARG), (dict(v=ODD), MXA_ERR_INVALID_ARG),
    (dict(out=ODD), MXA_ERR_INVALID_ARG), (dict(cu=ODD), MXA_ERR_INVALID_ARG), (dict(lens=ODD), MXA_ERR_INVALID_ARG),
    (dict(table=ODD), MXA_ERR_INVALID_ARG), (dict(lse=ODD), MXA_ERR_INVALID_ARG),
])
def test_prefill_call_refusals(kw, code):
    assert prefill_status(params(), **kw) == code


def test_prefill_layout_refusals():
    assert prefill_status(params(page_size=12, max_seqlen_k=12000)) == MXA_ERR_UNSUPPORTED
    assert prefill_status(params(max_pages_per_seq=1023)) == MXA_ERR_INVALID_ARG
    assert prefill_status(params(num_pages=4, page_size=16383), table=None) == MXA_ERR_INVALID_ARG
    # 2^17 tokens over 2^20 keys on 64 KV heads: more work than is laid out
    big = params(B=1, q_len=2**17, Hq=64 * 128, Hkv=64, page_size=1024, max_seqlen_k=2**20)
    assert prefill_status(big, total_q=2**17) == MXA_ERR_UNSUPPORTED


def test_prefill_without_tokens_is_nothing_to_do():
    assert prefill_status(params(), total_q=0, q=None, cu=None, k=None, v=None, lens=None, out=None, ws=None) == MXA_OK
    assert prefill_status(params(B=0), total_q=0) == MXA_OK
