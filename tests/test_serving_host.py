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
