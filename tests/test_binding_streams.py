"""Where the binding's own tensors come from when a call names its stream: the
pool of that stream, lent to the current one.  On the CPU, with the library's
entry points and torch's streams replaced by records of their use; the same
calls on a GPU are in test_gpu_streams.py."""
import contextlib

import pytest
import torch

from decode_attention_packed_b200 import mxa


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Record:
    """Tensors made, the stream whose pool each came from, and those lent to the current stream."""

    def __init__(self, monkeypatch):
        self.made, self.lent, self.inside = [], [], [None]

        def recording(make):
            def made(*args, **kw):
                t = make(*args, **kw)
                if kw.get("device") != "meta":
                    self.made.append((t, self.inside[-1]))
                return t
            return made

        @contextlib.contextmanager
        def stream(s):
            self.inside.append(s.cuda_stream)
            yield
            self.inside.pop()

        for where, name in ((mxa.torch, "empty"), (mxa.torch, "empty_like"), (mxa.torch.Tensor, "new_empty")):
            monkeypatch.setattr(where, name, recording(getattr(where, name)))
        monkeypatch.setattr(mxa.torch.cuda, "Stream", FakeStream)
        monkeypatch.setattr(mxa.torch.cuda, "ExternalStream", FakeStream)
        monkeypatch.setattr(mxa.torch.cuda, "default_stream", lambda: FakeStream(0))
        monkeypatch.setattr(mxa.torch.cuda, "current_stream", lambda: FakeStream(5000))
        monkeypatch.setattr(mxa.torch.cuda, "stream", stream)
        monkeypatch.setattr(mxa.torch.Tensor, "record_stream", lambda t, s: self.lent.append((t, s.cuda_stream)))
        monkeypatch.setattr(mxa, "_current_device", lambda: -1)  # where host tensors say they are
        monkeypatch.setattr(mxa, "_raw_stream", lambda device: 5000)
        plan, plan_window = mxa.mxa_plan, mxa.mxa_plan_window
        monkeypatch.setattr(mxa, "mxa_plan", lambda p, splits=0: plan(p, splits, 148))
        monkeypatch.setattr(mxa, "mxa_plan_window", lambda p, w, s, splits=0: plan_window(p, w, s, splits, 148))
        self.streams = []
        for name in ("mxa_decode_fwd_with_plan", "mxa_decode_fwd_window", "mxa_decode_fwd_f32out", "mxa_decode_fwd_varlen",
                     "mxa_prefill_fwd", "mxa_extend_tables"):
            monkeypatch.setattr(mxa._lib, name, lambda *args: self.streams.append(args[-1]) or mxa.MXA_OK)
        monkeypatch.setattr(mxa._lib, "mxa_prefill_workspace_size", lambda *args: 4096)


def calls():
    B, Hq, Hkv, D, page, width = 3, 8, 2, 64, 16, 64
    q = torch.zeros(B, 1, Hq, D, dtype=torch.float16)
    k, v = (torch.zeros(B * width, page, Hkv, D, dtype=torch.float16) for _ in range(2))
    table = torch.arange(B * width, dtype=torch.int32).view(B, width)
    lens, cu = torch.full((B,), 500, dtype=torch.int32), torch.arange(B + 1, dtype=torch.int32)
    packed, free = q.view(B, Hq, D), torch.arange(9, dtype=torch.int32)
    return {  # what is called, and the tensors it makes: results, and a workspace where there is one
        "decode": (lambda **kw: mxa.decode(q, k, v, table, lens, **kw), 3),
        "float32": (lambda **kw: mxa.decode(q, k, v, table, lens, out_dtype=torch.float32, **kw), 3),
        "window": (lambda **kw: mxa.decode(q, k, v, table, lens, causal=True, window=256, **kw), 3),
        "varlen": (lambda **kw: mxa.decode_varlen(packed, cu, k, v, table, lens, max_seqlen_q=1, **kw), 3),
        "prefill": (lambda **kw: mxa.prefill(packed, cu, k, v, table, lens, max_seqlen_q=1, **kw), 3),
        "tables": (lambda **kw: mxa.extend_tables(table, lens, cu, free, page_size=page, num_pages=B * width, total_q=B, **kw), 3),
        "prepare": (lambda **kw: mxa.prepare(q, k, table, **kw).workspace, 1),
        "prepare_prefill": (lambda **kw: mxa.prepare_prefill(packed, cu, k, table, max_seqlen_q=1, **kw).workspace, 1),
    }


@pytest.mark.parametrize("stream,handle", [(FakeStream(7000), 7000), (7000, 7000), (0, 0), (1, 0), (None, None)])
@pytest.mark.parametrize("which", sorted(calls()))
def test_tensors_come_from_the_calls_stream(monkeypatch, which, stream, handle):
    call, count = calls()[which]
    record = Record(monkeypatch)
    call(stream=stream)
    assert [at for _, at in record.made] == [handle] * count
    # each of them is lent to the current stream, where the caller reads and drops it
    assert [id(t) for t, _ in record.lent] == ([] if stream is None else [id(t) for t, _ in record.made])
    assert all(s == 5000 for _, s in record.lent)
    want = 5000 if stream is None else getattr(stream, "cuda_stream", stream)
    assert record.streams == [] if which.startswith("prepare") else record.streams == [want]


def test_the_callers_tensors_are_left_alone(monkeypatch):
    record = Record(monkeypatch)
    q = torch.zeros(2, 8, 64, dtype=torch.float16)
    k, v = (torch.zeros(4, 16, 2, 64, dtype=torch.float16) for _ in range(2))
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.full((2,), 9, dtype=torch.int32)
    cu = torch.arange(3, dtype=torch.int32)
    out, lse = torch.zeros_like(q), torch.zeros(8, 2)
    got = mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=1, out=out, lse=lse, stream=7000)
    assert got[0] is out and got[1] is lse
    assert len(record.made) == 1 and all(t is not out and t is not lse for t, _ in record.lent)


@pytest.mark.parametrize("stream", [FakeStream(5000), 5000])
@pytest.mark.parametrize("which", sorted(calls()))
def test_the_current_stream_by_name_is_none_at_all(monkeypatch, which, stream):
    # no other stream is entered and nothing lent: the call's host time is that without stream=
    call, count = calls()[which]
    record = Record(monkeypatch)
    call(stream=stream)
    assert [at for _, at in record.made] == [None] * count and record.lent == []
    assert record.streams == [] if which.startswith("prepare") else record.streams == [5000]
