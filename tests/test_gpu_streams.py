"""Calls on a stream of their own, named by hand: the tensors that the binding
makes are neither handed out again while the call still runs nor taken from
memory that work on the current stream still writes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa

BUSY = 50_000_000  # cycles, some 25 ms: longer than what the host does meanwhile


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(scope="module")
def problem():
    B, Hq, Hkv, D, page, width = 4, 8, 2, 128, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(2200)
    k, v = (torch.randn(B * width, page, Hkv, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, 1, Hq, D, generator=gen, device="cuda").bfloat16()
    table = torch.randperm(B * width, generator=gen, device="cuda").int().view(B, width)
    lens, cu = torch.tensor([2000, 1, 700, 2000]).int().cuda(), torch.arange(B + 1).int().cuda()
    free = torch.arange(64, dtype=torch.int32, device="cuda")
    packed, held, extended = q.view(B, Hq, D), lens - 1, table.clone()
    return {
        "decode": lambda **kw: mxa.decode(q, k, v, table, lens, **kw),
        "float32": lambda **kw: mxa.decode(q, k, v, table, lens, out_dtype=torch.float32, **kw),
        "window": lambda **kw: mxa.decode(q, k, v, table, lens, causal=True, window=600, sinks=4, **kw),
        "varlen": lambda **kw: mxa.decode_varlen(packed, cu, k, v, table, lens, max_seqlen_q=1, **kw),
        "prefill": lambda **kw: mxa.prefill(packed, cu, k, v, table, lens, max_seqlen_q=1, **kw),
        # a table of its own, where every call writes the same page again
        "tables": lambda **kw: mxa.extend_tables(extended, held, cu, free, page_size=page, num_pages=B * width,
                                                 total_q=B, **kw)[::2],
    }


NAMES = ["decode", "float32", "window", "varlen", "prefill", "tables"]


def bits(results):
    return [t.clone().view(torch.uint8) for t in results]


def stream_forms():
    s = torch.cuda.Stream()
    return [s, s.cuda_stream]


@pytest.mark.parametrize("which", NAMES)
@pytest.mark.parametrize("form", [0, 1])
def test_dropped_results_are_not_handed_out_while_the_call_runs(problem, which, form):
    call, s = problem[which], stream_forms()
    want = bits(call())
    torch.cuda.synchronize()
    with torch.cuda.stream(s[0]):
        torch.cuda._sleep(BUSY)
    results = call(stream=s[form])
    kept, size = results[0], results[1].numel() * results[1].element_size()
    del results  # the second result (and the workspace) dropped before the call has begun
    mine = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (size, size, 1 << 20, 4 << 20, 32 << 20) * 2]
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert all(bool((t == 7).all()) for t in mine)
    assert torch.equal(kept.view(torch.uint8), want[0])


@pytest.mark.parametrize("which", NAMES)
def test_results_lie_apart_from_what_the_current_stream_still_writes(problem, which):
    call, s = problem[which], torch.cuda.Stream()
    want = bits(call())
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for _ in range(2):  # freed on the current stream at once, written there later
        junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in (64, 512, 1024, 16384, 1 << 20, 4 << 20)]
        del junk
    results = call(stream=s)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert all(torch.equal(a, b) for a, b in zip(bits(results), want))


@pytest.mark.parametrize("which", NAMES)
def test_the_default_stream_by_its_handle(problem, which):
    want = bits(problem[which]())
    got = bits(problem[which](stream=0))
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("which", ["decode", "window", "varlen", "prefill"])
def test_a_side_stream_inside_a_capture(problem, which):
    call, s = problem[which], torch.cuda.Stream()
    want = bits(call())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        results = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        copies = [t.clone() for t in results]
        del results
    for _ in range(2):
        for t in copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bits(copies), want))
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
