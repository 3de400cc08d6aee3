"""The first call of a process made under stream capture: each entry point's
kernels are loaded, and its graph replayed, without a call before it."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

SCRIPT = """
import torch
from decode_attention_packed_b200 import mxa
d = "cuda"
B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
k, v = (torch.zeros(8, page, Hkv, D, dtype=torch.float16, device=d) for _ in range(2))
table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=d)
lens, cu = torch.tensor([20, 9], dtype=torch.int32, device=d), torch.tensor([0, 1, 2], dtype=torch.int32, device=d)
free, q = torch.arange(4, 8, dtype=torch.int32, device=d), torch.ones(B, Hq, D, dtype=torch.float16, device=d)
new = torch.ones(B, Hkv, D, dtype=torch.float16, device=d)
out = torch.empty_like(q)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    which = "%s"
    if which == "tables":
        slots, new_lens, used = mxa.extend_tables(table, lens, cu, free, page_size=page, num_pages=8, total_q=2)
    elif which == "write":
        mxa.write_cache(new, new, k, v, torch.zeros(2, dtype=torch.int32, device=d).copy_(cu[:2]))
    elif which == "prefill":
        mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=1, out=out)
    else:
        mxa.decode(q.view(B, 1, Hq, D), k, v, table, lens, causal=True, window=8, sinks=2, out=out.view(B, 1, Hq, D))
g.replay()
torch.cuda.synchronize()
assert mxa.mxa_device_error(True) == mxa.MXA_OK
if which == "tables":
    assert slots.tolist() == [1 * 16 + 4, 2 * 16 + 9] and new_lens.tolist() == [21, 10] and used.tolist() == [0]
elif which == "write":
    assert bool((k.view(-1, Hkv, D)[:2] == 1).all())
else:
    assert bool((out == 0).all())
"""


@pytest.mark.parametrize("which", ["tables", "write", "prefill", "window"])
def test_first_call_under_capture(which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", SCRIPT % which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
