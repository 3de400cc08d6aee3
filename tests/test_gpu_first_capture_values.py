"""The first call of a process made under stream capture, with outputs that
only its kernels can bring about: every buffer holds another value before, and
no result is zero."""
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

SCRIPT = """
import math
import torch
from decode_attention_packed_b200 import mxa
d, which = "cuda", "%s"
B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
k = torch.zeros(8, page, Hkv, D, dtype=torch.float16, device=d)  # every key weighs the same
v = torch.full_like(k, 3.0)
table = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=d)
lens, cu = torch.tensor([20, 9], dtype=torch.int32, device=d), torch.tensor([0, 1, 2], dtype=torch.int32, device=d)
free, q = torch.arange(4, 8, dtype=torch.int32, device=d), torch.ones(B, Hq, D, dtype=torch.float16, device=d)
k_new, v_new = torch.full((B, Hkv, D), 5.0, dtype=torch.float16, device=d), torch.full((B, Hkv, D), 6.0, dtype=torch.float16, device=d)
rows = (B, 1, Hq, D)
out, out32 = torch.full_like(q, 7.0), torch.full(rows, 7.0, device=d)
lse = torch.full((Hq, B), 7.0, device=d)           # packed: [Hq, total_q]
lse_rows = torch.full((B, Hq, 1), 7.0, device=d)
slots, new_lens, used = (torch.full((n,), -9, dtype=torch.int32, device=d) for n in (2, 2, 1))
where = torch.tensor([40, 3], dtype=torch.int32, device=d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    if which == "tables":
        mxa.extend_tables(table, lens, cu, free, page_size=page, num_pages=8, total_q=2, slots=slots, new_seqlens=new_lens,
                          pages_used=used)
    elif which == "write":
        mxa.write_cache(k_new, v_new, k, v, where)
    elif which == "prefill":
        mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=1, out=out, lse=lse)
    elif which == "varlen":
        mxa.decode_varlen(q, cu, k, v, table, lens, max_seqlen_q=1, out=out, lse=lse)
    elif which == "float32":
        mxa.decode(q.view(rows), k, v, table, lens, out=out32, lse=lse_rows)
    else:
        kw = dict(window=dict(causal=True, window=8, sinks=2), append=dict(k_new=k_new.view(B, 1, Hkv, D) * 0, v_new=v_new.view(B, 1, Hkv, D)),
                  decode={})[which]
        mxa.decode(q.view(rows), k, v, table, lens, out=out.view(rows), lse=lse_rows, **kw)
# captured, and nothing run
assert bool((out == 7).all()) and bool((out32 == 7).all()) and bool((lse == 7).all()) and bool((lse_rows == 7).all())
assert slots.tolist() == [-9, -9] and bool((k == 0).all())
g.replay()
torch.cuda.synchronize()
assert mxa.mxa_device_error(True) == mxa.MXA_OK
if which == "tables":
    assert slots.tolist() == [1 * 16 + 4, 2 * 16 + 9] and new_lens.tolist() == [21, 10] and used.tolist() == [0]
elif which == "write":
    for cache, new, old in ((k, 5.0, 0.0), (v, 6.0, 3.0)):
        flat = cache.view(-1, Hkv, D)
        assert bool((flat[[40, 3]] == new).all()) and int((flat != old).any(-1).any(-1).sum()) == 2
else:
    seen = dict(window=[10, 9], append=[21, 10]).get(which, [20, 9])
    # equal weights: the mean of the values, and the logarithm of their number
    mean = [(20 * 3 + 6) / 21, (9 * 3 + 6) / 10] if which == "append" else [3.0, 3.0]
    got = out32 if which == "float32" else out
    got_lse = lse.t() if which in ("prefill", "varlen") else lse_rows.view(B, Hq)
    for b in range(B):
        # a sum of at most 21 terms in float32, rounded once to half precision
        assert bool(((got.view(B, -1)[b].double() - mean[b]).abs() <= mean[b] * (2 ** -11 + 1e-5)).all())
        assert bool(((got_lse[b].double() - math.log(seen[b])).abs() <= 1e-5).all())
"""


@pytest.mark.parametrize("which", ["tables", "write", "prefill", "window", "decode", "varlen", "float32", "append"])
def test_first_call_under_capture_writes_its_results(which):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", SCRIPT % which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
