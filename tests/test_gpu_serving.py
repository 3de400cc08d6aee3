"""A serving loop over the paged cache, end to end on the GPU: block tables
extended from a free list, prompts written and attended in chunks, then
single tokens with and without a sliding window; every step checked against
the fp64 oracle on the keys and values as plain rows.  Once call by call and
once as one captured graph that is replayed step after step.
"""
import numpy as np
import pytest
import torch

import oracle
from tests.tolerance import assert_lse_close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Serving:
    """Requests over one pool; `rows[b]` is the plain (unpaged) truth."""

    def __init__(self, B, Hq, Hkv, D, page, width, dtype, seed):
        self.B, self.Hq, self.Hkv, self.D, self.page, self.width, self.dtype = B, Hq, Hkv, D, page, width, dtype
        self.gen = torch.Generator().manual_seed(seed)
        self.pages = B * width
        shape = (self.pages, page, Hkv, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(self.pages, generator=self.gen).int().cuda()
        self.rows = [[torch.empty(0, Hkv, D, dtype=dtype) for _ in range(2)] for _ in range(B)]

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen).to(self.dtype)

    def step(self, counts, window=0, sinks=0):
        """One step with counts[b] new tokens; returns what the oracle needs and the outputs."""
        total = sum(counts)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
        q, k_new, v_new = self.normal(total, self.Hq, self.D), self.normal(total, self.Hkv, self.D), self.normal(total, self.Hkv, self.D)
        cud = cu.cuda()
        slots, lens, used = mxa.extend_tables(self.table, self.lens, cud, self.free, page_size=self.page, num_pages=self.pages,
                                              total_q=total)
        mxa.write_cache(k_new.cuda(), v_new.cuda(), self.k, self.v, slots)
        out, lse = mxa.prefill(q.cuda(), cud, self.k, self.v, self.table, lens, max_seqlen_q=max(counts), window=window,
                               sinks=sinks)
        single = None
        if set(counts) == {1}:  # the decode entry point answers the same step
            single = mxa.decode(q.view(self.B, 1, self.Hq, self.D).cuda(), self.k, self.v, self.table, lens, causal=True,
                                window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_OK
        self.free, self.lens = self.free[int(used):].contiguous(), lens
        for b in range(self.B):
            s = slice(int(cu[b]), int(cu[b + 1]))
            self.rows[b] = [torch.cat([old, new[s]]) for old, new in zip(self.rows[b], (k_new, v_new))]
        assert lens.tolist() == [r[0].shape[0] for r in self.rows]
        self.check(q, cu, out.cpu(), lse.cpu(), window, sinks)
        if single is not None:
            self.check(q, cu, single[0].cpu().view(total, self.Hq, self.D), single[1].cpu().view(self.B, self.Hq).t(), window, sinks)

    def check(self, q, cu, out, lse, window, sinks):
        L = max(r[0].shape[0] for r in self.rows)
        k, v = (torch.zeros(self.B, max(1, L), self.Hkv, self.D, dtype=self.dtype) for _ in range(2))
        for b, (rk, rv) in enumerate(self.rows):
            k[b, :rk.shape[0]], v[b, :rv.shape[0]] = rk, rv
        args = dict(Hkv=self.Hkv, page_size=max(1, L), dtype="bf16" if self.dtype == torch.bfloat16 else "f16",
                    scale=self.D ** -0.5, causal=True, window=window, sinks=sinks)
        lens = np.array([r[0].shape[0] for r in self.rows], dtype=np.int32)
        ro, rl = oracle.decode_varlen(q, cu.numpy(), k, v, None, lens, **args)
        ra, _ = oracle.decode_varlen(q, cu.numpy(), k, v.abs(), None, lens, **args)
        u = torch.finfo(self.dtype).eps / 2  # as in the chunk attention's own tests
        err = np.abs(out.double().numpy() - ro)
        assert (err <= u * ra + u * (np.abs(ro) + u * ra) + 2e-4 * ra).all(), err.max()
        assert_lse_close(lse, rl)


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype", [(8, 2, 128, 16, torch.bfloat16), (6, 2, 64, 8, torch.float16),
                                                 (4, 1, 256, 32, torch.bfloat16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (96, 4)])
def test_prompts_in_chunks_then_single_tokens(Hq, Hkv, D, page, dtype, window, sinks):
    s = Serving(3, Hq, Hkv, D, page, 1024 // page, dtype, seed=D + window)
    s.step([70, 1, 300], window, sinks)
    s.step([130, 257, 1], window, sinks)
    s.step([0, 33, 64], window, sinks)
    for _ in range(3):
        s.step([1, 1, 1], window, sinks)


def test_one_graph_replayed_step_after_step():
    # tables, write, attention and the lengths' update captured once; every
    # replay serves the next token of every request
    B, Hq, Hkv, D, page, width, steps = 4, 8, 2, 128, 16, 8, 40
    dtype = torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(5)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    pages = B * width
    k, v = torch.zeros(pages, page, Hkv, D, dtype=dtype, device="cuda"), torch.zeros(pages, page, Hkv, D, dtype=dtype, device="cuda")
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    pool = torch.cat([torch.randperm(pages, device="cuda").int(), torch.zeros(pages, dtype=torch.int32, device="cuda")])
    free = pool[:pages].clone()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    q, kn, vn = normal(B, Hq, D), normal(B, Hkv, D), normal(B, Hkv, D)
    slots, new_lens, used = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B, 1))
    out, lse = torch.empty_like(q), torch.empty(Hq, B, device="cuda")
    prep = mxa.prepare_prefill(q, cu, k, table, max_seqlen_q=1)
    at = torch.arange(pages, device="cuda")

    def step():
        mxa.extend_tables(table, lens, cu, free, page_size=page, num_pages=pages, total_q=B, slots=slots, new_seqlens=new_lens,
                          pages_used=used)
        mxa.write_cache(kn, vn, k, v, slots)
        mxa.prefill(q, cu, k, v, table, new_lens, max_seqlen_q=1, window=40, sinks=2, prepared=prep, out=out, lse=lse)
        lens.copy_(new_lens)
        free.copy_(free[(at + used).clamp_max(pages - 1)])

    keep = [t.clone() for t in (table, lens, free)]
    step()  # loads the kernels
    for t, old in zip((table, lens, free), keep):
        t.copy_(old)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    truth = [torch.zeros(B, steps, Hkv, D, dtype=dtype) for _ in range(2)]
    for i in range(steps):
        for t, n in ((q, (B, Hq, D)), (kn, (B, Hkv, D)), (vn, (B, Hkv, D))):
            t.copy_(normal(*n))
        graph.replay()
        torch.cuda.synchronize()
        truth[0][:, i], truth[1][:, i] = kn.cpu(), vn.cpu()
        if i % 13 == 0 or i == steps - 1:
            assert mxa.mxa_device_error(True) == mxa.MXA_OK
            assert lens.tolist() == [i + 1] * B
            args = dict(Hkv=Hkv, page_size=steps, dtype="bf16", scale=D ** -0.5, causal=True, window=40, sinks=2)
            rows = (None, np.full(B, i + 1, dtype=np.int32))
            ro, rl = oracle.decode_varlen(q.cpu(), cu.cpu().numpy(), *truth, *rows, **args)
            ra, _ = oracle.decode_varlen(q.cpu(), cu.cpu().numpy(), truth[0], truth[1].abs(), *rows, **args)
            u = torch.finfo(dtype).eps / 2  # as above
            assert (np.abs(out.cpu().double().numpy() - ro) <= u * ra + u * (np.abs(ro) + u * ra) + 2e-4 * ra).all()
            assert_lse_close(lse.cpu(), rl)
