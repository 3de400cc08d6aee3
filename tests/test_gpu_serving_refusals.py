"""A serving step whose free list runs out: the requests that were served are
right, and what a refused one leaves is what the documentation says."""
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


@pytest.mark.parametrize("D,window,sinks", [(64, 0, 0), (128, 40, 3), (256, 0, 0)])
@pytest.mark.parametrize("num_free", [0, 2, 3, 5, 7])
def test_a_step_with_a_short_free_list(D, window, sinks, num_free):
    Hq, Hkv, page, width, dtype = 8, 2, 16, 8, torch.bfloat16
    held, new = np.array([20, 30, 0, 64, 15]), np.array([3, 40, 20, 1, 1])
    B, total = held.size, int(new.sum())
    gen = torch.Generator().manual_seed(2400 + D)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(dtype)

    # pages dealt to the rows for the keys they hold, the others free
    have = -(-held // page)
    pages = int(have.sum()) + 16
    order = torch.randperm(pages, generator=gen).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    first = np.concatenate([[0], np.cumsum(have)])
    for b in range(B):
        table[b, :have[b]] = order[first[b]:first[b + 1]]
    free = order[first[-1]:][:num_free].contiguous()
    k, v = normal(pages, page, Hkv, D), normal(pages, page, Hkv, D)
    q, k_new, v_new = normal(total, Hq, D), normal(total, Hkv, D), normal(total, Hkv, D)
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).int()
    before = torch.from_numpy(held).int()

    bt, slots, lens, used = oracle.extend_tables(table.numpy(), held, cu.numpy(), free.numpy(), page_size=page, num_pages=pages)
    served = lens == held + new
    assert served.any() and (num_free == 7 or not served.all())  # 7 pages serve every row
    k_want, v_want = k.clone(), v.clone()
    for t, s in enumerate(slots):
        if s >= 0:
            k_want.view(-1, Hkv, D)[s], v_want.view(-1, Hkv, D)[s] = k_new[t], v_new[t]

    kd, vd, td, qd, cd, ld = (x.cuda() for x in (k, v, table, q, cu, before))
    slots_d, lens_d, used_d = mxa.extend_tables(td, ld, cd, free.cuda(), page_size=page, num_pages=pages, total_q=total)
    mxa.write_cache(k_new.cuda(), v_new.cuda(), kd, vd, slots_d)
    out, lse = mxa.prefill(qd, cd, kd, vd, td, lens_d, max_seqlen_q=int(new.max()), window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert mxa.mxa_device_error(True) == mxa.MXA_OK
    assert td.cpu().numpy().tolist() == bt.tolist() and used_d.tolist() == [used]
    # a refused row shows in its length and in its slots
    assert lens_d.tolist() == lens.tolist()
    for b in range(B):
        s = slots_d[int(cu[b]):int(cu[b + 1])]
        assert bool((s >= 0).all()) if served[b] else bool((s == -1).all())
    # its keys and values were written nowhere
    assert torch.equal(kd.cpu().view(torch.int16), k_want.view(torch.int16))
    assert torch.equal(vd.cpu().view(torch.int16), v_want.view(torch.int16))
    # the served rows' outputs are right; a refused row's are finite, and for the caller to drop
    args = dict(Hkv=Hkv, page_size=page, dtype="bf16", scale=D ** -0.5, causal=True, window=window, sinks=sinks)
    table_now = torch.from_numpy(np.maximum(bt, 0)).int()
    ro, rl = oracle.decode_varlen(q, cu.numpy(), k_want, v_want, table_now, lens, **args)
    ra, _ = oracle.decode_varlen(q, cu.numpy(), k_want, v_want.abs(), table_now, lens, **args)
    rows = np.repeat(served, new)
    u = torch.finfo(dtype).eps / 2  # as in the chunk attention's own tests
    err = np.abs(out.cpu().double().numpy() - ro)
    assert (err <= u * ra + u * (np.abs(ro) + u * ra) + 2e-4 * ra)[rows].all()
    assert_lse_close(lse.cpu()[:, rows], rl[:, rows])
    assert torch.isfinite(out.float()).all()
