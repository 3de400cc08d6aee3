"""Pages that lie past 4 GB in their pool, and past 2^31 values: the same results
as from the same keys in a small pool, and nothing else written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from decode_attention_packed_b200 import mxa


@pytest.fixture(scope="module", autouse=True)
def _needs_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("D,Hkv", [(128, 8), (64, 16), (256, 4)])
def test_far_pages(D, Hkv):
    page, Hq, B, width, new = 64, 2 * Hkv, 2, 4, 70
    near, far = 16, 45000  # pages of 128 KB: 5.9 GB and 2.9e9 values a pool
    gen = torch.Generator(device="cuda").manual_seed(2500)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").half()

    small = [normal(near, page, Hkv, D) for _ in range(2)]
    big = [torch.empty(far, page, Hkv, D, dtype=torch.float16, device="cuda") for _ in range(2)]
    for s, b in zip(small, big):
        b[far - near:] = s
        b[:near] = 7.0  # where an address cut to 32 bits would land
    q, k_new, v_new = normal(B * new, Hq, D), normal(B * new, Hkv, D), normal(B * new, Hkv, D)
    one, k_one, v_one = normal(B, 1, Hq, D), normal(B, 1, Hkv, D), normal(B, 1, Hkv, D)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    before = torch.tensor([100, 3], dtype=torch.int32, device="cuda")
    results = []
    for k, v, base in ((*small, 0), (*big, far - near)):
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        table[0, :2], table[1, 0] = torch.tensor([5, 2], dtype=torch.int32, device="cuda") + base, 9 + base
        free = torch.tensor([11, 3, 15, 0], dtype=torch.int32, device="cuda") + base
        slots, lens, used = mxa.extend_tables(table, before, cu, free, page_size=page, num_pages=base + near, total_q=2 * new)
        mxa.write_cache(k_new, v_new, k, v, slots)
        got = [slots - base * page, *mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=new)]
        got += mxa.prefill(q, cu, k, v, table, lens, max_seqlen_q=new, window=60, sinks=2)
        got += mxa.decode(one, k, v, table, lens, causal=True, window=60, sinks=2, k_new=k_one, v_new=v_one)
        torch.cuda.synchronize()
        assert mxa.mxa_device_error(True) == mxa.MXA_OK
        results.append([t.cpu() for t in got] + [k[base:base + near].cpu(), v[base:base + near].cpu()])
    for a, b in zip(*results):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for b in big:
        assert bool((b[:near] == 7).all())
