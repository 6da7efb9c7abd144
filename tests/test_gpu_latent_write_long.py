"""engram_latent_write with more tokens than 2^32 threads of one workgroup for four of them would cover."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from latent_common import bits_bf16, make_rows  # noqa: E402


@pytest.mark.parametrize("fp8", [False, True])
def test_write_of_many_tokens(fp8):
    say(f"[gpu] latent write: 2^26 + 9 tokens, fp8={fp8}")
    n, dc, dr = (1 << 26) + 9, 128, 32
    at = torch.tensor([0, 3, 70_001, (1 << 25) + 5, (1 << 26) - 1, 1 << 26, n - 1])
    lay = eg.make_latent_layout(1, dc, dr, cache_format=eg.CACHE_MXFP8 if fp8 else eg.CACHE_BF16)
    pages = eg.make_page_layout(16, 1, 1)
    latent, rope = (torch.empty((n, d), dtype=torch.bfloat16, device="cuda") for d in (dc, dr))
    rng = np.random.default_rng(45)
    x = torch.from_numpy(rng.normal(0, 1, (len(at), dc + dr)).astype(np.float32)).bfloat16()
    latent[at.cuda()], rope[at.cuda()] = x[:, :dc].cuda(), x[:, dc:].cuda()
    plan = eg.BatchPlan(1, n, device="cuda")
    plan.slots.fill_(-1)
    plan.slots[at.cuda()] = torch.arange(len(at), device="cuda")
    plan.slots[n - 2] = 16  # past the pool
    cache, err = eg.make_latent_cache(lay, pages), torch.zeros(1, dtype=torch.int32, device="cuda")
    eg.engram_latent_write(lay, pages, latent, rope, plan, cache, err_count=err)
    want = make_rows(bits_bf16(x[:, :dc]), bits_bf16(x[:, dc:]), fp8)
    got = cache.view(torch.uint8).view(16, -1).cpu().numpy()
    assert np.array_equal(got[: len(at)], want) and (got[len(at):] == 0).all()
    assert int(err) == 1
