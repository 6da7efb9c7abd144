"""engram_linear with one workspace kept for steps of every length: sized once for the longest step, as a serving
program sizes it, then used for shorter ones, split and whole, eagerly and in a captured graph."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402


@pytest.mark.parametrize("K,N,glu", [(5120, 1030, False), (4096, 640, True)])
def test_one_workspace_for_steps_of_every_length(K, N, glu):
    say(f"[gpu] linear: one workspace for 1 .. 4000 tokens x {K} x {N}, gated {glu}")
    g = torch.Generator(device="cuda").manual_seed(K)
    lay = eg.make_linear_layout(K, N, glu=glu, stream_format=eg.STREAM_FP32)
    size = eg.engram_linear_workspace_bytes_up_to(lay, 4000)
    sizes = [eg.engram_linear_workspace_bytes(lay, m) for m in (1, 20, 64, 100, 200, 500, 1000, 2000, 4000)]
    assert max(sizes) > sizes[-1] == 0 and size >= max(sizes)  # (the longest step's own size would be too small)
    buf = torch.full((size + 512,), 171, dtype=torch.uint8, device="cuda")
    ws = buf[256:256 + size]

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").float()
    w = whole(2 * N if glu else N, K)
    if glu:  # gated products stay below 2^24
        w *= torch.rand(w.shape, generator=g, device="cuda") < 64 / K
    for M in (4000, 2000, 1, 20, 64, 100, 200, 500, 1000, 17, 333):
        x = whole(M, K)
        z = x.double() @ w.double().T
        ref = z[:, :N] * z[:, N:] if glu else z
        assert ref.abs().max() < 2 ** 24
        got = eg.engram_linear(lay, x.bfloat16(), w.bfloat16(), workspace=ws)
        assert torch.equal(got.double(), ref), M
    assert (buf[:256] == 171).all() and (buf[256 + size:] == 171).all()
    x, wb, out = whole(100, K).bfloat16(), w.bfloat16(), torch.empty((100, N), device="cuda")
    eg.engram_linear(lay, x, wb, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.engram_linear(lay, x, wb, out=out, workspace=ws)
    for k in range(3):
        x.neg_()
        ref = eg.engram_linear(lay, x, wb, workspace=ws)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref), k
