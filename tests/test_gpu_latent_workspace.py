"""Expanded attention with one workspace kept for steps of every length: eager, and in a captured graph between eager steps of
other lengths."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from test_gpu_latent_attention import Expanded, normal  # noqa: E402


@pytest.mark.parametrize("hd,H", [(128, 8), (64, 24)])
def test_one_workspace_for_steps_of_every_length(hd, H):
    say(f"[gpu] expanded: one workspace for steps of 1 .. 3000 tokens, {H} heads of {hd}")
    rng = np.random.default_rng(61)
    steps = [([3000], [0]), ([1], [5000]), ([300], [4000]), ([70, 9], [2000, 2500]), ([3], [600]), ([900], [5000]), ([2, 1, 40], [5, 2900, 0])]
    cases = [Expanded(rng, new, held, H, hd, 32) for new, held in steps]
    lay = cases[0].lay
    size = eg.engram_latent_attention_expanded_workspace_bytes_up_to(lay, max(c.st.T for c in cases), max(int(c.first[-1]) for c in cases))
    own = [eg.engram_latent_attention_expanded_workspace_bytes(lay, c.st.R, c.st.T, int(c.first[-1])) for c in cases]
    assert max(own) <= size and own[0] < max(own)  # (the longest step's own size would be too small)
    buf = torch.full((size + 512,), 171, dtype=torch.uint8, device="cuda")
    ws = buf[256:256 + size]
    for c in cases:
        want, lse = c.run().clone(), c.lse.clone()
        c.run(workspace=ws)
        assert torch.equal(c.out, want) and torch.equal(c.lse, lse)
        c.check(heads=[0, H - 1], tokens=[0, 1, 8, 39, 69, 299, 899, 2999])
    assert (buf[:256] == 171).all() and (buf[256 + size:] == 171).all()

    def call(c):
        args = [c.lay, c.q.cuda(), c.kv.cuda(), c.rope.cuda(), torch.from_numpy(c.first).cuda(), c.st.plan(eg)]
        out = torch.full_like(c.out, 5.0)
        return lambda: eg.engram_latent_attention_expanded(*args, out=out, workspace=ws), args[1], out
    (fa, qa, oa), (fb, _, ob) = call(cases[2]), call(cases[5])
    want = cases[5].run().clone()
    fa()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa()
    for k in range(4):
        qa.copy_(normal(rng, *qa.shape))
        fa()
        eager = oa.clone()
        oa.fill_(5.0)
        fb()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, eager) and torch.equal(ob, want), k
