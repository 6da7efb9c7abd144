"""The serving operators on int16 views of bf16 tensors: the bits of the bf16 call, outputs in the views' type."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402

I16, BF = torch.int16, torch.bfloat16


def normal(g, *shape):
    return torch.empty(shape, device="cuda").normal_(generator=g)


def test_int16_views_give_the_same_bits():
    say("[gpu] serving operators: int16 views of bf16 tensors")
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w, r = normal(g, 33, 72).to(BF), normal(g, 50, 72).to(BF), normal(g, 33, 50).to(BF)
    lay = eg.make_linear_layout(72, 50)
    got, ref = eg.engram_linear(lay, x.view(I16), w.view(I16), residual=r.view(I16)), eg.engram_linear(lay, x, w, residual=r)
    assert got.dtype is I16 and torch.equal(got, ref.view(I16))
    lay = eg.make_linear_layout(72, 50, stream_format=eg.STREAM_FP32)
    got = eg.engram_linear(lay, x.view(I16), w)
    assert got.dtype is torch.float32 and torch.equal(got, eg.engram_linear(lay, x, w))
    x, y, z = (normal(g, 1, 9, 2, 136).to(BF) for _ in range(3))
    lay = eg.make_norm_layout(2, 136, gate=eg.GATE_FEATURE)
    out, h = eg.engram_residual_norm(lay, x.view(I16), y.view(I16), gate=z.view(I16))
    ref, h_ref = eg.engram_residual_norm(lay, x, y, gate=z)
    assert out.dtype is I16 and h.dtype is I16
    assert torch.equal(out, ref.view(I16)) and torch.equal(h, h_ref.view(I16))
    lay = eg.make_norm_layout(2, 136, stream_format=eg.STREAM_FP32)
    out, h = eg.engram_residual_norm(lay, x.float(), y.view(I16))
    assert out.dtype is torch.float32 and h.dtype is BF
