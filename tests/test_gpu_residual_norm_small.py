"""engram_residual_norm's norms of rows whose mean square is a denormal number: epsilons of 0 and smaller than the
least normal number, rows from 1e-17 down to where the squares are still numbers."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402


@pytest.mark.parametrize("eps", [0.0, 1e-40])
@pytest.mark.parametrize("dim", [64, 1000, 5120, 20480])
def test_rows_with_denormal_mean_squares(dim, eps):
    say(f"[gpu] residual norm: small rows of {dim}, epsilon {eps}")
    # The squares are multiples of 2^-149, each within half of one: relative to a square of 2^-2k, 2^(2k - 150); the
    # division by dim adds as much once, the root halves the sum.  2^(2k - 150) covers both, over fp32's own 2^-18
    # (serving_common.norm_ref counts 90 and 64 roundings of 2^-24).
    for k in (57, 62, 64, 66, 68, 70):
        v = 2.0 ** -k
        off = 2.0 ** -17 + 2.0 ** (2 * k - 150)
        g = torch.Generator(device="cuda").manual_seed(k)
        sign = torch.randint(0, 2, (1, 3, 2, dim), generator=g, device="cuda").float() * 2 - 1
        x = sign * v
        size = v / (v * v + eps) ** 0.5
        lay = eg.make_norm_layout(2, dim, pre_eps=eps, stream_format=eg.STREAM_FP32)
        _, h = eg.engram_residual_norm(lay, x)
        assert ((h.double() - sign.double() * size).abs() <= size * (off + 2.0 ** -8)).all(), (k, h.flatten()[:4])
        lay = eg.make_norm_layout(2, dim, pre_norm=False, post_eps=eps, stream_format=eg.STREAM_FP32)
        out, _ = eg.engram_residual_norm(lay, torch.zeros_like(x), x.bfloat16())
        assert ((out.double() - sign.double() * size).abs() <= size * off).all(), (k, out.flatten()[:4])


def test_rows_of_zeros_without_an_epsilon():
    say("[gpu] residual norm: zero rows with an epsilon of 0 are NaN, others stay")
    x = torch.ones((1, 2, 1, 64), device="cuda")
    x[:, 1] = 0
    _, h = eg.engram_residual_norm(eg.make_norm_layout(1, 64, pre_eps=0.0, stream_format=eg.STREAM_FP32), x)
    assert (h[:, 0] == 1).all() and h[:, 1].isnan().all()
