"""Calls whose launch would need 2^32 threads, of which some would be lost without an error: refused before they write."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402


def test_residual_norm_of_2_to_the_26_rows():
    say("[gpu] residual norm: 2^26 + 8 rows of 8 features, 2^26, and fewer")
    lay = eg.make_norm_layout(1, 8, post_norm=False)
    w = torch.ones((1, 8), device="cuda")
    x = torch.ones((1, (1 << 26) + 8, 1, 8), dtype=torch.bfloat16, device="cuda")
    h = torch.full_like(x, 5.0)
    for n in ((1 << 26) + 8, 1 << 26):
        with pytest.raises(eg.EngramError):
            eg.engram_residual_norm(lay, x[:, :n], pre_weight=w, h=h[:, :n])
        assert (h == 5).all()
    n = (1 << 26) - 4  # the longest that fits
    eg.engram_residual_norm(lay, x[:, :n], pre_weight=w, h=h[:, :n])
    assert (h[:, :n] == 1).all() and (h[:, n:] == 5).all()


def test_gate_of_2_to_the_24_tokens():
    say("[gpu] gate: 2^24 + 1 tokens, 2^24, and one fewer")
    n = (1 << 24) + 1
    lay = eg.make_layout(4, 64, 6, 64, 32, 1000)
    w = torch.ones((4, 64), device="cuda")
    x = torch.zeros((1, n, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.ones((1, n, 5 * 64), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(x, 5.0)
    for m in (n, n - 1):
        with pytest.raises(eg.EngramError):
            eg.engram_gate_apply(lay, x[:, :m], kv[:, :m], w, w, out=out[:, :m])
        assert (out == 5).all()
    eg.engram_gate_apply(lay, x[:, 2:], kv[:, 2:], w, w, out=out[:, 2:])
    assert (out[:, :2] == 5).all() and (out[:, 2:] == out[0, -1, 0, 0]).all() and float(out[0, -1, 0, 0]) != 5
