"""engram_linear's activations at infinities, NaN and the largest finite arguments, plain and gated, against
their definitions in include/engram.h evaluated in 64 bits: which outputs are NaN, which infinite, and of which
sign.  Arguments come once from the bias (x = 0) and once from the product itself."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402

INF, NAN = math.inf, math.nan
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")
# every one exact in bf16, so that the product gives it unrounded
ARGS = [INF, -INF, NAN, 0.0, 4.0, -4.0, 2.0 ** 66, -2.0 ** 66, 2.0 ** 126, -2.0 ** 126]


def defined(z, act):
    if act == "relu":
        return torch.where(z.isnan(), z, z.clamp(min=0))
    if act == "gelu":  # z Phi(z)
        return z * (0.5 * torch.special.erfc(-z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))) / 2
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    return z


def same(got, ref, what):
    got, ref = got.double().cpu(), ref.cpu()
    assert torch.equal(got.isnan(), ref.isnan()), (what, got[0].tolist(), ref[0].tolist())
    wild = ref.isinf()
    assert torch.equal(got[wild], ref[wild]) and not got[~wild].isinf().any(), (what, got[0].tolist(), ref[0].tolist())
    # finite values: half a step of bf16 (2^-8), and far more than the 1e-6 of the activations' own error
    tame = ref.isfinite()
    assert ((got - ref)[tame].abs() <= 2.0 ** -7 * ref[tame].abs() + 1e-5).all(), what


# 1 and 12 tokens share K in a workgroup, 40 and 300 take tiles, 100 x 5120 splits K
@pytest.mark.parametrize("M,K", [(1, 64), (12, 72), (40, 64), (300, 136), (100, 5120)])
@pytest.mark.parametrize("act", ACTS)
def test_activations_at_their_limits(act, M, K):
    say(f"[gpu] linear: {act} of infinities and NaN, {M} tokens, K {K}")
    pairs = [(z, u) for z in ARGS for u in (1.0, -2.0, 0.0, INF)]
    for glu in (False, True):
        z = torch.tensor([p[0] for p in pairs] if glu else ARGS, dtype=torch.float64)
        u = torch.tensor([p[1] for p in pairs], dtype=torch.float64)
        ref = defined(z, act) * u if glu else defined(z, act)
        N = len(z)
        rows = torch.cat([z, u]) if glu else z
        for fp32 in (False, True):
            lay = eg.make_linear_layout(K, N, activation=ACTS.index(act), glu=glu,
                                        stream_format=eg.STREAM_FP32 if fp32 else eg.STREAM_BF16)
            # from the bias
            x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
            w = torch.ones((len(rows), K), dtype=torch.bfloat16, device="cuda")
            got = eg.engram_linear(lay, x, w, bias=rows.float().cuda())
            same(got, ref.expand(M, N), (act, glu, fp32, "bias"))
            # from the product: x = (1, 0, 0, ...)
            x[:, 0] = 1
            w.zero_()
            w[:, 0] = rows.bfloat16().cuda()
            got = eg.engram_linear(lay, x, w)
            same(got, ref.expand(M, N), (act, glu, fp32, "product"))
