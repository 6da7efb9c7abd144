"""Latent attention of values near the end of bf16's range: weights that grow by less than the reference follows must not
take their sums past fp32."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import say  # noqa: E402
from latent_common import attend_ref, bits_bf16, make_rows, near, row_values  # noqa: E402
from test_gpu_latent_attention import Absorbed, Expanded  # noqa: E402
from test_gpu_latent_tiles import with_long_table  # noqa: E402

GROW = 15.5  # powers of two from a request's first score to its last


def repeated(c, R):
    """The case of one request as R requests over the same pages: enough for a workgroup to take whole ones."""
    st = c.st
    st.new, st.held, st.R, st.T = st.new * R, st.held * R, R, st.new[0] * R + 2
    st.table, st.start, st.slots = np.repeat(st.table, R, 0), (np.arange(R + 1) * st.new[0]).astype(np.int32), np.full(st.T, -1, np.int64)
    return c


@pytest.mark.parametrize("H,dc,fp8,new,held,R,long", [
    (8, 128, False, 1, 500, 1000, False), (16, 512, True, 1, 300, 600, False), (24, 256, False, 1, 300, 600, False),
    (40, 512, True, 1, 300, 300, False), (64, 256, False, 1, 300, 300, False), (128, 512, True, 1, 300, 300, True),
    (128, 128, False, 1, 300, 600, True)])
def test_absorbed(H, dc, fp8, new, held, R, long):
    say(f"[gpu] absorbed: values of 2^116 H={H} {dc} fp8={fp8} {R} requests of {new} behind {held}, long table: {long}")
    rng = np.random.default_rng(51)
    c = Absorbed(rng, [new], [held], H, dc, 32, fp8, 16)
    n, m = c.st.n_blocks * 16, held + new
    lat, rope = torch.from_numpy(rng.normal(0, 1, (n, dc))) * 2.0 ** 116, torch.zeros((n, 32))
    # scores by one rope feature alone, ascending along the positions
    rope[c.st.slot_list(0, 0, m), 5] = torch.linspace(0, GROW / (c.scale * math.log2(math.e)), m)
    c.rows = make_rows(bits_bf16(lat.bfloat16()), bits_bf16(rope.bfloat16()), fp8)
    repeated(c, R)
    c.q = torch.zeros((c.st.T, H, dc + 32), dtype=torch.bfloat16)
    c.q[:, :, dc + 5] = 1.0
    if long:
        with_long_table(c, 32 * 1024 * 16)
    c.run()
    live = R * new
    assert torch.isfinite(c.out[:live].float()).all() and torch.isfinite(c.lse[:live]).all()
    lat, rope = row_values(c.rows[c.st.slot_list(0, 0, m)], dc, fp8)
    o, l, do, dl = attend_ref(c.q[:1, 0].double().numpy(), np.concatenate([lat, rope], 1), lat, np.array([held]), np.arange(m), c.scale, 0)
    near(c.out[:live], o[None], do[None])  # (every token and head: the same query)
    near(c.lse[:live], l[None], dl[None])


@pytest.mark.parametrize("H,hd,new,held", [(2, 64, [37, 1], [100, 300]), (3, 128, [200], [100]), (1, 128, [3], [2000]), (128, 128, [512], [200]),
                                           (128, 64, [2100], [30])])
def test_expanded(H, hd, new, held):
    say(f"[gpu] expanded: values of 2^116 H={H} {hd} {new} {held}")
    c = Expanded(np.random.default_rng(52), new, held, H, hd, 32)
    c.kv = c.kv * 2.0 ** 116
    c.kv[:, :, :hd] = 0.0
    c.rope = torch.zeros_like(c.rope)
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 3] = 1.0
    for r in range(c.st.R):
        a, b = int(c.first[r]), int(c.first[r + 1])
        c.kv[a: b, :, 3] = torch.linspace(0, GROW / (c.scale * math.log2(math.e)), b - a).bfloat16()[:, None]
    c.run()
    assert torch.isfinite(c.out[: sum(new)].float()).all()
    c.check(heads=[0, H - 1], tokens=[0, 1, 15, 36, 100, 199, 255, 256, 511, 1000, 2099])
