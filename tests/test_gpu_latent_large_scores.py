"""Latent attention with scores so large that a product with the scale, rounded to fp32, is off by many powers of two:
one key then takes everything, and outputs are its values, not NaN."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import say  # noqa: E402
from latent_common import EPS, U, row_values  # noqa: E402
from test_gpu_latent_attention import Absorbed, Expanded, normal  # noqa: E402
from test_gpu_latent_tiles import with_long_table  # noqa: E402


def check_head(out, lse, q, k, v, pos, key_pos, scale, window):
    """Returns the tokens whose result is certain: the distance of their two highest scores passes the bound of the scores'
    errors (an fp32 sum of D products, within (D + 2) 2^-23 of the sum of their magnitudes, and the scale's and the
    difference's roundings) by 200, so that the others' weights are below e^-200 and vanish.  Of these the weight is rounded
    to bf16 for the second product but not for its sum, and the output once: within 2 EPS and a few roundings of fp32."""
    certain = 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in range(len(pos)):
        j = np.nonzero((key_pos <= pos[i]) & ((key_pos > pos[i] - window) if window else True))[0]
        s = scale * (k[j] @ q[i])
        err = (q.shape[1] + 2) * 2.0 ** -23 * abs(scale) * (np.abs(k[j]) @ np.abs(q[i])).max() + 8 * U * np.abs(s).max()
        order = np.argsort(s)
        if len(j) > 1 and s[order[-1]] - s[order[-2]] < 2 * err + 200:
            continue
        certain += 1
        best = v[j[order[-1]]]
        assert (np.abs(got[i] - best) <= (2 * EPS + EPS * EPS + 16 * U) * np.abs(best)).all()
        assert abs(got_lse[i] - s[order[-1]]) <= err + 8 * U * abs(s[order[-1]]) + 2.0 ** -20
    return certain


@pytest.mark.parametrize("std", [2.0 ** 12, 2.0 ** 15, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("H,dc,fp8,window,new,held,long", [
    (8, 128, False, 0, [1, 1, 1], [300, 40, 7], False), (16, 512, True, 50, [1, 1], [300, 90], False),
    (16, 128, False, 0, [1, 2], [300, 40], False), (32, 512, True, 0, [1, 1], [90, 200], False), (40, 512, True, 30, [1, 2], [300, 33], False),
    (64, 256, False, 0, [1], [700], False), (128, 512, True, 0, [1, 1], [300, 63], True), (128, 512, False, 0, [1], [200], True),
    (128, 128, True, 0, [2], [129], True)])
def test_absorbed(H, dc, fp8, window, new, held, long, std):
    say(f"[gpu] absorbed: values of {std:g} H={H} {dc} fp8={fp8} window={window} {new} {held} long table: {long}")
    rng = np.random.default_rng(43)
    c = Absorbed(rng, new, held, H, dc, 32, fp8, 16, window)
    if fp8:  # (the scales' bytes)
        c.rows[:, dc: dc + dc // 32] += np.uint8(np.log2(std))
    else:
        c.rows = (torch.from_numpy(c.rows).view(torch.bfloat16) * std).view(torch.uint8).numpy()
    c.q = c.q * std
    if long:
        with_long_table(c, 32 * 1024 * 16)
    c.run()
    lat, rope = row_values(c.rows, dc, fp8)
    both, q, certain, tokens = np.concatenate([lat, rope], 1), c.q.double().numpy(), 0, 0
    for r in range(c.st.R):
        a, n, h = int(c.st.start[r]), c.st.new[r], c.st.held[r]
        at = c.st.slot_list(r, 0, h + n)
        for head in range(H):
            certain += check_head(c.out[a: a + n, head], c.lse[a: a + n, head], q[a: a + n, head], both[at], lat[at], np.arange(h, h + n),
                                  np.arange(h + n), c.scale, window)
            tokens += n
    assert certain > tokens // 2


@pytest.mark.parametrize("std", [2.0 ** 12, 2.0 ** 15, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("H,hd,window,new,held", [(2, 64, 0, [37, 1], [0, 300]), (3, 128, 50, [200, 5], [100, 400]), (1, 128, 0, [3], [2000]),
                                                  (128, 128, 0, [512], [200]), (128, 64, 70, [2100], [30])])
def test_expanded(H, hd, window, new, held, std):
    say(f"[gpu] expanded: values of {std:g} H={H} {hd} window={window} {new} {held}")
    rng = np.random.default_rng(44)
    c = Expanded(rng, new, held, H, hd, 32, window)
    c.q, c.kv, c.rope = c.q * std, c.kv * std, c.rope * std
    c.run()
    q, kv, rope, certain, tokens = c.q.double().numpy(), c.kv.double().numpy(), c.rope.double().numpy(), 0, 0
    for r in range(c.st.R):
        a, n, h, f = int(c.st.start[r]), c.st.new[r], c.st.held[r], int(c.first[r])
        pos = np.unique(np.linspace(0, n - 1, 20).astype(int))
        for head in (0, H - 1):
            k = np.concatenate([kv[f: f + h + n, head, :hd], rope[f: f + h + n]], 1)
            certain += check_head(c.out[a + torch.from_numpy(pos), head], c.lse[a + torch.from_numpy(pos), head], q[a + pos, head], k,
                                  kv[f: f + h + n, head, hd:], h + pos, np.arange(h + n), c.scale, window)
            tokens += len(pos)
    assert certain > tokens // 2
