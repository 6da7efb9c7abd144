"""The error count of the absorbed attention: a visible position on a page outside the pool is counted, whichever of a
request's tiles sees it first."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import say  # noqa: E402
from test_gpu_latent_attention import Absorbed  # noqa: E402
from test_gpu_latent_tiles import with_long_table  # noqa: E402


def bad_positions(c):
    """The visible positions on bad pages, each once for its request."""
    st, n = c.st, 0
    for r in range(st.R):
        if st.new[r]:
            lo = max(0, st.held[r] + 1 - c.window) if c.window else 0
            n += int((st.slot_list(r, lo, st.held[r] + st.new[r]) < 0).sum())
    return n


# heads, latent, fp8, window, new, held, block, a long table, and the first bad page of request 0: its new tokens are at
# positions held .., so that the first tile of the request (16 rows and 32 in the first two and the third, 64, 128) sees
# none of the bad positions
CASES = [
    (16, 128, False, 0, [9] + [0] * 7, [32], 4, False, 9),
    (16, 512, True, 20, [9] + [0] * 7, [32], 4, False, 9),
    (32, 256, True, 0, [9] + [0] * 7, [61], 2, False, 32),
    (32, 256, True, 0, [5], [62], 2, False, 32),
    (32, 512, False, 30, [5], [62], 2, False, 32),
    (128, 512, True, 0, [3], [63], 1, False, 64),
    (128, 512, True, 0, [3], [63], 1, True, 64),
    (128, 512, False, 0, [2], [64], 1, True, 65),
    (100, 128, True, 2, [6], [90], 1, True, 92),
]


@pytest.mark.parametrize("H,dc,fp8,window,new,held,block,long,page", CASES)
def test_pages_that_the_first_tile_does_not_see(H, dc, fp8, window, new, held, block, long, page):
    say(f"[gpu] absorbed: bad pages behind the first tile H={H} {dc} fp8={fp8} window={window} {new} {held} long table: {long}")
    held = held + [0] * (len(new) - len(held))
    c = Absorbed(np.random.default_rng(41), new, held, H, dc, 32, fp8, block, window)
    c.st.table[0, page:] = -1
    if long:
        with_long_table(c, 32 * 1024 * 16)
    want = bad_positions(c)
    assert want > 0
    c.run()
    c.check()
    assert int(c.err) == want


@pytest.mark.parametrize("H,long", [(8, False), (40, False), (128, True)])
@pytest.mark.parametrize("window", [0, 37])
def test_each_position_counts_once(H, long, window):
    """Bad pages at the front, in the middle and at the end, of requests whose units many workgroups share."""
    say(f"[gpu] absorbed: bad pages everywhere H={H} window={window} long table: {long}")
    c = Absorbed(np.random.default_rng(42), [3, 0, 7, 1], [200, 40, 150, 333], H, 128, 32, True, 16, window)
    t = c.st.table
    t[0, 0], t[0, 12], t[2, 5], t[2, 9], t[3, :] = -1, c.st.n_blocks, -3, 2 ** 30, -1
    if long:
        with_long_table(c, 32 * 1024 * 16)
    c.run()
    c.check()
    assert int(c.err) == bad_positions(c)
