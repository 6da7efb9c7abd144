"""The tile sizes of the latent attention that few rows or tokens do not reach, against the formulas in 64 bits:
tiles of 64 and 128 rows over the pages, tiles of 256 tokens over expanded rows, with scores that grow, masks,
values that are not finite and pages outside the pool in each."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from latent_common import attend_ref, bits_bf16, make_rows, near, row_values  # noqa: E402
from test_gpu_latent_attention import Absorbed, Expanded, normal  # noqa: E402


def with_long_table(c, positions):
    """The case with a table for so many positions a request: its tile size goes by the table."""
    st = c.st
    blocks = -(-positions // st.block)
    st.table = np.concatenate([st.table, np.full((st.R, blocks - st.max_blocks), -1, np.int32)], 1)
    st.max_blocks = blocks
    return c


# heads, latent, rope, fp8, window, new, held; a long table
TILES = [
    (40, 512, 64, True, 0, [1, 2], [90, 33], False),
    (64, 512, 64, False, 20, [1, 3], [70, 40], False),
    (48, 128, 32, True, 0, [1, 1], [65, 300], False),
    (128, 512, 64, True, 0, [1, 2, 0, 1], [150, 63, 10, 0], True),
    (100, 512, 64, False, 0, [1, 2], [97, 31], True),
    (128, 256, 64, True, 40, [2, 1], [100, 64], True),
    (70, 256, 32, False, 0, [3], [200], True),
    (128, 128, 64, True, 0, [2, 1], [129, 40], True),
    (128, 128, 32, False, 33, [1, 2], [100, 70], True),
]


def tile_case(rng, H, dc, dr, fp8, window, new, held, long, **kw):
    c = Absorbed(rng, new, held, H, dc, dr, fp8, 64, window, **kw)
    return with_long_table(c, 32 * 1024 * 16) if long else c


@pytest.mark.parametrize("H,dc,dr,fp8,window,new,held,long", TILES)
def test_absorbed_tiles(H, dc, dr, fp8, window, new, held, long):
    say(f"[gpu] absorbed tiles H={H} {dc}+{dr} fp8={fp8} window={window} {new} {held} long table: {long}")
    c = tile_case(np.random.default_rng(31), H, dc, dr, fp8, window, new, held, long)
    c.run()
    c.check()
    assert int(c.err) == 0


@pytest.mark.parametrize("H,dc,fp8,long", [(48, 256, True, False), (64, 512, False, False), (128, 512, True, True), (96, 512, False, True),
                                           (128, 256, False, True), (128, 128, True, True)])
def test_absorbed_tiles_with_scores_that_grow(H, dc, fp8, long):
    """Later keys score higher by far: the reference maximum moves again and again."""
    say(f"[gpu] absorbed tiles, growing scores H={H} {dc} fp8={fp8}")
    rng = np.random.default_rng(32)
    c = tile_case(rng, H, dc, 32, fp8, 0, [1], [250], long)
    lat = normal(rng, c.st.n_blocks * 64, dc).abs().float()
    p = np.arange(251)
    lat[c.st.slot_list(0, 0, 251)] *= torch.from_numpy(0.02 * p[:, None]).float()
    c.rows = make_rows(bits_bf16(lat.bfloat16()), bits_bf16(normal(rng, len(lat), 32)), fp8)
    c.q = c.q.abs()
    s = row_values(c.rows[c.st.slot_list(0, 0, 251)], dc, fp8)[0] @ c.q[0, 0, :dc].double().numpy() * c.scale * math.log2(math.e)
    assert s[-1] - s[0] > 3 * 16
    c.run()
    c.check()


@pytest.mark.parametrize("H,dc,fp8,long", [(40, 512, True, False), (64, 128, False, False), (128, 512, True, True), (128, 512, False, True),
                                           (70, 256, True, True), (128, 128, False, True)])
def test_absorbed_tiles_do_not_look_at_what_is_masked(H, dc, fp8, long):
    say(f"[gpu] absorbed tiles, values that are not finite H={H} {dc} fp8={fp8}")
    c = tile_case(np.random.default_rng(33), H, dc, 64, fp8, 0, [5, 1], [60, 70], long)
    st = c.st
    seen = np.zeros(len(c.rows), bool)
    for r in range(st.R):
        seen[st.slot_list(r, 0, st.held[r] + st.new[r])] = True
    c.rows[~seen] = 0xFF
    at = st.slot_list(0, 63, 64)[0]  # of the fourth new token
    if fp8:
        c.rows[at, 7] = 0x7F
    else:
        c.rows[at].view(np.uint16)[7] = 0x7F80
    c.run()
    assert not torch.isfinite(c.out[3:5, :, 7].float()).any()
    lat, rope = row_values(c.rows, dc, fp8)
    both = np.concatenate([lat, rope], 1)
    for r, n in ((0, 3), (1, 1)):
        first, h = int(st.start[r]), st.held[r]
        s = st.slot_list(r, 0, h + n)
        for head in range(0, H, 13):
            o, l, do, dl = attend_ref(c.q[first: first + n, head].double().numpy(), both[s], lat[s], np.arange(h, h + n), np.arange(h + n), c.scale, 0)
            near(c.out[first: first + n, head], o, do, f"request {r}")
            near(c.lse[first: first + n, head], l, dl, f"request {r}")


@pytest.mark.parametrize("H,dc,fp8,long", [(40, 512, False, False), (64, 256, True, False), (128, 512, True, True), (128, 512, False, True)])
def test_absorbed_tiles_leave_out_pages_outside_the_pool(H, dc, fp8, long):
    say(f"[gpu] absorbed tiles, pages outside the pool H={H} {dc} fp8={fp8}")
    c = tile_case(np.random.default_rng(34), H, dc, 64, fp8, 0, [1, 2, 1], [50, 200, 130], long)
    t = c.st.table
    t[0, :] = -1
    t[1, 1] = c.st.n_blocks
    t[2, 2] = -7
    c.run()
    assert int(c.err) > 0 and (c.out[0] == 0).all() and (c.lse[0] == -math.inf).all()
    c.check()


# ---------------------------------------------------------------- expanded, tiles of 256 tokens: heads enough to fill the device with them

LARGE = [
    (128, 64, 0, [250] * 8, [0, 1, 63, 64, 100, 7, 300, 20], 64),
    (128, 32, 70, [250] * 8, [0, 1, 63, 64, 100, 7, 300, 20], 64),
    (128, 64, 0, [512], [200], 128),
    (128, 64, 0, [512], [2600], 64),
    (128, 64, 256, [700, 1, 0, 790], [30, 2000, 5, 600], 128),
    (64, 64, 0, [2100], [100], 64),
    (64, 32, 300, [2100], [0], 64),
]


@pytest.mark.parametrize("hd,dr,window,new,held,H", LARGE)
def test_expanded_tiles(hd, dr, window, new, held, H):
    say(f"[gpu] expanded tiles H={H} {hd}+{dr} window={window} {new} {held}")
    c = Expanded(np.random.default_rng(35), new, held, H, hd, dr, window)
    c.run()
    c.check(heads=[0, H // 2, H - 1], tokens=[0, 1, 15, 16, 63, 64, 127, 128, 200, 249, 255, 256, 257, 500, 511, 699, 789, 1024, 2099])
    first = c.out.clone()
    c.run()
    assert torch.equal(first, c.out)


@pytest.mark.parametrize("hd", [64, 128])
def test_expanded_tiles_with_scores_that_grow(hd):
    say(f"[gpu] expanded tiles, growing scores {hd}")
    n = 2100 if hd == 64 else 512
    c = Expanded(np.random.default_rng(36), [n], [300], 128, hd, 32)
    c.kv[:, :, :hd] = c.kv[:, :, :hd].abs() * (0.02 * 251 / (n + 300) * torch.arange(n + 300, dtype=torch.float32))[:, None, None].bfloat16()
    c.q = c.q.abs()
    c.run()
    c.check(heads=[0, 77], tokens=[0, 100, 255, 256, 300, 511, 2099])


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("hd,n,held", [(128, 512, 200), (64, 2100, 30)])
def test_expanded_tiles_do_not_look_at_what_is_masked(hd, n, held, window):
    say(f"[gpu] expanded tiles, values that are not finite {hd} window={window}")
    H = 128
    c = Expanded(np.random.default_rng(37), [n], [held], H, hd, 64, window)
    bad = n - 150  # this token's key and value rows are not finite, and the value of the token three behind
    c.kv[held + bad, :, 3] = math.nan
    c.kv[held + bad, :, hd + 9] = math.inf
    c.kv[held + bad + 3, :, hd:] = math.nan
    c.run()
    assert torch.isfinite(c.out[:bad].float()).all() and torch.isfinite(c.lse[:n][:bad]).all()
    assert torch.isnan(c.out[bad].float()).any(-1).all() and torch.isnan(c.lse[bad]).all()
    tokens = np.array([0, bad // 2, bad - 70, bad - 20, bad - 2, bad - 1])
    if window:  # and those that have passed it
        tokens = np.concatenate([tokens, [bad + 3 + window, n - 1]])
        assert torch.isfinite(c.out[bad + 3 + window: n].float()).all()
    kv, rope, q = np.nan_to_num(c.kv.double().numpy(), posinf=0.0), c.rope.double().numpy(), c.q.double().numpy()
    for head in (0, 99):
        k = np.concatenate([kv[:, head, :hd], rope], 1)
        o, l, do, dl = attend_ref(q[tokens, head], k, kv[:, head, hd:], held + tokens, np.arange(held + n), c.scale, window)
        near(c.out[torch.from_numpy(tokens), head], o, do)
        near(c.lse[torch.from_numpy(tokens), head], l, dl)


def test_expanded_tiles_of_rows_at_the_ends():
    """Fewer rows than positions, none, and rows that end at the tensor's end."""
    say("[gpu] expanded tiles: rows of the last positions only")
    c = Expanded(np.random.default_rng(38), [250] * 8, [100, 0, 30, 10, 500, 64, 0, 9], 64, 128, 64, lens=[350, 100, 0, 260, 400, 5, 250, 200])
    c.run()
    c.check(heads=[0, 63])
    assert (c.out[500:750] == 0).all() and (c.lse[500:750] == -math.inf).all()
