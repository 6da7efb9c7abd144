"""Latent attention on the GPU, absorbed and expanded, against the formulas in 64 bits."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from latent_common import Step, attend_ref, bits_bf16, cache_on, make_rows, near, row_values  # noqa: E402


def normal(rng, *shape, std=1.0):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).bfloat16()


def random_rows(rng, n, dc, dr, fp8, std=1.0):
    """Cache rows of normal latents (as bytes); the codes drawn directly where the search would take long."""
    lat, rope = normal(rng, n, dc, std=std), normal(rng, n, dr, std=std)
    if not fp8 or n <= 300:
        return make_rows(bits_bf16(lat), bits_bf16(rope), fp8)
    out = np.zeros((n, dc + 16 + 2 * dr), np.uint8)
    scale = rng.integers(117, 121, (n, dc // 32))
    x = lat.float() / torch.from_numpy(np.repeat(2.0 ** (scale - 127), 32, 1)).float()
    out[:, :dc] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    out[:, dc: dc + dc // 32] = scale
    out[:, dc + 16:] = bits_bf16(rope).view(np.uint8).reshape(n, -1)
    return out


class Absorbed:
    """A case of absorbed attention: its inputs on the GPU and what has to come out."""

    def __init__(self, rng, new, held, H, dc=128, dr=32, fp8=False, block=16, window=0, max_tokens=0, std=1.0, extra=2, scale=None):
        self.st = Step(new, held, block, rng, max_tokens=sum(new) + extra)
        self.fp8, self.H, self.dc, self.dr, self.window, self.max_tokens = fp8, H, dc, dr, window, max_tokens
        self.rows = random_rows(rng, self.st.n_blocks * block, dc, dr, fp8, std)
        self.q = normal(rng, self.st.T, H, dc + dr)
        self.lay = eg.make_latent_layout(H, dc, dr, head_dim=64, scale=scale, window=window,
                                         cache_format=eg.CACHE_MXFP8 if fp8 else eg.CACHE_BF16)
        self.scale = float(np.float32(self.lay.scale))

    def run(self, **kw):
        st = self.st
        self.out = torch.full((st.T, self.H, self.dc), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((st.T, self.H), 5.0, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.cache = cache_on(self.rows, self.dc, self.dr, self.fp8, st)
        got = eg.engram_latent_attention(self.lay, st.pages(eg), self.q.cuda(), self.cache, st.plan(eg), st.table_on(),
                                         max_tokens=self.max_tokens, out=self.out, lse=self.lse, err_count=self.err, **kw)
        assert got is self.out
        return got

    def check(self, what=""):
        st = self.st
        lat, rope = row_values(self.rows, self.dc, self.fp8)
        both = np.concatenate([lat, rope], 1)
        q = self.q.double().numpy()
        touched = np.zeros(st.T, bool)
        for r in range(st.R):
            a, n, h = int(st.start[r]), st.new[r], st.held[r]
            if n == 0 or (self.max_tokens and n > self.max_tokens):
                continue
            slots = st.slot_list(r, 0, h + n)
            keys = np.where((slots >= 0)[:, None], both[slots], 0.0)
            vals = np.where((slots >= 0)[:, None], lat[slots], 0.0)
            touched[a: a + n] = True
            for head in range(self.H):
                o, l, do, dl = attend_ref(q[a: a + n, head], keys, vals, np.arange(h, h + n), np.arange(h + n), self.scale, self.window, alive=slots >= 0)
                near(self.out[a: a + n, head], o, do, f"{what} request {r} head {head} out")
                near(self.lse[a: a + n, head], l, dl, f"{what} request {r} head {head} lse")
        rest = torch.from_numpy(~touched)
        assert (self.out.cpu()[rest] == 5.0).all() and (self.lse.cpu()[rest] == 5.0).all(), f"{what}: other tokens' rows were written"


# heads, latent, rope, fp8, block, window, new tokens, held tokens
SHAPES = [
    (1, 128, 32, False, 16, 0, [1], [0]),
    (8, 128, 32, False, 16, 0, [1, 1, 1], [0, 62, 63]),
    (16, 512, 64, True, 64, 0, [1, 0, 1], [200, 9, 64]),
    (17, 512, 64, False, 24, 0, [1, 1], [127, 128]),
    (20, 256, 64, True, 1, 0, [2, 3], [70, 5]),
    (32, 512, 32, True, 16, 0, [1, 1], [500, 3]),
    (33, 256, 32, False, 16, 0, [1], [300]),
    (5, 128, 64, True, 256, 0, [13, 1, 40], [0, 90, 20]),
    (128, 512, 64, True, 64, 0, [1, 1], [65, 190]),
    (128, 512, 64, False, 64, 0, [2], [100]),
    (3, 512, 64, False, 16, 0, [70], [30]),
    (16, 512, 64, True, 16, 50, [1, 5], [300, 120]),
    (4, 256, 64, False, 24, 1, [9], [40]),
    (64, 128, 64, False, 16, 64, [3], [128]),
    (7, 512, 32, True, 16, 1000, [4], [30]),
]


@pytest.mark.parametrize("H,dc,dr,fp8,block,window,new,held", SHAPES)
def test_absorbed(H, dc, dr, fp8, block, window, new, held):
    say(f"[gpu] absorbed H={H} {dc}+{dr} fp8={fp8} block={block} window={window} {new} {held}")
    c = Absorbed(np.random.default_rng(H + dc + block), new, held, H, dc, dr, fp8, block, window)
    c.run()
    c.check()
    assert int(c.err) == 0
    first = c.out.clone(), c.lse.clone()
    c.run()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_over_many_ragged_requests(fp8):
    """More units than workgroups, tiles that begin and end inside workgroups, idle requests between."""
    say(f"[gpu] absorbed: 300 ragged requests fp8={fp8}")
    rng = np.random.default_rng(11)
    new, held = (rng.random(300) < 0.7).astype(int), rng.integers(0, 300, 300)
    held[::50] = 2000
    c = Absorbed(rng, new, held, 2, 128, 32, fp8, 16)
    c.run()
    c.check()


def test_absorbed_requests_behind_many_idle_ones():
    say("[gpu] absorbed: 4096 requests, three at work")
    rng = np.random.default_rng(12)
    new, held = np.zeros(4096, int), np.zeros(4096, int)
    for r, n, h in ((5, 1, 700), (2000, 3, 40), (4095, 1, 1)):
        new[r], held[r] = n, h
    c = Absorbed(rng, new, held, 16, 128, 32, False, 16)
    c.run()
    c.check()


def test_absorbed_one_long_request_in_many_parts():
    say("[gpu] absorbed: one request of 20,001 positions")
    c = Absorbed(np.random.default_rng(13), [1], [20_000], 3, 256, 32, True, 64)
    c.run()
    c.check()


def test_absorbed_takes_requests_up_to_max_tokens():
    say("[gpu] absorbed: max_tokens")
    c = Absorbed(np.random.default_rng(14), [1, 9, 2, 3, 1], [40, 7, 100, 3, 0], 8, max_tokens=2)
    c.run()
    c.check()


def test_absorbed_scores_of_any_size():
    """Scores far apart (one key takes all), growing along the keys (the reference maximum moves), equal, and a
    negative scale."""
    say("[gpu] absorbed: large, growing and equal scores")
    rng = np.random.default_rng(15)
    for std, scale in ((6.0, None), (1.0, 0.0), (1.0, -0.1), (0.01, None)):
        c = Absorbed(rng, [1, 2], [400, 130], 16, 128, 32, False, 16, std=std, scale=scale)
        c.run()
        c.check(f"std {std} scale {scale}")
    c = Absorbed(rng, [1], [600], 16, 128, 32, False, 16)
    lat = normal(rng, c.st.n_blocks * 16, 128).float()
    p = np.arange(601)
    lat[c.st.slot_list(0, 0, 601)] *= torch.from_numpy(0.02 * p[:, None]).float()  # later keys score higher
    c.rows = make_rows(bits_bf16(lat.bfloat16()), bits_bf16(normal(rng, len(lat), 32)), False)
    c.q = c.q.abs()
    c.run()
    c.check("growing")


@pytest.mark.parametrize("fp8", [False, True])
def test_absorbed_bad_pages_take_no_part(fp8):
    """Pages outside the pool: all of a request's (nothing is left), its first, one in the middle, its last."""
    say("[gpu] absorbed: pages outside the pool")
    c = Absorbed(np.random.default_rng(16), [1, 1, 1, 2, 1], [30, 200, 200, 200, 10], 16, 128, 32, fp8, 16)
    t = c.st.table
    t[0, :] = -1
    t[1, 0] = c.st.n_blocks
    t[2, 5] = -7
    t[3, 200 // 16] = 2 ** 30
    c.run()
    assert int(c.err) > 0
    assert (c.out[0] == 0).all() and torch.isinf(c.lse[0]).all() and (c.lse[0] < 0).all()
    c.check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window", [0, 9])
def test_absorbed_what_is_masked_is_not_looked_at(fp8, window):
    """Every slot that no visible position has holds NaN; so does the last new token's own row, and another holds
    infinities, which tokens before them must not notice."""
    say(f"[gpu] absorbed: NaN and infinities in masked places fp8={fp8} window={window}")
    rng = np.random.default_rng(17)
    c = Absorbed(rng, [6, 1, 40], [40, 77, 3], 8, 128, 32, fp8, 16, window)
    st = c.st
    seen = np.zeros(len(c.rows), bool)
    for r in range(st.R):
        lo = max(0, st.held[r] + 1 - window) if window else 0
        seen[st.slot_list(r, lo, st.held[r] + st.new[r])] = True
    c.rows[~seen] = 0xFF
    nan_at, inf_at = st.slot_list(0, 45, 46)[0], st.slot_list(2, 30, 31)[0]
    c.rows[nan_at] = 0xFF
    if fp8:
        c.rows[inf_at, 7] = 0x7F
        c.rows[nan_at, 128:136] = 120
    else:
        c.rows[inf_at].view(np.uint16)[7] = 0x7F80
    c.run()
    a = int(st.start[2]) + 27
    assert torch.isfinite(c.out[:5].float()).all() and torch.isfinite(c.out[a - 20: a].float()).all()
    assert torch.isnan(c.out[5].float()).all() and torch.isnan(c.lse[5]).all()
    assert not torch.isfinite(c.out[a, :, 7].float()).any()
    # tokens that see neither: the formula
    lat, rope = row_values(c.rows, 128, fp8)
    both = np.concatenate([lat, rope], 1)
    for r, n in ((0, 5), (1, 1), (2, 27)):
        first, h = int(st.start[r]), st.held[r]
        s = st.slot_list(r, 0, h + n)
        k, v = np.nan_to_num(both[s], nan=0.0), np.nan_to_num(lat[s], nan=0.0)
        for head in range(8):
            o, l, do, dl = attend_ref(c.q[first: first + n, head].double().numpy(), k, v, np.arange(h, h + n), np.arange(h + n), c.scale, window)
            near(c.out[first: first + n, head], o, do, f"request {r}")
            near(c.lse[first: first + n, head], l, dl, f"request {r}")


def test_absorbed_slices_of_wider_rows_and_no_lse():
    say("[gpu] absorbed: strided q and out, no lse, a given workspace")
    c = Absorbed(np.random.default_rng(18), [2, 1], [50, 9], 6, 256, 64, True, 16)
    c.run()
    st = c.st
    wide_q = torch.zeros((st.T, 2, 6, 320), dtype=torch.bfloat16, device="cuda")
    wide_q[:, 1] = c.q.cuda()
    wide_o = torch.full((st.T, 3, 6, 256), 9.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(eg.engram_latent_attention_workspace_bytes(c.lay), dtype=torch.uint8, device="cuda")
    eg.engram_latent_attention(c.lay, st.pages(eg), wide_q[:, 1], c.cache, st.plan(eg), st.table_on(), out=wide_o[:, 1], workspace=ws)
    live = slice(0, int(st.start[-1]))
    assert torch.equal(wide_o[live, 1], c.out[live])
    assert (wide_o[:, 0] == 9).all() and (wide_o[:, 2] == 9).all() and (wide_o[live.stop:] == 9).all()


def test_absorbed_rows_past_4_gib_of_the_cache():
    say("[gpu] absorbed: a cache of 5 GiB, the request's pages at its end")
    rng = np.random.default_rng(19)
    c = Absorbed(rng, [1], [150], 16, 512, 64, True, 64)
    st = c.st
    n_blocks = (5 << 30) // (64 * 656)
    small = cache_on(c.rows, 512, 64, True, st)
    big = torch.zeros((n_blocks, 64, 656), dtype=torch.uint8, device="cuda")
    big[n_blocks - st.n_blocks:] = small
    pages = eg.make_page_layout(64, st.max_blocks, n_blocks)
    table = (st.table_on() + (n_blocks - st.n_blocks)).int()
    c.run()
    out = torch.zeros_like(c.out)
    eg.engram_latent_attention(c.lay, pages, c.q.cuda(), big, st.plan(eg), table, out=out)
    assert torch.equal(out[:1], c.out[:1])
    lat, _, first = eg.engram_latent_read(c.lay, pages, big, st.plan(eg), table, 151)
    assert np.array_equal(lat.double().cpu().numpy(), row_values(c.rows[st.slot_list(0, 0, 151)], 512, True)[0])
    x = normal(rng, st.T, 576).cuda()
    plan = st.plan(eg)
    plan.slots.copy_(torch.where(plan.slots >= 0, plan.slots + (n_blocks - st.n_blocks) * 64, plan.slots))
    eg.engram_latent_write(c.lay, pages, x[:, :512], x[:, 512:], plan, big)
    eg.engram_latent_write(c.lay, st.pages(eg), x[:, :512], x[:, 512:], st.plan(eg), small)
    assert torch.equal(big[n_blocks - st.n_blocks:], small)


# ---------------------------------------------------------------- expanded


class Expanded:
    def __init__(self, rng, new, held, H, hd=64, dr=32, window=0, lens=None, min_tokens=1, extra=2, std=1.0):
        self.st = Step(new, held, 16, rng, max_tokens=sum(new) + extra)
        self.H, self.hd, self.dr, self.window, self.min_tokens = H, hd, dr, window, min_tokens
        st = self.st
        self.lens = lens or [h + n if n >= min_tokens else 0 for n, h in zip(st.new, st.held)]
        self.first = np.concatenate([[0], np.cumsum(self.lens)]).astype(np.int32)
        rows = int(self.first[-1])
        self.q = normal(rng, st.T, H, hd + dr)
        self.kv, self.rope = normal(rng, rows, H, 2 * hd, std=std), normal(rng, rows, dr)
        self.lay = eg.make_latent_layout(H, 128, dr, head_dim=hd, window=window)
        self.scale = float(np.float32(self.lay.scale))

    def run(self, **kw):
        st = self.st
        self.out = torch.full((st.T, self.H, self.hd), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((st.T, self.H), 5.0, device="cuda")
        eg.engram_latent_attention_expanded(self.lay, self.q.cuda(), self.kv.cuda(), self.rope.cuda(), torch.from_numpy(self.first).cuda(),
                                            st.plan(eg), min_tokens=self.min_tokens, out=self.out, lse=self.lse, **kw)
        return self.out

    def check(self, what="", heads=None, tokens=None):
        st = self.st
        q, kv, rope = self.q.double().numpy(), self.kv.double().numpy(), self.rope.double().numpy()
        touched = np.zeros(st.T, bool)
        for r in range(st.R):
            a, n, h, m, f = int(st.start[r]), st.new[r], st.held[r], self.lens[r], int(self.first[r])
            if n == 0 or n < self.min_tokens:
                continue
            touched[a: a + n] = True
            pos = np.arange(n) if tokens is None else np.array([t for t in tokens if t < n])
            for head in heads or range(self.H):
                k = np.concatenate([kv[f: f + m, head, : self.hd], rope[f: f + m]], 1)
                o, l, do, dl = attend_ref(q[a + pos, head], k, kv[f: f + m, head, self.hd:], h + pos, np.arange(h + n - m, h + n), self.scale, self.window)
                near(self.out[a + torch.from_numpy(pos), head], o, do, f"{what} request {r} head {head} out")
                near(self.lse[a + torch.from_numpy(pos), head], l, dl, f"{what} request {r} head {head} lse")
        rest = torch.from_numpy(~touched)
        assert (self.out.cpu()[rest] == 5.0).all() and (self.lse.cpu()[rest] == 5.0).all(), f"{what}: other tokens' rows were written"


@pytest.mark.parametrize("H,hd,dr,window,new,held", [
    (1, 64, 32, 0, [1], [0]),
    (4, 64, 32, 0, [37], [0]),
    (3, 128, 64, 0, [63, 64, 65], [0, 1, 64]),
    (5, 128, 32, 0, [1, 0, 130], [100, 40, 7]),
    (2, 64, 64, 0, [257, 1], [30, 300]),
    (2, 128, 64, 0, [600], [0]),
    (1, 128, 64, 0, [3], [2000]),
    (9, 64, 32, 0, [2], [1500]),
    (3, 128, 64, 50, [200, 5], [100, 400]),
    (2, 64, 64, 1, [70], [5]),
    (2, 128, 32, 300, [290], [1000]),
    (33, 64, 64, 0, [5, 6, 7], [1, 0, 9]),
])
def test_expanded(H, hd, dr, window, new, held):
    say(f"[gpu] expanded H={H} {hd}+{dr} window={window} {new} {held}")
    c = Expanded(np.random.default_rng(H + hd + sum(new)), new, held, H, hd, dr, window)
    c.run()
    c.check()
    first = c.out.clone(), c.lse.clone()
    c.run()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


@pytest.mark.parametrize("hd", [64, 128])
def test_expanded_long_prompts(hd):
    """Tiles of 256 tokens, whole and ragged, with and without tokens held before; some tokens are checked."""
    say(f"[gpu] expanded: prompts of 1500 and 777 tokens, head_dim {hd}")
    c = Expanded(np.random.default_rng(20), [1500, 777], [0, 333], 2, hd, 64)
    c.run()
    c.check(tokens=[0, 1, 15, 16, 63, 64, 255, 256, 257, 511, 700, 776, 1023, 1024, 1300, 1498, 1499])


def test_expanded_takes_requests_from_min_tokens_on():
    say("[gpu] expanded: min_tokens")
    c = Expanded(np.random.default_rng(21), [3, 10, 0, 9, 40], [7, 0, 5, 60, 2], 4, min_tokens=10)
    c.run()
    c.check()


def test_expanded_rows_are_the_last_positions():
    """Fewer rows than positions (a window's read, or a request that got none), and more."""
    say("[gpu] expanded: rows of the last positions only")
    c = Expanded(np.random.default_rng(22), [20, 20, 20, 5], [100, 0, 30, 10], 3, 128, 64, lens=[30, 8, 0, 40])
    c.run()
    c.check()
    assert (c.out[20:32] == 0).all() and (c.lse[20:32] == -math.inf).all()
    assert (c.out[40:60] == 0).all() and (c.lse[40:60] == -math.inf).all()


def test_expanded_without_any_row():
    say("[gpu] expanded: no rows")
    c = Expanded(np.random.default_rng(23), [3], [0], 2, lens=[0])
    c.run()
    assert (c.out[:3] == 0).all() and (c.lse[:3] == -math.inf).all() and (c.out[3:] == 5).all()


@pytest.mark.parametrize("window", [0, 11])
@pytest.mark.parametrize("new,held", [([150], [20]), ([600], [0]), ([20], [900])])
def test_expanded_what_is_masked_is_not_looked_at(window, new, held):
    say(f"[gpu] expanded: NaN and infinities in masked places {new} {held} window={window}")
    rng = np.random.default_rng(24)
    c = Expanded(rng, new, held, 2, 128, 64, window)
    n, h = new[0], held[0]
    bad = n - 7  # its key and value rows are not finite
    c.kv[h + bad, :, 3] = math.nan
    c.kv[h + bad, :, 128 + 9] = math.inf
    c.kv[h + bad + 2, :, 128:] = math.nan
    c.run()
    assert torch.isfinite(c.out[:bad].float()).all() and torch.isfinite(c.lse[:bad]).all()
    assert torch.isnan(c.out[bad].float()).any() and torch.isnan(c.lse[bad]).all()
    kv, rope, q = c.kv.double().numpy(), c.rope.double().numpy(), c.q.double().numpy()
    tokens = np.array(sorted({0, 1, bad // 2, bad - 64, bad - 20, bad - 2, bad - 1} & set(range(bad))))
    for head in range(2):
        k = np.concatenate([kv[: h + bad, head, :128], rope[: h + bad]], 1)
        o, l, do, dl = attend_ref(q[tokens, head], k, kv[: h + bad, head, 128:], h + tokens, np.arange(h + bad), c.scale, window)
        near(c.out[torch.from_numpy(tokens), head], o, do)
        near(c.lse[torch.from_numpy(tokens), head], l, dl)


def test_expanded_slices_of_wider_rows():
    say("[gpu] expanded: strided q, kv, rope and out, no lse")
    c = Expanded(np.random.default_rng(25), [70, 4], [9, 600], 3, 64, 32)
    c.run()
    st = c.st

    def wide(t):
        w = torch.zeros((t.shape[0], 2, *t.shape[1:]), dtype=torch.bfloat16, device="cuda")
        w[:, 1] = t.cuda()
        return w[:, 1]
    out = torch.full((st.T, 3, 3, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    eg.engram_latent_attention_expanded(c.lay, wide(c.q), wide(c.kv), wide(c.rope), torch.from_numpy(c.first).cuda(), st.plan(eg), out=out[:, 1])
    assert torch.equal(out[:74, 1], c.out[:74]) and (out[:, 0] == 9).all() and (out[:, 2] == 9).all() and (out[74:] == 9).all()


def test_expanded_over_many_requests():
    say("[gpu] expanded: 500 ragged requests, idle ones between")
    rng = np.random.default_rng(26)
    new, held = rng.integers(0, 9, 500) * (rng.random(500) < 0.6), rng.integers(0, 40, 500)
    c = Expanded(rng, new, held, 2, 64, 32)
    c.run()
    c.check()


@pytest.mark.parametrize("what", ["absorbed", "expanded"])
def test_captured_and_on_other_streams(what):
    """A captured call replays with new inputs, and calls on two streams at once do not disturb each other."""
    say(f"[gpu] {what}: captured, replayed, on two streams")
    rng = np.random.default_rng(27)
    if what == "absorbed":
        a, b = (Absorbed(rng, [1, 1, 2], h, 16, 128, 32, True, 16) for h in ([700, 30, 5], [3, 900, 64]))
    else:
        a, b = (Expanded(rng, [3, 40], h, 2, 64, 32) for h in ([1500, 7], [30, 800]))
    wants = [c.run().clone() for c in (a, b)]

    def inputs(c):
        st = c.st
        if what == "absorbed":
            args = [c.lay, st.pages(eg), c.q.cuda(), c.cache, st.plan(eg), st.table_on()]
            return lambda out: eg.engram_latent_attention(*args, out=out), args[2]
        args = [c.lay, c.q.cuda(), c.kv.cuda(), c.rope.cuda(), torch.from_numpy(c.first).cuda(), st.plan(eg)]
        return lambda out: eg.engram_latent_attention_expanded(*args, out=out), args[1]
    (fa, qa), (fb, _) = inputs(a), inputs(b)
    outs = [torch.full_like(w, 5.0) for w in wants]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for f, s, o in zip((fa, fb), streams, outs):
            with torch.cuda.stream(s):
                f(o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], wants[0]) and torch.equal(outs[1], wants[1])
    graph, held = torch.cuda.CUDAGraph(), torch.full_like(wants[0], 5.0)
    with torch.cuda.graph(graph):
        fa(held)
    for k in range(4):
        qa.copy_(normal(rng, *qa.shape))
        graph.replay()
        torch.cuda.synchronize()
        eager = torch.full_like(held, 5.0)
        fa(eager)
        fb(outs[1])
        torch.cuda.synchronize()
        assert torch.equal(held, eager) and torch.equal(outs[1], wants[1]), k
