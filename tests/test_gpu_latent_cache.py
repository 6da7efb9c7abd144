"""The latent cache on the GPU: rows written and read back, bit for bit, against a plain search for codes and scales."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from gpu_common import eg, say  # noqa: E402
from latent_common import Step, bits_bf16, cache_on, make_rows, row_bytes, row_values  # noqa: E402


def normal(rng, *shape, std=1.0):
    return torch.from_numpy(rng.normal(0, std, shape).astype(np.float32)).bfloat16()


def layout(dc, dr, fp8, **kw):
    return eg.make_latent_layout(4, dc, dr, cache_format=eg.CACHE_MXFP8 if fp8 else eg.CACHE_BF16, **kw)


def as_bytes(cache):
    return cache.contiguous().view(torch.uint8).cpu().numpy().reshape(cache.shape[0] * cache.shape[1], -1)


CASES = [(512, 64, True, 16, [3, 0, 1, 20], [5, 9, 31, 0]), (512, 32, True, 24, [1, 7], [40, 0]), (256, 64, True, 1, [5], [3]),
         (128, 32, True, 64, [70, 1, 1], [0, 64, 63]), (512, 64, False, 16, [9, 33], [16, 1]), (256, 32, False, 7, [2, 2, 2], [0, 5, 6]),
         (128, 64, False, 256, [1], [0])]


@pytest.mark.parametrize("dc,dr,fp8,block,new,held", CASES)
def test_rows_written_and_read_back(dc, dr, fp8, block, new, held):
    say(f"[gpu] latent cache {dc} + {dr} fp8={fp8} block={block}")
    rng = np.random.default_rng(dc + dr + block)
    st = Step(new, held, block, rng, max_tokens=sum(new) + 3)
    old = rng.integers(0, 256, (st.n_blocks * block, row_bytes(dc, dr, fp8)), dtype=np.uint8)
    if fp8:
        old[:, dc: dc + 16] = rng.integers(100, 140, (len(old), 16))
    cache = cache_on(old.copy(), dc, dr, fp8, st)
    wide = normal(rng, st.T, dc + dr + 8, std=3.0)
    lay, pages, plan = layout(dc, dr, fp8), st.pages(eg), st.plan(eg)
    dev = wide.cuda()
    back = eg.engram_latent_write(lay, pages, dev[:, :dc], dev[:, dc: dc + dr], plan, cache)
    assert back is cache
    want = old.copy()
    live = st.slots >= 0
    want[st.slots[live]] = make_rows(bits_bf16(wide[:, :dc]), bits_bf16(wide[:, dc: dc + dr]), fp8)[live]
    got = as_bytes(cache)
    if fp8:  # the scale field's bytes past the last scale are not looked at
        want[:, dc + dc // 32: dc + 16] = got[:, dc + dc // 32: dc + 16]
    assert np.array_equal(got, want)

    # back: the requests with tokens, one after the other; rows behind the last keep what they held
    lens = [n + h if n else 0 for n, h in zip(new, held)]
    rows = sum(lens)
    lat, rope = torch.full((rows + 2, dc), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((rows + 2, dr), 7.0, dtype=torch.bfloat16, device="cuda")
    l2, r2, first = eg.engram_latent_read(lay, pages, cache, plan, st.table_on(), rows + 2, latent=lat, rope=rope)
    assert l2 is lat and r2 is rope
    assert first.cpu().tolist() == [0, *np.cumsum(lens)]
    slots = np.concatenate([st.slot_list(r, 0, n) for r, n in enumerate(lens)])
    lv, rv = row_values(want[slots], dc, fp8)
    for name, g, w in (("latent", lat, lv), ("rope", rope, rv)):
        g = g.double().cpu().numpy()
        assert np.array_equal(g[:rows], w, equal_nan=True), name
        assert (g[rows:] == 7.0).all()


def test_every_bf16_value_is_quantised_to_the_nearest_code():
    """All 65,536 patterns, in blocks whose largest magnitude takes every exponent, and not-finite ones among them."""
    say("[gpu] latent cache: every bf16 value")
    bits = np.arange(65536, dtype=np.uint32).astype(np.uint16).reshape(-1, 512)
    rng = np.random.default_rng(0)
    mixed = rng.integers(0, 65536, (40, 512)).astype(np.uint16)          # any exponents together
    near = (rng.integers(0, 65536, (60, 16, 32)) & 0x83FF | rng.integers(0, 250, (60, 16, 1)) << 7).astype(np.uint16).reshape(60, 512)
    allz = np.zeros((2, 512), np.uint16)
    allz[1] = 0x8000
    full = np.full((1, 512), 0x7F80, np.uint16)                          # nothing finite
    bits = np.concatenate([bits, mixed, near, allz, full])
    n = len(bits)
    st = Step([n], [0], 16, rng)
    lay, pages, plan = layout(512, 64, True), st.pages(eg), st.plan(eg)
    cache = eg.make_latent_cache(lay, pages)
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    rope = torch.from_numpy(rng.integers(-32768, 32768, (n, 64)).astype(np.int16)).cuda().view(torch.bfloat16)
    eg.engram_latent_write(lay, pages, x, rope, plan, cache)
    want = make_rows(bits, bits_bf16(rope.cpu()), True)
    got = as_bytes(cache)[st.slots]
    lat = got[:, :512].copy()
    lat[(lat & 0x7F) == 0x7F] = 0x7F  # a NaN code's sign says nothing
    assert np.array_equal(lat, want[:, :512])
    assert np.array_equal(got[:, 512:], want[:, 512:])
    back, rb, _ = eg.engram_latent_read(lay, pages, cache, plan, st.table_on(), n)
    assert np.array_equal(back.double().cpu().numpy(), row_values(want, 512, True)[0], equal_nan=True)
    assert np.array_equal(bits_bf16(rb), bits_bf16(rope))


def test_every_scale_byte_reads_as_its_power_of_two():
    say("[gpu] latent cache: every scale byte and code")
    rng = np.random.default_rng(1)
    st = Step([256], [0], 32, rng)
    lay, pages, plan = layout(256, 32, True), st.pages(eg), st.plan(eg)
    rows = np.zeros((st.n_blocks * 32, row_bytes(256, 32, True)), np.uint8)
    for b in range(256):
        rows[st.slots[b], :256] = np.arange(256)
        rows[st.slots[b], 256: 264] = b
    back, _, _ = eg.engram_latent_read(lay, pages, cache_on(rows, 256, 32, True, st), plan, st.table_on(), 256)
    lv = row_values(rows[st.slots], 256, True)[0]
    want = torch.from_numpy(lv).to(torch.float32).to(torch.bfloat16)  # (a code times 2^-127 is exact in fp32; past bf16, rounded)
    assert np.array_equal(back.float().cpu().numpy(), want.float().numpy(), equal_nan=True)


@pytest.mark.parametrize("fp8", [False, True])
def test_requests_are_chosen_by_their_tokens_and_cut_at_max_rows(fp8):
    say("[gpu] latent read: min_tokens, window, max_rows, bad pages")
    rng = np.random.default_rng(2)
    new, held = [1, 6, 0, 4, 9], [30, 3, 12, 0, 21]
    st = Step(new, held, 8, rng)
    dc, dr = 128, 32
    rows = make_rows(rng.integers(0x3C00, 0x4200, (st.n_blocks * 8, dc)).astype(np.uint16), rng.integers(0x3C00, 0x4200, (st.n_blocks * 8, dr)).astype(np.uint16), fp8)
    cache = cache_on(rows, dc, dr, fp8, st)
    pages, plan, table = st.pages(eg), st.plan(eg), st.table_on()

    def read(max_rows, min_tokens, window=0, table=table):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        lat = torch.full((max_rows, dc), -3.0, dtype=torch.bfloat16, device="cuda")
        lat, rope, first = eg.engram_latent_read(layout(dc, dr, fp8, window=window), pages, cache, plan, table, max_rows, min_tokens=min_tokens, latent=lat, err_count=err)
        return lat.double().cpu().numpy(), first.cpu().tolist(), int(err)

    def values(spans):
        s = np.concatenate([st.slot_list(r, lo, hi) for r, lo, hi in spans])
        return row_values(rows[s], dc, fp8)[0]

    lat, first, err = read(100, 4)
    assert first == [0, 0, 9, 9, 13, 43] and err == 0
    assert np.array_equal(lat[:43], values([(1, 0, 9), (3, 0, 4), (4, 0, 30)])) and (lat[43:] == -3).all()
    # a window: from the first position that the first new token sees
    lat, first, err = read(100, 1, window=5)
    assert first == [0, 5, 14, 14, 18, 31] and err == 0
    assert np.array_equal(lat[:31], values([(0, 26, 31), (1, 0, 9), (3, 0, 4), (4, 17, 30)]))
    # the second does not fit, so that the smaller ones behind it wait too
    lat, first, err = read(39, 1)
    assert first == [0, 31, 31, 31, 31, 31] and err == 3
    assert np.array_equal(lat[:31], values([(0, 0, 31)])) and (lat[31:] == -3).all()
    lat, first, err = read(40, 1)
    assert first == [0, 31, 40, 40, 40, 40] and err == 2
    lat, first, err = read(0, 1)
    assert first == [0] * 6 and err == 4
    # pages outside the pool
    bad = st.table.copy()
    bad[0, 1], bad[4, 0] = st.n_blocks, -1
    lat, first, err = read(100, 1, table=torch.from_numpy(bad).cuda())
    assert err == 16 and first[-1] == 74
    want = values([(0, 0, 31), (1, 0, 9), (3, 0, 4), (4, 0, 30)])
    want[8:16] = 0
    want[44:52] = 0
    assert np.array_equal(lat[:74], want)


def test_slots_outside_the_pool_are_not_written():
    say("[gpu] latent write: slots outside the pool")
    rng = np.random.default_rng(3)
    st = Step([6], [0], 4, rng)
    lay, pages, plan = layout(128, 32, True), st.pages(eg), st.plan(eg)
    guard = torch.full((st.n_blocks + 2, 4, row_bytes(128, 32, True)), 9, dtype=torch.uint8, device="cuda")
    cache = guard[1:-1]
    plan.slots.copy_(torch.tensor([0, -1, st.n_blocks * 4, 2 ** 40, -2 ** 40, 1]))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = normal(rng, 6, 160).cuda()
    eg.engram_latent_write(lay, pages, x[:, :128], x[:, 128:], plan, cache, err_count=err)
    assert int(err) == 2
    assert (guard[0] == 9).all() and (guard[-1] == 9).all() and (guard[1:-1].view(-1, guard.shape[-1])[2:] == 9).all()
    assert not (cache.view(-1, cache.shape[-1])[:2] == 9).all()


def test_a_step_without_tokens_or_requests():
    say("[gpu] latent cache: nothing to do")
    lay, pages = layout(128, 32, False), eg.make_page_layout(4, 2, 3)
    cache = eg.make_latent_cache(lay, pages)
    for R in (0, 2):
        plan = eg.BatchPlan(R, 0)
        x = torch.zeros((0, 160), dtype=torch.bfloat16, device="cuda")
        eg.engram_latent_write(lay, pages, x[:, :128], x[:, 128:], plan, cache)
        table = torch.zeros((R, 2), dtype=torch.int32, device="cuda")
        first = torch.full((R + 1,), 5, dtype=torch.int32, device="cuda")
        eg.engram_latent_read(lay, pages, cache, plan, table, 4, row_start=first)
        assert first.tolist() == [0] * (R + 1)
    assert not cache.any()


def test_many_requests():
    say("[gpu] latent read: 4096 requests")
    rng = np.random.default_rng(4)
    new = rng.integers(0, 3, 4096)
    held = rng.integers(0, 5, 4096)
    st = Step(new, held, 2, rng)
    lay, pages, plan = layout(128, 32, False), st.pages(eg), st.plan(eg)
    rows = rng.integers(0x3C00, 0x4200, (st.n_blocks * 2, 160)).astype(np.uint16).view(np.uint8)
    lens = np.where(new > 0, new + held, 0)
    lat, rope, first = eg.engram_latent_read(lay, pages, cache_on(rows, 128, 32, False, st), plan, st.table_on(), int(lens.sum()))
    assert first.cpu().tolist() == [0, *np.cumsum(lens)]
    slots = np.concatenate([st.slot_list(r, 0, n) for r, n in enumerate(lens)])
    lv, rv = row_values(rows[slots], 128, False)
    assert np.array_equal(lat.double().cpu().numpy(), lv) and np.array_equal(rope.double().cpu().numpy(), rv)
    assert math.isfinite(lv.sum())
