"""Refusals of the latent operators (CPU, no GPU call): the library's argument checks through the C entry points,
and the binding's tensor checks."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402
from latent_common import e4m3_values, quantise_row  # noqa: E402

LAY = eg.make_latent_layout(4, 128, 32, head_dim=64)
FP8 = eg.make_latent_layout(4, 128, 32, head_dim=64, cache_format=eg.CACHE_MXFP8)
PAGES = eg.make_page_layout(16, 3, 10)
R, T, ROWS = 2, 5, 9
P, ODD = ctypes.c_void_p(256), ctypes.c_void_p(264)
lib = eg._lib


def test_layouts():
    assert eg.engram_latent_layout_check(LAY) == 0
    assert abs(LAY.scale - 96 ** -0.5) < 1e-7
    for dc in (128, 256, 512):
        for dr in (32, 64):
            assert eg.engram_latent_row_bytes(eg.make_latent_layout(1, dc, dr)) == 2 * (dc + dr)
            assert eg.engram_latent_row_bytes(eg.make_latent_layout(1, dc, dr, cache_format=eg.CACHE_MXFP8)) == dc + 16 + 2 * dr
    for change in (dict(heads=0), dict(heads=1025), dict(latent_dim=64), dict(latent_dim=384), dict(rope_dim=0), dict(rope_dim=48),
                   dict(rope_dim=128), dict(head_dim=96), dict(cache_format=2), dict(cache_format=-1), dict(window=-1),
                   dict(scale=math.nan), dict(scale=math.inf)):
        lay = eg.make_latent_layout(4, 128, 32, head_dim=64)
        for k, v in change.items():
            setattr(lay, k, v)
        assert eg.engram_latent_layout_check(lay) == -2, change
        assert eg.engram_latent_row_bytes(lay) == 0
        assert eg.engram_latent_attention_workspace_bytes(lay) == 0
        assert eg.engram_latent_attention_expanded_workspace_bytes(lay, 1, 1, 1) == 0
    assert lib.engram_latent_layout_check(None) == -1


def test_layout_struct_matches_the_header():
    import os
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "engram.h")).read()
    body = text[:text.index("} engram_latent_layout;")]
    body = body[body.rindex("typedef struct {"):]
    names = [line.split(";")[0].split()[-1] for line in body.splitlines()[1:] if ";" in line.split("/*")[0]]
    assert names == [f for f, _ in eg.LatentLayout._fields_]


def write(lay=LAY, pages=PAGES, latent=P, ls=128, rope=P, rs=32, slots=P, n=T, cache=P, err=None):
    return lib.engram_latent_write(lay, pages, latent, ls, rope, rs, slots, n, cache, err, None)


def read(lay=LAY, pages=PAGES, cache=P, ts=P, sp=P, r=R, table=P, n=T, least=1, rows=ROWS, first=P, latent=P, rope=P, err=None):
    return lib.engram_latent_read(lay, pages, cache, ts, sp, r, table, n, least, rows, first, latent, rope, err, None)


def absorbed(lay=LAY, pages=PAGES, q=P, qs=640, cache=P, ts=P, sp=P, r=R, table=P, n=T, most=0, out=P, os=512, lse=None, ws=P,
             wb=1 << 40, err=None):
    return lib.engram_latent_attention(lay, pages, q, qs, cache, ts, sp, r, table, n, most, out, os, lse, ws, wb, err, None)


def expanded(lay=LAY, q=P, qs=384, kv=P, ks=512, rope=P, rs=32, first=P, rows=ROWS, ts=P, sp=P, r=R, n=T, least=1, out=P, os=256,
             lse=None, ws=P, wb=1 << 40):
    return lib.engram_latent_attention_expanded(lay, q, qs, kv, ks, rope, rs, first, rows, ts, sp, r, n, least, out, os, lse, ws, wb, None)


BAD = eg.make_latent_layout(4, 128, 40)
BAD_PAGES = eg.make_page_layout(0, 3, 10)
ACCEPTED = -7  # (the checks passed: no gfx950 here)


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up pointers")
@pytest.mark.parametrize("call", [write, read, absorbed, expanded])
def test_good_arguments_reach_the_device_query(call):
    assert call() in (ACCEPTED, -6)


@pytest.mark.parametrize("call,change,status", [
    (write, dict(lay=None), -1), (write, dict(lay=BAD), -2), (write, dict(pages=None), -1), (write, dict(pages=BAD_PAGES), -2),
    (write, dict(n=-1), -3), (write, dict(n=1 << 31), -3), (write, dict(latent=None), -1), (write, dict(rope=None), -1),
    (write, dict(slots=None), -1), (write, dict(cache=None), -1), (write, dict(latent=ODD), -4), (write, dict(rope=ODD), -4),
    (write, dict(cache=ODD), -4), (write, dict(slots=ctypes.c_void_p(260)), -4), (write, dict(err=ctypes.c_void_p(258)), -4),
    (write, dict(ls=120), -3), (write, dict(ls=132), -3), (write, dict(rs=31), -3), (write, dict(rs=1 << 32), -3),
    (write, dict(n=0, latent=None, rope=None, slots=None, cache=None), 0),
    (read, dict(lay=None), -1), (read, dict(lay=BAD), -2), (read, dict(pages=BAD_PAGES), -2), (read, dict(cache=None), -1),
    (read, dict(ts=None), -1), (read, dict(sp=None), -1), (read, dict(table=None), -1), (read, dict(first=None), -1),
    (read, dict(latent=None), -1), (read, dict(rope=None), -1), (read, dict(r=-1), -3), (read, dict(r=4097), -3), (read, dict(n=-1), -3),
    (read, dict(least=0), -3), (read, dict(rows=-1), -3), (read, dict(rows=1 << 31), -3), (read, dict(latent=ODD), -4),
    (read, dict(rope=ODD), -4), (read, dict(cache=ODD), -4), (read, dict(ts=ctypes.c_void_p(258)), -4),
    (absorbed, dict(lay=None), -1), (absorbed, dict(lay=BAD), -2), (absorbed, dict(pages=None), -1), (absorbed, dict(r=-1), -3),
    (absorbed, dict(r=4097), -3), (absorbed, dict(n=-1), -3), (absorbed, dict(n=1 << 29), -3), (absorbed, dict(most=-1), -3),
    (absorbed, dict(q=None), -1), (absorbed, dict(cache=None), -1), (absorbed, dict(out=None), -1), (absorbed, dict(ts=None), -1),
    (absorbed, dict(table=None), -1), (absorbed, dict(q=ODD), -4), (absorbed, dict(out=ODD), -4), (absorbed, dict(lse=ctypes.c_void_p(258)), -4),
    (absorbed, dict(qs=639), -3), (absorbed, dict(qs=644), -3), (absorbed, dict(os=504), -3), (absorbed, dict(os=516), -3),
    (absorbed, dict(n=0, q=None, cache=None, out=None), 0), (absorbed, dict(r=0, ts=None, sp=None, table=None), 0),
    (expanded, dict(lay=None), -1), (expanded, dict(lay=BAD), -2), (expanded, dict(least=0), -3), (expanded, dict(rows=-1), -3),
    (expanded, dict(rows=1 << 31), -3), (expanded, dict(kv=None), -1), (expanded, dict(rope=None), -1), (expanded, dict(first=None), -1),
    (expanded, dict(q=None), -1), (expanded, dict(out=None), -1), (expanded, dict(kv=ODD), -4), (expanded, dict(rope=ODD), -4),
    (expanded, dict(qs=380), -3), (expanded, dict(ks=504), -3), (expanded, dict(ks=516), -3), (expanded, dict(rs=24), -3),
    (expanded, dict(os=248), -3), (expanded, dict(n=0), 0), (expanded, dict(r=0, ts=None, sp=None), 0),
])
def test_the_library_refuses(call, change, status):
    assert call(**change) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up pointers")
def test_workspaces_are_asked_for():
    # (the sizes are for 256 CUs where there is no device; the check stands behind the device query)
    assert eg.engram_latent_attention_workspace_bytes(eg.make_latent_layout(128, 512, 64)) > 0
    # many tiles need none, a few tokens over many rows do
    lay = eg.make_latent_layout(16, 512, 64)
    assert eg.engram_latent_attention_expanded_workspace_bytes(lay, 1, 8192, 8192) == 0
    assert eg.engram_latent_attention_expanded_workspace_bytes(lay, 1, 4, 8192) > 0


def tensors(**over):
    bf16 = torch.bfloat16
    d = dict(latent=torch.zeros((T, 128), dtype=bf16), rope=torch.zeros((T, 32), dtype=bf16), plan=eg.BatchPlan(R, T, device="cpu"),
             cache=torch.zeros((10, 16, 160), dtype=bf16), table=torch.zeros((R, 3), dtype=torch.int32),
             q=torch.zeros((T, 4, 160), dtype=bf16), out=None, lse=None, err=None, qx=torch.zeros((T, 4, 96), dtype=bf16),
             kv=torch.zeros((ROWS, 4, 128), dtype=bf16), kr=torch.zeros((ROWS, 32), dtype=bf16), first=torch.zeros(R + 1, dtype=torch.int32), lay=LAY)
    d.update(over)
    return d


CALLS = {
    "write": lambda d: eg.engram_latent_write(d["lay"], PAGES, d["latent"], d["rope"], d["plan"], d["cache"], err_count=d["err"]),
    "read": lambda d: eg.engram_latent_read(d["lay"], PAGES, d["cache"], d["plan"], d["table"], ROWS, latent=d.get("to"), row_start=d.get("start"), err_count=d["err"]),
    "absorbed": lambda d: eg.engram_latent_attention(d["lay"], PAGES, d["q"], d["cache"], d["plan"], d["table"], out=d["out"], lse=d["lse"], err_count=d["err"]),
    "expanded": lambda d: eg.engram_latent_attention_expanded(d["lay"], d["qx"], d["kv"], d["kr"], d["first"], d["plan"], out=d["out"], lse=d["lse"]),
}


@pytest.mark.parametrize("name", CALLS)
def test_host_tensors_stop_at_the_device_check(name):
    with pytest.raises(ValueError, match="must be on a GPU"):
        CALLS[name](tensors())


@pytest.mark.parametrize("name,change,kind,match", [
    ("write", dict(latent=torch.zeros((T, 120), dtype=torch.bfloat16)), ValueError, "latent has shape"),
    ("write", dict(latent=torch.zeros((T + 1, 128), dtype=torch.bfloat16)), ValueError, "latent has shape"),
    ("write", dict(latent=torch.zeros((T, 128))), TypeError, "latent has dtype"),
    ("write", dict(rope=torch.zeros((T, 64), dtype=torch.bfloat16)), ValueError, "rope has shape"),
    ("write", dict(rope=torch.zeros((32, T), dtype=torch.bfloat16).t()), ValueError, "rope: the last"),
    ("write", dict(cache=torch.zeros((10, 16, 161), dtype=torch.bfloat16)), ValueError, "cache has shape"),
    ("write", dict(cache=torch.zeros((10, 16, 160), dtype=torch.uint8)), TypeError, "cache has dtype"),
    ("write", dict(lay=FP8), TypeError, "cache has dtype"),
    ("write", dict(lay=FP8, cache=torch.zeros((10, 16, 160), dtype=torch.uint8)), ValueError, "cache has shape"),
    ("write", dict(err=torch.zeros(1)), TypeError, "err_count"),
    ("read", dict(table=torch.zeros((R, 4), dtype=torch.int32)), ValueError, "block_table has shape"),
    ("read", dict(table=torch.zeros((R, 3), dtype=torch.int64)), TypeError, "block_table has dtype"),
    ("read", dict(to=torch.zeros((ROWS - 1, 128), dtype=torch.bfloat16)), ValueError, "latent has shape"),
    ("read", dict(start=torch.zeros(R, dtype=torch.int32)), ValueError, "row_start has shape"),
    ("absorbed", dict(q=torch.zeros((T, 4, 128), dtype=torch.bfloat16)), ValueError, "q has shape"),
    ("absorbed", dict(q=torch.zeros((T, 4, 160))), TypeError, "q has dtype"),
    ("absorbed", dict(out=torch.zeros((T, 4, 160), dtype=torch.bfloat16)), ValueError, "out has shape"),
    ("absorbed", dict(lse=torch.zeros((T, 5))), ValueError, "lse has shape"),
    ("absorbed", dict(lse=torch.zeros((T, 4), dtype=torch.float64)), TypeError, "lse has dtype"),
    ("expanded", dict(kv=torch.zeros((ROWS, 4, 64), dtype=torch.bfloat16)), ValueError, "kv has shape"),
    ("expanded", dict(kv=torch.zeros((ROWS, 512), dtype=torch.bfloat16)), ValueError, "kv has shape"),
    ("expanded", dict(kr=torch.zeros((ROWS + 1, 32), dtype=torch.bfloat16)), ValueError, "rope has shape"),
    ("expanded", dict(first=torch.zeros(R, dtype=torch.int32)), ValueError, "row_start has shape"),
    ("expanded", dict(qx=torch.zeros((T, 3, 96), dtype=torch.bfloat16)), ValueError, "q has shape"),
])
def test_the_binding_refuses(name, change, kind, match):
    with pytest.raises(kind, match=match):
        CALLS[name](tensors(**change))


@pytest.mark.parametrize("name,arg", [("write", "latent"), ("write", "rope"), ("absorbed", "q"), ("expanded", "kv"), ("expanded", "qx"), ("read", "cache")])
def test_tensors_that_require_grad_are_refused(name, arg):
    d = tensors()
    d[arg] = d[arg].clone().requires_grad_()
    with pytest.raises(ValueError, match="no backward pass"):
        CALLS[name](d)
    with torch.no_grad(), pytest.raises(ValueError, match="must be on a GPU"):
        CALLS[name](d)


def test_the_oracle_of_codes_and_scales():
    """The search that the GPU's rows are held to, at values worked out by hand and against torch's conversion."""
    x = np.zeros(32)
    x[:6] = [448.0, -17.0, 2.0 ** -9, 3 * 2.0 ** -10, math.nan, -math.inf]
    codes, scales = quantise_row(x)
    assert scales[0] == 127
    # 448 is the last code; 17 lies halfway between 16 and 18 and goes to the even code; so does 1.5 2^-9
    assert codes[:6].tolist() == [0x7E, 0x80 | 0x58, 1, 2, 0x7F, 0x7F]
    assert quantise_row(np.full(32, 449.0))[1][0] == 128 and quantise_row(np.zeros(32))[1][0] == 1
    rng = np.random.default_rng(0)
    for _ in range(20):
        x = torch.from_numpy(rng.normal(0, 1, 64)).bfloat16().double().numpy() * 2.0 ** rng.integers(-20, 20)
        codes, scales = quantise_row(x)
        y = torch.from_numpy(x / np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32)).float()
        assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)
        assert (y.abs().view(2, 32).amax(1) <= 448).all() and (y.abs().view(2, 32).amax(1) > 224).all()
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, e4m3_values(), equal_nan=True)


@pytest.mark.parametrize("call,change", [(write, dict(ls=(1 << 28) + 8)), (write, dict(rs=(1 << 28) + 8)), (absorbed, dict(qs=(1 << 28) + 8)),
                                         (absorbed, dict(os=(1 << 28) + 8)), (expanded, dict(ks=(1 << 28) + 8)), (expanded, dict(rs=(1 << 28) + 8))])
def test_strides_are_2_to_the_28_at_most(call, change):
    assert call(**change) == -3
