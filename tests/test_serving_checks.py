"""The serving operators' refusals (CPU, no GPU call): layouts, then what each entry point says to missing,
misaligned, overlapping and wrongly shaped arguments before any device work; and the scalar plan of the GPU
tests against hand-worked steps."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402
from serving_common import plan_ref  # noqa: E402

LIB = eg._lib
P = ctypes.c_void_p(1 << 12)
ODD = ctypes.c_void_p((1 << 12) + 2)
HALF = ctypes.c_void_p((1 << 12) + 8)


def bad_fields(make, check, changes):
    assert check(ctypes.byref(make())) == 0
    assert check(None) == -1
    for change in changes:
        lay = make()
        for k, v in change.items():
            setattr(lay, k, v)
        assert check(ctypes.byref(lay)) == -2, change


def test_layout_checks():
    bad_fields(lambda: eg.make_page_layout(16, 64, 1000), LIB.engram_page_layout_check,
               [dict(block_size=0), dict(block_size=-4), dict(max_blocks=0), dict(n_blocks=0), dict(n_blocks=(1 << 30) + 1),
                dict(block_size=1 << 20, max_blocks=1 << 11)])
    bad_fields(lambda: eg.make_norm_layout(4, 5120), LIB.engram_norm_layout_check,
               [dict(hc=0), dict(hc=65), dict(dim=0), dict(dim=12), dict(dim=40968), dict(y_streams=2), dict(stream_format=2),
                dict(gate=3), dict(gate=-1), dict(post_norm=2), dict(pre_norm=-1), dict(alpha=float("inf")),
                dict(beta=float("nan")), dict(post_eps=-1.0), dict(pre_eps=float("inf"))])
    bad_fields(lambda: eg.make_linear_layout(5120, 777), LIB.engram_linear_layout_check,
               [dict(in_features=0), dict(in_features=4), dict(in_features=1004), dict(in_features=(1 << 20) + 8),
                dict(out_features=0), dict(out_features=(1 << 24) + 1), dict(activation=6), dict(activation=-1), dict(glu=2),
                dict(stream_format=-1)])


def plan_out(**over):
    out = eg._PlanOut(*[(i + 2) << 12 for i in range(9)])
    for k, v in over.items():
        setattr(out, k, v)
    return out


def test_plan_refusals():
    lay = eg.make_page_layout(16, 4, 10)
    ins = [ctypes.c_void_p((64 + i) << 12) for i in range(5)]

    def call(layout=lay, new=ins[0], held=ins[1], R=3, table=ins[2], free=ins[3], count=ins[4], tokens=8, out=None, err=None):
        return LIB.engram_batch_plan(layout, new, held, R, table, free, count, tokens, plan_out() if out is None else out, err,
                                     None)
    assert call(layout=eg.make_page_layout(0, 4, 10)) == -2
    for bad in (dict(R=-1), dict(R=4097), dict(tokens=-1), dict(tokens=1 << 31)):
        assert call(**bad) == -3, bad
    for bad in ("new", "held", "table", "free", "count"):
        assert call(**{bad: None}) == -1, bad
    for f in eg.BatchPlan.FIELDS:
        assert call(out=plan_out(**{f: None})) == -1, f
        assert call(out=plan_out(**{f: (1 << 12) + (4 if f == "slots" else 2)})) == -4 or f == "live", f
    assert call(err=ODD) == -4 and call(new=ODD) == -4 and call(count=ODD) == -4
    # what the call reads everywhere must not be written in place
    assert call(out=plan_out(seq_lens=65 << 12)) == -3
    assert call(out=plan_out(start_pos=65 << 12)) == -3
    assert call(out=plan_out(free_left=68 << 12)) == -3


def test_hash_refusals():
    hl, pl = eg.make_hash_layout(2, 4, 8, 2, 1000, 16), eg.make_page_layout(16, 4, 10)

    def call(h=hl, p=pl, n=8, R=2, **over):
        names = ["token_map", "multipliers", "primes", "offsets", "input_ids", "mask", "slots", "positions", "requests", "start",
                 "table", "history", "out", "err"]
        a = {k: P for k in names} | dict(mask=None, err=None) | over
        return LIB.engram_hash_ids_paged(h, p, a["token_map"], a["multipliers"], a["primes"], a["offsets"], a["input_ids"],
                                         a["mask"], n, a["slots"], a["positions"], a["requests"], a["start"], R, a["table"],
                                         a["history"], a["out"], a["err"], None)
    assert call(h=None) == -1 and call(p=None) == -1
    assert call(h=eg.make_hash_layout(2, 9, 8, 2, 1000, 16)) == -2 and call(p=eg.make_page_layout(16, 0, 10)) == -2
    assert call(n=-1) == -3 and call(R=-1) == -3
    assert call(n=0, token_map=None, history=None) == 0
    for k in ("token_map", "multipliers", "primes", "offsets", "input_ids", "slots", "positions", "requests", "start", "table",
              "history", "out"):
        assert call(**{k: None}) == -1, k
        assert call(**{k: ODD}) == -4, k
    assert call(err=ODD) == -4


def test_norm_refusals():
    lay = eg.make_norm_layout(2, 64, gate=eg.GATE_TOKEN)

    def call(layout=lay, x=P, y=P, ys=128, gate=P, gs=0, post=P, pre=P, mask=None, B=1, T=3, out=P, h=P):
        return LIB.engram_residual_norm(layout, x, y, ys, gate, gs, post, pre, mask, B, T, out, h, None)
    assert call(layout=eg.make_norm_layout(2, 60)) == -2
    assert call(B=-1) == -3 and call(T=-1) == -3 and call(B=1 << 30, T=1 << 30) == -3 and call(T=1 << 31) == -3
    assert call(B=0, x=None, y=None, out=None) == 0
    for bad in (dict(x=None), dict(y=None), dict(out=None), dict(h=None), dict(gate=None), dict(y=None, out=None, h=None)):
        assert call(**bad) == -1, bad
    assert call(layout=eg.make_norm_layout(2, 64), gate=P) == -1
    assert call(layout=eg.make_norm_layout(2, 64, pre_norm=False, gate=eg.GATE_TOKEN)) == -1
    assert call(layout=eg.make_norm_layout(2, 64, pre_norm=False), gate=None, y=None, out=None, h=None) == -1
    for k in ("x", "y", "post", "pre", "out", "h"):
        assert call(**{k: HALF}) == -4, k
    assert call(gate=ODD) == -4
    assert call(ys=120) == -3 and call(ys=132) == -3
    feat = eg.make_norm_layout(2, 64, gate=eg.GATE_FEATURE)
    assert call(layout=feat, gs=120) == -3 and call(layout=feat, gate=HALF, gs=128) == -4


def test_linear_refusals():
    lay = eg.make_linear_layout(64, 40)

    def call(layout=lay, x=P, xs=64, w=P, b=None, r=None, rs=0, M=3, out=P, os=40):
        return LIB.engram_linear(layout, x, xs, w, b, r, rs, M, out, os, None, 0, None)
    assert call(layout=eg.make_linear_layout(60, 40)) == -2
    assert call(M=-1) == -3 and call(M=1 << 31) == -3 and call(M=0, x=None, w=None, out=None) == 0
    for k in ("x", "w", "out"):
        assert call(**{k: None}) == -1 and call(**{k: HALF}) == -4, k
    assert call(b=HALF) == -4 and call(r=HALF, rs=40) == -4
    assert call(xs=56) == -3 and call(xs=68) == -3 and call(os=39) == -3 and call(r=HALF.__class__(1 << 13), rs=39) == -3
    assert call(xs=(1 << 28) + 8) == -3 and call(os=1 << 60) == -3
    assert call(r=P, rs=48, out=P, os=40) == -3  # in place with another stride


def test_binding_refusals():
    bf, i32 = torch.bfloat16, torch.int32
    lin = eg.make_linear_layout(64, 40)
    x, w = torch.zeros((3, 64), dtype=bf), torch.zeros((40, 64), dtype=bf)
    with pytest.raises(ValueError, match="must be on a GPU"):
        eg.engram_linear(lin, x, w)
    for bad, match in ((dict(x=x.float()), "x has dtype"), (dict(x=x[:, :56]), "x has shape"), (dict(w=w[:39]), "w has shape"),
                       (dict(w=torch.zeros((64, 40), dtype=bf).t()), "w must be contiguous"),
                       (dict(bias=torch.zeros(40, dtype=bf)), "bias has dtype"), (dict(bias=torch.zeros(39)), "bias has shape"),
                       (dict(residual=torch.zeros((3, 40))), "residual has dtype"),
                       (dict(residual=torch.zeros((4, 40), dtype=bf)), "residual has shape"),
                       (dict(out=torch.zeros((3, 80), dtype=bf)[:, ::2]), "out: the last 1"),
                       (dict(x=torch.zeros((2, 5, 64), dtype=bf)[:, :3], out=torch.zeros((2, 3, 40))), "x: the rows"),
                       (dict(out=torch.zeros((3, 40))), "out has dtype")):
        with pytest.raises((ValueError, TypeError), match=match):
            eg.engram_linear(lin, **(dict(x=x, w=w) | bad))
    norm = eg.make_norm_layout(2, 64, gate=eg.GATE_TOKEN)
    x, y = torch.zeros((1, 3, 2, 64), dtype=bf), torch.zeros((1, 3, 2, 64), dtype=bf)
    gate = torch.zeros((1, 3, 2))
    with pytest.raises(ValueError, match="must be on a GPU"):
        eg.engram_residual_norm(norm, x, y, gate=gate)
    for bad, match in ((dict(x=x[0]), "x has shape"), (dict(x=x.float()), "x has dtype"), (dict(gate=None), "gate kind"),
                       (dict(y=y[:, :2]), "y has shape"), (dict(y=y.float()), "y has dtype"), (dict(gate=gate[..., :1]), "gate"),
                       (dict(y=None), "need y"), (dict(out=torch.zeros((1, 3, 2, 64))), "out has dtype"),
                       (dict(post_weight=torch.zeros(64)), "post_weight has shape"),
                       (dict(token_mask=torch.zeros(3, dtype=torch.uint8)), "token_mask has shape"),
                       (dict(token_mask=torch.zeros((1, 3))), "token_mask has dtype")):
        with pytest.raises((ValueError, TypeError), match=match):
            eg.engram_residual_norm(norm, **(dict(x=x, y=y, gate=gate) | bad))
    with pytest.raises(ValueError, match="h needs pre_norm"):
        eg.engram_residual_norm(eg.make_norm_layout(2, 64, pre_norm=False), x, y, h=y)
    pages, plan = eg.make_page_layout(4, 2, 6), eg.BatchPlan(3, 8, device="cpu")
    args = dict(new_lens=torch.zeros(3, dtype=i32), cached_lens=torch.zeros(3, dtype=i32),
                block_table=torch.zeros((3, 2), dtype=i32), free_list=torch.zeros(6, dtype=i32),
                free_count=torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError, match="must be on a GPU"):
        eg.engram_batch_plan(pages, *args.values(), plan)
    for k, v in args.items():
        with pytest.raises(TypeError, match=k):
            eg.engram_batch_plan(pages, *(args | {k: v.long()}).values(), plan)
        with pytest.raises(ValueError, match=k):
            eg.engram_batch_plan(pages, *(args | {k: torch.zeros(7, dtype=i32)}).values(), plan)
    with pytest.raises(AttributeError):
        plan.slots = plan.slots[:5]
    plan, hl = eg.BatchPlan(3, 8, device="cpu"), eg.make_hash_layout(1, 3, 2, 2, 50, 8)
    args = dict(token_map=torch.zeros(50, dtype=i32), multipliers=torch.zeros((1, 3), dtype=torch.int64),
                primes=torch.zeros((1, 2, 2), dtype=torch.int64), offsets=torch.zeros((1, 4), dtype=torch.int64),
                input_ids=torch.zeros(8, dtype=torch.int64), plan=plan, block_table=torch.zeros((3, 2), dtype=i32),
                history=torch.zeros((6, 4), dtype=torch.int64))
    with pytest.raises(ValueError, match="must be on a GPU"):
        eg.engram_hash_ids_paged(hl, pages, **args)
    for k in ("multipliers", "primes", "offsets", "input_ids", "block_table", "history", "token_map"):
        with pytest.raises(ValueError, match=k):
            eg.engram_hash_ids_paged(hl, pages, **(args | {k: args[k][..., :1].contiguous()}))


def test_scalar_plan_by_hand():
    # two pages free (5 on top, then 3); request 0 grows into page 5, 1 is finished and gives back 7, 2 needs two
    table = np.array([[1, 0], [7, 0], [0, 0]], np.int32)
    plan, t, f, errors = plan_ref(2, 2, 8, [2, -1, 3], [1, 1, 0], table, np.array([3, 5, 9, 9, 9, 9, 9, 9]), 2, 6)
    assert f[:3].tolist() == [3, 5, 7]           # the page given back is on top
    assert t.tolist() == [[1, 7], [7, 0], [5, 3]]
    assert plan["token_start"] == [0, 2, 2, 5] and plan["seq_lens"] == [3, 0, 3] and plan["free_left"] == [0]
    assert plan["slots"] == [3, 14, 10, 11, 6, -1] and plan["positions"] == [1, 2, 0, 1, 2, -1] and errors == 0
    # one page too few: the last request is refused, its table untouched
    plan, t, f, errors = plan_ref(2, 2, 8, [2, -1, 3], [1, 1, 0], table, np.array([3, 5, 9, 9, 9, 9, 9, 9]), 1, 6)
    assert plan["status"] == [0, 0, 2] and plan["free_left"] == [1] and t[2].tolist() == [0, 0] and errors == 1


def test_linear_sizes_its_workspace_on_the_tensors_device(monkeypatch):
    """A call refused for want of a workspace asks for the size with the tensors' device current: the size
    follows that device's compute units, not those of the device that happens to be current."""
    current, asked, given = [0], [], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    def size(layout, M):
        asked.append(current[0])
        return 64

    def launch(where, device, fn, *args):
        given.append(args[-1])
        if args[-1] == 0:
            raise eg.EngramError(where, eg.ENGRAM_E_WORKSPACE)

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(eg, "engram_linear_workspace_bytes", size)
    monkeypatch.setattr(eg, "_launch", launch)
    monkeypatch.setattr(eg, "_rows", lambda name, t, lead, row, dtype, device: row[0])
    monkeypatch.setattr(eg, "_tensor", lambda name, t, shape, dtype, device: t.data_ptr())
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16)
    eg.engram_linear(eg.make_linear_layout(8, 4), x, w)
    assert asked == [1] and given == [0, 64] and current == [0]
