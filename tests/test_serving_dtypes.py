"""The types that the serving operators' binding takes and refuses (CPU, no GPU call: a tensor that passes the
checks is then refused for not being on a GPU)."""
import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402

I32, I64 = torch.int32, torch.int64


def hash_call(token_map):
    hl, pages, plan = eg.make_hash_layout(1, 3, 2, 2, 50, 8), eg.make_page_layout(4, 2, 6), eg.BatchPlan(3, 8, device="cpu")
    return eg.engram_hash_ids_paged(hl, pages, token_map, torch.zeros((1, 3), dtype=I64), torch.zeros((1, 2, 2), dtype=I64),
                                    torch.zeros((1, 4), dtype=I64), torch.zeros(8, dtype=I64), plan, torch.zeros((3, 2), dtype=I32),
                                    torch.zeros((6, 4), dtype=I64))


def test_token_maps_without_unsigned_types(monkeypatch):
    """torch versions that have no uint32 say what is wrong with a map of another type, as engram_hash_ids does."""
    monkeypatch.delattr(torch, "uint32")
    with pytest.raises(TypeError, match="token_map has dtype torch.int64"):
        hash_call(torch.zeros(50, dtype=I64))
    with pytest.raises(ValueError, match="must be on a GPU"):
        hash_call(torch.zeros(50, dtype=I32))


def test_int16_views_of_bf16_are_taken():
    bf, i16 = torch.bfloat16, torch.int16
    lin = dict(x=torch.zeros((3, 64), dtype=bf), w=torch.zeros((40, 64), dtype=bf), residual=torch.zeros((3, 40), dtype=bf),
               out=torch.zeros((3, 80), dtype=bf)[:, :40])
    four = torch.zeros((1, 3, 2, 64), dtype=bf)
    norm = dict(x=four, y=four, gate=four, out=four, h=four)
    cases = ((eg.engram_linear, eg.make_linear_layout(64, 40), lin),
             (eg.engram_residual_norm, eg.make_norm_layout(2, 64, gate=eg.GATE_FEATURE), norm))
    for call, layout, args in cases:
        for some in [[k] for k in args] + [list(args)]:
            with pytest.raises(ValueError, match="must be on a GPU"):
                call(layout, **(args | {k: args[k].view(i16) for k in some}))
            for wrong in (torch.float16, torch.int32, torch.uint8):
                with pytest.raises(TypeError, match=f"{some[0]} has dtype"):
                    call(layout, **(args | {some[0]: args[some[0]].to(wrong)}))


def test_int16_is_not_taken_for_other_types():
    x, w = torch.zeros((3, 64), dtype=torch.bfloat16), torch.zeros((40, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bias has dtype"):
        eg.engram_linear(eg.make_linear_layout(64, 40), x, w, bias=torch.zeros(40, dtype=torch.int16))
    with pytest.raises(TypeError, match="residual has dtype"):
        eg.engram_linear(eg.make_linear_layout(64, 40, stream_format=eg.STREAM_FP32), x, w,
                         residual=torch.zeros((3, 40), dtype=torch.int16))
