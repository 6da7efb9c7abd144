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
