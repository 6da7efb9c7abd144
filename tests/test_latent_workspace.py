"""The workspace of expanded attention that serves steps of every length (CPU: sizes for 256 CUs, host code only)."""
import random

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads", [1, 3, 16, 20, 128, 1024])
def test_enough_for_every_shorter_step(heads, hd):
    lay = eg.make_latent_layout(heads, 512, 64, head_dim=hd)
    rng = random.Random(heads + hd)
    whole = eg.engram_latent_attention_expanded_workspace_bytes_up_to(lay, (1 << 30) // heads, 1 << 30)
    assert 0 < whole <= 256 * 768 * (hd + 2) * 4
    for _ in range(3000):
        n, rows = int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 18))
        R = min(4096, int(2 ** rng.uniform(0, 7)))
        need = eg.engram_latent_attention_expanded_workspace_bytes(lay, R, n, rows)
        assert need <= eg.engram_latent_attention_expanded_workspace_bytes_up_to(lay, n, rows) <= whole, (R, n, rows)


@pytest.mark.parametrize("heads", [1, 16, 128])
def test_it_grows_with_tokens_and_rows(heads):
    lay = eg.make_latent_layout(heads, 512, 64)
    up_to = eg.engram_latent_attention_expanded_workspace_bytes_up_to
    at = [1, 2, 7, 63, 64, 65, 255, 256, 511, 512, 1000, 5000, 8192, 100_000]
    for a, b in zip(at, at[1:]):
        for m in at:
            assert up_to(lay, a, m) <= up_to(lay, b, m) and up_to(lay, m, a) <= up_to(lay, m, b)
    # the longest step's own size is not enough for shorter ones
    exact = eg.engram_latent_attention_expanded_workspace_bytes
    if heads == 16:
        assert exact(lay, 1, 8192, 16_896) == 0 < exact(lay, 1, 512, 16_896) <= up_to(lay, 8192, 16_896)


def test_what_no_call_takes_needs_none():
    up_to = eg.engram_latent_attention_expanded_workspace_bytes_up_to
    lay = eg.make_latent_layout(16, 512, 64)
    assert up_to(lay, 0, 4096) == up_to(lay, -1, 4096) == up_to(lay, 1, -1) == up_to(lay, 1, (1 << 30) + 1) == up_to(lay, 1 << 30, 1) == 0
    assert up_to(lay, 1, 511) == 0 < up_to(lay, 1, 512)
    assert up_to(eg.make_latent_layout(16, 512, 48), 1, 4096) == 0
    assert eg._lib.engram_latent_attention_expanded_workspace_bytes_up_to(None, 1, 4096) == 0
