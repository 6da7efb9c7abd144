"""The scale of latent attention (CPU): times log2 e it has to stay in fp32, or scores of zero would be NaN."""
import math

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402


@pytest.mark.parametrize("scale,status", [(0.0, 0), (1e-45, 0), (-1.0, 0), (2.0 ** 126, 0), (-(2.0 ** 126), 0), (1.7e38, 0), (2.0 ** 127, -2),
                                          (-(2.0 ** 127), -2), (3.4e38, -2), (math.inf, -2), (-math.inf, -2), (math.nan, -2)])
def test_scales(scale, status):
    lay = eg.make_latent_layout(4, 128, 32, scale=scale)
    assert eg.engram_latent_layout_check(lay) == status
    assert (eg.engram_latent_row_bytes(lay) > 0) == (status == 0)
