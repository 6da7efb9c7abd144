"""engram_linear on the tiles that test_gpu_linear's lists leave out, exact on whole numbers as there: the plain
256 x 128 tile over all of K, and the gated 256 x 256 tile with K in two, three and four parts (its join has a
mapping of waves to the tile of its own).  tests/test_linear_choice.py holds the lists against the choice."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_linear as lists  # noqa: E402

TILES = [(17237, 568, 329)]
GATED_TILES = [(235, 5544, 10839), (1640, 11624, 6515), (194, 8056, 5637)]


@pytest.mark.parametrize("M,K,N,gated", [(*s, False) for s in TILES] + [(*s, True) for s in GATED_TILES])
def test_exact_on_whole_numbers(M, K, N, gated):
    lists.test_exact_on_whole_numbers(M, K, N, (gated,))
