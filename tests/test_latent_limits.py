"""Sizes past what a launch can hold (CPU): refused, not cut."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402
from test_latent_checks import ACCEPTED, expanded  # noqa: E402


def call(heads, n, R):
    lay = eg.make_latent_layout(heads, 128, 32, head_dim=64)
    return expanded(lay=ctypes.byref(lay), qs=heads * 96, ks=heads * 128, os=heads * 64, n=n, r=R)


@pytest.mark.parametrize("heads,n,R", [(1024, 1 << 20, 4096), (1024, 786_432, 4096), (1024, 1 << 20, 1), (256, 1 << 22, 4096), (1, 1 << 30, 1)])
def test_expanded_attention_refuses_launches_of_2_to_the_32_threads(heads, n, R):
    assert (n // 64 + R) * heads >= 1 << 24 and n * heads <= 1 << 30
    assert call(heads, n, R) == -3


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on made-up pointers")
@pytest.mark.parametrize("heads,n,R", [(1024, 786_432, 4095), (1024, (1 << 20) - 128, 1), (1, (1 << 30) - 128, 1), (1024, 100, 4096)])
def test_and_takes_those_below(heads, n, R):
    assert call(heads, n, R) in (ACCEPTED, -6)
