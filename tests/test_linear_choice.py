"""engram_linear's choice of tile and split (hashed_gram_engram_amd/csrc/linear_choice.h), compiled for the host
(CPU): the shapes of the GPU tests take every tile that a call can take, whole and split over K, and a workspace
sized for all lengths up to a largest one serves each of them."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

pytest.importorskip("torch")

import hashed_gram_engram_amd as eg  # noqa: E402
import test_gpu_linear as lists  # noqa: E402
import test_gpu_linear_tiles as more  # noqa: E402

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hashed_gram_engram_amd", "csrc")
SOURCE = """
#include "linear_choice.h"
extern "C" void choices(int n, const int64_t* M, const int64_t* K, const int64_t* N, int glu, int cus, int64_t* tile,
                        int64_t* parts, int64_t* bytes) {
  for (int i = 0; i < n; ++i) {
    const engram::LinearChoice c = engram::choose(M[i], int(K[i]), int(N[i]), glu != 0, cus);
    tile[i] = c.tile;
    parts[i] = c.parts;
    bytes[i] = c.bytes;
  }
}
"""


@pytest.fixture(scope="module")
def choices(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cc").write_text(SOURCE)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "choice.cc"), "-o",
                    str(d / "choice.so")], check=True)
    fn = ctypes.CDLL(str(d / "choice.so")).choices

    def call(M, K, N, glu, cus=256):
        """Arrays of (tile, parts, workspace bytes)."""
        ins = [np.ascontiguousarray(a, np.int64) for a in np.broadcast_arrays(M, K, N)]
        outs = [np.empty(len(ins[0]), np.int64) for _ in range(3)]

        def p(a):
            return a.ctypes.data_as(ctypes.c_void_p)
        fn(len(ins[0]), *map(p, ins), int(glu), cus, *map(p, outs))
        return outs
    return call


@pytest.mark.parametrize("glu", [False, True])
def test_the_tested_shapes_take_every_tile_whole_and_split(choices, glu):
    tested = lists.SIZES + (lists.GATED_TILES + more.GATED_TILES if glu else lists.TILES + more.TILES)
    tile, parts, _ = choices(*np.array(tested).T, glu)
    have = set(zip(tile.tolist(), (parts > 1).tolist()))
    rng = np.random.default_rng(0)

    def sizes(lo, hi):
        return np.exp(rng.uniform(np.log(lo), np.log(hi), 1_000_000)).round()
    M, K, N = sizes(1, 20000), 8 * sizes(1, 2048), sizes(1, 60000)
    tile, parts, _ = choices(M, K, N, glu)
    reached = {}
    for i, key in enumerate(zip(tile.tolist(), (parts > 1).tolist())):
        reached.setdefault(key, (int(M[i]), int(K[i]), int(N[i])))
    missing = {key: shape for key, shape in reached.items() if key not in have}
    assert not missing, f"(tile, split): a shape that takes it, {missing}"
    assert len(reached) > 25


# (K, N, gated): few and many columns of tiles, K too short to split, one feature
@pytest.mark.parametrize("K,N,glu", [(5120, 5120, False), (10240, 5120, False), (5120, 10240, True), (4096, 17, False), (504, 640, False),
                                     (512, 640, False), (2232, 260, True), (1 << 20, 1, False), (6144, 25600, False)])
def test_a_workspace_for_all_lengths_serves_every_one(choices, K, N, glu):
    lay = eg.make_linear_layout(K, N, glu=glu)
    most = 4096
    each = choices(np.arange(1, most + 1), K, N, glu)[2]
    assert [eg.engram_linear_workspace_bytes(lay, m) for m in (1, 64, 512, most)] == [each[m - 1] for m in (1, 64, 512, most)]
    for M in (1, 16, 17, 64, 511, 512, 1000, most):
        assert eg.engram_linear_workspace_bytes_up_to(lay, M) == each[:M].max(), M
    # past the last length that is split the bound stays where it is
    far = choices(np.arange(1, 110_001), K, N, glu)[2]
    assert eg.engram_linear_workspace_bytes_up_to(lay, 110_000) == far.max()
    assert eg.engram_linear_workspace_bytes_up_to(lay, (1 << 31) - 1) == far.max() and far[98_304:].max() == 0


def test_the_size_for_one_length_is_not_a_size_for_fewer():
    """What engram.h says of 5120 -> 5120: one buffer of the largest step's size is too small for smaller ones."""
    lay = eg.make_linear_layout(5120, 5120)
    for_64, for_512, for_8192 = (eg.engram_linear_workspace_bytes(lay, m) for m in (64, 512, 8192))
    assert 3.8e6 < for_64 < 4e6 and 20e6 < for_512 < 22e6 and for_8192 == 0
    assert eg.engram_linear_workspace_bytes_up_to(lay, 8192) >= for_512


def test_sizes_of_bad_arguments_are_zero():
    lay = eg.make_linear_layout(5120, 5120)
    for M in (0, -1, 1 << 31):
        assert eg.engram_linear_workspace_bytes_up_to(lay, M) == 0
    assert eg.engram_linear_workspace_bytes_up_to(eg.make_linear_layout(5121, 5120), 64) == 0
    assert eg._lib.engram_linear_workspace_bytes_up_to(None, 64) == 0
