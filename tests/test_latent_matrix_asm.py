"""Matrix instructions of the latent kernels are the compiler's own (CPU, source only): it knows how long their results take, and
puts the waits before whatever reads them, its own register copies among them.  Inline assembly that issues one, or that
reads accumulation registers, would leave that to the code around it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hashed_gram_engram_amd", "csrc")
SOURCES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "latent*")))


@pytest.mark.parametrize("name", SOURCES)
def test_no_matrix_instruction_in_assembly(name):
    text = open(os.path.join(CSRC, name)).read()
    assert "v_mfma" not in text
    assert not re.search(r'"[=+&]*a"\s*\(', text)


def test_there_are_sources():
    assert "latent_absorbed_rows.hip" in SOURCES and "latent_expanded.hip" in SOURCES
