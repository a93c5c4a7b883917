"""A slot of scales in shared memory is given back to its TMA producer only behind
the tensor-memory stores that use its values (their completion is waited for):
plain loads before an arrival may be moved behind it."""
import glob
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "nvfp4_quantization_precision_gb300", "csrc")
FILES = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) if "sh.sf_empty" in open(f).read()]


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_slot_is_freed_behind_the_stores(path):
    text = open(path).read()
    frees = [i for i in range(len(text)) if text.startswith("bar_arrive(&sh.sf_empty", i)]
    assert frees
    for free in frees:
        body = text[text.rindex("warp_wait(&sh.sf_full", 0, free):free]
        assert body.index("tmem_st_x16") < body.rindex("tcgen05.wait::st") and "tmem_st_x8" in body


def test_found():
    assert FILES
