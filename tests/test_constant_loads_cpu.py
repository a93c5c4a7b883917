"""Loads that promise constant data (ld.global.nc), read from the kernels' source: a
kernel starts while the one before it still runs and may be writing what it reads,
so its data is not constant, and a line that L1 kept from before the wait would be
old.  The row segments' loads alone are of this kind, whose lines L1 does not keep."""
import os
import re

from nvfp4_quantization_precision_gb300 import build as fos_build

FILES = sorted(f for f in os.listdir(fos_build.CSRC) if f.endswith((".cu", ".cuh")))


def _text(name):
    with open(os.path.join(fos_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_constant_loads_keep_no_lines():
    seen = 0
    for name in FILES:
        for load in re.findall(r"ld\.global[\w.:]*\.nc[\w.:]*", _text(name)):
            seen += 1
            assert name == "fos_device.cuh" and ".L1::no_allocate" in load, (name, load)
    assert seen  # what the pattern looks for is there
