"""How the feed-forward operators' kernels load what the kernel before them may have
written, read from their source: they start while it still runs and wait for it,
and __ldg promises data that is constant from the start on, which the compiler
may use to move the load past the wait."""
import os
import re

from nvfp4_quantization_precision_gb300 import build as fos_build

KERNELS = ["fos_norm.cuh", "fos_quant8.cuh", "fos_linear.cuh", "fos_linear_pair.cuh", "norm.cu",
           "quant8.cu", "linear.cu"]


def _text(name):
    with open(os.path.join(fos_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_load_may_pass_the_wait():
    for name in KERNELS + ["fos_block8.cuh", "fos_act.cuh"]:
        assert "__ldg" not in _text(name), name


def test_every_kernel_waits_before_its_first_load():
    """chain_wait is the first call of every kernel, but for the products', which set
    their barriers up first and touch no tensor in it."""
    for name in KERNELS:
        for kernel in re.findall(r"__global__[^;{]*\)\s*\{(.*?)\n\}", _text(name), flags=re.S):
            before = kernel.split("chain_wait();")[0]
            assert before != kernel
            assert not re.search(r"a\.(x|w|h|dy|dh|rstd|part|sf\w|ep)\b|tma_load|bulk_load", before), before
