"""Buffer sizes of the feed-forward operators for sizes that their calls refuse:
an answer that says so, not a product that left 64 bits."""
import pytest

import nvfp4_quantization_precision_gb300 as fos
from nvfp4_quantization_precision_gb300 import build as fos_build

HUGE = [(1 << 62, 32), (1 << 62, 1 << 20), ((1 << 63) - 1, 32), (1 << 40, 1 << 40),
        (32, 1 << 62), ((1 << 30) + 1, 32), (4, (1 << 30) + 32)]


@pytest.fixture(scope="module")
def L():
    fos_build.build()
    return fos.lib()


@pytest.mark.parametrize("rows,cols", HUGE)
def test_refused_sizes_have_no_size(L, rows, cols):
    for layout in (0, 1):
        assert L.fos_scales8_bytes(rows, cols, layout) == -1
    assert L.fos_rms_norm_backward_workspace_bytes(rows, cols) == 0
    assert L.fos_act_backward_workspace_bytes(rows, cols) == 0
    with pytest.raises(ValueError):
        fos.scales8_shape(rows, cols)


def test_largest_sizes(L):
    """The limits of the calls, and the column-wise form of the most rows."""
    assert L.fos_scales8_bytes((1 << 30) - 1, 32, 0) == (1 << 30) - 1
    assert L.fos_scales8_bytes((1 << 30) - 1, 32, 1) == 1 << 32
    assert L.fos_scales8_bytes(32, 1 << 30, 1) == 1 << 32
    assert L.fos_rms_norm_backward_workspace_bytes((1 << 30) - 1, 1024) == 1024 * 1024 * 4
    assert L.fos_act_backward_workspace_bytes((1 << 30) - 1, 1024) == (1 << 23) * 1024 * 4
