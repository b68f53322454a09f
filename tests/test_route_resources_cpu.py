"""The routing kernels compile without scratch: a wave's choice is a chain of dependent steps, and spills would lengthen each."""

import tempfile
from pathlib import Path

import pytest

from test_kernel_resources import HIPCC, _resources


@pytest.mark.skipif(not Path(HIPCC).exists(), reason="hipcc not available")
def test_route_no_scratch():
    with tempfile.TemporaryDirectory() as d:
        kernels = {k: v for k, v in _resources("route.hip", d).items() if "kernel" in k}
    assert len(kernels) >= 27  # three types by four widths, for few tokens and for many, and three that place
    assert not {k: v for k, v in kernels.items() if v.get("ScratchSize", 0)}
