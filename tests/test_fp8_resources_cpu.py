"""The kernels of the 8-bit layers and the experts compile without scratch: register spills inside the
tile kernel's steps also make it wait for every load that is under way."""

import tempfile
from pathlib import Path

import pytest

from test_kernel_resources import HIPCC, _resources

SOURCES = ["fp8_products.hip", "fp8_quantize.hip", "combine.hip"]


@pytest.mark.skipif(not Path(HIPCC).exists(), reason="hipcc not available")
@pytest.mark.parametrize("source", SOURCES)
def test_no_scratch(source):
    with tempfile.TemporaryDirectory() as d:
        kernels = {k: v for k, v in _resources(source, d).items() if "kernel" in k}
    assert kernels
    assert not {k: v for k, v in kernels.items() if v.get("ScratchSize", 0)}
