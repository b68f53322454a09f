"""The kernels of sorted slots, the exchange and the adapters compile without scratch, but for outer products of ranks above
64, whose workgroups of 1024 threads leave 128 registers: they keep a few values of the loads to come there."""

import tempfile
from pathlib import Path

import pytest

from test_kernel_resources import HIPCC, _resources


@pytest.mark.skipif(not Path(HIPCC).exists(), reason="hipcc not available")
@pytest.mark.parametrize("source", ["sort_slots.hip", "exchange.hip", "adapters.hip"])
def test_no_scratch(source):
    with tempfile.TemporaryDirectory() as d:
        kernels = {k: v for k, v in _resources(source, d).items() if "kernel" in k}
    assert kernels
    for k, v in kernels.items():
        assert v.get("ScratchSize", 0) <= (64 if "outer_kernel" in k and "Li8E" in k else 0), k
