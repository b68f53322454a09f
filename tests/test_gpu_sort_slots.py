"""sort_slots against its definition: small and large counts on both sides of each kernel's limits."""

import weakref

import numpy as np
import pytest
import torch

import adapters_ref as ar
import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


def check(tl, ids, E, what):
    say(f"sort_slots {what} {ids.shape} E={E}")
    dev = ref.dev(ids)
    r = tl.sort_slots(dev, E)
    for got, want in zip((r.offsets, r.order, r.slots), ar.sort_slots(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want), what
    assert r.ids.data_ptr() == dev.data_ptr() and bool((r.weights == 1).all()) and r.weights.shape == ids.shape


@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (1, 32, 512), (2, 3, 3), (63, 1, 5), (64, 1, 32), (65, 1, 512), (100, 7, 40), (128, 8, 64),
                                   (129, 8, 64), (512, 8, 200), (513, 8, 200), (4096, 1, 33), (4097, 1, 33), (5000, 2, 512), (8192, 8, 256),
                                   (8193, 8, 256), (12000, 8, 300), (16384, 8, 77), (16385, 8, 64), (131073, 1, 17), (262144, 1, 90), (70000, 4, 511)])
def test_sort(tl, T, k, E):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    check(tl, ids, E, "uniform")
    ids[rng.random((T, k)) < 0.2] = -1
    check(tl, np.where(ids % 7 == 3, ids * 1000 + 10 ** 6, ids).astype(np.int32), E, "some none")


@pytest.mark.parametrize("T,k", [(40, 3), (700, 8), (30000, 5)])
def test_sort_repeated_and_extreme(tl, T, k):
    """The same index in every slot, runs of it, one that nothing names; indices at the ends of 32 bits."""
    check(tl, np.full((T, k), 3, np.int32), 9, "one")
    check(tl, np.full((T, k), -1, np.int32), 9, "none")
    runs = (np.arange(T * k) * 37 // (T * k)).reshape(T, k).astype(np.int32)
    check(tl, runs, 37, "runs")
    check(tl, runs[::-1].copy(), 37, "runs, descending")
    ends = np.array([2 ** 31 - 1, -2 ** 31, 0, 511, 512, -1], np.int32)
    check(tl, np.resize(ends, (T, k)), 512, "ends")
    check(tl, np.resize(ends, (T, k)), 1, "one expert")


def test_sort_shapes(tl):
    say("sort_slots shapes")
    ids = torch.tensor([2, -1, 0, 2], dtype=torch.int32, device="cuda")
    r = tl.sort_slots(ids, 3)
    assert r.ids.shape == (4, 1) and r.slots.cpu().tolist() == [[1], [-1], [0], [2]] and r.order.cpu().tolist() == [2, 0, 3, -1]
    w = torch.rand(4, 1, device="cuda")
    assert tl.sort_slots(ids.view(4, 1), 3, w).weights is w
    with pytest.raises(tl.TernaryError):
        tl.sort_slots(ids, 513)
    with pytest.raises(tl.TernaryError):
        tl.sort_slots(ids.view(1, 4).expand(4, 4).contiguous().view(1, 16).repeat(1, 3), 3)


def test_sort_agrees_with_route(tl):
    """Sorting a router's own choice again gives its own places, and combine takes the result."""
    say("sort_slots after route")
    for T in (5, 300, 9000):
        logits = torch.randn(T, 40, device="cuda")
        logits[T // 2] = -torch.inf
        r = tl.route(logits, 4)
        s = tl.sort_slots(r.ids, 40, r.weights)
        assert all(torch.equal(a, b) for a, b in zip(r, s))


def test_sort_captured(tl):
    """Captured once, replayed on other indices, with eager calls and another stream in between; the workspace is held
    until the launches are enqueued."""
    say("sort_slots captured")
    for T, k, E in ((50, 1, 20), (20000, 8, 100)):
        ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda")
        tl.sort_slots(ids, E)
        torch.cuda.synchronize()
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g):
            r = tl.sort_slots(ids, E)
        for rep in range(4):
            ids.copy_(torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda"))
            side.wait_stream(torch.cuda.current_stream())
            g.replay()
            with torch.cuda.stream(side):
                other = tl.sort_slots(ids, E)
            torch.cuda.synchronize()
            want = tl.sort_slots(ids, E)
            assert all(torch.equal(a, b) for a, b in zip(r, want)) and all(torch.equal(a, b) for a, b in zip(other, want)), rep


def test_sort_holds_its_workspace(tl, monkeypatch):
    say("sort_slots workspace")
    made, alive, make, call = [], [], tl._workspace, tl._call

    def recording(*a):
        t = make(*a)
        made.append(weakref.ref(t))
        return t

    def checked(name, *a):
        alive.extend(r() is not None for r in made)
        return call(name, *a)

    monkeypatch.setattr(tl, "_workspace", recording)
    monkeypatch.setattr(tl, "_call", checked)
    tl.sort_slots(torch.zeros(9000, 8, dtype=torch.int32, device="cuda"), 5)
    assert alive == [True]
