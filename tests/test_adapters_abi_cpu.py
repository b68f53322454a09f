"""Sorted slots, the exchange and the adapters without a GPU: what their entry points refuse, on the host, before any
launch, and what they take as an empty call.  No pointer here is ever followed."""

import pytest
import torch

F = 1 << 24  # 16-byte aligned, never dereferenced
NULL, SHAPE, GROUP, DTYPE, ALIGN, ALIAS = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    if not tl.LIB_PATH.exists():
        from gemm_ternary_linear_amd import build
        build.build()
    return tl


def sort(tl, ids=F, T=1000, k=8, E=64, ones=2 * F, off=3 * F, order=4 * F, slots=5 * F, ws=6 * F):
    return tl.lib().ternary_sort_slots(ids, T, k, E, ones, off, order, slots, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 24) + 1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE),
    (dict(ids=0), NULL), (dict(off=0), NULL), (dict(order=0), NULL), (dict(slots=0), NULL), (dict(ws=0), NULL), (dict(T=0, off=0), NULL),
    (dict(ids=F + 2), ALIGN), (dict(ones=2 * F + 1), ALIGN), (dict(off=3 * F + 2), ALIGN), (dict(order=4 * F + 1), ALIGN),
    (dict(slots=5 * F + 2), ALIGN), (dict(ws=6 * F + 8), ALIGN), (dict(order=F + 31996), ALIAS), (dict(slots=4 * F + 31996), ALIAS),
    (dict(ones=F), ALIAS), (dict(off=F + 16), ALIAS), (dict(ws=5 * F + 16), ALIAS), (dict(T=1 << 24, k=32, ws=1 << 60), ALIAS)])
def test_sort_refuses(tl, kw, status):
    assert sort(tl, **kw) == status


def test_sort_workspace(tl):
    f = tl.lib().ternary_sort_slots_workspace
    assert f(0, 8, 64) == 0 and f(64, 1, 512) == 0 and f(1 << 20, 8, 512) > 0
    assert f(-1, 1, 4) == f(5, 0, 4) == f(5, 1, 513) == SHAPE
    assert f(1 << 24, 32, 512) > 0


def dispatch(tl, x=F, dtype=0, T=8, N=256, slots=2 * F, w=3 * F, k=2, R=16, out=4 * F):
    return tl.lib().ternary_dispatch(x, dtype, T, N, slots, w, k, R, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE), (dict(N=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(R=-1), SHAPE),
    (dict(T=1 << 24, N=1 << 15), SHAPE), (dict(R=1 << 30, N=1 << 9), SHAPE),
    (dict(x=0), NULL), (dict(slots=0), NULL), (dict(out=0), NULL), (dict(x=F + 1), ALIGN), (dict(x=F + 2, dtype=2), ALIGN),
    (dict(slots=2 * F + 2), ALIGN), (dict(w=3 * F + 2), ALIGN), (dict(out=4 * F + 1), ALIGN), (dict(out=F + 4094), ALIAS),
    (dict(out=2 * F + 60), ALIAS), (dict(out=3 * F), ALIAS), (dict(T=0, x=0), 0), (dict(N=0, x=0), 0), (dict(R=0, out=0), 0)])
def test_dispatch_refuses(tl, kw, status):
    assert dispatch(tl, **kw) == status


def dispatch_back(tl, g=F, dtype=0, R=16, N=256, slots=2 * F, w=3 * F, T=8, k=2, x=4 * F, add=None, dx=5 * F, dw=6 * F):
    return tl.lib().ternary_dispatch_backward(g, dtype, R, N, slots, w, T, k, x, add, dx, dw, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE), (dict(N=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(R=-1), SHAPE),
    (dict(g=0), NULL), (dict(slots=0), NULL), (dict(dx=0), NULL), (dict(w=0), NULL), (dict(x=0), NULL), (dict(dw=0), NULL),
    (dict(w=0, dw=0), NULL), (dict(g=F + 1), ALIGN), (dict(x=4 * F + 1), ALIGN), (dict(add=7 * F + 1), ALIGN), (dict(dx=5 * F + 1), ALIGN),
    (dict(slots=2 * F + 2), ALIGN), (dict(w=3 * F + 1), ALIGN), (dict(dw=6 * F + 2), ALIGN), (dict(dx=F + 8190), ALIAS), (dict(dx=4 * F), ALIAS),
    (dict(dx=2 * F), ALIAS), (dict(add=5 * F + 2), ALIAS), (dict(add=6 * F), ALIAS), (dict(dw=5 * F + 4092), ALIAS), (dict(dw=3 * F), ALIAS),
    (dict(T=0, slots=0), 0)])
def test_dispatch_backward_refuses(tl, kw, status):
    assert dispatch_back(tl, **kw) == status


def combine_back(tl, g=F, y=2 * F, dtype=0, R=16, N=256, slots=3 * F, w=4 * F, T=8, k=2, dy=5 * F, dw=6 * F):
    return tl.lib().ternary_combine_backward(g, y, dtype, R, N, slots, w, T, k, dy, dw, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE), (dict(N=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(R=-1), SHAPE),
    (dict(g=0), NULL), (dict(y=0), NULL), (dict(slots=0), NULL), (dict(w=0), NULL), (dict(dy=0), NULL), (dict(dw=0), NULL),
    (dict(g=F + 1), ALIGN), (dict(y=2 * F + 1), ALIGN), (dict(slots=3 * F + 1), ALIGN), (dict(w=4 * F + 2), ALIGN), (dict(dy=5 * F + 1), ALIGN),
    (dict(dw=6 * F + 1), ALIGN), (dict(dy=2 * F), ALIAS), (dict(dy=F + 4094), ALIAS), (dict(dw=5 * F), ALIAS), (dict(dw=3 * F), ALIAS),
    (dict(T=0, g=0), 0)])
def test_combine_backward_refuses(tl, kw, status):
    assert combine_back(tl, **kw) == status


def adapters(tl, x=F, dtype=0, T=8, K=256, N=128, rank=64, a=2 * F, b=3 * F, E=4, s=4 * F, off=5 * F, order=6 * F, slots=7 * F, add=None, y=8 * F,
             hidden=9 * F, ws=10 * F):
    return tl.lib().ternary_linear_adapters(x, dtype, T, K, N, rank, a, b, E, s, off, order, slots, add, y, hidden, ws, None)


SHAPES = [(dict(dtype=2), DTYPE), (dict(dtype=-1), DTYPE), (dict(T=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE), (dict(rank=0), SHAPE),
          (dict(rank=129), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE), (dict(K=(1 << 24) + 1), SHAPE), (dict(T=1 << 24, N=1 << 15), SHAPE),
          (dict(E=512, N=1 << 19), SHAPE)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(x=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL), (dict(off=0), NULL), (dict(order=0), NULL), (dict(slots=0), NULL), (dict(y=0), NULL),
    (dict(ws=0), NULL), (dict(x=F + 1), ALIGN), (dict(a=2 * F + 1), ALIGN), (dict(b=3 * F + 1), ALIGN), (dict(s=4 * F + 2), ALIGN),
    (dict(off=5 * F + 2), ALIGN), (dict(order=6 * F + 2), ALIGN), (dict(slots=7 * F + 2), ALIGN), (dict(add=11 * F + 1), ALIGN), (dict(y=8 * F + 1), ALIGN),
    (dict(hidden=9 * F + 8), ALIGN), (dict(ws=10 * F + 8), ALIGN), (dict(y=F + 4094), ALIAS), (dict(y=2 * F), ALIAS), (dict(y=3 * F), ALIAS),
    (dict(y=4 * F), ALIAS), (dict(y=6 * F + 16), ALIAS), (dict(add=8 * F + 2), ALIAS), (dict(add=9 * F), ALIAS), (dict(hidden=8 * F + 2032), ALIAS),
    (dict(hidden=F), ALIAS), (dict(ws=9 * F + 496), ALIAS), (dict(ws=8 * F), ALIAS), (dict(T=0, x=0, ws=0), 0)])
def test_adapters_refuse(tl, kw, status):
    assert adapters(tl, **kw) == status


def back(tl, g=F, x=2 * F, hidden=3 * F, dtype=0, T=8, K=256, N=128, rank=16, a=4 * F, b=5 * F, E=4, s=6 * F, off=7 * F, order=8 * F, slots=9 * F,
         add=None, dx=10 * F, da=11 * F, db=12 * F, ws=13 * F):
    return tl.lib().ternary_linear_adapters_backward(g, x, hidden, dtype, T, K, N, rank, a, b, E, s, off, order, slots, add, dx, da, db, ws, None)


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(g=0), NULL), (dict(x=0), NULL), (dict(hidden=0), NULL), (dict(a=0), NULL), (dict(b=0), NULL), (dict(off=0), NULL), (dict(order=0), NULL),
    (dict(slots=0), NULL), (dict(dx=0), NULL), (dict(da=0), NULL), (dict(db=0), NULL), (dict(ws=0), NULL), (dict(T=0, da=0), NULL), (dict(g=F + 1), ALIGN),
    (dict(x=2 * F + 1), ALIGN), (dict(hidden=3 * F + 4), ALIGN), (dict(a=4 * F + 1), ALIGN), (dict(b=5 * F + 1), ALIGN), (dict(s=6 * F + 2), ALIGN),
    (dict(off=7 * F + 2), ALIGN), (dict(order=8 * F + 1), ALIGN), (dict(slots=9 * F + 1), ALIGN), (dict(add=14 * F + 1), ALIGN), (dict(dx=10 * F + 1), ALIGN),
    (dict(da=11 * F + 2), ALIGN), (dict(db=12 * F + 8), ALIGN), (dict(ws=13 * F + 4), ALIGN), (dict(dx=2 * F), ALIAS), (dict(dx=F + 2046), ALIAS),
    (dict(da=4 * F), ALIAS), (dict(db=11 * F + 32752), ALIAS), (dict(db=5 * F), ALIAS), (dict(ws=12 * F), ALIAS), (dict(ws=3 * F), ALIAS),
    (dict(add=10 * F + 2), ALIAS), (dict(add=11 * F), ALIAS)])
def test_adapters_backward_refuses(tl, kw, status):
    assert back(tl, **kw) == status


def test_adapters_workspaces(tl):
    f, g = tl.lib().ternary_linear_adapters_workspace, tl.lib().ternary_linear_adapters_backward_workspace
    assert f(8, 256, 128, 16, 4) == 0 and f(8, 256, 128, 64, 4) >= 4 * 8 * 64 and f(5000, 256, 128, 16, 4) >= 4 * 5000 * 16
    assert g(8, 256, 128, 16, 4) >= 4 * 8 * 16
    assert f(0, 256, 128, 16, 4) >= 0 and g(0, 256, 128, 16, 4) >= 0
    assert f(8, 0, 128, 16, 4) == g(8, 256, 128, 129, 4) == SHAPE
    assert f(1 << 20, 4096, 4096, 128, 512) > 0 and g(1 << 20, 4096, 4096, 128, 512) > 0


def test_binding_refuses(tl):
    z, i = torch.zeros, torch.int32
    for bad in [(z(4, 2), 8), (z(4, 2, 1, dtype=i), 8), (z(4, 2, dtype=i), 8, z(4, 1)), (z(4, 2, dtype=i), 8, z(4, 2).half()), (z(4, 2, dtype=i), 8)]:
        with pytest.raises(ValueError):
            tl.sort_slots(*bad)
    r = tl.Routing(z(4, 2, dtype=i), z(4, 2), z(9, dtype=i), z(8, dtype=i), z(4, 2, dtype=i))
    x, y = z(4, 32), z(8, 32)
    for f, good, bads in [
            (tl.dispatch, dict(x=x, routing=r), [dict(x=z(5, 32)), dict(x=x.double()), dict(x=z(4)), dict(routing=r._replace(order=z(7, dtype=i))), {}]),
            (tl.dispatch_backward, dict(grad=y, routing=r, x=x, add=x), [dict(grad=x), dict(x=z(4, 31)), dict(x=x.half()), dict(add=z(3, 32)), {}]),
            (tl.combine_backward, dict(grad=x, y=y, routing=r), [dict(grad=y), dict(y=x), dict(y=y.half()), {}])]:
        for bad in bads:  # the last: everything right, but in host memory
            with pytest.raises(ValueError):
                f(**(good | bad))
    h = torch.float16
    r = tl.Routing(z(4, 1, dtype=i), z(4, 1), z(4, dtype=i), z(4, dtype=i), z(4, 1, dtype=i))
    good = dict(x=z(4, 32, dtype=h), a=z(3, 8, 32, dtype=h), b=z(3, 24, 8, dtype=h), routing=r, scale=z(3))
    two = tl.Routing(z(2, 2, dtype=i), z(2, 2), z(4, dtype=i), z(4, dtype=i), z(2, 2, dtype=i))
    bads = [dict(x=z(4, 32)), dict(x=z(4, 31, dtype=h)), dict(a=z(3, 8, 32).bfloat16()), dict(a=z(2, 8, 32, dtype=h)), dict(b=z(3, 24, 7, dtype=h)),
            dict(b=z(24, 8, dtype=h)), dict(scale=z(4)), dict(scale=z(3, dtype=h)), dict(routing=two), dict(routing=r._replace(offsets=z(5, dtype=i))), {}]
    for bad in bads + [dict(add=z(4, 32, dtype=h)), dict(add=z(4, 24)), dict(hidden=z(4, 8, dtype=h)), dict(hidden=z(4, 9))]:
        with pytest.raises(ValueError):
            tl.linear_adapters(**(good | bad))
    good |= dict(grad=z(4, 24, dtype=h), hidden=z(4, 8))
    for bad in bads + [dict(grad=z(4, 32, dtype=h)), dict(hidden=z(4, 9)), dict(add=z(4, 24, dtype=h))]:
        with pytest.raises(ValueError):
            tl.linear_adapters_backward(**(good | bad))
