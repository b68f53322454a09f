"""The 8-bit and experts' entry points without a GPU: what they refuse, on the host, before any
launch, and what they take as an empty call.  No pointer here is ever followed."""

import numpy as np
import pytest
import torch

import fp8_ref as ref

F = 1 << 24  # 16-byte aligned, never dereferenced
NULL, SHAPE, GROUP, DTYPE, ALIGN, ALIAS = -1, -2, -3, -4, -5, -6


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    if not tl.LIB_PATH.exists():
        from gemm_ternary_linear_amd import build
        build.build()
    return tl


def quantize(tl, x=F, dtype=0, M=4, K=256, ld=None, block=0, act=0, q=2 * F, s=3 * F):
    ld = (2 * K if act == 1 else K) if ld is None else ld
    return tl.lib().ternary_fp8_quantize(x, dtype, M, K, ld, block, act, q, s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE), (dict(block=2), SHAPE), (dict(act=2), SHAPE),
    (dict(block=1, act=1), SHAPE), (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=(1 << 24) + 1), SHAPE),
    (dict(ld=255), SHAPE), (dict(act=1, ld=511), SHAPE), (dict(x=0), NULL), (dict(q=0), NULL), (dict(s=0), NULL),
    (dict(x=F + 1), ALIGN), (dict(x=F + 2, dtype=2), ALIGN), (dict(q=2 * F + 8), ALIGN), (dict(s=3 * F + 2), ALIGN),
    (dict(q=F + 1024), ALIAS), (dict(s=F + 2044), ALIAS), (dict(s=2 * F + 512), ALIAS),
    (dict(M=2, ld=4096, q=F + 8192), ALIAS),  # inside the second row
    (dict(M=0, x=0, q=0, s=0), 0)])
def test_quantize_refuses(tl, kw, status):
    assert quantize(tl, **kw) == status


def linear(tl, x=F, xs=2 * F, w=3 * F, ws=4 * F, M=4, N=256, K=256, y=5 * F, dtype=0):
    return tl.lib().ternary_fp8_linear(x, xs, w, ws, M, N, K, y, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=192), SHAPE),
    (dict(K=(1 << 20) + 128), SHAPE), (dict(M=(1 << 24) + 1), SHAPE), (dict(x=0), NULL), (dict(xs=0), NULL),
    (dict(w=0), NULL), (dict(ws=0), NULL), (dict(y=0), NULL), (dict(x=F + 8), ALIGN), (dict(w=3 * F + 4), ALIGN),
    (dict(xs=2 * F + 2), ALIGN), (dict(ws=4 * F + 1), ALIGN), (dict(y=5 * F + 8), ALIGN), (dict(y=F + 1008), ALIAS),
    (dict(y=3 * F + 65520), ALIAS), (dict(y=2 * F + 16), ALIAS), (dict(y=4 * F), ALIAS),
    (dict(M=0, x=0, y=0), 0), (dict(N=0, w=0), 0)])
def test_linear_refuses(tl, kw, status):
    assert linear(tl, **kw) == status


def route(tl, l=F, dtype=2, T=100, E=64, bias=None, score=0, groups=1, top_groups=1, k=8, ids=2 * F, w=3 * F,
          off=4 * F, order=5 * F, slots=6 * F, ws=7 * F):
    return tl.lib().ternary_route(l, dtype, T, E, bias, score, groups, top_groups, k, 1, 1.0, ids, w, off, order,
                                  slots, ws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE), (dict(score=2), SHAPE),
    (dict(groups=0), SHAPE), (dict(groups=3), SHAPE), (dict(E=130, groups=65), SHAPE), (dict(groups=4, top_groups=5), SHAPE),
    (dict(top_groups=0), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=4, k=5), SHAPE),
    (dict(groups=16, top_groups=1, k=5), SHAPE), (dict(T=1 << 24, E=512, k=32, ws=1 << 60), ALIAS),
    (dict(l=0), NULL), (dict(ids=0), NULL), (dict(w=0), NULL), (dict(off=0), NULL), (dict(order=0), NULL),
    (dict(slots=0), NULL), (dict(ws=0), NULL), (dict(T=0, off=0), NULL), (dict(l=F + 2), ALIGN), (dict(bias=8 * F + 2), ALIGN),
    (dict(ids=2 * F + 2), ALIGN), (dict(w=3 * F + 1), ALIGN), (dict(off=4 * F + 2), ALIGN), (dict(order=5 * F + 2), ALIGN),
    (dict(slots=6 * F + 2), ALIGN), (dict(ws=7 * F + 8), ALIGN), (dict(ids=F + 16), ALIAS), (dict(order=6 * F + 16), ALIAS),
    (dict(bias=4 * F + 256), ALIAS), (dict(ws=3 * F + 16), ALIAS)])
def test_route_refuses(tl, kw, status):
    assert route(tl, **kw) == status


def test_route_workspace(tl):
    L = tl.lib()
    assert L.ternary_route_workspace(0, 64) == 0 and L.ternary_route_workspace(32, 512) == 0 \
        and L.ternary_route_workspace(64, 64) == 0
    assert L.ternary_route_workspace(65, 64) >= 5 * 64 * 2
    assert L.ternary_route_workspace(-1, 64) == SHAPE and L.ternary_route_workspace(5, 513) == SHAPE
    assert L.ternary_route_workspace(1 << 24, 512) > 0


def experts(tl, x=F, xs=2 * F, n=8, t=3 * F, s=4 * F, E=4, N=256, K=256, g=-1, off=5 * F, order=6 * F, R=16, k=2, rows=0,
            y=7 * F, dtype=0):
    return tl.lib().ternary_linear_experts(x, xs, n, t, s, E, N, K, g, off, order, R, k, rows, y, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(g=64), GROUP), (dict(g=32), GROUP), (dict(g=0), GROUP), (dict(K=130), SHAPE), (dict(K=0), SHAPE),
    (dict(K=384, g=256), SHAPE), (dict(K=260, g=128), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE), (dict(N=-1), SHAPE),
    (dict(R=-1), SHAPE), (dict(R=(1 << 30) + 1), SHAPE), (dict(n=0), SHAPE), (dict(rows=2), SHAPE), (dict(rows=1, n=15), SHAPE),
    (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(x=0), NULL), (dict(xs=0), NULL), (dict(t=0), NULL), (dict(s=0), NULL),
    (dict(off=0), NULL), (dict(order=0), NULL), (dict(y=0), NULL), (dict(x=F + 8), ALIGN), (dict(t=3 * F + 8), ALIGN),
    (dict(s=4 * F + 1), ALIGN), (dict(off=5 * F + 2), ALIGN), (dict(order=6 * F + 1), ALIGN), (dict(y=7 * F + 8), ALIGN),
    (dict(xs=2 * F + 2), ALIGN), (dict(y=F + 1024), ALIAS), (dict(y=2 * F + 48), ALIAS), (dict(y=3 * F + 65520), ALIAS),
    (dict(y=4 * F), ALIAS), (dict(y=5 * F + 16), ALIAS), (dict(y=6 * F + 48), ALIAS),
    (dict(R=0, x=0, y=0), 0), (dict(N=0, t=0), 0), (dict(R=0, n=0), 0)])
def test_experts_refuse(tl, kw, status):
    assert experts(tl, **kw) == status


def combine(tl, y=F, dtype=0, R=16, N=256, slots=2 * F, w=3 * F, T=8, k=2, add=None, out=4 * F):
    return tl.lib().ternary_combine(y, dtype, R, N, slots, w, T, k, add, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), DTYPE), (dict(R=-1), SHAPE), (dict(N=-1), SHAPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE),
    (dict(y=0), NULL), (dict(slots=0), NULL), (dict(w=0), NULL), (dict(out=0), NULL), (dict(y=F + 1), ALIGN),
    (dict(add=5 * F + 1), ALIGN), (dict(out=4 * F + 1), ALIGN), (dict(slots=2 * F + 2), ALIGN), (dict(w=3 * F + 2), ALIGN),
    (dict(out=F + 8190), ALIAS), (dict(out=2 * F), ALIAS), (dict(out=3 * F + 60), ALIAS), (dict(add=4 * F + 2), ALIAS),
    (dict(T=0, slots=0), 0), (dict(N=0, y=0), 0)])
def test_combine_refuses(tl, kw, status):
    assert combine(tl, **kw) == status


def test_binding_refuses(tl):
    f8, z = torch.float8_e4m3fn, torch.zeros
    x, xs, w, ws = z(4, 256).to(f8), z(4, 2), z(300, 256).to(f8), z(3, 2)
    for bad in [dict(x=z(4, 192).to(f8), w=z(300, 192).to(f8)), dict(w=z(300, 128).to(f8)), dict(xs=z(4, 3)), dict(ws=z(2, 2)),
                dict(xs=z(4, 2).double()), dict(x=z(4, 256)), dict(w=z(300 * 256).to(f8)), dict(dtype=torch.float64), {}]:
        a = dict(x=x, xs=xs, w=w, ws=ws, dtype=torch.bfloat16) | bad
        with pytest.raises(ValueError):  # the last: everything right, but in host memory
            tl.fp8_linear(a["x"], a["xs"], a["w"], a["ws"], dtype=a["dtype"])
    for bad in [(z(4, 8).double(),), (z(4),), (z(4, 8), "column"), (z(4, 8), "row", "gelu"), (z(4, 7), "row", "swiglu"),
                (z(4, 0),), (z(4, 8),)]:
        with pytest.raises(ValueError):
            tl.fp8_quantize(*bad)
    for bad in [dict(logits=z(4)), dict(score="tanh"), dict(bias=z(9)), dict(bias=z(8).double()), {}]:
        with pytest.raises(ValueError):
            tl.route(**(dict(logits=z(4, 8), top_k=2) | bad))
    i = torch.int32
    r = tl.Routing(z(4, 2, dtype=i), z(4, 2), z(9, dtype=i), z(8, dtype=i), z(4, 2, dtype=i))
    codes, s = z(8, 2, 1, 1024, dtype=torch.uint8), z(8, 32).half()
    for bad in [dict(x=z(3, 256).to(f8)), dict(x=z(4, 384).to(f8)), dict(K=300), dict(codes=codes[:7]), dict(s=s.float()),
                dict(s=z(8, 32, 3).half()), dict(s=z(8, 33).half()), dict(rows="all"), dict(rows="sorted"),
                dict(r=r._replace(offsets=z(8, dtype=i))), dict(r=r._replace(order=z(7, dtype=i))),
                dict(r=r._replace(slots=z(4, 2))), {}]:
        a = dict(x=x, xs=xs, codes=codes, s=s, r=r, K=None, rows="tokens") | bad
        with pytest.raises(ValueError):
            tl.linear_experts(a["x"], a["xs"], a["codes"], a["s"], a["r"], K=a["K"], rows=a["rows"])
    for bad in [dict(y=z(7, 32)), dict(y=z(8, 32).double()), dict(add=z(4, 31)), dict(add=z(4, 32).half()), {}]:
        with pytest.raises(ValueError):
            tl.combine(**(dict(y=z(8, 32), routing=r) | bad))


def test_reference_codes_are_torchs():
    """The tests' own e4m3 rounding against torch's conversion, on the CPU."""
    rng = np.random.default_rng(5)
    v = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000), (ref.TABLE[1:126] + ref.TABLE[2:127]) / 2,
                        ref.TABLE[:127], [0.0, -0.0, 448, -448]])
    v = np.clip(v, -448, 448).astype(np.float32)
    assert np.array_equal(ref.nearest_code(v.astype(np.float64)), torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    with np.errstate(invalid="ignore"):
        t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, ref.TABLE, equal_nan=True)
