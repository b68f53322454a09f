"""linear_adapters and linear_adapters_backward against their 64-bit definitions."""

import numpy as np
import pytest
import torch

import adapters_ref as ar
import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
TYPES = ["bf16", "fp16"]


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


# T, E, rank, K, N
CASES = [(1, 1, 1, 1, 1), (1, 8, 16, 512, 260), (2, 3, 8, 64, 64), (5, 2, 3, 7, 9), (16, 1, 16, 128, 256), (17, 5, 17, 130, 257), (33, 64, 32, 256, 128),
         (63, 4, 33, 72, 500), (64, 2, 64, 1000, 136), (65, 3, 100, 264, 520), (70, 512, 12, 96, 80), (129, 1, 128, 520, 264), (130, 100, 8, 264, 200), (200, 6, 40, 333, 777),
         (300, 1, 16, 256, 1024), (520, 2, 64, 640, 384), (700, 9, 5, 320, 65)]


def draw_of(rng, T, E, runs=False, masked=True):
    """Each token's adapter: some have none, and an adapter may have no token."""
    of = np.sort(rng.integers(0, E, T)) if runs else rng.integers(0, E, T)
    if masked and T > 2:
        of = np.where(rng.random(T) < 0.1, -1, of)
        of[1] = -1
    return of.astype(np.int32)


def whole(rng, shape, hi):
    return rng.integers(-hi, hi + 1, shape).astype(np.float64)


def dev(v, dt, shift=0):
    return ar.shifted(torch.from_numpy(np.asarray(v, np.float32)).to(dt).cuda(), shift)


def rounded(v, dt):
    return torch.from_numpy(v).to(torch.float32).to(dt)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,rank,K,N", CASES)
def test_adapters_exact(tl, T, E, rank, K, N, dtype, shift):
    """Whole numbers whose sums fit 24 bits: y is the rounding of the exact sum.  x a^T needs up to 16 bits, and
    neighbouring columns of b cancel, so that no rounding of it to fewer bits would pass."""
    say(f"adapters exact {T} {E} {rank} {K} {N} {dtype} shift={shift}")
    rng, dt = np.random.default_rng(T + K + N + rank), ar.DT[dtype]
    of = draw_of(rng, T, E)
    x, a = whole(rng, (T, K), 30), whole(rng, (E, rank, K), 30)
    b = whole(rng, (E, N, rank), 3)
    s = 2.0 ** rng.integers(-1, 2, E)
    add = whole(rng, (T, N), 100)
    y, v = ar.adapters(x, a, b, s, of, add)
    has = of >= 0
    mags = [np.abs(v[of == e]) @ np.abs(b[e]).T for e in range(E)]
    assert np.abs(v).max(initial=0) < 2.0 ** 24 and max(m.max(initial=0) for m in mags) < 2.0 ** 23
    # two 16-bit numbers hold 16 bits of bf16 (two nearest roundings: any whole number below 2^16), 22 of fp16
    if np.abs(v).max(initial=0) >= 2.0 ** 16 and dtype == "bf16":
        a = np.sign(a)
        x = np.clip(x, -8, 8)
        y, v = ar.adapters(x, a, b, s, of, add)
        assert np.abs(v).max() < 2.0 ** 16
    if dtype == "fp16":
        y = np.where(np.abs(y) > 60000, np.nan, y)
    r = tl.sort_slots(ref.dev(of), E)
    xd = dev(x, dt, shift)
    xd[~torch.from_numpy(has)] = torch.nan  # not read
    args = (xd, dev(a, dt, shift), dev(b, dt, shift), r, ref.dev(s.astype(np.float32)))
    out, buf = ar.guarded((T, N), dt, shift=shift)
    hid, hbuf = ar.guarded((T, rank), torch.float32)
    addd = dev(add, dt, shift)
    assert tl.linear_adapters(*args, add=addd, out=out, hidden=hid) is out
    fine = torch.from_numpy(~np.isnan(y))
    assert torch.equal(out.cpu()[fine], rounded(np.nan_to_num(y), dt)[fine])
    assert ar.untouched(out, buf) and ar.untouched(hid, hbuf)
    assert np.array_equal(hid.cpu().numpy()[has], v[has].astype(np.float32)) and bool((hid.cpu()[~torch.from_numpy(has)] == 77).all())
    assert torch.equal(tl.linear_adapters(*args, add=addd).nan_to_num(), out.nan_to_num())
    inplace = addd.clone() if not shift else ar.shifted(addd, shift)
    tl.linear_adapters(*args, add=inplace, out=inplace)
    assert torch.equal(inplace.nan_to_num(), out.nan_to_num())
    plain = tl.linear_adapters(*args)
    y0 = y - add
    fine = torch.from_numpy(~np.isnan(y0))
    assert torch.equal(plain.cpu()[fine], rounded(np.nan_to_num(y0), dt)[fine]) and not plain[~torch.from_numpy(has)].any()


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,rank,K,N", CASES)
def test_adapters_backward_exact(tl, T, E, rank, K, N, dtype, shift):
    """The same of the gradients: dv and hidden of up to 16 bits, sums that fit 24."""
    say(f"adapters backward exact {T} {E} {rank} {K} {N} {dtype} shift={shift}")
    rng, dt = np.random.default_rng(T + K + N + rank), ar.DT[dtype]
    of = draw_of(rng, T, E, runs=T % 2 == 0)
    has = torch.from_numpy(of >= 0)
    g, b = whole(rng, (T, N), 6), whole(rng, (E, N, rank), 6)
    x, a = whole(rng, (T, K), 2), whole(rng, (E, rank, K), 2)
    hidden = whole(rng, (T, rank), 2000)
    add = whole(rng, (T, K), 50)
    s = np.ones(E)
    dx, da, db, dv = ar.adapters_backward(g, x, hidden, a, b, s, of, add)
    assert np.abs(dv).max(initial=0) < 2.0 ** 16 and max(np.abs(v).max(initial=0) for v in (dx, da, db)) < 2.0 ** 24
    r = tl.sort_slots(ref.dev(of), E)
    gd, xd, hd = dev(g, dt, shift), dev(x, dt, shift), ref.dev(hidden.astype(np.float32))
    for t in (gd, xd, hd):
        t[~has] = torch.nan  # not read
    args = (gd, xd, hd, dev(a, dt, shift), dev(b, dt, shift), r)
    addd = dev(add, dt, shift)
    out, buf = ar.guarded((T, K), dt, shift=shift)
    got = tl.linear_adapters_backward(*args, add=addd, out=out)
    assert got[0] is out and ar.untouched(out, buf)
    for name, t, want in zip(("dx", "da", "db"), got, (dx, da, db)):
        want = np.where(np.abs(want) > 60000, np.nan, want) if dtype == "fp16" else want
        fine = torch.from_numpy(~np.isnan(want))
        assert torch.equal(t.cpu()[fine], rounded(np.nan_to_num(want), dt)[fine]), name
    again = tl.linear_adapters_backward(*args, scale=torch.ones(E, device="cuda"), add=addd)
    assert all(torch.equal(p.nan_to_num(), q.nan_to_num()) for p, q in zip(got, again))
    inplace = ar.shifted(addd, shift) if shift else addd.clone()
    assert torch.equal(tl.linear_adapters_backward(*args, add=inplace, out=inplace)[0].nan_to_num(), out.nan_to_num())
    plain = tl.linear_adapters_backward(*args)[0]
    assert torch.equal(plain.cpu()[has].nan_to_num(posinf=0, neginf=0) if dtype == "fp16" else plain.cpu()[has],
                       rounded((dx - add)[has.numpy()], dt).nan_to_num(posinf=0, neginf=0) if dtype == "fp16" else rounded((dx - add)[has.numpy()], dt))
    assert not plain[~has].any()


def forward_bound(x, a, b, s, of, add, y, v, dt):
    """How far y may be from the 64-bit sum.  hidden: K exact products, added up in at most K + 16 sums of the matrix unit (and of
    waves and parts).  Two 16-bit numbers stand for it: cut to 8 bits, what is
    left is below 2^-7, and the nearest of 8 bits to that within 2^-9 of it (bf16: 2^-16); of 11 bits 2^-10 and 2^-12 (fp16: 2^-22, of the row's
    largest, which also covers what is below its smallest number).  2 rank products more, the scale, add and the output's rounding."""
    T, rank, K = x.shape[0], a.shape[1], x.shape[1]
    mv = ar.adapters(np.abs(x), np.abs(a), np.abs(b), np.abs(s), of)[1]
    dv = (K + 16) * ar.SUM * mv
    dsplit = 2.0 ** -16 * np.abs(v) if dt == torch.bfloat16 else 2.0 ** -22 * np.abs(v).max(1, keepdims=True) * np.ones((1, rank))
    lim = np.zeros(y.shape)
    for e in range(a.shape[0]):
        at = of == e
        lim[at] = abs(s[e]) * ((dv[at] + dsplit[at] + (2 * rank + 8) * ar.SUM * (np.abs(v[at]) + dv[at])) @ np.abs(b[e]).T)
    return lim * 1.001 + 4 * ar.STEP * np.abs(add) + ref.EPS[dt] * (np.abs(y) + lim) + ar.TINY[dt], dv


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,rank,K,N", [(1, 4, 16, 4096, 512), (40, 16, 8, 1024, 300), (300, 3, 64, 512, 640), (200, 1, 128, 256, 256)])
def test_adapters(tl, T, E, rank, K, N, dtype):
    say(f"adapters {T} {E} {rank} {K} {N} {dtype}")
    rng, dt = np.random.default_rng(T + K), ar.DT[dtype]
    of = draw_of(rng, T, E)
    x = dev(rng.standard_normal((T, K)) * np.exp(0.7 * rng.standard_normal(K)), dt)
    a, b = dev(rng.standard_normal((E, rank, K)) * K ** -0.5, dt), dev(0.05 * rng.standard_normal((E, N, rank)), dt)
    s, add = (0.5 + rng.random(E)).astype(np.float32), dev(rng.standard_normal((T, N)), dt)
    r = tl.sort_slots(ref.dev(of), E)
    hid = torch.zeros(T, rank, device="cuda")
    got = tl.linear_adapters(x, a, b, r, ref.dev(s), add=add, hidden=hid)
    w = [ar.wide(t) for t in (x, a, b)]
    y, v = ar.adapters(*w, s.astype(np.float64), of, ar.wide(add))
    lim, dv = forward_bound(*w, s.astype(np.float64), of, ar.wide(add), y, v, dt)
    assert np.all(np.abs(ar.wide(hid) - v) <= dv + 1e-40)
    assert np.all(np.abs(ar.wide(got) - y) <= lim)
    # the rounding of y aside, all that is left is far below a 16-bit rounding of hidden (2^-8, 2^-11 of it)
    off = ar.wide(tl.linear_adapters(x, a, b, r, ref.dev(s))) - rounded(y - ar.wide(add), dt).double().numpy()
    assert np.mean(off != 0) < 0.05


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,rank,K,N", [(1, 4, 16, 512, 1024), (40, 16, 8, 300, 512), (600, 2, 64, 512, 256), (200, 1, 128, 256, 256)])
def test_adapters_backward(tl, T, E, rank, K, N, dtype):
    say(f"adapters backward {T} {E} {rank} {K} {N} {dtype}")
    rng, dt = np.random.default_rng(T + K), ar.DT[dtype]
    of = draw_of(rng, T, E)
    g = dev(0.01 * rng.standard_normal((T, N)), dt)
    x = dev(rng.standard_normal((T, K)) * np.exp(0.7 * rng.standard_normal(K)), dt)
    a, b = dev(rng.standard_normal((E, rank, K)) * K ** -0.5, dt), dev(0.05 * rng.standard_normal((E, N, rank)), dt)
    hidden = rng.standard_normal((T, rank)).astype(np.float32)
    s, add = (0.5 + rng.random(E)).astype(np.float32), dev(0.01 * rng.standard_normal((T, K)), dt)
    r = tl.sort_slots(ref.dev(of), E)
    got = tl.linear_adapters_backward(g, x, ref.dev(hidden), a, b, r, ref.dev(s), add=add)
    gw, xw, aw, bw, hw, sw = ar.wide(g), ar.wide(x), ar.wide(a), ar.wide(b), hidden.astype(np.float64), s.astype(np.float64)
    want = ar.adapters_backward(gw, xw, hw, aw, bw, sw, of, ar.wide(add))
    dv = want[3]
    mag = ar.adapters_backward(np.abs(gw), np.abs(xw), np.abs(hw), np.abs(aw), np.abs(bw), sw, of, np.abs(ar.wide(add)))
    ddv = (N + 16) * ar.SUM * mag[3]  # as hidden in the forward call, N products
    lims = [np.zeros(w.shape) for w in want[:3]]
    for e in range(E):
        at = of == e
        if not at.any():
            continue
        n = at.sum()
        # what the two 16-bit numbers leave of dv (row's largest for dx, the tokens' largest for da) and of hidden
        if dt == torch.bfloat16:
            sx, sa, sb = 2.0 ** -16 * np.abs(dv[at]), 2.0 ** -16 * np.abs(dv[at]), 2.0 ** -16 * np.abs(hw[at])
        else:
            o = np.ones((n, rank))
            sx, sa, sb = 2.0 ** -22 * np.abs(dv[at]).max(1, keepdims=True) * o, 2.0 ** -22 * np.abs(dv[at]).max() * o, 2.0 ** -22 * np.abs(hw[at]).max() * o
        sums = (2 * rank + 8) * ar.SUM * (np.abs(dv[at]) + ddv[at])
        lims[0][at] = (ddv[at] + sx + sums) @ np.abs(aw[e])
        lims[1][e] = (ddv[at] + sa + (2 * n + 16) * ar.SUM * (np.abs(dv[at]) + ddv[at])).T @ np.abs(xw[at])
        lims[2][e] = sw[e] * (np.abs(gw[at]).T @ (sb + (2 * n + 16) * ar.SUM * np.abs(hw[at])))
    lims[0] += 4 * ar.STEP * np.abs(ar.wide(add))
    for name, t, w, lim in zip(("dx", "da", "db"), got, want, lims):
        assert np.all(np.abs(ar.wide(t) - w) <= lim * 1.001 + ref.EPS[dt] * (np.abs(w) + lim) + ar.TINY[dt]), name
    again = tl.linear_adapters_backward(g, x, ref.dev(hidden), a, b, r, ref.dev(s), add=add)
    assert all(torch.equal(p, q) for p, q in zip(got, again)), "the same inputs give the same bits"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,rank,K,N", [(2049, 3, 16, 136, 264), (2500, 40, 32, 264, 520), (4200, 5, 64, 264, 520), (4200, 2, 40, 77, 139),
                                          (5000, 1, 128, 264, 264), (9000, 7, 8, 1032, 72), (20000, 300, 16, 64, 320), (7001, 2, 24, 3600, 4001),
                                          (6500, 3, 48, 4000, 4096), (8200, 2, 90, 3201, 3104)])
def test_adapters_many_tokens(tl, T, E, rank, K, N, dtype):
    """Whole numbers again, at numbers of tokens that take the kernels' large tiles and several pieces of an adapter's tokens
    (the definitions here on the GPU, in 64 bits)."""
    say(f"adapters many tokens {T} {E} {rank} {K} {N} {dtype}")
    dt = ar.DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(T + rank)

    def whole_dev(*s, hi):
        return torch.randint(-hi, hi + 1, s, device="cuda", generator=g).double()

    of = torch.randint(-1, E, (T,), device="cuda", generator=g).sort().values if T % 2 else torch.randint(-1, E, (T,), device="cuda", generator=g)
    of[of == E - 2] = -1 if E > 2 else 0  # (an adapter without tokens)
    x, a, b, gr = whole_dev(T, K, hi=2), whole_dev(E, rank, K, hi=2), whole_dev(E, N, rank, hi=3), whole_dev(T, N, hi=2)
    add, addx, hidden = whole_dev(T, N, hi=50), whole_dev(T, K, hi=50), whole_dev(T, rank, hi=9)
    y, dx, v = add.clone(), addx.clone(), torch.zeros(T, rank, device="cuda", dtype=torch.float64)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for e in range(E):
        at = (of == e).nonzero()[:, 0]
        v[at] = x[at] @ a[e].t().contiguous()
        y[at] += v[at] @ b[e].t().contiguous()
        dv = gr[at] @ b[e]
        dx[at] += dv @ a[e]
        da[e], db[e] = dv.t().contiguous() @ x[at], gr[at].t().contiguous() @ hidden[at]
    for t in (v, y, dx, da, db):  # every sum fits 24 bits: |dv| and |v| below 2^16, and what they are multiplied and added up to
        assert float(t.abs().max()) < 2.0 ** 23
    r = tl.sort_slots(of.int(), E)
    hid = torch.zeros(T, rank, device="cuda")
    args = [t.to(dt) for t in (x, a, b)]
    assert torch.equal(tl.linear_adapters(*args, r, add=add.to(dt), hidden=hid), y.float().to(dt)) and torch.equal(hid.double(), v)
    got = tl.linear_adapters_backward(gr.to(dt), args[0], hidden.float(), *args[1:], r, add=addx.to(dt))
    for name, t, want in zip(("dx", "da", "db"), got, (dx, da, db)):
        assert torch.equal(t, want.float().to(dt)), name


@pytest.mark.parametrize("T", [0, 5, 200])
def test_adapters_nobody(tl, T):
    """No token, or none with an adapter: y is add or 0, gradients of the weights are 0."""
    say(f"adapters nobody T={T}")
    E, rank, K, N = 3, 8, 40, 72
    z = lambda *s: torch.full(s, torch.nan, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    r = tl.sort_slots(torch.full((T,), -1, dtype=torch.int32, device="cuda"), E)
    x, g, a, b, h = z(T, K), z(T, N), z(E, rank, K), z(E, N, rank), torch.full((T, rank), torch.nan, device="cuda")
    add = torch.randn(T, N, device="cuda").bfloat16()
    assert torch.equal(tl.linear_adapters(x, a, b, r, add=add), add) and not tl.linear_adapters(x, a, b, r).any()
    for more in (None, torch.randn(T, K, device="cuda").bfloat16()):
        dx, da, db = tl.linear_adapters_backward(g, x, h, a, b, r, add=more)
        assert torch.equal(dx, more) if more is not None else not dx.any()
        assert not da.any() and not db.any()


@pytest.mark.parametrize("dtype", TYPES)
def test_adapters_rows_apart(tl, dtype):
    """An infinity or a NaN of one token reaches that token's outputs only, one of an adapter's weights that adapter's."""
    say(f"adapters apart {dtype}")
    rng, dt = np.random.default_rng(1), ar.DT[dtype]
    T, E, rank, K, N = 150, 3, 24, 136, 200
    of = draw_of(rng, T, E, masked=False)
    r = tl.sort_slots(ref.dev(of), E)
    x, a, b = (dev(whole(rng, s, 2), dt) for s in ((T, K), (E, rank, K), (E, N, rank)))
    good = tl.linear_adapters(x, a, b, r)
    t = int(np.nonzero(of == 1)[0][3])
    for bad in (torch.nan, torch.inf, -torch.inf):
        y = x.clone()
        y[t, 77] = bad
        got = tl.linear_adapters(y, a, b, r)
        assert not torch.isfinite(got[t]).all() and torch.equal(torch.cat([got[:t], got[t + 1:]]), torch.cat([good[:t], good[t + 1:]]))
    # an infinite x times positive weights: infinite, not NaN
    got = tl.linear_adapters(torch.where(torch.arange(K, device="cuda") == 5, torch.inf, x[t:t + 1].float()).to(dt).expand(T, K).contiguous(),
                             a.abs() + 1, b.abs() + 1, r)
    assert bool((got == torch.inf).all())
    c = b.clone()
    c[2, 5, 3] = torch.nan
    got = tl.linear_adapters(x, a, c, r)
    want = good.clone()
    want[torch.from_numpy(of == 2).cuda(), 5] = torch.nan
    assert torch.equal(got.nan_to_num(5e4), want.nan_to_num(5e4))


def test_adapters_large_and_small(tl):
    """fp16: hidden beyond fp16's largest and below its smallest number, by token, still gives y of usual size."""
    say("adapters fp16 range")
    T, K, N, rank = 96, 256, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, K, device="cuda", generator=g).half()
    of = torch.arange(T, device="cuda", dtype=torch.int32) % 2
    a = torch.randn(2, rank, K, device="cuda", generator=g)
    b = torch.randn(2, N, rank, device="cuda", generator=g)
    a, b = (a * torch.tensor([6e3, 3e-7], device="cuda").view(2, 1, 1)).half(), (b * torch.tensor([1e-4, 1e4], device="cuda").view(2, 1, 1)).half()
    s = torch.tensor([1.0, 30.0], device="cuda")
    r = tl.sort_slots(of, 2)
    hid = torch.empty(T, rank, device="cuda")
    got = tl.linear_adapters(x, a, b, r, s, hidden=hid)
    assert float(hid.abs().max()) > 7e4 and float(hid[1::2].abs().max()) < 1e-4
    y, v = ar.adapters(ar.wide(x), ar.wide(a), ar.wide(b), ar.wide(s), of.cpu().numpy())
    lim, _ = forward_bound(ar.wide(x), ar.wide(a), ar.wide(b), ar.wide(s), of.cpu().numpy(), 0 * y, y, v, torch.float16)
    assert np.all(np.abs(ar.wide(got) - y) <= lim)
    # gradients: the tokens' hidden and dv span the same range
    dx, da, db = tl.linear_adapters_backward(torch.ones(T, N, device="cuda").half(), x, hid, a, b, r, s)
    want = ar.adapters_backward(np.ones((T, N)), ar.wide(x), ar.wide(hid), ar.wide(a), ar.wide(b), ar.wide(s), of.cpu().numpy())
    for t, w in zip((dx, da, db), want):
        t, w = ar.wide(t), np.where(np.abs(w) > 65504, np.sign(w) * np.inf, w)
        ok = np.isfinite(w) & (np.abs(w) < 65000)
        assert np.isfinite(t[ok]).all() and np.linalg.norm(t[ok] - w[ok]) <= 2.0 ** -10 * np.linalg.norm(w[ok])


@pytest.mark.parametrize("T", [4, 400])
def test_adapters_foreign_indices(tl, T):
    """Offsets, order and slots that describe no sorting: nothing outside the arguments is read or written."""
    say(f"adapters foreign indices T={T}")
    E, rank, K, N = 5, 16, 64, 96
    n = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, g, a, b, h = n(T, K), n(T, N), n(E, rank, K), n(E, N, rank), torch.randn(T, rank, device="cuda")
    r = tl.sort_slots(torch.randint(0, E, (T,), dtype=torch.int32, device="cuda"), E)
    i32 = dict(dtype=torch.int32, device="cuda")
    for off in ([0, T, -7, T + 100, 3, 2 ** 31 - 1], [-2 ** 31, -5, -1, 0, 0, 0], [5, 4, 3, 2, 1, 0], [T] * 6, [0, T, 0, T, 0, T], r.offsets.tolist()):
        order = torch.full((T,), 2 ** 31 - 1, **i32)
        order[::2] = -2 ** 31
        order[-1] = T
        for o in (order, r.order):
            bad = r._replace(offsets=torch.tensor(off, **i32), order=o, slots=torch.full_like(r.slots, 2 ** 31 - 1))
            out, buf = ar.guarded((T, N), torch.bfloat16)
            hid, hbuf = ar.guarded((T, rank), torch.float32)
            tl.linear_adapters(x, a, b, bad, out=out, hidden=hid)
            dx, dbuf = ar.guarded((T, K), torch.bfloat16)
            _, da, db = tl.linear_adapters_backward(g, x, h, a, b, bad, out=dx)
            torch.cuda.synchronize()
            assert ar.untouched(out, buf) and ar.untouched(hid, hbuf) and ar.untouched(dx, dbuf)


def test_adapters_far(tl):
    """Rows beyond 2^31 elements, forward and back."""
    say("adapters far")
    T, E, rank, K, N = 66000, 3, 8, 40, 33000
    n = lambda *s: torch.randint(-2, 3, s, device="cuda").bfloat16()  # noqa: E731
    x, a, b = n(T, K), n(E, rank, K), n(E, N, rank)
    r = tl.sort_slots(torch.randint(-1, E, (T,), dtype=torch.int32, device="cuda"), E)
    hid = torch.zeros(T, rank, device="cuda")
    y = tl.linear_adapters(x, a, b, r, hidden=hid)
    g = y.clamp_(-2, 2)
    dx, da, db = tl.linear_adapters_backward(g, x, hid, a, b, r)
    of = r.ids[:, 0].long()
    for t in [0, 1, 65075, 65076, T - 1, *range(40000, 40040)]:  # (2^31 / N = 65075.3)
        e = int(of[t])
        if e < 0:
            assert not y[t].any() and not dx[t].any()
            continue
        v = x[t].double() @ a[e].double().t().contiguous()
        assert torch.equal(hid[t].double(), v)
        assert torch.equal(y[t].double(), (v @ b[e].double().t().contiguous()).clamp(-2, 2))
        dv = g[t].double() @ b[e].double()
        # dv is whole and mostly below 2^16, where two 16-bit numbers hold it; beyond they are 2^-16 off.  The sums of whole
        # numbers are exact; dx is rounded once
        want, mags = dv @ a[e].double(), dv.abs() @ a[e].double().abs()
        off = 2.0 ** -16 * mags if float(dv.abs().max()) >= 2.0 ** 16 else 0 * mags
        assert bool(((dx[t].double() - want).abs() <= off + 2.0 ** -8 * (want.abs() + off)).all())
    at = (of == 1).nonzero()[:, 0]
    want = g[at][:, -64:].double().t().contiguous() @ hid[at].double()
    got, mags = db[1, -64:].double(), g[at][:, -64:].double().abs().t().contiguous() @ hid[at].double().abs()
    assert bool(((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * mags).all())


def layer(tl, x, codes, s, a, b, r, scale, hidden=None):
    """A shared ternary projection with each token's adapter beside it, as a user writes it."""
    y = tl.linear(x, codes, s, layout="tiled")
    return tl.linear_adapters(x, a, b, r, scale, add=y, out=y, hidden=hidden)


@pytest.mark.parametrize("T", [1, 7, 40, 300])
def test_adapters_beside_linear(tl, T):
    """The layer as a whole, serving and training, against 64 bits; captured and replayed on other requests."""
    say(f"adapters beside linear T={T}")
    rng = np.random.default_rng(T)
    E, rank, K, N = 6, 16, 512, 384
    q, s = rng.integers(-1, 2, (N, K)).astype(np.int8), ref.scales_of(rng, N).astype(np.float16)
    codes, sd = torch.from_numpy(ref.tile_codes(q)).cuda(), ref.dev(s)
    a, b = dev(whole(rng, (E, rank, K), 1), torch.bfloat16), dev(whole(rng, (E, N, rank), 1), torch.bfloat16)
    scale = torch.full((E,), 0.5, device="cuda")
    x = dev(whole(rng, (T, K), 4), torch.bfloat16)
    of = torch.from_numpy(draw_of(rng, T, E)).cuda()

    def step():
        r = tl.sort_slots(of, E)
        hidden = torch.zeros(T, rank, device="cuda")
        y = layer(tl, x, codes, sd, a, b, r, scale, hidden)
        g = y.clamp(-2, 2)
        base = tl.linear((g * sd.to(g.dtype)).contiguous(), back, ones, layout="tiled")  # the projection's own gradient of x
        return (y, hidden, *tl.linear_adapters_backward(g, x, hidden, a, b, r, scale, add=base, out=base))

    back = torch.from_numpy(ref.tile_codes(np.ascontiguousarray(q.T))).cuda()
    ones = torch.ones(K, dtype=torch.float16, device="cuda")
    first = step()
    w = q * s.astype(np.float64)[:, None]
    base = ar.wide(tl.linear(x, codes, sd, layout="tiled"))
    want, v = ar.adapters(ar.wide(x), ar.wide(a), ar.wide(b), ar.wide(scale), of.cpu().numpy(), base)
    assert np.abs(base - ar.wide(x) @ w.T).max() <= 2.0 ** -8 * np.abs(ar.wide(x) @ w.T).max()
    assert torch.equal(first[0].cpu(), rounded(want, torch.bfloat16)) and np.array_equal(first[1].cpu().numpy(), v)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kept = step()
    for rep in range(4):
        x.copy_(torch.randint(-4, 5, x.shape, device="cuda"))
        of.copy_(torch.randint(-1, E, of.shape, dtype=torch.int32, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, eager)), rep


def test_adapters_streams(tl):
    """Two calls at once, each on its own stream with its own workspace."""
    say("adapters streams")
    T, E, rank, K, N = 300, 4, 32, 512, 640
    n = lambda *s: torch.randn(*s, device="cuda").bfloat16()  # noqa: E731
    x, g, a, b, h = n(T, K), n(T, N), n(E, rank, K), n(E, N, rank), torch.randn(T, rank, device="cuda")
    r = tl.sort_slots(torch.randint(0, E, (T,), dtype=torch.int32, device="cuda"), E)
    want = (tl.linear_adapters(x, a, b, r), *tl.linear_adapters_backward(g, x, h, a, b, r))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for rep in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((tl.linear_adapters(x, a, b, r), *tl.linear_adapters_backward(g, x, h, a, b, r)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for one in got for p, q in zip(one, want))
