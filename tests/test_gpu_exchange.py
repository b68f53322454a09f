"""dispatch, dispatch_backward and combine_backward against their 64-bit definitions, and the chain that they belong to."""

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


CASES = [(1, 1, 1, 1), (1, 8, 4096, 64), (2, 3, 7, 3), (3, 2, 8, 9), (7, 3, 17, 5), (33, 32, 260, 40), (64, 4, 504, 8), (65, 5, 513, 9), (40, 8, 1023, 64),
         (12, 2, 1025, 4), (9, 6, 2048, 16), (10, 4, 4104, 9), (5, 2, 9000, 7), (300, 8, 1024, 512)]


def draw(rng, T, k, E, masked=True):
    ids = rng.integers(0, E, (T, k)).astype(np.int32)  # (the same expert twice in a token, too)
    if masked:
        ids[rng.random((T, k)) < 0.15] = -1
        ids[T // 2] = E + 5
    return ids, rng.random((T, k)).astype(np.float32)


def tensor(rng, shape, dt, shift=0):
    return ar.shifted(torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt).cuda(), shift)


def close(got, want, lim, what):
    err = np.abs(ar.wide(got) - want)
    assert np.all(err <= lim), (what, float((err - lim).max()))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", list(ar.DT))
@pytest.mark.parametrize("T,k,N,E", CASES)
def test_dispatch(tl, T, k, N, E, dtype, shift):
    say(f"dispatch {T} {k} {N} {dtype} shift={shift}")
    rng, dt = np.random.default_rng(T + N), ar.DT[dtype]
    ids, w = draw(rng, T, k, E)
    r = ar.routing(tl, ids, w, E)
    slots, x = r.slots.cpu().numpy(), tensor(rng, (T, N), dt, shift)
    used = int((slots >= 0).sum())
    for weighted in (False, True):
        out, buf = ar.guarded((T * k, N), dt, shift=shift)
        assert tl.dispatch(x, r, weighted=weighted, out=out) is out
        want = ar.dispatch(ar.wide(x), w.astype(np.float64) if weighted else np.ones((T, k)), slots)[:used]
        # a product in fp32, and the output's rounding
        close(out[:used], want, ref.EPS[dt] * np.abs(want) * (1 + 2.0 ** -20) + ar.STEP * np.abs(want) + ar.TINY[dt] if weighted else 0 * want, weighted)
        assert ar.untouched(out[:used], buf)
    assert torch.equal(tl.dispatch(x, r)[:used], tl.dispatch(x, r)[:used])


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", list(ar.DT))
@pytest.mark.parametrize("T,k,N,E", CASES)
def test_combine_backward(tl, T, k, N, E, dtype, shift):
    say(f"combine_backward {T} {k} {N} {dtype} shift={shift}")
    rng, dt = np.random.default_rng(T + N), ar.DT[dtype]
    ids, w = draw(rng, T, k, E)
    r = ar.routing(tl, ids, w, E)
    slots = r.slots.cpu().numpy()
    g, y = tensor(rng, (T, N), dt, shift), tensor(rng, (T * k, N), dt, shift)
    used = int((slots >= 0).sum())
    y[used:] = torch.nan  # places without a slot are not read
    out, buf = ar.guarded((T * k, N), dt, shift=shift)
    dy, dw = tl.combine_backward(g, y, r, out=out)
    assert dy is out
    wy, wdw = ar.combine_backward(ar.wide(g), np.nan_to_num(ar.wide(y)), w.astype(np.float64), slots)
    wy = wy[:used]
    close(dy[:used], wy, ref.EPS[dt] * np.abs(wy) * (1 + 2.0 ** -20) + ar.STEP * np.abs(wy) + ar.TINY[dt], "dy")
    mags = ar.combine_backward(np.abs(ar.wide(g)), np.abs(np.nan_to_num(ar.wide(y))), w.astype(np.float64), slots)[1]
    # a lane adds up eight products of each 512, a wave's 64 lanes in six steps: roundings of a product and of each sum
    close(dw, wdw, (8 * ref.up(N, 512) // 512 + 7) * ar.STEP * mags + 1e-40, "dweights")
    assert ar.untouched(out[:used], buf) and bool((dw[r.slots < 0] == 0).all())
    again = tl.combine_backward(g, y, r)
    assert torch.equal(again[0][:used], dy[:used]) and torch.equal(again[1], dw)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", list(ar.DT))
@pytest.mark.parametrize("T,k,N,E", CASES)
def test_dispatch_backward(tl, T, k, N, E, dtype, shift):
    say(f"dispatch_backward {T} {k} {N} {dtype} shift={shift}")
    rng, dt = np.random.default_rng(T + N), ar.DT[dtype]
    ids, w = draw(rng, T, k, E)
    r = ar.routing(tl, ids, w, E)
    slots = r.slots.cpu().numpy()
    g, x, a = tensor(rng, (T * k, N), dt, shift), tensor(rng, (T, N), dt, shift), tensor(rng, (T, N), dt, shift)
    g[int((slots >= 0).sum()):] = torch.nan
    gw, xw, aw = np.nan_to_num(ar.wide(g)), ar.wide(x), ar.wide(a)
    for weighted in (False, True):
        for add in (None, a):
            wt = w.astype(np.float64) if weighted else np.ones((T, k))
            out, buf = ar.guarded((T, N), dt, shift=shift)
            got = tl.dispatch_backward(g, r, x=x if weighted else None, add=add, out=out)
            want, wdw = ar.dispatch_backward(gw, wt, slots, xw, aw if add is not None else 0)
            mags, mdw = ar.dispatch_backward(np.abs(gw), wt, slots, np.abs(xw), np.abs(aw) if add is not None else 0)
            dx = got[0] if weighted else got
            assert dx is out and ar.untouched(out, buf)
            # k products and k sums, and the output's rounding
            close(dx, want, 2 * k * ar.STEP * mags + ref.EPS[dt] * np.abs(want) * (1 + 2.0 ** -20) + ar.TINY[dt], "dx")
            if weighted:
                # a lane adds up at most eight products of each 512, a wave's lanes in six steps, four waves
                close(got[1], wdw, (8 * ref.up(N, 512) // 512 + 12) * ar.STEP * mdw + 1e-40, "dweights")
                assert bool((got[1][r.slots < 0] == 0).all())
            if add is not None:
                buf2 = add.clone()
                again = tl.dispatch_backward(g, r, x=x if weighted else None, add=buf2, out=buf2)
                assert torch.equal(buf2, dx) and (not weighted or torch.equal(again[1], got[1]))


def test_exchange_edges(tl):
    """No tokens, empty rows, weights and rows that are not numbers where no slot is."""
    say("exchange edges")
    z = torch.zeros
    r = tl.sort_slots(z(0, 2, dtype=torch.int32, device="cuda"), 4)
    x = z(0, 16, device="cuda")
    assert tl.dispatch(x, r).shape == (0, 16) and tl.dispatch_backward(x, r).shape == (0, 16)
    assert [t.shape for t in tl.combine_backward(x, x, r)] == [(0, 16), (0, 2)]
    ids = torch.tensor([[0, -1], [-1, -1], [1, 0]], dtype=torch.int32, device="cuda")
    r = tl.sort_slots(ids, 2, torch.tensor([[.5, torch.nan], [torch.nan, torch.inf], [2, 4]], device="cuda"))
    e = z(3, 0, device="cuda")
    dy, dw = tl.combine_backward(e, z(6, 0, device="cuda"), r)
    assert dy.shape == (6, 0) and not dw.any()
    x = torch.tensor([[1.0, torch.inf], [torch.nan, 7], [3, -4]], device="cuda")
    out = tl.dispatch(x, r, weighted=True)
    assert out[:3].tolist() == [[0.5, torch.inf], [12, -16], [6, -8]]
    dx, dw = tl.dispatch_backward(torch.ones(6, 2, device="cuda"), r, x=x)
    assert dx.tolist() == [[.5, .5], [0, 0], [6, 6]] and dw.tolist() == [[torch.inf, 0], [0, 0], [-1, -1]]
    dy, dw = tl.combine_backward(x, torch.ones(6, 2, device="cuda"), r)
    assert dy[:3].tolist() == [[.5, torch.inf], [12, -16], [6, -8]] and dw.tolist() == [[torch.inf, 0], [0, 0], [-1, -1]]


def test_exchange_foreign_slots(tl):
    """Slots that name no row: nothing outside the arguments is read or written."""
    say("exchange foreign slots")
    T, k, N = 6, 3, 40
    r = tl.sort_slots(torch.zeros(T, k, dtype=torch.int32, device="cuda"), 2)
    far = torch.full_like(r.slots, 2 ** 31 - 1)
    far[::2] = -2 ** 31
    far[0, 0] = T * k
    bad = r._replace(slots=far)
    x, y = torch.ones(T, N, device="cuda"), torch.ones(T * k, N, device="cuda")
    out, buf = ar.guarded((T * k, N), torch.float32)
    tl.dispatch(x, bad, out=out)
    tl.combine_backward(x, y, bad, out=out)
    assert bool((buf == 77).all())
    dx, dw = tl.dispatch_backward(y, bad, x=x)
    assert not dx.any() and not dw.any() and not tl.combine_backward(x, y, bad)[1].any()


def test_exchange_far(tl):
    """Rows beyond 2^31 elements."""
    say("exchange far")
    T, k, N = 20000, 4, 40000
    r = tl.sort_slots(torch.randint(0, 9, (T, k), dtype=torch.int32, device="cuda"), 9, torch.rand(T, k, device="cuda"))
    x = torch.randn(T, N, device="cuda", dtype=torch.bfloat16)
    y = tl.dispatch(x, r, weighted=True)
    for p in (0, T * k // 2, 53687, 53688, T * k - 1):  # (2^31 / N = 53687.09)
        s = int(r.order[p])
        assert torch.equal(y[p], (x[s // k].float() * r.weights[s // k, s % k]).to(y.dtype))
    dy, dw = tl.combine_backward(x, y, r)
    assert torch.equal(dy, y)
    t = int(r.order[T * k - 1]) // k
    want = (y[r.slots[t].long()].double() * x[t].double()).sum(1)
    assert bool(((dw[t].double() - want).abs() <= 2e-5 * want.abs()).all())
    del dy
    dx = tl.dispatch_backward(y, r)
    want = y[r.slots[t].long()].double().sum(0)
    assert bool(((dx[t].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-6).all())


def test_exchange_many_tokens(tl):
    """More tokens and slots than a launch has workgroups."""
    say("exchange many tokens")
    T, k, N = 1100000, 5, 8
    r = tl.sort_slots(torch.randint(-1, 9, (T, k), dtype=torch.int32, device="cuda"), 9, torch.rand(T, k, device="cuda"))
    x, g = torch.randn(T, N, device="cuda"), torch.randn(T, N, device="cuda")
    y = tl.dispatch(x, r, out=torch.zeros(T * k, N, device="cuda"))
    has, at = r.slots >= 0, r.slots.long().clamp_min(0)
    assert torch.equal(y[at][has], x[:, None, :].expand(T, k, N)[has])
    dy, dw = tl.combine_backward(g, y, r, out=torch.zeros_like(y))
    want = torch.where(has, (x.double() * g.double()).sum(1, keepdim=True), 0.0)
    mags = (x.double() * g.double()).abs().sum(1, keepdim=True)
    assert bool(((dw.double() - want).abs() <= 16 * ar.STEP * mags).all())  # eight products, eight sums
    assert torch.equal(dy[at][has], (r.weights[:, :, None] * g[:, None, :])[has])
    dx, dw = tl.dispatch_backward(dy, r, x=x)
    w2 = torch.where(has, r.weights.double(), 0.0)
    want = (w2 * w2).sum(1, keepdim=True) * g.double()
    assert bool(((dx.double() - want).abs() <= 16 * ar.STEP * want.abs() + 1e-30).all())  # k products (and dy's), k sums, of one sign
    want, mags = w2 * (x.double() * g.double()).sum(1, keepdim=True), w2 * mags
    assert bool(((dw.double() - want).abs() <= 18 * ar.STEP * mags).all())


def test_exchange_other_stream(tl):
    """Calls on a stream of their own, and captured and replayed, give the eager results."""
    say("exchange streams")
    T, k, N, E = 200, 4, 520, 16
    r = tl.sort_slots(torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda"), E, torch.rand(T, k, device="cuda"))
    x, g = torch.randn(T, N, device="cuda").half(), torch.randn(T, N, device="cuda").half()
    out = torch.zeros(T * k, N, device="cuda").half()

    def chain():
        rows = tl.dispatch(x, r, weighted=True, out=out)
        dy, dw = tl.combine_backward(g, rows, r, out=torch.zeros_like(out))
        return (*tl.dispatch_backward(dy, r, x=x, add=g), dw, dy, rows.clone())

    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = chain()
    for rep in range(4):
        x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            apart = chain()
        torch.cuda.synchronize()
        want = chain()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)) and all(torch.equal(a, b) for a, b in zip(apart, want)), rep


@pytest.mark.parametrize("T", [3, 90])
def test_training_step_of_experts(tl, T):
    """A layer of ternary experts and its gradients, as a user writes them: route, the experts' products, combine, and
    back through combine_backward, the experts' transposed weights and dispatch_backward.  Whole numbers and
    power-of-two scales keep every product exact, so that gradients are known."""
    say(f"training step of experts T={T}")
    rng = np.random.default_rng(T)
    E, k, K, N = 6, 2, 256, 128
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = ref.scales_of(rng, E, 1).astype(np.float16)  # one scale an expert
    one = np.repeat(s, N, 1), np.repeat(s, K, 1)
    up = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    back = torch.stack([torch.from_numpy(ref.tile_codes(np.ascontiguousarray(e.T))) for e in q]).cuda()
    x = torch.from_numpy(rng.integers(-8, 9, (T, K)).astype(np.float32)).cuda()
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[0] = -1
    w = (rng.integers(1, 5, (T, k)) / 4).astype(np.float32)
    r = tl.sort_slots(ref.dev(ids), E, ref.dev(w))
    slots = r.slots.cpu().numpy()
    xq, xs = tl.fp8_quantize(x)
    y = tl.linear_experts(xq, xs, up, ref.dev(one[0]), r, dtype=torch.float32, out=torch.zeros(T * k, N, device="cuda"))
    out = tl.combine(y, r)
    g = torch.from_numpy(rng.integers(-2, 3, (T, N)).astype(np.float32)).cuda()
    dy, dw = tl.combine_backward(g, y, r, out=torch.zeros_like(y))
    gq, gs = tl.fp8_quantize(dy)
    dx = tl.dispatch_backward(tl.linear_experts(gq, gs, back, ref.dev(one[1]), r, rows="sorted", dtype=torch.float32,
                                                out=torch.zeros(T * k, K, device="cuda")), r)
    # the experts see x and dy as their codes and scales stand for them
    xw, gw = ref.wide(xq.view(torch.uint8).cpu().numpy(), xs.cpu().numpy()), ref.wide(gq.view(torch.uint8).cpu().numpy(), gs.cpu().numpy())
    _, order, _ = ar.sort_slots(ids, E)
    rows, of = np.zeros((T * k, N)), ids.reshape(-1)
    drows = np.zeros((T * k, K))
    for p, slot in enumerate(order):
        if slot >= 0:
            e = of[slot]
            rows[p] = (q[e] * float(s[e, 0])) @ xw[slot // k]
            drows[p] = (q[e].T * float(s[e, 0])) @ gw[p]
    def near(got, want, scale):
        assert np.abs(ar.wide(got) - want).max() <= 2.0 ** -18 * max(1.0, np.abs(scale).max())  # K + N sums of 24 bits
    near(out, ar.combine(rows, w.astype(np.float64), slots), K * 8)
    wy, wdw = ar.combine_backward(ar.wide(g), rows, w.astype(np.float64), slots)
    near(dw, wdw, K * 8 * N)
    used = int((slots >= 0).sum())
    assert np.array_equal(ar.wide(dy)[:used], wy[:used])
    near(dx, ar.dispatch_backward(drows, np.ones((T, k)), slots, np.zeros((T, K)))[0], N * 8)
