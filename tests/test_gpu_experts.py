"""route, linear_experts and combine against 64-bit references, and a whole mixture of experts."""

import weakref

import numpy as np
import pytest
import torch

import fp8_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def tl():
    import gemm_ternary_linear_amd as tl
    return tl


def check_route(tl, logits, k, score="softmax", bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """logits: float32 numpy or a device tensor."""
    lt = logits if torch.is_tensor(logits) else ref.dev(logits)
    T, E = lt.shape
    say(f"route T={T} E={E} k={k} {score} bias={bias is not None} groups={groups}/{top_groups}")
    r = tl.route(lt, k, score=score, bias=None if bias is None else ref.dev(bias), groups=groups, top_groups=top_groups,
                 renormalize=renormalize, scale=scale)
    ids, w = ref.route(lt.float().cpu().numpy(), k, score == "sigmoid", bias, groups, top_groups, renormalize, scale)
    off, order, slots = ref.sort_slots(ids, E)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    # 64-bit scores rounded once to 32 bits: half a step, and the 64-bit differences far below
    assert np.all(np.abs(r.weights.cpu().numpy() - w) <= 2.0 ** -24 * np.abs(w) * 1.001 + 2.0 ** -149)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    assert np.array_equal(r.order.cpu().numpy(), order)
    assert np.array_equal(r.slots.cpu().numpy(), slots)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(0, 8, 2), (1, 1, 1), (1, 64, 8), (2, 3, 3), (15, 65, 6), (16, 128, 8), (17, 100, 1), (64, 512, 32), (65, 64, 8),
                                   (63, 256, 10), (32, 96, 5), (33, 96, 5), (33, 64, 5), (64, 64, 3), (4096, 40, 2), (4097, 40, 2), (130, 129, 7), (333, 512, 32), (1000, 60, 4), (1024, 256, 8), (1, 512, 32), (1, 40, 32)])
def test_route(tl, T, E, k, score):
    rng = np.random.default_rng(T + E + k)
    logits = (2 * rng.standard_normal((T, E))).astype(np.float32)
    check_route(tl, logits, k, score)
    check_route(tl, logits, k, score, bias=(0.2 * rng.standard_normal(E)).astype(np.float32), renormalize=False, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (64, 64, 5, 5), (8, 4, 1, 2), (96, 3, 2, 9), (512, 2, 1, 32), (160, 8, 8, 6), (330, 5, 3, 7)])
@pytest.mark.parametrize("T", [7, 200])
def test_route_groups(tl, T, E, groups, top_groups, k, score):
    rng = np.random.default_rng(T + E)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[::5, :E // groups] = -np.inf       # a group without experts
    logits[1::5, 1:E // groups] = -np.inf     # one with a single expert
    check_route(tl, logits, k, score, (0.3 * rng.standard_normal(E)).astype(np.float32), groups, top_groups)
    check_route(tl, logits, k, score, None, groups, top_groups, renormalize=False)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T", [9, 100])
def test_route_ties_and_masks(tl, T, dtype):
    """Coarse logits (many ties), rows with few or no experts left, infinities and NaN."""
    rng = np.random.default_rng(T)
    l = np.round(rng.standard_normal((T, 70)) * 2) / 2
    l[1] = -np.inf
    l[2, 3:] = -np.inf
    l[3, ::2] = np.nan
    l[4, 5] = l[4, 60] = np.inf
    l[5] = 0
    l[6] = np.finfo(np.float32).min if dtype != "fp16" else -65504
    l[7, 1:] = -np.inf
    l[8] = 700 * rng.standard_normal(70)
    lt = torch.from_numpy(l.astype(np.float32)).to(DT[dtype]).cuda()
    bias = (0.25 * rng.integers(-2, 3, 70)).astype(np.float32)
    bias[9], bias[10] = -np.inf, np.nan
    for score in ("softmax", "sigmoid"):
        check_route(tl, lt, 5, score)
        check_route(tl, lt, 5, score, bias)
        check_route(tl, lt, 5, score, bias, groups=7, top_groups=3)


def test_route_many_tokens(tl):
    """Over the limits of one and of two kernels: ids against an order by 64-bit scores, the sort against its meaning."""
    for T, E, k in [(8192, 64, 4), (8193, 256, 8), (20011, 96, 6)]:
        say(f"route many T={T}")
        g = torch.Generator(device="cuda").manual_seed(T)
        l = torch.randn(T, E, generator=g, device="cuda")
        l[T // 2] = -torch.inf
        r = tl.route(l, k)
        ids = l.double().sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
        ids[T // 2] = -1
        assert torch.equal(r.ids, ids)
        off, order, slots = ref.sort_slots(ids.cpu().numpy(), E)
        for a, b in ((r.offsets, off), (r.order, order), (r.slots, slots)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_route_holds_its_workspace(tl, monkeypatch):
    """The workspace lives until the kernels are enqueued: freed before, another thread could be given it between
    them (the call lets other threads run)."""
    say("route workspace")
    made, alive, empty, call = [], [], torch.empty, tl._call

    def recording(*a, **kw):
        t = empty(*a, **kw)
        if kw.get("dtype") == torch.uint8:
            made.append(weakref.ref(t))
        return t

    def checked(name, *a):
        alive.extend(r() is not None for r in made)
        return call(name, *a)

    monkeypatch.setattr(tl.torch, "empty", recording)
    monkeypatch.setattr(tl, "_call", checked)
    r = tl.route(torch.randn(200, 64, device="cuda"), 8)
    assert alive == [True] and bool((r.ids >= 0).all())


def routing(tl, ids, w, E):
    off, order, slots = ref.sort_slots(ids, E)
    return tl.Routing(ref.dev(ids), ref.dev(w), ref.dev(off), ref.dev(order), ref.dev(slots))


def draw_ids(rng, T, E, k, masked, skew):
    pop = rng.standard_normal(E) * skew
    ids = np.argsort(-(pop + rng.standard_normal((T, E))), axis=1)[:, :k].astype(np.int32)
    if masked:
        ids[rng.choice(T, masked, replace=False)] = -1
        ids[0, k - 1] = -1
    return ids


def experts_ref(xw, q, s, g, ids, k, by_token):
    E, N, K = q.shape
    off, order, _ = ref.sort_slots(ids, E)
    y, used = np.zeros((ids.size, N)), int(off[E])
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        w = q[e] * (s[e].astype(np.float64)[:, None] if g == -1 else np.repeat(s[e].astype(np.float64), g, 1))
        rows = order[lo:hi] // k if by_token else np.arange(lo, hi)
        y[lo:hi] = xw[rows][:, :K] @ w.T
    return y, used


EXPERT_CASES = [
    # T, E, k, N, K, group, masked, skew
    (1, 8, 2, 64, 256, -1, 0, 0), (1, 64, 8, 256, 1024, 128, 0, 0), (2, 4, 1, 17, 260, -1, 0, 0), (5, 3, 3, 100, 128, 128, 1, 0),
    (9, 96, 6, 130, 140, -1, 2, 1), (16, 1, 1, 33, 512, 256, 0, 0), (33, 16, 4, 512, 1024, 128, 0, 0), (40, 8, 2, 260, 384, 128, 5, 2),
    (64, 5, 5, 48, 4, -1, 0, 0), (100, 512, 8, 20, 256, -1, 0, 0), (130, 4, 2, 300, 640, -1, 7, 1), (200, 70, 3, 144, 768, 256, 0, 3),
    (300, 2, 1, 256, 256, 128, 0, 0), (500, 8, 4, 272, 388, -1, 50, 1), (600, 3, 2, 132, 1280, 256, 0, 1), (1500, 8, 2, 128, 512, -1, 9, 1)]


@pytest.mark.parametrize("rows", ["tokens", "sorted"])
@pytest.mark.parametrize("T,E,k,N,K,g,masked,skew", EXPERT_CASES)
def test_experts_exact(tl, T, E, k, N, K, g, masked, skew, rows):
    """Whole-number codes, power-of-two scales: every output bit is known; rows past offsets[E] are left alone."""
    say(f"experts {T} {E} {k} {N} {K} g={g} {rows}")
    rng = np.random.default_rng(T + E + N + K)
    ids = draw_ids(rng, T, E, k, masked, skew)
    n, Kp = (T if rows == "tokens" else T * k), ref.up(K, 128)
    xq, xs = ref.codes_of(rng, n, Kp), ref.scales_of(rng, n, Kp // 128)
    xq[:, K:] = 0
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = ref.scales_of(rng, *((E, N) if g == -1 else (E, N, K // g))).astype(np.float16)
    y, used = experts_ref(ref.wide(xq, xs), q, s, g, ids, k, rows == "tokens")
    assert np.abs(y).max(initial=0) < 2.0 ** 19  # steps of 1/16: exact in 32 bits
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    r = routing(tl, ids, np.zeros(ids.shape, np.float32), E)
    for name, dt in DT.items():
        buf = torch.full((T * k * N + 64,), 77.0, dtype=dt, device="cuda")
        out = buf[32:32 + T * k * N].view(T * k, N)
        got = tl.linear_experts(ref.fp8_dev(xq), ref.dev(xs), codes, ref.dev(s), r, K=K, rows=rows, out=out)
        assert got is out and np.array_equal(out[:used].double().cpu().numpy(), ref.rounded(y[:used], dt)), name
        assert bool((buf[:32] == 77).all()) and bool((buf[32 + used * N:] == 77).all()), name


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,k,N,K,g", [(1, 16, 4, 256, 2048, -1), (30, 8, 2, 200, 1024, 128), (400, 4, 2, 300, 512, 256)])
def test_experts(tl, T, E, k, N, K, g, dtype):
    say(f"experts real {dtype} {T} {E} {k} {N} {K} g={g}")
    rng = np.random.default_rng(T + N)
    ids = draw_ids(rng, T, E, k, 0, 1)
    xq, xs = ref.quantize((rng.standard_normal((T, K)) * np.exp(0.7 * rng.standard_normal(K))).astype(np.float32), False)
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = (0.01 + 0.02 * rng.random((E, N) if g == -1 else (E, N, K // g))).astype(np.float16)
    xw = ref.wide(xq, xs)
    y, _ = experts_ref(xw, q, s, g, ids, k, True)
    off, order, _ = ref.sort_slots(ids, E)
    bound = np.zeros_like(y)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        w = q[e] * (s[e].astype(np.float64)[:, None] if g == -1 else np.repeat(s[e].astype(np.float64), g, 1))
        bound[lo:hi] = ref.product_bound(xw[order[lo:hi] // k], w, K // 128, DT[dtype], y[lo:hi])
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    r = routing(tl, ids, np.zeros(ids.shape, np.float32), E)
    args = (ref.fp8_dev(xq), ref.dev(xs), codes, ref.dev(s), r)
    got = tl.linear_experts(*args, dtype=DT[dtype])
    assert np.all(np.abs(got.double().cpu().numpy() - y) <= bound)
    assert torch.equal(got, tl.linear_experts(*args, dtype=DT[dtype])), "the same inputs give the same bits"


@pytest.mark.parametrize("T", [4, 500])
def test_experts_foreign_indices(tl, T):
    """Offsets and order that do not describe a routing: nothing outside the arguments is read or written, and the
    rows that they leave out stay as they were."""
    say(f"experts foreign indices T={T}")
    rng = np.random.default_rng(T)
    E, k, N, K = 5, 2, 48, 256
    xq, xs = ref.codes_of(rng, T, K), ref.scales_of(rng, T, K // 128)
    codes = torch.stack([torch.from_numpy(ref.tile_codes(rng.integers(-1, 2, (N, K)).astype(np.int8))) for _ in range(E)]).cuda()
    s = ref.dev(ref.scales_of(rng, E, N).astype(np.float16))
    R = T * k
    r = routing(tl, draw_ids(rng, T, E, k, 0, 0), np.zeros((T, k), np.float32), E)
    for off in ([0, R, -7, R + 100, 3, 2 ** 31 - 1], [-2 ** 31, -5, -1, 0, 0, 0], [5, 4, 3, 2, 1, 0], [R] * 6):
        order = torch.full((R,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
        order[::2] = -2 ** 31
        bad = r._replace(offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), order=order)
        buf = torch.full((R * N + 64,), 77.0, device="cuda")
        tl.linear_experts(ref.fp8_dev(xq), ref.dev(xs), codes, s, bad, out=buf[32:32 + R * N].view(R, N))
        torch.cuda.synchronize()
        assert bool((buf[:32] == 77).all()) and bool((buf[32 + R * N:] == 77).all())
        if max(off) <= 0 or off[0] >= R:
            assert bool((buf == 77).all())
    bad = r._replace(slots=torch.where(r.slots % 3 == 0, torch.full_like(r.slots, 2 ** 31 - 1), torch.full_like(r.slots, -9)))
    y = torch.full((R, 40), torch.nan, device="cuda")
    assert bool((tl.combine(y, bad) == 0).all())


@pytest.mark.parametrize("T", [3, 90, 700])
def test_experts_rows_apart(tl, T):
    """A NaN in one token's x shows in that token's rows only; a NaN scale of an expert in that channel only."""
    say(f"experts NaN T={T}")
    rng = np.random.default_rng(T)
    E, k, N, K = 6, 2, 80, 384
    ids = draw_ids(rng, T, E, k, 0, 0)
    xq, xs = ref.codes_of(rng, T, K), ref.scales_of(rng, T, K // 128)
    q = rng.integers(-1, 2, (E, N, K)).astype(np.int8)
    s = ref.scales_of(rng, E, N).astype(np.float16)
    y, _ = experts_ref(ref.wide(xq, xs), q, s, -1, ids, k, True)
    xq[T - 1, 200] = 0x7f
    s[2, 5] = np.nan
    off, order, _ = ref.sort_slots(ids, E)
    nan = np.zeros(y.shape, bool)
    nan[order // k == T - 1] = True
    nan[off[2]:off[3], 5] = True
    codes = torch.stack([torch.from_numpy(ref.tile_codes(e)) for e in q]).cuda()
    got = tl.linear_experts(ref.fp8_dev(xq), ref.dev(xs), codes, ref.dev(s), routing(tl, ids, np.zeros(ids.shape, np.float32), E),
                            dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(got), nan) and np.array_equal(got[~nan], y[~nan])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,N,add", [(1, 1, 1, False), (1, 8, 4096, True), (7, 3, 17, True), (33, 32, 260, False), (300, 8, 1024, True), (64, 4, 8, False)])
def test_combine(tl, T, k, N, add, dtype):
    say(f"combine {dtype} {T} {k} {N}")
    rng = np.random.default_rng(T + k + N)
    dt, R = DT[dtype], T * k
    y = torch.from_numpy(rng.standard_normal((R, N)).astype(np.float32)).to(dt).cuda()
    a = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).to(dt).cuda() if add else None
    ids = draw_ids(rng, T, max(k, 40), k, T // 4, 0)
    r = routing(tl, ids, rng.random((T, k)).astype(np.float32), max(k, 40))
    used = int((ids >= 0).sum())
    y[used:] = torch.nan  # places without a slot are not read
    w, sl = r.weights.double().cpu().numpy(), r.slots.cpu().numpy()
    yv = np.nan_to_num(y.double().cpu().numpy())
    terms = np.where(sl >= 0, w, 0)[:, :, None] * yv[np.maximum(sl, 0)]
    base = a.double().cpu().numpy() if add else 0
    want, mags = terms.sum(1) + base, np.abs(terms).sum(1) + np.abs(base)
    got = tl.combine(y, r, add=a)
    # k products and k sums, each half a step of fp32 of at most the magnitudes' sum; the output's rounding
    lim = 2 * k * 2.0 ** -24 * mags + ref.EPS[dt] * np.abs(want) + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    assert got.dtype == dt and np.all(np.abs(got.double().cpu().numpy() - want) <= lim)
    if add:
        assert torch.equal(tl.combine(y, r, add=a, out=a), got)


def mixture(tl, x, gate_q, gate_s, up, up_s, down, down_s, k, K, I, add=None, **kw):
    """A mixture of ternary experts, as a user of the operators writes it."""
    xq, xs = tl.fp8_quantize(x)
    r = tl.route(tl.fp8_linear(xq, xs, gate_q, gate_s, dtype=torch.float32), k, **kw)
    h = tl.linear_experts(xq, xs, up, up_s, r, K=K, dtype=x.dtype)
    hq, hs = tl.fp8_quantize(h, act="swiglu")
    return tl.combine(tl.linear_experts(hq, hs, down, down_s, r, K=I, rows="sorted", dtype=x.dtype), r, add=add), r


@pytest.fixture(scope="module")
def layer(tl):
    g = torch.Generator(device="cuda").manual_seed(9)
    E, k, K, I = 24, 4, 512, 200
    gate_q, gate_s = tl.fp8_quantize(0.1 * torch.randn(E, K, generator=g, device="cuda"), block="tile")
    def weights(N, K, groups):
        q = torch.randint(-1, 2, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
        s = (0.02 + 0.02 * torch.rand(E, N, *groups, generator=g, device="cuda")).half()
        return torch.stack([tl.tile(tl.pack(e)) for e in q]), s, q
    up, up_s, up_q = weights(2 * I, K, (K // 128,))
    down, down_s, down_q = weights(K, I, ())
    return dict(gate_q=gate_q, gate_s=gate_s, up=up, up_s=up_s, down=down, down_s=down_s, k=k, K=K, I=I), up_q, down_q


@pytest.mark.parametrize("T", [1, 2, 19, 150, 700])
def test_mixture(tl, layer, T):
    """The chain end to end against the layer in 64 bits with unquantised activations: 8-bit activations cost at
    most a relative 2^-4 each of two times; measured as a whole by the norm."""
    say(f"mixture T={T}")
    p, up_q, down_q = layer
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, p["K"], generator=g, device="cuda").to(torch.bfloat16)
    out, r = mixture(tl, x, add=x, score="sigmoid", **p)
    ids, w = r.ids.cpu().numpy(), r.weights.double().cpu().numpy()
    assert (ids >= 0).all() and np.allclose(w.sum(1), 1)
    xw = x.double().cpu().numpy()
    us = p["up_s"].double().cpu().numpy().repeat(128, 2)
    ds = p["down_s"].double().cpu().numpy()[:, :, None]
    want = xw.copy()
    for t in range(T):
        for j in range(p["k"]):
            e = ids[t, j]
            h = (up_q[e].cpu().numpy() * us[e]) @ xw[t]
            h = h[:p["I"]] / (1 + np.exp(-h[:p["I"]])) * h[p["I"]:]
            want[t] += w[t, j] * ((down_q[e].cpu().numpy() * ds[e]) @ h)
    err = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want - xw)
    assert err < 2.0 ** -3, err


def test_mixture_padded_captured(tl, layer):
    """Padded tokens take no slots and change nobody's result; captured, replayed, and on two streams at once."""
    say("mixture captured")
    p, _, _ = layer
    x = torch.randn(100, p["K"], device="cuda").to(torch.bfloat16)
    for T in (100, 40):
        xt = x[:T].clone()
        torch.cuda.synchronize()
        eager, _ = mixture(tl, xt, **p)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out, r = mixture(tl, xt, **p)
        for rep in range(4):
            xt.copy_(torch.randn_like(xt))
            gr.replay()
            torch.cuda.synchronize()
            want, wr = mixture(tl, xt, **p)
            assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(r, wr)), rep
        got = []
        for rep in range(10):
            gr.replay()
            with torch.cuda.stream(side):
                got.append(mixture(tl, xt, **p)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, want) for g in got) and torch.equal(out, want)
    xq, xs = tl.fp8_quantize(x)
    logits = tl.fp8_linear(xq, xs, p["gate_q"], p["gate_s"], dtype=torch.float32)
    masked = logits.clone()
    masked[60:] = -torch.inf
    a, b = tl.route(logits[:60].contiguous(), 4), tl.route(masked, 4)
    assert torch.equal(a.ids, b.ids[:60]) and bool((b.ids[60:] == -1).all()) and torch.equal(a.offsets, b.offsets)
    assert torch.equal(a.order, b.order[:240]) and bool((b.order[240:] == -1).all())
