"""The exchange of tokens with experts and the low-rank adapters, as they are timed and compared:
slots sorted by given indices, rows sent to their places and the gradients of that exchange, adapters
of many requests beside a shared projection and their gradients.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, through the package's entry points.
"""

import math

import torch

import numpy as np

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
_GENERIC = (1024, 2048, 4096, 5120, 8192)
# No case reads and writes more elements: 8191 tokens of the 7B-shaped gate projection, base output and result
MOST_ROWS = 8191 * (4096 + 2 * 18944)


def listed():
    return [
        # the adapters of a batch of decoding sequences, a few of them without one
        {"name": "sort-64x1", "op": "sort", "T": 64, "E": 32, "k": 1, "runs": False, "masked": 3},
        # a prompt's choices of another router
        {"name": "sort-8192x8", "op": "sort", "T": 8192, "E": 256, "k": 8, "runs": False, "masked": 5},
        # rows of a decoding batch for experts that take weighted inputs
        {"name": "dispatch-33x4096", "op": "dispatch", "T": 33, "E": 64, "k": 8, "N": 4096, "weighted": True, "dtype": "bf16", "masked": 0},
        # the same for a prompt, unweighted
        {"name": "dispatch-2047x4096", "op": "dispatch", "T": 2047, "E": 64, "k": 8, "N": 4096, "weighted": False, "dtype": "bf16", "masked": 3},
        # gradients of the experts' rows and of the router's weights, a short sequence
        {"name": "combine-back-96x1023", "op": "combine_back", "T": 96, "E": 64, "k": 8, "N": 1023, "dtype": "fp16", "masked": 0},
        # the same for a training batch
        {"name": "combine-back-2047x4096", "op": "combine_back", "T": 2047, "E": 64, "k": 8, "N": 4096, "dtype": "bf16", "masked": 3},
        # gradient of the tokens that experts of weighted inputs took, and of their weights
        {"name": "dispatch-back-4096x2048", "op": "dispatch_back", "T": 4096, "E": 64, "k": 8, "N": 2048, "weighted": True, "add": True, "dtype": "bf16", "masked": 0},
        # adapter beside the 7B-shaped query projection, decoding one sequence
        {"name": "adapters-1-4096x4096", "op": "adapters", "T": 1, "E": 8, "r": 16, "N": 4096, "K": 4096, "dtype": "bf16", "runs": False, "masked": 0, "add": True, "hidden": False},
        # the same for 64 decoding sequences of up to 32 adapters
        {"name": "adapters-64-4096x4096", "op": "adapters", "T": 64, "E": 32, "r": 16, "N": 4096, "K": 4096, "dtype": "bf16", "runs": False, "masked": 3, "add": True, "hidden": False},
        # prompts of several requests beside the 7B-shaped gate projection
        {"name": "adapters-8191-18944x4096", "op": "adapters", "T": 8191, "E": 8, "r": 64, "N": 18944, "K": 4096, "dtype": "bf16", "runs": True, "masked": 0, "add": True, "hidden": False},
        # one adapter trained on a short batch
        {"name": "adapters-back-513-4096x4096", "op": "adapters_back", "T": 513, "E": 1, "r": 16, "N": 4096, "K": 4096, "dtype": "fp16", "runs": True, "masked": 0, "add": True},
        # several adapters trained at once, tokens of a large batch
        {"name": "adapters-back-8191-4096x4096", "op": "adapters_back", "T": 8191, "E": 4, "r": 32, "N": 4096, "K": 4096, "dtype": "bf16", "runs": True, "masked": 0, "add": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine_back", "dispatch_back", "adapters", "adapters", "adapters_back", "adapters_back"])
    T = _log(rng, 1, 8192)
    masked = rng.choice([0, 0, T // 7])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "sort":
        E = rng.randint(1, 512)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(10, E)), "runs": rng.choice([True, False]), "masked": masked}
    if op in ("dispatch", "combine_back", "dispatch_back"):
        E = rng.randint(4, 256)
        k = rng.randint(1, min(8, E))
        N = rng.choice([_log(rng, 64, 8192), rng.choice(_GENERIC)])
        c = {"op": op, "T": min(T, max(1, MOST_ROWS // (4 * k * N))), "E": E, "k": k, "N": N, "dtype": rng.choice(["bf16", "fp16", "fp32"])}
        if op != "combine_back":
            c["weighted"] = rng.choice([True, False])
        if op == "dispatch_back":
            c["add"] = rng.choice([True, False])
        return c | {"masked": min(masked, c["T"] // 7)}
    K, N = (rng.choice([_log(rng, 64, 8192), rng.choice(_GENERIC)]) for _ in range(2))
    r = rng.choice([8, 16, 32, 64, rng.randint(1, 128)])
    E = rng.choice([1, _log(rng, 1, 64 if T <= 512 else 16)])
    T = min(T, 8191 * 4096 // max(K, N))
    c = {"op": op, "T": T, "E": E, "r": r, "N": N, "K": K, "dtype": dtype, "runs": rng.choice([True, T > 256]),
         "masked": min(masked, T // 7), "add": rng.choice([True, True, False])}
    return c if op == "adapters_back" else c | {"hidden": rng.choice([True, False])}


# ---------------------------------------------------------------- what a user has in hand

def _activations(gen, rows, K, dtype):
    """Hidden states: normal values, some channels larger than the rest."""
    x = torch.randn(rows, K, device="cuda", generator=gen)
    x *= torch.exp(0.7 * torch.randn(K, device="cuda", generator=gen))
    return x.to(dtype)


def _ids(gen, c):
    """int32 [T, k]: the experts of a router, or each token's adapter: of its own (a decoding batch), or of the
    request whose run of tokens it belongs to. Masked tokens have none."""
    T, E, k = c["T"], c["E"], c.get("k", 1)
    if c.get("runs"):
        cuts = torch.rand(max(1, E - 1), device="cuda", generator=gen).sort().values * T
        at = torch.searchsorted(cuts, torch.arange(T, device="cuda", dtype=torch.float32), right=True)
        of = torch.rand(E, device="cuda", generator=gen).argsort()
        ids = (of[at % E][:, None] + torch.arange(k, device="cuda")) % E
    else:
        logits = torch.randn(T, E, device="cuda", generator=gen) + 0.4 * torch.randn(E, device="cuda", generator=gen)
        ids = logits.topk(k, dim=1).indices
    ids = ids.to(torch.int32)
    if c["masked"]:
        ids[T - c["masked"]:] = -1
    return ids.contiguous()


def _sorted_slots(ids, E):
    flat = ids.reshape(-1)
    key = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=key.device, dtype=key.dtype))
    place = torch.arange(flat.numel(), device=key.device)
    slots = torch.empty_like(place).scatter_(0, order, place)
    order = torch.where(place >= offsets[E], torch.full_like(order, -1), order)
    slots = torch.where(key == E, torch.full_like(slots, -1), slots).view(ids.shape)
    return {"offsets": offsets.to(torch.int32), "order": order.to(torch.int32), "slots": slots.to(torch.int32)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, s, op = case, {"case": case}, case["op"]
    T, E = c["T"], c["E"]
    ids = _ids(gen, c)
    if op == "sort":
        return s | {"ids": ids}
    w = torch.rand(ids.shape, device="cuda", generator=gen)
    w = torch.where(ids < 0, torch.zeros_like(w), w / w.sum(1, keepdim=True))
    r = s["routing"] = {"ids": ids, "weights": w} | _sorted_slots(ids, E)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, by=1.0):
        return (by * torch.randn(*shape, device="cuda", generator=gen)).to(dt)

    if op in ("dispatch", "combine_back", "dispatch_back"):
        R, N = T * c["k"], c["N"]
        if op == "dispatch":
            s |= {"x": _activations(gen, T, N, dt), "out": torch.zeros(R, N, device="cuda", dtype=dt)}
        elif op == "combine_back":
            s |= {"grad": normal(T, N, by=0.01), "y": normal(R, N), "out": torch.zeros(R, N, device="cuda", dtype=dt)}
        else:
            s |= {"grad": normal(R, N, by=0.01), "x": _activations(gen, T, N, dt) if c["weighted"] else None,
                  "add": normal(T, N, by=0.01) if c["add"] else None}
        return s
    K, N, rank = c["K"], c["N"], c["r"]
    s |= {"x": _activations(gen, T, K, dt), "a": normal(E, rank, K, by=K ** -0.5), "b": normal(E, N, rank, by=0.05),
          "scale": 0.5 + 1.5 * torch.rand(E, device="cuda", generator=gen), "ids": ids[:, 0].long(),
          "most": int((r["offsets"][1:] - r["offsets"][:-1]).max())}
    if op == "adapters":
        s |= {"add": normal(T, N) if c["add"] else None,
              "hidden": torch.zeros(T, rank, device="cuda") if c["hidden"] else None}
    else:
        s |= {"grad": normal(T, N, by=0.01), "add": normal(T, K, by=0.01) if c["add"] else None}
        rows, back = _by_adapter(c, s)
        s["hidden"] = back(_down(c, s, rows(s["x"]), s["a"].float()))
    return s


# ---------------------------------------------------------------- plain forms

def _plain_dispatch(c, s):
    r, order = s["routing"], s["routing"]["order"].long()
    at = order.clamp_min(0)
    rows = s["x"].float()[at // c["k"]]
    if c["weighted"]:
        rows = rows * r["weights"].reshape(-1)[at][:, None]
    return torch.where((order >= 0)[:, None], rows, torch.zeros_like(rows)).to(s["x"].dtype)


def _plain_combine_back(c, s):
    r, order, slots = s["routing"], s["routing"]["order"].long(), s["routing"]["slots"].long()
    at = order.clamp_min(0)
    g = s["grad"].float()[at // c["k"]]
    dy = g * r["weights"].reshape(-1)[at][:, None]
    dy = torch.where((order >= 0)[:, None], dy, torch.zeros_like(dy)).to(s["y"].dtype)
    dw = (s["y"].float() * g).sum(1)[slots.clamp_min(0)]
    return {"y": dy, "weights": torch.where(slots >= 0, dw, torch.zeros_like(dw))}


def _plain_dispatch_back(c, s):
    r, slots = s["routing"], s["routing"]["slots"].long()
    rows = s["grad"].float()[slots.clamp_min(0)]
    rows = torch.where((slots >= 0)[:, :, None], rows, torch.zeros_like(rows))
    dx = (rows * r["weights"][:, :, None] if c["weighted"] else rows).sum(1)
    dx = (dx + s["add"].float() if s["add"] is not None else dx).to(s["grad"].dtype)
    return {"x": dx, "weights": (rows * s["x"].float()[:, None, :]).sum(2)} if c["weighted"] else dx


def _by_adapter(c, s):
    """Two functions: rows of tokens -> the rows of each adapter side by side [E, most, .], and back. As few tokens as
    adapters: each token with a copy of its own adapter instead."""
    r, T, E = s["routing"], c["T"], c["E"]
    has = s["ids"] >= 0
    if T <= E:
        return (lambda v: torch.where(has[:, None], v.float(), 0.0)[:, None, :]), (lambda v: torch.where(has[:, None], v[:, 0], 0.0))
    off = r["offsets"].long()
    at = off[:-1, None] + torch.arange(max(1, s["most"]), device="cuda")
    used = at < off[1:, None]
    tok = r["order"].long()[at.clamp_max(T - 1)].clamp_min(0)
    of = s["ids"].clamp_min(0)
    place = r["slots"].long()[:, 0].clamp_min(0) - off[of]

    def rows(v):
        return torch.where(used[:, :, None], v[tok].float(), 0.0)

    def back(v):
        return torch.where(has[:, None], v[of, place.clamp(0, v.shape[1] - 1)], 0.0)
    return rows, back


def _own(c, s, w):
    """An adapter's part of `w`, beside the rows that _by_adapter gives."""
    return w[s["ids"].clamp_min(0)] if c["T"] <= c["E"] else w


def _down(c, s, rows, a):
    return torch.bmm(rows, _own(c, s, a).transpose(1, 2).contiguous())


def _sum_by_adapter(c, s, grads):
    """Gradients of _own()'s copies, added up by adapter."""
    if c["T"] > c["E"]:
        return grads
    grads = torch.where((s["ids"] >= 0)[:, None, None], grads, 0.0)
    return torch.zeros(c["E"], *grads.shape[1:], device="cuda").index_add_(0, s["ids"].clamp_min(0), grads)


def _plain_adapters(c, s):
    rows, back = _by_adapter(c, s)
    v = _down(c, s, rows(s["x"]), s["a"].float())
    y = torch.bmm(v * _own(c, s, s["scale"])[:, None, None], _own(c, s, s["b"].float()).transpose(1, 2).contiguous())
    y = back(y)
    y = (y + s["add"].float() if s["add"] is not None else y).to(s["x"].dtype)
    return {"y": y, "hidden": back(v)} if c["hidden"] else y


def _plain_adapters_back(c, s):
    rows, back = _by_adapter(c, s)
    dt = s["x"].dtype
    g = rows(s["grad"]) * _own(c, s, s["scale"])[:, None, None]
    dv = torch.bmm(g, _own(c, s, s["b"].float()).contiguous())
    db = torch.bmm(g.transpose(1, 2).contiguous(), rows(s["hidden"]))
    da = torch.bmm(dv.transpose(1, 2).contiguous(), rows(s["x"]))
    dx = back(torch.bmm(dv, _own(c, s, s["a"].float()).contiguous()))
    dx = (dx + s["add"].float() if s["add"] is not None else dx).to(dt)
    return {"x": dx, "a": _sum_by_adapter(c, s, da).to(dt), "b": _sum_by_adapter(c, s, db).to(dt)}


def run(state):
    c, op, s = state["case"], state["case"]["op"], state
    if own:
        import gemm_ternary_linear_amd as tl
        if op == "sort":
            r = tl.sort_slots(s["ids"], c["E"])
            return {"offsets": r.offsets, "order": r.order, "slots": r.slots}
        r = tl.Routing(**s["routing"])
        if op == "dispatch":
            return tl.dispatch(s["x"], r, weighted=c["weighted"], out=s["out"])
        if op == "combine_back":
            return dict(zip(("y", "weights"), tl.combine_backward(s["grad"], s["y"], r, out=s["out"])))
        if op == "dispatch_back":
            got = tl.dispatch_backward(s["grad"], r, x=s["x"], add=s["add"])
            return dict(zip(("x", "weights"), got)) if c["weighted"] else got
        if op == "adapters":
            y = tl.linear_adapters(s["x"], s["a"], s["b"], r, s["scale"], add=s["add"], hidden=s["hidden"])
            return {"y": y, "hidden": s["hidden"]} if c["hidden"] else y
        return dict(zip("xab", tl.linear_adapters_backward(s["grad"], s["x"], s["hidden"], s["a"], s["b"], r, s["scale"], add=s["add"])))
    if op == "sort":
        return _sorted_slots(s["ids"], c["E"])
    return {"dispatch": _plain_dispatch, "combine_back": _plain_combine_back, "dispatch_back": _plain_dispatch_back,
            "adapters": _plain_adapters, "adapters_back": _plain_adapters_back}[op](c, s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c, op, T, E = case, case["op"], case["T"], case["E"]
    rows = T - c["masked"]
    if op == "sort":
        return {"bytes": 12 * T * c["k"] + 4 * (E + 1), "flops": T * c["k"]}
    e, N = SIZES[c["dtype"]], c["N"]
    if op == "dispatch":
        return {"bytes": rows * N * e * (1 + c["k"]) + T * c["k"] * (8 if c["weighted"] else 4), "flops": rows * c["k"] * N}
    if op == "combine_back":
        return {"bytes": rows * N * e * (1 + 2 * c["k"]) + 16 * T * c["k"], "flops": 3 * rows * c["k"] * N}
    if op == "dispatch_back":
        more = 1 + c["weighted"] + c["add"]
        return {"bytes": rows * N * e * c["k"] + T * N * e * more + T * c["k"] * (12 if c["weighted"] else 4),
                "flops": rows * c["k"] * N * (4 if c["weighted"] else 1)}
    K, r = c["K"], c["r"]
    touched = E * (1 - (1 - 1 / E) ** rows) if not c["runs"] else min(E, rows)  # adapters that some token takes, on average
    weights = int(touched * r * (K + N) * e)
    if op == "adapters":
        return {"bytes": rows * K * e + weights + T * N * e * (2 if c["add"] else 1) + (4 * T * r if c["hidden"] else 0),
                "flops": 2 * rows * r * (K + N)}
    return {"bytes": rows * (K + N) * e + 4 * rows * r + weights + T * K * e * (2 if c["add"] else 1) + E * r * (K + N) * e,
            "flops": 4 * rows * r * (K + N)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _order_of(ids, E):
    """numpy: places by expert, slots in ascending order."""
    flat = ids.reshape(-1).astype(np.int64)
    have = np.nonzero((flat >= 0) & (flat < E))[0]
    have = have[np.argsort(flat[have], kind="stable")]
    counts = np.bincount(flat[have], minlength=E)
    return have, np.concatenate([[0], np.cumsum(counts)])


def exact(case, seed):
    c, s, op = case, prepare(case, seed), case["op"]
    T, E = c["T"], c["E"]
    if op == "sort":
        have, offsets = _order_of(s["ids"].cpu().numpy(), E)
        order, slots = np.full(T * c["k"], -1), np.full(T * c["k"], -1)
        order[:have.size], slots[have] = have, np.arange(have.size)
        return {"offsets": offsets, "order": order, "slots": slots.reshape(T, c["k"])}
    have, offsets = _order_of(s["routing"]["ids"].cpu().numpy(), E)
    if op in ("dispatch", "combine_back", "dispatch_back"):
        k, N = c["k"], c["N"]
        have = torch.from_numpy(have).cuda()
        w = s["routing"]["weights"].double().reshape(-1)[have][:, None]
        if op == "dispatch":
            out = torch.zeros(T * k, N, device="cuda", dtype=torch.float64)
            out[:have.numel()] = s["x"].double()[have // k] * (w if c["weighted"] else 1)
            return out
        dw = torch.zeros(T * k, device="cuda", dtype=torch.float64)
        if op == "combine_back":
            g, y = s["grad"].double()[have // k], s["y"].double()[:have.numel()]
            dw[have] = (g * y).sum(1)
            out = torch.zeros(T * k, N, device="cuda", dtype=torch.float64)
            out[:have.numel()] = g * w
            return {"y": out, "weights": dw.view(T, k)}
        g = s["grad"].double()[:have.numel()]
        dx = torch.zeros(T, N, device="cuda", dtype=torch.float64) if s["add"] is None else s["add"].double()
        for j in range(k):
            mine = (have % k == j).nonzero()[:, 0]
            dx[have[mine] // k] += g[mine] * (w[mine] if c["weighted"] else 1)
        if not c["weighted"]:
            return dx
        dw[have] = (g * s["x"].double()[have // k]).sum(1)
        return {"x": dx, "weights": dw.view(T, k)}
    f64 = {"device": "cuda", "dtype": torch.float64}
    K, N, rank = c["K"], c["N"], c["r"]
    if op == "adapters":
        y = torch.zeros(T, N, **f64) if s["add"] is None else s["add"].double()
        hidden = torch.zeros(T, rank, **f64)
    else:
        y = torch.zeros(T, K, **f64) if s["add"] is None else s["add"].double()
        da, db = torch.zeros(E, rank, K, **f64), torch.zeros(E, N, rank, **f64)
    for e in range(E):
        tok = torch.from_numpy(have[offsets[e]:offsets[e + 1]]).cuda()
        if not tok.numel():
            continue
        a, b, by, x = s["a"][e].double(), s["b"][e].double(), float(s["scale"][e]), s["x"][tok].double()
        if op == "adapters":
            hidden[tok] = x @ a.t().contiguous()
            y[tok] += by * (hidden[tok] @ b.t().contiguous())
        else:
            g = by * s["grad"][tok].double()
            dv = g @ b
            y[tok] += dv @ a
            da[e], db[e] = dv.t().contiguous() @ x, g.t().contiguous() @ s["hidden"][tok].double()
    if op == "adapters":
        return {"y": y, "hidden": hidden} if c["hidden"] else y
    return {"x": y, "a": da, "b": db}
