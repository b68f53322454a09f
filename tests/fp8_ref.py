"""Plain 64-bit definitions of the 8-bit and experts' operators (numpy, CPU), and the
inputs their tests share.  No code of the library is used."""

import numpy as np
import torch

BLOCK = 128
EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step


def up(n, m):
    return (n + m - 1) // m * m


def e4m3_table():
    """The value of each of the 256 codes."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = np.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v[c] = -mag if c & 128 else mag
    return v


TABLE = e4m3_table()


def nearest_code(v):
    """float64 [...] -> the e4m3 code of the nearest value, ties to the even code, the largest beyond 448."""
    pos = TABLE[:127]  # 0 .. 448, ascending
    mag = np.minimum(np.abs(v), 448.0)
    hi = np.clip(np.searchsorted(pos, mag), 1, 126)
    lo = hi - 1
    dl, dh = mag - pos[lo], pos[hi] - mag
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = code | np.where(np.signbit(v), 128, 0)
    return np.where(np.isnan(v), 0x7f, code).astype(np.uint8)


def quantize(x, tile):
    """float32 [M, K] -> codes [M, Kp], scales, with the stored scale and the quotient rounded to fp32."""
    M, K = x.shape
    kb, rows = up(K, BLOCK) // BLOCK, BLOCK if tile else 1
    full = np.zeros((up(M, rows), kb * BLOCK), np.float32)
    full[:M, :K] = x
    t = full.reshape(-1, rows, kb, BLOCK)
    big = np.fmax.reduce(np.abs(t), axis=(1, 3))
    big = np.where(np.isnan(big), np.float32(0), big)
    s = (big / np.float32(448)).astype(np.float32)
    with np.errstate(all="ignore"):
        d = np.where(s[:, None, :, None] > 0, t / s[:, None, :, None], np.where(np.isnan(t), t, np.float32(0)))
    return nearest_code(d.astype(np.float64)).reshape(full.shape)[:M], s


def wide(q, s, rows=1):
    """Codes and scales -> the float64 values they stand for."""
    s = np.repeat(np.repeat(np.asarray(s, np.float64), BLOCK, 1), rows, 0)
    return TABLE[q] * s[:q.shape[0]]


def codes_of(rng, *shape):
    """Small whole numbers -8 .. 8 as codes: products and sums of them are exact in fp32."""
    return nearest_code(rng.integers(-8, 9, shape).astype(np.float64))


def scales_of(rng, *shape):
    return np.ldexp(np.float32(1), rng.integers(-2, 3, shape)).astype(np.float32)


def route(logits, k, sigmoid, bias, groups, top_groups, renorm, scale):
    """One token at a time: ids, float64 weights."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    for t in range(T):
        l = np.minimum(logits[t].astype(np.float64), float(np.finfo(np.float32).max))
        with np.errstate(invalid="ignore"):
            free = (logits[t] > -np.inf) & (b > -np.inf)
        p = np.zeros(E)
        if free.any():
            with np.errstate(over="ignore"):
                if sigmoid:
                    p[free] = 1 / (1 + np.exp(-l[free]))
                else:
                    e = np.exp(l[free] - l[free].max())
                    p[free] = e / e.sum()
        c = [(p[i] + b[i] if free[i] else -np.inf) for i in range(E)]
        if groups > 1:
            per = E // groups
            worth = []
            for g in range(groups):
                best = sorted((v for v in c[g * per:(g + 1) * per] if v > -np.inf), reverse=True)[:2]
                worth.append(sum(best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            c = [v if i // per in kept else -np.inf for i, v in enumerate(c)]
        best = [i for i in sorted(range(E), key=lambda i: (-c[i], i))[:k] if c[i] > -np.inf]
        ids[t, :len(best)] = best
        w[t, :len(best)] = p[best]
        if renorm and w[t].sum() > 0:
            w[t] /= w[t].sum()
    return ids, w * scale


def sort_slots(ids, E):
    """offsets, order, slots of ids [T, k] (-1: none)."""
    flat = ids.reshape(-1)
    order, offsets = [], [0]
    for e in range(E):
        order += np.nonzero(flat == e)[0].tolist()
        offsets.append(len(order))
    slots = np.full(flat.size, -1, np.int32)
    slots[order] = np.arange(len(order))
    order = np.array(order + [-1] * (flat.size - len(order)), np.int32)
    return np.array(offsets, np.int32), order, slots.reshape(ids.shape)


def tile_codes(q):
    """int [N, K] of 0, +1, -1 -> the tiled layout [ceil(N/16), ceil(K/256), 1024], byte by byte's rule."""
    N, K = q.shape
    full = np.zeros((up(N, 16), up(K, 256)), np.uint8)
    full[:N, :K] = np.where(q < 0, 2, q)
    b = full.reshape(full.shape[0], -1, 4)
    packed = b[..., 0] | b[..., 1] << 2 | b[..., 2] << 4 | b[..., 3] << 6
    t = packed.reshape(full.shape[0] // 16, 16, full.shape[1] // 256, 4, 16)
    return np.ascontiguousarray(t.transpose(0, 2, 3, 1, 4)).reshape(full.shape[0] // 16, -1, 1024)


def fp8_dev(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).cuda().view(torch.float8_e4m3fn)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rounded(y, dtype):
    """float64 -> dtype, to nearest even, as float64 (exact where y fits in fp32)."""
    return torch.from_numpy(np.ascontiguousarray(y)).to(torch.float32).to(dtype).double().numpy()


def product_bound(xw, ww, nb, dtype, y):
    """How far an output may be from the 64-bit sum `y`.  Of a block, 128 exact products are summed in
    fp32 and the nb blocks' scaled sums after them: at most 128 + 2 nb + 4 roundings (sums, the
    scales' product, its product with the sum, a channel scale), each at most 2^-23 of the sum of
    magnitudes (2^-23 and not 2^-24, as the matrix unit may cut where it aligns); then the output's."""
    mags = np.abs(xw) @ np.abs(ww).T
    return (128 + 2 * nb + 4) * 2.0 ** -23 * mags + EPS[dtype] * (np.abs(y) + 1e-30) + (2.0 ** -25 if dtype == torch.float16 else 0)
