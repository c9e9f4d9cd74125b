"""Plain references of the operators around a paged cache (plan of pages and slots, norms with
rotation, the FP4 cache), in Python's integers and 64-bit floats, with error bounds where a kernel
rounds."""
from __future__ import annotations

import numpy as np


# ---- pages and slots -------------------------------------------------------------------------

def plan(table, ctx, add, ring, state, page, rows, padded):
    """What the plan leaves: table, slots, positions, lengths, ring, state (numpy, int64)."""
    table, ring = np.array(table, np.int64), np.array(ring, np.int64)
    B, width = table.shape
    P = len(ring)
    head, free = int(state[0]) % 2 ** 32 % P, min(max(int(state[1]), 0), P)
    wanted = taken = 0
    back, lens, tokens = [], [], []
    for b in range(B):
        c, a = min(max(int(ctx[b]), 0), width * page), int(add[b])
        after = max(c + a, 0)
        fits = after <= width * page and not (padded and a > rows)
        held, need = -(-c // page), -(-after // page)
        lack = max(need - held, 0) if fits else 0
        wanted += lack
        served = fits and (lack == 0 or wanted <= free)
        if served:
            for j in range(held, need):
                table[b, j] = ring[(head + taken) % P]
                taken += 1
            back += table[b, need:held].tolist()
        lens.append(after if served else c)
        new = []
        for q in range(c, c + min(max(a, 0), rows)):
            pg = int(table[b, q // page]) if served else -1
            new.append((pg * page + q % page if 0 <= pg < P else -1, q))
        tokens += new + [(-1, 0)] * (rows - len(new)) if padded else new
    if not padded:
        tokens = tokens[:rows] + [(-1, 0)] * (rows - len(tokens))
    back = back[:P - free]
    for i, pg in enumerate(back):
        ring[(head + free + i) % P] = pg
    tokens = np.array(tokens, np.int64).reshape(-1, 2)
    shape = (B, rows) if padded else (rows,)
    state = np.array([(head + taken) % P, free - taken + len(back)])
    return table, tokens[:, 0].reshape(shape), tokens[:, 1].reshape(shape), np.array(lens, np.int64), ring, state


def random_pool(rng, B, page, ctx, spare):
    """A table whose requests hold pages for ctx tokens, the ring of the other pages and its state;
    spare: free pages."""
    held = [-(-int(c) // page) for c in ctx]
    P = sum(held) + spare
    order = rng.permutation(P)
    width = max(held, default=0) + spare + 1
    table, at = np.full((B, width), -77, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    head = int(rng.integers(P))
    ring = np.full(P, -55, np.int32)
    ring[(head + np.arange(spare)) % P] = order[at:]
    return table, ring, np.array([head, spare], np.int32)


# ---- norms with rotation -----------------------------------------------------------------------

U = 2.0 ** -24             # half a step of fp32
HALF_STEP = {"bf16": 2.0 ** -8, "f32": U}
# Neighbours are never less than 2^-133 (bf16) or 2^-149 (fp32) apart, below 2^-126: half of that
# for the one rounding to bf16, and in fp32 for each of some ten.
LEAST = {"bf16": 2.0 ** -134 + 1e-44, "f32": 1e-44}


def _turn(x, cos, sin, R, interleaved, back=False):
    """The first R values of rows turned, and the same of absolute values (for bounds)."""
    z, size = x.copy(), np.abs(x)
    a, b = (np.s_[..., 0:R:2], np.s_[..., 1:R:2]) if interleaved else (np.s_[..., :R // 2], np.s_[..., R // 2:R])
    s = -sin if back else sin
    z[a], z[b] = x[a] * cos - x[b] * s, x[b] * cos + x[a] * s
    size[a] = size[b] = np.abs(x[a]) + np.abs(x[b])
    return z, size


def _angles(positions, inv_freq):
    t = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float32).astype(np.float64)
    # cosines and sines: two of fp32's last places (2 U each) and the angle's own, 2^-25 of an eighth of a
    # turn from its rounding to fp32 and 2^-51 of it from the products in 64 bits
    return np.cos(t)[:, None], np.sin(t)[:, None], 5 * U + 2.0 ** -51 * np.abs(t).max(initial=0.0)


def norm_rope(x, w, positions, inv_freq, eps, interleaved, out):
    """z of rows x [T, H, D] (64-bit) and its bound; out: "bf16" or "f32"."""
    D, R = x.shape[-1], 2 * len(inv_freq)
    cos, sin, off = _angles(positions, inv_freq)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    z, size = _turn(y, cos, sin, R, interleaved)
    # r: half the error of a sum of 8 products and 5 exchanges and its mean (16 U), and a Newton step's 2 U;
    # y: two products more; z: two products and a sum
    bound = size * ((8 + 2 + 2 + 3) * U + off) * 1.01 + HALF_STEP[out] * np.abs(z) + LEAST[out]
    return z, bound


def norm_rope_backward(dz, x, w, positions, inv_freq, eps, interleaved, out):
    """dx and dw of rows (64-bit) and their bounds."""
    D, R = x.shape[-1], 2 * len(inv_freq)
    cos, sin, off = _angles(positions, inv_freq)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dy, size = _turn(dz, cos, sin, R, interleaved, back=True)
    e_dy, e_n = size * (3 * U + off), 11 * U * np.abs(n)
    g = dy * w
    e_g = np.abs(w) * e_dy + U * np.abs(g)
    m = (g * n).mean(-1, keepdims=True)
    # 8 products in a chain and 5 exchanges, and the mean
    e_m = (e_g * np.abs(n) + np.abs(g) * e_n + 15 * U * np.abs(g * n)).mean(-1, keepdims=True)
    dx = r * (g - n * m)
    e_dx = r * (e_g + e_n * np.abs(m) + np.abs(n) * e_m + 2 * U * (np.abs(g) + np.abs(n * m))) + 11 * U * np.abs(dx)
    rows = x.shape[0] * x.shape[1]
    each = np.abs(dy * n)
    # a lane's rows one after the other (1 / 16 of a workgroup's, of 1024 workgroups), 32 lanes, 32
    # workgroups and 32 of those sums: what a term goes through
    e_dw = (e_dy * np.abs(n) + np.abs(dy) * e_n).sum((0, 1)) + (128 + rows / 4096) * U * each.sum((0, 1))
    return (dx, 1.01 * e_dx + HALF_STEP[out] * np.abs(dx) + LEAST[out]), ((dy * n).sum((0, 1)), 1.01 * e_dw + 1e-44)


# ---- the FP4 cache -------------------------------------------------------------------------------

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def quantise4(x):
    """[..., D] rows -> (codes [..., D / 2], exponent bytes [..., D / 32]) by the cache's rule, block by
    block in 64 bits."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(b).all(-1)
        b = np.where(bad[..., None], 0.0, b)
        most = np.abs(b).max(-1)
        e = np.full(most.shape, -125)
        while True:                                    # the least exponent that will do
            small = (most > 6 * np.ldexp(1.0, e)) & (e < 125)
            if not small.any():
                break
            e += small
        e = np.where(most == 0, 0, e)
        y = np.ldexp(b, -e[..., None])
    middles = (E2M1[1:8] + E2M1[:7]) / 2
    code = np.zeros(y.shape, np.uint8)
    for i, middle in enumerate(middles):               # ties to the even code
        code += (np.abs(y) > middle) if i % 2 == 0 else (np.abs(y) >= middle)
    code |= np.signbit(y).astype(np.uint8) << 3
    code[bad] = 0
    code = code.reshape(x.shape)
    return code[..., ::2] | code[..., 1::2] << 4, np.where(bad, 255, e + 127).astype(np.uint8)


def values4(codes, sf):
    """[..., D / 2] codes, [..., D / 32] exponents -> [..., D] in 64 bits."""
    codes = np.asarray(codes)
    v = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(np.shape(sf) + (32,))
    scale = np.where(np.asarray(sf) == 255, np.nan, np.ldexp(1.0, np.asarray(sf).astype(np.int64) - 127))
    return (v * scale[..., None]).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))


def random_cache4(rng, pages, H, page, D, values=None):
    """Random codes, scales of several sizes (a fifth of the cache's blocks far smaller).  values: a
    function of rng and a shape that gives the bytes of the values' scales instead."""
    out = []
    for kind in range(2):
        codes = rng.integers(0, 256, (pages, H, page, D // 2)).astype(np.uint8)
        sf = (127 - 2 + rng.integers(-4, 3, (pages, H, page, D // 32))).astype(np.uint8)
        sf[rng.random(sf.shape) < 0.2] -= 20
        if kind and values:
            sf = values(rng, sf.shape).astype(np.uint8)
        out.append((codes, sf))
    return out


def form4(sf):
    """What the attention makes of values with these bytes of scales: "fp16" where all are from 2^-18 to
    2^13, "bf16" where none is, else "both"."""
    inside = (np.asarray(sf) >= 127 - 18) & (np.asarray(sf) <= 127 + 13)
    return "fp16" if inside.all() else "both" if inside.any() else "bf16"


def attention4(q, cache, table, ctx, lens, mask, scale, page, form=None):
    """q [B, N, Hq, D] float; mask [B, N, N] bool.  Returns o, lse and the bounds of both; NaN where a
    scale that is NaN reaches.  form: "fp16" or "bf16" where all values are read in it, for bounds of
    each column by itself."""
    (kc, ks), (vc, vs) = cache
    P, H = kc.shape[:2]
    B, N, Hq, D = q.shape
    G, most, eps = Hq // H, table.shape[1] * page, 2.0 ** -23
    o, bo = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, bl = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        c, n = min(max(int(ctx[b]), 0), most), min(max(int(lens[b]), 0), N)
        L = min(c + n, most)
        pos = np.arange(L)
        pg = table[b, pos // page].astype(np.int64) if L else np.zeros(0, np.int64)
        there = (pg >= 0) & (pg < P)
        at = np.where(there, pg, 0)
        for h in range(H):
            keys, values = (values4(codes[at, h, pos % page], sf[at, h, pos % page]) for codes, sf in cache)
            for i in range(n):
                seen = there.copy()
                for j in range(L - c):
                    seen[c + j] &= bool(mask[b, i, j])
                w = np.nonzero(seen)[0]
                if len(w) == 0:
                    continue
                key, val = keys[w], values[w]
                for g in range(G):
                    x = q[b, i, h * G + g].astype(np.float64)
                    with np.errstate(all="ignore"):
                        s = key @ x * scale
                        # a score's error: its sum's, and a few roundings of the scaled value
                        es = np.max((D + 8) * eps * (np.abs(key) @ np.abs(x)) * abs(scale))
                        m = s.max()
                        p = np.exp(s - m)
                        z = p.sum()
                        o[b, i, h * G + g] = p @ val / z
                        lse[b, i, h * G + g] = m + np.log(z)
                        # the sums run over len(w) terms, of the weights and of the values
                        rel = 2 * es + (len(w) + 64) * eps + 2.0 ** -20
                        # A weight is kept to fp16's 11 bits, half a step of which is 2^-11, and to half of
                        # fp16's least number 2^-24 in units of 2^-11 of the largest: 2^-36.  (Values out of
                        # fp16's range: to 16 bits, and to 2^-92 of the values' unit.)
                        with_nan = np.where(np.isnan(val), 0.0, np.abs(val))
                        least = (2.0 ** -36 * with_nan.sum(0) + len(w) * 2.0 ** -92 * with_nan.max()) / z + 2.0 ** -92
                        bo[b, i, h * G + g] = (np.abs(p) @ np.abs(val) / z * (2.0 ** -11 + 2 * rel) + least
                                               + 2.0 ** -8 * np.abs(o[b, i, h * G + g]))
                        if form:
                            # A weight is kept to fp16's half step, 2^-11, and to 2^-36 of the largest; or to 16
                            # bits and (as a product) to 2^-92.  Its exponent, a power of two up to 45 beside
                            # |s - m|, is rounded to 24 bits.
                            fp16 = form == "fp16"
                            each = (2.0 ** -11 if fp16 else 2.0 ** -16) + 2 * rel + 2.0 ** -24 * (np.abs(s - m) + 46)
                            least = 2.0 ** -36 * with_nan.sum(0) if fp16 else 2.0 ** -92 * (with_nan.sum(0) + len(w))
                            bo[b, i, h * G + g] = ((p * each) @ np.abs(val) / z + least / z + 2.0 ** -92
                                                   + 2.0 ** -8 * np.abs(o[b, i, h * G + g]))
                        bl[b, i, h * G + g] = rel + 2.0 ** -20 + 4 * eps * abs(m)
    return o, lse, bo, bl
