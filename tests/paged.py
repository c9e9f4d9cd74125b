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
