"""Plain 64-bit references of the few-token operators, with error bounds, and their inputs.

Each reference returns, beside the exact values, a bound on what a kernel may be off by,
derived from the arithmetic it is allowed: fp32 sums (unit roundoff 2^-24, taken twice for
sums that truncate), the exponentials' few units, and the one rounding to bf16 (2^-8) or of a
softmax weight to 11 bits (2^-11) where there is one.
"""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = np.float32(448.0)
EPS = 2.0 ** -23            # of an fp32 sum's step, truncation included


def e4m3(codes) -> np.ndarray:
    """Values of e4m3 codes in float64."""
    c = np.asarray(codes, np.uint8)
    e, m = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


# ---- the cache -----------------------------------------------------------------------------

def quantise_rows(x: np.ndarray):
    """[..., D] fp32 rows -> (codes, fp32 scales) by the cache's rule."""
    x = np.ascontiguousarray(x, np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        bad = ~np.isfinite(x).all(-1)
        s = np.where(bad, np.float32(1), amax / E4M3_MAX).astype(np.float32)
        s = np.where(s == 0, np.float32(1), s).astype(np.float32)
        q = np.clip(x / s[..., None], -E4M3_MAX, E4M3_MAX).astype(np.float32)
    q = np.where(bad[..., None], np.float32(0), q)
    codes = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes, np.where(bad, np.float32(np.nan), s).astype(np.float32)


def random_cache(rng, pages, H, page, D):
    """Codes and scales of random rows, scales of several sizes."""
    out = []
    for _ in range(2):
        x = rng.standard_normal((pages, H, page, D)).astype(np.float32)
        x *= np.exp2(rng.integers(-6, 7, (pages, H, page, 1))).astype(np.float32)
        out.append(quantise_rows(x))
    return out


# ---- attention -----------------------------------------------------------------------------

def attention(q, cache, table, ctx, lens, mask, scale, page):
    """q [B, N, Hq, D] float; cache [(codes, sf), (codes, sf)]; mask [B, N, N] bool.
    Returns o, lse and the bounds of both."""
    (kc, ks), (vc, vs) = cache
    P, H, _, D = kc.shape
    B, N, Hq, _ = q.shape
    G, most = Hq // H, table.shape[1] * page
    o, bo = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, bl = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        c, n = min(max(int(ctx[b]), 0), most), min(max(int(lens[b]), 0), N)
        L = min(c + n, most)
        pos = np.arange(L)
        pg = table[b, pos // page].astype(np.int64) if L else np.zeros(0, np.int64)
        there = (pg >= 0) & (pg < P)
        at = np.where(there, pg, 0)
        for i in range(n):
            seen = there.copy()
            for j in range(L - c):
                seen[c + j] &= bool(mask[b, i, j])
            w = np.nonzero(seen)[0]
            if len(w) == 0:
                continue
            for h in range(H):
                key = e4m3(kc[at[w], h, w % page]) * ks[at[w], h, w % page].astype(np.float64)[:, None]
                val = e4m3(vc[at[w], h, w % page]) * vs[at[w], h, w % page].astype(np.float64)[:, None]
                for g in range(G):
                    x = q[b, i, h * G + g].astype(np.float64)
                    s = key @ x * scale
                    # a score's error: its sum's, and a few roundings of the scaled value
                    es = np.max((D + 8) * EPS * (np.abs(key) @ np.abs(x)) * abs(scale))
                    m = s.max()
                    p = np.exp(s - m)
                    z = p.sum()
                    o[b, i, h * G + g] = p @ val / z
                    lse[b, i, h * G + g] = m + np.log(z)
                    # the sums run over len(w) terms, of the weights and of the values
                    rel = 2 * es + (len(w) + 64) * EPS + 2.0 ** -20
                    # a weight times its value's scale is kept to 11 bits, and to 2^-35 of the
                    # largest weight (1) times the largest scale, whichever is more
                    code = np.abs(e4m3(vc[at[w], h, w % page])).sum(0)
                    least = 2.0 ** -35 * float(vs[at[w], h, w % page].max()) * code / z
                    bo[b, i, h * G + g] = (np.abs(p) @ np.abs(val) / z * (2.0 ** -11 + 2 * rel) + least
                                           + 2.0 ** -8 * np.abs(o[b, i, h * G + g]) + 1e-37)
                    bl[b, i, h * G + g] = rel + 2.0 ** -20 + 4 * EPS * abs(m)
    return o, lse, bo, bl


def chain(N):
    """The mask of drafted tokens one after the other."""
    return np.tril(np.ones((N, N), bool))


def random_tree(rng, N):
    """Mask of a random tree: a token sees itself and its ancestors."""
    m = np.zeros((N, N), bool)
    for i in range(N):
        parent = int(rng.integers(-1, i)) if i else -1
        if parent >= 0:
            m[i] = m[parent]
        m[i, i] = True
    return m


def pack_mask(mask):
    """[B, N, N] bool -> the call's int64 words [B, N, ceil(N / 64)]."""
    B, N, _ = mask.shape
    W = (N + 63) // 64
    bits = np.zeros((B, N, 64 * W), np.uint64)
    bits[:, :, :N] = mask
    words = (bits.reshape(B, N, W, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
    return words.view(np.int64)


# ---- mixture of experts ----------------------------------------------------------------------

def quantise_blocks(w: np.ndarray):
    """[E, N, K] fp32 -> (codes, fp32 scales per 128 x 128 block)."""
    E, N, K = w.shape
    b = w.reshape(E, N // 128, 128, K // 128, 128)
    s = (np.abs(b).max((2, 4)) / E4M3_MAX).astype(np.float32)
    q = np.clip(b / s[:, :, None, :, None], -E4M3_MAX, E4M3_MAX).astype(np.float32)
    codes = torch.from_numpy(np.ascontiguousarray(q)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    return codes.reshape(E, N, K), s


def moe(x, w1, s1, w2, s2, ids, weights, parts):
    """y of the layer and its bound before the rounding of y; parts: bf16 parts
    that the hidden values are kept as."""
    T, H = x.shape
    E, _, I = w2.shape
    y, by = np.zeros((T, H)), np.zeros((T, H))
    x = x.astype(np.float64)
    for e in range(E):
        hit = np.nonzero((ids == e).any(1))[0]
        if len(hit) == 0:
            continue
        a1 = e4m3(w1[e]) * np.repeat(np.repeat(s1[e].astype(np.float64), 128, 0), 128, 1)
        a2 = e4m3(w2[e]) * np.repeat(np.repeat(s2[e].astype(np.float64), 128, 0), 128, 1)
        z = x[hit] @ a1.T
        bz = (H + 16) * EPS * (np.abs(x[hit]) @ np.abs(a1).T)
        g, u, bg, bu = z[:, :I], z[:, I:], bz[:, :I], bz[:, I:]
        silu = g / (1 + np.exp(-g))
        h = silu * u
        bh = 1.1 * np.abs(u) * bg + np.abs(silu) * bu + 1.1 * bg * bu + 16 * EPS * np.abs(h)
        bh += (2.0 ** -14 if parts == 2 else EPS) * np.abs(h)
        c = np.where(ids[hit] == e, weights[hit].astype(np.float64), 0).sum(1)[:, None]
        size = (np.abs(h) @ np.abs(a2).T) * np.abs(np.where(ids[hit] == e, weights[hit], 0)).sum(1)[:, None]
        y[hit] += c * (h @ a2.T)
        by[hit] += np.abs(c) * (bh @ np.abs(a2).T) + (I + 32 + 16) * EPS * size
    return y, by + 64 * EPS * np.abs(y)
