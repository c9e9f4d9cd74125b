"""Cases of the attention over the FP4 cache by the form that it reads values in: fp16 where their scales
are in its range, else bf16 with weights in two parts."""
from __future__ import annotations

import numpy as np

from tests import few_tokens as ft
from tests import paged


def _bytes(*ranges):
    every = np.concatenate([np.arange(lo, hi + 1) for lo, hi in ranges])
    return lambda rng, shape: rng.choice(every, shape)


# bytes of the values' scales: of values of several sizes, of all fp16 holds, of what it does not
VALUES = {"fp16": _bytes((121, 127)), "fp16's range": _bytes((109, 140)), "bf16": _bytes((100, 108), (141, 149))}

# B, N, H, G, D, page, longest context, positions that the table has beyond it
SHAPES = {
    "decode D=64": (9, 1, 2, 4, 64, 16, 601, 0),
    "decode D=128": (9, 1, 2, 4, 128, 64, 601, 0),
    "decode D=256": (9, 1, 2, 4, 256, 16, 601, 0),
    "17 query heads": (2, 1, 3, 17, 128, 16, 70, 0),
    "trees D=64": (4, 24, 2, 8, 64, 16, 100, 0),
    "trees D=128": (4, 17, 2, 4, 128, 16, 100, 0),
    "trees D=256": (4, 16, 2, 2, 256, 16, 100, 0),
    "long trees": (2, 65, 2, 2, 64, 16, 90, 0),
    "split D=64": (3, 3, 2, 4, 64, 16, 3000, 9000),
    "split D=128": (1, 1, 2, 4, 128, 16, 5000, 0),
    "split D=256": (2, 3, 2, 2, 256, 16, 1500, 5000),
    "split short": (10, 5, 2, 4, 128, 16, 100, 5000),
    "two row tiles D=64": (2, 12, 2, 8, 64, 16, 2500, 9000),
    "two row tiles D=128": (2, 12, 2, 8, 128, 16, 2500, 9000),
    "two row tiles whole": (130, 5, 2, 8, 128, 16, 300, 1200),
    "dealt": (10, 7, 2, 4, 128, 16, 700, 9000),
    "sixteen waves": (33, 1, 8, 2, 64, 16, 700, 5000),
    "sixteen waves split": (32, 1, 8, 2, 64, 16, 2500, 24000),
    "many short": (300, 1, 2, 3, 128, 16, 120, 0),
}


def case(B, N, H, G, D, page, longest, room, values, seed, q_scale=1.0, scale=None, change=None):
    """A random case, with NaN scales wherever no one may look: q, cache, table, ctx, lens, mask, scale, page,
    and the bytes of the values' scales that are read."""
    rng = np.random.default_rng(seed)
    ctx, lens = rng.integers(0, longest + 1, B), rng.integers(min(N, 2), N + 1, B)
    ctx[0], lens[0] = longest, N
    if B > 2:
        ctx[B // 2], ctx[-1] = 0, min(32, longest)
    MP = -(-(longest + N) // page) + 1
    pages = B * MP + 2
    cache = paged.random_cache4(rng, pages, H, page, D, values)
    table = rng.permutation(pages)[:B * MP].reshape(B, MP).astype(np.int32)
    live = np.zeros((pages, page), bool)
    for b in range(B):
        p = np.arange(ctx[b] + lens[b])
        live[table[b, p // page], p % page] = True
    if change:
        change(rng, cache, table, ctx, lens)
    for codes, sf in cache:
        codes.transpose(0, 2, 1, 3)[~live] = 0x7F
        sf.transpose(0, 2, 1, 3)[~live] = 255
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)])
    q = q_scale * rng.standard_normal((B, N, H * G, D))
    table = np.concatenate([table, np.full((B, room // page), -7, np.int32)], 1)
    return dict(q=q.astype(np.float32), cache=cache, table=table, ctx=ctx.astype(np.int32), lens=lens.astype(np.int32), mask=mask,
                scale=D ** -0.5 if scale is None else scale, page=page, read=cache[1][1].transpose(0, 2, 1, 3)[live])


def at(c, b, position):
    """Page and place in it of a request's position."""
    return int(c["table"][b, position // c["page"]]), position % c["page"]
