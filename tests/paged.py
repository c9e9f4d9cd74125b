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
