"""GPU tests of the few-token operators at their edges: strides of single tokens, values that are not
finite, scales of any size, and grids past a launch's limit.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests.parity import announce, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


def same_bits(a, b):
    kind = torch.int16 if a.element_size() == 2 else torch.int32
    return a.shape == b.shape and torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def ints(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


# room: positions that the table has beyond ctx; with many, requests are split over workgroups
def call_of(B=3, N=1, H=2, G=4, D=128, page=16, ctx=300, room=0, seed=0):
    """q, cache, table of a random call; the table's pages past ctx + N are none."""
    rng = np.random.default_rng(seed)
    MP = -(-(ctx + N) // page)
    cache = tuple((dev(c), dev(s)) for c, s in ft.random_cache(rng, B * MP, H, page, D))
    table = np.concatenate([rng.permutation(B * MP).reshape(B, MP), np.full((B, room // page), -7)], 1).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, N, H * G, D)).astype(np.float32)).bfloat16().cuda()
    return q, cache, dev(table)


# ---- strides --------------------------------------------------------------------------------------

@pytest.mark.parametrize("room", [0, 5000])
def test_single_tokens_of_wider_rows(room):
    announce(f"single tokens of wider rows, {room}")
    q, cache, table = call_of(B=5, room=room)
    ctx = ints(0, 1, 40, 299, 300)
    o, lse = dg.fp8_tree_attention(q, cache, table, ctx)
    wide = torch.full((5, 3, 14, 128), float("nan"), device="cuda").bfloat16()
    wide[:, 2:, 3:11] = q
    for part in (wide[:, 2:, 3:11], wide[:, 2, 3:11].unsqueeze(1)):
        got = dg.fp8_tree_attention(part, cache, table, ctx)
        assert same_bits(got[0], o) and same_bits(got[1], lse)
    heads = torch.zeros(5, 1, 8, 256, device="cuda").bfloat16()
    for bad in (heads[..., :128], heads[..., ::2], heads[..., :128].transpose(2, 3).contiguous().transpose(2, 3),
                torch.zeros(5, 1, 16, 128, device="cuda").bfloat16()[:, :, ::2]):
        with pytest.raises(ValueError, match="dense"):
            dg.fp8_tree_attention(bad, cache, table, ctx)


# ---- values that are not finite -----------------------------------------------------------------------

SHAPES = [(1, 4, 64), (1, 3, 128), (1, 16, 256), (3, 4, 128), (24, 8, 64), (17, 4, 128)]     # N, G, D


@pytest.mark.parametrize("N,G,D", SHAPES)
@pytest.mark.parametrize("ctx,room", [(1, 0), (40, 0), (300, 5000), (5000, 0)])
def test_queries_with_nan_give_nan(N, G, D, ctx, room):
    """Rows of NaN queries are NaN where they see anything, 0 and -inf where not; the others keep
    their bits."""
    announce(f"NaN queries N={N} G={G} D={D} ctx={ctx} room={room}")
    q, cache, table = call_of(3, N, 2, G, D, ctx=ctx, room=room)
    ctxs, lens = ints(ctx, 0, ctx // 2 + 1), ints(N, N, max(N - 1, 1))
    mask = np.stack([ft.chain(N)] * 3)
    mask[1, 0] = False                                # sees nothing
    words = dev(ft.pack_mask(mask))
    o, lse = dg.fp8_tree_attention(q, cache, table, ctxs, lens, words)
    bad = torch.zeros(3, N, 2 * G, dtype=torch.bool, device="cuda")
    bad[0, 0, 0] = bad[1, 0] = bad[1, -1, 1] = bad[2, -1, -1] = bad[2, 0, G] = True
    x = q.clone()
    x[bad] = torch.where(torch.arange(D, device="cuda") == D - 5, float("nan"), x[bad])
    ob, lb = dg.fp8_tree_attention(x, cache, table, ctxs, lens, words)
    sees = lse > -float("inf")
    assert not sees[1, 0].any() and sees[0].all() and sees[2, 0].all()
    assert ob[bad & sees].isnan().all() and lb[bad & sees].isnan().all()
    keep = ~(bad & sees)
    assert same_bits(ob[keep], o[keep]) and same_bits(lb[keep], lse[keep])


@pytest.mark.parametrize("N,G,D", SHAPES)
@pytest.mark.parametrize("ctx,room,first,last", [(1, 0, 0, 1), (40, 0, 0, 40), (300, 5000, 0, 300), (300, 5000, 299, 300),
                                                 (5000, 0, 0, 5000), (5000, 0, 0, 4000), (5000, 0, 1000, 5000), (5000, 0, 0, 1)])
def test_cached_rows_of_nan_reach_every_row(N, G, D, ctx, room, first, last):
    """Keys or values of NaN in positions [first, last), alone or among others, whole or a split
    request's parts."""
    announce(f"NaN rows of the cache N={N} G={G} D={D} ctx={ctx} room={room} {first}:{last}")
    q, cache, table = call_of(2, N, 2, G, D, ctx=ctx, room=room)
    ctxs, lens = ints(ctx, ctx), ints(N, N)
    mask = dev(ft.pack_mask(np.zeros((2, N, N), bool)))     # the context alone
    o, lse = dg.fp8_tree_attention(q, cache, table, ctxs, lens, mask)
    at = torch.arange(first, last, device="cuda")
    slots = (table[0, at // 16] * 16 + at % 16).int()
    k, v = dg.fp8_kv_cache_read(cache, slots, dtype=torch.float32)
    spoilt = torch.full_like(k, 2.0)
    spoilt[:, 1, 7] = float("nan")                    # key head 1 of request 0
    for keys, values in ((spoilt, v), (k, spoilt)):
        dg.fp8_kv_cache_write(keys, values, cache, slots)
        ob, lb = dg.fp8_tree_attention(q, cache, table, ctxs, lens, mask)
        assert ob[0, :, G:].isnan().all() and not ob[0, :, :G].isnan().any()
        assert lb[0, :, G:].isnan().all() if keys is spoilt else not lb.isnan().any()
        assert same_bits(ob[1], o[1]) and same_bits(lb[1], lse[1])


def test_parts_of_nan_are_joined():
    """However many of a split request's first keys are NaN, whole parts of it among them."""
    announce("NaN parts")
    q, cache, table = call_of(1, 1, 1, 4, 128, ctx=5000)
    scales = cache[0][1].clone()
    for last in range(32, 1400, 32):
        at = torch.arange(last, device="cuda")
        cache[0][1].copy_(scales)
        cache[0][1][table[0, at // 16].long(), 0, at % 16] = float("nan")
        o, lse = dg.fp8_tree_attention(q, cache, table, ints(5000))
        assert o.isnan().all() and lse.isnan().all(), last


@pytest.mark.parametrize("N,G,D", SHAPES)
@pytest.mark.parametrize("ctx,room", [(1, 0), (40, 0), (300, 5000), (5000, 0)])
def test_queries_with_infinities_give_nan(N, G, D, ctx, room):
    """Scores of infinity less infinity: NaN where the row sees anything, also where all its scores
    are -infinity, 0 and -inf where it sees nothing."""
    announce(f"infinite queries N={N} G={G} D={D} ctx={ctx} room={room}")
    q, cache, table = call_of(2, N, 2, G, D, ctx=ctx, room=room)
    (kc, ks), _ = cache
    kc[..., D - 9] = 0x38                             # 1 in every key, so that scores have one sign
    ctxs, lens = ints(ctx, 0), ints(N, N)
    mask = np.stack([ft.chain(N)] * 2)
    mask[1, 0] = False
    words = dev(ft.pack_mask(mask))
    o, lse = dg.fp8_tree_attention(q, cache, table, ctxs, lens, words)
    bad = torch.zeros(2, N, 2 * G, dtype=torch.bool, device="cuda")
    bad[0, 0, 0] = bad[0, -1, G] = bad[1, 0] = bad[1, -1, -1] = True
    for value in (-float("inf"), float("inf")):
        x = q.clone()
        x[bad] = torch.where(torch.arange(D, device="cuda") == D - 9, value, x[bad])
        ob, lb = dg.fp8_tree_attention(x, cache, table, ctxs, lens, words)
        sees = lse > -float("inf")
        assert sees[0].all() and not sees[1, 0].any()
        assert ob[bad & sees].isnan().all() and lb[bad & sees].isnan().all()
        keep = ~(bad & sees)
        assert same_bits(ob[keep], o[keep]) and same_bits(lb[keep], lse[keep])


# ---- scales of any size ------------------------------------------------------------------------------

@pytest.mark.parametrize("low,high", [(-126, -118), (-118, -104), (-104, -88), (-88, -60), (60, 119)])
def test_cache_quotients_at_any_scale(low, high):
    """Quotients on and next to the midpoints of codes, for the smallest and largest scales of normal
    numbers."""
    announce(f"quotients at scales of 2^{low} to 2^{high}")
    rng = np.random.default_rng(high + 200)
    grid = ft.e4m3(np.arange(127, dtype=np.uint8))
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.zeros((1024, 1, 256), np.float32)
    for r in range(1024):
        amax = np.float32(448 * np.exp2(rng.uniform(low, high)))
        v = (mid * (amax / np.float32(448))).astype(np.float32)
        near = np.concatenate([v, np.nextafter(v, np.float32(0 if r % 2 else np.inf))])
        x[r, 0, :252], x[r, 0, 255] = near[:252] * rng.choice([-1, 1], 252), amax
    cache = dg.make_fp8_kv_cache(64, 1, 16, 256)
    dg.fp8_kv_cache_write(dev(x), dev(x), cache, torch.arange(1024, dtype=torch.int32, device="cuda"))
    want, scale = ft.quantise_rows(x)
    for codes, sf in cache:
        np.testing.assert_array_equal(codes.cpu().numpy().reshape(1024, 1, 256), want)
        np.testing.assert_array_equal(sf.cpu().numpy().reshape(1024, 1), scale)


def against_reference(q, cache, table, ctxs, lens, mask):
    """The call's outputs, checked against the 64-bit result within its bound."""
    B, N, _, D = q.shape
    o, lse = dg.fp8_tree_attention(q, cache, table, ctxs, lens, dev(ft.pack_mask(mask)))
    host = [(c.cpu().numpy(), s.cpu().numpy()) for c, s in cache]
    ro, rl, bo, bl = ft.attention(q.float().cpu().numpy(), host, table.cpu().numpy(), ctxs.tolist(), lens.tolist(), mask,
                                  D ** -0.5, cache[0][0].shape[2])
    off = np.abs(o.double().cpu().numpy() - ro)
    assert (off <= bo).all(), float((off / bo).max())
    seen = np.isfinite(rl)
    assert np.array_equal(np.isneginf(lse.cpu().numpy()), ~seen)
    assert (np.abs(lse.double().cpu().numpy()[seen] - rl[seen]) <= bl[seen]).all()
    return o, lse


@pytest.mark.parametrize("N,G,D", SHAPES)
@pytest.mark.parametrize("room", [0, 5000])
def test_negative_value_scales(N, G, D, room):
    """A cache of the caller's own may have them: all of a request's, or some."""
    announce(f"negative value scales N={N} G={G} D={D} room={room}")
    q, cache, table = call_of(2, N, 2, G, D, ctx=130, room=room)
    mask = np.stack([ft.chain(N)] * 2)
    args = ints(130, 61), ints(N, N), mask
    _, lse = against_reference(q, cache, table, *args)
    sf = cache[1][1]
    sf.neg_()
    assert same_bits(against_reference(q, cache, table, *args)[1], lse)
    sf[:, :, ::3].neg_()
    against_reference(q, cache, table, *args)


@pytest.mark.parametrize("N,G,D,ctx,room", [(6, 4, 64, 10, 0), (6, 4, 128, 3, 5000), (8, 2, 256, 0, 0), (24, 8, 64, 40, 0),
                                            (40, 2, 128, 0, 5000), (130, 1, 128, 5, 0), (130, 1, 64, 700, 5000)])
@pytest.mark.parametrize("factor", [2.0 ** 30, 2.0 ** 60, float("inf")])
def test_large_values_of_unseen_tokens_do_not_touch_others(N, G, D, ctx, room, factor):
    """A drafted token's values far larger than all others leave the rows that do not see it as they
    were, bit for bit, and the others within their bound."""
    announce(f"large unseen values N={N} G={G} D={D} ctx={ctx} room={room} {factor}")
    q, cache, table = call_of(1, N, 2, G, D, ctx=ctx, room=room)
    ctxs, lens = ints(ctx), ints(N)
    mask = np.stack([ft.chain(N)])
    mask[0, 1:, 0] = np.arange(1, N) % 3 == 0          # who sees token 0
    mask[0, 3:, 2] = False                            # and token 2: itself alone
    o, lse = against_reference(q, cache, table, ctxs, lens, mask)
    for token in (0, 2):
        at = ctx + token
        cache[1][1][table[0, at // 16].long(), :, at % 16] *= factor
    sees = torch.from_numpy(mask[0, :, 0] | mask[0, :, 2]).cuda()
    if np.isfinite(factor):
        ob, lb = against_reference(q, cache, table, ctxs, lens, mask)
    else:
        ob, lb = dg.fp8_tree_attention(q, cache, table, ctxs, lens, dev(ft.pack_mask(mask)))
        assert not ob[0, sees].isfinite().any()
    assert same_bits(ob[0, ~sees], o[0, ~sees]) and same_bits(lb, lse)


@pytest.mark.parametrize("G,D,ctx,room", [(4, 64, 10, 0), (3, 128, 31, 5000), (16, 256, 32, 0), (8, 128, 300, 5000), (33, 64, 0, 0)])
def test_a_single_token_that_does_not_see_itself(G, D, ctx, room):
    announce(f"blind single tokens G={G} D={D} ctx={ctx} room={room}")
    q, cache, table = call_of(2, 1, 2, G, D, ctx=ctx, room=room)
    ctxs, lens, mask = ints(ctx, ctx), ints(1, 1), np.array([[[False]], [[True]]])
    o, lse = against_reference(q, cache, table, ctxs, lens, mask)
    for factor in (2.0 ** 60, float("inf"), float("nan")):
        sf = cache[1][1].clone()
        cache[1][1][table[0, ctx // 16].long(), :, ctx % 16] *= factor
        ob, lb = dg.fp8_tree_attention(q, cache, table, ctxs, lens, dev(ft.pack_mask(mask)))
        assert same_bits(ob, o) and same_bits(lb, lse)
        cache[1][1].copy_(sf)


@pytest.mark.parametrize("N,G,D", SHAPES)
@pytest.mark.parametrize("ctx,room", [(40, 0), (300, 5000), (5000, 0)])
@pytest.mark.parametrize("power", [-118, -60, 60, 118])
def test_values_of_any_size(N, G, D, ctx, room, power):
    """Values multiplied by a power of two multiply o by it, up to the largest numbers of bf16 and
    down to the smallest normal ones."""
    announce(f"values of 2^{power} N={N} G={G} D={D} ctx={ctx} room={room}")
    q, cache, table = call_of(2, N, 2, G, D, ctx=ctx, room=room)
    q = q * 2.0 ** -6                                 # weights that are nearly even
    ctxs, lens = ints(ctx, ctx // 3), ints(N, N)
    o, lse = dg.fp8_tree_attention(q, cache, table, ctxs, lens)
    sf = cache[1][1]
    assert 448 * sf.max() < 2.0 ** 9                  # so that no value passes 2^127
    sf.copy_(torch.from_numpy(np.ldexp(sf.cpu().numpy(), power)))
    ob, lb = dg.fp8_tree_attention(q, cache, table, ctxs, lens)
    want = np.ldexp(o.double().cpu().numpy(), power)
    got = ob.double().cpu().numpy()
    # Sums are put down 2^13 too small, over a sum of weights of 1/2 or more: below the normal
    # numbers of fp32 each of some (16 + 3 * 80 parts) roundings is 2^-150 * 2^14 of o, and then
    # bf16 may round to the other side.  Otherwise nothing is lost.
    off = 0.0 if power > -64 else 2.0 ** -128 + 2.0 ** -7 * np.abs(want)
    assert same_bits(lb, lse) and (np.abs(got - want) <= off).all()


# ---- past a grid's limit ---------------------------------------------------------------------------------

def test_cache_copies_of_more_than_2_to_the_32_threads():
    """2^27 rows of 256 values and a few: 64 GiB of keys, of which a few tokens are stored."""
    announce("cache copies past 2^32 threads")
    D, T = 256, (1 << 27) + 5
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("too little memory")
    at = torch.tensor([0, 1, 77, (1 << 26) - 1, 1 << 26, (1 << 26) + 1, (1 << 27) - 1, 1 << 27, T - 2, T - 1], device="cuda")
    n = len(at)
    few = torch.randn(n, 1, D, device="cuda").bfloat16()
    k = torch.empty(T, 1, D, dtype=torch.bfloat16, device="cuda")
    k[at] = few
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    slots[at] = torch.arange(n, dtype=torch.int32, device="cuda") * 3
    cache, want = dg.make_fp8_kv_cache(2, 1, 16, D), dg.make_fp8_kv_cache(2, 1, 16, D)
    dg.fp8_kv_cache_write(k, k, cache, slots)
    dg.fp8_kv_cache_write(few, few, want, slots[at])
    for (codes, sf), (wc, ws) in zip(cache, want):
        assert torch.equal(codes, wc) and torch.equal(sf, ws)
    v = torch.empty_like(k)
    near = torch.cat([at, torch.tensor([2, (1 << 26) + 2, T - 3], device="cuda")])
    k[near], v[near] = 5.0, 5.0
    dg.fp8_kv_cache_read(cache, slots, out=(k, v))
    for rows in (k, v):
        assert same_bits(rows[at], dg.fp8_kv_cache_read(want, slots[at])[0]) and not rows[near[n:]].any()
    del k, v, rows, slots
    torch.cuda.empty_cache()


def test_joining_more_than_2_to_the_32_threads():
    """32768 requests of 8192 query heads, D = 64: 2^34 values of o, two runs, so that the second
    kernel looks at every row."""
    announce("joined rows past 2^32 threads")
    B, Hq, D, turn = 32768 + 16, 8192, 64, 16
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("too little memory")
    small_q, cache, table = call_of(turn, 1, 1, Hq, D, ctx=16)
    ctx = torch.arange(turn, dtype=torch.int32, device="cuda")
    want, want_lse = dg.fp8_tree_attention(small_q, cache, table, ctx)
    assert dg.get_fp8_tree_attention_workspace_bytes(B, 1, Hq, 1, D, 16, table.shape[1]) > 0
    q = small_q.repeat(B // turn, 1, 1, 1)
    o, lse = dg.fp8_tree_attention(q, cache, table.repeat(B // turn, 1), ctx.repeat(B // turn))
    del q
    o, lse = o.view(B // turn, turn, 1, Hq, D), lse.view(B // turn, turn, 1, Hq)
    for i in range(B // turn):
        assert torch.equal(o[i], want) and torch.equal(lse[i], want_lse), i
    del o, lse
    torch.cuda.empty_cache()
