"""GPU parity of the few-token operators (FP8 cache, tree attention, few-token mixture of experts)
against the 64-bit references of tests/few_tokens.py, at the sizes and masks where they can go
wrong.  Cache codes, scales and rows are compared bit for bit; sums within the references' bounds.
"""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests.parity import announce, dev

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu()


def same_bits(a, b):
    return a.shape == b.shape and torch.equal(bits(a), bits(b))


# ---- the cache -----------------------------------------------------------------------------------

def cache_of(pages, H, page, D, fill=0xA5):
    return tuple((torch.full((pages, H, page, D), fill, dtype=torch.uint8, device="cuda"),
                  torch.full((pages, H, page), 7.5, device="cuda")) for _ in range(2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (1, 8, 128, 64), (7, 3, 128, 16), (65, 2, 256, 32), (300, 5, 64, 128),
                                        (1000, 8, 128, 64), (33, 1, 256, 4096)])
def test_cache_write_and_read(T, H, D, page, dtype):
    announce(f"cache T={T} H={H} D={D} page={page} {dtype}")
    rng = np.random.default_rng(T + H + D)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    x = rng.standard_normal((2, T, H, D)).astype(np.float32) * np.exp2(rng.integers(-20, 20, (2, T, H, 1))).astype(np.float32)
    x[0, 0, 0] = 0                                     # a row of zeros
    x[1, -1, -1, ::2] = -0.0
    x[1, T // 2, 0] *= np.float32(2.0 ** -130)          # scales below the normal numbers
    skip = T // 3
    slots_given = slots.copy()
    if T > 2:
        slots_given[skip], slots_given[skip + 1] = -1, pages * page   # not stored
    t = [dev(v).to(TYPES[dtype]) for v in x]
    # tokens as slices of a wider row: keys and values side by side
    wide = torch.zeros(T, 2 * H + 1, D, dtype=TYPES[dtype], device="cuda")
    wide[:, :H], wide[:, H:2 * H] = t[0], t[1]
    cache = cache_of(pages, H, page, D)
    got = dg.fp8_kv_cache_write(wide[:, :H], wide[:, H:2 * H], cache, dev(slots_given))
    assert got is cache
    k, v = dg.fp8_kv_cache_read(cache, dev(slots_given), dtype=TYPES[dtype])
    torch.cuda.synchronize()
    for (codes, sf), src, rows in zip(cache, t, (k, v)):
        want, scale = ft.quantise_rows(src.float().cpu().numpy())
        pool, scales = np.full(codes.shape, 0xA5, np.uint8), np.full(sf.shape, 7.5, np.float32)
        live = (slots_given >= 0) & (slots_given < pages * page)
        at = slots_given[live]
        pool[at // page, :, at % page], scales[at // page, :, at % page] = want[live], scale[live]
        np.testing.assert_array_equal(codes.cpu().numpy(), pool)
        np.testing.assert_array_equal(sf.cpu().numpy().view(np.int32), scales.view(np.int32))
        values = (ft.e4m3(want).astype(np.float32) * scale[..., None]).astype(np.float32)
        values[~live] = 0
        assert same_bits(rows, torch.from_numpy(values).to(TYPES[dtype]).cuda())


def test_cache_rows_that_are_not_finite():
    announce("cache: NaN and infinite rows")
    x = torch.randn(6, 2, 128, device="cuda")
    x[1, 0, 17], x[2, 1, 127], x[3, 0, 0] = float("nan"), float("inf"), -float("inf")
    cache = cache_of(1, 2, 16, 128)
    dg.fp8_kv_cache_write(x, x.flip(0).contiguous(), cache, torch.arange(6, dtype=torch.int32, device="cuda"))
    k, v = dg.fp8_kv_cache_read(cache, torch.arange(6, dtype=torch.int32, device="cuda"), dtype=torch.float32)
    bad = torch.zeros(6, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = bad[3, 0] = True
    for rows, want in ((k, bad), (v, bad.flip(0))):
        assert torch.equal(rows.isnan().all(-1), want) and torch.equal(rows.isnan().any(-1), want)
    assert not cache[0][0].eq(0x7F).any() and torch.equal(cache[0][1][0, :, :6].isnan(), bad.t())


def test_cache_every_quotient_is_correctly_rounded():
    """Quotients on and next to the midpoints of codes, over many scales."""
    announce("cache: quotients at midpoints")
    rng = np.random.default_rng(5)
    grid = ft.e4m3(np.arange(127, dtype=np.uint8))
    mid = (grid[1:] + grid[:-1]) / 2
    x = np.zeros((512, 1, 256), np.float32)
    for r in range(512):
        amax = np.float32(448 * np.exp2(rng.uniform(-8, 8)))
        s = np.float32(amax / np.float32(448))
        v = (mid * s).astype(np.float32)
        near = np.concatenate([v, np.nextafter(v, np.float32(0))])
        x[r, 0, :252], x[r, 0, 255] = near[:252] * rng.choice([-1, 1], 252), amax
    cache = cache_of(32, 1, 16, 256)
    dg.fp8_kv_cache_write(dev(x), dev(x), cache, torch.arange(512, dtype=torch.int32, device="cuda"))
    want, scale = ft.quantise_rows(x)
    np.testing.assert_array_equal(cache[0][0].cpu().numpy().reshape(512, 1, 256), want)
    np.testing.assert_array_equal(cache[1][1].cpu().numpy().reshape(512, 1), scale)


def test_cache_into_given_rows_and_single_tokens():
    announce("cache: out=, T = 0, T = 1")
    cache = cache_of(2, 2, 16, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    dg.fp8_kv_cache_write(e, e, cache, none)
    assert dg.fp8_kv_cache_read(cache, none)[0].shape == (0, 2, 64)
    x = torch.randn(1, 2, 64, device="cuda").bfloat16()
    slot = torch.tensor([31], dtype=torch.int32, device="cuda")
    dg.fp8_kv_cache_write(x, 2 * x, cache, slot)
    out = (torch.empty(1, 2, 64, device="cuda"), torch.empty(1, 2, 64, device="cuda"))
    got = dg.fp8_kv_cache_read(cache, slot, out=out)
    assert got[0] is out[0] and torch.equal(out[1], 2 * out[0])
    assert ((out[0] - x.float()).abs() <= x.float().abs() / 16 + x.float().abs().amax() / 448 / 512).all()


def test_cache_larger_than_32_bit_offsets():
    """The last pages of pools of 4.7 GB: offsets past 2^32."""
    announce("cache and attention past 2^32")
    H, page, D, pages = 8, 64, 128, 72000
    free, _ = torch.cuda.mem_get_info()
    if free < 16 << 30:
        pytest.skip("too little memory")
    cache = dg.make_fp8_kv_cache(pages, H, page, D)
    T = 130
    x = torch.randn(2, T, H, D, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(T, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).int()
    dg.fp8_kv_cache_write(x[0], x[1], cache, slots)
    small = dg.make_fp8_kv_cache(3, H, page, D)
    dg.fp8_kv_cache_write(x[0], x[1], small, pos.int())
    for a, b in zip(dg.fp8_kv_cache_read(cache, slots), dg.fp8_kv_cache_read(small, pos.int())):
        assert same_bits(a, b)
    q = torch.randn(1, 1, 32, D, device="cuda").bfloat16()
    ctx = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    for a, b in zip(dg.fp8_tree_attention(q, cache, table, ctx), dg.fp8_tree_attention(q, small, near, ctx)):
        assert same_bits(a, b)


# ---- attention -----------------------------------------------------------------------------------------

def attention_case(B, N, H, G, D, page, ctx, lens, mask, seed, scale=None, hide=(), q_scale=1.0, room=0):
    """A random case run on the GPU, with 0x7F codes and NaN scales wherever no one may look.
    room: positions that the table has beyond the longest request (with many, requests are split)."""
    rng = np.random.default_rng(seed)
    ctx, lens = np.asarray(ctx, np.int32), np.asarray(lens, np.int32)
    MP = max(1, -(-int((np.clip(ctx, 0, None) + np.clip(lens, 0, N)).max()) // page)) + 1
    pages = B * MP + 2
    cache = ft.random_cache(rng, pages, H, page, D)
    table = rng.permutation(pages)[:B * MP].reshape(B, MP).astype(np.int32)
    live = np.zeros((pages, page), bool)
    for b in range(B):
        p = np.arange(min(max(ctx[b], 0) + min(max(lens[b], 0), N), MP * page))
        live[table[b, p // page], p % page] = True
    for codes, sf in cache:
        codes.transpose(0, 2, 1, 3)[~live] = 0x7F
        sf.transpose(0, 2, 1)[~live] = np.nan
    for b, p, value in hide:
        table[b, p] = value
    table = np.concatenate([table, np.full((B, room // page), -7, np.int32)], 1)
    q = torch.from_numpy((q_scale * rng.standard_normal((B, N, H * G, D))).astype(np.float32)).bfloat16()
    scale = D ** -0.5 if scale is None else scale
    words = None if mask is None else dev(ft.pack_mask(mask))
    on_gpu = tuple((dev(c), dev(s)) for c, s in cache)
    o, lse = dg.fp8_tree_attention(q.cuda(), on_gpu, dev(table), dev(ctx), dev(lens), words, scale)
    torch.cuda.synchronize()
    full = np.stack([ft.chain(N)] * B) if mask is None else mask
    return (o.float().cpu().numpy(), lse.cpu().numpy()), ft.attention(q.float().numpy(), cache, table, ctx, lens, full, scale, page)


def check_attention(got, want):
    (o, lse), (ro, rl, bo, bl) = got, want
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty) and not o[empty].any()
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= bo).all(), float((np.abs(o - ro) / np.maximum(bo, 1e-30)).max())
    off = np.abs(lse[~empty] - rl[~empty])
    assert (off <= bl[~empty]).all(), float((off / bl[~empty]).max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_lengths(D, page):
    announce(f"decode D={D} page={page}")
    ctx = [0, 1, 14, 15, 16, 17, 31, 32, 33, 63, 64, 127, 200, 601]
    B = len(ctx)
    got, want = attention_case(B, 1, 2, 4, D, page, ctx, [1] * (B - 1) + [0], None, D + page)
    check_attention(got, want)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 17, 33])
def test_query_heads_of_a_key_head(G):
    announce(f"attention G={G}")
    got, want = attention_case(2, 1, 3, G, 128, 16, [70, 33], [1, 1], None, G)
    check_attention(got, want)


@pytest.mark.parametrize("N,G,D", [(2, 1, 64), (3, 4, 128), (5, 8, 64), (16, 2, 256), (17, 4, 128), (24, 8, 64), (33, 4, 64),
                                   (64, 1, 128), (65, 2, 64), (130, 1, 128), (20, 16, 128), (40, 2, 256)])
def test_trees(N, G, D):
    announce(f"tree N={N} G={G} D={D}")
    rng = np.random.default_rng(N)
    ctx, lens = [100, 0, 37, 5], [N, N - 1, max(N // 2, 1), 0]
    mask = np.stack([ft.random_tree(rng, N) for _ in ctx])
    got, want = attention_case(4, N, 2, G, D, 16, ctx, lens, mask, N)
    check_attention(got, want)


def test_chain_is_the_mask_that_is_not_given():
    announce("chain")
    a = attention_case(2, 19, 2, 4, 128, 32, [50, 0], [19, 12], None, 3)
    b = attention_case(2, 19, 2, 4, 128, 32, [50, 0], [19, 12], np.stack([ft.chain(19)] * 2), 3)
    check_attention(*a)
    assert np.array_equal(a[0][0], b[0][0]) and np.array_equal(a[0][1], b[0][1])


def test_masks_that_leave_rows_empty():
    announce("empty rows")
    rng = np.random.default_rng(7)
    mask = rng.random((3, 40, 40)) < 0.05            # rows of nothing, rows that miss themselves
    mask[0, :7] = False
    got, want = attention_case(3, 40, 2, 4, 128, 16, [0, 0, 9], [40, 21, 40], mask, 8)
    assert np.isneginf(want[1]).any()
    check_attention(got, want)


def test_lengths_out_of_range_are_clamped():
    announce("clamped lengths")
    got, want = attention_case(4, 3, 1, 2, 64, 16, [-5, 20, 7, 40], [3, 99, -4, 3], None, 9)
    check_attention(got, want)


def test_hidden_pages():
    announce("hidden pages")
    got, want = attention_case(2, 2, 2, 4, 128, 16, [70, 64], [2, 2], None, 10, hide=((0, 1, -1), (0, 3, 1 << 30), (1, 0, 9999)))
    check_attention(got, want)


def test_scores_far_apart():
    """Scores over hundreds, so that most weights vanish, and a scale of 0 and below."""
    announce("scores far apart")
    for scale, qs in ((1.0, 30.0), (0.0, 1.0), (-0.5, 2.0)):
        got, want = attention_case(2, 3, 2, 4, 128, 16, [150, 40], [3, 2], None, 11, scale=scale, q_scale=qs)
        check_attention(got, want)


@pytest.mark.parametrize("N,G,D", [(1, 4, 64), (1, 3, 128), (1, 16, 256), (3, 4, 128), (16, 2, 256), (17, 4, 128), (24, 8, 64),
                                   (65, 2, 64), (130, 1, 128)])
def test_short_requests_in_a_long_table(N, G, D):
    """Split over workgroups by the table's size, with lengths around tiles and steps, trees, hidden
    pages and rows that see nothing."""
    announce(f"split short N={N} G={G} D={D}")
    rng = np.random.default_rng(N)
    ctx, lens = [100, 0, 37, 5, 31, 32, 33, 0, 601, 16], [N, N - 1, max(N // 2, 1), 0, N, N, 1, N, N, N]
    mask = np.stack([ft.random_tree(rng, N) for _ in ctx])
    mask[2, 0] = mask[7, N // 2] = False
    got, want = attention_case(10, N, 2, G, D, 16, ctx, lens, mask, N, hide=((0, 1, -1), (8, 3, 1 << 30), (4, 0, -9)), room=5000)
    assert np.isneginf(want[1]).any()
    check_attention(got, want)


@pytest.mark.parametrize("B,N,H,G,D,most", [(5, 7, 2, 4, 128, 700), (300, 1, 8, 1, 64, 100), (70, 3, 8, 2, 128, 900), (40, 2, 16, 1, 256, 300),
                                            (9, 20, 1, 2, 64, 760), (66, 1, 16, 1, 128, 2040)])
def test_whole_requests_in_a_long_table(B, N, H, G, D, most):
    """Short or many requests, which stay whole whatever the table's size."""
    announce(f"whole in a long table B={B} N={N} H={H} G={G} D={D}")
    rng = np.random.default_rng(B)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)])
    ctx, lens = rng.integers(0, most + 1, B), rng.integers(0, N + 1, B)
    ctx[0], ctx[B // 2], lens[0] = most - N, 0, N
    got, want = attention_case(B, N, H, G, D, 16, ctx, lens, mask, B, room=5000)
    check_attention(got, want)


@pytest.mark.parametrize("B,N,G,ctx", [(70, 1, 2, 1500), (1, 1, 4, 5000), (3, 1, 8, 2500), (70, 1, 2, 60), (2, 12, 8, 1500)])
def test_requests_split_over_workgroups(B, N, G, ctx):
    announce(f"split B={B} N={N} G={G} ctx={ctx}")
    rng = np.random.default_rng(B)
    lens = rng.integers(0, N + 1, B)
    lens[0] = N
    got, want = attention_case(B, N, 1, G, 64, 16, rng.integers(0, ctx + 1, B), lens, None, B + N)
    check_attention(got, want)


@pytest.mark.parametrize("B,N,H,G,D", [(400, 1, 2, 4, 64), (800, 1, 2, 1, 64), (300, 1, 2, 3, 128), (600, 1, 2, 1, 128), (150, 1, 2, 4, 256),
                                       (600, 1, 1, 2, 256), (250, 9, 2, 2, 64), (400, 5, 2, 4, 64), (800, 9, 2, 2, 64), (160, 5, 2, 4, 128),
                                       (270, 9, 2, 2, 128), (1030, 5, 1, 4, 128)])
def test_many_short_requests(B, N, H, G, D):
    """More workgroups than are resident with many waves each."""
    announce(f"many short B={B} N={N} H={H} G={G} D={D}")
    rng = np.random.default_rng(B)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)]) if N > 1 else None
    got, want = attention_case(B, N, H, G, D, 16, rng.integers(0, 120, B), rng.integers(0, N + 1, B), mask, B)
    check_attention(got, want)


def random_call(B=5, N=9, H=2, G=4, D=128, page=16, ctx=300, seed=0):
    rng = np.random.default_rng(seed)
    MP = -(-(ctx + N) // page)
    cache = tuple((dev(c), dev(s)) for c, s in ft.random_cache(rng, B * MP, H, page, D))
    table = dev(rng.permutation(B * MP).reshape(B, MP).astype(np.int32))
    q = torch.randn(B, N, H * G, D, device="cuda").bfloat16()
    lens = dev(rng.integers(0, N + 1, B).astype(np.int32))
    return [q, cache, table, dev(rng.integers(0, ctx + 1, B).astype(np.int32)), lens]


def test_unseen_tokens_do_not_touch_others():
    """NaN keys and values of one drafted token reach the rows that see it and no others."""
    announce("NaN in unseen tokens")
    q, cache, table, _, _ = random_call(B=1, N=6)
    ctx, lens = (torch.tensor([v], dtype=torch.int32, device="cuda") for v in (40, 6))
    mask = np.stack([ft.chain(6)])
    mask[0, 4, 2] = False
    words = dev(ft.pack_mask(mask))
    clean, clean_lse = dg.fp8_tree_attention(q, cache, table, ctx, lens, words)
    x = torch.randn(1, 2, 128, device="cuda")
    x[0, 1, 5] = float("nan")                        # key head 1 only
    slot = (table[0, 42 // 16] * 16 + 42 % 16).view(1).int()
    k, v = dg.fp8_kv_cache_read(cache, slot, dtype=torch.float32)
    for keys, values in ((x, v), (k, x)):
        dg.fp8_kv_cache_write(keys, values, cache, slot)
        o, lse = dg.fp8_tree_attention(q, cache, table, ctx, lens, words)
        sees = torch.tensor([False, False, True, True, False, True], device="cuda")
        assert o[0, sees, 4:].isnan().all() and not o[0, ~sees].isnan().any() and not o[0, :, :4].isnan().any()
        assert same_bits(o[0, [0, 1, 4], 4:], clean[0, [0, 1, 4], 4:])
        if keys is k:
            assert torch.equal(lse, clean_lse)       # a value's NaN is not in the scores
        dg.fp8_kv_cache_write(k, v, cache, slot)


@pytest.mark.parametrize("ctx", [300, 5000])
def test_strided_queries_given_outputs_and_workspaces(ctx):
    announce(f"strides, out=, workspace, {ctx}")
    args = random_call(ctx=ctx)
    q = args[0]
    o, lse = dg.fp8_tree_attention(*args)
    wide = torch.full((5, 9, 12, 128), float("nan"), device="cuda").bfloat16()
    wide[:, :, 2:10] = q
    ws = torch.full((dg.make_fp8_tree_attention_workspace(q, args[1], args[2]).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    out = (torch.full_like(o, 3.0), torch.full_like(lse, 3.0))
    for _ in range(3):
        got = dg.fp8_tree_attention(wide[:, :, 2:10], *args[1:], out=out, workspace=ws)
        assert got[0] is out[0] and same_bits(out[0], o) and same_bits(out[1], lse)
        out[0].fill_(3.0)
    none = dg.fp8_tree_attention(q[:0], args[1], args[2][:0], args[3][:0])
    assert none[0].shape == (0, 9, 8, 128)


def test_attention_binding_rejects():
    announce("attention refusals")
    q, cache, table, ctx, lens = random_call()
    mask = torch.zeros(5, 9, 1, dtype=torch.int64, device="cuda")
    for change, error in ((dict(q=q.float()), TypeError), (dict(q=q[..., :64]), ValueError), (dict(table=table.long()), TypeError),
                          (dict(table=table[:4]), ValueError), (dict(ctx=ctx[:4]), ValueError), (dict(lens=lens.long()), TypeError),
                          (dict(lens=lens[:4]), ValueError), (dict(mask=mask.int()), TypeError), (dict(mask=mask[:, :8]), ValueError),
                          (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError), (dict(q=q[:, :8]), ValueError),
                          (dict(cache=((cache[0][0].int(), cache[0][1]), cache[1])), TypeError),
                          (dict(cache=((cache[0][0][:2], cache[0][1]), cache[1])), ValueError)):
        a = dict(q=q, cache=cache, table=table, ctx=ctx, lens=lens, mask=mask) | change
        with pytest.raises(error):
            dg.fp8_tree_attention(a["q"], a["cache"], a["table"], a["ctx"], a["lens"], a["mask"])
    with pytest.raises(dg.DGError, match="multiple of H"):
        dg.fp8_tree_attention(q[:, :, :7].contiguous(), cache, table, ctx, lens)
    with pytest.raises(dg.DGError, match="needed"):
        dg.fp8_tree_attention(q, cache, table.repeat(1, 20), ctx, lens, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="uint8"):
        dg.fp8_tree_attention(q, cache, table, ctx, lens, workspace=torch.zeros(16, device="cuda"))


# ---- mixture of experts ------------------------------------------------------------------------------------

def moe_case(T, E, k, H, I, ids, dtype, seed):
    rng = np.random.default_rng(seed)
    w1, s1 = ft.quantise_blocks(rng.standard_normal((E, 2 * I, H)).astype(np.float32) / np.float32(H ** 0.5))
    w2, s2 = ft.quantise_blocks(rng.standard_normal((E, H, I)).astype(np.float32) / np.float32(I ** 0.5))
    x = torch.from_numpy((2 * rng.standard_normal((T, H))).astype(np.float32)).bfloat16()
    wt = rng.standard_normal((T, k)).astype(np.float32)
    ids = np.asarray(ids(rng), np.int32)
    args = [x.cuda(), (dev(w1), dev(s1)), (dev(w2), dev(s2)), dev(ids), dev(wt)]
    y = dg.fp8_moe_few_tokens(*args, dtype=TYPES[dtype])
    torch.cuda.synchronize()
    want, bound = ft.moe(x.double().numpy(), w1, s1, w2, s2, ids, wt, 2 if dtype == "bf16" else 3)
    got = y.double().cpu().numpy()
    none = ~((ids >= 0) & (ids < E)).any(1)
    assert not got[none].any()
    bound = bound + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23) * np.abs(want) + 1e-37
    worst = float((np.abs(got - want) / bound).max()) if T else 0.0
    assert worst <= 1, worst
    return args, y


def routed(T, E, k, drop=0.0):
    def make(rng):
        ids = np.stack([rng.permutation(max(E, k))[:k] for _ in range(T)]) if T else np.zeros((0, k))
        ids = np.where(ids < E, ids, -1)
        return np.where(rng.random(ids.shape) < drop, -1, ids)
    return make


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,H,I", [
    (1, 1, 1, 128, 128), (1, 8, 2, 1024, 512), (2, 5, 5, 256, 384), (5, 40, 8, 384, 128), (6, 3, 2, 128, 640), (8, 16, 4, 640, 256),
    (9, 8, 2, 256, 256), (16, 4, 4, 256, 128), (17, 4, 4, 256, 256), (32, 3, 3, 384, 128), (33, 2, 2, 128, 256), (64, 64, 6, 256, 128),
    (65, 9, 3, 128, 128), (130, 7, 4, 256, 256), (256, 20, 16, 128, 128), (3, 1024, 16, 128, 128)])
def test_moe(T, E, k, H, I, dtype):
    announce(f"moe T={T} E={E} k={k} H={H} I={I} {dtype}")
    moe_case(T, E, k, H, I, routed(T, E, k), dtype, T + E)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,H,I", [(256, 8, 2, 1280, 256), (130, 20, 3, 1792, 128), (17, 4, 2, 5120, 128), (64, 6, 4, 5248, 384),
                                       (9, 5, 1, 5120, 640), (200, 3, 1, 1408, 1024)])
def test_moe_many_rows_of_y(T, E, k, H, I, dtype):
    """Sizes whose second product is taken by waves that share the columns."""
    announce(f"moe many rows T={T} E={E} k={k} H={H} I={I} {dtype}")
    moe_case(T, E, k, H, I, routed(T, E, k, 0.1), dtype, T + E)
    moe_case(T, E, k, H, I, lambda rng: rng.choice([-1, 1, 2], (T, k)), dtype, T)
    if T == 17:
        moe_case(T, E, k, H, I, lambda rng: np.full((T, k), -1), dtype, T)
        args, y = moe_case(T, E, k, H, I, lambda rng: np.where(np.arange(T)[:, None] == 3, [1, 0], [-1, -1]), dtype, T)
        for _ in range(3):
            assert same_bits(dg.fp8_moe_few_tokens(*args, dtype=TYPES[dtype]), y)


@pytest.mark.parametrize("T", [1, 3, 12, 40, 100])
def test_moe_dropped_slots(T):
    announce(f"moe dropped slots T={T}")
    moe_case(T, 6, 4, 256, 256, routed(T, 6, 4, 0.6), "bf16", T)
    moe_case(T, 6, 4, 256, 256, lambda rng: np.full((T, 4), -1), "f32", T)
    moe_case(T, 6, 4, 256, 256, lambda rng: rng.choice([-2 ** 31, -7, 6, 2 ** 31 - 1, 2, 5], (T, 4)), "f32", T)


@pytest.mark.parametrize("T,dtype", [(4, "bf16"), (16, "f32"), (48, "bf16"), (64, "f32"), (70, "f32"), (256, "bf16")])
def test_moe_all_tokens_to_one_expert_and_repeated_ids(T, dtype):
    announce(f"moe skewed T={T}")
    moe_case(T, 9, 3, 256, 256, lambda rng: np.tile([7, -1, 7], (T, 1)), dtype, T)
    moe_case(T, 9, 3, 256, 256, lambda rng: rng.integers(0, 2, (T, 3)) * 4, dtype, T)


def test_moe_bad_tokens_stay_alone():
    """A token with NaN or infinite values spoils its own row only."""
    announce("moe NaN token")
    args, clean = moe_case(20, 6, 3, 256, 256, routed(20, 6, 3), "f32", 1)
    x = args[0].clone()
    x[3, 100], x[11, 0] = float("nan"), float("inf")
    y = dg.fp8_moe_few_tokens(x, *args[1:], dtype=torch.float32)
    keep = torch.ones(20, dtype=torch.bool, device="cuda")
    keep[3] = keep[11] = False
    assert same_bits(y[keep], clean[keep]) and y[3].isnan().all() and not y[11].isfinite().all()


def test_moe_given_output_workspace_and_refusals():
    announce("moe out=, workspace, refusals")
    args, y = moe_case(13, 8, 4, 384, 256, routed(13, 8, 4), "bf16", 2)
    ws = torch.full((dg.make_fp8_moe_few_tokens_workspace(args[0], args[2], args[3]).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full_like(y, 9.0)
    for _ in range(3):
        assert dg.fp8_moe_few_tokens(*args, out=out, workspace=ws) is out and same_bits(out, y)
        out.fill_(9.0)
    assert dg.fp8_moe_few_tokens(args[0][:0], args[1], args[2], args[3][:0], args[4][:0]).shape == (0, 384)
    x, w1, w2, ids, wt = args
    for bad, error in (((x.float(), w1, w2, ids, wt), TypeError), ((x, w1, w2, ids.long(), wt), TypeError),
                       ((x, w1, w2, ids, wt.bfloat16()), TypeError), ((x, w1, w2, ids[:5], wt), ValueError),
                       ((x[:, :256].contiguous(), w1, w2, ids, wt), ValueError), ((x, (w1[0], w2[1]), w2, ids, wt), ValueError),
                       ((x, w2, w2, ids, wt), ValueError), ((x.t().contiguous().t(), w1, w2, ids, wt), ValueError)):
        with pytest.raises(error):
            dg.fp8_moe_few_tokens(*bad)
    with pytest.raises(TypeError):
        dg.fp8_moe_few_tokens(*args, dtype=torch.float16)
    with pytest.raises(dg.DGError, match="T must be"):
        dg.fp8_moe_few_tokens(torch.zeros(257, 384, dtype=torch.bfloat16, device="cuda"), w1, w2,
                              torch.zeros(257, 4, dtype=torch.int32, device="cuda"), torch.zeros(257, 4, device="cuda"))


def test_moe_weights_past_32_bit_offsets():
    """The last of 80 experts of 4096 x 16384 + 4096 x 8192 values: offsets past 2^32."""
    announce("moe past 2^32")
    E, H, I, T = 80, 4096, 8192, 3
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("too little memory")
    w1 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=torch.uint8, device="cuda")
    s1, s2 = torch.ones(E, 2 * I // 128, H // 128, device="cuda"), torch.ones(E, H // 128, I // 128, device="cuda")
    x = torch.randn(T, H, device="cuda").bfloat16()
    one, half = 0x38, 0x30                            # 1 and 1/2
    # expert 79: hidden value 8191 is silu(x[4095]) * x[0], and y[4095] half of it
    w1[79, 8191, 4095], w1[79, 16383, 0], w2[79, 4095, 8191] = one, one, half
    ids = torch.full((T, 1), 79, dtype=torch.int32, device="cuda")
    y = dg.fp8_moe_few_tokens(x, (w1, s1), (w2, s2), ids, torch.ones(T, 1, device="cuda"), dtype=torch.float32)
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    g = x[:, 4095].double()
    want[:, 4095] = g / (1 + torch.exp(-g)) * x[:, 0].double() / 2
    assert torch.equal(y == 0, want == 0) and (y.double() - want).abs().max() <= 1e-6 * want.abs().max()


# ---- streams, graphs, repetition ------------------------------------------------------------------------------

def step(state):
    """Cache write, attention, read and MoE of one decode step, into fixed outputs."""
    s = state
    dg.fp8_kv_cache_write(s["k"], s["v"], s["cache"], s["slots"])
    dg.fp8_tree_attention(s["q"], s["cache"], s["table"], s["ctx"], s["lens"], None, out=s["o"], workspace=s["ws_a"])
    dg.fp8_kv_cache_read(s["cache"], s["slots"], out=s["rows"])
    dg.fp8_moe_few_tokens(s["x"], s["w1"], s["w2"], s["ids"], s["wt"], out=s["y"], workspace=s["ws_m"])


def decode_state(seed=0, ctx=700):
    torch.manual_seed(seed)
    rng = np.random.default_rng(seed)
    q, cache, table, ctx, lens = random_call(seed=seed, ctx=ctx)
    s = dict(q=q, cache=cache, table=table, ctx=ctx, lens=lens)
    s["k"], s["v"] = torch.randn(2, 30, 2, 128, device="cuda").bfloat16()
    s["slots"] = dev(rng.permutation(cache[0][0].shape[0] * 16)[:30].astype(np.int32))
    s["x"] = torch.randn(30, 256, device="cuda").bfloat16()
    s["w1"] = dg.per_block_cast_to_fp8(torch.randn(12, 512, 256, device="cuda") / 16)
    s["w2"] = dg.per_block_cast_to_fp8(torch.randn(12, 256, 256, device="cuda") / 16)
    s["ids"] = dev(rng.integers(-1, 12, (30, 4)).astype(np.int32))
    s["wt"] = torch.rand(30, 4, device="cuda")
    s["ws_a"] = dg.make_fp8_tree_attention_workspace(q, cache, table)
    s["ws_m"] = dg.make_fp8_moe_few_tokens_workspace(s["x"], s["w2"], s["ids"])
    s["o"] = (torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"))
    s["rows"] = (torch.empty(30, 2, 128, device="cuda"), torch.empty(30, 2, 128, device="cuda"))
    s["y"] = torch.empty(30, 256, device="cuda")
    return s


def outputs(s):
    return [*s["o"], *s["rows"], s["y"]]


@pytest.mark.parametrize("most", [700, 5000])
def test_a_step_is_bitwise_repeatable_and_capturable(most):
    announce(f"graph replays, {most}")
    s = decode_state(ctx=most)
    changes = [(s["ctx"].clone(), s["lens"].clone(), s["ids"].clone()),
               ((s["ctx"] // 3), (9 - s["lens"]).int(), s["ids"].flip(0).contiguous()),
               (torch.zeros_like(s["ctx"]), torch.zeros_like(s["lens"]), torch.full_like(s["ids"], -1))]
    eager = []
    for ctx, lens, ids in changes:
        s["ctx"].copy_(ctx), s["lens"].copy_(lens), s["ids"].copy_(ids)
        step(s)
        first = [t.clone() for t in outputs(s)]
        step(s)
        assert all(same_bits(a, b) for a, b in zip(first, outputs(s)))
        eager.append(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    for turn in range(2):
        for (ctx, lens, ids), want in zip(changes, eager):
            s["ctx"].copy_(ctx), s["lens"].copy_(lens), s["ids"].copy_(ids)
            for t in outputs(s):
                t.fill_(5.0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(same_bits(a, b) for a, b in zip(want, outputs(s)))
            (torch.ones(1000, device="cuda") * 2).sum().item()


def test_on_another_stream():
    announce("another stream")
    s = decode_state(1, ctx=5000)
    step(s)
    want = [t.clone() for t in outputs(s)]
    for t in outputs(s):
        t.zero_()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        step(s)
    torch.cuda.current_stream().wait_stream(other)
    assert all(same_bits(a, b) for a, b in zip(want, outputs(s)))


def test_slices_of_indices_lengths_masks_and_weights():
    """Small arrays at any element of a longer one."""
    announce("slices")
    s = decode_state(2)
    N = s["q"].shape[1]
    s["mask"] = dev(ft.pack_mask(np.stack([ft.random_tree(np.random.default_rng(b), N) for b in range(5)])))

    def run(s, o):
        step(s)
        dg.fp8_tree_attention(s["q"], s["cache"], s["table"], s["ctx"], s["lens"], s["mask"], out=o, workspace=s["ws_a"])

    def aside(t):
        wide = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        wide[1:] = t.reshape(-1)
        return wide[1:].view(t.shape)

    want_o = tuple(torch.empty_like(t) for t in s["o"])
    run(s, want_o)
    want = [t.clone() for t in (*outputs(s), *want_o)]
    for name in ("slots", "table", "ctx", "lens", "mask", "ids", "wt"):
        s[name] = aside(s[name])
        assert s[name].data_ptr() % 16
    s["o"] = (s["o"][0], aside(s["o"][1]))
    o = (torch.empty_like(want_o[0]), aside(want_o[1]))
    run(s, o)
    assert all(same_bits(a, b) for a, b in zip(want, (*outputs(s), *o)))
