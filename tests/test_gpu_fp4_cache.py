"""GPU parity of the FP4 key/value cache and of attention over it against the 64-bit references of
tests/paged.py, at the sizes and masks where they can go wrong.  Codes, scales and rows are compared
bit for bit; attention within bounds that count its roundings."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests import paged
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
    return tuple((torch.full((pages, H, page, D // 2), fill, dtype=torch.uint8, device="cuda"),
                  torch.full((pages, H, page, D // 32), fill, dtype=torch.uint8, device="cuda")) for _ in range(2))


def written(cache, sources, slots, fill=0xA5):
    """What a write of the rows leaves in the cache."""
    out = []
    for (codes, sf), src in zip(cache, sources):
        page = codes.shape[2]
        want, scale = paged.quantise4(src.float().cpu().numpy())
        pool, scales = np.full(codes.shape, fill, np.uint8), np.full(sf.shape, fill, np.uint8)
        live = (slots >= 0) & (slots < codes.shape[0] * page)
        at = slots[live]
        pool[at // page, :, at % page], scales[at // page, :, at % page] = want[live], scale[live]
        out.append((pool, scales, want, scale, live))
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 64, 16), (1, 8, 128, 64), (7, 3, 128, 16), (65, 2, 256, 32), (300, 5, 64, 128),
                                        (1000, 8, 128, 64), (33, 1, 256, 4096)])
def test_cache_write_and_read(T, H, D, page, dtype):
    announce(f"fp4 cache T={T} H={H} D={D} page={page} {dtype}")
    rng = np.random.default_rng(T + H + D)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    x = rng.standard_normal((2, T, H, D)).astype(np.float32) * np.exp2(rng.integers(-20, 20, (2, T, H, D // 32))).astype(np.float32).repeat(32, -1)
    x[0, 0, 0] = 0                                     # a row of zeros
    x[1, -1, -1, ::2] = -0.0
    x[1, T // 2, 0] *= np.float32(2.0 ** -130)          # scales at the lower end, and below the normal numbers
    if T > 2:
        slots[T // 3], slots[T // 3 + 1] = -1, pages * page   # not stored
    t = [dev(v).to(TYPES[dtype]) for v in x]
    # tokens as slices of a wider row: keys and values side by side
    wide = torch.zeros(T, 2 * H + 1, D, dtype=TYPES[dtype], device="cuda")
    wide[:, :H], wide[:, H:2 * H] = t[0], t[1]
    cache = cache_of(pages, H, page, D)
    got = dg.fp4_kv_cache_write(wide[:, :H], wide[:, H:2 * H], cache, dev(slots))
    assert got is cache
    for out in TYPES.values():
        rows = dg.fp4_kv_cache_read(cache, dev(slots), dtype=out)
        for (codes, sf), r, (pool, scales, want, scale, live) in zip(cache, rows, written(cache, t, slots)):
            np.testing.assert_array_equal(codes.cpu().numpy(), pool)
            np.testing.assert_array_equal(sf.cpu().numpy(), scales)
            values = paged.values4(want, scale).astype(np.float32)
            values[~live] = 0
            assert r.dtype == out and same_bits(r, torch.from_numpy(values).to(out).cuda())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_every_rounding(dtype):
    """Middles of neighbouring values and what is next to them, over all scales, with a largest value
    on either side of each power of two's limit."""
    announce(f"fp4 cache: middles {dtype}")
    middles = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((4 * 251, 1, 64), np.float64)
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    for e in range(-125, 126):
        for k, most in enumerate((6.0, 6.0 * (1 + step), 3.0 * (1 + step), 4.0)):
            row = np.concatenate([middles, -middles, middles * (1 - step), -middles * (1 + step)])
            if most * 2.0 ** e < 3e38:
                x[4 * (e + 125) + k, 0, :28] = np.clip(row, -most, most) * 2.0 ** e
                x[4 * (e + 125) + k, 0, 31] = most * 2.0 ** e
            x[4 * (e + 125) + k, 0, 32:] = 5.5 * 2.0 ** min(e, 120)
    t = torch.from_numpy(x).to(TYPES[dtype]).cuda()
    cache = cache_of(63, 1, 16, 64)
    slots = np.arange(len(x), dtype=np.int32)
    dg.fp4_kv_cache_write(t, -t, cache, dev(slots))
    for (codes, sf), (pool, scales, *_) in zip(cache, written(cache, (t, -t), slots)):
        np.testing.assert_array_equal(sf.cpu().numpy(), scales)
        np.testing.assert_array_equal(codes.cpu().numpy(), pool)


def test_cache_smallest_and_largest():
    announce("fp4 cache: ends of fp32")
    x = np.zeros((8, 1, 64), np.float32)
    x[0, 0, :4] = [3.4028235e38, -3.4e38, 2.0 ** 127, 1.0]
    x[1, 0, :4] = [1e-45, -1e-40, 2.0 ** -126, 0]
    x[2, 0, :4] = [6 * 2.0 ** -125, 0.25 * 2.0 ** -125, 0.3 * 2.0 ** -125, 0]
    x[3, 0, :4] = [1e-45, 0, 0, 0]
    x[4, 0, :4] = [6 * 2.0 ** 125, 2.0 ** 122, 2.0 ** 123, 0]
    t = dev(x)
    cache = cache_of(1, 1, 16, 64)
    slots = np.arange(8, dtype=np.int32)
    dg.fp4_kv_cache_write(t, -t, cache, dev(slots))
    for (codes, sf), (pool, scales, *_) in zip(cache, written(cache, (t, -t), slots)):
        np.testing.assert_array_equal(sf.cpu().numpy(), scales)
        np.testing.assert_array_equal(codes.cpu().numpy(), pool)
    rows = dg.fp4_kv_cache_read(cache, dev(slots), dtype=torch.float32)
    assert rows[0].isfinite().all()


def test_cache_blocks_that_are_not_finite():
    announce("fp4 cache: NaN and infinite blocks")
    for D in (64, 128, 256):
        x = torch.randn(6, 2, D, device="cuda")
        x[1, 0, 17], x[2, 1, D - 1], x[3, 0, 32] = float("nan"), float("inf"), -float("inf")
        cache = cache_of(1, 2, 16, D)
        slots = torch.arange(6, dtype=torch.int32, device="cuda")
        dg.fp4_kv_cache_write(x, x.flip(0).contiguous(), cache, slots)
        bad = torch.zeros(6, 2, D // 32, dtype=torch.bool, device="cuda")
        bad[1, 0, 0] = bad[2, 1, -1] = bad[3, 0, 1] = True
        for dtype in TYPES.values():
            k, v = dg.fp4_kv_cache_read(cache, slots, dtype=dtype)
            for rows, want in ((k, bad), (v, bad.flip(0))):
                assert torch.equal(rows.isnan(), want.repeat_interleave(32, -1))
        assert torch.equal(cache[0][1][0, :, :6].transpose(0, 1) == 255, bad)


def test_cache_into_given_rows_and_single_tokens():
    announce("fp4 cache: out=, T = 0, T = 1")
    cache = cache_of(2, 2, 16, 64)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    e = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    dg.fp4_kv_cache_write(e, e, cache, none)
    assert dg.fp4_kv_cache_read(cache, none)[0].shape == (0, 2, 64) and (cache[0][0] == 0xA5).all()
    x = torch.randn(1, 2, 64, device="cuda").bfloat16()
    slot = torch.tensor([31], dtype=torch.int32, device="cuda")
    dg.fp4_kv_cache_write(x, 2 * x, cache, slot)
    out = (torch.empty(1, 2, 64, device="cuda"), torch.empty(1, 2, 64, device="cuda"))
    got = dg.fp4_kv_cache_read(cache, slot, out=out)
    assert got[0] is out[0] and torch.equal(out[1], 2 * out[0])
    # written again, rows keep their values: codes up to 3 may become twice that of half the scale
    dg.fp4_kv_cache_write(*out, cache, slot)
    assert all(torch.equal(a, b) for a, b in zip(out, dg.fp4_kv_cache_read(cache, slot, dtype=torch.float32)))


def test_make_cache_is_empty():
    cache = dg.make_fp4_kv_cache(3, 2, 16, 128)
    k, v = dg.fp4_kv_cache_read(cache, torch.arange(48, dtype=torch.int32, device="cuda"))
    assert k.shape == (48, 2, 128) and not k.any() and not v.any()


def test_cache_larger_than_32_bit_offsets():
    """The last pages of pools of 5.0 GB: offsets past 2^32."""
    announce("fp4 cache and attention past 2^32")
    H, page, D, pages = 8, 64, 128, 152000
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("too little memory")
    cache = dg.make_fp4_kv_cache(pages, H, page, D)
    T = 130
    x = torch.randn(2, T, H, D, device="cuda").bfloat16()
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device="cuda")
    pos = torch.arange(T, device="cuda")
    slots = (table[0].long()[pos // page] * page + pos % page).int()
    dg.fp4_kv_cache_write(x[0], x[1], cache, slots)
    small = dg.make_fp4_kv_cache(3, H, page, D)
    dg.fp4_kv_cache_write(x[0], x[1], small, pos.int())
    for a, b in zip(dg.fp4_kv_cache_read(cache, slots), dg.fp4_kv_cache_read(small, pos.int())):
        assert same_bits(a, b)
    q = torch.randn(1, 1, 32, D, device="cuda").bfloat16()
    ctx = torch.tensor([T - 1], dtype=torch.int32, device="cuda")
    near = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    for a, b in zip(dg.fp4_tree_attention(q, cache, table, ctx), dg.fp4_tree_attention(q, small, near, ctx)):
        assert same_bits(a, b)


# ---- attention -----------------------------------------------------------------------------------------

def attention_case(B, N, H, G, D, page, ctx, lens, mask, seed, scale=None, hide=(), q_scale=1.0, room=0, change=None):
    """A random case run on the GPU, with NaN scales wherever no one may look.  room: positions that the
    table has beyond the longest request (with many, requests are split); change(cache, table): what else is
    made of the cache."""
    rng = np.random.default_rng(seed)
    ctx, lens = np.asarray(ctx, np.int32), np.asarray(lens, np.int32)
    MP = max(1, -(-int((np.clip(ctx, 0, None) + np.clip(lens, 0, N)).max()) // page)) + 1
    pages = B * MP + 2
    cache = paged.random_cache4(rng, pages, H, page, D)
    table = rng.permutation(pages)[:B * MP].reshape(B, MP).astype(np.int32)
    live = np.zeros((pages, page), bool)
    for b in range(B):
        p = np.arange(min(max(ctx[b], 0) + min(max(lens[b], 0), N), MP * page))
        live[table[b, p // page], p % page] = True
    for codes, sf in cache:
        codes.transpose(0, 2, 1, 3)[~live] = 0x7F
        sf.transpose(0, 2, 1, 3)[~live] = 255
    if change:
        change(cache, table)
    for b, p, value in hide:
        table[b, p] = value
    table = np.concatenate([table, np.full((B, room // page), -7, np.int32)], 1)
    q = torch.from_numpy((q_scale * rng.standard_normal((B, N, H * G, D))).astype(np.float32)).bfloat16()
    scale = D ** -0.5 if scale is None else scale
    words = None if mask is None else dev(ft.pack_mask(mask))
    on_gpu = tuple((dev(c), dev(s)) for c, s in cache)
    o, lse = dg.fp4_tree_attention(q.cuda(), on_gpu, dev(table), dev(ctx), dev(lens), words, scale)
    torch.cuda.synchronize()
    full = np.stack([ft.chain(N)] * B) if mask is None else mask
    return (o.float().cpu().numpy(), lse.cpu().numpy()), paged.attention4(q.float().numpy(), cache, table, ctx, lens, full, scale, page)


def check_attention(got, want):
    (o, lse), (ro, rl, bo, bl) = got, want
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty) and not o[empty].any()
    assert np.array_equal(np.isnan(o), np.isnan(ro)) and np.array_equal(np.isnan(lse), np.isnan(rl))
    assert np.isfinite(o[~np.isnan(ro)]).all()
    ok = ~np.isnan(ro)
    assert (np.abs(o - ro)[ok] <= bo[ok]).all(), float((np.abs(o - ro)[ok] / np.maximum(bo[ok], 1e-300)).max())
    ok = ~empty & ~np.isnan(rl)
    off = np.abs(lse[ok] - rl[ok])
    assert (off <= bl[ok]).all(), float((off / bl[ok]).max())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_decode_lengths(D, page):
    announce(f"fp4 decode D={D} page={page}")
    ctx = [0, 1, 14, 15, 16, 17, 31, 32, 33, 63, 64, 127, 200, 601]
    B = len(ctx)
    check_attention(*attention_case(B, 1, 2, 4, D, page, ctx, [1] * (B - 1) + [0], None, D + page))


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 17, 33])
def test_query_heads_of_a_key_head(G):
    announce(f"fp4 attention G={G}")
    check_attention(*attention_case(2, 1, 3, G, 128, 16, [70, 33], [1, 1], None, G))


@pytest.mark.parametrize("N,G,D", [(2, 1, 64), (3, 4, 128), (5, 8, 64), (16, 2, 256), (17, 4, 128), (24, 8, 64), (33, 4, 64),
                                   (64, 1, 128), (65, 2, 64), (130, 1, 128), (20, 16, 128), (40, 2, 256)])
def test_trees(N, G, D):
    announce(f"fp4 tree N={N} G={G} D={D}")
    rng = np.random.default_rng(N)
    ctx, lens = [100, 0, 37, 5], [N, N - 1, max(N // 2, 1), 0]
    mask = np.stack([ft.random_tree(rng, N) for _ in ctx])
    check_attention(*attention_case(4, N, 2, G, D, 16, ctx, lens, mask, N))


def test_chain_is_the_mask_that_is_not_given():
    announce("fp4 chain")
    a = attention_case(2, 19, 2, 4, 128, 32, [50, 0], [19, 12], None, 3)
    b = attention_case(2, 19, 2, 4, 128, 32, [50, 0], [19, 12], np.stack([ft.chain(19)] * 2), 3)
    check_attention(*a)
    assert np.array_equal(a[0][0], b[0][0]) and np.array_equal(a[0][1], b[0][1])


def test_masks_that_leave_rows_empty():
    announce("fp4 empty rows")
    rng = np.random.default_rng(7)
    mask = rng.random((3, 40, 40)) < 0.05            # rows of nothing, rows that miss themselves
    mask[0, :7] = False
    got, want = attention_case(3, 40, 2, 4, 128, 16, [0, 0, 9], [40, 21, 40], mask, 8)
    assert np.isneginf(want[1]).any()
    check_attention(got, want)
    blind = np.zeros((2, 1, 1), bool)                # single tokens that do not see themselves
    check_attention(*attention_case(2, 1, 2, 4, 128, 16, [0, 33], [1, 1], blind, 9))


def test_lengths_out_of_range_are_clamped():
    announce("fp4 clamped lengths")
    check_attention(*attention_case(4, 3, 1, 2, 64, 16, [-5, 20, 7, 40], [3, 99, -4, 3], None, 9))


def test_hidden_pages():
    announce("fp4 hidden pages")
    check_attention(*attention_case(2, 2, 2, 4, 128, 16, [70, 64], [2, 2], None, 10, hide=((0, 1, -1), (0, 3, 1 << 30), (1, 0, 9999))))


def test_scores_far_apart():
    """Scores over hundreds, so that most weights vanish, and a scale of 0 and below."""
    announce("fp4 scores far apart")
    for scale, qs in ((1.0, 30.0), (0.0, 1.0), (-0.5, 2.0)):
        check_attention(*attention_case(2, 3, 2, 4, 128, 16, [150, 40], [3, 2], None, 11, scale=scale, q_scale=qs))


@pytest.mark.parametrize("N,G,D", [(1, 4, 64), (1, 3, 128), (1, 16, 256), (3, 4, 128), (16, 2, 256), (17, 4, 128), (24, 8, 64),
                                   (65, 2, 64), (130, 1, 128)])
def test_short_requests_in_a_long_table(N, G, D):
    """Split over workgroups by the table's size, with lengths around tiles and steps, trees, hidden
    pages and rows that see nothing."""
    announce(f"fp4 split short N={N} G={G} D={D}")
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
    announce(f"fp4 whole in a long table B={B} N={N} H={H} G={G} D={D}")
    rng = np.random.default_rng(B)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)])
    ctx, lens = rng.integers(0, most + 1, B), rng.integers(0, N + 1, B)
    ctx[0], ctx[B // 2], lens[0] = most - N, 0, N
    check_attention(*attention_case(B, N, H, G, D, 16, ctx, lens, mask, B, room=5000))


@pytest.mark.parametrize("B,N,H,G,D,most,room", [(2, 12, 2, 8, 64, 9000, 0), (2, 12, 2, 8, 128, 9000, 0), (10, 7, 2, 4, 128, 700, 9000),
                                                  (6, 9, 2, 4, 64, 1900, 9000), (3, 5, 2, 8, 128, 4000, 9000), (130, 5, 2, 4, 64, 1500, 0),
                                                  (130, 5, 2, 8, 128, 1500, 0), (40, 5, 8, 4, 64, 3500, 0)])
def test_two_row_tiles(B, N, H, G, D, most, room):
    """Tables long enough, or workgroups many enough, for 32 rows in each: split, dealt in turn, whole."""
    announce(f"fp4 two row tiles B={B} N={N} H={H} G={G} D={D} room={room}")
    rng = np.random.default_rng(B + D)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)])
    ctx, lens = rng.integers(0, most + 1, B), rng.integers(0, N + 1, B)
    ctx[0], ctx[B // 2], lens[0] = most - N, 0, N
    check_attention(*attention_case(B, N, H, G, D, 16, ctx, lens, mask, B, room=room))


@pytest.mark.parametrize("B,N,G,most,room", [(33, 1, 2, 3000, 5000), (34, 4, 4, 2100, 9000), (33, 2, 4, 2000, 50000), (32, 1, 2, 6000, 20000)])
def test_sixteen_waves_a_workgroup(B, N, G, most, room):
    """Heads of 64 in tables of long requests: whole ones, short ones dealt to the runs, split ones."""
    announce(f"fp4 sixteen waves B={B} N={N} G={G} room={room}")
    rng = np.random.default_rng(room)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)])
    ctx, lens = rng.integers(0, most + 1, B), rng.integers(0, N + 1, B)
    ctx[0], ctx[B // 2], lens[0] = most - N, 0, N
    check_attention(*attention_case(B, N, 8, G, 64, 16, ctx, lens, mask, B, room=room))


@pytest.mark.parametrize("B,N,G,ctx", [(70, 1, 2, 1500), (1, 1, 4, 5000), (3, 1, 8, 2500), (70, 1, 2, 60), (2, 12, 8, 1500), (70, 1, 2, 4500)])
def test_requests_split_over_workgroups(B, N, G, ctx):
    announce(f"fp4 split B={B} N={N} G={G} ctx={ctx}")
    rng = np.random.default_rng(B)
    lens = rng.integers(0, N + 1, B)
    lens[0] = N
    check_attention(*attention_case(B, N, 1, G, 64, 16, rng.integers(0, ctx + 1, B), lens, None, B + N))


@pytest.mark.parametrize("B,N,H,G,D", [(400, 1, 2, 4, 64), (800, 1, 2, 1, 64), (300, 1, 2, 3, 128), (600, 1, 2, 1, 128), (150, 1, 2, 4, 256),
                                       (600, 1, 1, 2, 256), (250, 9, 2, 2, 64), (400, 5, 2, 4, 64), (800, 9, 2, 2, 64), (160, 5, 2, 4, 128),
                                       (270, 9, 2, 2, 128), (1030, 5, 1, 4, 128)])
def test_many_short_requests(B, N, H, G, D):
    """More workgroups than are resident with many waves each."""
    announce(f"fp4 many short B={B} N={N} H={H} G={G} D={D}")
    rng = np.random.default_rng(B)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(B)]) if N > 1 else None
    check_attention(*attention_case(B, N, H, G, D, 16, rng.integers(0, 120, B), rng.integers(0, N + 1, B), mask, B))


@pytest.mark.parametrize("N,D,room", [(1, 128, 0), (6, 64, 0), (6, 128, 0), (6, 128, 5000), (6, 128, 9000), (6, 64, 9000), (20, 256, 0)])
def test_scales_that_are_nan(N, D, room):
    """NaN scales of keys and values in the context and in drafted tokens: what sees them, and of values
    the 32 that they belong to, is NaN and nothing else."""
    announce(f"fp4 NaN N={N} D={D} room={room}")
    rng = np.random.default_rng(N)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(3)])

    def change(cache, table):
        (_, ks), (_, vs) = cache
        vs[table[0, 1], 0, 5, D // 32 - 1] = 255       # a context token's value
        ks[table[1, 0], 1, 7, 0] = 255                 # a context token's key
        for j in (1, 2, N - 1):                        # values of drafted tokens of request 2, at 40 + j
            if j < N:
                vs[table[2, (40 + j) // 16], 0, (40 + j) % 16, j % (D // 32)] = 255
        if N > 3:
            ks[table[2, 43 // 16], 1, 43 % 16, 1] = 255

    got, want = attention_case(3, N, 2, 4, D, 16, [40, 33, 40], [N, N, N], mask, 5, room=room, change=change)
    assert np.isnan(want[0]).any() and (N == 1 or not np.isnan(want[0]).all((2, 3)).all())
    check_attention(got, want)


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("far", [60, 124])
@pytest.mark.parametrize("room", [5000, 9000])
def test_values_of_very_different_sizes(N, far, room):
    """Scales of 2^far and 2^-far of values, some hidden from some rows: sums do not overflow, and small
    blocks keep their bits beside large ones."""
    announce(f"fp4 large values N={N} far={far} room={room}")
    rng = np.random.default_rng(far)
    mask = np.stack([ft.random_tree(rng, N) for _ in range(2)])

    def change(cache, table):
        vs = cache[1][1]
        vs[...] = np.where(vs == 255, 255, 127 - 2)
        vs[:, :, :, 0] = np.where(vs[:, :, :, 0] == 255, 255, 127 + far)
        if far < 90:                                   # below that terms may count as 0
            vs[:, :, :, 1] = np.where(vs[:, :, :, 1] == 255, 255, 127 - far)
        vs[table[1, 2], 0, 9] = 127 + far              # one drafted token (position 41), all blocks

    got, want = attention_case(2, N, 2, 4, 128, 16, [300, 40], [N, N], mask, far, change=change, room=room if N == 5 else 0)
    check_attention(got, want)


def test_extreme_keys_and_queries():
    """A query with an infinity or a NaN is NaN and leaves the others alone."""
    announce("fp4 queries that are not finite")
    q, cache, table, ctx, lens = random_call()
    o, lse = dg.fp4_tree_attention(q, cache, table, ctx, lens)
    bad = q.clone()
    bad[0, 0, 1, 5], bad[1, 1, 3, 100], bad[3, 0, 7, 0] = float("inf"), float("nan"), -float("inf")
    o2, lse2 = dg.fp4_tree_attention(bad, cache, table, ctx, lens)
    hit = ~torch.isfinite(bad).all(-1)
    seen = hit & ~torch.isneginf(lse)
    assert seen.any() and o2[seen].isnan().all() and lse2[seen].isnan().all()
    assert same_bits(o2[~hit], o[~hit]) and same_bits(lse2[~hit], lse[~hit])


@pytest.mark.parametrize("room", [0, 9000])
@pytest.mark.parametrize("seed", range(6))
def test_a_row_depends_on_its_own_query_alone(seed, room):
    """Other queries of the same call changed, larger and not finite: a row keeps its bits."""
    announce(f"fp4 rows apart seed={seed} room={room}")
    q, cache, table, ctx, lens = random_call(seed=seed)
    table = torch.cat([table, torch.full((table.shape[0], room // 16), -1, dtype=torch.int32, device="cuda")], 1)
    o, lse = dg.fp4_tree_attention(q, cache, table, ctx, lens)
    for change in (float("nan"), float("inf"), 30.0, -3.0):
        other = q.clone()
        other[:, ::2, ::3] *= change
        o2, lse2 = dg.fp4_tree_attention(other, cache, table, ctx, lens)
        same = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
        same[:, ::2, ::3] = False
        assert same_bits(o2[same], o[same]) and same_bits(lse2[same], lse[same])


def random_call(B=5, N=9, H=2, G=4, D=128, page=16, ctx=300, seed=0):
    rng = np.random.default_rng(seed)
    MP = -(-(ctx + N) // page)
    cache = tuple((dev(c), dev(s)) for c, s in paged.random_cache4(rng, B * MP, H, page, D))
    table = dev(rng.permutation(B * MP).reshape(B, MP).astype(np.int32))
    q = torch.randn(B, N, H * G, D, device="cuda").bfloat16()
    lens = dev(rng.integers(1, N + 1, B).astype(np.int32))
    return [q, cache, table, dev(rng.integers(0, ctx + 1, B).astype(np.int32)), lens]


@pytest.mark.parametrize("ctx", [300, 5000])
def test_strided_queries_given_outputs_and_workspaces(ctx):
    announce(f"fp4 strides, out=, workspace, {ctx}")
    args = random_call(ctx=ctx)
    q = args[0]
    o, lse = dg.fp4_tree_attention(*args)
    wide = torch.full((5, 9, 12, 128), float("nan"), device="cuda").bfloat16()
    wide[:, :, 2:10] = q
    ws = torch.full((dg.make_fp4_tree_attention_workspace(q, args[1], args[2]).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    assert (ws.numel() > 0) == (ctx == 5000)
    out = (torch.full_like(o, 3.0), torch.full_like(lse, 3.0))
    for _ in range(3):
        got = dg.fp4_tree_attention(wide[:, :, 2:10], *args[1:], out=out, workspace=ws)
        assert got[0] is out[0] and same_bits(out[0], o) and same_bits(out[1], lse)
        out[0].fill_(3.0)
    none = dg.fp4_tree_attention(q[:0], args[1], args[2][:0], args[3][:0])
    assert none[0].shape == (0, 9, 8, 128)


@pytest.mark.parametrize("ctx", [300, 5000])
def test_graph_replays_with_changed_lengths(ctx):
    announce(f"fp4 graph {ctx}")
    q, cache, table, lens, tree = random_call(ctx=ctx, seed=4)
    k, v = (torch.randn(7, 2, 128, device="cuda").bfloat16() for _ in range(2))
    slots = torch.arange(7, dtype=torch.int32, device="cuda")
    ws = dg.make_fp4_tree_attention_workspace(q, cache, table)

    def step():
        dg.fp4_kv_cache_write(k, v, cache, slots)
        return dg.fp4_tree_attention(q, cache, table, lens, tree, workspace=ws) + dg.fp4_kv_cache_read(cache, slots)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        lens.copy_((lens * 3 + 17 * i) % (ctx + 1)), slots.add_(5), k.copy_(torch.randn_like(k)), q.mul_(-1)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        assert all(same_bits(a, b) for a, b in zip(replayed, step()))


def test_other_stream_and_two_calls_at_once():
    announce("fp4 streams")
    args, more = random_call(ctx=5000, seed=5), random_call(ctx=5000, seed=6)
    want = dg.fp4_tree_attention(*args), dg.fp4_tree_attention(*more)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, (s, a) in enumerate(zip(streams, (args, more))):
            with torch.cuda.stream(s):
                got[i] = dg.fp4_tree_attention(*a)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert same_bits(a[0], b[0]) and same_bits(a[1], b[1])


def test_binding_rejects():
    announce("fp4 refusals")
    q, cache, table, ctx, lens = random_call()
    k = torch.randn(3, 2, 128, device="cuda").bfloat16()
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    eight = dg.make_fp8_kv_cache(4, 2, 16, 128)
    (kc, ks), (vc, vs) = cache
    for bad, error, text in ((eight, TypeError, "k scales must be uint8"), (((kc, ks[..., :2]), (vc, vs)), ValueError, ""),
                             (((kc, ks), (vc, vs[..., :2].contiguous())), ValueError, "cache shapes"),
                             (((kc[:, :1].contiguous(), ks), (vc, vs)), ValueError, "cache shapes"),
                             (((kc.cpu(), ks), (vc, vs)), ValueError, "device tensor")):
        with pytest.raises(error, match=text or "contiguous"):
            dg.fp4_kv_cache_write(k, k, bad, slots)
        with pytest.raises(error, match=text or "contiguous"):
            dg.fp4_kv_cache_read(bad, slots)
        with pytest.raises(error, match=text or "contiguous"):
            dg.fp4_tree_attention(q, bad, table, ctx)
    with pytest.raises((TypeError, ValueError)):
        dg.fp8_tree_attention(q, cache, table, ctx)
    with pytest.raises(ValueError, match="shape mismatch"):
        dg.fp4_kv_cache_write(k[..., :64], k[..., :64], cache, slots)
    with pytest.raises(TypeError, match="slots must be int32"):
        dg.fp4_kv_cache_write(k, k, cache, slots.long())
    with pytest.raises(TypeError, match="q must be bfloat16"):
        dg.fp4_tree_attention(q.float(), cache, table, ctx)
    with pytest.raises(ValueError, match="must be"):
        dg.fp4_tree_attention(q[..., :64], cache, table, ctx)
    with pytest.raises(dg.DGError, match="overlap"):
        dg.fp4_tree_attention(q, cache, table, ctx, out=(q, torch.empty(5, 9, 8, device="cuda")))
    long = torch.zeros(5, 400, dtype=torch.int32, device="cuda")
    with pytest.raises(dg.DGError, match="needed"):
        dg.fp4_tree_attention(q, cache, long, ctx, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
