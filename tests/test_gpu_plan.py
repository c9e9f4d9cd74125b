"""GPU results of the plan of pages and slots against the request-by-request reference of
tests/paged.py: all whole numbers, compared for equality."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import paged
from tests.parity import announce, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


def check(table, ctx, add, ring, state, page, rows, padded):
    want = paged.plan(table, ctx, add, ring, state, page, rows, padded)
    t, r, s = dev(table), dev(ring), dev(np.asarray(state, np.int32))
    c, a = dev(np.asarray(ctx, np.int32)), dev(np.asarray(add, np.int32))
    slots, positions, lens, new_state = dg.kv_cache_plan(t, c, a, (r, s), page, rows, padded)
    for got, ref, what in zip((t, slots, positions, lens, r, new_state), want,
                              ("table", "slots", "positions", "lens", "ring", "state")):
        assert got.dtype == torch.int32
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=what)
    assert np.array_equal(c.cpu().numpy(), ctx) and np.array_equal(s.cpu().numpy(), state)
    return t, r, new_state, lens


def lengths(rng, B, page, most, grow):
    """Contexts from 0 on, on and around page borders; changes in either direction."""
    ctx = rng.integers(0, most + 1, B)
    edge = rng.random(B) < 0.4
    ctx[edge] = np.maximum(ctx[edge] // page * page + rng.integers(-1, 2, B)[edge], 0)
    add = rng.integers(-most // 2, grow + 1, B)
    add[rng.random(B) < 0.2] = 0
    done = rng.random(B) < 0.1
    add[done] = -ctx[done]
    return ctx.astype(np.int32), add.astype(np.int32)


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("B,page,most,grow", [(1, 16, 0, 1), (1, 16, 40, 70), (7, 16, 100, 40), (64, 64, 300, 3), (255, 16, 60, 33),
                                              (256, 32, 200, 1), (257, 16, 100, 20), (1024, 16, 70, 5), (1025, 16, 40, 9), (3000, 128, 500, 2),
                                              (2, 4096, 9000, 5000)])
@pytest.mark.parametrize("enough", [True, False])
def test_random_batches(B, page, most, grow, padded, enough):
    announce(f"plan B={B} page={page} most={most} grow={grow} padded={padded} enough={enough}")
    rng = np.random.default_rng(B + page + padded)
    ctx, add = lengths(rng, B, page, most, grow)
    lack = int(np.maximum(-(-(ctx + np.maximum(add, 0)) // page) - -(-ctx // page), 0).sum())
    table, ring, state = paged.random_pool(rng, B, page, ctx, lack + 3 if enough else lack // 2 + 1)
    new = int(np.maximum(add, 0).sum())
    for rows in ((grow, max(grow - 1, 0)) if padded else (new, new + 37, max(new - 5, 0))):
        check(table, ctx, add, ring, state, page, rows, padded)


def test_first_request_without_room_ends_the_service():
    """Requests after the first that lacks pages get none, but those that need none are served."""
    announce("plan: pool short")
    rng = np.random.default_rng(3)
    ctx = [16, 15, 40, 8, 32]
    table, ring, state = paged.random_pool(rng, 5, 16, ctx, 3)
    t, r, s, lens = check(table, ctx, [16, 1, 48, 4, 1], ring, state, 16, 100, False)
    assert lens.tolist() == [32, 16, 40, 12, 32] and s.tolist()[1] == 2


def test_longer_than_the_table_or_the_rows():
    announce("plan: table and rows short")
    rng = np.random.default_rng(4)
    ctx = [60, 64, 10, 5]
    table, ring, state = paged.random_pool(rng, 4, 16, ctx, 12)
    table = np.ascontiguousarray(table[:, :4])
    check(table, ctx, [4, 1, 3, 60], ring, state, 16, 200, False)
    check(table, ctx, [4, 1, 3, 60], ring, state, 16, 3, True)
    check(table, ctx, [4, 1, 3, 60], ring, state, 16, 0, True)
    big = np.iinfo(np.int32).max
    check(table, ctx, [1, big, big, 2], ring, state, 16, 64, False)
    check(table, ctx, [1, big, -big - 1, 2], ring, state, 16, 5, True)


def test_lengths_and_states_out_of_range():
    announce("plan: clamped")
    rng = np.random.default_rng(5)
    table, ring, _ = paged.random_pool(rng, 3, 16, [20, 30, 0], 9)
    table[1, 0], table[0, 1] = -3, 1 << 20                # pages of no cache: no slots
    for state in ([-1, 4], [len(ring) + 3, 4], [2, -7]):
        check(table, [20, 30, -9], [3, 2, 5], ring, state, 16, 12, False)
    full = len(ring)                                      # all free: more than there are
    check(table, [0, 0, 0], [1, 16, 17], ring, [5, full + 100], 16, 40, False)


@pytest.mark.parametrize("B", [2, 9, 700])
def test_shared_pages_come_back_from_each_request(B):
    """More pages come back than the ring has places for: the first ones are kept, and the free
    pages that a growing request takes in the same call are not written over."""
    announce(f"plan: shared pages B={B}")
    rng = np.random.default_rng(B)
    P, width = 3 * B, 8
    ring = rng.permutation(P).astype(np.int32)
    table = np.repeat(rng.permutation(P)[None, :width], B, 0).astype(np.int32)[:, :6].copy()
    table = np.concatenate([table, np.full((B, 4), -1, np.int32)], 1)
    ctx = np.full(B, 6 * 16, np.int32)
    add = np.where(np.arange(B) % 2 == 0, -6 * 16, 16).astype(np.int32)
    for free in (B // 2, P - 3, P):
        _, _, state, _ = check(table, ctx, add, ring, [P - 2, free], 16, 16 * B, False)
        assert state[1].item() <= P


def test_no_requests():
    announce("plan: B = 0")
    pool = dg.make_kv_page_pool(5)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, positions, lens, state = dg.kv_cache_plan(none.view(0, 3), none, none, pool, 16, 7)
    assert slots.tolist() == [-1] * 7 and positions.tolist() == [0] * 7 and lens.shape == (0,) and state.tolist() == [0, 5]
    slots = dg.kv_cache_plan(none.view(0, 3), none, none, pool, 16, 7, padded=True)[0]
    assert slots.shape == (0, 7)


def test_many_steps_lose_no_page():
    """A batch that grows, loses drafts, ends and starts again over many steps: every page is held
    once or free once, and the ring goes round."""
    announce("plan: many steps")
    rng = np.random.default_rng(6)
    B, page, P, width = 9, 16, 60, 12
    table = np.full((B, width), -1, np.int32)
    ring, state, ctx = rng.permutation(P).astype(np.int32), np.array([17, P], np.int32), np.zeros(B, np.int32)
    rounds = 0
    for step in range(60):
        add = rng.integers(-20, 40, B).astype(np.int32)
        done = rng.random(B) < 0.15
        add[done] = -ctx[done]
        t, r, s, lens = check(table, ctx, add, ring, state, page, 300, False)
        table, ring, ctx = (x.cpu().numpy() for x in (t, r, lens))
        rounds += int(s[0]) < state[0]
        state = s.cpu().numpy()
        held = [p for b in range(B) for p in table[b, :-(-int(ctx[b]) // page)]]
        free = ring[(state[0] + np.arange(state[1])) % P].tolist()
        assert sorted(held + free) == list(range(P))
    assert rounds >= 1


def test_given_outputs_other_stream_and_a_graph():
    announce("plan: out=, stream, graph")
    rng = np.random.default_rng(7)
    B, page, rows = 40, 16, 300
    ctx, add = lengths(rng, B, page, 100, 12)
    table, ring, state = paged.random_pool(rng, B, page, ctx, 80)
    t, r, s, c, a = dev(table), dev(ring), dev(state), dev(ctx), dev(add)
    out = tuple(torch.full(n, 9, dtype=torch.int32, device="cuda") for n in ((rows,), (rows,), (B,), (2,)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dg.kv_cache_plan(t, c, a, (r, s), page, rows, out=out)
    torch.cuda.current_stream().wait_stream(side)
    want = paged.plan(table, ctx, add, ring, state, page, rows, False)
    np.testing.assert_array_equal(out[0].cpu().numpy(), want[1])
    with torch.cuda.graph(graph):
        got = dg.kv_cache_plan(t, c, a, (r, s), page, rows, out=out)
        # what a decode loop does at the end of its step
        c.copy_(out[2]), s.copy_(out[3])
    assert got[0] is out[0] and got[3] is out[3]
    t.copy_(dev(table)), r.copy_(dev(ring))
    for step in range(4):
        want = paged.plan(table, ctx, add, ring, state, page, rows, False)
        graph.replay()
        torch.cuda.synchronize()
        for x, ref in zip((t, out[0], out[1], out[2], r, out[3]), want):
            np.testing.assert_array_equal(x.cpu().numpy(), ref)
        table, ctx, ring, state = want[0], want[3], want[4], want[5]
        add = np.where(ctx > 50, -30, rng.integers(0, 8, B)).astype(np.int32)
        a.copy_(dev(add))


def test_slices_at_their_own_alignment():
    announce("plan: unaligned slices")
    rng = np.random.default_rng(8)
    ctx, add = lengths(rng, 6, 16, 60, 20)
    table, ring, state = paged.random_pool(rng, 6, 16, ctx, 40)
    want = paged.plan(table, ctx, add, ring, state, 16, 90, False)

    def shifted(x):
        longer = torch.zeros(x.size + 1, dtype=torch.int32, device="cuda")
        longer[1:] = dev(np.asarray(x, np.int32)).flatten()
        return longer[1:].view(x.shape)

    t, r, s, c, a = (shifted(x) for x in (table, ring, state, ctx, add))
    got = dg.kv_cache_plan(t, c, a, (r, s), 16, 90, out=tuple(shifted(np.zeros(n, np.int32)) for n in (90, 90, 6, 2)))
    for x, ref in zip((t, *got[:3], r, got[3]), want):
        np.testing.assert_array_equal(x.cpu().numpy(), ref)


def test_binding_rejects():
    announce("plan refusals")
    pages, state = dg.make_kv_page_pool(9)
    table = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    ctx, add = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    for bad, error, text in (((table, ctx.long(), add, (pages, state), 16, 8), TypeError, "context_lens must be int32"),
                             ((table, ctx[:2], add, (pages, state), 16, 8), ValueError, "must be"),
                             ((table.t().contiguous().t(), ctx, add, (pages, state), 16, 8), ValueError, "contiguous"),
                             ((table, ctx, add, (pages, state[:1]), 16, 8), ValueError, "state"),
                             ((table, ctx, add, (pages.view(3, 3), state), 16, 8), ValueError, "num_pages"),
                             ((table, ctx, add, (pages, state), 17, 8), dg.DGError, "page_size=17"),
                             ((table, ctx, add, (pages, state), 16, -1), ValueError, "rows=-1"),
                             ((table, ctx, table[0, :3], (pages, state), 16, 8), dg.DGError, "overlap"),
                             ((table, ctx.cpu(), add, (pages, state), 16, 8), ValueError, "device tensor")):
        with pytest.raises(error, match=text):
            dg.kv_cache_plan(*bad)
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (8, 8, 3, 2)]
    with pytest.raises(ValueError, match="out shapes"):
        dg.kv_cache_plan(table, ctx, add, (pages, state), 16, 9, out=out)
    with pytest.raises(dg.DGError, match="overlaps"):
        dg.kv_cache_plan(table, ctx, add, (pages, state), 16, 8, out=out[:2] + [ctx, out[3]])
    assert not table.any() and state.tolist() == [0, 9]
