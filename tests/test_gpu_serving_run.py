"""The operators around a paged cache in one run, as they are used: pages and slots, norms with the
rotation, the cache's write, attention over it; a step of a batch in a graph, and the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests import paged
from tests.parity import announce, dev, to64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


@pytest.mark.parametrize("bits", ["fp4", "fp8"])
@pytest.mark.parametrize("B,H,G,D,N,page", [(3, 2, 4, 128, 1, 16), (5, 1, 8, 64, 6, 32), (2, 2, 2, 256, 3, 16)])
def test_steps_of_a_batch(B, H, G, D, N, page, bits):
    """Several replays of a captured step against the request-by-request plan, the 64-bit rotation and
    attention over what the cache holds."""
    announce(f"run {bits} B={B} H={H} G={G} D={D} N={N}")
    rng = np.random.default_rng(B + D)
    make, write, attend = (getattr(dg, name) for name in (f"make_{bits}_kv_cache", f"{bits}_kv_cache_write", f"{bits}_tree_attention"))
    pages, width, steps = 40, 12, 5
    table, ctx = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    ring, state = rng.permutation(pages).astype(np.int32), np.array([7, pages], np.int32)
    t, c, r, s = dev(table), dev(ctx), dev(ring), dev(state)
    add = torch.zeros(B, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(B * N, H * G + 2 * H, D, dtype=torch.bfloat16, device="cuda")
    w = [(1 + 0.2 * torch.randn(D, device="cuda")).bfloat16() for _ in range(2)]
    freq = dev((10000.0 ** (-np.arange(D // 4) * 4.0 / D)).astype(np.float32))
    cache = make(pages, H, page, D)
    ws = getattr(dg, f"make_{bits}_tree_attention_workspace")(qkv[:, :H * G].unflatten(0, (B, N)), cache, t)

    def step():
        slots, positions, lens, pool = dg.kv_cache_plan(t, c, add, (r, s), page, N, padded=True)
        q, k = dg.qk_norm_rope(qkv[:, :H * G], qkv[:, H * G:H * G + H], *w, positions.view(-1), freq)
        write(k, qkv[:, H * G + H:], cache, slots.view(-1))
        o, lse = attend(q.unflatten(0, (B, N)), cache, t, c, lens - c, workspace=ws)
        return slots, positions, lens, pool, q, k, o, lse

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
        c.copy_(out[2]), s.copy_(out[3])
    for i in range(steps):
        change = rng.integers(0, N + 1, B).astype(np.int32)
        if i == 3:
            change[0] = -int(ctx[0])                       # the first request starts again
        add.copy_(dev(change))
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        want = paged.plan(table, ctx, change, ring, state, page, N, True)
        graph.replay()
        torch.cuda.synchronize()
        slots, positions, lens, pool, q, k, o, lse = out
        for got, ref in zip((t, slots, positions, lens, r, pool), want):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        for got, first, n, weight in ((q, 0, H * G, w[0]), (k, H * G, H, w[1])):
            ref, bound = paged.norm_rope(to64(qkv[:, first:first + n]), to64(weight), want[2].reshape(-1), freq.cpu().numpy(), 1e-6,
                                         False, "bf16")
            assert (np.abs(to64(got) - ref) <= bound).all()
        pool_of = [(codes.cpu().numpy(), sf.cpu().numpy()) for codes, sf in cache]
        reference = paged.attention4 if bits == "fp4" else ft.attention
        mask = np.stack([ft.chain(N)] * B)
        new = np.asarray(want[3] - ctx)
        ro, rl, bo, bl = reference(to64(q).reshape(B, N, H * G, D), pool_of, want[0].astype(np.int32), ctx, np.maximum(new, 0), mask,
                                   D ** -0.5, page)
        assert (np.abs(to64(o) - ro) <= bo).all()
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse.cpu().numpy()), empty)
        assert (np.abs(lse.cpu().numpy()[~empty] - rl[~empty]) <= bl[~empty]).all()
        table, ctx, ring, state = want[0].astype(np.int32), want[3].astype(np.int32), want[4].astype(np.int32), want[5].astype(np.int32)
    assert ctx.max() > 0


@pytest.mark.parametrize("argv", [[], ["--cache", "fp8", "--places", "3", "--requests", "5"],
                                  ["--places", "1", "--requests", "2", "--prompt", "1", "--answer", "1", "--layers", "1"]])
def test_example(argv):
    announce(f"serve_requests {argv}")
    spec = importlib.util.spec_from_file_location("serve_requests", os.path.join(ROOT, "examples", "serve_requests.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    answers, waits = example.main(argv)
    assert min(answers) >= 1 and (argv or waits > 0)
