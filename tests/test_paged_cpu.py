"""The operators around a paged cache on the CPU: refusals of the C entry points before any HIP call,
sizes of workspaces, the compiled kernels' registers, and the references against closed forms.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import paged
from tests.test_resource_gate import HIPCC, kernel_reports

A = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(16)]    # far apart, never dereferenced
BAD = ctypes.c_void_p(0x10002)
BIG = 1 << 40
INVALID = dg.DG_ERR_INVALID_ARG
NO_DEVICE = (dg.DG_ERR_HIP, dg.DG_ERR_UNSUPPORTED)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dg.load_library()


def err(lib):
    return lib.dg_last_error().decode()


# ---- the plan ----------------------------------------------------------------------------------

def plan(lib, table=A[0], ctx=A[1], add=A[2], ring=A[3], state=A[4], slots=A[5], positions=A[6], lens=A[7], new_state=A[8],
         B=4, rows=100, padded=0, MP=20, P=50, page=64):
    return lib.dg_kv_cache_plan(table, ctx, add, ring, state, slots, positions, lens, new_state, B, rows, padded, MP, P,
                                page, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(B=-1), "negative"), (dict(rows=-1), "negative"), (dict(padded=2), "padded"), (dict(page=17), "page_size=17"),
    (dict(P=0), "num_pages=0"), (dict(P=1 << 26), "2^31"), (dict(MP=0), "max_pages=0"), (dict(MP=1 << 25), "2^30"),
    (dict(B=65537), "B=65537"), (dict(rows=BIG), "rows"), (dict(rows=1 << 30, padded=1), "rows"),
    (dict(table=None), "page_table is NULL"), (dict(ctx=BAD), "context_lens is not"), (dict(add=None), "add_lens is NULL"),
    (dict(ring=None), "pool_pages is NULL"), (dict(state=BAD), "pool_state is not"), (dict(slots=None), "slots is NULL"),
    (dict(positions=BAD), "positions is not"), (dict(lens=None), "new_lens is NULL"), (dict(new_state=None), "new_state is NULL"),
    (dict(lens=A[1]), "overlap"), (dict(new_state=A[4]), "overlap"), (dict(slots=A[6]), "overlap"), (dict(ring=A[0]), "overlap"),
    (dict(add=A[0]), "overlap"), (dict(slots=ctypes.c_void_p(0x10000000 + 4 * 79)), "overlap"),
])
def test_plan_rejects(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert plan(lib, **kw) == INVALID
    assert needle in err(lib)


def test_plan_without_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert plan(lib) in NO_DEVICE and plan(lib, ctx=A[2]) in NO_DEVICE         # inputs may be the same
    assert plan(lib, B=0, table=None, ctx=None, add=None, lens=None) in NO_DEVICE
    assert plan(lib, rows=0, slots=None, positions=None) in NO_DEVICE
    assert plan(lib, slots=ctypes.c_void_p(0x10000000 + 4 * 80)) in NO_DEVICE  # right behind the table


def test_reference_plan():
    """Two requests take one page each, one gives one back; the ring goes round its end."""
    table = [[3, -1], [0, 1], [-1, -1]]
    t, slots, positions, lens, ring, state = paged.plan(table, [16, 20, 0], [1, -5, 2], [9, 7, 5, 4, 8], [4, 3], 16, 4, False)
    assert t.tolist() == [[3, 8], [0, 1], [9, -1]]
    assert slots.tolist() == [-1, -1, -1, -1]             # pages 8 and 9 of a cache of five
    assert positions.tolist() == [16, 0, 1, 0] and lens.tolist() == [17, 15, 2]
    assert ring.tolist() == [9, 7, 1, 4, 8] and state.tolist() == [1, 2]


# ---- norms with rotation -------------------------------------------------------------------------

def rope(lib, q=A[0], k=A[1], dt=dg.DG_BF16, qs=4096, ks=1024, wq=A[2], wk=A[3], wdt=dg.DG_BF16, positions=A[4], freq=A[5],
         qo=A[6], ko=A[7], qos=4096, kos=1024, eps=1e-6, pairs=0, T=10, Hq=32, H=8, D=128, R=128):
    return lib.dg_qk_norm_rope(q, k, dt, qs, ks, wq, wk, wdt, positions, freq, qo, ko, qos, kos, eps, pairs, T, Hq, H, D, R, None)


def rope_grad(lib, dq=A[8], dk=A[9], q=A[0], k=A[1], dt=dg.DG_BF16, dqs=4096, dks=1024, qs=4096, ks=1024, wq=A[2], wk=A[3],
              wdt=dg.DG_BF16, positions=A[4], freq=A[5], qo=A[6], ko=A[7], qos=4096, kos=1024, dwq=A[10], dwk=A[11], eps=1e-6,
              pairs=0, T=10, Hq=32, H=8, D=128, R=128, ws=A[12], ws_bytes=1 << 22):
    return lib.dg_qk_norm_rope_backward(dq, dk, q, k, dt, dqs, dks, qs, ks, wq, wk, wdt, positions, freq, qo, ko, qos, kos, dwq, dwk,
                                        eps, pairs, T, Hq, H, D, R, ws, ws_bytes, None)


ROPE_WRONG = [
    (dict(T=-1), "negative"), (dict(H=-1), "negative"), (dict(D=96), "D must be"), (dict(Hq=1 << 17), "65535"),
    (dict(T=1 << 28), "2^31"), (dict(T=BIG), "2^31"), (dict(R=24), "R=24"), (dict(R=144), "R=144"), (dict(R=-16), "R=-16"),
    (dict(dt=0), "dtype"), (dict(wdt=7), "w_dtype"), (dict(pairs=2), "interleaved"), (dict(eps=0.0), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(qs=4088), "q_stride"), (dict(ks=1028), "k_stride"), (dict(qos=4095), "q"),
    (dict(kos=1 << 32), "k"), (dict(q=None), "q is NULL"), (dict(k=BAD), "k is not 16-byte"), (dict(wq=BAD), "q_weight is not"),
    (dict(positions=None), "positions is NULL"), (dict(freq=BAD), "inv_freq is not"), (dict(ko=None), "NULL"), (dict(qo=BAD), "16-byte"),
    (dict(qo=A[1]), "overlaps an input"), (dict(ko=A[6]), "overlap"), (dict(ko=A[3]), "overlaps an input"),
]


@pytest.mark.parametrize("kw,needle", ROPE_WRONG + [(dict(qo=A[0], qos=4104), "overlaps an input")])
def test_rope_rejects(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert rope(lib, **kw) == INVALID
    assert needle in err(lib)


@pytest.mark.parametrize("kw,needle", ROPE_WRONG + [
    (dict(dqs=4088), "dq_stride"), (dict(dk=None), "dk is NULL"), (dict(qo=A[0]), "overlaps an input"), (dict(qo=A[8]), "overlaps an input"),
    (dict(dwq=BAD), "dq_weight is not"), (dict(dwk=A[2]), "overlaps an input"), (dict(dwk=A[10]), "overlap"), (dict(ws=None), "workspace is NULL"),
    (dict(ws_bytes=64), "needed"), (dict(ws=A[6]), "overlap"),
])
def test_rope_gradients_reject(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert rope_grad(lib, **kw) == INVALID
    assert needle in err(lib)


def test_rope_without_work_or_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert rope(lib, T=0, q=None, positions=None) == dg.DG_OK and rope(lib, Hq=0, H=0, q=None, k=None) == dg.DG_OK
    assert rope(lib) in NO_DEVICE and rope(lib, qo=A[0], ko=A[1]) in NO_DEVICE and rope(lib, wq=None, wk=None, R=0, freq=None) in NO_DEVICE
    # slices of one row, in place and beside each other
    q, k = ctypes.c_void_p(0x10000000), ctypes.c_void_p(0x10000000 + 8192)
    side = dict(q=q, k=k, qs=6144, ks=6144)
    assert rope(lib, **side, qo=q, ko=k, qos=6144, kos=6144) in NO_DEVICE
    assert rope(lib, **side, qo=k, ko=q, qos=6144, kos=6144) == INVALID
    # queries and keys that are one tensor: neither may be written over while the other is read
    one = dict(q=q, k=q, qs=1024, ks=1024, Hq=8, qos=1024, kos=1024)
    assert rope(lib, **one) in NO_DEVICE
    assert rope(lib, **one, qo=q) == INVALID and rope(lib, **one, ko=q) == INVALID
    assert rope_grad(lib) in NO_DEVICE and rope_grad(lib, dwq=None, dwk=None, ws=None, ws_bytes=0) in NO_DEVICE
    assert rope_grad(lib, T=0, dwq=None, dwk=None) == dg.DG_OK and rope_grad(lib, T=0, ws=None) in NO_DEVICE
    f = lib.dg_qk_norm_rope_backward_workspace_bytes
    assert f(-1, 32, 8, 128) == 0 and f(10, 32, 8, 96) == 0 and f(0, 32, 8, 128) == 0
    assert all(0 < f(T, 32, 8, D) <= 1100 * D * 4 for T in (1, 333, 16384, 1 << 25) for D in (64, 128, 256))


def test_reference_norm_rope():
    """A quarter turn swaps a pair; the gradient is orthogonal to the row where eps is nothing."""
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 16] = 3, 4
    f = np.zeros(16, np.float32)
    f[0] = np.float32(np.pi / 2)
    z, _ = paged.norm_rope(x, 1.0, [1], f, 0.0, False, "f32")
    np.testing.assert_allclose(z[0, 0, [0, 16]], np.array([-4, 3]) * 8 / 5, atol=1e-6)
    rng = np.random.default_rng(0)
    x, dz, w = rng.standard_normal((5, 2, 64)), rng.standard_normal((5, 2, 64)), rng.standard_normal(64)
    for interleaved in (False, True):
        (dx, _), (dw, _) = paged.norm_rope_backward(dz, x, w, np.arange(5), f, 1e-30, interleaved, "f32")
        np.testing.assert_allclose((dx * x).sum(-1), 0, atol=1e-12)
        a = torch.tensor(x, requires_grad=True)
        b = torch.tensor(w, requires_grad=True)
        y = a * torch.rsqrt(a.square().mean(-1, keepdim=True)) * b
        t = torch.arange(5).double()[:, None] * torch.tensor(f).double()
        c, s = t.cos()[:, None], t.sin()[:, None]
        p, q = (y[..., 0:32:2], y[..., 1:32:2]) if interleaved else (y[..., :16], y[..., 16:32])
        u, v = p * c - q * s, p * s + q * c
        turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
        (torch.cat([turned, y[..., 32:]], -1) * torch.tensor(dz)).sum().backward()
        np.testing.assert_allclose(dx, a.grad.numpy(), atol=1e-12)
        np.testing.assert_allclose(dw, b.grad.numpy(), atol=1e-12)


# ---- the FP4 cache -------------------------------------------------------------------------------

def write4(lib, k=A[0], v=A[1], dt=dg.DG_BF16, ks=1024, vs=1024, slots=A[2], kc=A[3], kf=A[4], vc=A[5], vf=A[6],
           T=16, H=8, D=128, P=10, page=64):
    return lib.dg_fp4_kv_cache_write(k, v, dt, ks, vs, slots, kc, kf, vc, vf, T, H, D, P, page, None)


def read4(lib, kc=A[3], kf=A[4], vc=A[5], vf=A[6], slots=A[2], k=A[0], v=A[1], dt=dg.DG_BF16, T=16, H=8, D=128, P=10, page=64):
    return lib.dg_fp4_kv_cache_read(kc, kf, vc, vf, slots, k, v, dt, T, H, D, P, page, None)


def at(base, off):
    return ctypes.c_void_p(base.value + off)


CODES, SCALES = 10 * 8 * 64 * 64, 10 * 8 * 64 * 4        # bytes of the caches above


@pytest.mark.parametrize("kw,needle", [
    (dict(D=96), "D=96"), (dict(page=17), "page_size=17"), (dict(T=-1), "negative"), (dict(P=0), "num_pages=0"), (dict(P=1 << 26), "2^31"),
    (dict(dt=3), "dtype"), (dict(ks=1016), "k_stride"), (dict(vs=1028), "16 bytes"), (dict(k=None), "k is NULL"),
    (dict(v=BAD), "v is not 16-byte"), (dict(kf=BAD), "k_sf is not"), (dict(vc=A[3]), "overlap"), (dict(kf=at(A[3], CODES - 16)), "overlap"),
    (dict(vf=at(A[4], SCALES - 16)), "overlap"), (dict(k=at(A[5], CODES - 16)), "overlap"), (dict(slots=at(A[6], SCALES - 16)), "overlap"),
    (dict(T=BIG), "too large"), (dict(H=1 << 20), "H="),
])
def test_fp4_write_rejects(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert write4(lib, **kw) == INVALID
    assert needle in err(lib)


@pytest.mark.parametrize("kw,needle", [
    (dict(D=32), "D=32"), (dict(page=100), "page_size=100"), (dict(T=-1), "negative"), (dict(P=0), "num_pages=0"), (dict(dt=0), "dtype"),
    (dict(k=None), "k is NULL"), (dict(k=A[1]), "overlap"), (dict(v=at(A[3], CODES - 16)), "overlap"), (dict(slots=BAD), "slots is not"),
])
def test_fp4_read_rejects(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert read4(lib, **kw) == INVALID
    assert needle in err(lib)


def test_fp4_cache_without_work_or_device(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert write4(lib, T=0, k=None) == dg.DG_OK and read4(lib, T=0, k=None) == dg.DG_OK
    assert write4(lib) in NO_DEVICE and read4(lib) in NO_DEVICE
    # right behind one another, by the FP4 cache's sizes
    assert write4(lib, kf=at(A[3], CODES), vf=at(A[3], CODES + SCALES)) in NO_DEVICE


def attn4(lib, q=A[0], qs=4096, kc=A[1], kf=A[2], vc=A[3], vf=A[4], table=A[5], ctx=A[6], tree=A[7], mask=A[8],
          o=A[9], lse=A[10], scale=0.1, B=4, N=3, Hq=32, H=8, D=128, P=50, page=64, MP=40, ws=A[11], ws_bytes=1 << 27):
    return lib.dg_fp4_tree_attention(q, qs, kc, kf, vc, vf, table, ctx, tree, mask, o, lse, scale, B, N, Hq, H, D, P,
                                     page, MP, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(B=-1), "B, N, Hq"), (dict(H=0), "H >= 1"), (dict(MP=0), "max_pages >= 1"), (dict(D=100), "D must be"),
    (dict(page=48), "page_size"), (dict(Hq=33), "multiple of H"), (dict(MP=1 << 25), "2^30"), (dict(N=1 << 20), "2^20"),
    (dict(P=0), "num_pages=0"), (dict(qs=4088), "q_stride=4088"), (dict(scale=float("nan")), "scale"), (dict(q=None), "q is NULL"),
    (dict(kf=BAD), "k_sf is not"), (dict(table=None), "page_table is NULL"), (dict(mask=BAD), "tree_mask is not"), (dict(o=None), "o is NULL"),
    (dict(ws_bytes=16), "needed"), (dict(ws=None), "workspace is NULL"), (dict(o=A[0]), "overlap"),
    (dict(o=at(A[3], 50 * 8 * 64 * 64 - 16)), "overlaps the cache"), (dict(lse=at(A[4], 50 * 8 * 64 * 4 - 4)), "overlaps the cache"),
])
def test_fp4_attention_rejects(lib, kw, needle):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    assert attn4(lib, **kw) == INVALID
    assert needle in err(lib)


def test_fp4_attention_workspace_is_a_function_of_the_sizes(lib):
    f = lib.dg_fp4_tree_attention_workspace_bytes
    assert f(1, 1, 32, 8, 128, 64, 128) > 0 and f(32, 1, 32, 8, 128, 64, 400) > 0
    assert f(32, 1, 32, 8, 128, 64, 128) == 0         # 256 workgroups of whole requests: nothing to join
    assert f(0, 1, 32, 8, 128, 64, 128) == 0 and f(32, 1, 33, 8, 128, 64, 128) == 0 and f(32, 1, 32, 8, 96, 64, 128) == 0
    assert f(1, 1, 8, 8, 128, 16, 1) == 0             # one step a head: never split
    assert f(4, 3, 32, 8, 128, 64, 20) == 0 and f(4, 3, 32, 8, 128, 64, 40) > 0
    assert all(f(B, N, 64, 8, D, 64, 200) <= 1 << 28 for B in (1, 7, 64, 500) for N in (1, 16, 64, 200) for D in (64, 128, 256))
    if not torch.cuda.is_available():
        assert attn4(lib, B=0, q=None) == dg.DG_OK and attn4(lib) in NO_DEVICE and attn4(lib, tree=None, mask=None) in NO_DEVICE


def test_reference_fp4_rows():
    """Codes of a row of known values, the limit between two scales, and rows that are not finite."""
    x = np.zeros((4, 64))
    x[0, :9] = [6, -4, 3, 2, 1.5, 1, 0.5, 0.25, 0.26]
    x[1, :3] = [6.01, 0.5, -1.5]                       # scale 2: 0.25 and -0.75, ties
    x[2, 3], x[3, 40] = np.nan, np.inf
    codes, sf = paged.quantise4(x)
    v = paged.values4(codes, sf)
    np.testing.assert_array_equal(v[0, :9], [6, -4, 3, 2, 1.5, 1, 0.5, 0, 0.5])
    np.testing.assert_array_equal(v[1, :3], [6, 0, -2])
    assert codes[0, 0] == 7 | 14 << 4 and sf[0, 0] == 127 and sf[1, 0] == 128 and (sf[:2, 1] == 127).all()
    assert np.isnan(v[2, :32]).all() and not v[2, 32:].any() and np.isnan(v[3, 32:]).all() and sf[2, 0] == 255
    every = paged.values4(np.arange(256, dtype=np.uint8).reshape(4, 64), np.full((4, 4), 127))
    again, s = paged.quantise4(every)                  # every code is its own nearest
    np.testing.assert_array_equal(paged.values4(again, s), every)


def test_reference_attention4_closed_forms():
    """Equal keys average what is seen; nothing seen gives 0 and -inf; a NaN scale of a value stays in
    its 32 values."""
    rng = np.random.default_rng(0)
    D, page = 64, 16
    cache = paged.random_cache4(rng, 2, 1, page, D)
    cache[0][0][:] = 0
    cache[1][1][1, 0, 2, 1] = 255
    table = np.array([[1, 0]], np.int32)
    q = rng.standard_normal((1, 2, 1, D))
    mask = np.array([[[True, False], [False, False]]])
    o, lse, bo, _ = paged.attention4(q, cache, table, [5], [2], mask, 0.3, page)
    vals = paged.values4(cache[1][0][1, 0], cache[1][1][1, 0])
    np.testing.assert_allclose(o[0, 0, 0, :32], vals[:6, :32].mean(0), atol=1e-12)
    np.testing.assert_allclose(o[0, 1, 0, :32], vals[:5, :32].mean(0), atol=1e-12)
    np.testing.assert_allclose(lse[0, :, 0], np.log([6, 5]), rtol=1e-12)
    assert np.isnan(o[0, :, 0, 32:]).all() and np.isfinite(bo[0, :, 0, :32]).all()
    o, lse, _, _ = paged.attention4(q, cache, table, [0], [2], mask, 0.3, page)
    assert not o[0, 1].any() and np.isneginf(lse[0, 1]).all()


# ---- the compiled kernels --------------------------------------------------------------------------

@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src,least", [("plan_kernel.hip", 2), ("norm_rope_kernel.hip", 49), ("kv4_cache_kernel.hip", 12),
                                       ("tree_attn4_kernel.hip", 24)])
def test_no_vgpr_spill_no_scratch(src, least):
    reports = kernel_reports(src)
    assert len(reports) >= least, sorted(reports)
    bad = [f"{n}: {r}" for n, r in reports.items() if int(r["VGPRs Spill"]) or int(r["ScratchSize [bytes/lane]"])
           or r["Dynamic Stack"] != "False"]
    assert not bad, "\n".join(bad)
