"""The few-token operators on the CPU: refusals of the C entry points and of the binding before
any HIP call, sizes of workspaces, the compiled kernels' registers, and the 64-bit references
against closed forms.
"""
import ctypes
import os

import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests.test_resource_gate import HIPCC, kernel_reports

A = [ctypes.c_void_p(0x10000000 * (i + 1)) for i in range(14)]    # far apart, never dereferenced
BAD = ctypes.c_void_p(0x10002)
BIG = 1 << 40
INVALID = dg.DG_ERR_INVALID_ARG
NO_DEVICE = (dg.DG_ERR_HIP, dg.DG_ERR_UNSUPPORTED, dg.DG_OK)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return dg.load_library()


def err(lib):
    return lib.dg_last_error().decode()


# ---- refusals through the C ABI ----------------------------------------------------------------

def write(lib, k=A[0], v=A[1], dt=dg.DG_BF16, ks=1024, vs=1024, slots=A[2], kc=A[3], kf=A[4], vc=A[5], vf=A[6],
          T=16, H=8, D=128, P=10, page=64):
    return lib.dg_fp8_kv_cache_write(k, v, dt, ks, vs, slots, kc, kf, vc, vf, T, H, D, P, page, None)


def read(lib, kc=A[3], kf=A[4], vc=A[5], vf=A[6], slots=A[2], k=A[0], v=A[1], dt=dg.DG_BF16, T=16, H=8, D=128, P=10,
         page=64):
    return lib.dg_fp8_kv_cache_read(kc, kf, vc, vf, slots, k, v, dt, T, H, D, P, page, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(D=96), "D=96"), (dict(page=17), "page_size=17"), (dict(page=8), "page_size=8"), (dict(page=8192), "page_size"),
    (dict(T=-1), "negative"), (dict(H=-1), "negative"), (dict(P=-1), "negative"), (dict(P=0), "num_pages=0"),
    (dict(P=1 << 26), "2^31"), (dict(dt=3), "dtype"), (dict(ks=1016), "k_stride"), (dict(vs=1028), "16 bytes"),
    (dict(k=None), "k is NULL"), (dict(v=BAD), "v is not 16-byte"), (dict(slots=None), "slots is NULL"),
    (dict(kc=None), "k_codes is NULL"), (dict(vf=BAD), "v_sf is not"), (dict(v=A[3]), "overlap"),
    (dict(vc=A[3]), "overlap"), (dict(kf=A[3]), "overlap"), (dict(T=BIG), "too large"),
    (dict(T=1 << 30), "2^31"), (dict(H=1 << 20), "H="),
])
def test_write_rejects(lib, kw, needle):
    assert write(lib, **kw) == INVALID
    assert needle in err(lib)


@pytest.mark.parametrize("kw,needle", [
    (dict(D=32), "D=32"), (dict(page=100), "page_size=100"), (dict(T=-1), "negative"), (dict(P=0), "num_pages=0"),
    (dict(dt=0), "dtype"), (dict(k=None), "k is NULL"), (dict(k=A[1]), "overlap"), (dict(v=A[5]), "overlap"),
    (dict(slots=BAD), "slots is not"), (dict(H=BIG), "H="),
])
def test_read_rejects(lib, kw, needle):
    assert read(lib, **kw) == INVALID
    assert needle in err(lib)


def test_cache_calls_without_work_or_device(lib):
    assert write(lib, T=0, k=None) == dg.DG_OK and write(lib, H=0, ks=0, vs=0, k=None) == dg.DG_OK
    assert read(lib, T=0, k=None) == dg.DG_OK and err(lib) == ""
    assert write(lib) in NO_DEVICE and read(lib) in NO_DEVICE


def attn(lib, q=A[0], qs=4096, kc=A[1], kf=A[2], vc=A[3], vf=A[4], table=A[5], ctx=A[6], tree=A[7], mask=A[8],
         o=A[9], lse=A[10], scale=0.1, B=4, N=3, Hq=32, H=8, D=128, P=50, page=64, MP=20, ws=A[11], ws_bytes=1 << 27):
    return lib.dg_fp8_tree_attention(q, qs, kc, kf, vc, vf, table, ctx, tree, mask, o, lse, scale, B, N, Hq, H, D, P,
                                     page, MP, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(B=-1), "B, N, Hq"), (dict(H=0), "H >= 1"), (dict(MP=0), "max_pages >= 1"), (dict(D=100), "D must be"),
    (dict(page=48), "page_size"), (dict(Hq=33), "multiple of H"), (dict(MP=1 << 25), "2^30"),
    (dict(N=1 << 20), "2^20"), (dict(N=1 << 15, Hq=32), "2^20"), (dict(B=1 << 18), "2^20"), (dict(P=0), "num_pages=0"),
    (dict(P=1 << 30), "num_pages"), (dict(qs=4088), "q_stride=4088"), (dict(qs=4100), "multiple of 8"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(q=None), "q is NULL"),
    (dict(table=None), "page_table is NULL"), (dict(ctx=BAD), "context_lens is not"), (dict(tree=BAD), "tree_lens is not"),
    (dict(mask=BAD), "tree_mask is not"), (dict(o=None), "o is NULL"), (dict(lse=BAD), "lse is not"),
    (dict(ws_bytes=16), "needed"), (dict(ws=None), "workspace is NULL"), (dict(o=A[0]), "overlap"),
    (dict(lse=A[9]), "overlap"), (dict(o=A[3]), "overlaps the cache"), (dict(ws=A[5]), "overlap"),
])
def test_attention_rejects(lib, kw, needle):
    assert attn(lib, **kw) == INVALID
    assert needle in err(lib)


def test_attention_without_work_or_device(lib):
    assert attn(lib, B=0, q=None) == dg.DG_OK and attn(lib, N=0, q=None) == dg.DG_OK
    assert attn(lib) in NO_DEVICE and attn(lib, tree=None, mask=None) in NO_DEVICE


def test_attention_workspace_is_a_function_of_the_sizes(lib):
    f = lib.dg_fp8_tree_attention_workspace_bytes
    assert f(32, 1, 32, 8, 128, 64, 128) > 0
    assert f(0, 1, 32, 8, 128, 64, 128) == 0 and f(32, 1, 33, 8, 128, 64, 128) == 0 and f(32, 1, 32, 8, 96, 64, 128) == 0
    assert f(1, 1, 8, 8, 128, 16, 1) == 0             # one step a head: never split
    assert all(f(B, N, 64, 8, D, 64, 200) <= 1 << 28 for B in (1, 7, 64, 500) for N in (1, 16, 64, 200) for D in (64, 128, 256))


def moe(lib, x=A[0], w1=A[1], s1=A[2], w2=A[3], s2=A[4], ids=A[5], wt=A[6], y=A[7], dt=dg.DG_BF16, T=4, k=2, E=8, H=1024,
        I=512, ws=A[8], ws_bytes=1 << 27):
    return lib.dg_fp8_moe_few_tokens(x, w1, s1, w2, s2, ids, wt, y, dt, T, k, E, H, I, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,needle", [
    (dict(T=-1), "T must be"), (dict(T=257), "T must be"), (dict(k=0), "topk"), (dict(k=17), "topk"), (dict(E=0), "E must"),
    (dict(E=1025), "E must"), (dict(H=100), "H must"), (dict(H=0), "H must"), (dict(I=192), "I must"), (dict(I=BIG), "I must"),
    (dict(H=1 << 18), "H must"), (dict(dt=5), "y_dtype"), (dict(x=None), "x is NULL"), (dict(w1=BAD), "w1 is not"),
    (dict(s2=None), "s2 is NULL"), (dict(ids=BAD), "topk_ids is not"), (dict(wt=None), "topk_weights is NULL"),
    (dict(y=None), "y is NULL"), (dict(ws=None), "workspace is NULL"), (dict(ws=BAD), "workspace is not"),
    (dict(ws_bytes=64), "needed"), (dict(y=A[0]), "overlap"), (dict(ws=A[3]), "overlap"), (dict(ws=A[7]), "overlap"),
])
def test_moe_rejects(lib, kw, needle):
    assert moe(lib, **kw) == INVALID
    assert needle in err(lib)


def test_moe_without_work_or_device(lib):
    assert moe(lib, T=0, x=None, ws=None) == dg.DG_OK
    assert moe(lib) in NO_DEVICE
    f = lib.dg_fp8_moe_few_tokens_workspace_bytes
    assert f(0, 2, 8, 1024, 512) == 0 and f(4, 2, 8, 1000, 512) == 0 and f(4, 2, 8, 1024, 512) > 0


# ---- refusals of the binding --------------------------------------------------------------------

def host_cache(pages=4, H=2, page=16, D=64):
    return tuple((torch.zeros(pages, H, page, D, dtype=torch.uint8), torch.ones(pages, H, page)) for _ in range(2))


def test_binding_rejects_host_tensors():
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        dg.fp8_kv_cache_write(k, k, host_cache(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        dg.fp8_kv_cache_read(host_cache(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensor"):
        dg.fp8_tree_attention(torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16), host_cache(),
                              torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    w1 = (torch.zeros(2, 256, 128, dtype=torch.uint8), torch.ones(2, 2, 1))
    w2 = (torch.zeros(2, 128, 128, dtype=torch.uint8), torch.ones(2, 1, 1))
    with pytest.raises(ValueError, match="device tensor"):
        dg.fp8_moe_few_tokens(torch.zeros(1, 128, dtype=torch.bfloat16), w1, w2, torch.zeros(1, 1, dtype=torch.int32),
                              torch.ones(1, 1))


# ---- the compiled kernels ---------------------------------------------------------------------------

@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
@pytest.mark.parametrize("src,least", [("kv_cache_kernel.hip", 12), ("tree_attn_kernel.hip", 11), ("moe_few_kernel.hip", 12)])
def test_no_vgpr_spill_no_scratch(src, least):
    reports = kernel_reports(src)
    assert len(reports) >= least, sorted(reports)
    bad = [f"{n}: {r}" for n, r in reports.items() if int(r["VGPRs Spill"]) or int(r["ScratchSize [bytes/lane]"])
           or r["Dynamic Stack"] != "False"]
    assert not bad, "\n".join(bad)


# ---- the references against closed forms ---------------------------------------------------------------

def test_reference_codes_are_e4m3():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ft.e4m3(codes), want)


def test_reference_rows():
    x = np.array([[1.0, -2.0, 448.0, 0.0], [0, 0, 0, 0], [1, np.nan, 2, 3], [np.inf, 1, 2, 3]], np.float32)
    codes, s = ft.quantise_rows(x)
    np.testing.assert_array_equal(s[:2], [1, 1])
    assert np.isnan(s[2:]).all() and not codes[2:].any() and not codes[1].any()
    np.testing.assert_array_equal(ft.e4m3(codes[0]), [1, -2, 448, 0])


def test_reference_attention_closed_forms():
    """Equal keys average what is seen; a dominant key takes all; nothing seen gives 0 and -inf."""
    rng = np.random.default_rng(0)
    D, page = 64, 16
    vcodes, vs = ft.quantise_rows(rng.standard_normal((2, 1, page, D)).astype(np.float32))
    cache = [(np.zeros((2, 1, page, D), np.uint8), np.ones((2, 1, page), np.float32)), (vcodes, vs)]
    table = np.array([[1, 0]], np.int32)
    q = rng.standard_normal((1, 2, 1, D))
    mask = np.array([[[True, False], [False, False]]])
    o, lse, _, _ = ft.attention(q, cache, table, [5], [2], mask, 0.3, page)
    vals = ft.e4m3(vcodes[1, 0]) * vs[1, 0].astype(np.float64)[:, None]
    np.testing.assert_allclose(o[0, 0, 0], vals[:6].mean(0), rtol=1e-12)
    np.testing.assert_allclose(o[0, 1, 0], vals[:5].mean(0), rtol=1e-12)
    np.testing.assert_allclose(lse[0, :, 0], np.log([6, 5]), rtol=1e-12)
    o, lse, _, _ = ft.attention(q, cache, table, [0], [2], mask, 0.3, page)
    assert not o[0, 1].any() and np.isneginf(lse[0, 1]).all()
    cache[0][0][1, 0, 3] = 0x7E                     # key 3: 448 everywhere
    o, _, _, _ = ft.attention(np.abs(q), cache, table, [5], [2], mask, 1.0, page)
    np.testing.assert_allclose(o[0, 1, 0], vals[3], rtol=1e-9)


def test_reference_masks():
    rng = np.random.default_rng(1)
    m = np.stack([ft.random_tree(rng, 70) for _ in range(2)])
    w = ft.pack_mask(m)
    assert w.shape == (2, 70, 2) and w.dtype == np.int64
    for i, j in ((0, 0), (69, 69), (63, 63), (64, 3), (66, 65)):
        assert bool((int(w[1, i, j // 64]) >> (j % 64)) & 1) == bool(m[1, i, j])


def test_reference_moe_against_torch():
    rng = np.random.default_rng(2)
    T, E, k, H, I = 3, 4, 2, 128, 128
    w1, s1 = ft.quantise_blocks(rng.standard_normal((E, 2 * I, H)).astype(np.float32))
    w2, s2 = ft.quantise_blocks(rng.standard_normal((E, H, I)).astype(np.float32))
    x = rng.standard_normal((T, H))
    ids = np.array([[0, 1], [3, -1], [2, 2]], np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    y, bound = ft.moe(x, w1, s1, w2, s2, ids, wt, 3)
    for t in range(T):
        want = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            a1 = torch.from_numpy(w1[e]).view(torch.float8_e4m3fn).double() * torch.from_numpy(s1[e]).double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            a2 = torch.from_numpy(w2[e]).view(torch.float8_e4m3fn).double() * torch.from_numpy(s2[e]).double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            z = a1 @ torch.from_numpy(x[t])
            want += float(wt[t, j]) * (a2 @ (torch.nn.functional.silu(z[:I]) * z[I:]))
        np.testing.assert_allclose(y[t], want.numpy(), rtol=1e-10, atol=1e-12 * float(want.abs().max()))
    assert (bound >= 0).all() and bound.max() < 0.05 * np.abs(y).max()
