"""GPU parity of the norms of queries and keys with the rotation, and of their gradients, against the
64-bit formulas of tests/paged.py within bounds that count each rounding."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import paged
from tests.parity import announce, dev, to64

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


def frequencies(R, base=10000.0):
    return (base ** (-np.arange(R // 2) * 2.0 / max(R, 1))).astype(np.float32)


def case(T, Hq, H, D, R, dtype, seed, far=5000, w_dtype=None, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    qkv = (rand(T, Hq + 2 * H, D) * size).to(TYPES[dtype])
    wt = TYPES[w_dtype or dtype]
    w = [(1 + 0.3 * rand(D)).to(wt) for _ in range(2)]
    rng = np.random.default_rng(seed)
    positions = dev(rng.integers(-far // 50, far, T).astype(np.int32))
    d = [rand(T, n, D).to(TYPES[dtype]) for n in (Hq, H)]
    return (qkv[:, :Hq], qkv[:, Hq:Hq + H]), w, positions, dev(frequencies(R)), d


def within(got, want, what):
    ref, bound = want
    off = np.abs(to64(got) - ref)
    assert np.isfinite(to64(got)).all() and (off <= bound).all(), f"{what}: {(off / bound).max()} of the bound"


def check_forward(x, w, positions, freq, dtype, eps=1e-6, interleaved=False, out=None):
    got = dg.qk_norm_rope(*x, *w, positions, freq, eps=eps, interleaved=interleaved, out=out)
    for t, y, v, name in zip(x, got, w, "qk"):
        assert y.shape == t.shape and y.dtype == t.dtype
        within(y, paged.norm_rope(to64(t), 1.0 if v is None else to64(v), positions.cpu().numpy(), freq.cpu().numpy(), eps,
                                  interleaved, dtype), name)
    return got


def check_backward(d, x, w, positions, freq, dtype, eps=1e-6, interleaved=False, **kw):
    got = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, eps=eps, interleaved=interleaved, **kw)
    for i in range(2):
        dx, dw = paged.norm_rope_backward(to64(d[i]), to64(x[i]), 1.0 if w[i] is None else to64(w[i]), positions.cpu().numpy(),
                                          freq.cpu().numpy(), eps, interleaved, dtype)
        within(got[i], dx, "dx of " + "qk"[i])
        if w[i] is None:
            assert got[2 + i] is None
        else:
            assert got[2 + i].dtype == torch.float32
            within(got[2 + i], dw, "dw of " + "qk"[i])
    return got


SIZES = [(1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (5, 32, 8, 128, 128), (3, 7, 1, 64, 16), (65, 3, 3, 128, 32), (33, 5, 2, 256, 256),
         (130, 1, 1, 128, 64), (17, 16, 1, 256, 64), (2, 129, 17, 64, 32), (257, 2, 1, 64, 48), (9, 4, 4, 128, 0), (40, 8, 2, 256, 240)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,H,D,R", SIZES)
def test_small(T, Hq, H, D, R, dtype, interleaved):
    announce(f"norm rope T={T} Hq={Hq} H={H} D={D} R={R} {dtype} {interleaved}")
    x, w, positions, freq, d = case(T, Hq, H, D, R, dtype, T + D)
    check_forward(x, w, positions, freq, dtype, interleaved=interleaved)
    check_backward(d, x, w, positions, freq, dtype, interleaved=interleaved)


@pytest.mark.parametrize("dtype,interleaved,T,Hq,H,D,R", [("bf16", False, 3001, 32, 8, 128, 128), ("f32", True, 1203, 16, 2, 64, 32),
                                                         ("bf16", True, 901, 24, 3, 256, 64), ("f32", False, 5001, 1, 1, 256, 256),
                                                         ("bf16", False, 40001, 1, 2, 64, 64)])
def test_many_rows(dtype, interleaved, T, Hq, H, D, R):
    """More rows than a step of all workgroups: several steps each, and several rows a lane."""
    announce(f"norm rope many T={T} Hq={Hq} H={H} D={D} R={R} {dtype} {interleaved}")
    x, w, positions, freq, d = case(T, Hq, H, D, R, dtype, T)
    check_forward(x, w, positions, freq, dtype, interleaved=interleaved)
    first = check_backward(d, x, w, positions, freq, dtype, interleaved=interleaved)
    again = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, interleaved=interleaved)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("w_dtype,none", [("f32", ()), ("bf16", (0,)), ("f32", (1,)), ("bf16", (0, 1))])
def test_weights_of_another_type_or_none(w_dtype, none):
    announce(f"norm rope weights {w_dtype} {none}")
    x, w, positions, freq, d = case(21, 6, 2, 128, 64, "bf16" if w_dtype == "f32" else "f32", 5, w_dtype=w_dtype)
    w = [None if i in none else v for i, v in enumerate(w)]
    dtype = "bf16" if w_dtype == "f32" else "f32"
    check_forward(x, w, positions, freq, dtype)
    check_backward(d, x, w, positions, freq, dtype)


def test_gradients_against_differences():
    """The sum of all outputs' products with fixed numbers, its slope by differences in 64 bits."""
    announce("norm rope gradients by differences")
    x, w, positions, freq, d = case(3, 2, 1, 64, 32, "f32", 9, far=50)
    for interleaved in (False, True):
        got = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, eps=1e-3, interleaved=interleaved)
        p, f = positions.cpu().numpy(), freq.cpu().numpy()
        rng = np.random.default_rng(1)
        for i in range(2):
            def loss(xx, ww):
                return float((paged.norm_rope(xx, ww, p, f, 1e-3, interleaved, "f32")[0] * to64(d[i])).sum())
            for _ in range(6):
                vx, vw, h = rng.standard_normal(x[i].shape), rng.standard_normal(64), 1e-5
                slope = (loss(to64(x[i]) + h * vx, to64(w[i])) - loss(to64(x[i]) - h * vx, to64(w[i]))) / (2 * h)
                assert abs(slope - (to64(got[i]) * vx).sum()) <= 1e-5 * np.abs(to64(got[i]) * vx).sum()
                slope = (loss(to64(x[i]), to64(w[i]) + h * vw) - loss(to64(x[i]), to64(w[i]) - h * vw)) / (2 * h)
                assert abs(slope - (to64(got[2 + i]) * vw).sum()) <= 1e-5 * np.abs(to64(got[2 + i]) * vw).sum()


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Angles of up to 2^31: fp32 products would be wrong by whole turns."""
    announce("norm rope far positions")
    x, w, _, freq, d = case(8, 4, 2, 128, 128, "f32", 11)
    positions = torch.tensor([0, 1, 100003, 1 << 20, (1 << 24) + 1, (1 << 30) + 7, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device="cuda")
    check_forward(x, w, positions, freq, "f32", interleaved=interleaved)
    check_backward(d, x, w, positions, freq, "f32", interleaved=interleaved)


def test_rotation_keeps_lengths_and_differences():
    """Without weights a row's length is that of its norm, and products of queries and keys go by the
    difference of their positions."""
    announce("norm rope closed forms")
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(1, 1, 128, generator=g, device="cuda").expand(40, 1, 128).contiguous()
    y = torch.randn(1, 1, 128, generator=g, device="cuda").expand(40, 1, 128).contiguous()
    at = torch.arange(40, dtype=torch.int32, device="cuda") * 7
    q, k = dg.qk_norm_rope(x, y, None, None, at, dev(frequencies(128)))
    np.testing.assert_allclose(q.double().square().mean(-1).sqrt().cpu().numpy(), 1.0, rtol=2e-6)
    s = (q[:, 0].double() @ k[:, 0].double().t()).cpu().numpy()
    for off in range(0, 40, 9):
        along = np.diagonal(s, off)
        np.testing.assert_allclose(along, along[0], atol=128 * 40 * 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_small_and_large_rows(dtype):
    """Zeros, rows far below eps, and rows whose squares pass fp32's largest number."""
    announce(f"norm rope small and large {dtype}")
    x, w, positions, freq, d = case(6, 3, 2, 128, 128, dtype, 13)
    x = [t.clone() for t in x]
    for t in x:
        t[0] = 0
        t[1] *= 1e-20
        t[2] *= 1e25
        t[3] = 3e38 * t[3].sign()
        t[4, 0, 5] = 3e38
    got = check_forward(x, w, positions, freq, dtype)
    assert not got[0][0].any()
    check_backward(d, x, w, positions, freq, dtype)


def test_rows_that_are_not_finite():
    """A NaN or an infinity stays in its row, and in the weight's gradient."""
    announce("norm rope NaN")
    x, w, positions, freq, d = case(4, 3, 2, 128, 64, "f32", 15)
    x = [t.clone() for t in x]
    clean = dg.qk_norm_rope(*x, *w, positions, freq) + dg.qk_norm_rope_backward(*d, *x, *w, positions, freq)[:2]
    x[0][1, 2, 7], x[1][2, 0, 100] = float("nan"), float("inf")
    got = dg.qk_norm_rope(*x, *w, positions, freq) + dg.qk_norm_rope_backward(*d, *x, *w, positions, freq)[:2]
    assert got[0][1, 2].isnan().all() and got[1][2, 0, 100].isnan() and got[2][1, 2].isnan().all()
    for i, (a, b) in enumerate(zip(clean, got)):
        keep = torch.ones(a.shape[:2], dtype=torch.bool)
        keep[(1, 2) if i % 2 == 0 else (2, 0)] = False
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_and_given_outputs(dtype):
    announce(f"norm rope in place {dtype}")
    T, Hq, H, D = 70, 6, 2, 128
    x, w, positions, freq, d = case(T, Hq, H, D, D, dtype, 17)
    want = dg.qk_norm_rope(*x, *w, positions, freq)
    dwant = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq)
    fused = torch.full((T, Hq + 2 * H + 1, D), 7.0, dtype=TYPES[dtype], device="cuda")
    q, k = fused[:, 1:1 + Hq], fused[:, 1 + Hq:1 + Hq + H]
    q.copy_(x[0]), k.copy_(x[1])
    # gradients into slices of one row, beside each other
    wide = torch.full_like(fused, 5.0)
    ws = torch.full((dg.make_qk_norm_rope_backward_workspace(q, k).numel(),), 0xFF, dtype=torch.uint8, device="cuda")
    out = (wide[:, :Hq], wide[:, Hq:Hq + H])
    for _ in range(2):
        got = dg.qk_norm_rope_backward(*d, q, k, *w, positions, freq, out=out, workspace=ws)
        assert got[0] is out[0] and all(torch.equal(a, b) for a, b in zip(got, dwant))
    assert (wide[:, Hq + H:] == 5).all()
    got = dg.qk_norm_rope(q, k, *w, positions, freq, out=(q, k))
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert (fused[:, 0] == 7).all() and (fused[:, 1 + Hq + H:] == 7).all()


def test_nothing_to_do():
    announce("norm rope empty")
    for T, Hq, H in ((0, 4, 2), (3, 0, 2), (3, 4, 0), (0, 0, 0)):
        x, w, positions, freq, d = case(T, Hq, H, 64, 32, "bf16", 19)
        check_forward(x, w, positions, freq, "bf16")
        got = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq)
        for i, n in enumerate((Hq, H)):
            assert got[i].shape == (T, n, 64) and (T * n > 0 or not got[2 + i].any())


def test_graph_and_other_stream():
    announce("norm rope graph")
    x, w, positions, freq, d = case(50, 8, 2, 128, 128, "bf16", 21)
    x = [t.clone() for t in x]
    ws = dg.make_qk_norm_rope_backward_workspace(*x)

    def both():
        return dg.qk_norm_rope(*x, *w, positions, freq) + dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(on_side, both()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for step in range(4):
        for t in x:
            t.copy_(torch.randn_like(t))
        positions.add_(100)
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(replayed, both()))


def test_offsets_past_32_bits():
    """Rows of a wide buffer whose last ones start past 2^32 bytes."""
    announce("norm rope past 2^32")
    T, wide = 1100, 1 << 22
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("too little memory")
    buffer = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    x, w, positions, freq, d = case(T, 3, 1, 128, 128, "bf16", 23)
    q, k = (buffer[:, at:at + t.shape[1] * 128].unflatten(1, (-1, 128)) for at, t in zip((64, wide - 128), x))
    q.copy_(x[0]), k.copy_(x[1])
    want, dwant = dg.qk_norm_rope(*x, *w, positions, freq), dg.qk_norm_rope_backward(*d, *x, *w, positions, freq)
    dgot = dg.qk_norm_rope_backward(*d, q, k, *w, positions, freq)
    dg.qk_norm_rope(q, k, *w, positions, freq, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and all(torch.equal(a, b) for a, b in zip(dgot, dwant))


def test_binding_rejects():
    announce("norm rope refusals")
    (q, k), w, positions, freq, d = case(4, 4, 2, 64, 32, "bf16", 25)
    for bad, error, text in (((q, k.float(), *w, positions, freq), TypeError, "all be bfloat16"),
                             ((q.half(), k.half(), *w, positions, freq), TypeError, "all be bfloat16"),
                             ((q, k[:3], *w, positions, freq), ValueError, "shape mismatch"),
                             ((q, k[..., ::2], *w, positions, freq), ValueError, "shape mismatch"),
                             ((q[:, ::2], k, *w, positions, freq), ValueError, "dense"),
                             ((q, k, w[0][:32], w[1], positions, freq), ValueError, "q_weight"),
                             ((q, k, w[0], w[1].float(), positions, freq), TypeError, "one type"),
                             ((q, k, *w, positions.long(), freq), TypeError, "positions must be int32"),
                             ((q, k, *w, positions[:3], freq), ValueError, "positions"),
                             ((q, k, *w, positions, freq.double()), TypeError, "inv_freq must be float32"),
                             ((q, k, *w, positions, freq[:5]), dg.DGError, "R=10"),
                             ((q, k, *w, positions, dev(frequencies(96))), dg.DGError, "R=96"),
                             ((q, k, *w, positions, freq, 0.0), dg.DGError, "eps"),
                             ((q, k, *w, positions, freq, float("nan")), dg.DGError, "eps"),
                             ((q, k, *w, positions.cpu(), freq), ValueError, "device tensor"),
                             ((q.cpu(), k.cpu(), *w, positions, freq), ValueError, "device tensor")):
        with pytest.raises(error, match=text):
            dg.qk_norm_rope(*bad)
        with pytest.raises(error, match=text):
            dg.qk_norm_rope_backward(torch.zeros_like(bad[0]), torch.zeros_like(bad[0][:, :2]), *bad)
    y = dg.qk_norm_rope(q, k, *w, positions, freq)
    with pytest.raises(dg.DGError, match="overlap"):
        dg.qk_norm_rope(q, k, *w, positions, freq, out=(y[0], y[0][:, 1:3]))
    with pytest.raises(dg.DGError, match="overlaps an input"):
        dg.qk_norm_rope(q, k, *w, positions, freq, out=(y[0], q[:, 1:3]))      # keys over queries
    with pytest.raises(dg.DGError, match="overlap"):
        dg.qk_norm_rope_backward(*d, q, k, *w, positions, freq, out=(d[0], y[1]))
    with pytest.raises(dg.DGError, match="needed"):
        dg.qk_norm_rope_backward(*d, q, k, *w, positions, freq, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape mismatch"):
        dg.qk_norm_rope(q, k, *w, positions, freq, out=(y[1], y[1]))
