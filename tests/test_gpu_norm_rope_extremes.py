"""The norms with rotation and their gradients at weights and rows far from 1, and where a value is
infinite: what the formula does not mix stays apart."""
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests.parity import announce
from tests.test_gpu_norm_rope import case, check_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 32), (128, 48), (256, 64), (128, 128)])
def test_infinite_weights_stay_in_their_place(D, R, dtype, interleaved):
    """Values from R on are the norm times the weight: infinite with their weight, whatever stands beside them."""
    announce(f"norm rope infinite weights D={D} R={R} {dtype} {interleaved}")
    x, w, positions, freq, _ = case(37, 3, 2, D, R, dtype, D + R)
    clean = dg.qk_norm_rope(*x, *w, positions, freq, interleaved=interleaved)
    w = [v.clone() for v in w]
    hit = [d for d in (R, R + 5, D - 2) if R <= d < D]
    for v in w:
        v[hit] = float("inf")
    got = dg.qk_norm_rope(*x, *w, positions, freq, interleaved=interleaved)
    keep = torch.ones(D, dtype=torch.bool)
    keep[hit] = False
    for t, y, z in zip(x, got, clean):
        assert torch.equal(y[..., keep], z[..., keep])
        if hit:
            assert torch.equal(y[..., hit].float(), t[..., hit].float().sign() * float("inf"))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,R", [(64, 0), (64, 32), (256, 64)])
def test_infinite_gradients_stay_in_their_place(D, R, dtype, interleaved):
    """An infinite gradient of a value that is not turned: the sums of the other places' weights are as without
    it, its own is infinite; other rows are not touched."""
    announce(f"norm rope infinite gradients D={D} R={R} {dtype} {interleaved}")
    x, w, positions, freq, d = case(21, 3, 2, D, R, dtype, D + R)
    clean = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, interleaved=interleaved)
    d = [t.clone() for t in d]
    at = D - 2
    for t in d:
        t[4, 1, at] = float("inf")
    got = dg.qk_norm_rope_backward(*d, *x, *w, positions, freq, interleaved=interleaved)
    keep = torch.ones(D, dtype=torch.bool)
    keep[at] = False
    for i in range(2):
        assert torch.equal(got[2 + i][keep], clean[2 + i][keep])
        assert got[2 + i][at] == float("inf") * x[i][4, 1, at].float().sign()
        rows = torch.ones(x[i].shape[:2], dtype=torch.bool)
        rows[4, 1] = False
        assert torch.equal(got[i][rows], clean[i][rows])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [6, 3001])
@pytest.mark.parametrize("size,weight", [(1e37, 1e-6), (3e37, 1e-30), (1e-8, 1e34), (1.0, 1e36), (1.0, 1e-36)])
def test_weights_that_undo_the_norm(size, weight, T, interleaved):
    """Rows far from 1 and weights as far the other way or further: the norm is applied to the row first, and no
    product on the way leaves fp32's range where the result does not."""
    announce(f"norm rope size={size} weight={weight} T={T} {interleaved}")
    x, w, positions, freq, d = case(T, 3, 2, 64, 32, "f32", 31, size=size)
    w = [v * weight for v in w]
    check_forward(x, w, positions, freq, "f32", eps=2.0 ** -60, interleaved=interleaved)
