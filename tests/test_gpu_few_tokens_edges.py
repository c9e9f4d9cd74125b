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
