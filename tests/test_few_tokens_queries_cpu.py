"""How the binding reads the query's strides, on host tensors that say they are on a device, with the
call replaced by a recorder: a query whose heads are not dense is refused whatever its sizes, since
the call has one stride only, from token to token.
"""
import os

import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnDevice)


@pytest.fixture
def attend(monkeypatch):
    """attend(q) -> (the recorded call's arguments, what the binding returned)."""
    if not os.path.exists(dg.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    calls = []
    monkeypatch.setattr(dg, "_call", lambda fn, device, *args: calls.append(args))

    def run(q, H=4, D=128):
        B = q.shape[0]
        cache = tuple((on(torch.zeros(8, H, 16, D, dtype=torch.uint8)), on(torch.ones(8, H, 16))) for _ in range(2))
        calls.clear()
        out = dg.fp8_tree_attention(q, cache, on(torch.zeros(B, 2, dtype=torch.int32)),
                                    on(torch.zeros(B, dtype=torch.int32)), workspace=on(torch.zeros(1 << 20, dtype=torch.uint8)))
        return calls, out
    run.calls = calls
    return run


def rows(*shape):
    return on(torch.zeros(*shape, dtype=torch.bfloat16))


@pytest.mark.parametrize("B,N", [(4, 1), (1, 1), (4, 3), (1, 3)])
@pytest.mark.parametrize("name,make", [
    ("half of a wider head", lambda B, N: rows(B, N, 8, 256)[..., :128]),
    ("every second head", lambda B, N: rows(B, N, 16, 128)[:, :, ::2]),
    ("heads last", lambda B, N: rows(B, N, 128, 8).transpose(2, 3)),
    ("every second value", lambda B, N: rows(B, N, 8, 256)[..., ::2])])
def test_queries_that_are_not_dense_are_refused(attend, B, N, name, make):
    q = make(B, N)
    assert q.shape == (B, N, 8, 128)
    with pytest.raises(ValueError, match="dense"):
        attend(q)
    assert not attend.calls


@pytest.mark.parametrize("name,make,stride", [
    ("dense", lambda: rows(4, 1, 8, 128), 1024),
    ("heads of a wider row", lambda: rows(4, 12, 128)[:, 2:10].unsqueeze(1), 1536),
    ("heads of a wider row, by token", lambda: rows(4, 1, 12, 128)[:, :, 2:10], 1536),
    ("the last of each request's tokens", lambda: rows(4, 5, 8, 128)[:, 4:], 5120),
    ("one head", lambda: rows(4, 1, 4, 128)[:, :, 1:2], 512),
    ("tokens of a wider row", lambda: rows(4, 3, 12, 128)[:, :, 2:10], 1536),
    ("one request", lambda: rows(1, 3, 12, 128)[:, :, 2:10], 1536)])
def test_queries_of_wider_rows_pass_their_stride(attend, name, make, stride):
    q = make()
    calls, (o, lse) = attend(q, H=1)
    assert len(calls) == 1 and calls[0][1] == stride
    assert o.shape == q.shape and lse.shape == q.shape[:3] and o.is_contiguous()


@pytest.mark.parametrize("q", [rows(4, 0, 8, 128), rows(4, 5, 8, 128)[:, 5:], rows(1, 0, 8, 128), rows(0, 0, 8, 128),
                               rows(0, 3, 8, 128), rows(4, 3, 0, 128)], ids=lambda q: str(tuple(q.shape)))
def test_queries_of_nothing(attend, q):
    """No requests, tokens or heads are no work and no error, as in the C call."""
    calls, (o, lse) = attend(q)
    assert len(calls) == 1 and o.shape == q.shape and lse.shape == q.shape[:3]
    stride = calls[0][1]
    assert stride >= q.shape[2] * 128 and stride % 8 == 0
