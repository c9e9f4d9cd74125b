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
