"""GPU parity of the attention over the FP4 cache in each of the forms that it reads values in, within the
bounds of that form, at the ends of scales, and of what a row may not depend on."""
import numpy as np
import pytest
import torch

import fp8_fine_grained_e4m3_amd as dg
from tests import few_tokens as ft
from tests import fp4_forms as forms
from tests import paged
from tests.parity import announce, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dg.load_library()
    yield


def run(c):
    cache = tuple((dev(codes), dev(sf)) for codes, sf in c["cache"])
    q = torch.from_numpy(c["q"]).bfloat16()
    o, lse = dg.fp4_tree_attention(q.cuda(), cache, dev(c["table"]), dev(c["ctx"]), dev(c["lens"]), dev(ft.pack_mask(c["mask"])), c["scale"])
    torch.cuda.synchronize()
    return o, lse


def check(c, form):
    o, lse = (t.float().cpu().numpy().astype(np.float64) for t in run(c))
    q = torch.from_numpy(c["q"]).bfloat16().double().numpy()
    ro, rl, bo, bl = paged.attention4(q, c["cache"], c["table"], c["ctx"], c["lens"], c["mask"], c["scale"], c["page"], form)
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), empty) and not o[empty].any()
    assert np.array_equal(np.isnan(o), np.isnan(ro)) and np.array_equal(np.isnan(lse), np.isnan(rl))
    ok = ~np.isnan(ro)
    assert np.isfinite(o[ok]).all()
    assert (np.abs(o - ro)[ok] <= bo[ok]).all(), f"o: {np.max(np.abs(o - ro)[ok] / bo[ok])} of the bound"
    ok = ~empty & ~np.isnan(rl)
    off = np.abs(lse[ok] - rl[ok])
    assert (off <= bl[ok]).all(), f"lse: {np.max(off / bl[ok])} of the bound"


@pytest.mark.parametrize("values", list(forms.VALUES))
@pytest.mark.parametrize("shape", list(forms.SHAPES))
def test_each_form(shape, values):
    announce(f"fp4 {values}: {shape}")
    c = forms.case(*forms.SHAPES[shape], forms.VALUES[values], 1)
    form = paged.form4(c["read"])
    assert form == values[:4]
    check(c, form)


@pytest.mark.parametrize("values", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N", [1, 3])
def test_opposite_values(N, D, values):
    """Weights of nearly the same size and opposite values, which leave little but the weights' roundings."""
    announce(f"fp4 opposite values D={D} N={N} {values}")

    def change(rng, cache, table, ctx, lens):
        codes, sf = cache[1]
        for b in range(len(ctx)):                        # every odd position the negative of the one before
            p = np.arange(1, ctx[b] + lens[b], 2)
            to, of = (table[b, p // 16], slice(None), p % 16), (table[b, (p - 1) // 16], slice(None), (p - 1) % 16)
            codes[to], sf[to] = codes[of] ^ 0x88, sf[of]

    c = forms.case(6, N, 2, 16, D, 16, 33, 0, forms.VALUES[values], D + N, q_scale=0.004, change=change)
    assert paged.form4(c["read"]) == values
    check(c, values)


@pytest.mark.parametrize("byte", [100, 108, 109, 140, 141, 150])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_scale_around_the_range(D, byte):
    """A single block of a value on either side of fp16's range, in a step that all see and in one that is masked."""
    announce(f"fp4 one scale of 2^{byte - 127}, D={D}")
    for block in range(D // 32):
        def change(rng, cache, table, ctx, lens):
            sf = cache[1][1]
            sf[table[0, 1], 0, 3, block] = byte          # position 19 of 70 + 4
            sf[table[0, 4], 1, 9, block] = byte          # position 73, the last one
            sf[table[1, 0], 1, 5, block] = byte          # of 4 + 1: the only step, masked

        c = forms.case(2, 4, 2, 4, D, 16, 70, 0, forms.VALUES["fp16"], D + byte, change=change)
        c["ctx"][1], c["lens"][1] = 4, 2
        check(c, "fp16")


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("room", [0, 9000])
def test_small_columns_beside_large_ones(D, N, room):
    """Sums of a block of 2^124 pass fp32's range: the other blocks keep their 16 bits."""
    announce(f"fp4 small beside large D={D} N={N} room={room}")

    def change(rng, cache, table, ctx, lens):
        sf = cache[1][1]
        sf[..., 0] = 127 + 124

    c = forms.case(2, N, 2, 4, D, 16, 300, room, forms.VALUES["fp16"], D + N, change=change)
    check(c, "bf16")


@pytest.mark.parametrize("N", [1, 5])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("room", [0, 9000])
def test_smallest_and_largest_scales(D, N, room):
    """Blocks of keys and values with the scales 2^-126 and 2^125, queries that bring all to one size."""
    announce(f"fp4 ends of scales D={D} N={N} room={room}")

    def change(rng, cache, table, ctx, lens):
        for _, sf in cache:
            sf[..., 0], sf[..., 1] = 1, 252

    c = forms.case(3, N, 2, 4, D, 16, 200, room, forms.VALUES["fp16"], D + N, scale=0.05, change=change)
    c["q"][..., :32] *= 2.0 ** 124
    c["q"][..., 32:64] *= 2.0 ** -121
    check(c, "bf16")


@pytest.mark.parametrize("D,N,G,room", [(64, 9, 2, 0), (128, 9, 4, 0), (256, 9, 4, 0), (128, 20, 4, 5000), (64, 12, 8, 9000), (128, 12, 8, 9000)])
@pytest.mark.parametrize("byte", [100, 150, 240, 255])
def test_a_hidden_values_scale_changes_no_bit(D, N, G, room, byte):
    """The scale of a drafted token's value goes out of fp16's range, or NaN: rows that do not see the token keep
    their bits, and those that see it are as the reference."""
    announce(f"fp4 hidden scale 2^{byte - 127}, D={D} N={N} room={room}")
    c = forms.case(3, N, 2, G, D, 16, 200, room, forms.VALUES["fp16"], D + N)
    o, lse = run(c)
    for token, block in ((N // 3, 0), (N // 3 + 1, D // 32 - 1)):
        for b in range(3):
            page, place = forms.at(c, b, int(c["ctx"][b]) + token)
            if token < c["lens"][b]:
                c["cache"][1][1][page, :, place, block] = byte
    misses = ~c["mask"][:, :, [N // 3, N // 3 + 1]].any(-1)
    assert misses[0].any() and not misses[0].all()
    o2, lse2 = run(c)
    keep = torch.from_numpy(misses).cuda()
    assert torch.equal(o2[keep].view(torch.int16), o[keep].view(torch.int16)) and torch.equal(lse2[keep], lse[keep])
    check(c, "fp16")


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -140, -(2.0 ** -128)])
def test_scales_of_scores_next_to_zero(scale):
    """Products of queries and keys next to fp32's largest number, brought to little or nothing by the scale."""
    announce(f"fp4 scale of scores {scale}")
    c = forms.case(3, 5, 2, 4, 128, 16, 200, 0, forms.VALUES["fp16"], 3, q_scale=2.0 ** 119, scale=scale)
    check(c, "fp16")
