"""Which form the cases of tests/fp4_forms.py have the attention read values in, and the bounds by form."""
import numpy as np
import pytest

from tests import fp4_forms as forms
from tests import paged


@pytest.mark.parametrize("values", list(forms.VALUES))
@pytest.mark.parametrize("shape", ["decode D=64", "decode D=128", "decode D=256", "long trees"])
def test_cases_have_their_form(shape, values):
    c = forms.case(*forms.SHAPES[shape], forms.VALUES[values], 1)
    assert paged.form4(c["read"]) == values[:4]


def test_form_of_scales():
    assert paged.form4([109, 140]) == "fp16" and paged.form4([108, 141, 0, 255]) == "bf16" and paged.form4([108, 109]) == "both"


@pytest.mark.parametrize("form,bits", [("fp16", 11), ("bf16", 16)])
def test_bounds_tell_the_forms_apart(form, bits):
    """Two keys of nearly the same weight whose values are opposite: weights rounded to their bits stay in
    the bound, and to four bits fewer do not."""
    rng = np.random.default_rng(0)
    D, page, rows = 64, 16, 64
    cache = paged.random_cache4(rng, 1, 1, page, D, forms.VALUES["fp16"])
    cache[1][0][0, 0, 1] = cache[1][0][0, 0, 0] ^ 0x88
    cache[1][1][0, 0, 1] = cache[1][1][0, 0, 0]
    q = 0.002 * rng.standard_normal((1, 1, rows, D))
    ref, _, bound, _ = paged.attention4(q, cache, np.zeros((1, 1), np.int32), [1], [1], np.ones((1, 1, 1), bool), 1.0, page, form)
    key, val = (paged.values4(codes[0, 0, :2], sf[0, 0, :2]) for codes, sf in cache)
    e = np.exp(q[0, 0] @ key.T)
    for keep, right in ((bits, True), (bits - 4, False)):
        m, k = np.frexp(e)
        rounded = np.ldexp(np.round(m * 2.0 ** keep), k - keep)
        o = rounded @ val / e.sum(1, keepdims=True)
        assert (np.abs(o - ref[0, 0]) <= bound[0, 0]).all() == right
