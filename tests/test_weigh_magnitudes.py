"""Scales and scores at the ends of fp32's range: what counts is their product."""

import ctypes

import numpy as np
import pytest

from oracle import eviction as E
from test_weigh import RANGE, SCALE, _weigh, batch, check

gpu = pytest.mark.gpu


def scaled(x, by_q, by_k=1.0):
    """The batch's queries and (bf16) keys times powers of two, exactly."""
    bf = lambda b, by: ((b.astype(np.uint32) << 16).view(np.float32) * np.float32(by)).view(np.uint32) >> 16
    x["q"] = bf(x["q"], by_q).astype(np.uint16)
    if x["fp8"]:
        x["ks"] = np.where(x["ks"] == 255, 255, x["ks"].astype(int) + int(np.log2(by_k))).astype(np.uint8)
    else:
        x["k"] = bf(x["k"], by_k).astype(np.uint16)
    return x


@pytest.mark.parametrize("scale,code", [(2.0 ** 126, 0), (2.0 ** 127, 0), (2.36e38, RANGE), (3.4e38, RANGE)])
def test_scales_beyond_range_are_refused(pkvlib, scale, code):
    """Where scale times log2(e) is no fp32 number.  (B = 0: nothing is launched.)"""
    assert _weigh(pkvlib, B=0, scale=scale) == code


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows", [([200, 33], [1, 1]), ([700, 9, 64], [8, 3, 1]), ([300, 130], [100, 130]),
                                       ([1000, 40, 17], [300, 33, 1])])
@pytest.mark.parametrize("by_q,by_k,scale", [
    (2.0 ** -40, 1.0, 2.0 ** 40 * SCALE),            # a scale whose product with a sentinel of 1e30 overflows
    (2.0 ** -90, 2.0 ** -27, 2.0 ** 117 * SCALE),
    (2.0 ** 80, 2.0 ** 30, 2.0 ** -110 * SCALE),     # scores of 1e33: maxima far below -1e30 among them
    (2.0 ** 60, 2.0 ** 55, 2.0 ** -115 * SCALE),
])
def test_only_the_product_of_scale_and_scores_counts(pkvlib, lens, rows, by_q, by_k, scale, fp8):
    x = scaled(batch(lens, rows, 8, 2, seed=sum(lens), fp8=fp8, pad=1), by_q, by_k)
    got = check(x, scale=scale, decay=0.0)
    assert np.isfinite(got[E.weigh(x["q"], x["k"], x["scores"], x["tables"], x["lens"], x["qsl"], scale, 0.0,
                                   k_scale=x["ks"])[1] > 0]).all()


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,rows", [([200, 33], [1, 1]), ([300, 130], [100, 130])])
@pytest.mark.parametrize("more", [1.0, 2.0 ** 6])
def test_all_scores_far_below_zero(pkvlib, lens, rows, more, fp8):
    """Every score of every row lies near -1e33, times the scale near -7 or -450:
    a row's sum is one from its largest score down, not from a fixed one."""
    x = batch(lens, rows, 4, 2, seed=7, fp8=fp8)
    x["q"][: x["qsl"][-1]] |= 0x8000  # all negative against keys that are all positive
    if fp8:
        x["k"] &= 0x7F
    else:
        x["k"] &= 0x7FFF
    check(scaled(x, 2.0 ** 60, 2.0 ** 45), scale=more * 2.0 ** -105 * SCALE, decay=0.0)
