"""The 4-bit rows from the sentences of include/srkv.h, in numpy: apart from int4_ref.py, whose test for rows
that get NaN parameters takes |lo| where the header takes lo (rows from about -1.7e38 down)."""
from __future__ import annotations

import numpy as np

import int4_ref as ref

BF16_MAX = 2.0 ** 128 - 2.0 ** 120
PAST_BF16 = 2.0 ** 128 - 2.0 ** 119  # from here on a value rounds to infinity (a tie goes to even)


def bf16_up(x):
    """x >= 0 (float64) to the next bf16 upwards, subnormal ones among them, and the gap below it."""
    _, e = np.frexp(np.maximum(x, 2.0 ** -126))
    step = np.ldexp(1.0, e - 8)
    return np.ceil(x / step) * step, step


def quantize_rows(x):
    """Rows x [..., d] (float64, bf16 values): codes [..., d] int64, scale and lo [...] float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        lo = x.min(-1)
        span = (x.max(-1).astype(np.float32) - lo.astype(np.float32)).astype(np.float64)
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(span)
        span = np.where(bad, 0, span)
        scale, step = bf16_up(span / 15)
        scale = np.where(lo + 15 * scale >= PAST_BF16, scale - step, scale)
        diff = x.astype(np.float32) - lo.astype(np.float32)[..., None]
        codes = np.rint(diff / np.where(scale > 0, scale, 1).astype(np.float32)[..., None])
    codes = np.where(bad[..., None] | (scale < 2.0 ** -126)[..., None], 0, codes).astype(np.int64)
    return codes, np.where(bad, np.nan, scale), np.where(bad, np.nan, lo)


def check_slab(slab, k, v, d):
    """A slab's words against the rows they came from, code for code."""
    kc, vc, ks, kl, vs, vl = ref.unpack(slab, d)
    for codes, scale, lo, x in ((kc, ks, kl, k), (vc, vs, vl, v)):
        c, s, m = quantize_rows(x)
        np.testing.assert_array_equal(scale, s)
        np.testing.assert_array_equal(lo, m)
        np.testing.assert_array_equal(codes, c)
