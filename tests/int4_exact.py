"""The 4-bit rows and the step over them from the sentences of include/srkv.h, in 64 bits (numpy): apart from
int4_ref.py, whose rule for NaN rows takes |lo| where the header takes lo (rows from about -1.7e38 down), and
whose bound on the step's output charges every rounding at the largest row and logit, so that on long requests
it passes the outputs themselves."""
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


def attended(cfg, L, sel):
    """The attended tokens of a request as a mask [blocks][128]."""
    t = np.arange(-(-L // 128) * 128).reshape(-1, 128)
    W = L - cfg["local_tokens"]
    kept = np.isin(t // 128, np.asarray(sel, np.int64)) & (t >= cfg["init_tokens"]) & (t < W)
    return ((t < cfg["init_tokens"]) | (t >= W) | kept) & (t < L)


def gather(kv, pages, L, sel, cfg, h, d):
    """The attended rows of one (request, kv head): codes [N][d] and scales, minima [N] of keys and values."""
    on = attended(cfg, L, sel)
    parts = []
    for b in np.flatnonzero(on.any(1)):
        k, v, ks, kl, vs, vl = ref.unpack(kv[pages[b], h], d)
        parts.append([a[on[b]] for a in (k, ks, kl, v, vs, vl)])
    return [np.concatenate(a) for a in zip(*parts)] if parts else None


def query_error(q):
    """What the group's query [G][d] (bf16 values) loses as fp16 times one power of two: the largest magnitude goes to
    [2^14, 2^15), elements whose codes sit in the upper nibble of a byte 16 times lower."""
    top = np.abs(q).max()
    e = np.clip(np.frexp(top)[1] - 1, -112, 100) if top > 0 else -112
    f = np.ldexp(np.where(np.arange(q.shape[1]) % 8 // 2 % 2 == 1, 2.0 ** -4, 1.0), 14 - e)
    return np.abs((q * f).astype(np.float16).astype(np.float64) / f - q)


def attend(q, rows, random=False):
    """Output [G][d] over gathered rows, and what the step's arithmetic may differ from it.

    Roundings at half a step each (finfo.eps / 2 of the type), p the softmax weights, every sum one of this
    unit and head, each element of its own:
      * logits: what the query loses in fp16; d products and the rows' two parameters in fp32 (2^-23, the
        tensor cores' sums may truncate) of sum |q| ks ck + |kl| sum |q|; the difference from the reference,
        2^-24 of it; 2^-20 for the exponentials (the weight's, the merges').  A logit off by e moves the output by
        p e |V - out|;
      * weight times scale in fp16: 2^-11 of sum p vs cv; below fp16's normal range half a subnormal step, 2^-25:
        the largest product p vs that a warp has met is an operand of 2^10 at least, in half of the rows 16 times
        less, so 2^-31 of the unit's largest product, a token;
      * sums over the tokens in fp32: a lane adds four times a page (128 tokens), then come some hundred
        merges: n = N / 32 + 128 times 2^-24 of sum p (vs cv + |vl|), and of the output for the weights' own sum;
        the products of a page on the tensor cores, 2^-19 of the same;
      * the output in bf16: 2^-8 of it.
    random: the rows are random, so that the roundings of different tokens are independent and of mean 0.  N of them,
    r_t each at most, then pass 8 sqrt(sum r_t^2) with a probability below 2 exp(-32) = 3e-14 (Hoeffding's
    inequality): 2^-11 8 sqrt(sum (p vs cv)^2) for the operands, 8 sqrt(n) instead of n for the sums.
    """
    G, d = q.shape
    if rows is None:
        return np.zeros((G, d)), np.zeros((G, d))
    kc, ks, kl, vc, vs, vl = rows
    K, V = kl[:, None] + kc * ks[:, None], vl[:, None] + vc * vs[:, None]
    z = q @ K.T / np.sqrt(d)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = p @ V
    N, kcs, vcs = len(K), kc * ks[:, None], vc * vs[:, None]
    size = (np.abs(q) @ kcs.T + np.abs(q).sum(1, keepdims=True) * np.abs(kl)) / np.sqrt(d)
    dz = (query_error(q) @ kcs.T / np.sqrt(d) + (d + 16) * 2.0 ** -23 * size
          + 2.0 ** -24 * (z.max(1, keepdims=True) - z) + 2.0 ** -20)
    n, operands = N / 32 + 128, p @ vcs
    if random:
        n = min(n, 8 * np.sqrt(n))
        operands = np.minimum(operands, 8 * np.sqrt(p ** 2 @ vcs ** 2))
    sums = p @ (vcs + np.abs(vl)[:, None])
    bound = (2.0 ** -11 * operands + 15 * N * 2.0 ** -31 * (p * vs).max(1, keepdims=True)
             + n * 2.0 ** -24 * (sums + np.abs(out)) + 2.0 ** -19 * sums)
    for g in range(G):
        bound[g] += (p[g] * dz[g]) @ np.abs(V - out[g])
    return out, 1.01 * bound + 2.0 ** -8 * (np.abs(out) + bound)


def decode_unit(q, kv, pages, L, sel, cfg, h, random=False):
    """attend() of one (request, kv head): q [G][d] float64, kv [P][Hkv][bytes], its block table row, its kept blocks."""
    return attend(q, gather(kv, pages, L, sel, cfg, h, q.shape[1]), random)
