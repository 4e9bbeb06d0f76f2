"""The bound that the GPU tests hold the 4-bit decode to is far below the outputs, and mistakes pass it (no GPU):
planted in the restatement, each has to leave the bound."""
import numpy as np
import pytest

import int4_exact as exact
import int4_ref as ref


def random_rows(N, d, seed, offset=0.0):
    """N rows as the quantiser makes them from normal data: codes, scales, minima of keys and values."""
    rng = np.random.default_rng(seed)
    out = []
    for shift in (offset, 0.0):
        c, s, lo = exact.quantize_rows(ref.to_bf16(rng.standard_normal((N, d)) + shift))
        out += [c, s, lo]
    return out


def query(G, d, seed):
    return ref.to_bf16(np.random.default_rng(seed).standard_normal((G, d)))


@pytest.mark.parametrize("N,share", [(1, 0.1), (200, 0.1), (3000, 0.1), (30000, 0.15), (118000, 0.25)])
@pytest.mark.parametrize("d", [64, 128])
def test_the_bound_is_far_below_the_outputs(N, share, d):
    out, bound = exact.attend(query(4, d, 1), random_rows(N, d, 2), random=True)
    rms = (out ** 2).mean() ** 0.5
    assert np.median(bound) < share * rms and bound.max() < 0.5 * rms + 2.0 ** -7 * np.abs(out).max()


def dropped(rows, lo, hi):
    keep = np.ones(len(rows[0]), bool)
    keep[lo:hi] = False
    return [a[keep] for a in rows]


def changed(rows, i, f):
    rows = list(rows)
    rows[i] = f(rows[i].copy())
    return rows


def some(lo, hi, f):
    def g(a):
        a[lo:hi] = f(a[lo:hi])
        return a
    return g


MISTAKES = {
    "a group of 32 tokens is lost": lambda r: dropped(r, 640, 672),
    "a group of 32 tokens counts twice": lambda r: [np.concatenate((a, a[640:672])) for a in r],
    "a page's value scales are off by a bf16 step in eight": lambda r: changed(r, 4, some(128, 256, lambda a: a * 1.0625)),
    "a page's value minima are lost": lambda r: changed(r, 5, some(128, 256, lambda a: a * 0)),
    "all value minima are lost": lambda r: changed(r, 5, lambda a: a * 0),
    "a page's keys are the next page's": lambda r: changed(r, 0, lambda a: np.roll(a, 128, 0)),
    "key minima are lost": lambda r: changed(r, 2, lambda a: a * 0),
    "key scales are off by one row": lambda r: changed(r, 1, lambda a: np.roll(a, 1)),
    "value codes of neighbours change places": lambda r: changed(r, 3, lambda a: a.reshape(-1, 2, a.shape[1])[:, ::-1].reshape(a.shape)),
    "elements change places": lambda r: changed(r, 3, lambda a: np.roll(a, 1, 1)),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", list(MISTAKES))
def test_mistakes_leave_the_bound(name, d):
    q, rows = query(4, d, 3), random_rows(1536, d, 4, offset=0.5)
    want, bound = exact.attend(q, rows, random=True)
    got, _ = exact.attend(q, MISTAKES[name](rows))
    assert (np.abs(ref.to_bf16(got) - want) > 2 * bound).any()
    assert (np.abs(ref.to_bf16(want) - want) <= bound).all()


@pytest.mark.parametrize("d", [64, 128])
def test_zeros_and_lost_heads_leave_the_bound_at_every_length(d):
    for N in (1, 700, 30000):
        q, rows = query(3, d, 5), random_rows(N, d, 6)
        want, bound = exact.attend(q, rows, random=True)
        assert (np.abs(want) > bound).mean() > 0.7
        if N > 1:
            assert (np.abs(want[[1, 2, 0]] - want) > bound).any(1).all()


def test_what_a_query_loses():
    q = np.zeros((2, 64))
    q[0] = 1.5
    q[1] = ref.to_bf16(np.linspace(1, 2, 64) * 2.0 ** -16)
    assert (exact.query_error(q) == 0).all()
    q[0, 0] = 2.0 ** 14  # now the second head's elements reach fp16's subnormals, in the upper nibbles first
    err = exact.query_error(q)
    assert (err[0] == 0).all() and (err[1] > 0).any()
    assert (err <= 2.0 ** -25 * 2.0 ** 4).all()
