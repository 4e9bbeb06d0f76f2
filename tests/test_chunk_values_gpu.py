"""Attended values that are not finite: their element of the row is infinite or NaN however small their weight, in a page
that all rows of a tile see and in one that some see, whatever the other rows are; a row whose logits are all -infinity
is 0 whatever the values."""
import pytest
import torch

import chunk_ref as ref
from test_chunk_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def hold(case, name, r, t, col, value, heads=slice(None)):
    getattr(case, name)[int(case.table[r, t // 128]), heads, t % 128, col] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("t", [10, 130, 210], ids=["in a whole page", "before every row", "hidden from some"])
@pytest.mark.parametrize("n", [1, 3, 12, 200])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
def test_a_weight_of_zero_does_not_hide_an_attended_value(dtype, d, n, t, value):
    """Token t's weight is below 2^-500 of the others'."""
    made = []
    for _ in range(2):
        case = ref.Case([(n, 209)], Hq=4, Hkv=2, d=d, dtype=dtype, seed=81)
        case.q[:, :, 0] = 8.0
        if t < 209 + n:
            hold(case, "k", 0, t, 0, -8.0 * d)
        made.append(case)
    clean, case = made
    want = attend(clean)
    if t < 209 + n:
        hold(case, "v", 0, t, 5, value)
    out = attend(case)
    sees = torch.arange(209, 209 + n, device=DEV) >= t
    assert not out[sees][:, :, 5].isfinite().any()
    keep = [e for e in range(d) if e != 5]
    assert torch.equal(out[..., keep], want[..., keep]) and torch.equal(out[~sees], want[~sees])


@pytest.mark.parametrize("reqs", [[(1, 300)], [(1, 300)] * 160, [(9, 300)] * 160, [(200, 209)], [(1, 30000)],
                                  [(150, 30000)]],
                         ids=["token", "tokens", "few", "chunk", "divided", "divided chunk"])
@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 128), (F32, 64), (F32, 128)])
def test_rows_without_a_finite_logit_are_zero(dtype, d, reqs):
    """The keys of head 0 give -infinity; head 1 is as it was."""
    case = ref.Case(reqs, Hq=4, Hkv=2, d=d, dtype=dtype, seed=82)
    want = attend(case).clone()
    case.q[:, :2] = 0
    case.q[:, :2, 0] = 1
    for r, (n, p) in enumerate(reqs):
        case.k[case.table[r, :-(-(n + p) // 128)].long(), 0, :, 0] = -float("inf")
        for t in (10, p - 1, p):
            hold(case, "v", r, t, 5, float("nan"), 0)
            hold(case, "v", r, t, 7, float("inf"), 0)
    out = attend(case)
    assert (out[:, :2] == 0).all()
    assert torch.equal(out[:, 2:], want[:, 2:])
