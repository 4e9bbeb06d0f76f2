"""Chunks of a few rows, which the warps of a CTA share by tokens (fp32, up to 8 and 16 rows) or one of the two tiles
leaves to the other (bf16): against 64 bits at the borders, and with values that are not finite in hidden places."""
import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv
from test_chunk_gpu import attend, check

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [False, True])
def test_a_few_rows(dtype, d, window):
    reqs = [(n, p) for n in (1, 4, 7, 8, 9, 15, 16, 17, 127, 128, 129) for p in (0, 49, 64 - n, 190, 1300) if p >= 0]
    check(ref.Case(reqs, Hq=2, Hkv=2, d=d, dtype=dtype, seed=51, init=70, local=90), window)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n", [5, 12])
def test_hidden_values_that_are_not_finite(dtype, n):
    """Token 202 (a new one: later rows attend it) and token 150 (outside every window) hold a NaN."""
    kw = dict(Hq=2, Hkv=2, d=64, dtype=dtype, seed=52, init=100, local=40)
    clean, case = ref.Case([(n, 200)], **kw), ref.Case([(n, 200)], **kw)
    for t in (150, 202):
        case.v[int(case.table[0, t // 128]), :, t % 128, 5] = float("nan")
    out, want = attend(case, window=True), attend(clean, window=True)
    keep = [e for e in range(64) if e != 5]
    assert torch.equal(out[:2], want[:2])
    assert out[2:, :, 5].isnan().all()
    assert torch.equal(out[2:][:, :, keep], want[2:][:, :, keep])


@pytest.mark.parametrize("d", [64, 128])
def test_rows_without_a_token_and_pages_that_are_not_there(d):
    kw = dict(Hq=2, Hkv=2, d=d, dtype=F32, seed=53)
    case = ref.Case([(3, 700), (2, 300)], **kw, init=0, local=0)
    assert not attend(case, window=True).any() and int(case.flags) == 0
    case = ref.Case([(3, 700), (2, 300)], **kw)
    want = attend(case).clone()
    case.table[0] = -1
    out = attend(case)
    assert not out[:3].any() and torch.equal(out[3:], want[3:]) and int(case.flags) == srkv.EFLAG_PAGE_RANGE
