"""Long page lists among others: that the plan divides them, and that every page of a divided list counts once.  The
values of the second part are counts (equal logits, a page's values its own), so that a page left out or taken twice
shows whatever the list's length."""
import math

import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv
from test_chunk_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def planned(case, window=False):
    """The output, and what the plan left in the workspace: its items, and the lists that it divided."""
    ws = torch.zeros(srkv.chunk_workspace_size(case.cfg, case.T, len(case.reqs)), dtype=torch.uint8, device=DEV)
    out = attend(case, window, workspace=ws)
    torch.cuda.synchronize()
    assert int(case.flags) == 0
    return out, *ws[:8].view(torch.int32).tolist()


def count(case):
    """Every logit 0; block b of a request holds 1 + b // d in column b % d."""
    d = case.cfg["head_dim"]
    case.q.normal_()
    for r, (n, p) in enumerate(case.reqs):
        L = n + p
        blocks = case.table[r, :-(-L // 128)].long()
        b = torch.arange(len(blocks), device=DEV)
        v = torch.zeros(len(blocks), d, device=DEV)
        v[b, b % d] = (1 + b // d).float()
        case.k[blocks] = 0
        case.v[blocks] = v.to(case.dtype)[:, None, None, :]
        if L % 128:  # behind the sequence
            case.k[blocks[-1], :, L % 128:] = float("nan")
            case.v[blocks[-1], :, L % 128:] = float("nan")
    return case


def check_counts(case, out, window=False):
    d, Hq = case.cfg["head_dim"], case.cfg["num_q_heads"]
    init, local = (case.cfg["init_tokens"], case.cfg["local_tokens"]) if window else (1 << 30, 0)
    for r, (n, p) in enumerate(case.reqs):
        lo, L = int(case.offsets[r]), n + p
        t = torch.arange(L, device=DEV)
        one = torch.zeros(L, d, dtype=torch.float64, device=DEV)
        one[t, t // 128 % d] = (1 + t // 128 // d).double()
        upto = torch.cat((one.new_zeros(1, d), one.cumsum(0)))
        del one
        end = torch.arange(p, L, device=DEV) + 1
        first = end.clamp(max=init)
        start = torch.maximum(first, end - local) if local else end
        total = upto[first] + upto[end] - upto[start]
        want = total / (first + end - start).clamp(min=1).unsqueeze(1)
        want = want.unsqueeze(1).expand(n, Hq, d)
        # weights are 1 and sums are whole numbers below 2^24, so all is exact but the reciprocal, its product
        # and the rounding to the type
        tol = (torch.finfo(case.dtype).eps / 2 + 2.0 ** -21) * want
        bad = ~((out[lo:lo + n].double() - want).abs() <= tol)
        assert not bad.any(), (r, int(bad.sum()), bad.nonzero()[:3].tolist())


def test_a_long_token_beside_a_prompt_is_divided():
    """As a step of a server that starts a prompt while others decode: 64 full tiles, and lists of 1024 pages."""
    case = count(ref.Case([(4096, 0), (1, 131071)], Hq=32, Hkv=8, d=128, seed=71))
    out, items, merges = planned(case)
    assert merges >= 8 and items >= 65 * 8 + 8 * 6, (items, merges)
    check_counts(case, out)


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_one_list_of_one_head_is_divided(dtype, d, n):
    case = count(ref.Case([(n, 400000)], Hq=1, Hkv=1, d=d, dtype=dtype, seed=72))
    out, items, merges = planned(case)
    assert merges == 1 and items >= 100, (items, merges)
    check_counts(case, out)


@pytest.mark.parametrize("reqs,Hkv", [([(1, 511)] * 200 + [(1, 131071)] + [(1, 511)] * 120, 8),
                                      ([(1, 1023)] * 300 + [(1, 131071)] + [(1, 1023)] * 300, 1),
                                      ([(1, 600)] * 320 + [(300, 65000), (3, 99999)], 8)],
                         ids=["320 short", "600 short of one head", "two long"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_a_long_list_among_many_is_divided(reqs, Hkv, dtype, d):
    case = count(ref.Case(reqs, Hq=Hkv, Hkv=Hkv, d=d, dtype=dtype, seed=73))
    out, items, merges = planned(case)
    lists = sum(-(-n // (256 if dtype == BF else d)) for n, _ in reqs) * Hkv
    assert merges >= Hkv and items >= lists + 4 * Hkv, (items, lists, merges)
    check_counts(case, out)
    assert torch.equal(planned(case)[0], out)


@pytest.mark.parametrize("reqs", [[(1, 65535)], [(300, 130772)], [(2, 30000), (257, 66000), (1, 131071)]],
                         ids=["token", "rows", "mixed"])
@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_every_page_counts_once(reqs, window, dtype, d):
    case = count(ref.Case(reqs, Hq=2, Hkv=1, d=d, dtype=dtype, seed=74, init=1000, local=20001))
    check_counts(case, planned(case, window)[0], window)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_random_values_over_131072_tokens(dtype, d):
    """Two tiles over a thousand pages against 64 bits, as a whole.  Logits are N(0, 1) and values independent of them, so
    with weights w the output's mean square is that of w v, summed.  Rounding each weight (by up to 2^-8, evenly: 2^-8 /
    sqrt 3 in the mean square) and each output (the same) adds sqrt(2 / 3) 2^-8 of that; what fp32 adds (a logit
    is a sum of d products of up to 12 in all, whose roundings are as good as independent: sqrt(d) 2^-24 12 < 2^-16) the
    rest.  One page left out is 2^-5."""
    case = ref.Case([(300, 130772)], Hq=4, Hkv=1, d=d, dtype=dtype, seed=75)
    out = attend(case)
    want, _ = ref.attention(case, False)
    error = float((out.double() - want).square().mean().sqrt() / want.square().mean().sqrt())
    assert error <= (math.sqrt(2 / 3) * 2.0 ** -8 if dtype == BF else 0.0) + 2.0 ** -16, error
