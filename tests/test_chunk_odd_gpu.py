"""Values that are not finite in pages that some rows see in part, as many of them as a tile can meet: every row
gets those that it attends and no others."""
import pytest
import torch

import chunk_ref as ref
from test_chunk_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("Hq,Hkv,d", [(1, 1, 128), (2, 2, 64), (8, 2, 64), (3, 1, 128)])
@pytest.mark.parametrize("window", [False, True])
def test_every_32nd_value_is_infinite(Hq, Hkv, d, window):
    reqs = [(300, 700), (1, 900), (129, 383)]
    kw = dict(Hq=Hq, Hkv=Hkv, d=d, seed=31, init=140, local=333)
    clean, case = ref.Case(reqs, **kw), ref.Case(reqs, **kw)
    for r, (n, p) in enumerate(reqs):
        L = n + p
        for t in range(5, L, 32):
            case.v[int(case.table[r, t // 128]), :, t % 128, t % d] = float("inf")
    got, want = attend(case, window).float(), attend(clean, window).float()
    assert int(case.flags) == 0
    for r, (n, p) in enumerate(reqs):
        lo = int(case.offsets[r])
        pos = torch.arange(p, p + n, device=DEV).unsqueeze(1)
        t = torch.arange(5, p + n, 32, device=DEV)
        on = t <= pos
        if window:
            on &= (t < 140) | (t > pos - 333)
        hit = torch.zeros(n, d, dtype=torch.bool, device=DEV)
        for i, x in enumerate(t.tolist()):
            hit[:, x % d] |= on[:, i]
        hit = hit.unsqueeze(1).expand(n, Hq, d)
        g, w = got[lo:lo + n], want[lo:lo + n]
        assert (g[hit] == float("inf")).all()
        assert torch.equal(g[~hit], w[~hit])
