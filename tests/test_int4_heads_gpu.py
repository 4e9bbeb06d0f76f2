"""The 4-bit decode with heads of one group whose queries are of very different magnitudes: each is as accurate as alone."""
import numpy as np
import pytest
import torch

import int4_exact as exact
import int4_ref as ref
from test_int4_gpu import int4_case, make, step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 24])
@pytest.mark.parametrize("head_dim,group", [(64, 3), (64, 8), (128, 4), (128, 5)])
def test_a_head_does_not_cost_its_neighbours_bits(batch, head_dim, group):
    case = make(seq_lens=[2000 - 31 * r for r in range(batch)], num_q_heads=2 * group, num_kv_heads=2, head_dim=head_dim,
                topk_percent=1.0, seed=141)
    powers = torch.tensor([60, 0, -3, 30, 1, 0, -60, 2][:group], device="cuda").double().repeat(2)
    case.q.copy_(case.q.double() * 2.0 ** powers[None, :, None])
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    host, q, out = kv.cpu().numpy(), ref.host(case.q), ref.host(buf.out)
    table, L = case.block_table.cpu().numpy(), case.seq_lens.tolist()
    for r, h in {(0, 0), (batch // 2, 1), (batch - 1, 1)}:
        rows = exact.gather(host, table[r], L[r], range(100), case.cfg, h, head_dim)
        for j in range(h * group, (h + 1) * group):
            if powers[j] > 10:  # one token has all of the weight, or two whose logits fp32 cannot tell apart
                assert np.isfinite(out[r, j]).all()
                continue
            want, bound = exact.attend(q[r, j:j + 1], rows, random=True)
            assert np.median(bound) < 0.25 * (want ** 2).mean() ** 0.5
            assert (np.abs(out[r, j] - want) <= bound).all(), (r, j)
