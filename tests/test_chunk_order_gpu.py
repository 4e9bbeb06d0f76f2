"""A chunk call reads what the kernels before it in its stream wrote, tables, lengths and offsets too, although its own
kernels start ahead of their end."""
import pytest
import torch

import chunk_ref as ref
from test_chunk_gpu import attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("reqs,other", [([(1, 6000)], [(1, 900)]), ([(2, 300), (1, 4000)], [(1, 5000), (2, 100)]),
                                        ([(200, 500)], [(200, 20)])], ids=["token", "tokens", "chunk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_tables_lengths_and_caches_written_just_before(reqs, other, dtype):
    cases = [ref.Case(x, dtype=dtype, seed=61 + i) for i, x in enumerate((reqs, other))]
    want = [attend(c).clone() for c in cases]
    pages, blocks = max(c.pages for c in cases), max(c.max_blocks for c in cases)
    live = ref.Case(reqs, dtype=dtype, seed=60)  # whose contents change from call to call
    live.k, live.v = (torch.zeros(pages, *live.k.shape[1:], dtype=dtype, device="cuda") for _ in "kv")
    live.table = torch.full((len(reqs), blocks), -1, dtype=torch.int32, device="cuda")
    out, ws = torch.zeros_like(want[0]), None
    got = []
    for i in range(60):
        c = cases[i % 2]
        live.k[:c.pages].copy_(c.k)
        live.v[:c.pages].copy_(c.v)
        live.q.copy_(c.q)
        live.offsets.copy_(c.offsets)
        live.lens.copy_(c.lens)
        live.table.fill_(-1)
        live.table[:, :c.max_blocks].copy_(c.table)
        got.append(attend(live, out=out, workspace=ws).clone())
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2]), i
