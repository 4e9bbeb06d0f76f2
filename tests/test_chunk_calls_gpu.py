"""Appends at far positions, and what the calls make of each other's results and of wrong offsets."""
import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv
from test_append_rope_gpu import Run
from test_chunk_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def test_a_negative_frequency_turns_as_far_the_other_way():
    """At far positions, where a frequency held less exactly than its opposite would show."""
    d, p = 64, (1 << 31) - 256
    cfg = ref.Case([(1, 0)], 1, 1, d, F32).cfg
    g = torch.Generator(device=DEV).manual_seed(96)
    f = 10000.0 ** -torch.rand(32, dtype=torch.float64, generator=g, device=DEV)
    q = torch.randn(1, 1, d, generator=g, device=DEV)
    mirror = torch.ones(d, device=DEV)
    mirror[32:] = -1
    table = torch.zeros(1, p // 128 + 1, dtype=torch.int32, device=DEV)
    k, v = (torch.zeros(1, 1, 128, d, device=DEV) for _ in "kv")
    reps, outs = torch.zeros(1, 1, d, device=DEV), []
    for freqs, x in ((f, q), (-f, q * mirror)):
        out = torch.zeros_like(q)
        srkv.append_kv_rope(cfg, x, x, x, freqs, k, v, table, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                            torch.tensor([p], dtype=torch.int32, device=DEV), reps, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1] * mirror)
