"""Chunks whose lists are far from equal: one longer than all CTAs' average load, among as many as there are CTAs
and more, so that all are divided; and single calls captured into a graph before any other of their kind was made."""
import os
import subprocess
import sys

import pytest
import torch

import chunk_ref as ref
from test_chunk_gpu import attend, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 64), (torch.float32, 64), (torch.float32, 128)])
@pytest.mark.parametrize("long", [[(40, 16000), (300, 12000)], [(1, 40000)]], ids=["chunks", "token"])
def test_one_list_outlasts_the_others(dtype, d, long):
    reqs = [(40, 0)] * 19 + long + [(33, 20)] * 19
    case = ref.Case(reqs, Hq=8, Hkv=8, d=d, dtype=dtype, seed=41)
    out = check(case)
    assert torch.equal(attend(case), out)  # the same bits, whoever takes which piece


FIRST = """
import torch
import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv
dtype, d = getattr(torch, "{dtype}"), {d}
case = ref.Case([(1, 700), (1, 40), (1, 127)], Hq=8, Hkv=2, d=d, dtype=dtype, seed=42)
out, q2 = torch.zeros(3, 8, d, dtype=dtype, device="cuda"), torch.zeros(3, 8, d, dtype=dtype, device="cuda")
ws = torch.empty(srkv.chunk_workspace_size(case.cfg, 3, 3), dtype=torch.uint8, device="cuda")
freqs = torch.ones(d // 2, dtype=torch.float64, device="cuda")
before = case.lens - 1
k1, v1 = torch.ones(3, 2, d, dtype=dtype, device="cuda"), torch.ones(3, 2, d, dtype=dtype, device="cuda")
reps = torch.zeros(case.k.shape[0], 2, d, device="cuda")
def step():
    srkv.append_kv_rope(case.cfg, case.q, k1, v1, freqs, case.k, case.v, case.table, case.offsets, before, reps, q2,
                        case.flags)
    srkv.chunk_attention(case.cfg, q2, case.k, case.v, case.table, case.offsets, case.lens, out, ws, case.flags)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = out.clone()
step()
torch.cuda.synchronize()
assert got.abs().sum() > 0 and torch.equal(got, out) and int(case.flags) == 0
print("the same")
"""


@pytest.mark.parametrize("dtype,d", [("bfloat16", 128), ("float32", 128)])
def test_the_first_call_of_a_process_may_be_a_captured_one(dtype, d):
    here = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTHONPATH": os.pathsep.join([here, os.path.dirname(here)])}
    done = subprocess.run([sys.executable, "-c", FIRST.format(dtype=dtype, d=d)], env=env, capture_output=True, text=True,
                          timeout=300)
    assert done.returncode == 0 and "the same" in done.stdout, done.stderr[-2000:]
