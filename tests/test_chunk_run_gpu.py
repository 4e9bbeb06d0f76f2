"""A request's way through the calls as a server makes them: its prompt in chunks beside other requests that decode,
then decode steps over the pages and vectors that the chunks left."""
import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_a_prompt_in_chunks_then_decode_steps(dtype, d):
    Hq, Hkv, B = 8, 2, 3
    final = [1500, 700, 130]
    case = ref.Case([(0, n) for n in final], Hq, Hkv, d, dtype, seed=21, init=128, local=300)
    cfg = case.cfg
    g = torch.Generator(device=DEV).manual_seed(22)
    qkv = [torch.randn(n, Hq + 2 * Hkv, d, generator=g, device=DEV).to(dtype) for n in final]
    f = ref.freqs(d)
    buf = srkv.DecodeBuffers(cfg, B, case.max_blocks, case.pages)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    case.k.fill_(float("nan"))
    case.v.fill_(float("nan"))
    # what each step brings of every request: pieces of prompts, then single tokens; the last is a decode step
    steps = [[900, 0, 0], [1, 600, 0], [500, 1, 100], [98, 98, 29], [1, 1, 1]]
    at = [0] * B
    for step in steps:
        offsets = torch.tensor([0] + [sum(step[:i + 1]) for i in range(B)], dtype=torch.int32, device=DEV)
        new = torch.cat([x[a:a + n] for x, a, n in zip(qkv, at, step)])
        q, kn, vn = new.split((Hq, Hkv, Hkv), 1)
        q_rot = torch.zeros(len(new), Hq, d, dtype=dtype, device=DEV)
        srkv.append_kv_rope(cfg, q, kn, vn, f, case.k, case.v, case.table, offsets, lens, buf.reps, q_rot,
                            buf.error_flags)
        lens += offsets.diff()
        out, windowed = torch.zeros_like(q_rot), torch.zeros_like(q_rot)
        ws = torch.empty(srkv.chunk_workspace_size(cfg, len(new), B), dtype=torch.uint8, device=DEV)
        srkv.chunk_attention(cfg, q_rot, case.k, case.v, case.table, offsets, lens, out, ws, buf.error_flags)
        srkv.chunk_attention_window(cfg, q_rot, case.k, case.v, case.table, offsets, lens, windowed, ws,
                                    buf.error_flags)
        at = [a + n for a, n in zip(at, step)]
        assert at == lens.tolist() and int(buf.error_flags) == 0
        case.reqs, case.offsets, case.lens, case.q = [(n, 0) for n in step], offsets, lens, q_rot
        case.T = len(new)
        for got, window in ((out, False), (windowed, True)):
            want, tol = ref.attention(case, window)
            assert ((got.double() - want).abs() <= tol).all()
    # the vectors are those of a fresh build
    reps = torch.zeros_like(buf.reps)
    ids = torch.cat([case.table[r, :-(-n // 128)] for r, n in enumerate(final)])
    valid = torch.cat([torch.tensor([min(128, n - 128 * b) for b in range(-(-n // 128))]) for n in final])
    srkv.build_block_reps(cfg, case.k, ids, valid.int().to(DEV), reps)
    assert torch.equal(reps[ids.long()], buf.reps[ids.long()])
    # the last step was one token a request: the decode calls over the same cache say the same
    both = {}
    for name, topk in (("all", 1.0), ("none", 0.0)):
        c = dict(cfg, topk_percent=topk)
        b = srkv.DecodeBuffers(c, B, case.max_blocks, case.pages)
        srkv.retrieval_decode(c, q_rot, case.k, case.v, buf.reps, case.table, lens, None, b.sel, b.nsel, b.out,
                              b.workspace, b.error_flags)
        assert int(b.error_flags) == 0
        both[name] = b.out
    for got, dec, window in ((out, both["all"], False), (windowed, both["none"], True)):
        want, tol = ref.attention(case, window)
        assert ((got.double() - dec.double()).abs() <= 2 * tol).all()
