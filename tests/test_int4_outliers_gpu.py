"""The 4-bit decode where a few value rows are far larger than the rest and their keys leave them next to no weight:
the output is the other rows', at the accuracy it has without them."""
import pytest
import torch

import int4_exact as exact
import int4_ref as ref
from block_sparse_retrieval_gb300 import srkv, synth

pytestmark = pytest.mark.gpu

DEV = "cuda"
i32 = torch.int32


def outlier_case(batch, group, d, where, seed):
    """Queries of a common direction per kv head; keys of the outliers point against it (weights of about e^-70), their
    values are 1e9 times larger.  where: which tokens of a request are outliers."""
    H = 2
    case = synth.make_case(seq_lens=[1300 + 111 * (r % 5) for r in range(batch)], num_q_heads=H * group, num_kv_heads=H,
                           head_dim=d, init_tokens=256, local_tokens=512, topk_percent=1.0, dense_boundary=0,
                           device=DEV, seed=seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    base = torch.randn(H, d, generator=g, device=DEV)
    base *= d ** 0.5 / base.norm(dim=-1, keepdim=True)
    q = case.q.float().view(batch, H, group, d)
    case.q.copy_((2 * base[None, :, None] + 0.3 * q).reshape(batch, H * group, d))
    for r, L in enumerate(case.seq_lens.tolist()):
        for t in where(L):
            page = int(case.block_table[r, t // 128])
            case.k_cache[page, :, t % 128] = (-35.0 / d ** 0.5 * base).bfloat16()
            case.v_cache[page, :, t % 128] *= 1e9
    return case


WHERE = {
    "first-page": lambda L: range(128),         # met first: the references start at theirs
    "scattered": lambda L: range(0, L, 37),     # one in each 32 tokens or nearly
    "last": lambda L: range(L - 40, L),         # met last
}


@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("batch,group,d", [(1, 4, 128), (24, 4, 128), (1, 8, 128), (24, 8, 64), (24, 2, 64)])
def test_values_without_weight_cost_the_others_nothing(batch, group, d, where):
    case = outlier_case(batch, group, d, WHERE[where], 41)
    buf = srkv.DecodeBuffers(case.cfg, batch, case.max_blocks, case.num_pages, device=DEV)
    srkv.build_block_reps(case.cfg, case.k_cache, case.page_ids, case.page_valid, buf.reps)
    kv = torch.zeros(case.num_pages, 2, ref.slab_bytes(d), dtype=torch.uint8, device=DEV)
    srkv.quantize_kv_int4(case.cfg, case.k_cache, case.v_cache, torch.arange(case.num_pages, dtype=i32, device=DEV), kv)
    srkv.retrieval_decode_int4(case.cfg, case.q, kv, buf.reps, case.block_table, case.seq_lens, None, buf.sel, buf.nsel,
                               buf.out, buf.workspace, buf.error_flags)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    host, q, out = kv.cpu().numpy(), ref.host(case.q), ref.host(buf.out)
    table, L = case.block_table.cpu().numpy(), case.seq_lens.tolist()
    for r, h in {(0, 0), (batch // 2, 1), (batch - 1, 1)}:
        heads = slice(h * group, (h + 1) * group)
        want, bound = exact.decode_unit(q[r, heads], host, table[r], L[r],
                                        buf.sel[r, h, :int(buf.nsel[r, h])].tolist(), case.cfg, h)
        rms = (want ** 2).mean() ** 0.5
        assert rms < 10 and (bound < rms / 8).all()  # the outliers' values are of the order of 1e9
        err = abs(out[r, heads] - want)
        assert (err <= bound).all(), (r, h, float((err / bound).max()))
