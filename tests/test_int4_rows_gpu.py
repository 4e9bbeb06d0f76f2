"""Rows at the ends of the number range in a 4-bit cache: only a row that is not finite, or whose range passes fp32,
is held as NaN; every other one reads back finite, within half a step, and is attended."""
import numpy as np
import pytest
import torch

import int4_exact as exact
import int4_ref as ref
from block_sparse_retrieval_gb300 import srkv, synth

pytestmark = pytest.mark.gpu

DEV = "cuda"
i32 = torch.int32
MAX = exact.BF16_MAX


def config(d):
    return dict(num_q_heads=2, num_kv_heads=1, head_dim=d, block_size=128, init_tokens=128, local_tokens=128,
                topk_percent=0.5, dense_boundary=0, dtype=srkv.BF16)


def rows_at_the_ends(d, seed):
    """128 rows [128][d] and which of them may be NaN: bounds (lowest, highest) of every kind, values between."""
    rng = np.random.default_rng(seed)
    pairs = [(-2.5e38, 0.0), (-3e38, 0.0), (-MAX, 0.0), (0.0, MAX), (-MAX, -MAX), (MAX, MAX), (-1.75e38, 1.5e38),
             (-1.6e38, 1.75e38), (-2.0 ** 127, 2.0 ** 127 - 2.0 ** 119), (0.05 * 2.0 ** 128, MAX),
             (0.03 * 2.0 ** 128, MAX), (2.0 ** 120, MAX), (-2.0 ** 122, MAX), (-3.3e38, -1e30), (-3.3e38, 1e37),
             (-MAX, MAX), (-2.0 ** 127, 2.0 ** 127), (-2e38, 2e38)]
    while len(pairs) < 128:  # the tops just below bf16's last value, where rounding the scale up reaches past it
        top = MAX - 2.0 ** 120 * int(rng.integers(0, 4))
        pairs.append((top - 2.0 ** rng.uniform(126, 128) * rng.uniform(0.9, 1), top))
    x = np.empty((128, d))
    for i, (a, b) in enumerate(pairs):
        x[i] = a + (b / 2 - a / 2) * 2 * rng.random(d)
        x[i, 0], x[i, d - 1] = a, b
    return ref.to_bf16(np.clip(x, -MAX, MAX))


@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_the_ends_of_the_range(d):
    cfg = config(d)
    x, y = rows_at_the_ends(d, 1), rows_at_the_ends(d, 2)
    k, v = (torch.tensor(a[None, None], device=DEV).bfloat16() for a in (x, y))
    kv = torch.zeros(1, 1, ref.slab_bytes(d), dtype=torch.uint8, device=DEV)
    ids = torch.zeros(1, dtype=i32, device=DEV)
    srkv.quantize_kv_int4(cfg, k, v, ids, kv)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    srkv.dequantize_kv_int4(cfg, kv, ids, ko, vo)
    one, reps = torch.zeros_like(kv), torch.zeros(1, 1, d, device=DEV)
    table = torch.zeros(1, 1, dtype=i32, device=DEV)
    for t in range(128):  # and the same rows as appended tokens
        srkv.append_kv_int4(cfg, k[:, :, t].contiguous(), v[:, :, t].contiguous(), one, table,
                            torch.tensor([t], dtype=i32, device=DEV), reps)
    torch.cuda.synchronize()
    exact.check_slab(kv[0, 0].cpu().numpy(), x, y, d)
    assert torch.equal(one, kv)
    for a, got in ((x, ref.host(ko[0, 0])), (y, ref.host(vo[0, 0]))):
        with np.errstate(over="ignore"):
            span = (a.max(-1).astype(np.float32) - a.min(-1).astype(np.float32)).astype(np.float64)
        finite = np.isfinite(span)
        assert finite.sum() > 60 and (~finite).sum() >= 2
        np.testing.assert_array_equal(np.isfinite(got).all(-1), finite)
        assert np.isnan(got[~finite]).all()
        # half a step of at most (1 + 2^-7) / 15 of the range; where the scale was taken one down, the top is
        # short of 15 of its gaps of 2^-7 (1 / 15 of the range each); the read-back's rounding
        step = span[finite] / 15
        tol = step[:, None] * (0.5 * (1 + 2.0 ** -7) + 15 * 2.0 ** -7) + 2.0 ** -8 * np.abs(a[finite])
        assert (np.abs(got[finite] / 2 - a[finite] / 2) <= tol / 2).all()


def test_a_step_over_keys_far_below_zero():
    """Keys from -2.5e38 up and a query small enough for logits of a few units: no output is NaN."""
    case = synth.make_case(seq_lens=[700], num_q_heads=4, num_kv_heads=1, head_dim=128, init_tokens=128,
                           local_tokens=256, topk_percent=0.5, dense_boundary=0, device=DEV, seed=31)
    g = torch.Generator(device=DEV).manual_seed(32)
    case.k_cache.copy_(-2.5e38 * torch.rand(case.k_cache.shape, generator=g, device=DEV))
    q = torch.randn(case.q.shape, generator=g, device=DEV)
    case.q.copy_((q - q.mean(-1, keepdim=True)) * 1e-38 * 4)
    buf = srkv.DecodeBuffers(case.cfg, 1, case.max_blocks, case.num_pages, device=DEV)
    buf.reps.copy_(case.k_cache.double().mean(2))  # (128 of these keys pass fp32's range when they are summed)
    kv = torch.zeros(case.num_pages, 1, ref.slab_bytes(128), dtype=torch.uint8, device=DEV)
    srkv.quantize_kv_int4(case.cfg, case.k_cache, case.v_cache, torch.arange(case.num_pages, dtype=i32, device=DEV), kv)
    srkv.retrieval_decode_int4(case.cfg, case.q, kv, buf.reps, case.block_table, case.seq_lens, None, buf.sel, buf.nsel,
                               buf.out, buf.workspace, buf.error_flags)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0 and torch.isfinite(buf.out).all()
    want, bound = ref.decode_unit(ref.host(case.q)[0], kv.cpu().numpy(), case.block_table[0].tolist(), 700,
                                  buf.sel[0, 0, :int(buf.nsel[0, 0])].tolist(), case.cfg, 0)
    # the limit that the rows' own half steps leave plays no part: both sides read the same slabs
    assert (np.abs(ref.host(buf.out)[0] - want) <= bound).all()
