"""The 4-bit decode held to bounds far below its outputs (int4_exact.py), to structured values whose sums are exact, and
its selection to scores in 64 bits."""
import numpy as np
import pytest
import torch

import int4_exact as exact
import int4_ref as ref
from block_sparse_retrieval_gb300 import srkv
from test_int4_gpu import CASES, int4_case, make, step

pytestmark = pytest.mark.gpu

DEV = "cuda"


def run(case, kv, buf):
    buf.out.fill_(float("nan"))
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0


def units(case):
    return [(r, h) for r in range(case.batch) for h in range(case.cfg["num_kv_heads"])]


def check(case, kv, buf, which=None, share=0.25):
    """The step's output within the bound of random data, and that bound within `share` of the output's size."""
    cfg = case.cfg
    G = cfg["num_q_heads"] // cfg["num_kv_heads"]
    host, q, out = kv.cpu().numpy(), ref.host(case.q), ref.host(buf.out)
    table, L = case.block_table.cpu().numpy(), case.seq_lens.tolist()
    sel, nsel = buf.sel.cpu().numpy(), buf.nsel.cpu().numpy()
    for r, h in which or units(case):
        heads = slice(h * G, (h + 1) * G)
        want, bound = exact.decode_unit(q[r, heads], host, table[r], L[r], sel[r, h, :nsel[r, h]], cfg, h, random=True)
        err = np.abs(out[r, heads] - want)
        assert (err <= bound).all(), (r, h, float((err / np.maximum(bound, 1e-300)).max()))
        assert np.median(bound) <= share * (want ** 2).mean() ** 0.5, (r, h)


@pytest.mark.parametrize("name", list(CASES))
def test_decode_within_a_bound_below_the_outputs(name):
    case = CASES[name]()
    kv, buf = int4_case(case)
    run(case, kv, buf)
    check(case, kv, buf)


@pytest.mark.parametrize("head_dim,group", [(64, 3), (64, 8), (128, 4), (128, 5)])
def test_long_dense_steps(head_dim, group):
    case = make(seq_lens=[30000 + 128 * i for i in range(24)], num_q_heads=2 * group, num_kv_heads=2, head_dim=head_dim,
                topk_percent=1.0, shared_prefix_tokens=8192, seed=115)
    kv, buf = int4_case(case)
    run(case, kv, buf)
    check(case, kv, buf, [(0, 1), (11, 0), (23, 1)])


@pytest.mark.parametrize("group", [4, 8])
@pytest.mark.parametrize("log_q,log_k,log_v", [(98, -98, 0), (-100, 100, 0), (14, -13, 60), (5, 0, -60), (0, 0, 95), (-20, 20, -96),
                                               (4, 0, 0), (-8, 0, 0)])
def test_magnitudes_to_the_documented_ends(group, log_q, log_k, log_v):
    """Queries to 2^101, keys to match, values to 2^98 and down to V scales of 2^-100, as accurate as at 1."""
    case = make(seq_lens=[3000, 2000] * (1 if group == 4 else 10), num_q_heads=2 * group, topk_percent=1.0, seed=137)
    for t, n in ((case.q, log_q), (case.k_cache, log_k), (case.v_cache, log_v)):
        t.mul_(2.0 ** n)
    kv, buf = int4_case(case)
    run(case, kv, buf)
    check(case, kv, buf, [(0, 0), (1, 1)], share=0.5)


# ---- every 32 tokens, once -----------------------------------------------------------------------------

COUNTS = {
    "layer": dict(seq_lens=[65536], num_q_heads=32, num_kv_heads=8, init_tokens=1024, local_tokens=7192),
    "all-of-two-odd": dict(seq_lens=[9999, 4001], num_q_heads=16, num_kv_heads=2, topk_percent=1.0),
    "kept-by-a-pool": dict(seq_lens=[131000], num_q_heads=2, num_kv_heads=1, topk_percent=0.9),
    "odd-bounds": dict(seq_lens=[3001, 2777, 4095, 130, 1, 0] * 5, init_tokens=77, local_tokens=333),
    "odd-bounds-wide": dict(seq_lens=[3001, 2777, 4095, 130, 1, 0] * 5, num_q_heads=14, init_tokens=77,
                            local_tokens=333, head_dim=64),
    "longest": dict(seq_lens=[25600 * 128 - 5], num_q_heads=4, num_kv_heads=1, topk_percent=1.0),
    "longest-wide": dict(seq_lens=[25600 * 128 - 5], num_q_heads=8, num_kv_heads=1, head_dim=64, topk_percent=0.7),
    "a-thousand": dict(seq_lens=[(37 * i) % 700 for i in range(1000)], init_tokens=100, local_tokens=130),
    "seventy": dict(seq_lens=[(97 * i) % 1500 for i in range(70)], num_q_heads=4, init_tokens=128, local_tokens=200),
    **{f"long-{d}-{g}": dict(seq_lens=[30000 + 128 * i for i in range(24)], num_q_heads=2 * g, head_dim=d, topk_percent=1.0)
       for d, g in ((64, 3), (64, 8), (128, 4), (128, 5))},
}


@pytest.mark.parametrize("name", list(COUNTS))
def test_every_attended_token_counts_once(name):
    """A query of zeros weighs all tokens alike.  Each 32 tokens of a page have a value in one element of their own (15
    times a power of two of the page: code 15, the others 0), so that the outputs are counts over the length: exact
    but for the division and the rounding to bf16.  A part of a page that is lost, doubled, misplaced or scaled as
    another's moves an element by a good part of itself."""
    case = make(**{"seed": 131, **COUNTS[name]})
    cfg, d, H = case.cfg, case.cfg["head_dim"], case.cfg["num_kv_heads"]
    case.q.zero_()
    case.v_cache.zero_()
    table, L = case.block_table.cpu().numpy(), case.seq_lens.tolist()
    w = torch.arange(4, device=DEV).repeat_interleave(32)
    for r, n in enumerate(L):
        nb = -(-n // 128)
        if nb == 0:
            continue
        pages = case.block_table[r, :nb].long()
        unit = 15.0 * 2.0 ** (pages % 3 - 1).double()
        for h in range(H):
            at = (torch.arange(nb, device=DEV)[:, None] * 4 + w + 5 * h + 11 * r) % d
            v = torch.zeros(nb, 128, d, device=DEV)
            v.scatter_(2, at[..., None], unit[:, None, None].float().expand(nb, 128, 1))
            case.v_cache[pages, h] = v.bfloat16()
    kv, buf = int4_case(case)
    run(case, kv, buf)
    out, sel, nsel = ref.host(buf.out).reshape(case.batch, H, -1, d), buf.sel.cpu().numpy(), buf.nsel.cpu().numpy()
    for r, n in enumerate(L):
        for h in range(H):
            on = exact.attended(cfg, n, sel[r, h, :nsel[r, h]])
            want = np.zeros(d)
            for b in range(len(on)):
                for g in range(4):
                    want[(b * 4 + g + 5 * h + 11 * r) % d] += on[b, 32 * g:32 * g + 32].sum() * 15 * 2.0 ** (table[r, b] % 3 - 1)
            want /= max(1, on.sum())
            assert (np.abs(out[r, h] - want) <= 2.0 ** -8 * (1 + 2.0 ** -10) * want).all(), (r, h)


# ---- one token each -------------------------------------------------------------------------------------

@pytest.mark.parametrize("batch", [1, 24])
@pytest.mark.parametrize("head_dim,group", [(64, 3), (64, 8), (128, 4), (128, 7)])
def test_a_query_along_one_key_finds_its_value(batch, head_dim, group):
    """Each head's query is six times some token's key, which then has all of the weight: keys, values and their rows
    belong together at every place of a page."""
    case = make(seq_lens=[5000 - 61 * r for r in range(batch)], num_q_heads=2 * group, num_kv_heads=2, head_dim=head_dim,
                topk_percent=1.0, seed=132)
    rng = np.random.default_rng(133)
    target = np.zeros((batch, 2 * group), int)
    for r, n in enumerate(case.seq_lens.tolist()):
        for j in range(2 * group):
            t = target[r, j] = (0, n - 1, int(rng.integers(n)))[min(2, (r + j) % 7)]
            case.q[r, j] = 6 * case.k_cache[int(case.block_table[r, t // 128]), j // group, t % 128]
    kv, buf = int4_case(case)
    run(case, kv, buf)
    host, q, out = kv.cpu().numpy(), ref.host(case.q), ref.host(buf.out)
    table = case.block_table.cpu().numpy()
    for r, n in enumerate(case.seq_lens.tolist()):
        for h in range(2):
            heads = slice(h * group, (h + 1) * group)
            rows = exact.gather(host, table[r], n, range(100), case.cfg, h, head_dim)
            want, bound = exact.attend(q[r, heads], rows)
            assert (np.abs(out[r, heads] - want) <= bound).all()
            K = rows[2][:, None] + rows[0] * rows[1][:, None]
            z = q[r, heads] @ K.T / np.sqrt(head_dim)
            for j in range(group):
                t = target[r, h * group + j]
                value = ref.values(host[table[r, t // 128], h], head_dim)[1][t % 128]
                # out = sum p V, so out - V_t = sum over the others of p (V - V_t): at most 1 - p_t of the
                # range of V, which lies within 12 (normal values)
                rest = 1 - 1 / np.exp(z[j] - z[j, t]).sum()
                assert rest < 0.05 and (np.abs(want[j] - value) <= 12 * rest + 1e-12).all() and bound[j].max() < 0.03


# ---- the selection ----------------------------------------------------------------------------------------

def check_selection(case, buf, tied=True):
    """sel and nsel against scores in 64 bits: the formula's count, ascending candidates, no kept score below a dropped
    one by more than the fp32 score's error, and among blocks on one page (equal vectors: equal scores) the lower ones."""
    cfg, d = case.cfg, case.cfg["head_dim"]
    H = cfg["num_kv_heads"]
    G = cfg["num_q_heads"] // H
    q = ref.host(case.q).reshape(case.batch, H, G, d)
    reps, table = buf.reps.double().cpu().numpy(), case.block_table.cpu().numpy()
    for r, L in enumerate(case.seq_lens.tolist()):
        W, lo = L - cfg["local_tokens"], cfg["init_tokens"] // 128
        n = -(-W // 128) - lo if W > cfg["init_tokens"] else 0
        k = min(n, int(np.ceil(cfg["topk_percent"] * n - 1e-9)))
        pages = table[r, lo:lo + n]
        for h in range(H):
            assert int(buf.nsel[r, h]) == k
            kept = buf.sel[r, h, :k].cpu().numpy() - lo
            assert (np.diff(kept) > 0).all() and (k == 0 or (kept[0] >= 0 and kept[-1] < n))
            if not 0 < k < n:
                continue
            on = np.isin(np.arange(n), kept)
            qs = q[r, h].sum(0)
            # the sum of G heads and the product of d, in fp32
            tol = (G + d + 8) * 2.0 ** -24 * (np.abs(q[r, h]).sum(0) @ np.abs(reps[pages, h]).max(0)) * 2
            s = reps[pages, h] @ qs
            assert s[on].min() >= s[~on].max() - tol, (r, h)
            for p in set(pages) if tied else ():
                mine = on[pages == p]
                assert (np.diff(mine.astype(int)) <= 0).all(), (r, h, p)


@pytest.mark.parametrize("batch,seq_len", [(1, 40000), (20, 40000), (5, 120000)])
@pytest.mark.parametrize("distinct", [1, 3, 40])
def test_equal_scores_keep_the_lower_blocks(batch, seq_len, distinct):
    """Blocks that share a few pages have equal scores; the steps score by clusters (one kernel), by 256 threads a CTA
    and, in the larger two, by 512."""
    case = make(seq_lens=[seq_len] * batch, topk_percent=0.37, shared_prefix_tokens=seq_len // 128 * 128, seed=134)
    case.k_cache += 3.0
    pages = case.block_table[:, :distinct].clone()
    case.block_table[:, 2:-4] = pages[:, torch.arange(case.max_blocks - 6, device=DEV) % distinct]
    kv, buf = int4_case(case)
    run(case, kv, buf)
    check_selection(case, buf)
    check(case, kv, buf, [(0, 0), (batch - 1, 1)], share=1)


@pytest.mark.parametrize("batch,seq_len", [(1, 60000), (3, 9000), (20, 50000), (70, 9000)])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_the_best_blocks_are_kept(batch, seq_len, head_dim):
    case = make(seq_lens=[seq_len - 77 * r for r in range(batch)], head_dim=head_dim, seed=135)
    kv, buf = int4_case(case)
    run(case, kv, buf)
    check_selection(case, buf, tied=False)
    check(case, kv, buf, [(0, 0), (batch - 1, 1)])


def test_the_bf16_step_keeps_the_lower_of_equal_blocks_too():
    """The scoring kernel of large shares behind the bf16 step."""
    case = make(seq_lens=[40000] * 20, topk_percent=0.37, shared_prefix_tokens=39936, seed=136)
    pages = case.block_table[:, :3].clone()
    case.block_table[:, 2:-4] = pages[:, torch.arange(case.max_blocks - 6, device=DEV) % 3]
    _, buf = int4_case(case)
    srkv.retrieval_decode(case.cfg, case.q, case.k_cache, case.v_cache, buf.reps, case.block_table, case.seq_lens, None,
                          buf.sel, buf.nsel, buf.out, buf.workspace, buf.error_flags)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    check_selection(case, buf)
