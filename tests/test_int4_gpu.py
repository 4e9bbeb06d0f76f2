"""GPU tests of the 4-bit cache: pages compressed, read back, tokens appended, and the decode over
them, each against the 64-bit restatement in int4_ref.py."""
import numpy as np
import pytest
import torch

import int4_ref as ref
from block_sparse_retrieval_gb300 import srkv, synth

pytestmark = pytest.mark.gpu

DEV = "cuda"
i32 = torch.int32


def config(Hq=8, Hkv=2, d=128, **over):
    return dict(dict(num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, block_size=128, init_tokens=256,
                     local_tokens=512, topk_percent=0.2, dense_boundary=0, dtype=srkv.BF16), **over)


def flags():
    return torch.zeros(1, dtype=i32, device=DEV)


def cache(cfg, pages, fill=0):
    return torch.full((pages, cfg["num_kv_heads"], ref.slab_bytes(cfg["head_dim"])), fill,
                      dtype=torch.uint8, device=DEV)


def random_pages(cfg, pages, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (pages, cfg["num_kv_heads"], 128, cfg["head_dim"])
    gain = torch.rand(shape[3], generator=g, device=DEV) + 0.5
    k = torch.randn(shape, generator=g, device=DEV) * gain + torch.randn(shape[3], generator=g, device=DEV)
    return k.bfloat16(), torch.randn(shape, generator=g, device=DEV).bfloat16()


def special_rows(k):
    """Rows where the quantiser can go wrong, in page 0, head 0."""
    d = k.shape[-1]
    ramp = torch.arange(d, device=DEV) / (d - 1)
    rows = [torch.zeros(d), torch.full((d,), -3.25), 15 * ramp, 15.0 * (ramp > 0.5), 1e-30 * ramp - 2e-30,
            3e38 * ramp, -1e-3 - ramp, 256 + ramp * 2,
            torch.arange(d) % 16 / 2.0,                     # quotients on halves: scale 0.5
            torch.cat((torch.tensor([0.0, 30.0]), torch.arange(d - 2) % 31)),  # ties: scale 2
            torch.cat((torch.tensor([-1.0, 2.0]), torch.full((d - 2,), 2.0 ** -30)))]
    for i, r in enumerate(rows):
        k[0, 0, i] = r.to(DEV).bfloat16()
    n = len(rows)
    k[0, 0, n, 3] = float("nan")
    k[0, 0, n + 1, d - 1] = float("inf")
    k[0, 0, n + 2, 0] = -float("inf")
    k[0, 0, n + 3, 1], k[0, 0, n + 3, 2] = 3.3e38, -3.3e38  # the range passes fp32
    return n


def check_slab(slab, k, v, d):
    """A slab's words against the rows they came from, code for code."""
    kc, vc, ks, kl, vs, vl = ref.unpack(slab, d)
    for codes, scale, lo, x in ((kc, ks, kl, k), (vc, vs, vl, v)):
        c, s, m = ref.quantize_rows(x)
        np.testing.assert_array_equal(scale, s)
        np.testing.assert_array_equal(lo, m)
        np.testing.assert_array_equal(codes, c)


@pytest.mark.parametrize("d,Hkv", [(128, 1), (128, 3), (64, 1), (64, 5)])
def test_quantizer_matches_the_definition_code_for_code(d, Hkv):
    cfg = config(Hq=Hkv, Hkv=Hkv, d=d)
    k, v = random_pages(cfg, 3, 1)
    special_rows(k)
    special_rows(v)
    kv, f = cache(cfg, 3), flags()
    srkv.quantize_kv_int4(cfg, k, v, torch.arange(3, dtype=i32, device=DEV), kv, None, f)
    torch.cuda.synchronize()
    assert int(f.item()) == 0
    got, kh, vh = kv.cpu().numpy(), ref.host(k), ref.host(v)
    for p in range(3):
        for h in range(Hkv):
            check_slab(got[p, h], kh[p, h], vh[p, h], d)


@pytest.mark.parametrize("d", [64, 128])
def test_pages_go_where_the_ids_say_and_bad_ids_are_flagged(d):
    cfg = config(d=d)
    k, v = random_pages(cfg, 6, 2)
    kv = cache(cfg, 9, 0x5A)
    src = torch.tensor([4, 6, 0, 2, -1, 5], dtype=i32, device=DEV)   # 6 and -1 are outside
    dst = torch.tensor([8, 1, 9, 0, 3, 6], dtype=i32, device=DEV)    # 9 is outside
    f = flags()
    srkv.quantize_kv_int4(cfg, k, v, src, kv, dst, f)
    torch.cuda.synchronize()
    assert int(f.item()) == srkv.EFLAG_PAGE_RANGE
    got, kh, vh = kv.cpu().numpy(), ref.host(k), ref.host(v)
    written = {8: 4, 0: 2, 6: 5}
    for p in range(9):
        for h in range(2):
            if p in written:
                check_slab(got[p, h], kh[written[p], h], vh[written[p], h], d)
            else:
                assert (got[p, h] == 0x5A).all()
    # and back into other pages of another pair of caches
    ko = torch.full((5, 2, 128, d), 7.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    f = flags()
    srkv.dequantize_kv_int4(cfg, kv, torch.tensor([8, 0, 9, 6], dtype=i32, device=DEV), ko, vo,
                            torch.tensor([1, 5, 2, 4], dtype=i32, device=DEV), f)
    torch.cuda.synchronize()
    assert int(f.item()) == srkv.EFLAG_PAGE_RANGE
    for p, s in ((1, 8), (4, 6)):
        for h in range(2):
            kx, vx = ref.values(got[s, h], d)
            np.testing.assert_array_equal(ref.host(ko[p, h]), ref.to_bf16(kx))
            np.testing.assert_array_equal(ref.host(vo[p, h]), ref.to_bf16(vx))
    assert (ko[[0, 2, 3]] == 7).all() and (vo[[0, 2, 3]] == 7).all()


def test_rows_that_are_not_finite_read_back_as_nan():
    cfg = config(Hq=1, Hkv=1)
    k, v = random_pages(cfg, 1, 3)
    n = special_rows(k)
    ids, kv = torch.zeros(1, dtype=i32, device=DEV), cache(cfg, 1)
    srkv.quantize_kv_int4(cfg, k, v, ids, kv)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    srkv.dequantize_kv_int4(cfg, kv, ids, ko, vo)
    torch.cuda.synchronize()
    bad = torch.isnan(ko[0, 0]).all(-1).cpu()
    assert bad.tolist() == [n <= t < n + 4 for t in range(128)]
    assert torch.isfinite(vo).all()
    # half a step of the row's scale (at most (max - min) / 15 * (1 + 2^-7)), and the read-back's rounding
    good = ~bad
    good[4:6] = False  # rows of ranges where the bound's own arithmetic under- or overflows
    x, y = ref.host(k[0, 0])[good.numpy()], ref.host(ko[0, 0])[good.numpy()]
    step = (x.max(-1) - x.min(-1)) / 15 * (1 + 2.0 ** -7)
    assert (np.abs(x - y) <= step[:, None] / 2 + 2.0 ** -8 * np.abs(y) + 2.0 ** -23 * np.abs(x)).all()


def test_rows_of_nearly_one_value_are_held_as_their_minimum():
    """Ranges around 2^-122, where the scale passes 2^-126: codes 0 below it, codes of the definition above.
    All values are multiples of 2^-133, bf16's smallest, so nothing here rounds."""
    cfg = config()
    k, _ = random_pages(cfg, 1, 7)
    steps = torch.randint(0, 16, k.shape, generator=torch.Generator().manual_seed(8)).to(DEV)
    steps[..., 0], steps[..., 1] = 0, 15
    unit = 2.0 ** torch.randint(-133, -120, k.shape[:3], generator=torch.Generator().manual_seed(9)).double()
    k = (steps.double() * unit.to(DEV)[..., None]).bfloat16()
    kv = cache(cfg, 1)
    srkv.quantize_kv_int4(cfg, k, k, torch.zeros(1, dtype=i32, device=DEV), kv)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    srkv.dequantize_kv_int4(cfg, kv, torch.zeros(1, dtype=i32, device=DEV), ko, vo)
    torch.cuda.synchronize()
    small = (unit < 2.0 ** -126)[..., None].to(DEV)  # 15 steps of `unit`: the scale is `unit`
    want = torch.where(small, torch.zeros_like(k), k)
    assert small.any() and not small.all()
    assert torch.equal(ko, want) and torch.equal(vo, want)


def test_empty_lists_and_batches_do_nothing():
    cfg = config()
    k, v = random_pages(cfg, 2, 4)
    kv = cache(cfg, 2, 0x11)
    none = torch.zeros(0, dtype=i32, device=DEV)
    srkv.quantize_kv_int4(cfg, k, v, none, kv)
    srkv.dequantize_kv_int4(cfg, kv, none, k, v)
    before = k.clone()
    e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)
    srkv.append_kv_int4(cfg, e(0, 2, 128), e(0, 2, 128), kv, e(0, 4, dt=i32), e(0, dt=i32),
                        e(2, 2, 128, dt=torch.float32))
    torch.cuda.synchronize()
    assert (kv == 0x11).all() and torch.equal(k, before)


@pytest.mark.parametrize("d,Hkv", [(128, 8), (128, 3), (64, 2)])
def test_appended_tokens_equal_quantised_pages_and_keep_the_vectors(d, Hkv):
    """Tokens appended one by one give the page that compressing the whole page gives (rows not
    yet written keep what they held), and the vector is the mean of the keys as held."""
    cfg = config(Hq=Hkv, Hkv=Hkv, d=d)
    B, max_blocks, P = 3, 3, 12
    lens = [0, 126, 250]  # the first token; across a page's end; inside a page
    table = torch.tensor([[7, 2, 9], [0, 5, 3], [11, 4, 8]], dtype=i32, device=DEV)
    k, v = random_pages(cfg, P, 5)
    kv = cache(cfg, P, 0x37)
    reps = torch.full((P, Hkv, d), -5.0, device=DEV)
    before = kv.cpu().numpy().copy()
    f, n_new = flags(), 9
    L = torch.tensor(lens, dtype=i32, device=DEV)
    written = {}
    for step in range(n_new):
        src = [(int(table[r, (lens[r] + step) // 128]), (lens[r] + step) % 128) for r in range(B)]
        kn = torch.stack([k[p, :, t] for p, t in src])
        vn = torch.stack([v[p, :, t] for p, t in src])
        srkv.append_kv_int4(cfg, kn, vn, kv, table, L, reps, f)
        for p, t in src:
            written.setdefault(p, []).append(t)
        L += 1
    torch.cuda.synchronize()
    assert int(f.item()) == 0
    got, kh, vh = kv.cpu().numpy(), ref.host(k), ref.host(v)
    for p in range(P):
        rows = written.get(p, [])
        for h in range(Hkv):
            now, was = ref.unpack(got[p, h], d), ref.unpack(before[p, h], d)
            others = [t for t in range(128) if t not in rows]
            for a, b in zip(now, was):
                np.testing.assert_array_equal(a[others], b[others])
            if not rows:
                assert (reps[p, h] == -5).all()
                continue
            for i, x in ((0, kh), (1, vh)):
                c, s, m = ref.quantize_rows(x[p, h, rows])
                np.testing.assert_array_equal(now[i][rows], c)
                np.testing.assert_array_equal(now[2 + 2 * i][rows], s)
                np.testing.assert_array_equal(now[3 + 2 * i][rows], m)
            held = ref.values(got[p, h], d)[0][:max(rows) + 1]
            want = held.mean(0)
            # n fp32 additions, the row values' and the quotient's rounding: (n + 2) 2^-24 of the sum
            tol = (len(held) + 2) * 2.0 ** -24 * np.abs(held).mean(0)
            assert (np.abs(reps[p, h].double().cpu().numpy() - want) <= tol).all(), (p, h)


def test_a_token_written_again_gives_the_same_cache():
    cfg = config(d=128)
    k, v = random_pages(cfg, 4, 6)
    table = torch.tensor([[3, 1]], dtype=i32, device=DEV)
    kv, reps = cache(cfg, 4), torch.zeros(4, 2, 128, device=DEV)
    ids = torch.arange(4, dtype=i32, device=DEV)
    srkv.quantize_kv_int4(cfg, k, v, ids, kv)
    L = torch.tensor([200], dtype=i32, device=DEV)
    put = lambda t: srkv.append_kv_int4(cfg, k[0, :, t][None].contiguous(), v[0, :, t][None].contiguous(),
                                        kv, table, L, reps)
    put(11)
    torch.cuda.synchronize()
    first, vec = kv.clone(), reps.clone()
    put(12)  # a draft token, refused: the length stays and another takes its place
    put(11)
    torch.cuda.synchronize()
    assert torch.equal(kv, first) and torch.equal(reps, vec)


def test_append_outside_the_table_or_the_cache_is_flagged_and_writes_nothing():
    cfg = config()
    kv, reps = cache(cfg, 4, 0x77), torch.full((4, 2, 128), 3.0, device=DEV)
    kn = torch.randn(4, 2, 128, device=DEV).bfloat16()
    table = torch.tensor([[0, 1], [2, 3], [4, 1], [1, -1]], dtype=i32, device=DEV)
    lens = torch.tensor([256, -1, 5, 130], dtype=i32, device=DEV)  # past the table; negative; pages 4, -1
    f = flags()
    srkv.append_kv_int4(cfg, kn, kn, kv, table, lens, reps, f)
    torch.cuda.synchronize()
    assert int(f.item()) == srkv.EFLAG_SEQ_LEN | srkv.EFLAG_PAGE_RANGE
    assert (kv == 0x77).all() and (reps == 3).all()


# ---- the decode ------------------------------------------------------------------------------------

def int4_case(case):
    """A synthetic case with its pages compressed, and the vectors of the bf16 keys."""
    buf = srkv.DecodeBuffers(case.cfg, case.batch, case.max_blocks, case.num_pages, device=DEV)
    srkv.build_block_reps(case.cfg, case.k_cache, case.page_ids, case.page_valid, buf.reps)
    kv = cache(case.cfg, case.num_pages)
    ids = torch.arange(case.num_pages, dtype=i32, device=DEV)
    srkv.quantize_kv_int4(case.cfg, case.k_cache, case.v_cache, ids, kv)
    return kv, buf


def step(case, kv, buf, q=None):
    srkv.retrieval_decode_int4(case.cfg, case.q if q is None else q, kv, buf.reps, case.block_table,
                               case.seq_lens, case.prompt_lens, buf.sel, buf.nsel, buf.out,
                               buf.workspace, buf.error_flags)


def check(case, kv, buf, q=None, units=None):
    """The step's output against the 64-bit restatement with the step's own selection."""
    cfg = case.cfg
    Hkv, d = cfg["num_kv_heads"], cfg["head_dim"]
    G = cfg["num_q_heads"] // Hkv
    host, qh = kv.cpu().numpy(), ref.host(case.q if q is None else q)
    bt, L = case.block_table.cpu().numpy(), case.seq_lens.tolist()
    sel, nsel, out = buf.sel.cpu().numpy(), buf.nsel.cpu().numpy(), ref.host(buf.out)
    worst = 0.0
    for r, h in units or [(r, h) for r in range(case.batch) for h in range(Hkv)]:
        want, bound = ref.decode_unit(qh[r, h * G:(h + 1) * G], host, bt[r], L[r],
                                      sel[r, h, :nsel[r, h]], cfg, h)
        err = np.abs(out[r, h * G:(h + 1) * G] - want)
        assert (err <= bound).all(), (r, h, float((err / np.maximum(bound, 1e-300)).max()))
        worst = max(worst, float((err / np.maximum(bound, 1e-300)).max()))
    return worst


def same_selection(case, buf):
    """The step keeps the blocks that srkv_score_topk keeps."""
    other = srkv.DecodeBuffers(case.cfg, case.batch, case.max_blocks, case.num_pages, device=DEV)
    srkv.score_topk(case.cfg, case.q, buf.reps, case.block_table, case.seq_lens, case.prompt_lens,
                    other.sel, other.nsel)
    torch.cuda.synchronize()
    assert torch.equal(other.nsel, buf.nsel) and torch.equal(other.sel, buf.sel)


def make(**kw):
    base = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, init_tokens=256, local_tokens=512,
                topk_percent=0.2, dense_boundary=0, device=DEV)
    return synth.make_case(**{**base, **kw})


CASES = {
    "llama8b-16k": lambda: synth.llama8b_layer(seq_len=16384, device=DEV, seed=81),
    "ragged-5": lambda: synth.ragged_batch(n_requests=5, lo=9000, hi=14000, device=DEV, seed=82),
    "short-and-empty": lambda: make(seq_lens=[700, 1, 0, 129, 130, 1030, 5000], init_tokens=1024,
                                    local_tokens=1024, seed=83),
    "one-token": lambda: make(seq_lens=[1], seed=84),
    "empty-but-one": lambda: make(seq_lens=[0, 0, 0, 5], extra_blocks=2, seed=85),
    "odd-bounds": lambda: make(seq_lens=[3001, 2777, 4095], init_tokens=77, local_tokens=333, seed=86),
    "no-init-no-window": lambda: make(seq_lens=[2560, 1999], init_tokens=0, local_tokens=0,
                                      topk_percent=0.4, seed=87),
    "nothing-attended": lambda: make(seq_lens=[2560], init_tokens=0, local_tokens=0, topk_percent=0.0,
                                     seed=88),
    "dense": lambda: make(seq_lens=[5000, 900], dense_boundary=32768, seed=89),
    "group-1": lambda: make(seq_lens=[4000] * 3, num_q_heads=3, num_kv_heads=3, seed=90),
    "group-3-many-units": lambda: make(seq_lens=[2000, 3000, 2500] * 8, num_q_heads=15, num_kv_heads=5,
                                       seed=91),
    "group-8": lambda: make(seq_lens=[6000, 2222], num_q_heads=16, num_kv_heads=2, seed=92),
    "d64-one-kernel": lambda: make(seq_lens=[7000], num_q_heads=4, num_kv_heads=1, head_dim=64, seed=93),
    "d64-group-7": lambda: make(seq_lens=[3000, 0, 257, 4444] * 5, num_q_heads=14, num_kv_heads=2,
                                head_dim=64, init_tokens=100, local_tokens=300, seed=94),
    "shared-prefix": lambda: make(seq_lens=[2000, 3000], shared_prefix_tokens=1024, seed=95),
    "d64-group-6-one-kernel": lambda: make(seq_lens=[5000, 3333], num_q_heads=6, num_kv_heads=1,
                                           head_dim=64, seed=105),
    "group-5": lambda: make(seq_lens=[5000, 77], num_q_heads=10, num_kv_heads=2, seed=106),
    "group-2-seventy-requests": lambda: make(seq_lens=[(97 * i) % 1500 for i in range(70)], num_q_heads=4,
                                             num_kv_heads=2, init_tokens=128, local_tokens=200, seed=107),
    # prompts on both sides of the dense boundary, several requests to a lane of the plan
    "prompts-around-the-boundary": lambda: make(seq_lens=[900 + 71 * (i % 23) for i in range(45)],
                                                prompt_lens=[700 + 40 * (i % 17) for i in range(45)],
                                                dense_boundary=1000, seed=117),
    # more kept blocks than go out with the selection: the rest from the shared pool
    "long-mostly-kept": lambda: make(seq_lens=[131000], num_q_heads=2, num_kv_heads=1,
                                     topk_percent=0.9, seed=108),
    # more candidates than the one-kernel path takes
    "longer-than-one-kernel": lambda: make(seq_lens=[150000], num_q_heads=2, num_kv_heads=1,
                                           head_dim=64, topk_percent=0.1, seed=109),
}


@pytest.mark.parametrize("name", list(CASES))
def test_decode_matches_64_bits(name):
    case = CASES[name]()
    kv, buf = int4_case(case)
    buf.out.fill_(float("nan"))
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    same_selection(case, buf)
    check(case, kv, buf)


@pytest.mark.parametrize("batch", [1, 20])
@pytest.mark.parametrize("distinct", [1, 3, 40])
def test_scores_that_are_equal_or_close_keep_the_lower_blocks(batch, distinct):
    """Blocks that share a few pages have equal scores (hundreds in one bin of any digit), and keys with a
    large common part scores that agree in their top bits."""
    case = make(seq_lens=[40000] * batch, topk_percent=0.37, seed=110)
    case.k_cache += 3.0
    pages = case.block_table[:, :distinct].clone()
    case.block_table[:, 2:-4] = pages[:, torch.arange(case.max_blocks - 6, device=DEV) % distinct]
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    same_selection(case, buf)
    check(case, kv, buf, units=[(0, 0), (batch - 1, 1)])


def test_a_cache_past_32_bit_offsets():
    """The last pages of a cache of more than 2^32 bytes: written, appended to, read back, attended."""
    cfg = config(Hq=32, Hkv=8, init_tokens=128, local_tokens=128)
    P = (1 << 32) // (8 * 17408) + 200
    kv = torch.empty(P, 8, 17408, dtype=torch.uint8, device=DEV)
    assert kv.numel() > 1 << 32
    n = 12
    k, v = random_pages(cfg, n, 111)
    ids = torch.arange(n, dtype=i32, device=DEV)
    top = (P - 1 - ids).contiguous()
    srkv.quantize_kv_int4(cfg, k, v, ids, kv, top)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    L = torch.tensor([n * 128 - 30], dtype=i32, device=DEV)
    table = top.view(1, n).contiguous()
    reps = torch.zeros(P, 8, 128, device=DEV)
    reps[top.long()] = k.float().mean(2)
    srkv.append_kv_int4(cfg, k[:1, :, 3].contiguous(), v[:1, :, 3].contiguous(), kv, table, L, reps)
    srkv.dequantize_kv_int4(cfg, kv, top, ko, vo, ids)
    buf = srkv.DecodeBuffers(cfg, 1, n, 1, device=DEV)
    q = random_pages(cfg, 1, 112)[0][:, :, :4].reshape(1, 32, 128).contiguous()
    L += 1
    srkv.retrieval_decode_int4(cfg, q, kv, reps, table, L, None, buf.sel, buf.nsel, buf.out, buf.workspace,
                               buf.error_flags)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    got = kv[top.long()].cpu().numpy()
    kh, vh = ref.host(k), ref.host(v)
    row = n * 128 - 30
    kh[n - 1, :, row % 128], vh[n - 1, :, row % 128] = kh[0, :, 3], vh[0, :, 3]
    for p in (0, n - 1):
        for h in range(8):
            check_slab(got[p, h], kh[p, h], vh[p, h], 128)
            np.testing.assert_array_equal(ref.host(ko[p, h]), ref.to_bf16(ref.values(got[p, h], 128)[0]))
    sel, nsel = buf.sel.cpu().numpy(), buf.nsel.cpu().numpy()
    for h in (0, 7):
        want, bound = ref.decode_unit(ref.host(q)[0, 4 * h:4 * h + 4], got, np.arange(n), row + 1,
                                      sel[0, h, :nsel[0, h]], cfg, h)
        assert (np.abs(ref.host(buf.out)[0, 4 * h:4 * h + 4] - want) <= bound).all()


@pytest.mark.parametrize("head_dim,group", [(64, 3), (64, 8), (128, 4), (128, 5)])
def test_long_dense_steps_repeat_bit_for_bit(head_dim, group):
    """Rings that turn over hundreds of times, every group size's: the three-kernel path gives the same
    bits on every call, and those of the definition."""
    case = make(seq_lens=[30000 + 128 * i for i in range(24)], num_q_heads=2 * group, num_kv_heads=2,
                head_dim=head_dim, topk_percent=1.0, shared_prefix_tokens=8192, seed=115)
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    first = buf.out.clone()
    check(case, kv, buf, units=[(0, 1), (23, 0)])
    for _ in range(50):
        step(case, kv, buf)
        assert torch.equal(buf.out, first)
    assert int(buf.error_flags.item()) == 0


def test_two_streams_at_once():
    """Two requests' steps on two streams over one cache, each with buffers of its own, against the same
    steps one after the other."""
    cases = [make(seq_lens=[9000, 4000], seed=113), make(seq_lens=[6000, 2000] * 12, seed=114)]
    sets = [(c, *int4_case(c)) for c in cases]
    want = []
    for c, kv, buf in sets:
        step(c, kv, buf)
        torch.cuda.synchronize()
        want.append(buf.out.clone())
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (c, kv, buf), s in zip(sets, streams):
            with torch.cuda.stream(s):
                step(c, kv, buf)
    torch.cuda.synchronize()
    for (c, kv, buf), w in zip(sets, want):
        assert int(buf.error_flags.item()) == 0 and torch.equal(buf.out, w)


def test_streams_given_by_hand_and_no_flags():
    """Every call with a stream object, then with its handle, neither of them current, and no error flags."""
    case = make(seq_lens=[2000, 1500], seed=118)
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    want, pages = buf.out.clone(), kv.clone()
    ids = torch.arange(case.num_pages, dtype=i32, device=DEV)
    new = case.k_cache[:2, :, 5].contiguous()
    at = case.seq_lens.clone()  # the last blocks have room
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        kv.zero_(), buf.out.zero_()
        k, v = torch.zeros_like(case.k_cache), torch.zeros_like(case.v_cache)
        torch.cuda.synchronize()
        srkv.quantize_kv_int4(case.cfg, case.k_cache, case.v_cache, ids, kv, stream=stream)
        srkv.retrieval_decode_int4(case.cfg, case.q, kv, buf.reps, case.block_table, case.seq_lens,
                                   case.prompt_lens, buf.sel, buf.nsel, buf.out, buf.workspace,
                                   stream=stream)
        s.synchronize()
        # (the one-kernel path's fp32 sums may differ in order: a step of bf16, 2^-7, where they round apart)
        assert torch.equal(kv, pages) and torch.allclose(buf.out.float(), want.float(), rtol=2.0 ** -7, atol=1e-3)
        reps = buf.reps.clone()
        torch.cuda.synchronize()
        srkv.append_kv_int4(case.cfg, new, new, kv, case.block_table, at, reps, stream=stream)
        srkv.dequantize_kv_int4(case.cfg, kv, ids, k, v, stream=stream)
        s.synchronize()
        for r in range(2):
            L = int(at[r])
            row = k[int(case.block_table[r, L // 128]), :, L % 128].float()
            step_of = (new[r].float().amax(-1) - new[r].float().amin(-1)) / 15
            # half a step of codes, the scale's rounding over 15 codes, and a rounding to bf16
            assert ((row - new[r].float()).abs() <= (step_of * (0.5 + 2.0 ** -7 * 8))[:, None]
                    + 2.0 ** -8 * new[r].float().abs().amax(-1, keepdim=True)).all()


def test_two_graphs_over_one_workspace():
    """Steps of two batches captured with the same workspace, replayed in turn on one stream."""
    cases = [make(seq_lens=[3000, 1234] * 12, seed=119), make(seq_lens=[2500, 0, 129] * 9, seed=120)]
    sets = [(c, *int4_case(c)) for c in cases]
    shared = max((b.workspace for _, _, b in sets), key=lambda t: t.numel())
    want, graphs = [], []
    s = torch.cuda.Stream()
    for c, kv, buf in sets:
        buf.workspace = shared
        step(c, kv, buf)
        torch.cuda.synchronize()
        want.append(buf.out.clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            step(c, kv, buf)
    for _ in range(10):
        for _, _, buf in sets:
            buf.out.fill_(float("nan"))
        for g in graphs:
            g.replay()
        for (_, _, buf), w in zip(sets, want):
            assert torch.equal(buf.out, w)


@pytest.mark.parametrize("prefix", [False, True])
def test_pages_read_back_feed_the_full_precision_calls(prefix):
    """Read back into bf16 pages and attended there at once, with nothing between the launches: the bits of
    the same calls with the stream waited for in between."""
    case = make(seq_lens=[5000 + 64 * i for i in range(12)], num_q_heads=16, num_kv_heads=4,
                shared_prefix_tokens=2048, seed=121)
    kv, _ = int4_case(case)
    buf = srkv.DecodeBuffers(case.cfg, case.batch, case.max_blocks, case.num_pages, device=DEV, prefix=True)
    srkv.build_block_reps(case.cfg, case.k_cache, case.page_ids, case.page_valid, buf.reps)
    ids = torch.arange(case.num_pages, dtype=i32, device=DEV)
    k, v = torch.empty_like(case.k_cache), torch.empty_like(case.v_cache)

    def run(wait):
        k.zero_(), v.zero_()
        srkv.dequantize_kv_int4(case.cfg, kv, ids, k, v, error_flags=buf.error_flags)
        if wait:
            torch.cuda.synchronize()
        if prefix:
            srkv.retrieval_decode_prefix(case.cfg, case.q, k, v, buf.reps, case.block_table, case.seq_lens,
                                         None, 16, buf.sel, buf.nsel, buf.out, buf.workspace,
                                         buf.error_flags)
        else:
            srkv.sparse_paged_decode(case.cfg, case.q, k, v, case.block_table, case.seq_lens, buf.sel,
                                     buf.nsel, buf.out, buf.workspace, buf.error_flags)
        return buf.out.clone()

    srkv.score_topk(case.cfg, case.q, buf.reps, case.block_table, case.seq_lens, None, buf.sel, buf.nsel)
    want = run(True)
    assert torch.isfinite(want).all() and (want != 0).any()
    for _ in range(10):
        assert torch.equal(run(False), want)
    assert int(buf.error_flags.item()) == 0


def test_a_cache_without_pages_is_refused():
    case = make(seq_lens=[0, 0, 0], extra_blocks=2, seed=85)
    assert case.num_pages == 0
    kv, buf = int4_case(case)
    with pytest.raises(srkv.SrkvError, match="invalid argument"):
        step(case, kv, buf)


def test_rows_that_are_not_attended_never_reach_the_output():
    """NaN rows (scale and minimum NaN) wherever nothing is attended: behind the last token, in
    blocks that are not kept, and in the part of a kept block outside the offload range."""
    for seq_lens, kw in (([3001, 1500], dict(init_tokens=77, local_tokens=333)),
                         ([2000, 2100] * 12, dict(num_q_heads=16, num_kv_heads=4))):
        case = make(seq_lens=seq_lens, seed=96, **kw)
        kv, buf = int4_case(case)
        step(case, kv, buf)
        torch.cuda.synchronize()
        want = buf.out.clone()
        d, Hkv = case.cfg["head_dim"], case.cfg["num_kv_heads"]
        sel, nsel = buf.sel.cpu().numpy(), buf.nsel.cpu().numpy()
        rows = kv[:, :, 128 * d:].view(torch.bfloat16).view(-1, Hkv, 2, 128, 2)
        INIT, LOCAL = case.cfg["init_tokens"], case.cfg["local_tokens"]
        for r, L in enumerate(seq_lens):
            for b in range(-(-L // 128)):
                page = int(case.block_table[r, b])
                t = np.arange(b * 128, b * 128 + 128)
                for h in range(Hkv):
                    kept = b in sel[r, h, :nsel[r, h]]
                    on = ((t < INIT) | (t >= L - LOCAL) | kept) & (t < L)
                    rows[page, h, :, torch.from_numpy(~on).to(DEV)] = float("nan")
        buf.out.zero_()
        step(case, kv, buf)
        torch.cuda.synchronize()
        assert torch.isfinite(buf.out).all()
        if case.batch * Hkv > 36:  # three kernels: the same bits
            assert torch.equal(buf.out, want)
        check(case, kv, buf)


def test_an_attended_nan_row_makes_its_head_nan():
    for batch, kernels in ((1, 1), (24, 3)):
        case = make(seq_lens=[1500] * batch, seed=97)
        assert srkv.retrieval_decode_launches(case.cfg, batch, case.max_blocks) == kernels
        page = int(case.block_table[0, 0])
        case.v_cache[page, 1, 5, 3] = float("inf")
        kv, buf = int4_case(case)
        step(case, kv, buf)
        torch.cuda.synchronize()
        out = buf.out.view(batch, 2, 4, 128)
        assert torch.isnan(out[0, 1]).all()
        rest = torch.ones(batch, 2, dtype=torch.bool, device=DEV)
        rest[0, 1] = False
        assert torch.isfinite(out[rest]).all()


def test_a_request_of_nan_rows_alone_is_nan():
    for batch in (1, 24):
        case = make(seq_lens=[1] + [1500] * (batch - 1), seed=98)
        case.k_cache[int(case.block_table[0, 0])] = float("nan")
        kv, buf = int4_case(case)
        step(case, kv, buf)
        torch.cuda.synchronize()
        assert torch.isnan(buf.out[0]).all() and torch.isfinite(buf.out[1:]).all()


@pytest.mark.parametrize("group", [4, 8])
def test_a_query_that_is_not_finite_is_its_heads_own(group):
    case = make(seq_lens=[1500] * 2, num_q_heads=2 * group, topk_percent=1.0, seed=116)
    case.q[0, group + 1, 5], case.q[1, 2, 0] = float("inf"), float("nan")
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    bad = torch.zeros(2, 2 * group, dtype=torch.bool, device=DEV)
    bad[0, group + 1] = bad[1, 2] = True
    assert torch.isnan(buf.out[bad]).all() and torch.isfinite(buf.out[~bad]).all()
    case.q[0, group + 1, 5] = case.q[1, 2, 0] = 0
    kv, other = int4_case(case)
    step(case, kv, other)
    torch.cuda.synchronize()
    assert torch.equal(other.out[~bad], buf.out[~bad])
    check(case, kv, other)


@pytest.mark.parametrize("scale_q,scale_k,scale_v", [(1e4, 1e-4, 1.0), (1e-6, 1e6, 1e5), (1.0, 1.0, 1e-6),
                                                     (1.0, 1.0, 1e9), (30.0, 1.0, 1.0), (1.0, 1.0, 1e30),
                                                     (1.0, 1.0, 1e-29), (1e-30, 1e30, 1.0), (1e29, 1e-29, 1.0)])
def test_magnitudes(scale_q, scale_k, scale_v):
    """Queries, keys and values far from 1, and logits that leave a few tokens all the weight."""
    case = make(seq_lens=[3000, 2000], seed=99)
    case.q.mul_(scale_q)
    case.k_cache.mul_(scale_k)
    case.v_cache.mul_(scale_v)
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    check(case, kv, buf)


def test_value_scales_that_differ_between_tokens():
    """Small and constant value rows (scale 0) among large ones: the weights' reference follows
    weight times scale."""
    case = make(seq_lens=[2500] * 2, seed=100)
    case.v_cache[:, :, ::3] *= 1e-5
    case.v_cache[:, :, 1::7] = 0.75
    case.v_cache[:, :, 5::50] *= 1e4
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    check(case, kv, buf)


def test_constant_rows_alone():
    case = make(seq_lens=[600, 300], seed=101)
    case.k_cache.fill_(0.5)
    case.v_cache.fill_(-2.5)
    kv, buf = int4_case(case)
    step(case, kv, buf)
    torch.cuda.synchronize()
    assert (buf.out == -2.5).all()


def test_bad_pages_lengths_are_flagged_as_in_the_other_calls():
    case = make(seq_lens=[3000, 2000], seed=102)
    kv, buf = int4_case(case)
    case.block_table[0, 1] = case.num_pages  # an initial page outside the cache: skipped
    case.seq_lens[1] = case.max_blocks * 128 + 7
    step(case, kv, buf)
    torch.cuda.synchronize()
    got = int(buf.error_flags.item())
    assert got & srkv.EFLAG_PAGE_RANGE and got & srkv.EFLAG_SEQ_LEN
    assert torch.isfinite(buf.out).all()


@pytest.mark.parametrize("batch", [2, 12])
def test_a_run_of_appends_and_steps_as_a_server_makes_them(batch):
    """Prompt pages compressed, then tokens appended and decoded in turn; captured once into a graph
    and replayed, on a stream of its own."""
    n = 5
    lens = [1000 + 97 * r for r in range(batch)]
    case = make(seq_lens=[L + n for L in lens], num_q_heads=16, num_kv_heads=4, seed=103)
    cfg, Hkv, d = case.cfg, 4, 128
    kv, buf = int4_case(case)
    g = torch.Generator(device=DEV).manual_seed(5)
    new = [[torch.randn(batch, Hkv, d, generator=g, device=DEV).bfloat16() for _ in "kv"] for _ in range(n)]
    L = torch.tensor(lens, dtype=i32, device=DEV)
    kn, vn = (torch.zeros(batch, Hkv, d, dtype=torch.bfloat16, device=DEV) for _ in "kv")

    def token():
        srkv.append_kv_int4(cfg, kn, vn, kv, case.block_table, L, buf.reps, buf.error_flags)
        L.add_(1)
        srkv.retrieval_decode_int4(cfg, case.q, kv, buf.reps, case.block_table, L, None, buf.sel,
                                   buf.nsel, buf.out, buf.workspace, buf.error_flags)

    start = (kv.clone(), buf.reps.clone(), L.clone())
    outs = []
    for a, b in new:
        kn.copy_(a), vn.copy_(b)
        token()
        outs.append(buf.out.clone())
    torch.cuda.synchronize()
    assert int(buf.error_flags.item()) == 0
    end = synth.Case(**{**case.__dict__, "seq_lens": L, "prompt_lens": L})
    check(end, kv, buf, units=[(0, 0), (batch - 1, 3)])
    # the same tokens through a captured graph
    for t, x in zip((kv, buf.reps, L), start):
        t.copy_(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            token()
        for (a, b), want in zip(new, outs):
            kn.copy_(a), vn.copy_(b)
            graph.replay()
            assert torch.equal(buf.out, want)
    torch.cuda.synchronize()


def test_refusals_reach_python():
    cfg = config()
    case = make(seq_lens=[600], seed=104)
    kv, buf = int4_case(case)
    wide = dict(case.cfg, num_q_heads=18)  # group 9
    q = torch.zeros(1, 18, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(srkv.SrkvError, match="unsupported"):
        srkv.retrieval_decode_int4(wide, q, kv, buf.reps, case.block_table, case.seq_lens, None,
                                   buf.sel, buf.nsel, q.clone(), buf.workspace)
    with pytest.raises(srkv.SrkvError, match="workspace"):
        srkv.retrieval_decode_int4(case.cfg, case.q, kv, buf.reps, case.block_table, case.seq_lens, None,
                                   buf.sel, buf.nsel, buf.out, buf.workspace[:256])
    with pytest.raises(ValueError, match="kv_int4 must have shape"):
        srkv.append_kv_int4(cfg, *(x[:1, :, 0].contiguous() for x in (case.k_cache, case.v_cache)),
                            kv[..., :-1], case.block_table, case.seq_lens, buf.reps)
    with pytest.raises(ValueError, match="contiguous"):
        srkv.retrieval_decode_int4(case.cfg, case.q, kv.transpose(0, 1).contiguous().transpose(0, 1),
                                   buf.reps, case.block_table, case.seq_lens, None, buf.sel, buf.nsel,
                                   buf.out, buf.workspace)
    with pytest.raises(ValueError, match="must be torch.float32"):
        srkv.retrieval_decode_int4(case.cfg, case.q, kv, buf.reps.double(), case.block_table,
                                   case.seq_lens, None, buf.sel, buf.nsel, buf.out, buf.workspace)
    off = torch.zeros(kv.numel() + 8, dtype=torch.uint8, device=DEV)[8:].view(kv.shape)  # 8-byte aligned
    with pytest.raises(srkv.SrkvError, match="invalid argument"):
        srkv.quantize_kv_int4(case.cfg, case.k_cache, case.v_cache, case.page_ids, off)
    with pytest.raises(ValueError, match="CUDA tensor on device"):
        srkv.dequantize_kv_int4(case.cfg, kv, case.page_ids.cpu(), case.k_cache, case.v_cache)
