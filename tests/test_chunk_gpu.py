"""Attention of chunks of new tokens over the paged cache, against 64 bits, within the bounds that the kernels'
roundings give (chunk_ref.attention).  What is behind a request's last token is NaN throughout."""
import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def attend(case, window=False, q=None, out=None, workspace=None, stream=None):
    out = torch.full((case.T, case.cfg["num_q_heads"], case.cfg["head_dim"]), 7.0, dtype=case.dtype,
                     device=DEV) if out is None else out
    if workspace is None:
        workspace = torch.full((srkv.chunk_workspace_size(case.cfg, case.T, len(case.reqs)),), 255,
                               dtype=torch.uint8, device=DEV)
    call = srkv.chunk_attention_window if window else srkv.chunk_attention
    call(case.cfg, case.q if q is None else q, case.k, case.v, case.table, case.offsets, case.lens, out,
         workspace, case.flags, stream=stream)
    return out


def check(case, window=False, flags=0):
    out = attend(case, window)
    torch.cuda.synchronize()
    assert int(case.flags) == flags
    want, tol = ref.attention(case, window)
    bad = ~((out.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((out.double() - want).abs().max()))
    return out


# one token to a few pages, ends at, before and behind a page's end, several requests, empty chunks among them
SHAPES = [[(1, 0)], [(1, 127)], [(1, 128)], [(2, 3)], [(128, 0)], [(129, 0)], [(127, 129)], [(70, 1000)],
          [(1, 5000)], [(300, 411)], [(5, 0), (0, 0), (1, 700), (0, 50), (130, 255), (33, 95)],
          [(1, 40 * i) for i in range(40)]]


@pytest.mark.parametrize("reqs", SHAPES, ids=lambda r: "+".join(f"{n}@{p}" for n, p in r[:3]))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_chunks_of_all_lengths(reqs, d, dtype):
    check(ref.Case(reqs, d=d, dtype=dtype, seed=1))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (15, 5), (32, 8), (7, 1), (16, 2), (100, 1), (300, 1)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_head_layouts(Hq, Hkv, dtype):
    check(ref.Case([(37, 200), (1, 301), (140, 3)], Hq=Hq, Hkv=Hkv, d=64, dtype=dtype, seed=2))


@pytest.mark.parametrize("init,local", [(0, 1), (0, 0), (1, 0), (4, 1), (4, 128), (100, 129), (128, 127), (129, 700),
                                        (300, 1111), (1024, 7192), (5000, 3), (0, 100000)])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)], ids=["bf16-128", "bf16-64", "fp32-64"])
def test_windows(init, local, dtype, d):
    check(ref.Case([(200, 1900), (1, 2500), (0, 3), (300, 0), (1, 0), (64, 256)], d=d, dtype=dtype, seed=3,
                   init=init, local=local), window=True)


def test_a_row_that_sees_nothing_is_zero():
    case = ref.Case([(3, 500), (1, 0)], init=0, local=0)
    assert not attend(case, window=True).any()
    assert int(case.flags) == 0


@pytest.mark.parametrize("reqs", [[(1, 65535)], [(2, 30000), (1, 60000)], [(513, 20000)]])
def test_long_lists_are_divided(reqs):
    check(ref.Case(reqs, Hq=8, Hkv=2, d=128, seed=4))


def test_many_tiles():
    check(ref.Case([(1500, 100), (700, 0), (1, 3000)], Hq=32, Hkv=8, d=64, seed=5))
    check(ref.Case([(1500, 100), (700, 0), (1, 3000)], Hq=32, Hkv=8, d=64, seed=5, init=64, local=200), window=True)


def test_logits_far_apart_and_equal():
    # rows whose maximum moves at every page, by more than a weight's whole range, up and down; and equal logits
    case = ref.Case([(40, 1000)], Hq=4, Hkv=1, d=64, seed=6)
    k, _ = case.tokens(0)
    ramp = torch.linspace(-30, 30, 1040, device=DEV)
    for sign, head in ((1, 0), (-1, 1)):
        case.q[:, head] = 0
        case.q[:, head, 0] = sign * 8.0
    blocks = case.table[0, :9].long()
    x = torch.zeros(9 * 128, device=DEV)
    x[:1040] = ramp
    keys = case.k[blocks].transpose(1, 2).flatten(0, 1)
    keys[:1040, 0, 0] = x[:1040].to(BF)
    case.k[blocks] = keys.view(9, 128, 1, 64).transpose(1, 2).contiguous()
    case.q[:, 2] = 0  # equal logits
    check(case)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_attend_cannot_reach_it(dtype, value):
    """Token 300 of 400 (a new one: later rows attend it) and token 150 (outside every window) hold `value`."""
    case = ref.Case([(200, 200)], Hq=4, Hkv=2, d=64, dtype=dtype, seed=7, init=100, local=40)
    for name in "kv":
        clean = ref.Case([(200, 200)], Hq=4, Hkv=2, d=64, dtype=dtype, seed=7, init=100, local=40)
        x = getattr(case, name)
        x.copy_(getattr(clean, name))
        for t in (150, 300):
            x[int(case.table[0, t // 128]), :, t % 128, 5] = value
        out = attend(case, window=True)
        want = attend(clean, window=True)
        pos = torch.arange(200, 400, device=DEV)
        sees = (pos >= 300) & (pos < 340)  # t > p - 40
        assert torch.equal(out[~sees], want[~sees])
        if name == "v":
            got = out[sees][:, :, 5].float()
            assert (got.isnan().all() if value != value else (got == value).all() or got.isnan().all())
            keep = [e for e in range(64) if e != 5]
            assert torch.equal(out[sees][:, :, keep], want[sees][:, :, keep])
        elif value != value:
            assert out[sees].isnan().all()
        x.copy_(getattr(clean, name))


def test_a_query_that_is_not_finite_spoils_its_own_row_alone():
    case = ref.Case([(50, 300)], seed=8)
    want = attend(case).clone()
    case.q[7, 3, 0] = float("nan")
    out = attend(case)
    assert out[7, 3].isnan().all()
    out[7, 3] = want[7, 3]
    assert torch.equal(out, want)


def test_query_strides_and_rows_outside_every_request():
    case = ref.Case([(9, 100), (20, 10)], seed=9)
    want = attend(case)
    wide = torch.full((case.T + 5, 8 + 6, 128), float("nan"), dtype=BF, device=DEV)
    wide[2:2 + case.T, 3:11] = case.q
    offsets, T = case.offsets, case.T
    case.offsets, case.T = offsets + 2, T + 5
    out = attend(case, q=wide[:, 3:11])
    assert torch.equal(out[2:2 + T], want)
    assert (out[:2] == 7).all() and (out[2 + T:] == 7).all()


def test_workspace_contents_and_repeats_do_not_matter():
    case = ref.Case([(300, 5000), (1, 20000)], seed=10)
    ws = torch.full((srkv.chunk_workspace_size(case.cfg, case.T, 2),), 255, dtype=torch.uint8, device=DEV)
    a = attend(case, workspace=ws)
    for _ in range(5):
        assert torch.equal(attend(case, workspace=ws), a)
    ws.zero_()
    assert torch.equal(attend(case, workspace=ws), a)


def test_streams_and_graphs_sharing_a_workspace():
    one, two = ref.Case([(200, 3000)], seed=11), ref.Case([(1, 9000), (40, 100)], seed=12)
    want = [attend(one), attend(two)]
    ws = torch.empty(max(srkv.chunk_workspace_size(c.cfg, c.T, len(c.reqs)) for c in (one, two)),
                     dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.zeros_like(w) for w in want], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip((one, two), outs):
            attend(c, out=o, workspace=ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for c, o in zip((one, two), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(c, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_lengths_change_under_a_captured_graph():
    case = ref.Case([(64, 2000), (64, 2000)], seed=13)
    out = torch.zeros(128, 8, 128, dtype=BF, device=DEV)
    ws = torch.empty(srkv.chunk_workspace_size(case.cfg, 128, 2), dtype=torch.uint8, device=DEV)
    attend(case, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend(case, out=out, workspace=ws)
    case.lens.copy_(torch.tensor([1500, 70]))
    case.offsets.copy_(torch.tensor([0, 100, 128]))
    g.replay()
    want, tol = ref.attention(case, False)
    assert ((out.double() - want).abs() <= tol).all()


def test_what_the_device_refuses():
    """Bad pages, lengths and offsets: nothing out of range is read, the rest is right, and a flag says so."""
    case = ref.Case([(10, 300), (20, 100), (5, 50)], seed=14)
    want = attend(case).clone()
    torch.cuda.synchronize()
    good = case.table.clone()
    for bad in (-1, case.pages, 1 << 30):
        case.flags.zero_()
        case.table[0, 1] = bad  # tokens 128 .. 255 of the first request are left out
        out = attend(case)
        assert int(case.flags) == srkv.EFLAG_PAGE_RANGE
        assert torch.equal(out[10:], want[10:])
        k, v = ref.Case([(10, 300), (20, 100), (5, 50)], seed=14).tokens(0)
        keep = torch.cat((torch.arange(128), torch.arange(256, 310))).to(DEV)
        q = case.q[9].double()
        for j in range(8):
            w = torch.softmax(q[j] @ k[keep, j // 4].T / 128 ** 0.5, -1)
            o = w @ v[keep, j // 4]
            assert ((out[9, j].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -6 * (w @ v[keep, j // 4].abs())).all()
        case.table.copy_(good)
    # a length behind the table is cut to it; the chunk's rows are the last ones of that
    case.flags.zero_()
    case.lens[2] = case.max_blocks * 128 + 1
    attend(case)
    assert int(case.flags) & srkv.EFLAG_SEQ_LEN
    # a chunk longer than its sequence: its first rows attend nothing
    case.flags.zero_()
    case.lens[2] = 2
    out = attend(case)
    assert int(case.flags) == srkv.EFLAG_CHUNK and not out[30:33].any() and out[33].any()
    case.flags.zero_()
    case.lens[2] = -3
    out = attend(case)
    assert int(case.flags) == srkv.EFLAG_CHUNK | srkv.EFLAG_SEQ_LEN and not out[30:].any()
    case.lens[2] = 55
    for offsets in ([0, 30, 10, 35], [0, 10, 30, 36], [-1, 10, 30, 35], [35, 0, 35, 0]):
        case.flags.zero_()
        case.offsets.copy_(torch.tensor(offsets))
        attend(case)
        assert int(case.flags) & srkv.EFLAG_CHUNK
    torch.cuda.synchronize()


def test_offsets_that_ask_for_more_tiles_than_there_are_rows():
    case = ref.Case([(64, 100)] * 2 + [(0, 0)] * 62, seed=15)
    want = attend(case)
    case.offsets.copy_(torch.tensor([0, 128] * 32 + [0]))
    attend(case)
    assert int(case.flags) & srkv.EFLAG_CHUNK
    case.flags.zero_()
    case.offsets.copy_(torch.tensor([0, 64] + [128] * 63))
    assert torch.equal(attend(case), want) and int(case.flags) == 0


def test_pages_past_32_bits():
    """A cache of 2.2e9 elements: a page whose offset passes 32 bits."""
    pages = 16500
    k = torch.zeros(pages, 8, 128, 128, dtype=BF, device=DEV)
    v = torch.zeros_like(k)
    small = ref.Case([(20, 200)], Hq=32, Hkv=8, seed=16, fill=0.0, slack=0)
    want = attend(small)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device=DEV)
    k[table[0].long()], v[table[0].long()] = small.k[small.table[0].long()], small.v[small.table[0].long()]
    small.k, small.v, small.table = k, v, table
    assert torch.equal(attend(small), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("reqs", [[(1, 13 * i % 400) for i in range(700)], [(i % 90, 3 * i) for i in range(600)],
                                  [(8000, 0)]], ids=["700 tokens", "600 chunks", "8000 rows"])
def test_more_requests_or_tiles_than_are_held_on_chip(reqs, dtype):
    Hq, Hkv = (33, 1) if len(reqs) == 1 else (4, 2)  # 264000 rows of one head: a thousand tiles
    case = ref.Case(reqs, Hq=Hq, Hkv=Hkv, d=64, dtype=dtype, seed=18, init=20, local=100)
    if len(reqs) > 1:
        check(case)
    check(case, window=True)


def test_positions_near_the_largest():
    """A sequence of 2^31 - 128 tokens, windowed (only the pages in sight exist)."""
    L = (1 << 31) - 128
    for dtype in (BF, F32):
        case = ref.Case([(5, 395)], Hq=4, Hkv=1, d=64, dtype=dtype, seed=19, init=0, local=300)
        want = attend(case, window=True)
        blocks = L // 128
        table = torch.full((1, blocks), -1, dtype=torch.int32, device=DEV)
        # 400 tokens end 112 before a page's end; as many tokens before the far end
        far = L - 112
        table[0, far // 128 - 3:far // 128 + 1] = case.table[0, :4]
        case.table, case.lens = table, torch.tensor([far], dtype=torch.int32, device=DEV)
        got = attend(case, window=True)
        assert int(case.flags) == 0 and torch.equal(got, want)
        case.cfg["local_tokens"] = (1 << 31) - 1  # everything, hidden pages among it
        case.lens = torch.tensor([400], dtype=torch.int32, device=DEV)
        case.table = ref.Case([(5, 395)], Hq=4, Hkv=1, d=64, dtype=dtype, seed=19).table
        assert torch.equal(attend(case, window=True), attend(case))


def test_no_rows_is_no_work():
    case = ref.Case([(0, 100), (0, 0)], seed=17)
    attend(case)
    assert int(case.flags) == 0
