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


class Server:
    """Steps of a batch, each an append and the two attentions over it, with nothing between; everything that changes
    from step to step is made beforehand, the workspace, caches and rotated queries are shared."""

    def __init__(self, past, steps, dtype, d, Hq=8, Hkv=2):
        B = len(past)
        total = [p + sum(s[r] for s in steps) for r, p in enumerate(past)]
        self.case = c = ref.Case([(0, n) for n in total], Hq, Hkv, d, dtype, seed=91, init=128, local=300)
        g = torch.Generator(device=DEV).manual_seed(92)
        self.f = ref.freqs(d)
        self.k0, self.v0 = c.k.clone(), c.v.clone()
        self.reps = torch.zeros(c.pages, Hkv, d, device=DEV)
        most = max(sum(s) for s in steps)
        self.q_rot = torch.zeros(most, Hq, d, dtype=dtype, device=DEV)
        self.ws = torch.zeros(srkv.chunk_workspace_size(c.cfg, most, B), dtype=torch.uint8, device=DEV)
        self.steps = []
        for s in steps:
            n = sum(s)
            ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
            qkv = torch.randn(n, Hq + 2 * Hkv, d, generator=g, device=DEV).to(dtype).split((Hq, Hkv, Hkv), 1)
            outs = [torch.zeros(n, Hq, d, dtype=dtype, device=DEV) for _ in range(2)]
            after = [p + m for p, m in zip(past, s)]
            self.steps.append((s, qkv, ints([sum(s[:i]) for i in range(B + 1)]), ints(past), ints(after), outs))
            past = after

    def run(self, wait):
        c = self.case
        c.k.copy_(self.k0)
        c.v.copy_(self.v0)
        for s, (q, kn, vn), offsets, past, lens, outs in self.steps:
            q_rot = self.q_rot[:sum(s)]
            srkv.append_kv_rope(c.cfg, q, kn, vn, self.f, c.k, c.v, c.table, offsets, past, self.reps, q_rot, c.flags)
            wait()
            for call, out in zip((srkv.chunk_attention, srkv.chunk_attention_window), outs):
                call(c.cfg, q_rot, c.k, c.v, c.table, offsets, lens, out, self.ws, c.flags)
                wait()

    def take(self):
        torch.cuda.synchronize()
        got = []
        for *_, outs in self.steps:
            for o in outs:
                got.append(o.clone())
                o.zero_()
        return got


@pytest.mark.parametrize("past,steps", [([6000], [[1]] * 12), ([300, 4000], [[2, 1], [1, 1], [40, 1], [1, 5]] * 3),
                                        ([500, 0, 90], [[200, 130, 1], [1, 1, 38], [300, 0, 1]] * 2)],
                         ids=["token", "tokens", "chunks"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_an_append_directly_followed_by_attention(past, steps, dtype, d):
    server = Server(past, steps, dtype, d)
    server.run(torch.cuda.synchronize)
    want = server.take()
    # the last step against 64 bits
    c, (s, _, offsets, _, lens, _) = server.case, server.steps[-1]
    c.reqs, c.offsets, c.lens, c.q, c.T = [(n, 0) for n in s], offsets, lens, server.q_rot[:sum(s)], sum(s)
    for out, window in zip(want[-2:], (False, True)):
        exact, tol = ref.attention(c, window)
        assert ((out.double() - exact).abs() <= tol).all()
    for _ in range(5):
        server.run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(server.take(), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        server.run(lambda: None)
    for _ in range(3):
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(server.take(), want))
    assert int(c.flags) == 0


@pytest.mark.parametrize("past", [[9000], [700, 5000, 90], [400 + 37 * i for i in range(40)]],
                         ids=["one", "three", "forty"])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_an_append_directly_followed_by_a_decode_step(past, dtype, d):
    """Decode steps over what the rotated append wrote just before, and the chunk attention beside them."""
    server = Server(past, [[1] * len(past)] * 8, dtype, d)
    c = server.case
    bufs = [srkv.DecodeBuffers(c.cfg, len(past), c.max_blocks, c.pages) for _ in server.steps]

    def run(wait):
        c.k.copy_(server.k0)
        c.v.copy_(server.v0)
        server.reps.zero_()
        for (s, (q, kn, vn), offsets, past_r, lens, outs), b in zip(server.steps, bufs):
            q_rot = server.q_rot[:len(past)]
            srkv.append_kv_rope(c.cfg, q, kn, vn, server.f, c.k, c.v, c.table, offsets, past_r, server.reps, q_rot, c.flags)
            wait()
            srkv.retrieval_decode(c.cfg, q_rot, c.k, c.v, server.reps, c.table, lens, None, b.sel, b.nsel, b.out,
                                  b.workspace, b.error_flags)
            wait()
            srkv.chunk_attention(c.cfg, q_rot, c.k, c.v, c.table, offsets, lens, outs[0], server.ws, c.flags)
            wait()

    def take():
        decoded = []
        torch.cuda.synchronize()
        for b in bufs:
            assert int(b.error_flags) == 0
            decoded += [b.out.clone(), b.nsel.clone()]
            b.out.zero_()
        return server.take() + decoded

    run(torch.cuda.synchronize)
    want = take()
    for _ in range(4):
        run(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(take(), want))
    assert int(c.flags) == 0


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_two_calls_at_once(dtype, d):
    """On two streams, with a workspace each."""
    cases = [ref.Case([(300, 900), (1, 9000)], d=d, dtype=dtype, seed=97),
             ref.Case([(1, 4000), (70, 3000), (5, 60)], d=d, dtype=dtype, seed=98)]
    want = [attend(c).clone() for c in cases]
    ws = [torch.zeros(srkv.chunk_workspace_size(c.cfg, c.T, len(c.reqs)), dtype=torch.uint8, device=DEV) for c in cases]
    outs = [[torch.zeros_like(w) for _ in range(20)] for w in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for c, w, o, stream in zip(cases, ws, outs, streams):
            attend(c, out=o[i], workspace=w, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for w, os in zip(want, outs) for o in os)
    assert all(int(c.flags) == 0 for c in cases)


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (64, 1), (256, 2), (129, 1)])
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
def test_large_groups(Hq, Hkv, dtype, d):
    case = ref.Case([(5, 300), (1, 700)], Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, seed=99)
    want, tol = ref.attention(case, False)
    assert ((attend(case).double() - want).abs() <= tol).all() and int(case.flags) == 0


def test_one_token_of_a_fused_projection_in_place():
    run = Run([(1, 300)], seed=100)
    run.append()
    want, k = run.q_out.clone(), run.case.k.clone()
    assert run.q.data_ptr() != run.q_out.data_ptr()
    run.q_out = run.q  # a single token's heads are contiguous
    run.append()
    assert torch.equal(run.q, want) and torch.equal(run.case.k.view(torch.uint8), k.view(torch.uint8))


@pytest.mark.parametrize("offsets,good", [([0, 10, 30, 36], [0, 1]), ([-1, 10, 30, 35], [1, 2]),
                                          ([0, 40, 30, 35], [2]), ([0, 10, 1 << 30, 35], [0])])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_requests_beside_wrong_offsets(dtype, offsets, good):
    run = Run([(10, 300), (20, 100), (5, 50)], dtype=dtype, seed=94)
    c = run.case
    (want, tol), k0, v0 = ref.attention(c, False), c.k.clone(), c.v.clone()
    run.append()
    q_rot, k1 = run.q_out.clone(), c.k.clone()
    ends, wrong = c.offsets.tolist(), torch.tensor(offsets, dtype=torch.int32, device=DEV)
    c.k.copy_(k0)
    c.v.copy_(v0)
    c.offsets = wrong
    out = attend(c)
    assert int(c.flags) == srkv.EFLAG_CHUNK
    run.q_out.fill_(7)
    c.flags.zero_()
    run.append()
    assert int(c.flags) == srkv.EFLAG_CHUNK
    left = torch.ones(c.T, dtype=torch.bool, device=DEV)
    for r in range(3):
        rows, pages = slice(ends[r], ends[r + 1]), c.table[r][c.table[r] >= 0].long()
        if r in good:
            left[rows] = False
            assert ((out[rows].double() - want[rows]).abs() <= tol[rows]).all()
            assert torch.equal(run.q_out[rows], q_rot[rows])
        held = k1 if r in good else k0
        assert torch.equal(c.k[pages].view(torch.uint8), held[pages].view(torch.uint8))
    assert (out[left] == 7).all() and (run.q_out[left] == 7).all()


@pytest.mark.parametrize("reqs", [[(20, 300)] * 4, [(300, 100)] * 4], ids=["tokens", "pages"])
def test_offsets_that_go_down(reqs):
    """A row is what its own request makes of it, or as it was."""
    run = Run(reqs, seed=95)
    c, n = run.case, reqs[0][0]
    (want, tol), k0, v0 = ref.attention(c, False), c.k.clone(), c.v.clone()
    run.append()
    q_rot, k1 = run.q_out.clone(), c.k.clone()
    c.k.copy_(k0)
    c.v.copy_(v0)
    c.offsets = torch.tensor([0, n, n // 2, 3 * n, 4 * n], dtype=torch.int32, device=DEV)  # the third begins elsewhere
    out = attend(c)
    assert int(c.flags) & srkv.EFLAG_CHUNK
    near = (out.double() - want).abs() <= tol
    assert near[3 * n:].all() and near[:n // 2].all()
    run.q_out.fill_(7)
    c.flags.zero_()
    run.append()
    assert int(c.flags) & srkv.EFLAG_CHUNK
    for rows in (slice(0, n // 2), slice(3 * n, 4 * n)):
        got = run.q_out[rows]
        right, old = (got == q_rot[rows]).flatten(1).all(1), (got == 7).flatten(1).all(1)
        assert (right | old).all()
    for r in (0, 3):
        pages = c.table[r][c.table[r] >= 0].long()
        same = lambda x: (c.k[pages].view(torch.uint8) == x[pages].view(torch.uint8)).flatten(3).all(3)
        assert (same(k1) | same(k0)).all()


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
