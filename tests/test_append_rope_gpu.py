"""Chunks of new tokens rotated and appended, against 64 bits: rows within half a step of the type and the
fp32 rotation, values and vectors to the bit, and everything else in the cache left alone."""
import fractions
import math

import pytest
import torch

import chunk_ref as ref
from block_sparse_retrieval_gb300 import srkv

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


class Run:
    def __init__(self, reqs, Hq=8, Hkv=2, d=128, dtype=BF, rope=None, seed=0, strided=True, **kw):
        self.case = c = ref.Case(reqs, Hq, Hkv, d, dtype, seed, **kw)
        g = torch.Generator(device=DEV).manual_seed(seed + 1)
        qkv = torch.randn(c.T, Hq + 2 * Hkv, d, generator=g, device=DEV).to(dtype)
        self.q, self.kn, self.vn = qkv.split((Hq, Hkv, Hkv), 1)
        if not strided:
            self.q, self.kn, self.vn = (x.contiguous() for x in (self.q, self.kn, self.vn))
        self.freqs = ref.freqs(d if rope is None else rope)
        self.q_out = torch.full((c.T, Hq, d), 7.0, dtype=dtype, device=DEV)
        self.reps = torch.full((c.pages, Hkv, d), 5.0, device=DEV)

    def append(self, inter=False, queries=True, stream=None):
        c = self.case
        srkv.append_kv_rope(c.cfg, self.q if queries else None, self.kn, self.vn, self.freqs, c.k, c.v, c.table,
                            c.offsets, c.past, self.reps, self.q_out if queries else None, c.flags,
                            stream=stream, interleaved=inter)

    def check(self, inter=False):
        """Appends, and looks at all that the call writes and at all that it must not."""
        c = self.case
        k0, v0, reps0 = c.k.clone(), c.v.clone(), self.reps.clone()
        self.append(inter)
        torch.cuda.synchronize()
        assert int(c.flags) == 0
        pos = torch.cat([torch.arange(p, p + n, device=DEV) for n, p in c.reqs])
        r = torch.cat([torch.full((n,), i, device=DEV) for i, (n, _) in enumerate(c.reqs)])
        page, row = c.table[r, pos // 128].long(), pos % 128
        for got, new in ((self.q_out, self.q), (c.k[page, :, row], self.kn)):
            y, size = ref.rotate(new, pos, self.freqs, inter)
            assert ((got.double() - y).abs() <= ref.rotation_bound(y, size, c.dtype)).all()
            assert torch.equal(got[..., 2 * len(self.freqs):], new[..., 2 * len(self.freqs):])
        k0[page, :, row] = c.k[page, :, row]
        v0[page, :, row] = self.vn
        assert torch.equal(c.k.view(torch.uint8), k0.view(torch.uint8))  # NaN where it was
        assert torch.equal(c.v.view(torch.uint8), v0.view(torch.uint8))
        held = torch.zeros(c.pages, dtype=torch.int32, device=DEV)
        held.scatter_reduce_(0, page, (row + 1).int(), "amax")
        ids = held.nonzero()[:, 0].int()
        srkv.build_block_reps(c.cfg, c.k, ids, held[ids.long()], reps0)
        assert torch.equal(self.reps, reps0)


SHAPES = [[(1, 0)], [(1, 127)], [(1, 128)], [(2, 127)], [(128, 0)], [(129, 127)], [(300, 50)], [(1, 65499)],
          [(5, 0), (0, 0), (1, 700), (0, 50), (130, 255), (33, 95)], [(1, 40 * i) for i in range(70)],
          [(1, 40 * i) for i in range(1100)], [(1500, 77), (2, 0)]]


@pytest.mark.parametrize("reqs", SHAPES, ids=lambda r: f"{len(r)}x" + "+".join(f"{n}@{p}" for n, p in r[:3]))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_chunks_of_all_lengths(reqs, d, dtype):
    Run(reqs, d=d, dtype=dtype, seed=1).check()


@pytest.mark.parametrize("rope", [0, 16, 32, 48, 64])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_part_of_a_head_rotated(rope, inter, dtype):
    for d in (64, 128):
        Run([(40, 100), (3, 9)], d=d, rope=rope, dtype=dtype, seed=2).check(inter)
    if rope:
        Run([(40, 100), (3, 9)], d=128, rope=64 + rope, dtype=dtype, seed=2).check(inter)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (15, 5), (32, 8), (64, 8), (9, 1)])
def test_head_layouts(Hq, Hkv):
    Run([(37, 200), (1, 301)], Hq=Hq, Hkv=Hkv, d=64, seed=3, strided=Hq % 2 == 0).check()


def test_angles_of_far_positions():
    """Positions up to the largest that a table can hold: the angle is reduced without rounding."""
    Hkv, d = 1, 64
    far = [(1 << 31) - 256, 1234567890, 99999999, 131071]
    cfg = ref.Case([(1, 0)], 1, 1, d, F32).cfg
    f = torch.cat((ref.freqs(48, 500000.0), torch.tensor([3.0, 100.0, -1.5, 1e-9, 6.283185307179586, 0.0, 2.0, 0.5],
                                                          dtype=torch.float64, device=DEV)))
    for p in far:
        blocks = p // 128 + 1
        table = torch.zeros(1, blocks, dtype=torch.int32, device=DEV)
        k, v = (torch.zeros(1, Hkv, 128, d, device=DEV) for _ in "kv")
        q, kn, vn = (torch.randn(1, 1, d, device=DEV) for _ in "qkv")
        q_out, reps = torch.zeros_like(q), torch.zeros(1, 1, d, device=DEV)
        srkv.append_kv_rope(cfg, q, kn, vn, f, k, v, table, torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                            torch.tensor([p], dtype=torch.int32, device=DEV), reps, q_out)
        # the angle modulo a turn in exact arithmetic on the frequency as given
        pi = fractions.Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
        a = [float((fractions.Fraction(x) * p) % (2 * pi)) for x in f.tolist()]
        cos = torch.tensor([math.cos(x) for x in a], dtype=torch.float64, device=DEV)
        sin = torch.tensor([math.sin(x) for x in a], dtype=torch.float64, device=DEV)
        for got, x in ((q_out[0, 0], q[0, 0]), (k[0, 0, p % 128], kn[0, 0])):
            one, two = x[:32].double(), x[32:].double()
            y = torch.cat((one * cos - two * sin, two * cos + one * sin))
            size = torch.hypot(one, two).repeat(2)
            # a fraction of a turn good to 2^-54, times the position
            tol = ref.rotation_bound(y, size, F32) + 2 * math.pi * p * 2.0 ** -53 * size
            assert ((got.double() - y).abs() <= tol).all(), p


def test_without_queries_and_in_place():
    run = Run([(9, 100), (20, 10)], seed=4, strided=False)
    run.append(queries=False)
    assert (run.q_out == 7).all()
    k, reps = run.case.k.clone(), run.reps.clone()
    run.append()
    assert torch.equal(run.case.k.view(torch.uint8), k.view(torch.uint8)) and torch.equal(run.reps, reps)
    want = run.q_out.clone()
    run.q_out = run.q
    run.append()
    assert torch.equal(run.q, want)


def test_rows_outside_every_request_are_left_alone():
    run = Run([(9, 100), (20, 10)], seed=5)
    c = run.case
    run.append()
    want, k = run.q_out.clone(), c.k.clone()
    pad = lambda x: torch.cat((x[:2], x, x[:3]))
    run.q, run.kn, run.vn = pad(run.q), pad(run.kn), pad(run.vn)
    run.q_out = torch.full((c.T + 5, 8, 128), 7.0, dtype=BF, device=DEV)
    c.offsets += 2
    run.append()
    assert torch.equal(run.q_out[2:-3], want) and (run.q_out[:2] == 7).all() and (run.q_out[-3:] == 7).all()
    assert torch.equal(c.k.view(torch.uint8), k.view(torch.uint8))


def test_in_pieces_as_in_one_go():
    """A prompt in one chunk, in odd pieces and token by token: the same cache and vectors."""
    whole = Run([(400, 60)], seed=6, strided=False)
    whole.append()
    for sizes in ([1] * 400, [68, 1, 127, 128, 76], [399, 1]):
        part = Run([(400, 60)], seed=6, strided=False)
        c = part.case
        q, kn, vn = part.q, part.kn, part.vn
        at = 0
        for n in sizes:
            out = torch.zeros(n, 8, 128, dtype=BF, device=DEV)
            srkv.append_kv_rope(c.cfg, q[at:at + n], kn[at:at + n], vn[at:at + n], part.freqs, c.k, c.v, c.table,
                                torch.tensor([0, n], dtype=torch.int32, device=DEV), c.past, part.reps, out, c.flags)
            assert torch.equal(out, whole.q_out[at:at + n])
            at += n
            c.past += n
        assert torch.equal(c.k.view(torch.uint8), whole.case.k.view(torch.uint8))
        assert torch.equal(part.reps, whole.reps)


def test_without_rotation_it_is_the_plain_append():
    run = Run([(1, 200), (1, 127), (1, 0)], rope=0, seed=7, strided=False)
    c = run.case
    k, v, reps = c.k.clone(), c.v.clone(), run.reps.clone()
    srkv.append_kv(c.cfg, run.kn, run.vn, k, v, c.table, c.past, reps)
    run.append()
    assert torch.equal(c.k.view(torch.uint8), k.view(torch.uint8))
    assert torch.equal(c.v.view(torch.uint8), v.view(torch.uint8)) and torch.equal(run.reps, reps)


def test_streams_and_graphs():
    run = Run([(70, 100), (1, 3)], seed=8)
    run.append()
    want, k = run.q_out.clone(), run.case.k.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run.q_out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    run.append(stream=side)
    side.synchronize()
    assert torch.equal(run.q_out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run.append()
    run.q_out.zero_()
    g.replay()
    assert torch.equal(run.q_out, want) and torch.equal(run.case.k.view(torch.uint8), k.view(torch.uint8))


def test_what_the_device_refuses():
    run = Run([(10, 300), (150, 100), (5, 50)], seed=9)
    c = run.case
    k0, v0 = c.k.clone(), c.v.clone()

    def again():
        c.k.copy_(k0)
        c.v.copy_(v0)
        c.flags.zero_()
        run.q_out.fill_(7)
        run.append()
        return int(c.flags)

    assert again() == 0
    k1, q1 = c.k.clone(), run.q_out.clone()
    good, past = c.table.clone(), c.past.clone()
    for bad in (-1, c.pages, 1 << 30):  # that page is skipped, the rest goes on
        c.table[1, 1] = bad
        assert again() == srkv.EFLAG_PAGE_RANGE
        page = int(good[1, 1])
        want = k1.clone()
        want[page] = k0[page]
        assert torch.equal(c.k.view(torch.uint8), want.view(torch.uint8)) and torch.equal(run.q_out, q1)
        c.table.copy_(good)
    for bad in (-1, c.max_blocks * 128 - 149, (1 << 31) - 1):  # that request is skipped
        c.past[1] = bad
        assert again() == srkv.EFLAG_SEQ_LEN
        assert (run.q_out[10:160] == 7).all() and torch.equal(run.q_out[160:], q1[160:])
        c.past.copy_(past)
    for offsets in ([0, 30, 10, 165], [0, 10, 160, 166], [-1, 10, 160, 165], [165, 0, 165, 0]):
        c.offsets.copy_(torch.tensor(offsets))
        assert again() & srkv.EFLAG_CHUNK
    torch.cuda.synchronize()
