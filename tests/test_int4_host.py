"""The 4-bit cache's entry points on the host (no GPU): argument checks of the library, shape checks of the
binding, and the tests' own restatement of the format.  No call reaches a launch."""
import ctypes

import numpy as np
import pytest
import torch

import int4_ref as ref
from block_sparse_retrieval_gb300 import build, srkv

CFG = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=128, init_tokens=256,
           local_tokens=512, topk_percent=0.2, dense_boundary=0, dtype=srkv.BF16)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the checks reject the call first
ODD = ctypes.c_void_p((1 << 20) + 8)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return srkv.load()


def test_slab_bytes(lib):
    assert srkv.kv_int4_slab_bytes(CFG) == 17408 == ref.slab_bytes(128)
    assert srkv.kv_int4_slab_bytes(dict(CFG, head_dim=64)) == 9216 == ref.slab_bytes(64)
    assert srkv.kv_int4_slab_bytes(dict(CFG, head_dim=96)) == 0
    assert lib.srkv_kv_int4_slab_bytes(None) == 0


def quantize(lib, cfg=CFG, **o):
    a = {**dict(k=FAKE, v=FAKE, pages=10, ids=FAKE, n=3, kv=FAKE, slabs=10, to=None), **o}
    c = ctypes.byref(srkv.config(cfg)) if cfg else None
    return lib.srkv_quantize_kv_int4(c, a["k"], a["v"], a["pages"], a["ids"], a["n"], a["kv"],
                                     a["slabs"], a["to"], None, None)


def dequantize(lib, cfg=CFG, **o):
    a = {**dict(k=FAKE, v=FAKE, pages=10, ids=FAKE, n=3, kv=FAKE, slabs=10, to=None), **o}
    c = ctypes.byref(srkv.config(cfg)) if cfg else None
    return lib.srkv_dequantize_kv_int4(c, a["kv"], a["slabs"], a["ids"], a["n"], a["k"], a["v"],
                                       a["pages"], a["to"], None, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
def test_page_calls_check_their_arguments(lib, call):
    assert call(lib, n=0) == OK
    assert call(lib, cfg=None) == INVALID
    assert call(lib, dict(CFG, head_dim=96)) == INVALID
    for bad in (dict(k=None), dict(v=None), dict(kv=None), dict(ids=None), dict(k=ODD), dict(v=ODD),
                dict(kv=ODD), dict(n=-1), dict(pages=-1), dict(slabs=-1), dict(pages=0), dict(slabs=0)):
        assert call(lib, **bad) == INVALID, bad
    assert call(lib, dict(CFG, dtype=srkv.F32)) == UNSUPPORTED
    assert call(lib, dict(CFG, num_q_heads=64, num_kv_heads=64), n=1 << 25) == UNSUPPORTED


def append(lib, cfg=CFG, **o):
    a = {**dict(k=FAKE, v=FAKE, kv=FAKE, pages=10, bt=FAKE, max_blocks=8, lens=FAKE, batch=2, reps=FAKE),
         **o}
    c = ctypes.byref(srkv.config(cfg)) if cfg else None
    return lib.srkv_append_kv_int4(c, a["k"], a["v"], a["kv"], a["pages"], a["bt"], a["max_blocks"],
                                   a["lens"], a["batch"], a["reps"], None, None)


def test_append_checks_its_arguments(lib):
    assert append(lib, batch=0) == OK
    assert append(lib, cfg=None) == INVALID
    for bad in (dict(k=None), dict(v=None), dict(kv=None), dict(bt=None), dict(lens=None),
                dict(reps=None), dict(k=ODD), dict(v=ODD), dict(kv=ODD), dict(reps=ODD), dict(batch=-1),
                dict(max_blocks=0), dict(max_blocks=1 << 24), dict(pages=0), dict(pages=-1)):
        assert append(lib, **bad) == INVALID, bad
    assert append(lib, dict(CFG, dtype=srkv.F32)) == UNSUPPORTED


def decode(lib, cfg=CFG, **o):
    a = {**dict(q=FAKE, kv=FAKE, reps=FAKE, pages=10, bt=FAKE, max_blocks=8, lens=FAKE, batch=1, sel=FAKE,
                kmax=8, nsel=FAKE, out=FAKE, ws=None, ws_bytes=0), **o}
    c = ctypes.byref(srkv.config(cfg)) if cfg else None
    return lib.srkv_retrieval_decode_int4(c, a["q"], a["kv"], a["reps"], a["pages"], a["bt"],
                                          a["max_blocks"], a["lens"], None, a["batch"], a["sel"],
                                          a["kmax"], a["nsel"], a["out"], a["ws"], a["ws_bytes"], None,
                                          None)


def test_decode_checks_its_arguments(lib):
    assert decode(lib, batch=0) == OK
    assert decode(lib, cfg=None) == INVALID
    for bad in (dict(q=None), dict(kv=None), dict(reps=None), dict(bt=None), dict(lens=None),
                dict(sel=None), dict(nsel=None), dict(out=None), dict(q=ODD), dict(kv=ODD),
                dict(out=ODD), dict(batch=-1), dict(max_blocks=0), dict(pages=0), dict(kmax=-1)):
        assert decode(lib, **bad) == INVALID, bad
    assert decode(lib) == WORKSPACE
    assert decode(lib, ws=FAKE, ws_bytes=256) == WORKSPACE
    assert decode(lib, dict(CFG, num_q_heads=18)) == UNSUPPORTED  # group 9
    assert decode(lib, dict(CFG, dtype=srkv.F32)) == UNSUPPORTED
    assert decode(lib, max_blocks=25601, kmax=1 << 20) == UNSUPPORTED
    assert decode(lib, dict(CFG, dense_boundary=1), max_blocks=100, kmax=8) == INVALID  # below kmax_bound


# ---- the binding's shape checks ------------------------------------------------------------------------

B, MAXB, P, KMAX = 3, 10, 24, 4
bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


def shaped(**over):
    z = torch.zeros
    return {**dict(q=z(B, 8, 128, dtype=bf), k_cache=z(P, 2, 128, 128, dtype=bf),
                   v_cache=z(P, 2, 128, 128, dtype=bf), kv=z(P + 5, 2, 17408, dtype=u8),
                   reps=z(P + 5, 2, 128, dtype=f32), block_table=z(B, MAXB, dtype=i32),
                   seq_lens=z(B, dtype=i32), prompt_lens=z(B, dtype=i32), sel=z(B, 2, KMAX, dtype=i32),
                   nsel=z(B, 2, dtype=i32), out=z(B, 8, 128, dtype=bf), workspace=z(256, dtype=u8),
                   ids=z(7, dtype=i32), to=z(7, dtype=i32), k_new=z(B, 2, 128, dtype=bf),
                   v_new=z(B, 2, 128, dtype=bf)), **over}


def call_quantize(a):
    srkv.quantize_kv_int4(CFG, a["k_cache"], a["v_cache"], a["ids"], a["kv"], a["to"])


def call_dequantize(a):
    srkv.dequantize_kv_int4(CFG, a["kv"], a["ids"], a["k_cache"], a["v_cache"], a["to"])


def call_append(a):
    srkv.append_kv_int4(CFG, a["k_new"], a["v_new"], a["kv"], a["block_table"], a["seq_lens"], a["reps"])


def call_decode(a):
    srkv.retrieval_decode_int4(CFG, a["q"], a["kv"], a["reps"], a["block_table"], a["seq_lens"],
                               a["prompt_lens"], a["sel"], a["nsel"], a["out"], a["workspace"])


CALLS = [call_quantize, call_dequantize, call_append, call_decode]


@pytest.mark.parametrize("call", CALLS)
def test_right_shapes_reach_the_device_check(lib, call):
    with pytest.raises(ValueError, match="CUDA tensor"):
        call(shaped())


z = torch.zeros
WRONG = [
    (call_quantize, dict(kv=z(P, 2, 17407, dtype=u8))), (call_quantize, dict(kv=z(P, 3, 17408, dtype=u8))),
    (call_quantize, dict(to=z(6, dtype=i32))), (call_quantize, dict(v_cache=z(P - 1, 2, 128, 128, dtype=bf))),
    (call_quantize, dict(k_cache=z(P, 2, 128, 64, dtype=bf))), (call_quantize, dict(ids=z(7, 1, dtype=i32))),
    (call_dequantize, dict(kv=z(P, 2, 9216, dtype=u8))), (call_dequantize, dict(to=z(8, dtype=i32))),
    (call_dequantize, dict(k_cache=z(P, 1, 128, 128, dtype=bf))),
    (call_append, dict(k_new=z(B, 1, 128, dtype=bf))), (call_append, dict(v_new=z(B + 1, 2, 128, dtype=bf))),
    (call_append, dict(seq_lens=z(B + 1, dtype=i32))), (call_append, dict(reps=z(P, 2, 128, dtype=f32))),
    (call_append, dict(kv=z(P, 2, 17408, 1, dtype=u8))),
    (call_decode, dict(q=z(B, 4, 128, dtype=bf))), (call_decode, dict(out=z(B, 8, 64, dtype=bf))),
    (call_decode, dict(kv=z(P, 2, 128, 128, dtype=u8))), (call_decode, dict(reps=z(P, 2, 128, dtype=f32))),
    (call_decode, dict(sel=z(B, 1, KMAX, dtype=i32))), (call_decode, dict(nsel=z(B * 2, dtype=i32))),
    (call_decode, dict(prompt_lens=z(B - 1, dtype=i32))), (call_decode, dict(seq_lens=z(B, 1, dtype=i32))),
]


@pytest.mark.parametrize("i", range(len(WRONG)))
def test_a_wrong_shape_stops_before_the_library(lib, i):
    call, over = WRONG[i]
    with pytest.raises(ValueError, match="must have shape|needs at least"):
        call(shaped(**over))


# ---- the restatement the GPU tests compare with ----------------------------------------------------------

def test_quantised_rows_lie_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((200, 128)) * np.exp(np.linspace(-20, 20, 200))[:, None]
    x = ref.to_bf16(x)
    c, s, lo = ref.quantize_rows(x)
    assert c.min() == 0 and c.max() == 15
    # half a step; the difference's rounding to fp32 adds 2^-24 of the range (15 steps)
    assert (np.abs(lo[:, None] + c * s[:, None] - x) <= s[:, None] * (0.5 + 15 * 2.0 ** -24)).all()
    assert (s >= (x.max(1) - x.min(1)) / 15 * (1 - 2.0 ** -23)).all()
    assert (s <= (x.max(1) - x.min(1)) / 15 * (1 + 2.0 ** -7)).all()


def test_constant_and_bad_rows_of_the_restatement():
    x = np.zeros((4, 64))
    x[1], x[2, 5], x[3, 0] = 2.5, np.nan, np.inf
    c, s, lo = ref.quantize_rows(x)
    assert (c == 0).all() and (s[:2] == 0).all() and (lo[:2] == [0, 2.5]).all()
    assert np.isnan(s[2:]).all() and np.isnan(lo[2:]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_every_code_of_a_slab_has_its_own_place(d):
    """Each code set alone comes back alone, at the place the format gives it."""
    rng = np.random.default_rng(d)
    for t, e in [(0, 0), (127, d - 1)] + [(int(rng.integers(128)), int(rng.integers(d))) for _ in range(40)]:
        slab = np.zeros(ref.slab_bytes(d), np.uint8)
        w = slab.view(np.uint32)
        w[t * (d // 8) + e // 8] |= np.uint32(9 << ref.shift(e % 8))
        w[16 * d + ((t // 32 * (d // 4) + e // 4) * 4 + t % 32 // 8) * 4 + e % 4] |= np.uint32(
            13 << ref.shift(t % 8))
        k, v, *_ = ref.unpack(slab, d)
        assert k[t, e] == 9 and k.sum() == 9 and v[t, e] == 13 and v.sum() == 13
