"""The chunk calls on the host (no GPU): argument checks of the library and of the binding.  No call reaches a
launch."""
import ctypes

import pytest
import torch

from block_sparse_retrieval_gb300 import build, srkv

CFG = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=128, init_tokens=256, local_tokens=512,
           topk_percent=0.2, dense_boundary=0, dtype=srkv.BF16)
FAKE = ctypes.c_void_p(1 << 20)  # never dereferenced: the checks reject the call first
ODD = ctypes.c_void_p((1 << 20) + 8)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return srkv.load()


def append(lib, cfg=CFG, **o):
    a = {**dict(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, off=FAKE, T=5, f=FAKE, R=128, inter=0, qo=FAKE,
                kc=FAKE, vc=FAKE, pages=10, bt=FAKE, mb=8, lens=FAKE, B=2, reps=FAKE), **o}
    return lib.srkv_append_kv_rope(ctypes.byref(srkv.config(cfg)) if cfg else None, a["q"], a["qs"], a["k"], a["ks"],
                                   a["v"], a["vs"], a["off"], a["T"], a["f"], a["R"], a["inter"], a["qo"], a["kc"],
                                   a["vc"], a["pages"], a["bt"], a["mb"], a["lens"], a["B"], a["reps"], None, None)


def test_append_checks_its_arguments(lib):
    assert append(lib, B=0) == OK and append(lib, T=0) == OK
    assert append(lib, cfg=None) == INVALID
    assert append(lib, dict(CFG, head_dim=96)) == INVALID
    for bad in (dict(q=None), dict(qo=None), dict(k=None), dict(v=None), dict(off=None), dict(f=None), dict(kc=None),
                dict(vc=None), dict(bt=None), dict(lens=None), dict(reps=None), dict(q=ODD), dict(k=ODD), dict(v=ODD),
                dict(qo=ODD), dict(kc=ODD), dict(vc=ODD), dict(reps=ODD), dict(f=ctypes.c_void_p((1 << 20) + 4)),
                dict(qs=1023), dict(qs=1020), dict(qs=1016), dict(ks=255), dict(ks=248), dict(vs=0), dict(vs=-256),
                dict(T=-1), dict(B=-1), dict(R=-2), dict(R=17), dict(R=130), dict(mb=0), dict(mb=1 << 24),
                dict(pages=0), dict(pages=-1)):
        assert append(lib, **bad) == INVALID, bad
    assert append(lib, R=24) == UNSUPPORTED
    assert append(lib, B=1 << 29) == UNSUPPORTED


def attend(lib, name, cfg=CFG, **o):
    a = {**dict(q=FAKE, qs=1024, k=FAKE, v=FAKE, pages=10, bt=FAKE, mb=8, off=FAKE, T=5, lens=FAKE, B=2, out=FAKE,
                ws=None, ws_bytes=0), **o}
    return getattr(lib, name)(ctypes.byref(srkv.config(cfg)) if cfg else None, a["q"], a["qs"], a["k"], a["v"],
                              a["pages"], a["bt"], a["mb"], a["off"], a["T"], a["lens"], a["B"], a["out"], a["ws"],
                              a["ws_bytes"], None, None)


@pytest.mark.parametrize("name", ["srkv_chunk_attention", "srkv_chunk_attention_window"])
def test_attention_checks_its_arguments(lib, name):
    assert attend(lib, name, B=0) == OK and attend(lib, name, T=0) == OK
    assert attend(lib, name, cfg=None) == INVALID
    assert attend(lib, name, dict(CFG, local_tokens=-1)) == INVALID
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(off=None), dict(lens=None),
                dict(out=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(out=ODD), dict(qs=1016), dict(qs=1028),
                dict(T=-1), dict(B=-1), dict(mb=0), dict(mb=1 << 24), dict(pages=0), dict(pages=-1)):
        assert attend(lib, name, **bad) == INVALID, bad
    assert attend(lib, name, pages=1 << 31) == UNSUPPORTED
    assert attend(lib, name, T=1 << 29) == UNSUPPORTED
    need = srkv.chunk_workspace_size(CFG, 5, 2)
    assert attend(lib, name) == WORKSPACE
    assert attend(lib, name, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert attend(lib, name, ws=ODD, ws_bytes=need) == WORKSPACE


def at(byte):
    return ctypes.c_void_p((1 << 20) + byte)


def test_outputs_that_lie_in_their_inputs_are_refused(lib):
    """5 rows of 8 heads of 128 bf16: 10240 bytes packed, 4 * stride * 2 + 2048 strided."""
    need = srkv.chunk_workspace_size(CFG, 5, 2)
    for name in ("srkv_chunk_attention", "srkv_chunk_attention_window"):
        for o in (dict(), dict(out=at(10240 - 16)), dict(q=at(10240 - 16)), dict(qs=2048, out=at(4 * 4096 + 2048 - 16))):
            assert attend(lib, name, ws=at(1 << 22), ws_bytes=need, **o) == INVALID, o
    far = dict(k=at(1 << 21), v=at(1 << 21))
    for o in (dict(qs=2048), dict(qo=at(16)), dict(q=at(10240 - 16)), dict(k=FAKE), dict(v=FAKE),
              dict(v=at(10240 - 16)), dict(k=at(1 << 10), ks=1024)):
        assert append(lib, **{**far, **o}) == INVALID, o


def test_workspace_size(lib):
    sizes = [srkv.chunk_workspace_size(CFG, t, b) for t, b in ((1, 1), (64, 64), (8192, 1), (131072, 64))]
    assert all(x % 256 == 0 for x in sizes) and sizes == sorted(sizes) and sizes[0] > 0
    assert sizes[-1] < 256 << 20
    assert srkv.chunk_workspace_size(dict(CFG, head_dim=96), 1, 1) == 0
    assert srkv.chunk_workspace_size(CFG, -1, 1) == 0 and lib.srkv_chunk_workspace_size(None, 1, 1) == 0


# ---- the binding: shapes before anything reaches the library (which sees only pointers)

B, T, MAXB, P = 3, 9, 10, 24
bf, i32, f32, f64 = torch.bfloat16, torch.int32, torch.float32, torch.float64


def tensors():
    z = lambda *s, dt=bf: torch.zeros(*s, dtype=dt)
    return dict(q=z(T, 8, 128), k_new=z(T, 2, 128), v_new=z(T, 2, 128), f=z(64, dt=f64), k=z(P, 2, 128, 128),
                v=z(P, 2, 128, 128), bt=z(B, MAXB, dt=i32), off=z(B + 1, dt=i32), lens=z(B, dt=i32),
                reps=z(P, 2, 128, dt=f32), q_out=z(T, 8, 128), out=z(T, 8, 128), ws=z(256, dt=torch.uint8), flags=None)


def call_append(**o):
    a = {**tensors(), **o}
    srkv.append_kv_rope(CFG, a["q"], a["k_new"], a["v_new"], a["f"], a["k"], a["v"], a["bt"], a["off"], a["lens"],
                        a["reps"], a["q_out"], a["flags"])


def call_chunk(**o):
    a = {**tensors(), **o}
    srkv.chunk_attention(CFG, a["q"], a["k"], a["v"], a["bt"], a["off"], a["lens"], a["out"], a["ws"], a["flags"])


def call_window(**o):
    a = {**tensors(), **o}
    srkv.chunk_attention_window(CFG, a["q"], a["k"], a["v"], a["bt"], a["off"], a["lens"], a["out"], a["ws"],
                                a["flags"])


@pytest.mark.parametrize("call", [call_append, call_chunk, call_window])
def test_the_binding_checks_shapes_then_devices(call):
    with pytest.raises(ValueError, match="CUDA"):  # every shape right: as far as the device
        call()
    bad = dict(q=(T, 7, 128), k=(P, 2, 128, 64), v=(P - 1, 2, 128, 128), off=(B,), lens=(B + 1,), bt=(B,),
               flags=(2,))
    if call is call_append:
        bad.update(k_new=(T, 8, 128), v_new=(T + 1, 2, 128), reps=(P - 1, 2, 128), q_out=(T + 1, 8, 128), f=(8, 8))
    else:
        bad.update(out=(T + 1, 8, 128))
    for name, shape in bad.items():
        with pytest.raises(ValueError, match="shape|rows"):
            call(**{name: torch.zeros(*shape)})


def test_queries_and_their_output_go_together():
    with pytest.raises(ValueError, match="together"):
        call_append(q_out=None)
    with pytest.raises(ValueError, match="together"):
        call_append(q=None)
