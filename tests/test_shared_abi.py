"""Attention behind shared prefixes on the host: argument checks of the C entry points
(nothing here reaches a launch), workspace sizes, and checks of the binding."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
from gated_deltanet_linear_core_gb300 import _lib as E

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host-only validation tests use fake device addresses")
A = 0x7f0000000000  # fake 16-byte-aligned address (never dereferenced)


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_core_gb300 import build
    build.build()
    return E.load()


def shared(lib, **kw):
    a = dict(q=A, kc=A + 0x1000, vc=A + 0x2000, table=A + 0x3000, lens=A + 0x4000, pre=A + 0x4100, cu=A + 0x4200, scale=0.0,
             gate=None, out=A + 0x5000, lse=None, B=4, K=1, hq=16, hkv=2, D=256, page=16, n_pages=100, max_pages=50, G=2,
             ws=A + 0x10000, ws_bytes=1 << 40, dt=E.GDN_BF16)
    a.update(kw)
    return lib.gdn_attn_decode_shared(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["pre"], a["cu"], a["scale"],
                                      a["gate"], a["out"], a["lse"], a["B"], a["K"], a["hq"], a["hkv"], a["D"], a["page"],
                                      a["n_pages"], a["max_pages"], a["G"], a["ws"], a["ws_bytes"], a["dt"], None)


@no_gpu
def test_refusals(lib):
    for bad in (dict(dt=5), dict(B=-1), dict(K=17), dict(K=-1), dict(hq=15), dict(hq=0), dict(hkv=0), dict(D=0),
                dict(page=0), dict(n_pages=0), dict(max_pages=0), dict(scale=-0.5), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(G=0), dict(G=-1), dict(G=1 << 25), dict(cu=None), dict(q=None), dict(kc=None),
                dict(vc=None), dict(table=None), dict(lens=None), dict(pre=None), dict(out=None)):
        assert shared(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(D=264), dict(D=12), dict(max_pages=1 << 27), dict(page=1 << 30, hkv=2), dict(hq=131072, hkv=2),
                dict(B=1 << 22, K=16, hq=32)):
        assert shared(lib, **bad) == E.GDN_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 2), dict(kc=A + 8), dict(vc=A + 4), dict(table=A + 2), dict(lens=A + 1), dict(pre=A + 2),
                dict(cu=A + 2), dict(out=A + 2), dict(gate=A + 2), dict(lse=A + 2), dict(ws=A + 4)):
        assert shared(lib, **bad) == E.GDN_ERR_ALIGN, bad
    need = lib.gdn_attn_decode_shared_workspace_size(4, 1, 16, 2, 256, 16, 2, E.GDN_BF16)
    assert shared(lib, ws=None) == E.GDN_ERR_WORKSPACE
    assert shared(lib, ws_bytes=need - 1) == E.GDN_ERR_WORKSPACE
    assert shared(lib, B=0) == E.GDN_OK and shared(lib, K=0, q=None) == E.GDN_OK


@no_gpu
def test_selftest_refusals(lib):
    def call(stop_at, page, ws):
        return lib.gdn_selftest_attn_decode_shared(A, A, A, A, A, A, A, 2, 1, 16, 2, 256, page, 100, 50, ws, 1 << 40, stop_at,
                                                   None)
    assert call(-1, 16, A) == E.GDN_ERR_INVALID_ARG
    assert call(0, 6, A) == E.GDN_ERR_UNSUPPORTED
    assert call(0, 16, None) == E.GDN_ERR_WORKSPACE


def test_workspace_sizes(lib):
    f = gdn.gdn_attn_decode_shared_workspace_size
    assert f(0, 1, 16, 2, 256, 16, torch.bfloat16) == 0 and f(1, 17, 16, 2, 256, 16, torch.bfloat16) == 0
    assert f(4, 1, 16, 2, 256, 16, torch.bfloat16, 0) == 0
    for dt in (torch.bfloat16, torch.float32):
        for sizes in ([f(4, K, 16, 2, 256, 16, dt) for K in (1, 2, 4, 8, 16)], [f(B, 2, 16, 2, 256, 16, dt) for B in (1, 30, 900)],
                      [f(4000, 1, 16, 2, 256, 16, dt, G) for G in (1, 100, 4000)]):
            assert sizes[0] > 0 and sizes == sorted(sizes)


def test_binding_refuses_host_tensors():
    z = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_attn_decode_shared(z, c, c, i, i[:, 0], i[:, 0])
