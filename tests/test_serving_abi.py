"""Serving operators on the host: argument checks of the C entry points (nothing
here reaches a launch) and workspace sizes."""
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


def attn(lib, **kw):
    a = dict(q=A, kc=A + 0x1000, vc=A + 0x2000, table=A + 0x3000, lens=A + 0x4000, scale=0.0, gate=None,
             out=A + 0x5000, lse=None, B=2, K=1, hq=16, hkv=2, D=256, page=16, n_pages=100, max_pages=50,
             ws=A + 0x10000, ws_bytes=1 << 40, dt=E.GDN_BF16)
    a.update(kw)
    return lib.gdn_attn_decode(a["q"], a["kc"], a["vc"], a["table"], a["lens"], a["scale"], a["gate"], a["out"],
                               a["lse"], a["B"], a["K"], a["hq"], a["hkv"], a["D"], a["page"], a["n_pages"],
                               a["max_pages"], a["ws"], a["ws_bytes"], a["dt"], None)


@no_gpu
def test_attention_refusals(lib):
    for bad in (dict(dt=5), dict(B=-1), dict(K=17), dict(K=-1), dict(hq=15), dict(hq=0), dict(hkv=0), dict(D=0),
                dict(page=0), dict(n_pages=0), dict(max_pages=0), dict(scale=-0.5), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(q=None), dict(kc=None), dict(vc=None), dict(table=None),
                dict(lens=None), dict(out=None)):
        assert attn(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(D=264), dict(D=12), dict(max_pages=1 << 27), dict(page=1 << 30, hkv=2),
                dict(hq=131072, hkv=2)):
        assert attn(lib, **bad) == E.GDN_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 2), dict(kc=A + 8), dict(vc=A + 4), dict(table=A + 2), dict(lens=A + 1), dict(out=A + 2),
                dict(gate=A + 2), dict(lse=A + 2), dict(ws=A + 4)):
        assert attn(lib, **bad) == E.GDN_ERR_ALIGN, bad
    need = lib.gdn_attn_decode_workspace_size(2, 1, 16, 2, 256, 16, E.GDN_BF16)
    assert attn(lib, ws=None) == E.GDN_ERR_WORKSPACE
    assert attn(lib, ws_bytes=need - 1) == E.GDN_ERR_WORKSPACE
    assert attn(lib, B=0) == E.GDN_OK and attn(lib, K=0, q=None) == E.GDN_OK


@no_gpu
def test_selftest_refusals(lib):
    def call(stop_at, page, ws):
        return lib.gdn_selftest_attn_decode(A, A, A, A, A, A, 2, 1, 16, 2, 256, page, 100, 50, ws, 1 << 40, stop_at, None)
    assert call(-1, 16, A) == E.GDN_ERR_INVALID_ARG
    assert call(0, 6, A) == E.GDN_ERR_UNSUPPORTED
    assert call(0, 16, None) == E.GDN_ERR_WORKSPACE


def test_workspace_sizes(lib):
    f = gdn.gdn_attn_decode_workspace_size
    assert f(0, 1, 16, 2, 256, 16, torch.bfloat16) == 0 and f(1, 17, 16, 2, 256, 16, torch.bfloat16) == 0
    for dt in (torch.bfloat16, torch.float32):
        sizes = [f(4, K, 16, 2, 256, 16, dt) for K in (1, 2, 4, 8, 16)]
        assert sizes[0] > 0 and sizes == sorted(sizes)
        # the lengths do not matter, nor does the batch
        assert f(4, 2, 16, 2, 256, 16, dt) == f(4000, 2, 16, 2, 256, 16, dt)


def append(lib, **kw):
    a = dict(k=A, v=A + 0x1000, kc=A + 0x2000, vc=A + 0x3000, table=A + 0x4000, lens=A + 0x5000, cu=None, B=2, T=6,
             hkv=2, D=256, page=16, n_pages=100, max_pages=50, dt=E.GDN_BF16)
    a.update(kw)
    return lib.gdn_kv_append(a["k"], a["v"], a["kc"], a["vc"], a["table"], a["lens"], a["cu"], a["B"], a["T"],
                             a["hkv"], a["D"], a["page"], a["n_pages"], a["max_pages"], a["dt"], None)


@no_gpu
def test_append_refusals(lib):
    for bad in (dict(dt=5), dict(B=-1), dict(B=0), dict(T=-1), dict(T=7), dict(T=1 << 31), dict(hkv=0), dict(D=0), dict(page=0),
                dict(n_pages=0), dict(max_pages=0), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None),
                dict(table=None), dict(lens=None)):
        assert append(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(D=12), dict(D=512), dict(max_pages=1 << 27), dict(hkv=1 << 20)):
        assert append(lib, **bad) == E.GDN_ERR_UNSUPPORTED, bad
    for bad in (dict(k=A + 2), dict(v=A + 8), dict(kc=A + 8), dict(vc=A + 8), dict(table=A + 2), dict(lens=A + 2),
                dict(cu=A + 2)):
        assert append(lib, **bad) == E.GDN_ERR_ALIGN, bad
    assert append(lib, T=0) == E.GDN_OK


def accept(lib, **kw):
    a = dict(p=A, q=A + 0x1000, draft=A + 0x2000, u=A + 0x3000, nd=None, slots=None, B=2, K=3, V=1000, n=A + 0x4000,
             tok=A + 0x5000, ns=None, dt=E.GDN_F32)
    a.update(kw)
    return lib.gdn_draft_accept(a["p"], a["q"], a["draft"], a["u"], a["nd"], a["slots"], a["B"], a["K"], a["V"],
                                a["n"], a["tok"], a["ns"], a["dt"], None)


@no_gpu
def test_acceptance_refusals(lib):
    for bad in (dict(dt=5), dict(B=-1), dict(K=-1), dict(K=16), dict(V=0), dict(V=(1 << 24) + 1), dict(p=None),
                dict(draft=None), dict(u=None), dict(n=None), dict(tok=None), dict(slots=A), dict(ns=A)):
        assert accept(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(p=A + 4), dict(q=A + 4), dict(draft=A + 2), dict(u=A + 2), dict(nd=A + 2), dict(n=A + 2),
                dict(tok=A + 2), dict(slots=A + 2, ns=A), dict(slots=A, ns=A + 2)):
        assert accept(lib, **bad) == E.GDN_ERR_ALIGN, bad
    assert accept(lib, B=0) == E.GDN_OK


def test_binding_refuses_host_tensors():
    z = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_attn_decode(z, c, c, i, i[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_kv_append(z[0], z[0], c, c, i, i[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_draft_accept(torch.zeros((1, 2, 9)), None, torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2)))


def test_binding_refuses_a_stream_of_another_device(monkeypatch):
    """It would run on the tensors' device's current stream, not on the one named."""
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0x1234
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    ran = []
    with pytest.raises(ValueError, match="stream: on cuda:1, the tensors are on cuda:0"):
        gdn._on_stream(0, Stream(), (), lambda: ran.append(1))
    assert not ran
