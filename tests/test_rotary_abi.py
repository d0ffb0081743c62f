"""Rotary operators on the host: argument checks of the C entry points (nothing here
reaches a launch) and of the binding."""
import pytest
import torch

import gated_deltanet_linear_core_gb300 as gdn
from gated_deltanet_linear_core_gb300 import _lib as E

no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="host-only validation tests use fake device addresses")
A = 0x7f0000000000  # fake 16-byte-aligned address (never dereferenced)
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_core_gb300 import build
    build.build()
    return E.load()


def rope(lib, **kw):
    a = dict(x=A, xt=1024, xh=128, pos=A + 0x1000, n_axes=1, axes=None, f=A + 0x2000, w=None, eps=1e-6, mscale=1.0, flags=0,
             out=A + 0x3000, ot=1024, oh=128, T=4, H=8, D=128, R=64, dt=E.GDN_BF16)
    a.update(kw)
    return lib.gdn_rope(a["x"], a["xt"], a["xh"], a["pos"], a["n_axes"], a["axes"], a["f"], a["w"], a["eps"], a["mscale"],
                        a["flags"], a["out"], a["ot"], a["oh"], a["T"], a["H"], a["D"], a["R"], a["dt"], None)


@no_gpu
def test_rope_refusals(lib):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(dt=5), dict(T=-1), dict(T=1 << 31), dict(H=0), dict(D=0), dict(R=0), dict(R=63), dict(R=130), dict(R=-2),
                dict(n_axes=0), dict(flags=2), dict(mscale=nan), dict(mscale=inf), dict(w=A, eps=0.0), dict(w=A, eps=nan),
                dict(w=A, eps=inf), dict(w=A, eps=-1.0), dict(x=None), dict(out=None), dict(pos=None), dict(f=None),
                dict(xt=-1024), dict(xh=-128), dict(xt=BIG), dict(xh=BIG), dict(ot=BIG), dict(oh=BIG),
                # outputs whose rows overlap
                dict(ot=512), dict(oh=64), dict(ot=0), dict(oh=0), dict(ot=128, oh=128), dict(ot=128, oh=384),
                dict(out=A, ot=2048)):
        assert rope(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(D=12, R=4), dict(D=264), dict(H=65537, oh=128, ot=65537 * 128), dict(n_axes=17)):
        assert rope(lib, **bad) == E.GDN_ERR_UNSUPPORTED, bad
    for bad in (dict(x=A + 8), dict(out=A + 2), dict(pos=A + 2), dict(axes=A + 2), dict(f=A + 2), dict(w=A + 2),
                dict(xt=1028), dict(xh=132), dict(ot=1028), dict(oh=132)):
        assert rope(lib, **bad) == E.GDN_ERR_ALIGN, bad
    assert rope(lib, T=0, x=None, out=None) == E.GDN_OK


def append(lib, **kw):
    a = dict(q=A, qt=4096, qh=256, k=A + 0x1000, kt=512, kh=256, v=A + 0x2000, vt=512, vh=256, o=A + 0x3000, kc=A + 0x4000,
             vc=A + 0x5000, table=A + 0x6000, lens=A + 0x7000, cu=None, pos=None, n_axes=1, axes=None, f=A + 0x8000, qw=None,
             kw=None, eps=1e-6, mscale=1.0, flags=0, B=2, T=6, hq=16, hkv=2, D=256, R=64, page=16, n_pages=100, max_pages=50,
             dt=E.GDN_BF16)
    a.update(kw)
    return lib.gdn_rope_kv_append(
        a["q"], a["qt"], a["qh"], a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"], a["o"], a["kc"], a["vc"], a["table"],
        a["lens"], a["cu"], a["pos"], a["n_axes"], a["axes"], a["f"], a["qw"], a["kw"], a["eps"], a["mscale"], a["flags"],
        a["B"], a["T"], a["hq"], a["hkv"], a["D"], a["R"], a["page"], a["n_pages"], a["max_pages"], a["dt"], None)


@no_gpu
def test_append_refusals(lib):
    nan = float("nan")
    for bad in (dict(dt=5), dict(B=-1), dict(B=0), dict(T=-1), dict(T=7), dict(T=1 << 31), dict(hq=0), dict(hkv=0), dict(D=0),
                dict(R=0), dict(R=257), dict(R=258), dict(page=0), dict(n_pages=0), dict(max_pages=0), dict(n_axes=0),
                dict(n_axes=3), dict(flags=4), dict(mscale=nan), dict(qw=A, eps=0.0), dict(kw=A, eps=nan), dict(q=None),
                dict(k=None), dict(v=None), dict(o=None), dict(kc=None), dict(vc=None), dict(table=None), dict(lens=None),
                dict(f=None), dict(qt=-8), dict(kh=-8), dict(vt=BIG), dict(o=A, qt=8192), dict(o=A, qh=512)):
        assert append(lib, **bad) == E.GDN_ERR_INVALID_ARG, bad
    for bad in (dict(D=12, R=2), dict(D=512), dict(max_pages=1 << 27), dict(hkv=1 << 20), dict(hq=1 << 20),
                dict(n_axes=17, pos=A)):
        assert append(lib, **bad) == E.GDN_ERR_UNSUPPORTED, bad
    for bad in (dict(q=A + 2), dict(k=A + 8), dict(v=A + 8), dict(o=A + 8), dict(kc=A + 8), dict(vc=A + 8), dict(table=A + 2),
                dict(lens=A + 2), dict(cu=A + 2), dict(pos=A + 2), dict(axes=A + 1), dict(f=A + 2), dict(qw=A + 2),
                dict(kw=A + 2), dict(qt=4100), dict(qh=260), dict(kt=516), dict(kh=260), dict(vt=516), dict(vh=260)):
        assert append(lib, **bad) == E.GDN_ERR_ALIGN, bad
    assert append(lib, T=0, B=0, q=None) == E.GDN_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    c = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 3), dtype=torch.int32)
    f = torch.ones(32)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_rope(x, f, i[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_rope_kv_append(x, x, x, c, c, i, i[:, 0], f)


def test_binding_checks_shapes():
    x = torch.zeros((5, 2, 64))
    for bad in (x[0], x[:, :1], x[:4], x[:, :, :32]):
        with pytest.raises(ValueError, match="k: shape"):
            gdn._rows(bad, "k", -1, torch.float32, 5, 64, 2)
    with pytest.raises(ValueError, match="contiguous"):
        gdn._rows(torch.zeros((5, 64, 2)).transpose(1, 2), "k", -1, torch.float32, 5, 64, 2)
    with pytest.raises(TypeError, match="dtype"):
        gdn._rows(x.half(), "k", -1, torch.float32, 5, 64, 2)
    with pytest.raises(ValueError, match="different devices"):
        gdn._rows(x, "k", 0, torch.float32, 5, 64, 2)
    i = torch.zeros(5, dtype=torch.int32)
    for f, pos, match in ((torch.ones(33), i, "inv_freq"), (torch.ones(0), i, "inv_freq"), (torch.ones((2, 3)), i, "inv_freq"),
                          (torch.ones(32), i[:4], "positions"), (torch.ones(32), torch.zeros((5, 3), dtype=torch.int32), "positions")):
        with pytest.raises(ValueError, match=match):
            gdn._rotation(f, pos, None, 5, 64, -1)
