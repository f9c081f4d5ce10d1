"""Host-only checks of gdn_short_conv, gdn_ssm_scan, gdn_q4_linear and gdn_q4_gated: what they refuse before the GPU is
touched, and what their Python forms say."""
import ctypes

import pytest
import torch

OK, INVALID, UNSUPPORTED, ALIGNMENT, CUDA, WORKSPACE = 0, 1, 2, 3, 4, 7
P = ctypes.c_void_p
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_03_gb300 import _build, gdn
    _build.build()
    return gdn.load_library()


def at(i):
    """Aligned addresses, 64 MB apart, that are never dereferenced: every call here fails its checks first."""
    return 64 * MB * (i + 1)


def conv(lib, **kw):
    a = dict(n=2, T=5, C=64, W=4, x=at(0), xs=64, w=at(1), bias=at(2), act=1, cu=at(3), si=at(4), so=at(5), slots=None, n_slots=2,
             out=at(6))
    a.update(kw)
    return lib.gdn_short_conv(a["n"], a["T"], a["C"], a["W"], P(a["x"]), a["xs"], P(a["w"]), P(a["bias"]), a["act"], P(a["cu"]),
                              P(a["si"]), P(a["so"]), P(a["slots"]), a["n_slots"], P(a["out"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(C=60), UNSUPPORTED), (dict(C=0), INVALID), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(W=0), INVALID),
    (dict(act=2), UNSUPPORTED), (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(n_slots=1), INVALID),
    (dict(n_slots=-1), INVALID), (dict(cu=None), INVALID), (dict(cu=None, T=2, x=None), INVALID), (dict(w=None), INVALID),
    (dict(out=None), INVALID), (dict(xs=56), INVALID), (dict(xs=68), ALIGNMENT), (dict(xs=2 ** 41), INVALID),
    (dict(x=at(0) + 8), ALIGNMENT), (dict(w=at(1) + 4), ALIGNMENT), (dict(bias=at(2) + 4), ALIGNMENT), (dict(cu=at(3) + 4), ALIGNMENT),
    (dict(si=at(4) + 8), ALIGNMENT), (dict(so=at(5) + 8), ALIGNMENT), (dict(slots=at(7) + 4), ALIGNMENT), (dict(out=at(6) + 8), ALIGNMENT),
    (dict(out=at(0)), INVALID), (dict(out=at(0) + 16), INVALID), (dict(so=at(4) + 16), INVALID), (dict(so=at(6)), INVALID),
    (dict(T=2 ** 31 - 1, C=2 ** 20), UNSUPPORTED)])
def test_conv_refuses(lib, kw, status):
    assert conv(lib, **kw) == status


def scan(lib, **kw):
    a = dict(n=2, T=5, C=64, N=16, G=2, x=at(0), xs=64, dt=at(1), ds=64, a=at(2), b=at(3), bs=32, c=at(4), cs=32, skip=at(5), z=at(6),
             zs=64, bias=at(7), sp=1, cu=at(8), ml=3, si=at(9), so=at(10), slots=None, n_slots=2, out=at(11), odt=0, ws=at(12),
             wsb=32 * MB)
    a.update(kw)
    return lib.gdn_ssm_scan(a["n"], a["T"], a["C"], a["N"], a["G"], P(a["x"]), a["xs"], P(a["dt"]), a["ds"], P(a["a"]), P(a["b"]),
                            a["bs"], P(a["c"]), a["cs"], P(a["skip"]), P(a["z"]), a["zs"], P(a["bias"]), a["sp"], P(a["cu"]), a["ml"],
                            P(a["si"]), P(a["so"]), P(a["slots"]), a["n_slots"], P(a["out"]), a["odt"], P(a["ws"]), a["wsb"], None)


SHAPES = [(dict(C=0), INVALID), (dict(C=60), UNSUPPORTED), (dict(C=24), UNSUPPORTED), (dict(N=8), UNSUPPORTED), (dict(N=0), INVALID),
          (dict(G=0), INVALID), (dict(G=3), UNSUPPORTED), (dict(ml=-1), INVALID), (dict(T=2 ** 30, C=2 ** 20, G=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", SHAPES + [
    (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(odt=2), UNSUPPORTED), (dict(sp=2), INVALID),
    (dict(n_slots=1), INVALID), (dict(cu=None), INVALID), (dict(x=None), INVALID), (dict(dt=None), INVALID), (dict(a=None), INVALID),
    (dict(b=None), INVALID), (dict(c=None), INVALID), (dict(out=None), INVALID), (dict(xs=56), INVALID), (dict(ds=68), ALIGNMENT),
    (dict(bs=24), INVALID), (dict(cs=36), ALIGNMENT), (dict(zs=0), INVALID), (dict(x=at(0) + 2), ALIGNMENT),
    (dict(b=at(3) + 8), ALIGNMENT), (dict(a=at(2) + 4), ALIGNMENT), (dict(skip=at(5) + 4), ALIGNMENT), (dict(bias=at(7) + 4), ALIGNMENT),
    (dict(out=at(0)), INVALID), (dict(so=at(9) + 16), INVALID), (dict(so=at(2)), INVALID), (dict(ws=at(12) + 16), ALIGNMENT)])
def test_scan_refuses(lib, kw, status):
    assert scan(lib, **kw) == status


@pytest.mark.parametrize("kw,status", SHAPES)
def test_scan_workspace_refuses(lib, kw, status):
    a = dict(n=2, T=5, C=64, N=16, G=2, ml=3)
    a.update(kw)
    st = ctypes.c_int(-1)
    assert lib.gdn_ssm_scan_workspace_size(a["n"], a["T"], a["C"], a["N"], a["G"], a["ml"], st) == 0
    assert st.value == status


def q4(lib, gated, **kw):
    a = dict(rows=3, n=40, k=256, group=64, x=at(0), xs=256, codes=at(1), scales=at(2), offsets=at(3), codes2=at(4), scales2=at(5),
             offsets2=at(6), act=0, out=at(7), odt=0, ws=at(8), wsb=32 * MB)
    a.update(kw)
    first = (a["rows"], a["n"], a["k"], a["group"], P(a["x"]), a["xs"], P(a["codes"]), P(a["scales"]), P(a["offsets"]))
    if gated:
        return lib.gdn_q4_gated(*first, P(a["codes2"]), P(a["scales2"]), P(a["offsets2"]), a["act"], P(a["out"]), a["odt"], P(a["ws"]),
                                a["wsb"], None)
    return lib.gdn_q4_linear(*first, P(a["out"]), a["odt"], P(a["ws"]), a["wsb"], None)


MANY = dict(rows=100, n=4000, k=2048, xs=2048)                # a call that needs a workspace


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(k=96), UNSUPPORTED), (dict(group=32), UNSUPPORTED),
    (dict(group=128, k=192), UNSUPPORTED), (dict(k=65536 + 64, xs=2 ** 17), UNSUPPORTED), (dict(odt=2), UNSUPPORTED),
    (dict(rows=2 ** 31 - 1), UNSUPPORTED), (dict(n=2 ** 31 - 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(codes=None), INVALID),
    (dict(scales=None), INVALID), (dict(out=None), INVALID), (dict(xs=248), INVALID), (dict(xs=260), ALIGNMENT),
    (dict(x=at(0) + 8), ALIGNMENT), (dict(codes=at(1) + 8), ALIGNMENT), (dict(scales=at(2) + 2), ALIGNMENT),
    (dict(offsets=at(3) + 2), ALIGNMENT), (dict(out=at(7) + 2), ALIGNMENT), (dict(out=at(0)), INVALID), (dict(out=at(2) + 16), INVALID),
    (dict(MANY, ws=None), WORKSPACE), (dict(MANY, wsb=100 * 2048 * 2), WORKSPACE), (dict(MANY, ws=at(8) + 16), ALIGNMENT),
    (dict(MANY, ws=at(1)), INVALID)])
def test_q4_refuses(lib, gated, kw, status):
    assert q4(lib, gated, **kw) == status
    assert q4(lib, gated, rows=0) == OK


def test_q4_workspace(lib):
    st = ctypes.c_int(-1)
    size = lambda *a: (lib.gdn_q4_workspace_size(*a, st), st.value)  # noqa: E731
    assert size(1, 40, 256, 64, 0) == (0, OK) and size(1000, 40, 256, 64, 1) == (0, OK)
    assert size(100, 40, 256, 64, 0) == (0, OK) and size(1000, 4000, 2048, 64, 1) == (0, OK)
    assert size(100, 4000, 2048, 64, 0)[0] >= 100 * 2048 * 2 and size(1000, 400, 256, 64, 0)[0] >= 1000 * 256 * 2
    for bad, status in (((-1, 40, 256, 64, 0), INVALID), ((1, 40, 250, 64, 0), UNSUPPORTED), ((1, 40, 256, 64, 2), UNSUPPORTED)):
        assert size(*bad) == (0, status)


@pytest.mark.parametrize("kw,status", [(dict(act=2), UNSUPPORTED), (dict(codes2=None), INVALID), (dict(scales2=None), INVALID),
                                       (dict(offsets2=None), INVALID), (dict(offsets=None), INVALID), (dict(codes2=at(4) + 8), ALIGNMENT),
                                       (dict(out=at(4)), INVALID)])
def test_gated_refuses(lib, kw, status):
    assert q4(lib, True, **kw) == status


def test_python_forms_want_cuda_tensors(lib):
    from gated_deltanet_linear_03_gb300 import linear, ssm
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ssm.short_conv(x, torch.zeros(64, 4))
    with pytest.raises(ValueError, match="CUDA"):
        ssm.scan(x, x, torch.zeros(64, 16), x.view(4, 1, 64)[..., :16], x.view(4, 1, 64)[..., :16])
    w = linear.quantize(torch.randn(8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        linear.q4_linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        linear.q4_gated(x, w, w)
    turned = linear.quantize(torch.randn(64, 8).T)
    assert turned.codes.is_contiguous() and turned.scales.is_contiguous() and turned.offsets.is_contiguous()
    with pytest.raises(ValueError):
        linear.quantize(torch.randn(8, 96))
    with pytest.raises(ValueError):
        linear.quantize(torch.randn(8, 64), group=32)
