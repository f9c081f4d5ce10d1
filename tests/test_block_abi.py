"""Host-only checks of gdn_kv_append, gdn_kv_read, gdn_attend and gdn_block_norm: what they refuse before the GPU is
touched, and the workspace sizes of gdn_attend."""
import ctypes

import pytest

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 7
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


def append(lib, **kw):
    a = dict(n=2, T=5, hq=4, hkv=2, d=128, rot=64, q=at(0), qs=512, k=at(1), ks=256, v=at(2), vs=256, cos=at(3),
             sin=at(4), npos=100, il=0, cu=at(5), past=at(6), table=at(7), max_pages=4, n_pages=8, page=32, fmt=0,
             kp=at(8), vp=at(9), ksc=at(10), vsc=at(11), oi=at(12), oo=at(13), slots=None, n_slots=2, qo=at(14))
    a.update(kw)
    return lib.gdn_kv_append(a["n"], a["T"], a["hq"], a["hkv"], a["d"], a["rot"], P(a["q"]), a["qs"], P(a["k"]), a["ks"],
                             P(a["v"]), a["vs"], P(a["cos"]), P(a["sin"]), a["npos"], a["il"], P(a["cu"]), P(a["past"]),
                             P(a["table"]), a["max_pages"], a["n_pages"], a["page"], a["fmt"], P(a["kp"]), P(a["vp"]),
                             P(a["ksc"]), P(a["vsc"]), P(a["oi"]), P(a["oo"]), P(a["slots"]), a["n_slots"], P(a["qo"]), None)


def read(lib, **kw):
    a = dict(n=2, T=5, hkv=2, d=128, cu=at(0), table=at(1), max_pages=4, n_pages=8, page=32, fmt=0, kp=at(2), vp=at(3),
             ksc=at(4), vsc=at(5), ko=at(6), vo=at(7), odt=0)
    a.update(kw)
    return lib.gdn_kv_read(a["n"], a["T"], a["hkv"], a["d"], P(a["cu"]), P(a["table"]), a["max_pages"], a["n_pages"],
                           a["page"], a["fmt"], P(a["kp"]), P(a["vp"]), P(a["ksc"]), P(a["vsc"]), P(a["ko"]), P(a["vo"]),
                           a["odt"], None)


def workspace(lib, n=2, T=5, hq=4, hkv=2, d=128, mq=3, mk=100):
    st = ctypes.c_int(-1)
    need = lib.gdn_attend_workspace_size(n, T, hq, hkv, d, mq, mk, st)
    return need, st.value


def attend(lib, **kw):
    a = dict(n=2, T=5, hq=4, hkv=2, d=128, q=at(0), kp=at(1), vp=at(2), ksc=at(3), vsc=at(4), table=at(5), max_pages=4,
             n_pages=8, page=32, fmt=0, cu=at(6), lens=at(7), mq=3, mk=100, scale=0.1, window=0, sinks=0, out=at(8),
             odt=0, ws=at(9), wsb=32 * MB)
    a.update(kw)
    return lib.gdn_attend(a["n"], a["T"], a["hq"], a["hkv"], a["d"], P(a["q"]), P(a["kp"]), P(a["vp"]), P(a["ksc"]),
                          P(a["vsc"]), P(a["table"]), a["max_pages"], a["n_pages"], a["page"], a["fmt"], P(a["cu"]),
                          P(a["lens"]), a["mq"], a["mk"], a["scale"], a["window"], a["sinks"], P(a["out"]), a["odt"],
                          P(a["ws"]), a["wsb"], None)


def norm(lib, **kw):
    a = dict(rows=4, dim=256, x=at(0), gate=at(1), act=0, res=at(2), rdt=0, post=at(3), pre=at(4), sw=None, scale=1.0,
             eps=1e-6, ro=at(5), out=at(6))
    a.update(kw)
    return lib.gdn_block_norm(a["rows"], a["dim"], P(a["x"]), P(a["gate"]), a["act"], P(a["res"]), a["rdt"], P(a["post"]),
                              P(a["pre"]), P(a["sw"]), a["scale"], a["eps"], P(a["ro"]), P(a["out"]), None)


POOL = [(dict(d=96), UNSUPPORTED), (dict(d=0), INVALID), (dict(page=24), UNSUPPORTED), (dict(page=8192), UNSUPPORTED),
        (dict(page=0), INVALID), (dict(fmt=2), UNSUPPORTED), (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID),
        (dict(n_pages=2**25, page=64), UNSUPPORTED)]       # pool rows are counted in 31 bits


@pytest.mark.parametrize("kw,status", POOL + [
    (dict(hkv=0), INVALID), (dict(T=-1), INVALID), (dict(n=-1), INVALID), (dict(n=0), INVALID), (dict(hq=5), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(rot=-16), INVALID), (dict(rot=144), INVALID), (dict(cos=None), INVALID),
    (dict(sin=None), INVALID), (dict(npos=-1), INVALID), (dict(il=2), INVALID), (dict(qo=None), INVALID),
    (dict(q=None), INVALID), (dict(ks=255), INVALID), (dict(vs=260), ALIGNMENT), (dict(qs=500), INVALID),
    (dict(qs=516), ALIGNMENT), (dict(k=at(1) + 8), ALIGNMENT), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(cu=None), INVALID), (dict(past=None), INVALID), (dict(table=None), INVALID), (dict(oi=None), INVALID),
    (dict(n_slots=1), INVALID), (dict(kp=at(9)), INVALID), (dict(oo=at(1)), INVALID), (dict(qo=at(2)), INVALID),
    (dict(q=at(14), qs=520), INVALID),                      # in place, the queries are packed
    (dict(ksc=at(8) + 64), INVALID), (dict(T=2**30, hq=2**12, qs=2**19), UNSUPPORTED)])
def test_append_refuses(lib, kw, status):
    assert append(lib, **kw) == status


def test_append_of_no_sequences_is_done(lib):
    assert append(lib, n=0, T=0) == 0


@pytest.mark.parametrize("kw,status", POOL + [
    (dict(hkv=0), INVALID), (dict(n=-1), INVALID), (dict(T=-1), INVALID), (dict(n=0), INVALID), (dict(odt=5), UNSUPPORTED),
    (dict(cu=None), INVALID), (dict(ko=None), INVALID), (dict(vo=at(7) + 8), ALIGNMENT), (dict(ko=at(2)), INVALID),
    (dict(vo=at(6)), INVALID)])
def test_read_refuses(lib, kw, status):
    assert read(lib, **kw) == status


def test_read_of_no_tokens_is_done(lib):
    assert read(lib, T=0) == 0


@pytest.mark.parametrize("kw,status", POOL + [
    (dict(hkv=3), INVALID), (dict(hq=0), INVALID), (dict(mq=-1), INVALID), (dict(mq=0), INVALID), (dict(mk=-1), INVALID),
    (dict(mk=129), INVALID),                                # more than the table's pages hold
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID),
    (dict(sinks=-1), INVALID), (dict(odt=5), UNSUPPORTED), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=at(0) + 8), ALIGNMENT), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE),
    (dict(ws=at(9) + 16), ALIGNMENT), (dict(out=at(0)), INVALID), (dict(out=at(9)), INVALID), (dict(ws=at(1)), INVALID),
    (dict(T=2**28, hq=8), UNSUPPORTED)])                    # query rows are counted in 31 bits
def test_attend_refuses(lib, kw, status):
    assert attend(lib, **kw) == status


def test_attend_of_no_tokens_is_done(lib):
    assert attend(lib, T=0, mq=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), INVALID), (dict(dim=0), INVALID), (dict(dim=260), UNSUPPORTED), (dict(dim=16392), UNSUPPORTED),
    (dict(rdt=5), UNSUPPORTED), (dict(act=2), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(x=None), INVALID), (dict(res=None), INVALID), (dict(pre=None), INVALID),
    (dict(ro=None), INVALID), (dict(out=None), INVALID), (dict(x=at(0) + 8), ALIGNMENT), (dict(gate=at(1) + 2), ALIGNMENT),
    (dict(out=at(2)), INVALID), (dict(ro=at(0)), INVALID), (dict(ro=at(6)), INVALID), (dict(x=at(6) + 256), INVALID)])
def test_norm_refuses(lib, kw, status):
    assert norm(lib, **kw) == status


def test_norm_of_no_rows_is_done(lib):
    assert norm(lib, rows=0) == 0


def test_workspace_sizes(lib):
    assert workspace(lib, T=0, n=2, mq=0) == (0, 0)
    small, st = workspace(lib)
    assert st == 0 and small > 0
    # bounds may be loose: no sequence is longer than all of them together
    assert workspace(lib, T=5, mq=1000) == workspace(lib, T=5, mq=5)
    # few rows: parts of 64 cached tokens, at most two a CTA, so a long cache costs no more than so many CTAs
    assert workspace(lib, n=1, T=1, mq=1, mk=2**30) == workspace(lib, n=1, T=1, mq=1, mk=2**29)
    # prompts: a list of items that grows with the rows, beside parts that do not
    a, b = (workspace(lib, n=1, T=t, mq=t, mk=t)[0] for t in (4096, 65536))
    assert 0 < b - a < 64 * (65536 - 4096)
    assert workspace(lib, n=-1)[1] == INVALID and workspace(lib, hkv=3)[1] == INVALID
    assert workspace(lib, d=96)[1] == UNSUPPORTED


def test_python_refuses_tensors_that_are_not_on_a_gpu():
    import torch
    from gated_deltanet_linear_03_gb300 import attn, norm as norm_module
    x, w = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    with pytest.raises(ValueError, match="CUDA"):
        norm_module.block_norm(x, x, w)
    cache = attn.alloc_cache(4, 2, 32, 64, 1, device="cpu")
    table, cu, lens = torch.zeros(1, 4, dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        attn.attend(torch.zeros(1, 4, 64, dtype=torch.bfloat16), *cache[:4], table, cu, lens, max_q_len=1, max_kv_len=32)
    kv = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        attn.kv_append(kv, kv, None, None, cu, lens, table, *cache)
