"""gdn_attend and table entries: what a page outside the pool reads as, for both kernels and both formats."""
import math

import pytest
import torch

import attn_helpers as ref
from test_gpu_attend import F8, I8, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d,m", [(64, 1), (128, 1), (256, 1), (64, 40), (64, 270), (128, 70), (256, 140)])
def test_pages_outside_the_pool_read_as_zeros(attn, d, m, dtype):
    """Whatever the pool holds, its first rows included: here codes 0x7F (NaN in 8-bit floats) and NaN scales."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    page, lens = 16, [m + 150]
    cache = ref.make_cache(lens, 2, d, page, dtype, 7)
    n_pages = cache.k_pages.shape[0]
    used = set(cache.table[0, :-(-lens[0] // page)].tolist())
    zero, spoilt = [p for p in range(n_pages) if p not in used][:2]
    for pages, scales in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        raw = pages.view(torch.uint8)
        raw[zero], scales[zero] = 0, 2.0 ** -60 / ref.QMAX[dtype]
        raw[spoilt], scales[spoilt] = 0x7F, math.nan
    # the spoilt page is moved to the front of the pool, where a row that does not exist might be looked for
    order = list(range(n_pages))
    order[0], order[spoilt] = order[spoilt], order[0]
    back = torch.tensor([order.index(p) for p in range(n_pages)], dtype=torch.int32)
    moved = ref.Cache(back[cache.table.long()], *[x.view(torch.uint8)[order].view(x.dtype) if x.element_size() == 1 else x[order]
                                                  for x in cache.args])
    zero = int(back[zero])
    q = torch.randn(m, 4, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    gone = (1, 4, 5)                                        # pages of the middle; every query sees them
    for bad in (-1, n_pages, 2 ** 31 - 1, -2 ** 31):
        a, b = moved.table.clone(), moved.table.clone()
        a[0, list(gone)], b[0, list(gone)] = bad, zero
        out, cu = run(attn, q, ref.Cache(a, *moved.args), [m], lens)
        assert gdn.device_error() == 6
        check(out, *ref.attend(q, ref.Cache(b, *moved.args), cu, lens))



@pytest.mark.parametrize("kv", [64, 5000])
def test_replays_without_queries(attn, kv):
    """A captured call of a few items, replayed while its sequences come and go: without any query it writes nothing, and the
    kernel after it may change the lengths."""
    lens = [kv, kv - 7]
    cache = ref.make_cache(lens, 2, 128, 32, I8, 3)
    c = cache.on("cuda")
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    qd, cu, length = q.cuda(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    none, both = torch.zeros_like(cu), cu.clone()
    out = torch.empty(2, 8, 128, device="cuda")
    ws = torch.empty(attn.attend_workspace_size(2, 2, 8, 2, 128, 1, kv), dtype=torch.uint8, device="cuda")
    kw = dict(max_q_len=1, max_kv_len=kv, out=out, workspace=ws)
    attn.attend(qd, *c.args, c.table, cu, length, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attend(qd, *c.args, c.table, cu, length, **kw)
    want, tol = ref.attend(q, cache, [0, 1, 2], lens)
    for _ in range(20):
        cu.copy_(none)
        out.fill_(5.0)
        graph.replay()
        cu.copy_(both)
        torch.cuda.synchronize()
        assert (out == 5).all()
        graph.replay()
        cu.copy_(none)
        torch.cuda.synchronize()
        check(out, want, tol)


@pytest.mark.parametrize("d,hq,hkv,page", [(64, 4, 2, 16), (128, 8, 1, 48), (256, 4, 2, 32)])
@pytest.mark.parametrize("m", [1, 5, 200])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 0), (40, 5), (129, 20)])
def test_pages_that_the_window_has_left(attn, window, sinks, m, d, hq, hkv, page):
    """Pages that no query sees any more are given away: their entries are outside the pool, or the pages hold anything.  That
    is no error and changes nothing, although tiles that are read begin inside or before them."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    lens = [m + 700, m + 333]
    new = [m, m]
    cache = ref.make_cache(lens, hkv, d, page, F8, 9)
    clean = ref.Cache(*[x.clone() for x in (cache.table, *cache.args)])
    gone = []
    for n, length in enumerate(lens):
        for j in range(-(-length // page)):
            if j * page >= sinks and (j + 1) * page - 1 <= length - m - window:
                gone.append(int(cache.table[n, j]))
                cache.table[n, j] = -1
    assert len(gone) > 5
    for pages, scales in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        pages.view(torch.uint8)[gone] = 0x7F
        scales[gone] = math.nan
    q = torch.randn(2 * m, hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for table in (cache.table, clean.table):
        out, cu = run(attn, q, ref.Cache(table, *cache.args), new, lens, window=window, sinks=sinks)
        assert gdn.device_error() == 0
        check(out, *ref.attend(q, clean, cu, lens, window, sinks))
