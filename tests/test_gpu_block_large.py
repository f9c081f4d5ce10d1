"""gdn_kv_append, gdn_kv_read and gdn_block_norm on memory beyond 2^32 bytes, and captured in graphs."""
import pytest
import torch

import attn_helpers as ref
from test_gpu_kv_cache import F8, I8, Run, check_rotated, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


@pytest.fixture(scope="module")
def norm():
    from gated_deltanet_linear_03_gb300 import norm as n
    return n


@pytest.mark.parametrize("dtype", [I8, F8])
def test_pool_past_32_bits(attn, dtype):
    """The same tokens in the last pages of a large pool and in a small one."""
    hkv, d, page, T = 1, 256, 64, 150
    n_pages = (1 << 32) // (page * d) + 64
    ids = [n_pages - 1, n_pages - 30, n_pages - 5]
    small = Run(attn, [T], 2, hkv, d, 64, page, dtype, seed=1)
    q, k, v = small.inputs([T])
    want, _ = small.append([T], q, k, v)
    *pool, opened = attn.alloc_cache(n_pages, hkv, page, d, 1, dtype)
    table = i32([ids])
    got, opened = attn.kv_append(k.cuda(), v.cuda(), small.cos.cuda(), small.sin.cuda(), i32([0, T]), i32([0]), table, *pool, opened,
                                 q=q.cuda())
    assert torch.equal(got, want) and torch.equal(opened, small.open)
    for at, p in enumerate(ids):
        for x, y in zip(pool, small.pool):
            assert torch.equal(x[p].view(torch.uint8), y[small.table[0, at]].view(torch.uint8))
    a, b = attn.kv_read(*pool, table, i32([0, T]), T), small.read()[:2]
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_queries_past_32_bits(attn):
    """The last tokens' queries are those of a call with these tokens alone."""
    T, hq, d, page, last = 540000, 16, 256, 4096, 40
    assert T * hq * d * 2 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(T, hq, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    k = torch.randn(T, 1, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    ang = torch.arange(T, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    cos, sin = ang.cos().float(), ang.sin().float()
    *pool, opened = attn.alloc_cache(-(-T // page), 1, page, d, 1)
    table = torch.arange(-(-T // page), dtype=torch.int32, device="cuda")[None]
    a, _ = attn.kv_append(k, k, cos, sin, i32([0, T]), i32([0]), table, *pool, opened, q=q)
    part = slice(T - last, T)
    b, _ = attn.kv_append(k[part], k[part], cos, sin, i32([0, last]), i32([T - last]), table, *pool, opened, q=q[part])
    assert torch.equal(a[part], b)
    run = type("Tables", (), dict(cos=cos.cpu(), sin=sin.cpu(), rot=64, interleaved=False))
    check_rotated(b, q[part].cpu(), torch.arange(T - last, T), run)


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_norm_past_32_bits(norm, residual):
    rows, dim, last = 270001, 8192, 7
    assert rows * dim * 2 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, dim, device="cuda", generator=gen, dtype=torch.bfloat16)
    r = torch.randn(rows, dim, device="cuda", generator=gen, dtype=residual)
    w = 1 + 0.2 * torch.randn(dim, device="cuda", generator=gen)
    kw = dict(post_weight=w, scale=0.5)
    want = norm.block_norm(x[-last:].clone(), r[-last:].clone(), w, gate=x[-last:].clone(), **kw)
    got = norm.block_norm(x, r, w, gate=x, residual_out=r, out=x, **kw)
    assert all(torch.equal(a[-last:], b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [I8, F8])
def test_a_layer_in_a_graph(attn, norm, dtype):
    """One token of three sequences through norm, append and attention, captured once and replayed as the lengths grow; the
    same calls without a graph give the same, bit for bit."""
    n, hq, hkv, d, page, steps, dim = 3, 8, 2, 64, 16, 40, 512
    graphed = Run(attn, [60] * n, hq, hkv, d, 32, page, dtype, seed=2)
    eager = Run(attn, [60] * n, hq, hkv, d, 32, page, dtype, seed=2)
    start = [1, 9, 17]
    q, k, v = graphed.inputs(start)
    for r in (graphed, eager):
        r.append(start, q, k, v)
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = 1 + 0.2 * torch.randn(dim, device="cuda", generator=gen)
    cos, sin, cu = graphed.cos.cuda(), graphed.sin.cuda(), i32(list(range(n + 1)))
    x, res = (torch.zeros(n, dim, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.zeros(n, hkv, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))

    def layer(r, past, lens):
        res2, h = norm.block_norm(x, res, w, post_weight=w, gate=x)
        q, _ = attn.kv_append(k, v, cos, sin, cu, past, r.table, *r.pool, r.open, q=h.view(n, hq, d))
        y = attn.attend(q, *r.pool, r.table, cu, lens, max_q_len=1, max_kv_len=60)
        return (*norm.block_norm(y.view(n, dim), res2, w, scale=w), y)

    past, lens = i32(start), i32([s + 1 for s in start])
    saved = [t.clone() for t in (*graphed.pool, graphed.open)]
    layer(graphed, past, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(graphed, past, lens)
    for t, s in zip((*graphed.pool, graphed.open), saved):
        t.copy_(s)
    for _ in range(steps):
        for t in (x, res, k, v):
            t.normal_(generator=gen)
        graph.replay()
        want = layer(eager, past.clone(), lens.clone())
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        past += 1
        lens += 1
    for a, b in zip((*graphed.pool, graphed.open), (*eager.pool, eager.open)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
