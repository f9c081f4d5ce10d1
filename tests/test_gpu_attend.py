"""gdn_attend against the plain 64-bit form: types, head layouts, lengths, pages that end inside a tile, masks that
leave rows empty, splits over the cache, bounds, and values at the edges of the number formats."""
import math

import pytest
import torch

import attn_helpers as ref

pytestmark = pytest.mark.gpu
I8, F8 = torch.int8, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(attn, q, cache, new, lens, *, max_q=None, max_kv=None, **kw):
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    c = cache.on("cuda")
    out = attn.attend(q.cuda(), *c.args, c.table, i32(cu), i32(lens), max_q_len=max_q or max(max(new), 1),
                      max_kv_len=max(lens) if max_kv is None else max_kv, out_dtype=kw.pop("out_dtype", torch.float32), **kw)
    torch.cuda.synchronize()
    return out, cu


def check(out, want, tol):
    err = (out.double().cpu() - want).abs()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()          # half an ulp at the bottom of a binade
    assert torch.isfinite(out.float()).all()
    worst = (err / tol).max().item()
    assert worst <= 1, f"{worst:.3g} of the bound"


def case(attn, new, lens, hq, hkv, d, page, dtype, seed=0, window=0, sinks=0, out_dtype=torch.float32, sm_scale=None, q_std=1.0, **kw):
    cache = ref.make_cache(lens, hkv, d, page, dtype, seed)
    q = (q_std * torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(seed + 1))).to(torch.bfloat16)
    out, cu = run(attn, q, cache, new, lens, window=window, sinks=sinks, out_dtype=out_dtype, sm_scale=sm_scale, **kw)
    want, tol = ref.attend(q, cache, cu, lens, window, sinks, sm_scale)
    check(out, want, tol)
    return out


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("hq,hkv,d,page", [(16, 2, 256, 64), (32, 8, 128, 32), (8, 1, 64, 16), (5, 1, 128, 48), (4, 4, 64, 128), (17, 1, 256, 16)])
def test_single_tokens(attn, hq, hkv, d, page, dtype):
    """One query a sequence, caches from one token to several tiles."""
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 300]
    case(attn, [1] * len(lens), lens, hq, hkv, d, page, dtype, seed=d + page)


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_bf16_output(attn, d, dtype):
    case(attn, [1, 3], [40, 200], 4, 2, d, 32, dtype, seed=d, out_dtype=torch.bfloat16)


@pytest.mark.parametrize("new,lens", [([5], [5]), ([7, 1, 0, 3], [130, 64, 9, 3]), ([2, 2], [2, 500]), ([33], [33]), ([17, 40], [80, 40])])
@pytest.mark.parametrize("hq,hkv,d", [(16, 2, 256), (6, 2, 128), (3, 1, 64)])
def test_several_queries(attn, new, lens, hq, hkv, d):
    case(attn, new, lens, hq, hkv, d, 32, I8, seed=len(new) + d)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (63, 4), (64, 17), (100, 0), (128, 70), (1000, 3), (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [1, 200, 517]), ([9, 70], [300, 400])])
def test_window_and_sinks(attn, window, sinks, new, lens):
    case(attn, new, lens, 8, 2, 128, 48, I8, seed=window % 1000 + sinks, window=window, sinks=sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new,lens", [([300], [300]), ([257, 1, 64], [257, 900, 700]), ([130], [1000])])
def test_prompts(attn, new, lens, d):
    case(attn, new, lens, 4, 2, d, 64, I8, seed=d)


@pytest.mark.parametrize("window,sinks", [(50, 0), (130, 3), (64, 64), (200, 100)])
def test_prompts_with_window(attn, window, sinks):
    case(attn, [300, 90], [300, 500], 8, 1, 64, 16, F8, seed=window, window=window, sinks=sinks)
    case(attn, [300], [700], 6, 3, 256, 48, I8, seed=window, window=window, sinks=sinks)


@pytest.mark.parametrize("m", [2, 40, 200])
def test_rows_that_see_nothing_are_zero(attn, m):
    """Queries at negative positions (more queries than cached tokens), and an empty cache."""
    cache = ref.make_cache([3, 0, 20], 2, 64, 16, I8, 5)
    new, lens = [m, m, 1], [1, 0, 20]
    q = torch.randn(sum(new), 4, 64, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, new, lens)
    want = torch.zeros(sum(new), 4, 64, dtype=torch.float64)
    tol = torch.full_like(want, 1e-30)
    for n, (i, L) in enumerate(zip(new, lens)):
        last = slice(cu[n + 1] - min(i, L), cu[n + 1])
        if L:
            o, t = ref.attend(q[last], ref.Cache(cache.table[n:n + 1], *cache.args), [0, min(i, L)], [L])
            want[last], tol[last] = o, t
    check(out, want, tol)
    assert (out[:m - 1] == 0).all() and (out[m:2 * m] == 0).all()


def test_nothing_to_do(attn):
    cache = ref.make_cache([10], 1, 64, 16, I8, 1)
    q = torch.empty(0, 2, 64, dtype=torch.bfloat16)
    out, _ = run(attn, q, cache, [0], [10])
    assert out.shape == (0, 2, 64)


@pytest.mark.parametrize("new", [[1], [150]])
def test_long_cache_is_split_and_joined(attn, new):
    """Thousands of tokens behind few rows: many CTAs carry one item; a second call must not see the first's parts."""
    a = case(attn, new, [5003], 4, 1, 128, 64, I8, seed=3)
    case(attn, [1, 1], [5, 700], 4, 1, 128, 64, I8, seed=4)
    assert torch.equal(a, case(attn, new, [5003], 4, 1, 128, 64, I8, seed=3))     # no order of atomics in the result


def test_many_sequences(attn):
    """More items than CTAs, lengths and empty sequences mixed."""
    lens = [(37 * i * i) % 211 for i in range(700)]
    new = [0 if i % 11 == 3 else 1 + i % 2 for i in range(700)]
    lens = [max(x, m) for x, m in zip(lens, new)]
    case(attn, new, lens, 2, 1, 64, 16, I8, seed=8)


def test_generous_bounds_and_workspace(attn):
    """Bounds far above the lengths (as a captured graph uses them) give the same rows."""
    lens = [100, 3, 260]
    cache = ref.make_cache(lens, 2, 128, 32, I8, 9)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    wide = ref.Cache(torch.nn.functional.pad(cache.table, (0, 200), value=-7), *cache.args)
    a, cu = run(attn, q, wide, [1, 1, 1], lens, max_kv=6000, max_q=3)
    want, tol = ref.attend(q, cache, cu, lens)
    check(a, want, tol)
    need = attn.attend_workspace_size(3, 3, 8, 2, 128, 1, 260)
    guard = torch.full((need + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    b, _ = run(attn, q, cache, [1, 1, 1], lens, workspace=guard[256:256 + need])
    check(b, want, tol)
    assert (guard[:256] == 0xA5).all() and (guard[256 + need:] == 0xA5).all()


@pytest.mark.parametrize("m", [1, 100])
def test_outputs_stay_inside(attn, m):
    lens = [m + 77]
    cache = ref.make_cache(lens, 2, 128, 32, I8, 2)
    q = torch.randn(m, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    guard = torch.full(((1 << 15) + m * 4 * 128 * 4,), 7, dtype=torch.uint8, device="cuda")
    inner = guard[1 << 14:(1 << 14) + m * 4 * 128 * 4].view(torch.float32).view(m, 4, 128)
    out, cu = run(attn, q, cache, [m], lens, out=inner)
    check(out, *ref.attend(q, cache, cu, lens))
    assert (guard[:1 << 14] == 7).all() and (guard[(1 << 14) + m * 4 * 128 * 4:] == 7).all()


@pytest.mark.parametrize("m", [1, 130])
@pytest.mark.parametrize("scale_by", [2.0 ** -40, 2.0 ** 40])
def test_magnitudes(attn, scale_by, m):
    """Values and queries far from 1: the weights stay in range whatever the scales are."""
    lens = [m + 100]
    cache = ref.make_cache(lens, 1, 64, 16, I8, 4, spread=3.0)
    cache.v_scales *= scale_by
    q = (torch.randn(m, 2, 64, generator=torch.Generator().manual_seed(2)) / scale_by).to(torch.bfloat16)
    sm = 0.1 * scale_by
    out, cu = run(attn, q, cache, [m], lens, sm_scale=sm)
    want, tol = ref.attend(q, cache, cu, lens, sm_scale=sm)
    check(out, want, tol)


@pytest.mark.parametrize("m", [1, 130])
def test_zero_blocks_and_queries(attn, m):
    """Blocks of zeros (their scales 2^-60 / 127) among others, a zero query: uniform weights."""
    from gated_deltanet_linear_03_gb300.attn import KV_BLOCK
    lens = [m + 90]
    cache = ref.make_cache(lens, 1, 128, 16, I8, 11)
    for j in (0, 2, 5):
        p = int(cache.table[0, j])
        cache.v_pages[p] = 0
        cache.v_scales[p] = 2.0 ** -60 / 127
        cache.k_pages[p, :, KV_BLOCK // 2:] = 0
    q = torch.randn(m, 3, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q[0, 1] = 0
    out, cu = run(attn, q, cache, [m], lens)
    check(out, *ref.attend(q, cache, cu, lens))


@pytest.mark.parametrize("m", [1, 140])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_nonfinite_scales_reach_only_who_sees_them(attn, bad, m):
    """A block that reads as NaN (its scale not finite) poisons the rows that see it and no others; behind the mask
    (past the window, or after the query) it is not noticed."""
    lens = [m + 200]
    cache = ref.make_cache(lens, 1, 64, 16, I8, 12)
    clean = ref.Cache(*[x.clone() for x in (cache.table, *cache.args)])
    hit = (m + 200 - 20) // 16 if m > 1 else 3
    page = int(cache.table[0, hit])
    cache.k_pages[page] = 0
    cache.v_pages[page] = 0
    cache.k_scales[page] = bad
    cache.v_scales[page] = bad
    q = torch.randn(m, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    cu = [0, m]
    window = 64
    c = cache.on("cuda")
    out = attn.attend(q.cuda(), *c.args, c.table, i32(cu), i32(lens), max_q_len=m, max_kv_len=lens[0], window=window,
                      out_dtype=torch.float32).cpu()
    pos = lens[0] - m + torch.arange(m)
    sees = (pos >= hit * 16) & (pos - window < hit * 16 + 15)
    want, tol = ref.attend(q, clean, cu, lens, window)
    assert out[sees].isnan().all()
    check(out[~sees], want[~sees], tol[~sees])


@pytest.mark.parametrize("m", [1, 70])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_nonfinite_scales_behind_the_mask_of_a_loaded_tile(attn, bad, m):
    """The spoilt blocks share a 64-token tile with visible ones: before the window, and after the last token of the page."""
    lens = [m + 194]
    cache = ref.make_cache(lens, 1, 128, 64, I8, 13)
    clean = ref.Cache(*[x.clone() for x in (cache.table, *cache.args)])
    first = lens[0] - m - 31                       # the first token that the first query sees
    assert first // 16 % 4 != 0
    for j in (first // 16 - 1, -(-lens[0] // 16)):
        page = int(cache.table[0, j * 16 // 64])
        cache.k_scales[page, :, j % 4] = bad
        cache.v_scales[page, :, j % 4] = bad
    q = torch.randn(m, 2, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, [m], lens, window=32)
    check(out, *ref.attend(q, clean, cu, lens, 32))


def test_bad_pages_and_lengths_are_recorded(attn):
    """Table entries outside the pool read as zeros and record GDN_ERR_INTERNAL; so do lengths beyond the bounds."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    lens = [40]
    cache = ref.make_cache(lens, 1, 64, 16, I8, 1)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    for bad in (-1, cache.k_pages.shape[0], 2 ** 31 - 1):
        table = cache.table.clone()
        table[0, 1] = bad
        out, _ = run(attn, q, ref.Cache(table, *cache.args), [1], lens)
        assert torch.isfinite(out).all()
        assert gdn.device_error() == 6
    run(attn, q, cache, [1], lens, max_kv=39)
    assert gdn.device_error() == 6
    run(attn, q, cache, [1], lens)
    assert gdn.device_error() == 0


def test_graph_follows_lengths(attn):
    """A captured call replayed as the cache grows."""
    lens = [500]
    cache = ref.make_cache(lens, 2, 128, 32, I8, 21)
    c = cache.on("cuda")
    q = torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    qd, cu, length = q.cuda(), i32([0, 1]), i32([1])
    out = torch.empty(1, 4, 128, device="cuda")
    ws = torch.empty(attn.attend_workspace_size(1, 1, 4, 2, 128, 1, 500), dtype=torch.uint8, device="cuda")
    kw = dict(max_q_len=1, max_kv_len=500, out=out, workspace=ws)
    attn.attend(qd, *c.args, c.table, cu, length, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.attend(qd, *c.args, c.table, cu, length, **kw)
    for L in (1, 64, 65, 333, 500):
        length.fill_(L)
        graph.replay()
        torch.cuda.synchronize()
        check(out, *ref.attend(q, cache, [0, 1], [L]))


def test_other_stream(attn):
    lens = [90]
    cache = ref.make_cache(lens, 1, 64, 16, I8, 1)
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    stream = torch.cuda.Stream()
    c = cache.on("cuda")
    args = (q.cuda(), *c.args, c.table, i32([0, 1]), i32(lens))
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        a = attn.attend(*args, max_q_len=1, max_kv_len=90, out_dtype=torch.float32)
    b = attn.attend(*args, max_q_len=1, max_kv_len=90, out_dtype=torch.float32, stream=None)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    check(a, *ref.attend(q, cache, [0, 1], lens))


def test_offsets_past_32_bits(attn):
    """A pool of more than 2^32 bytes whose last pages are used."""
    hkv, d, page = 1, 256, 64
    n_pages = (1 << 32) // (page * d) + 64
    k = torch.zeros(n_pages, hkv, page, d, dtype=I8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.ones(n_pages, hkv, page // 16, device="cuda")
    vs = torch.ones_like(ks)
    small = ref.make_cache([150], hkv, d, page, I8, 3)
    ids = torch.tensor([n_pages - 1, n_pages - 30, n_pages - 5], device="cuda")
    for j in range(3):
        p = int(small.table[0, j])
        k[ids[j]], v[ids[j]] = small.k_pages[p].cuda(), small.v_pages[p].cuda()
        ks[ids[j]], vs[ids[j]] = small.k_scales[p].cuda(), small.v_scales[p].cuda()
    for m in (1, 60):
        q = torch.randn(m, 4, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
        out = attn.attend(q.cuda(), k, v, ks, vs, ids.to(torch.int32)[None].contiguous(), i32([0, m]), i32([150]), max_q_len=m,
                          max_kv_len=150, out_dtype=torch.float32)
        check(out, *ref.attend(q, small, [0, m], [150]))


def test_refusals(attn):
    from gated_deltanet_linear_03_gb300.gdn import GdnError
    cache = ref.make_cache([40], 2, 64, 16, I8, 1).on("cuda")
    q = torch.randn(1, 4, 64, device="cuda").to(torch.bfloat16)
    good = dict(max_q_len=1, max_kv_len=40)
    call = lambda q=q, c=cache.args, t=cache.table, cu=i32([0, 1]), n=i32([40]), **kw: attn.attend(q, *c, t, cu, n, **{**good, **kw})  # noqa: E731
    call()
    with pytest.raises(ValueError):
        call(q=q.float())
    with pytest.raises(ValueError):
        call(q=q.cpu())
    with pytest.raises(ValueError):
        call(t=cache.table.long())
    with pytest.raises(ValueError):
        call(n=i32([40, 40]))
    with pytest.raises(ValueError):
        call(c=(cache.k_pages, cache.v_pages[:, :1], cache.k_scales, cache.v_scales))
    with pytest.raises(ValueError):
        call(c=(cache.k_pages.float(), *cache.args[1:]))
    with pytest.raises(GdnError):
        call(q=q[:, :3].contiguous())                     # heads do not divide
    with pytest.raises(GdnError):
        call(max_kv_len=10 ** 6)                          # more than the table can name
    with pytest.raises(GdnError):
        call(window=-1)
    with pytest.raises(GdnError):
        call(sm_scale=math.nan)
    with pytest.raises(GdnError):
        call(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(GdnError):
        call(out=q)                                       # overlaps an input


@pytest.mark.parametrize("m", [1, 40, 130])
def test_garbage_past_the_end_is_not_read(attn, m):
    """NaN codes in the rows after a sequence's last token, NaN scales after its last block, NaN pages around it."""
    lens = [m + 45]
    cache = ref.make_cache(lens, 2, 128, 32, F8, 14)
    clean = ref.Cache(*[x.clone() for x in (cache.table, *cache.args)])
    used = cache.table[0, :-(-lens[0] // 32)].tolist()
    for pages, scales in ((cache.k_pages, cache.k_scales), (cache.v_pages, cache.v_scales)):
        raw = pages.view(torch.uint8)
        for page in range(pages.shape[0]):
            if page not in used:
                raw[page] = 0x7F
                scales[page] = math.nan
        raw[used[-1], :, lens[0] % 32:] = 0xFF
        scales[used[-1], :, -(-(lens[0] % 32) // 16):] = math.nan
    q = torch.randn(m, 4, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, [m], lens)
    check(out, *ref.attend(q, clean, cu, lens))


@pytest.mark.parametrize("d,hq,hkv", [(256, 6, 3), (128, 8, 2), (64, 8, 1)])
def test_repeated_calls_agree(attn, d, hq, hkv):
    """Short runs (a unit or two a CTA) many times over: nothing is read before the product that writes it has finished."""
    cache = ref.make_cache([700], hkv, d, 48, I8, 30)
    q = torch.randn(300, hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    first = None
    for _ in range(40):
        out, cu = run(attn, q, cache, [300], [700], window=200, sinks=100)
        if first is None:
            first = out
            check(out, *ref.attend(q, cache, cu, [700], 200, 100))
        assert torch.equal(out, first)
