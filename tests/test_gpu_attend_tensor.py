"""gdn_attend's tensor-core kernel where only the other kernel was tested: bf16 outputs, memory around its outputs and its
workspace, pools and queries beyond 2^32 bytes."""
import pytest
import torch

import attn_helpers as ref
from test_gpu_attend import F8, I8, check, i32, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


def takes_tensor_kernel(attn, n, hq, hkv, d, max_q):
    """The workspace of that kernel lists items, so it grows with the tokens of a call; the other's does not.  Asked for one
    cached token: more tokens never bring a call back to the other kernel."""
    size = lambda T: attn.attend_workspace_size(n, T, hq, hkv, d, max_q, 1)  # noqa: E731
    return size(max_q + 100000) > size(max_q)


ROWS = {64: 300, 128: 130, 256: 270}            # query rows of a key/value head that take it at any length


@pytest.mark.parametrize("d", [64, 128, 256])
def test_which_kernel(attn, d):
    assert takes_tensor_kernel(attn, 1, 2, 1, d, ROWS[d] // 2)
    assert not takes_tensor_kernel(attn, 1, 2, 1, d, 8)


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (64, 3, 1), (128, 8, 4), (128, 5, 1), (256, 4, 2), (256, 7, 1)])
def test_bf16_output(attn, d, hq, hkv, window, dtype):
    """Whole items leave through another store than parts and fp32 rows."""
    assert takes_tensor_kernel(attn, 3, hq, hkv, d, 300)
    new, lens = [300, 41, 300], [300, 90, 1000]
    cache = ref.make_cache(lens, hkv, d, 48, dtype, d + hq)
    q = torch.randn(sum(new), hq, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, new, lens, window=window, out_dtype=torch.bfloat16)
    check(out, *ref.attend(q, cache, cu, lens, window))


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_outputs_and_workspace_stay_inside(attn, d, out_dtype):
    m, hq, hkv = 301, 4, 2
    assert takes_tensor_kernel(attn, 1, hq, hkv, d, m)
    lens = [m + 77]
    cache = ref.make_cache(lens, hkv, d, 32, I8, 2)
    q = torch.randn(m, hq, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    edge, size = 1 << 14, m * hq * d * out_dtype.itemsize
    guard = torch.full((2 * edge + size,), 7, dtype=torch.uint8, device="cuda")
    need = attn.attend_workspace_size(1, m, hq, hkv, d, m, lens[0])
    work = torch.full((2 * edge + need,), 0xA5, dtype=torch.uint8, device="cuda")
    out, cu = run(attn, q, cache, [m], lens, out=guard[edge:edge + size].view(out_dtype).view(m, hq, d),
                  workspace=work[edge:edge + need])
    check(out, *ref.attend(q, cache, cu, lens))
    assert (guard[:edge] == 7).all() and (guard[edge + size:] == 7).all()
    assert (work[:edge] == 0xA5).all() and (work[edge + need:] == 0xA5).all()


def test_pool_past_32_bits(attn):
    """A pool of more than 2^32 bytes whose last pages are used; rows of one page alone would not reach that far."""
    hkv, d, page, hq, m = 1, 256, 64, 4, 80
    assert takes_tensor_kernel(attn, 1, hq, hkv, d, m)
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
    q = torch.randn(m, hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out = attn.attend(q.cuda(), k, v, ks, vs, ids.to(torch.int32)[None].contiguous(), i32([0, m]), i32([150]), max_q_len=m,
                      max_kv_len=150, out_dtype=torch.float32)
    check(out, *ref.attend(q, small, [0, m], [150]))


def test_queries_past_32_bits(attn):
    """More than 2^32 bytes of queries and outputs: the last rows are those of a call with the last tokens alone.  Both round
    weights (2^-11) and outputs (2^-8) once, in sums of at most 64 tokens that may be cut at other places."""
    T, hq, hkv, d, page, window, last = 540000, 16, 2, 256, 64, 64, 500
    assert T * hq * d * 2 > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(1)
    n_pages = -(-T // page)
    k, v = (torch.randint(-127, 128, (n_pages, hkv, page, d), dtype=I8, device="cuda", generator=gen) for _ in range(2))
    ks, vs = (torch.full((n_pages, hkv, page // 16), 0.01, device="cuda") for _ in range(2))
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(T, hq, d, device="cuda", generator=gen, dtype=torch.bfloat16)
    kw = dict(max_kv_len=T, window=window)
    a = attn.attend(q, k, v, ks, vs, table, i32([0, T]), i32([T]), max_q_len=T, **kw)
    b = attn.attend(q[-last:].contiguous(), k, v, ks, vs, table, i32([0, last]), i32([T]), max_q_len=last, **kw)
    x, y = a[-last:].float(), b.float()
    assert torch.isfinite(x).all() and x.abs().max() > 0.1
    assert ((x - y).abs() <= 2.0 ** -7 * y.abs() + 2 * 1.27 * 2.0 ** -10).all()
