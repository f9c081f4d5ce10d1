"""gdn_attend where a row's running reference has to move, where sequences are described wrongly, and on a stream of the
caller's with memory of its own."""
import pytest
import torch

import attn_helpers as ref
from test_gpu_attend import F8, I8, check, i32, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


@pytest.mark.parametrize("order", ["rising", "falling", "jumps"])
@pytest.mark.parametrize("m", [1, 130])
@pytest.mark.parametrize("d,dtype", [(64, I8), (128, F8), (256, I8)])
def test_scores_that_outgrow_the_reference(attn, d, dtype, m, order):
    """Scores whose size changes over the cache by many powers of two, so that a row's largest weight lies in its first, its
    last or any unit."""
    lens = [m + 570]
    cache = ref.make_cache(lens, 2, d, 32, dtype, 40)
    unit = torch.arange(cache.table.shape[1]) // 2          # pages of 32 tokens
    by = {"rising": 1.0 + 4.0 * unit, "falling": 1.0 + 4.0 * unit.flip(0), "jumps": 1.0 + 40.0 * (unit % 3 == 1)}[order]
    for p, f in zip(cache.table[0].tolist(), by.tolist()):
        cache.k_scales[p] *= f
    q = (2 * torch.randn(m, 4, d, generator=torch.Generator().manual_seed(3))).to(torch.bfloat16)
    out, cu = run(attn, q, cache, [m], lens)
    check(out, *ref.attend(q, cache, cu, lens))


@pytest.mark.parametrize("m", [20, 300])
def test_sequences_out_of_order_are_recorded(attn, m):
    """cu_seqlens that goes back: more rows than tokens, which the call's workspace has no room for."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    lens = [m] * 5
    cache = ref.make_cache(lens, 2, 64, 16, I8, 1).on("cuda")
    q = torch.randn(m, 4, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    attn.attend(q, *cache.args, cache.table, i32([0, m, 0, m, 0, m]), i32(lens), max_q_len=m, max_kv_len=m)
    torch.cuda.synchronize()
    assert gdn.device_error() == 6
    out = attn.attend(q, *cache.args, cache.table[:1], i32([0, m]), i32(lens[:1]), max_q_len=m, max_kv_len=m)
    torch.cuda.synchronize()
    assert gdn.device_error() == 0 and torch.isfinite(out.float()).all()


def test_stream_argument(attn):
    """Outputs and workspace of a call on a given stream come from that stream's memory: what the current stream frees and
    takes meanwhile does not reach them."""
    from gated_deltanet_linear_03_gb300 import norm
    m, lens = 300, [300]
    cache = ref.make_cache(lens, 2, 128, 16, I8, 5)
    c = cache.on("cuda")
    q = torch.randn(m, 8, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    args = (q.cuda(), *c.args, c.table, i32([0, m]), i32(lens))
    x = torch.randn(64, 256, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    w = torch.ones(256, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append((attn.attend(*args, max_q_len=m, max_kv_len=m, out_dtype=torch.float32, stream=stream),
                     *norm.block_norm(x, x, w, stream=stream)))
        junk = [torch.full((1 << 20,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        del junk
    torch.cuda.synchronize()
    check(outs[0][0], *ref.attend(q, cache, [0, m], lens))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("window", [0, 20])
def test_more_sequences_than_a_planning_pass(attn, window):
    """1100 short prompts: the items are listed 1024 sequences at a time, and most runs hold several items."""
    lens = [33 + n % 29 for n in range(1100)]
    new = [33 if n % 7 else 0 for n in range(1100)]
    cache = ref.make_cache(lens, 1, 64, 32, I8, 6)
    q = torch.randn(sum(new), 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, new, lens, window=window)
    check(out, *ref.attend(q, cache, cu, lens, window))


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 1), (128, 4, 2), (256, 4, 1)])
def test_negative_scale_of_prompts(attn, d, hq, hkv):
    lens = [400]
    cache = ref.make_cache(lens, hkv, d, 16, F8, 7)
    q = torch.randn(150, hq, d, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    out, cu = run(attn, q, cache, [150], lens, sm_scale=-0.07)
    check(out, *ref.attend(q, cache, cu, lens, sm_scale=-0.07))
