"""gdn_kv_append: a sequence that cannot be stored is left out as a whole, its queries and open block too."""
import pytest
import torch

from test_gpu_kv_cache import F8, I8, Run, check_rotated, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


@pytest.mark.parametrize("why", ["tables", "table", "negative", "overflow", "slot", "slot above"])
@pytest.mark.parametrize("rot", [0, 32])
@pytest.mark.parametrize("d,dtype,in_place", [(64, I8, False), (256, F8, True)])
def test_left_out_as_a_whole(attn, d, dtype, in_place, rot, why):
    """The second of three sequences does not fit; part of its tokens would, taken alone."""
    from gated_deltanet_linear_03_gb300 import gdn
    if why == "tables" and rot == 0:
        pytest.skip("no tables without a rotation")
    assert gdn.device_error() == 0
    new, at = [20, 21, 18], slice(20, 41)
    run = Run(attn, [40, 40, 40], 4, 2, d, rot, 16, dtype, seed=1)
    good = Run(attn, [40, 40, 40], 4, 2, d, rot, 16, dtype, seed=1)
    q, k, v = run.inputs(new)
    want, pos = good.append(new, q, k, v)
    check_rotated(want, q, pos, good)
    past, slots, cos, sin, table = [0, 0, 0], [0, 1, 2], run.cos.cuda(), run.sin.cuda(), run.table
    if why == "tables":
        cos, sin = cos[:20].contiguous(), sin[:20].contiguous()
    elif why == "table":
        table, new[0] = table[:, :1].contiguous(), 16
    elif why == "negative":
        past[1] = -5
    elif why == "overflow":
        past[1] = 2 ** 31 - 10
    else:
        slots[1] = -1 if why == "slot" else 3
    if why == "table":
        new[2] = 16
        q, k, v = (torch.cat([x[:16], x[20:41], x[41:57]]) for x in (q, k, v))
        at = slice(16, 37)
    cu = [0, new[0], new[0] + new[1], sum(new)]
    qd = q.cuda()
    out = qd if in_place else torch.full_like(qd, 9.0)
    before = out[at].clone()
    opened = torch.full_like(run.open, -3.0)
    pages = [x.clone() for x in run.pool]
    attn.kv_append(k.cuda(), v.cuda(), cos if rot else None, sin if rot else None, i32(cu), i32(past), table, *run.pool, run.open,
                   open_out=opened, q=qd, q_out=out, slots=i32(slots))
    torch.cuda.synchronize()
    assert gdn.device_error() == 6
    assert torch.equal(out[at], before)
    assert (opened[1] == -3).all()
    for p in run.table[1].tolist():
        if p >= 0:
            assert all(torch.equal(x[p].view(torch.uint8), y[p].view(torch.uint8)) for x, y in zip(run.pool, pages))
    # the others are as they should be
    first, last = slice(0, new[0]), slice(cu[2], cu[3])
    assert torch.equal(out[first], want[:new[0]])
    assert torch.equal(out[last], want[41:41 + new[2]])
    got = attn.kv_read(*run.pool, run.table, i32([0, 16, 16, 32]), 32)
    ref = attn.kv_read(*good.pool, good.table, i32([0, 16, 16, 32]), 32)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_tokens_of_no_sequence(attn):
    """Rows behind the last sequence's (a batch padded to a fixed size) are neither stored nor rotated, and no error."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    run = Run(attn, [40, 40], 4, 2, 128, 64, 16, I8, seed=1)
    q, k, v = (x.cuda() for x in run.inputs([20, 30]))
    out = torch.full_like(q, 9.0)
    attn.kv_append(k, v, run.cos.cuda(), run.sin.cuda(), i32([0, 20, 33]), i32([0, 0]), run.table, *run.pool, run.open, q=q, q_out=out)
    torch.cuda.synchronize()
    assert gdn.device_error() == 0
    pos = torch.cat([torch.arange(20), torch.arange(13)])
    check_rotated(out[:33], q[:33].cpu(), pos, run)
    assert (out[33:] == 9).all()


@pytest.mark.parametrize("pad", [0, 4, 64])
def test_one_token_of_a_wider_row(attn, pad):
    """A single token's q, k and v as slices of one row: no other token stands a stride away, so any stride is right, also for
    a query that is rotated in place."""
    hq, hkv, d = 6, 2, 128
    whole = Run(attn, [9], hq, hkv, d, 32, 16, I8, seed=3)
    part = Run(attn, [9], hq, hkv, d, 32, 16, I8, seed=3)
    q, k, v = whole.inputs([1])
    width = (hq + 2 * hkv) * d + pad
    fused = torch.zeros(2 * width, dtype=torch.bfloat16, device="cuda")
    fused[:width - pad] = torch.cat([x.flatten() for x in (q, k, v)]).cuda()
    qs, ks, vs = (fused.as_strided((1, h, d), (width, d, 1), at * d) for h, at in ((hq, 0), (hkv, hq), (hkv, hq + hkv)))
    want, _ = whole.append([1], q, k, v)
    got, _ = part.append([1], qs, ks, vs, q_out=qs)
    assert got is qs and torch.equal(got, want)
    for x, y in zip(whole.pool, part.pool):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
