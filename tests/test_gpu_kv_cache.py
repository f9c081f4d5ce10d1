"""gdn_kv_append and gdn_kv_read against plain forms: rotation, quantisation, unfinished blocks, ragged sequences."""
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


def tables(positions, rot):
    half = rot // 2
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))
    return torch.cos(ang).float(), torch.sin(ang).float()


class Run:
    """Sequences that grow in the cache, and what the cache ought to hold (bf16 rows of every sequence)."""

    def __init__(self, attn, cap, hq, hkv, d, rot, page, dtype, interleaved=False, seed=0, bad=-1):
        self.attn, self.hq, self.hkv, self.d, self.rot, self.dtype, self.interleaved = attn, hq, hkv, d, rot, dtype, interleaved
        gen = torch.Generator().manual_seed(seed)
        table, n_pages = ref.make_table(cap, page, gen, bad=bad)
        self.gen, self.page, self.table = gen, page, table.cuda()
        *self.pool, self.open = attn.alloc_cache(n_pages, hkv, page, d, len(cap), dtype)
        self.cos, self.sin = tables(max(cap), rot)
        self.lens = [0] * len(cap)
        self.rows = [[torch.zeros(0, hkv, d, dtype=torch.bfloat16) for _ in range(2)] for _ in cap]

    def inputs(self, new):
        T = sum(new)
        rand = lambda h: torch.randn(T, h, self.d, generator=self.gen).to(torch.bfloat16)  # noqa: E731
        return rand(self.hq), rand(self.hkv), rand(self.hkv)

    def append(self, new, q, k, v, **kw):
        cu = [0]
        for m in new:
            cu.append(cu[-1] + m)
        rot = dict(cos=self.cos.cuda(), sin=self.sin.cuda()) if self.rot else dict(cos=None, sin=None)
        qo, opened = self.attn.kv_append(k.cuda() if not k.is_cuda else k, v.cuda() if not v.is_cuda else v, rot["cos"], rot["sin"],
                                         i32(cu), i32(self.lens), self.table, *self.pool, self.open,
                                         q=(q.cuda() if not q.is_cuda else q) if q is not None else None,
                                         interleaved=self.interleaved, **kw)
        torch.cuda.synchronize()
        self.open = opened
        pos = torch.cat([torch.arange(p, p + m) for p, m in zip(self.lens, new)]) if sum(new) else torch.zeros(0, dtype=torch.long)
        kr = ref.rotate(k.cpu(), pos, self.cos if self.rot else None, self.sin, self.interleaved)
        for i, m in enumerate(new):
            at = slice(cu[i], cu[i + 1])
            self.rows[i][0] = torch.cat([self.rows[i][0].double(), kr[at]])
            self.rows[i][1] = torch.cat([self.rows[i][1].double(), v.cpu()[at].double()])
            self.lens[i] += m
        return qo, pos

    def read(self, **kw):
        cu = [0]
        for m in self.lens:
            cu.append(cu[-1] + m)
        k, v = self.attn.kv_read(*self.pool, self.table, i32(cu), cu[-1], **kw)
        torch.cuda.synchronize()
        return k, v, cu

    def check(self):
        """Every cached value is within its code's rounding of the bf16 row; V's codes are the definition's, bit for bit."""
        k, v, cu = self.read(out_dtype=torch.float32)
        for i, L in enumerate(self.lens):
            for j, got in enumerate((k, v)):
                x = self.rows[i][j]
                got = got[cu[i]:cu[i + 1]].cpu().double()
                pad = torch.zeros(-(-L // 16) * 16, self.hkv, self.d, dtype=torch.float64)
                pad[:L] = x
                amax = pad.view(-1, 16, self.hkv, self.d).abs().amax(dim=(1, 3)).repeat_interleave(16, 0)[:L, :, None]
                # the row's own rounding to bf16 (a rotated key in 32 bits first: 2^-22 of its pair), then the code's:
                # half a step of 1/127, or 2^-4 relative (2^-10 of a step below the smallest normal), and 32-bit scaling
                near = 2.0 ** -8 * x.abs() + 2.0 ** -21 * amax
                step = 0.5 / 127 * amax if self.dtype == I8 else 2.0 ** -4 * x.abs() + 2.0 ** -10 / 448 * amax
                bound = step * (1 + 2.0 ** -6) + near * 1.1 + 1e-30
                assert ((got - x).abs() <= bound).all(), (i, j)
                if j == 1:
                    blocks = pad.to(torch.bfloat16).view(-1, 16, self.hkv, self.d).transpose(1, 2)
                    codes, scales = ref.quantise(blocks, self.dtype)
                    want = (codes.float() * scales[..., None, None]).transpose(1, 2).reshape(-1, self.hkv, self.d)[:L]
                    assert torch.equal(got.float(), want), i


def check_rotated(qo, q, pos, run):
    want = ref.rotate(q, pos, run.cos if run.rot else None, run.sin, run.interleaved)
    big = q.double().abs().amax(-1, keepdim=True)
    # one rounding to bf16, after two products and a sum in 32 bits
    assert ((qo.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -21 * big).all()
    assert torch.equal(qo.cpu()[..., run.rot:], q[..., run.rot:])


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot,page", [(16, 2, 256, 64, 64), (32, 8, 128, 128, 32), (8, 1, 64, 16, 16), (3, 3, 128, 0, 48), (5, 1, 256, 256, 16)])
def test_growing_sequences(attn, hq, hkv, d, rot, page, interleaved, dtype):
    """Prompts, single tokens, pieces that cross blocks and pages, and sequences left alone."""
    run = Run(attn, [200, 70, 17, 40], hq, hkv, d, rot, page, dtype, interleaved, seed=d + rot)
    for new in ([37, 1, 0, 16], [1, 1, 1, 1], [0, 30, 15, 0], [100, 16, 1, 15], [1, 0, 0, 1]):
        q, k, v = run.inputs(new)
        qo, pos = run.append(new, q, k, v)
        check_rotated(qo, q, pos, run)
        run.check()


@pytest.mark.parametrize("dtype", [I8, F8])
def test_cache_does_not_depend_on_the_pieces(attn, dtype):
    """The same tokens at once, one at a time, and in odd pieces: codes, scales and open blocks agree bit for bit."""
    total, pools = 83, []
    for pieces in ([83], [1] * 83, [5, 16, 11, 32, 18, 1], [40, 43]):
        run = Run(attn, [total], 4, 2, 128, 64, 32, dtype, seed=5)
        _, k, v = run.inputs([total])
        at = 0
        for m in pieces:
            run.append([m], None, k[at:at + m], v[at:at + m])
            at += m
        k_out, v_out, _ = run.read(out_dtype=torch.float32)
        pools.append([k_out, v_out, run.open[:, :, :, :total % 16].clone(), *(s.clone() for s in run.pool[2:])])
    for other in pools[1:]:
        for a, b in zip(pools[0], other):
            assert torch.equal(a, b)


def test_open_blocks(attn):
    """open_out apart from open_in, and slots in another order: rows [0, length % 16) hold the bf16 tokens, others are untouched."""
    run = Run(attn, [100, 100, 100], 0, 2, 64, 0, 16, I8, seed=2)
    run.open = torch.full((5, 2, 2, 16, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    slots = i32([4, 0, 2])
    for new in ([3, 33, 16], [13, 0, 5], [20, 2, 1]):
        _, k, v = run.inputs(new)
        before = run.open
        run.append(new, None, k, v, open_out=torch.full_like(before, -3.0), slots=slots)
        for i, s in enumerate((4, 0, 2)):
            left = run.lens[i] % 16
            for j in range(2):
                want = run.rows[i][j][run.lens[i] - left:].to(torch.bfloat16).transpose(0, 1)
                assert torch.equal(run.open[s, j, :, :left].cpu(), want)
                assert (run.open[s, j, :, left:] == -3).all()
        assert (run.open[1] == -3).all() and (run.open[3] == -3).all()
        run.check()


def test_slices_of_one_projection(attn):
    """q, k and v as slices of [T, (hq + 2 hkv) d], and q rotated in place."""
    hq, hkv, d, T = 6, 2, 128, 45
    for dtype in (I8, F8):
        a = Run(attn, [T], hq, hkv, d, 32, 16, dtype, seed=3)
        b = Run(attn, [T], hq, hkv, d, 32, 16, dtype, seed=3)
        q, k, v = a.inputs([T])
        fused = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], dim=1).cuda()
        qs, ks, vs = (x.view(T, -1, d) for x in fused.split([hq * d, hkv * d, hkv * d], dim=1))
        assert not ks.is_contiguous()
        qa, pos = a.append([T], q, k, v)
        qb, _ = b.append([T], qs, ks, vs)
        assert torch.equal(qa, qb)
        for x, y in zip(a.pool, b.pool):
            assert torch.equal(x.view(torch.int8), y.view(torch.int8))
        own = q.cuda()
        c = Run(attn, [T], hq, hkv, d, 32, 16, dtype, seed=3)
        qc, _ = c.append([T], own, k, v, q_out=own)
        assert qc is own and torch.equal(qc, qa)


@pytest.mark.parametrize("dtype", [I8, F8])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_nonfinite_values_spoil_their_block_only(attn, bad, dtype):
    run = Run(attn, [64], 0, 2, 64, 0, 32, dtype, seed=4)
    _, k, v = run.inputs([64])
    clean = Run(attn, [64], 0, 2, 64, 0, 32, dtype, seed=4)
    clean.append([64], None, k, v)
    kb, vb = k.clone(), v.clone()
    kb[20, 1, 5] = bad
    vb[40, 0, 63] = bad
    run.append([64], None, kb, vb)
    got, want = run.read(out_dtype=torch.float32), clean.read(out_dtype=torch.float32)
    for j, (t, h) in enumerate(((20, 1), (40, 0))):
        hit = torch.zeros(64, 2, dtype=torch.bool)
        hit[t // 16 * 16:t // 16 * 16 + 16, h] = True
        assert got[j].cpu()[hit].isnan().all()
        assert torch.equal(got[j].cpu()[~hit], want[j].cpu()[~hit])


def test_small_large_and_zero_blocks(attn):
    """Blocks of zeros, of the smallest and the largest magnitudes."""
    run = Run(attn, [96], 0, 1, 64, 0, 16, I8, seed=4)
    _, k, v = run.inputs([96])
    for x in (k, v):
        x[:16] = 0
        x[16:32] *= 2.0 ** -100          # below the floor: reads as zero
        x[32:48] *= 2.0 ** -50
        x[48:64] *= 2.0 ** 120
    run.append([96], None, k, v)
    got = run.read(out_dtype=torch.float32)
    for x, y in ((k, got[0]), (v, got[1])):
        y = y.cpu().double()
        assert (y[:32] == 0).all() and torch.isfinite(y).all()
        amax = x[32:].double().view(4, 16, 64).abs().amax(dim=(1, 2)).repeat_interleave(16)[:, None]
        assert ((y[32:, 0] - x[32:, 0].double()).abs() <= 0.5001 / 127 * amax).all()


def test_positions_out_of_range_are_recorded(attn):
    """Beyond the cos/sin tables, the block table or the pool: GDN_ERR_INTERNAL, nothing written for that sequence."""
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    for what in ("tables", "table", "page", "negative"):
        run = Run(attn, [32, 32], 2, 1, 64, 16, 16, I8, seed=1)
        q, k, v = run.inputs([20, 20])
        good = Run(attn, [32, 32], 2, 1, 64, 16, 16, I8, seed=1)
        good.append([20, 20], q, k, v)
        if what == "tables":
            short = (run.cos[:25].contiguous().cuda(), run.sin[:25].contiguous().cuda())
            attn.kv_append(k.cuda(), v.cuda(), *short, i32([0, 20, 40]), i32([0, 16]), run.table, *run.pool, run.open, q=q.cuda())
        elif what == "table":
            attn.kv_append(k.cuda(), v.cuda(), run.cos.cuda(), run.sin.cuda(), i32([0, 20, 40]), i32([0, 0]),
                           run.table[:, :1].contiguous(), *run.pool, run.open)
        elif what == "page":
            run.table[1, 0] = run.pool[0].shape[0]
            attn.kv_append(k.cuda(), v.cuda(), run.cos.cuda(), run.sin.cuda(), i32([0, 20, 40]), i32([0, 0]), run.table, *run.pool, run.open)
        else:
            attn.kv_append(k.cuda(), v.cuda(), run.cos.cuda(), run.sin.cuda(), i32([0, 20, 40]), i32([0, -3]), run.table, *run.pool, run.open)
        assert gdn.device_error() == 6
        if what in ("tables", "page", "negative"):        # the other sequence is as it should be
            a = attn.kv_read(*run.pool, run.table[:1].contiguous(), i32([0, 20]), 20)
            b = attn.kv_read(*good.pool, good.table[:1].contiguous(), i32([0, 20]), 20)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert gdn.device_error() == 0


def test_writes_stay_inside(attn):
    """Pages of other sequences and the bytes around the pool keep their contents."""
    hkv, d, page = 2, 128, 16
    guard = torch.full((2 * (1 << 14) + 6 * hkv * page * d,), 0x5A, dtype=torch.uint8, device="cuda")
    pages = guard[1 << 14:(1 << 14) + 6 * hkv * page * d].view(torch.int8).view(6, hkv, page, d)
    v_pages = torch.full((6, hkv, page, d), 77, dtype=I8, device="cuda")
    ks, vs = (torch.full((6, hkv, 1), -5.0, device="cuda") for _ in range(2))
    opened = torch.zeros(1, 2, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(20, hkv, d, device="cuda").to(torch.bfloat16)
    attn.kv_append(k, k, None, None, i32([0, 20]), i32([0]), i32([[4, 1]]), pages, v_pages, ks, vs, opened)
    torch.cuda.synchronize()
    for p in (0, 2, 3, 5):
        assert (pages[p] == 0x5A).all() and (v_pages[p] == 77).all() and (ks[p] == -5).all() and (vs[p] == -5).all()
    assert (guard[:1 << 14] == 0x5A).all() and (guard[(1 << 14) + 6 * hkv * page * d:] == 0x5A).all()


def test_refusals(attn):
    from gated_deltanet_linear_03_gb300.gdn import GdnError
    *pool, opened = attn.alloc_cache(4, 2, 16, 64, 1)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cos, sin = (t.cuda() for t in tables(40, 32))
    table = i32([[0, 1]])

    def call(k=k, v=k, cos=cos, sin=sin, cu=i32([0, 3]), past=i32([0]), table=table, pool=pool, opened=opened, **kw):
        return attn.kv_append(k, v, cos, sin, cu, past, table, *pool, opened, **kw)

    call()
    for bad in (dict(k=k.float()), dict(k=k.cpu()), dict(v=k[:2]), dict(sin=None), dict(cos=cos[:, :8].contiguous()), dict(past=i32([0, 0])),
                dict(cu=i32([0, 3]).long()), dict(opened=opened.float()), dict(opened=opened[:, :1].contiguous()), dict(slots=i32([0, 1])),
                dict(q_out=k), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(pool=[pool[0][:, :, :8].contiguous(), *pool[1:]])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(GdnError):
        call(cos=cos[:, :4].contiguous(), sin=sin[:, :4].contiguous())      # rot must be a multiple of 16
    with pytest.raises(GdnError):
        call(q=torch.zeros(3, 3, 64, dtype=torch.bfloat16, device="cuda"))  # heads do not divide
    with pytest.raises(GdnError):
        call(k=torch.zeros(3, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128].view(3, 2, 64))   # token stride
    with pytest.raises(GdnError):
        call(k=opened.view(-1)[:384].view(3, 2, 64))                        # an input inside open_out
    with pytest.raises(ValueError):
        attn.kv_read(*pool, table, i32([0, 3, 4]), 4)
