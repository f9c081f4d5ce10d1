"""gdn_q4_linear and gdn_q4_gated against the plain 64-bit form."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def linear():
    from gated_deltanet_linear_03_gb300 import linear as m
    return m


def matrix(linear, n_out, k, group, offsets, seed):
    """Every code occurs; scales of both signs and of very different sizes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n_out, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = (torch.randn(n_out, k // group, generator=g, device="cuda") * k ** -0.5
              * torch.exp(torch.randn(n_out, 1, generator=g, device="cuda"))).to(BF)
    offs = (torch.randn(n_out, k // group, generator=g, device="cuda") * 4 * k ** -0.5).to(BF) if offsets else None
    return linear.Q4(codes, scales, offs)


def rounds(linear, x, w):
    """Calls that need a workspace may round the weights to fp16; in the others codes enter the products as they are."""
    return linear.workspace_size(x.shape[0], w.codes.shape[0], x.shape[1], x.shape[1] // w.scales.shape[1]) > 0


def rows_of(rows, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, k, generator=g, device="cuda").to(BF)


@pytest.mark.parametrize("group,offsets", [(64, True), (64, False), (128, True), (128, False)])
@pytest.mark.parametrize("rows,n_out,k", [(1, 1, 128), (1, 17, 256), (2, 1000, 2048), (7, 16, 1152), (9, 333, 640), (16, 50, 4096),
                                          (17, 129, 512), (33, 2047, 1024), (65, 200, 384), (130, 300, 2176), (40, 200, 1664), (150, 1001, 384),
                                          (600, 250, 128)])
def test_sizes(linear, rows, n_out, k, group, offsets):
    w, x = matrix(linear, n_out, k, group, offsets, seed=k), rows_of(rows, k, seed=rows)
    ref.check(linear.q4_linear(x, w, out_dtype=F32), *ref.q4_product(x, w))
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w, rounded=rounds(linear, x, w)))


@pytest.mark.parametrize("rows", [1, 3, 8, 12, 16, 24, 32, 40, 64, 100, 509])
@pytest.mark.parametrize("n_out,k", [(4100, 4096), (520, 192), (96, 8192)])
def test_rows(linear, rows, n_out, k):
    w, x = matrix(linear, n_out, k, 64, True, seed=n_out), rows_of(rows, k, seed=rows)
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w, rounded=rounds(linear, x, w)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("group,offsets", [(64, True), (128, False)])
@pytest.mark.parametrize("rows,n_out,k", [(1, 1, 128), (1, 5632, 2048), (5, 77, 256), (13, 1001, 384), (30, 40, 2048), (64, 513, 1024),
                                          (200, 260, 640), (64, 513, 1664), (200, 1000, 640), (90, 100, 2048), (300, 450, 128)])
def test_gated(linear, rows, n_out, k, group, offsets, act):
    gate, up = (matrix(linear, n_out, k, group, offsets, seed=s) for s in (1, 2))
    x = rows_of(rows, k, seed=rows)
    ref.check(linear.q4_gated(x, gate, up, act=act, out_dtype=F32), *ref.gated(x, gate, up, act))
    ref.check(linear.q4_gated(x, gate, up, act=act), *ref.gated(x, gate, up, act, rounded=rounds(linear, x, gate)))


@pytest.mark.parametrize("rows,k", [(1, 16384), (40, 16384), (64, 12288), (3, 65536), (70, 65536)])
def test_long_rows(linear, rows, k):
    w, x = matrix(linear, 40, k, 128, True, seed=1), rows_of(rows, k, seed=2)
    ref.check(linear.q4_linear(x, w, out_dtype=F32), *ref.q4_product(x, w))
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w, rounded=rounds(linear, x, w)))


def test_a_vocabulary(linear):
    w, x = matrix(linear, 131071, 2048, 64, True, seed=3), rows_of(2, 2048, seed=4)
    out = linear.q4_linear(x, w, out_dtype=F32)
    for at in (0, 65500, 131000):
        part = linear.Q4(*(t[at:at + 71] for t in w))
        y, e = ref.q4_product(x, part)
        ref.check(out[:, at:at + 71], y, e)


def test_beyond_32_bit_offsets(linear):
    """600000 outputs of 8192 inputs: 2.46e9 bytes of codes; 5000 rows by them: 3e9 outputs."""
    n, k = 600_000, 8192
    w = linear.Q4(torch.randint(0, 256, (n, k // 2), device="cuda", dtype=torch.uint8),
                  (torch.rand(n, k // 128, device="cuda") * 0.01).to(BF), None)
    x = rows_of(1, k, seed=5)
    out = linear.q4_linear(x, w, out_dtype=F32)
    part = linear.Q4(w.codes[-100:], w.scales[-100:])
    y, e = ref.q4_product(x, part)
    ref.check(out[:, -100:], y, e)
    small = linear.Q4(w.codes[:, :64].contiguous(), w.scales[:, :1].contiguous())
    x = rows_of(5000, 128, seed=6)
    out = linear.q4_linear(x, small)
    part = linear.Q4(small.codes[-300:], small.scales[-300:])
    ref.check(out[-70:, -300:], *ref.q4_product(x[-70:], part, rounded=True))


def test_slices_shapes_and_outputs(linear):
    w = matrix(linear, 96, 256, 64, True, seed=7)
    proj = rows_of(12, 3 * 256, seed=8)
    x = proj[:, 256:512]
    want = linear.q4_linear(x.contiguous(), w)
    assert torch.equal(linear.q4_linear(x, w), want)
    assert torch.equal(linear.q4_linear(x.contiguous().view(3, 4, 256), w), want.view(3, 4, 96))
    assert torch.equal(linear.q4_linear(x[5], w), want[5])
    out = torch.full((14, 96), 5.0, dtype=BF, device="cuda")
    assert linear.q4_linear(x, w, out=out[1:13]).data_ptr() == out[1].data_ptr()
    assert torch.equal(out[1:13], want) and (out[[0, 13]] == 5).all()
    assert linear.q4_linear(x[:0], w).shape == (0, 96)


@pytest.mark.parametrize("k", [512, 2048])
@pytest.mark.parametrize("rows", [1, 20, 64, 300])
def test_not_finite_rows_stay_alone(linear, rows, k):
    w, x = matrix(linear, 200, k, 64, True, seed=9), rows_of(rows, k, seed=10)
    want = linear.q4_linear(x, w)
    x[rows // 2, 100] = float("nan")
    if rows > 4:
        x[rows // 2 + 2, 7] = float("inf")
    out = linear.q4_linear(x, w)
    bad = [rows // 2] + ([rows // 2 + 2] if rows > 4 else [])
    assert not torch.isfinite(out[bad]).any()
    rest = [i for i in range(rows) if i not in bad]
    assert torch.equal(out[rest], want[rest])


@pytest.mark.parametrize("k", [512, 2048])
def test_large_and_small_values(linear, k):
    """Activations up to 1e30 and down to 1e-30 in one call: every row keeps its own precision."""
    w, x = matrix(linear, 300, k, 64, True, seed=11), rows_of(40, k, seed=12).float()
    x = (x * 10.0 ** torch.linspace(-30, 30, 40, device="cuda")[:, None]).to(BF)
    ref.check(linear.q4_linear(x, w, out_dtype=F32), *ref.q4_product(x, w))
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w, rounded=rounds(linear, x, w)))


@pytest.mark.parametrize("rows,k", [(3, 1024), (50, 1024), (50, 2048)])
def test_weights_of_very_different_sizes(linear, rows, k):
    """Rows of weights up to 1e30 and down to 1e-30, and groups in a row a million times smaller than others."""
    w, x = matrix(linear, 200, k, 64, True, seed=21), rows_of(rows, k, seed=22)
    f = 10.0 ** torch.linspace(-30, 30, 200, device="cuda")[:, None] * 10.0 ** (-6 * torch.rand(200, k // 64, device="cuda"))
    w = linear.Q4(w.codes, (w.scales * f).to(BF), (w.offsets * f).to(BF))
    ref.check(linear.q4_linear(x, w, out_dtype=F32), *ref.q4_product(x, w))
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w, rounded=rounds(linear, x, w)))


@pytest.mark.parametrize("k", [512, 2048])
def test_rows_of_zeros(linear, k):
    w, x = matrix(linear, 200, k, 64, True, seed=23), rows_of(40, k, seed=24)
    x[3] = 0
    zero = linear.Q4(w.codes, w.scales.clone(), w.offsets.clone())
    zero.scales[7], zero.offsets[7] = 0, 0
    out = linear.q4_linear(x, zero)
    assert (out[3] == 0).all() and (out[:, 7] == 0).all()
    ref.check(out, *ref.q4_product(x, zero, rounded=rounds(linear, x, zero)))


@pytest.mark.parametrize("offsets", [True, False])
@pytest.mark.parametrize("group", [64, 128])
def test_quantize(linear, offsets, group):
    """A value within its group's range is at most half a scale off, and what the roundings of the scale and offset to bf16 move
    it by: 15 scales and the offset, each by 2^-9 relative to itself at most."""
    w = torch.randn(50, 512, device="cuda")
    q = linear.quantize(w, group, offsets)
    got = linear.values(q)
    assert torch.equal(got.double(), ref.q4_values(q).float().double())
    s = q.scales.float().repeat_interleave(group, dim=1)
    o = q.offsets.float().abs().repeat_interleave(group, dim=1) if offsets else 0
    assert ((got - w).abs() <= 0.5 * s + 15 * s * 2.0 ** -8 + 2.0 ** -8 * o + 1e-6).all()
    zero = linear.quantize(torch.zeros(4, 256, device="cuda"), group, offsets)
    assert (linear.values(zero) == 0).all()


@pytest.mark.parametrize("rows", [1, 3, 40])
def test_streams_and_graphs(linear, rows):
    w, x = matrix(linear, 1000, 2048, 64, True, seed=13), rows_of(rows, 2048, seed=14)
    y, e = ref.q4_product(x, w, rounded=rounds(linear, x, w))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    out = linear.q4_linear(x, w, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    ref.check(out, y, e)
    graph, keep = torch.cuda.CUDAGraph(), x.clone()
    with torch.cuda.graph(graph):
        out = linear.q4_linear(keep, w)
    for seed in (15, 16):
        keep.copy_(rows_of(rows, 2048, seed=seed))
        graph.replay()
        y, e = ref.q4_product(keep, w, rounded=rounds(linear, keep, w))
        ref.check(out, y, e)


def test_calls_at_once(linear):
    """Calls of every kind on two streams at the same time, which share the SMs and their tensor memory, give what they give alone."""
    made = []
    for seed, (rows, n_out, k) in enumerate([(33, 4096, 4096), (100, 20000, 1024), (500, 3000, 2048), (1, 9000, 2048), (9, 700, 8192),
                                             (20, 520, 6144)]):
        w, up, x = matrix(linear, n_out, k, 64, True, seed), matrix(linear, n_out, k, 64, True, seed + 50), rows_of(rows, k, seed)
        made += [lambda x=x, w=w: linear.q4_linear(x, w), lambda x=x, w=w, up=up: linear.q4_gated(x, w, up),
                 lambda x=x, w=w: linear.q4_linear(x, w, out_dtype=F32)]
    want = [f() for f in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(6):
        got = [None] * len(made)
        for i in range(len(made)):                    # the two streams meet in another pairing every time
            for s, j in ((0, i), (1, (5 * i + turn) % len(made))):
                with torch.cuda.stream(streams[s]):
                    out = made[j]()
                    if s == 0:
                        got[i] = out
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("rows,n_out,k", [(1, 1, 64), (2, 9, 1536), (1, 2431, 1024), (1, 2433, 2048), (2, 5000, 8192), (1, 40, 16384), (3, 40, 4096),
                                          (9, 129, 2048), (16, 260, 6144)])
def test_divisions_of_few_rows(linear, rows, n_out, k):
    """Sizes around those at which warps share a row's inputs, CTAs get a second turn, or the call goes to another kernel."""
    gate, up, x = matrix(linear, n_out, k, 64, True, 31), matrix(linear, n_out, k, 64, True, 32), rows_of(rows, k, 33)
    ref.check(linear.q4_linear(x, gate), *ref.q4_product(x, gate, rounded=rounds(linear, x, gate)))
    ref.check(linear.q4_linear(x, gate, out_dtype=F32), *ref.q4_product(x, gate))
    ref.check(linear.q4_gated(x, gate, up), *ref.gated(x, gate, up, "silu", rounded=rounds(linear, x, gate)))


def test_no_rows(linear):
    w = matrix(linear, 40, 256, 64, True, 1)
    assert linear.q4_linear(rows_of(0, 256, 1), w).shape == (0, 40) and linear.q4_gated(rows_of(0, 256, 1), w, w).shape == (0, 40)
