"""4-bit products whose weights are much larger than what tells them apart: a product in 32 bits keeps it, one by weights of 16 bits
does not.  Bounds are those of 32-bit arithmetic for every kernel and output type (layer_helpers.q4_product without `rounded`)."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def linear():
    from gated_deltanet_linear_03_gb300 import linear as m
    return m


def offset_matrix(linear, n_out, k, group, seed, ratio=200.0):
    """Scales near 1 and offsets of `ratio` of them: neighbouring codes differ by a two-hundredth of a weight."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.randint(0, 256, (n_out, k // 2), generator=g, device="cuda").to(torch.uint8)
    scales = (1 + torch.rand(n_out, k // group, generator=g, device="cuda")).to(BF)
    return linear.Q4(codes, scales, (ratio * scales.float() * (0.7 + torch.rand(n_out, k // group, generator=g, device="cuda"))).to(BF))


def differences(rows, k, group, seed):
    """Rows with 1 at one input and -1 at another of the same group: a product is the difference of two weights."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros(rows, k, device="cuda")
    base = torch.randint(0, k // group, (rows,), generator=g, device="cuda") * group
    i = torch.randint(0, group, (rows,), generator=g, device="cuda")
    j = (i + 1 + torch.randint(0, group - 1, (rows,), generator=g, device="cuda")) % group
    at = torch.arange(rows, device="cuda")
    x[at, base + i], x[at, base + j] = 1.0, -1.0
    return x.to(BF)


SHAPES = [(1, 520, 2048), (2, 700, 1024), (5, 333, 640), (33, 4100, 1024), (33, 1000, 4096), (100, 513, 2048), (300, 450, 128), (509, 1208, 1984),
          (40, 20000, 1024), (70, 600, 16384)]


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("rows,n_out,k", SHAPES)
def test_differences_of_weights(linear, rows, n_out, k, group):
    if k % group:
        k += 64
    w, x = offset_matrix(linear, n_out, k, group, seed=k), differences(rows, k, group, seed=rows)
    for dtype in (BF, F32):
        ref.check(linear.q4_linear(x, w, out_dtype=dtype), *ref.q4_product(x, w))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,n_out,k", [(1, 520, 2048), (33, 1000, 4096), (64, 513, 1664), (300, 450, 128), (509, 1208, 1984)])
def test_differences_through_a_gate(linear, rows, n_out, k, act):
    gate, up = (offset_matrix(linear, n_out, k, 64, seed=s) for s in (1, 2))
    x = differences(rows, k, 64, seed=rows)
    f = 1 / 32                              # both factors about 1
    gate, up = (linear.Q4(w.codes, (w.scales * f), (w.offsets * f)) for w in (gate, up))
    (a, ea), (b, eb) = ref.q4_product(x, gate), ref.q4_product(x, up)
    y, _ = ref.gated(x, gate, up, act)
    # slopes of both activations are below 1.13, their size below that of the argument; the exponential's form is good to 2^-18
    bound = 1.13 * ea * (b.abs() + eb) + a.abs() * eb + 2.0 ** -18 * y.abs() + 2.0 ** -20 * (a.abs() * b.abs()).clamp_max(1e-6)
    ref.check(linear.q4_gated(x, gate, up, act=act), y, bound)


@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("offsets", [True, False])
@pytest.mark.parametrize("rows,n_out,k", SHAPES)
def test_a_large_group_beside_small_ones(linear, rows, n_out, k, offsets, group):
    """One group of every row 1000 times larger than the others, at inputs that are zero: the others keep 32 bits' worth.  With
    the row's largest 15 |scale| + |offset| in [2^-2, 2^-1), a half below 2^-14 is off by 2^-25 at most, once as -8 scale and once as the
    weight: 2^-22 of the largest."""
    if k % group:
        k += 64
    w = offset_matrix(linear, n_out, k, group, seed=n_out, ratio=-7.0)
    large = torch.arange(n_out, device="cuda") % (k // group)
    scales, offs = w.scales.clone(), w.offsets.clone()
    at = torch.arange(n_out, device="cuda")
    scales[at, large], offs[at, large] = scales[at, large] * 1000, offs[at, large] * 1000
    w = linear.Q4(w.codes, scales, offs if offsets else None)
    x = torch.randn(rows, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows))
    x.view(rows, -1, group)[:, : max(1, k // group // 2)] = 0                    # half of the groups
    x = x.to(BF)
    y, e = ref.q4_product(x, w)
    top = (15 * scales.double().abs() + (offs.double().abs() if offsets else 0)).amax(dim=1)
    e = e + 2.0 ** -22 * x.double().abs().sum(-1, keepdim=True) * top
    ref.check(linear.q4_linear(x, w), y, e)
    ref.check(linear.q4_linear(x, w, out_dtype=F32), y, e)


@pytest.mark.parametrize("rows", [1, 2, 3, 16, 24, 40, 100])
def test_offsets_alone_and_sums_that_cancel(linear, rows):
    """Codes of zero and equal scales: a product is the offsets' part, in which sums over groups cancel one another."""
    k, n_out = 2048, 1500
    w = offset_matrix(linear, n_out, k, 64, seed=3)
    w = linear.Q4(torch.zeros_like(w.codes), w.scales, w.offsets)
    x = torch.randn(rows, k // 64, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows)).to(BF).float()
    x[:, :, 32:] = -x[:, :, :32]
    x[:, :, 0] += 1
    x = x.to(BF).view(rows, k)
    ref.check(linear.q4_linear(x, w), *ref.q4_product(x, w))
    ref.check(linear.q4_linear(x, w, out_dtype=F32), *ref.q4_product(x, w))


@pytest.mark.parametrize("rows", [2, 40, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_rows_in_every_kernel(linear, rows, dtype):
    """x as a slice of a wider projection gives the same bits as its copy."""
    for n_out, k in ((300, 512), (4100, 2048)):
        w = offset_matrix(linear, n_out, k, 64, seed=k, ratio=-7.0)
        wide = torch.randn(rows, 3 * k + 8, device="cuda", generator=torch.Generator(device="cuda").manual_seed(rows)).to(BF)
        x = wide[:, k + 8:2 * k + 8]
        assert torch.equal(linear.q4_linear(x, w, out_dtype=dtype), linear.q4_linear(x.contiguous(), w, out_dtype=dtype))
        assert torch.equal(linear.q4_gated(x, w, w, out_dtype=dtype), linear.q4_gated(x.contiguous(), w, w, out_dtype=dtype))
