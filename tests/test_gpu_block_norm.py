"""gdn_block_norm against the plain 64-bit form."""
import pytest
import torch

import attn_helpers as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def norm():
    from gated_deltanet_linear_03_gb300 import norm as n
    return n


def inputs(rows, dim, residual, seed=0, big=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=(big * r(rows, dim)).to(BF), gate=(3 * r(rows, dim)).to(BF), residual=(big * r(rows, dim)).to(residual),
                post=1 + 0.3 * r(dim), pre=1 + 0.3 * r(dim), scale=0.5 + 0.2 * r(dim))


def check(got, want):
    """32-bit arithmetic: sums of squares of dim terms (tree of depth < 32: 2^-19), a reciprocal root, an exponential
    (2^-20 for |gate| < 16), a few products: 2^-17 of the added term and of the result; then one rounding."""
    (r, h), (rw, hw, add) = got, want
    half = 2.0 ** -8 if r.dtype == BF else 0.0
    assert ((r.cpu().double() - rw).abs() <= half * rw.abs() + 2.0 ** -17 * add + 2.0 ** -23 * rw.abs() + 1e-37).all()
    rms = (rw ** 2).mean(-1, keepdim=True).sqrt()
    spread = 2.0 ** -17 * hw.abs() + 2.0 ** -16 * (add + 0.01 * rw.abs()) / rms.clamp_min(1e-30) * 2.5
    assert ((h.cpu().double() - hw).abs() <= 2.0 ** -8 * hw.abs() + spread + 1e-37).all()


@pytest.mark.parametrize("residual", [BF, F32])
@pytest.mark.parametrize("rows,dim", [(1, 8), (1, 2048), (3, 248), (2, 256), (7, 264), (5, 1000), (2, 5120), (1, 8192), (2, 8200), (3, 16384)])
def test_sizes(norm, rows, dim, residual):
    i = inputs(rows, dim, residual, seed=dim)
    d = {k: t.cuda() for k, t in i.items()}
    got = norm.block_norm(d["x"], d["residual"], d["pre"], post_weight=d["post"], gate=d["gate"], scale=d["scale"])
    check(got, ref.block_norm(i["x"], i["residual"], i["pre"], i["post"], i["gate"], "sigmoid", i["scale"]))


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "sigmoid", "silu"])
@pytest.mark.parametrize("scale", ["number", "channel"])
@pytest.mark.parametrize("residual", [BF, F32])
def test_options(norm, post, gate, scale, residual):
    i = inputs(9, 520, residual, seed=3)
    d = {k: t.cuda() for k, t in i.items()}
    got = norm.block_norm(d["x"], d["residual"], d["pre"], post_weight=d["post"] if post else None, gate=d["gate"] if gate else None,
                          gate_act=gate or "sigmoid", scale=d["scale"] if scale == "channel" else -0.75, eps=1e-5)
    check(got, ref.block_norm(i["x"], i["residual"], i["pre"], i["post"] if post else None, i["gate"] if gate else None, gate or "sigmoid",
                              i["scale"] if scale == "channel" else -0.75, 1e-5))


def test_many_rows_and_leading_dimensions(norm):
    i = inputs(1999, 2048, F32, seed=1)
    d = {k: t.cuda() for k, t in i.items()}
    got = norm.block_norm(d["x"], d["residual"], d["pre"], post_weight=d["post"], gate=d["gate"], gate_act="silu", scale=0.5)
    check(got, ref.block_norm(i["x"], i["residual"], i["pre"], i["post"], i["gate"], "silu", 0.5))
    shaped = norm.block_norm(d["x"][:6].view(2, 3, 2048), d["residual"][:6].view(2, 3, 2048), d["pre"], post_weight=d["post"],
                             gate=d["gate"][:6].view(2, 3, 2048), gate_act="silu", scale=0.5)
    assert torch.equal(shaped[0].view(6, -1), got[0][:6]) and torch.equal(shaped[1].view(6, -1), got[1][:6])


def test_in_place(norm):
    i = inputs(5, 1024, BF, seed=2)
    d = {k: t.cuda() for k, t in i.items()}
    kw = dict(post_weight=d["post"], gate=d["gate"], scale=0.5)
    want = norm.block_norm(d["x"], d["residual"], d["pre"], **kw)
    x, r = d["x"].clone(), d["residual"].clone()
    got = norm.block_norm(x, r, d["pre"], residual_out=r, out=x, **kw)
    assert got[0] is r and got[1] is x and torch.equal(r, want[0]) and torch.equal(x, want[1])
    g = d["gate"].clone()
    got = norm.block_norm(d["x"], d["residual"], d["pre"], post_weight=d["post"], gate=g, scale=0.5, out=g)
    assert torch.equal(g, want[1])


def test_zero_rows_and_extreme_values(norm):
    """A row of zeros stays finite through eps; a saturated gate is 0 or 1; a NaN stays in its row."""
    i = inputs(4, 256, F32, seed=5)
    i["x"][0] = 0
    i["residual"][0] = 0
    i["gate"][1, :128] = 200.0
    i["gate"][1, 128:] = -200.0
    i["x"][2, 7] = float("nan")
    d = {k: t.cuda() for k, t in i.items()}
    for act in ("sigmoid", "silu"):
        r, h = norm.block_norm(d["x"], d["residual"], d["pre"], post_weight=d["post"], gate=d["gate"], gate_act=act, scale=1.0)
        assert (r[0] == 0).all() and (h[0] == 0).all()
        assert h[2].isnan().all()
        rw, hw, add = ref.block_norm(i["x"], i["residual"], i["pre"], i["post"], i["gate"], act, 1.0)
        for row in (1, 3):
            check((r[row:row + 1], h[row:row + 1]), (rw[row:row + 1], hw[row:row + 1], add[row:row + 1]))


def test_nothing_to_do(norm):
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    r, h = norm.block_norm(e, e, torch.ones(64, device="cuda"))
    assert r.shape == h.shape == (0, 64)


def test_refusals(norm):
    from gated_deltanet_linear_03_gb300.gdn import GdnError
    d = {k: t.cuda() for k, t in inputs(2, 64, BF).items()}
    norm.block_norm(d["x"], d["residual"], d["pre"])
    for a in ((d["x"].float(), d["residual"], d["pre"]), (d["x"].cpu(), d["residual"], d["pre"]), (d["x"], d["residual"].half(), d["pre"]),
              (d["x"], d["residual"][:1], d["pre"]), (d["x"], d["residual"], d["pre"][:32].contiguous()), (d["x"].t(), d["residual"], d["pre"])):
        with pytest.raises(ValueError):
            norm.block_norm(*a)
    with pytest.raises(ValueError):
        norm.block_norm(d["x"], d["residual"], d["pre"], gate_act="relu")
    with pytest.raises(GdnError):
        norm.block_norm(d["x"], d["residual"], d["pre"], eps=-1.0)
    with pytest.raises(GdnError):
        norm.block_norm(d["x"], d["residual"], d["pre"], scale=float("inf"))
    with pytest.raises(GdnError):
        norm.block_norm(d["x"][:, :60].contiguous(), d["residual"][:, :60].contiguous(), d["pre"][:60].contiguous())   # dim % 8
    with pytest.raises(GdnError):
        norm.block_norm(d["x"], d["residual"], d["pre"], residual_out=d["x"])      # an output over an input
