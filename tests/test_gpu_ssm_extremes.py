"""gdn_ssm_scan at the ends of its inputs' ranges: step widths of zero and without end, decays that leave fp32, and plans that only
long or narrow inputs reach."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, F32, i32
from test_gpu_ssm_scan import JOINED, both, cu_of, inputs

pytestmark = pytest.mark.gpu
LOW, HIGH = torch.finfo(BF).min, torch.finfo(BF).max


@pytest.fixture(scope="module")
def ssm():
    from gated_deltanet_linear_03_gb300 import ssm as s
    return s


def scan(ssm, i, lens, cu="given", **kw):
    state = torch.full_like(i["past"], 7.0)
    out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens) if cu else None, d=i["d"], z=i["z"], dt_bias=i["bias"],
                   state_in=i["past"], state_out=state, max_len=max(lens), out_dtype=F32, **kw)
    return out, state


# single tokens, one pass, pieces
PLANS = [([1, 1, 1], None), ([45, 9, 1], "given"), ([1800, 700, 3], "given")]


@pytest.mark.parametrize("lens,cu", PLANS)
@pytest.mark.parametrize("low", [float("-inf"), LOW, -2.4e38, -1e30, -1000.0, -104.0, -100.0, -88.0])
@pytest.mark.parametrize("where", ["dt", "bias"])
def test_tokens_without_a_step(ssm, lens, cu, low, where):
    """dt of -inf or the lowest number: a width of zero, which leaves the state as it is (a padded token)."""
    i = inputs(lens, 64, 16, seed=21)
    if where == "dt":
        i["dt"][::3] = low
    else:
        i["bias"][::3] = low
    both(ssm, i, lens, cu=cu)


@pytest.mark.parametrize("lens,cu", PLANS)
@pytest.mark.parametrize("n_state", [16, 128])
def test_widths_as_large_as_numbers_are(ssm, lens, cu, n_state):
    """dt of bf16's largest number: the width is that number, everything before is forgotten."""
    i = inputs(lens, 32, n_state, seed=22)
    i["a"].clamp_max_(-0.01)
    for row in (0, 8, 17, 1000):
        if row < sum(lens):
            i["dt"][row], i["x"][row] = HIGH, (1e-37 * torch.randn(32, device="cuda")).to(BF)
    both(ssm, i, lens, cu=cu)


@pytest.mark.parametrize("lens,cu", PLANS)
@pytest.mark.parametrize("what", ["dt", "bias", "x"])
def test_nan_and_infinity_are_kept(ssm, lens, cu, what):
    """A NaN (or a width of +inf) is seen in the outputs and the state of its channel, and in no other channel."""
    i = inputs(lens, 32, 16, seed=23)
    want, _ = scan(ssm, i, lens, cu)
    for value in (float("nan"), float("inf")):
        j = {k: v.clone() for k, v in i.items()}
        if what == "bias":
            j["bias"][5] = value
        else:
            j[what][0, 5] = value
        out, state = scan(ssm, j, lens, cu)
        assert not torch.isfinite(out[0, 5]) and not torch.isfinite(state[0, 5]).all() or lens[0] > 1
        if value != value:
            assert torch.isnan(out[:lens[0], 5]).all() and torch.isnan(state[0, 5]).all()
        else:
            assert not torch.isfinite(out[0, 5])
        rest = [c for c in range(32) if c != 5]
        assert torch.equal(out[:, rest], want[:, rest]) and torch.isfinite(state[:, rest]).all()


@pytest.mark.parametrize("lens,cu", PLANS + [([41], "given"), ([8], "given"), ([1801], "given")])
@pytest.mark.parametrize("n_state", [16, 64, 128])
def test_a_decay_without_end(ssm, lens, cu, n_state):
    """a = -inf forgets everything at every token, as a = -1e30 does, whatever the lengths."""
    i = inputs(lens, 32, n_state, seed=24)
    i["a"][::4, 1], i["a"][1::4] = -1e30, -1e30
    want = scan(ssm, i, lens, cu)
    i["a"][::4, 1], i["a"][1::4] = float("-inf"), float("-inf")
    got = scan(ssm, i, lens, cu)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens,cu", PLANS)
@pytest.mark.parametrize("low", [float("-inf"), LOW, -100.0])
def test_a_decay_without_end_and_no_step(ssm, lens, cu, low):
    """A token whose width is zero leaves the state as it is, for a = -inf too."""
    i = inputs(lens, 32, 16, seed=31)
    i["a"][:, 3] = -1e30
    i["dt"][::2] = low
    want = scan(ssm, i, lens, cu)
    i["a"][:, 3] = float("-inf")
    got = scan(ssm, i, lens, cu)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("lens,cu", PLANS)
def test_a_that_is_not_a_number_is_seen(ssm, lens, cu):
    i = inputs(lens, 32, 16, seed=32)
    want = scan(ssm, i, lens, cu)
    i["a"][7, 2] = float("nan")
    got = scan(ssm, i, lens, cu)
    rest = [c for c in range(32) if c != 7]
    assert torch.isnan(got[0][:, 7]).all() and torch.isnan(got[1][:, 7, 2]).all()
    assert torch.equal(got[0][:, rest], want[0][:, rest]) and torch.equal(got[1][:, rest], want[1][:, rest])


def test_growth_behind_zeros_in_pieces(ssm):
    """A state of zero stays zero however much a piece's tokens would have let it grow."""
    lens, C = [3000], 64
    i = inputs(lens, C, 16, seed=25)
    i["a"] = torch.full_like(i["a"], 1.0)
    i["past"].zero_()
    i["dt"] = torch.full_like(i["dt"], 0.25)
    i["x"][:2960] = 0
    kw = dict(dt_softplus=False, d=i["d"], z=i["z"], max_len=3000, out_dtype=F32)
    state = torch.empty_like(i["past"])
    out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), state_in=i["past"], state_out=state, **kw)
    y, e, h, he = ref.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], lens, i["d"], i["z"], None, False, i["past"])
    assert (out[:2960] == 0).all()
    # no piece begins with a state but those of the last 40 tokens, which decay over 64 tokens at most (widths of 1/4: exact sums)
    ref.check(out, y, e + 2.0 ** -19 * y.abs())
    ref.check(state, h, he + 2.0 ** -19 * h.abs())


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_growth_and_decay_beyond_fp32_in_pieces(ssm, sign):
    """From 1e-30 by e^120, which fp32 does not hold as a factor, to what it holds; and back."""
    lens, C = [3000], 64
    i = inputs(lens, C, 16, seed=26)
    i["a"] = torch.full_like(i["a"], sign)
    i["past"] = i["past"] * (1e-30 if sign > 0 else 1e22)
    i["dt"] = torch.full_like(i["dt"], 0.0400390625)            # exact in bf16; sums of 3000 in fp32 are off by 2^-24 of 120 each at most
    i["x"].zero_()
    state = torch.empty_like(i["past"])
    ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), state_in=i["past"], state_out=state, dt_softplus=False, max_len=3000)
    h = i["past"].double() * torch.exp(torch.tensor(sign * 3000 * 0.0400390625, dtype=torch.float64))
    # 3000 factors, each good to 2^-21 (its exponential and the product), or fewer by pieces whose exponents are rounded as often
    assert ((state.double() - h).abs() <= 3000 * 2.0 ** -21 * h.abs()).all()


@pytest.mark.parametrize("n_state,channels,groups,lens", [(16, 64, 4, [3000, 1, 900]), (64, 96, 2, [60, 2600, 300, 0, 7]), (128, 48, 3, [1500, 40]),
                                                          (32, 1536, 4, [1, 1999, 3])])
def test_groups_in_pieces(ssm, n_state, channels, groups, lens):
    i = inputs(lens, channels, n_state, groups, seed=27)
    both(ssm, i, lens)


def test_a_narrow_long_sequence(ssm):
    """More than a hundred pieces of one sequence, each of which begins with what all before it leave."""
    both(ssm, inputs([12000], 128, 16, seed=28), [12000])


@pytest.mark.parametrize("lens", [[3, 0, 2], [0, 0, 0], [1200, 0, 900], [0, 5]])
def test_a_slot_outside_the_pool_of_a_sequence_without_tokens(ssm, lens):
    """Recorded like any other, also where states stay in place."""
    from gated_deltanet_linear_03_gb300 import gdn
    i = inputs(lens, 64, 16, seed=29)
    n = len(lens)
    slots = [k if lens[k] or k != lens.index(0) else n for k in range(n)]
    g = torch.Generator(device="cuda").manual_seed(1)
    w, conv = torch.randn(64, 4, generator=g, device="cuda"), torch.randn(n, 3, 64, generator=g, device="cuda").to(BF)
    for in_place in (True, False):
        assert gdn.device_error() == 0
        state = i["past"].clone()
        ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), state_in=state, state_out=state if in_place else state.clone(),
                 slots=i32(slots), max_len=max(lens))
        assert gdn.device_error() == 6
        past = conv.clone()
        ssm.short_conv(i["x"], w, cu_of(lens), state_in=past, state_out=past if in_place else past.clone(), slots=i32(slots))
        assert gdn.device_error() == 6
        if in_place:
            rest = [k for k in range(n) if not lens[k]]
            assert torch.equal(past[rest], conv[rest]) and torch.equal(state[rest], i["past"][rest])


def test_outputs_are_rounded_once_to_bf16(ssm):
    lens = [500, 33]
    i = inputs(lens, 64, 16, seed=30)
    out, state = scan(ssm, i, lens)
    kept = torch.empty_like(state)
    half = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), d=i["d"], z=i["z"], dt_bias=i["bias"], state_in=i["past"], state_out=kept,
                    max_len=max(lens))
    assert torch.equal(half, out.to(BF)) and torch.equal(kept, state)
