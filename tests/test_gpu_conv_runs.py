"""gdn_short_conv in long runs of tokens: strided rows, and as many tokens as 32 bits count."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF
from test_gpu_short_conv import cu_of, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    from gated_deltanet_linear_03_gb300 import ssm as s
    return s


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens", [[700, 1, 3000, 0, 25, 900], [9000]])
def test_slices_of_a_projection(ssm, width, lens):
    C = 2048
    i = inputs(lens, C, width, seed=width)
    wide = torch.randn(sum(lens), 2 * C + 8, device="cuda").to(BF)
    x = wide[:, 8:8 + C]
    state = torch.full_like(i["past"], 7.0)
    out = ssm.short_conv(x, i["weight"], cu_of(lens), bias=i["bias"], state_in=i["past"], state_out=state)
    y, e, s = ref.conv(x, i["weight"], lens, i["bias"], "silu", i["past"])
    ref.check(out, y, e)
    assert torch.equal(state.double(), s)


def test_almost_as_many_tokens_as_32_bits_count(ssm):
    """2147483000 tokens of 8 channels: where the last run begins, a whole run more would pass 2^31.  34 GB each of x and out."""
    T, C = 2147483000, 8
    x = torch.zeros(T, C, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-3000:] = torch.randn(3000, C, generator=g, device="cuda").to(BF)
    w = torch.randn(C, 2, generator=g, device="cuda")
    out = torch.full((T, C), 3.0, dtype=BF, device="cuda")
    state = torch.empty(1, 1, C, dtype=BF, device="cuda")
    ssm.short_conv(x, w, torch.tensor([0, T], dtype=torch.int32, device="cuda"), state_out=state, out=out)
    y, e, _ = ref.conv(x[-3000:], w, [3000], None, "silu", None)
    ref.check(out[-2999:], y[1:], e[1:])
    assert (out[:64] == 0).all() and (out[T // 2:T // 2 + 64] == 0).all() and torch.equal(state[0], x[-1:])
