"""4-bit products of activations and weights near the ends of their types' ranges."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, F32
from test_gpu_q4_weights import offset_matrix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def linear():
    from gated_deltanet_linear_03_gb300 import linear as m
    return m


@pytest.mark.parametrize("rows,n_out,k", [(1, 300, 512), (2, 300, 512), (3, 300, 512), (5, 40, 4096), (16, 77, 256), (24, 200, 512), (60, 300, 512),
                                          (70, 200, 4096)])
@pytest.mark.parametrize("offsets", [True, False])
def test_the_largest_inputs_and_weights(linear, rows, n_out, k, offsets):
    """Activations near the end of bf16's range by small weights, and weights near it by small activations: nothing overflows that the
    result does not."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    w = offset_matrix(linear, n_out, k, 64, seed=5, ratio=-7.0)
    if not offsets:
        w = linear.Q4(w.codes, w.scales, None)
    x = (torch.rand(rows, k, generator=g, device="cuda") * 2 - 1)
    for fx, fw in ((3.3e38, 1e-6), (1e-6, 5e36)):              # weights up to 30 fw and 24 fw are numbers of 32 bits
        big = linear.Q4(w.codes, (w.scales * fw).to(BF), None if w.offsets is None else (w.offsets * fw).to(BF))
        v = (x * fx).to(BF)
        for dtype in (BF, F32):
            ref.check(linear.q4_linear(v, big, out_dtype=dtype), *ref.q4_product(v, big))
