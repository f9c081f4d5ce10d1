"""The hybrid stack of examples/hybrid_block.py: decoding token by token gives what a prefill of everything gives."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
def test_decode_equals_prefill(dtype):
    """Both ways round the same values to bf16 at the same places, but sum in other orders, so that a rounding may fall
    the other way: about 20 roundings of relative size 2^-9 behind one another, each carried on with a gain near 1, give
    2^-9 sqrt(20) = 0.9 %.  The tokens that are still in an unfinished block of 16 when they are decoded see its
    8-bit scale as it was then: up to half a step, 1/254 (int8) or 1/16 (e4m3) of a value, on at most 15 of 61 to 224
    tokens, and the attention layer is one of the two that add up.  Twice the sum of these stays below 5 % (int8) and 10 %
    (e4m3)."""
    import hybrid_block
    decoded, whole = hybrid_block.run(24, dtype)
    assert torch.isfinite(decoded).all() and torch.isfinite(whole).all()
    rel = ((decoded - whole).square().mean() / whole.square().mean()).sqrt().item()
    assert rel <= (0.05 if dtype is torch.int8 else 0.10), rel
