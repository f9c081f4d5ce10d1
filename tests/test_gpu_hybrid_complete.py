"""The complete hybrid stack of examples/hybrid_block.py: short convolutions, the selective scan and 4-bit products beside the
recurrence, attention and norms, decoded token by token, prefilled at once and in pieces."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def far(a, b):
    return ((a - b).square().mean() / b.square().mean()).sqrt().item()


@pytest.mark.parametrize("dtype,limit", [(torch.int8, 0.06), (torch.float8_e4m3fn, 0.12)])
def test_decode_equals_prefill(dtype, limit):
    """Both ways round the same values to bf16 at the same places, but sum in other orders, so that a rounding may fall the other
    way: four layers of about 10 roundings of relative size 2^-9 behind one another, each carried on with a gain near 1, give
    2^-9 sqrt(40) = 1.3 %; products of many rows round their weights to fp16, another 2^-12 sqrt(20) = 0.1 %.  Tokens in an
    unfinished block of 16 see its 8-bit scale as it was: half a step, 1/254 (int8) or 1/16 (e4m3) of a value, on at most 15 of 61
    to 224 tokens, and the attention layer is one of four that add up.  Twice the sum of these stays below 6 % and 12 %."""
    import hybrid_block
    decoded, whole = hybrid_block.run(24, dtype, complete=True)
    assert torch.isfinite(decoded).all() and torch.isfinite(whole).all()
    assert far(decoded, whole) <= limit


@pytest.mark.parametrize("prompts", [(700, 3, 1), (1, 1), (40,)])
def test_pieces(prompts):
    """A prompt in two pieces: states of the convolutions, the recurrence and the scan, and the cache, carry over.  The bound is
    the one above; the 16-token blocks are quantised afresh, so the cache does not add to it."""
    import hybrid_block
    gen = torch.Generator().manual_seed(3)
    xs = [torch.randn(m, hybrid_block.DIM, generator=gen).to(torch.bfloat16).cuda() for m in prompts]
    whole = hybrid_block.Hybrid(len(prompts), complete=True).forward(torch.cat(xs), list(prompts)).float()
    first = [max(1, m // 3) for m in prompts]
    served = hybrid_block.Hybrid(len(prompts), complete=True)
    a = served.forward(torch.cat([x[:f] for x, f in zip(xs, first)]), first).float().split(first)
    rest = [m - f for m, f in zip(prompts, first)]
    b = [None] * len(prompts)
    if sum(rest):
        b = served.forward(torch.cat([x[f:] for x, f in zip(xs, first)]), rest).float().split(rest)
    got = torch.cat([torch.cat([p, q]) if q is not None else p for p, q in zip(a, b)])
    assert far(got, whole) <= 0.06
