"""gdn_attend of prompts under a sliding window whose scores are all far below zero.  A softmax does not depend on an offset
that all scores of a row share, so neither may a row whose window begins behind the first tile of its item."""
import pytest
import torch

import attn_helpers as ref
from test_gpu_attend import F8, I8, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


def shifted(lens, new, hq, hkv, d, page, dtype, target, seed, zero_every=0):
    """A cache and queries whose products are near -target: component 0 of every key is -8 and of every query
    target sqrt(d) / 8, the others are noise.  With `zero_every` each such block of V is zero."""
    gen = torch.Generator().manual_seed(seed)
    table, n_pages = ref.make_table(lens, page, gen)
    out = []
    for which in "kv":
        x = torch.randn(n_pages, hkv, page // ref.BLOCK, ref.BLOCK, d, generator=gen)
        if which == "k":
            x[..., 0] = -8.0
        elif zero_every:
            for i, length in enumerate(lens):
                for b in range(zero_every - 1, -(-length // ref.BLOCK), zero_every):
                    x[table[i, b * ref.BLOCK // page], :, b * ref.BLOCK % page // ref.BLOCK] = 0
        codes, scales = ref.quantise(x.to(torch.bfloat16), dtype)
        out.append((codes.view(torch.int8).view(n_pages, hkv, page, d).contiguous().view(dtype), scales.contiguous()))
    q = torch.randn(sum(new), hq, d, generator=gen)
    q[..., 0] = target * d ** 0.5 / 8
    return ref.Cache(table, out[0][0], out[1][0], out[0][1], out[1][1]), q.to(torch.bfloat16)


def compare(attn, lens, new, hq, hkv, d, page, dtype, target, window, sinks, seed, zero_every=0):
    cache, q = shifted(lens, new, hq, hkv, d, page, dtype, target, seed, zero_every)
    out, cu = run(attn, q, cache, new, lens, window=window, sinks=sinks)
    check(out, *ref.attend(q, cache, cu, lens, window, sinks))


@pytest.mark.parametrize("target", [84, 90, 300])
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 8])
def test_scores_far_below_zero(attn, group, d, sinks, target):
    """Many items of several units each; the window of most rows begins in a later unit than that of the item's first row."""
    m = 400 // group + 13
    compare(attn, [m, m + 50, m + 260], [m, m, m - 1], 8, 8 // group, d, 32, I8, target, 70, sinks, d + group)


@pytest.mark.parametrize("target", [84, 300])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 4), (128, 8, 8), (256, 4, 4)])
def test_pieces_behind_a_long_cache(attn, d, hq, hkv, target):
    """The first tokens stay visible and the window lies far behind them: a run that begins at the far tile must not lose it."""
    compare(attn, [2900] * 3, [300, 290, 301], hq, hkv, d, 48, F8, target, 500, 5, d)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_zero_blocks_among_scores_below_zero(attn, d):
    """Blocks of zero values, whose tokens count in the denominator at scores near -50."""
    compare(attn, [450, 500], [400, 410], 4, 4, d, 32, I8, 50, 70, 0, d, zero_every=2)
