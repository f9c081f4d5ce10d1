"""Python integers beyond a C int's range in calls of gdn_attend."""
import pytest
import torch

import attn_helpers as ref
from test_gpu_attend import I8, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_03_gb300 import attn as a
    return a


@pytest.mark.parametrize("m", [1, 300])
def test_windows_beyond_32_bits(attn, m):
    from gated_deltanet_linear_03_gb300.gdn import GdnError
    lens = [m + 90]
    cache = ref.make_cache(lens, 2, 64, 16, I8, 3)
    q = torch.randn(m, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 40), dict(window=3, sinks=2 ** 32 + 1)):
        out, cu = run(attn, q, cache, [m], lens, **kw)
        check(out, *ref.attend(q, cache, cu, lens))
    for kw in (dict(window=-2 ** 32), dict(sinks=-2 ** 32), dict(window=-2 ** 40 + 3), dict(max_kv=2 ** 32 + lens[0])):
        with pytest.raises(GdnError):
            run(attn, q, cache, [m], lens, **kw)
