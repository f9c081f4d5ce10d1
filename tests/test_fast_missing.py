"""Without the Python binding's C++ part the modules' own code makes every call."""
import sys

import pytest
import torch

import gated_deltanet_linear_03_gb300 as pkg
from gated_deltanet_linear_03_gb300 import gdn, linear, ssm


@pytest.fixture
def missing(monkeypatch):
    monkeypatch.setitem(sys.modules, "gated_deltanet_linear_03_gb300._fast", None)
    monkeypatch.delattr(pkg, "_fast", raising=False)
    monkeypatch.setattr(gdn, "_fast", None)


def test_says_so_once_and_takes_no_call(missing):
    from gated_deltanet_linear_03_gb300 import _build
    _build.build()
    with pytest.warns(RuntimeWarning, match="_fast.so"):
        fast = gdn.fast_calls()
    assert gdn.fast_calls() is fast
    x = torch.zeros(2, 8, dtype=torch.bfloat16)
    assert fast.short_conv(x, x, None, None, 1, None, None, None, None) is None and fast.scan(x) is None
    assert fast.q4_linear(x, None, 0, None, 0) is None and fast.q4_gated(x, None, None, 0, None, 0) is None
    with pytest.raises(ValueError, match="CUDA"):
        ssm.short_conv(x, torch.zeros(8, 4))


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:_fast.so")
def test_calls_give_the_same(missing):
    from test_fast_calls import calls, same
    got = [fn(*args, **kw) for _, fn, args, kw in calls()]
    here = torch.cuda.current_stream()
    for out, (name, fn, args, kw) in zip(got, calls()):
        assert same(out, fn(*args, **kw, stream=here)), name
