"""The Python binding's C++ part: it gives what the modules' own code gives, and leaves to it what it does not take."""
import importlib.util
import os

import pytest
import torch

from layer_helpers import BF, i32

import gated_deltanet_linear_03_gb300 as pkg
from gated_deltanet_linear_03_gb300 import gdn, linear, ssm


@pytest.fixture(scope="module")
def fast():
    if not os.path.exists(os.path.join(os.path.dirname(pkg.__file__), "_fast.so")):
        pytest.skip("_fast.so not built")
    return gdn.fast_calls()


def test_leaves_what_it_does_not_take(fast):
    x, w = torch.zeros(2, 8, dtype=BF), torch.zeros(8, 4)
    assert fast.short_conv(x, w, None, None, 1, None, None, None, None) is None              # no CUDA tensors
    assert fast.short_conv(x, w) is None and fast.scan(x) is None and fast.q4_linear() is None and fast.q4_gated(x) is None
    nothing = (None, 1, "x", torch.zeros(3, 3))
    for a in nothing:
        for b in nothing:
            assert fast.short_conv(a, b, b, a, b, a, b, a, b) is None
            assert fast.scan(a, b, a, b, a, b, a, b, a, b, a, b, a, b, a, b) is None
            assert fast.q4_linear(a, b, a, b, a) is None and fast.q4_gated(a, (b, a, b), b, a, b, a) is None


def test_bind_refuses(fast):
    spec = importlib.util.find_spec("gated_deltanet_linear_03_gb300._fast")
    assert spec is not None
    for bad in ((), (1,) * 6, (1,) * 7, ("a",) * 6 + (RuntimeError,), (0,) * 6 + (RuntimeError,)):
        with pytest.raises((TypeError, ValueError)):
            fast.bind(*bad)


def calls(seed=0):
    """(name, function, arguments) of small calls, each in every form that the modules have of it."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T, C, N, G, lens = 21, 64, 16, 2, [3, 0, 17, 1]
    cu = i32([0, 3, 3, 20, 21])
    proj = r(T, 3 * C).to(BF)
    x, dt, z = proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:]
    bc = r(T, 2, G, N).to(BF)
    a, skip, bias = -r(C, N).exp(), r(C), r(C)
    w, pool, slots = r(C, 4), r(6, 3, C).to(BF), i32([5, 0, 2, 3])
    states = r(6, C, N)
    yield "short_conv", ssm.short_conv, (x, w, cu), dict(bias=bias, state_in=pool, slots=slots)
    yield "short_conv", ssm.short_conv, (x, w), dict(act="none")
    yield "scan", ssm.scan, (x, dt, a, bc[:, 0], bc[:, 1], cu), dict(d=skip, z=z, dt_bias=bias, state_in=states, slots=slots, max_len=17)
    yield "scan", ssm.scan, (x, dt, a, bc[:, 0], bc[:, 1]), dict(dt_softplus=False, out_dtype=torch.float32)
    m, up = linear.quantize(r(40, 256), group=64), linear.quantize(r(40, 256), group=64)
    sym = linear.quantize(r(40, 256), group=64, offsets=False)
    wide = r(33, 512).to(BF)
    for rows in (1, 2, 5, 33):
        yield "q4_linear", linear.q4_linear, (wide[:rows, :256], m), {}
        yield "q4_linear", linear.q4_linear, (wide[:rows, 256:].contiguous().view(1, rows, 256), sym), dict(out_dtype=torch.float32)
        yield "q4_gated", linear.q4_gated, (wide[:rows, :256], m, up), dict(act="gelu")


def same(a, b):
    """Equal element for element.  A NaN equals a NaN: without the softplus a step may be negative, and where exp(dt a) leaves fp32's
    range a state of zero makes inf * 0."""
    return a.dtype == b.dtype and a.shape == b.shape and torch.allclose(a, b, rtol=0, atol=0, equal_nan=True)


@pytest.mark.gpu
def test_gives_what_the_modules_give(fast):
    """The same bits with the stream left out, which goes the short way, and named, which does not; into memory that is given too."""
    here = torch.cuda.current_stream()
    for name, fn, args, kw in calls():
        want = fn(*args, **kw, stream=here)
        got = fn(*args, **kw)
        assert same(got, want), name
        out = torch.full_like(want, 3.0)
        back = fn(*args, **{k: v for k, v in kw.items() if k != "out_dtype"}, out=out)
        assert back.data_ptr() == out.data_ptr() and same(out, want), name


@pytest.mark.gpu
def test_takes_the_short_way(fast, monkeypatch):
    """Calls in which nothing is unusual do not reach the modules' own code."""
    made = list(calls())
    for module in (ssm, linear):
        monkeypatch.setattr(module, "load_library", lambda: pytest.fail("the long way"))
    for _, fn, args, kw in made:
        fn(*args, **kw)


@pytest.mark.gpu
def test_runs_on_the_current_stream(fast):
    """On another current stream the call and its memory belong to that stream: work that is queued there before it is seen."""
    made = list(calls(3))
    want = [fn(*args, **kw) for _, fn, args, kw in made]
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        for (name, fn, args, kw), expected in zip(made, want):
            first = args[0].clone()
            late = torch.zeros(64, 1 << 20, device="cuda").sum()            # keeps the stream busy
            fresh = torch.empty_like(first)
            fresh.copy_(first + 0 * late.to(BF))
            got = fn(fresh, *args[1:], **kw)
            other.synchronize()
            assert same(got, expected), name


@pytest.mark.gpu
def test_states_and_captured_calls(fast):
    """States in place, by the short way inside a captured graph."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w = torch.randn(5, 64, generator=g, device="cuda").to(BF), torch.randn(64, 4, generator=g, device="cuda")
    past = torch.randn(5, 3, 64, generator=g, device="cuda").to(BF)
    a, b = past.clone(), past.clone()
    want = [ssm.short_conv(x, w, state_in=a, state_out=a, stream=torch.cuda.current_stream()) for _ in range(2)][1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssm.short_conv(x, w, state_in=b, state_out=b)
    graph.replay()
    graph.replay()
    assert torch.equal(got, want) and torch.equal(a, b)


@pytest.mark.gpu
def test_what_is_wrong_is_said(fast):
    """A wrong call is refused in the modules' words, and nothing is written."""
    x, w = torch.zeros(4, 64, dtype=BF, device="cuda"), torch.zeros(64, 4, device="cuda")
    out = torch.full_like(x, 3.0)
    m = linear.quantize(torch.randn(40, 256, device="cuda"), group=64)
    y = torch.zeros(2, 256, dtype=BF, device="cuda")
    for call in (lambda: ssm.short_conv(x.float(), w, out=out), lambda: ssm.short_conv(x, w.half(), out=out),
                 lambda: ssm.short_conv(x, w[:, ::2], out=out), lambda: ssm.short_conv(x.cpu(), w, out=out),
                 lambda: ssm.short_conv(x, w, out=out[:, :32]), lambda: ssm.short_conv(x, w, i32([0, 4]).long(), out=out),
                 lambda: linear.q4_linear(y, m._replace(codes=m.codes[:, ::2])), lambda: linear.q4_linear(y.half(), m),
                 lambda: linear.q4_linear(y, m, out_dtype=torch.float16), lambda: linear.q4_gated(y, m, m, out=y)):
        with pytest.raises((ValueError, gdn.GdnError)):
            call()
    with pytest.raises((ValueError, KeyError, gdn.GdnError)):
        ssm.short_conv(x, w, act="tanh", out=out)
    assert (out == 3).all()
