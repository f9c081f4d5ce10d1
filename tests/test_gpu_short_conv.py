"""gdn_short_conv against the plain 64-bit form: prompts, single tokens, pieces, states."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    from gated_deltanet_linear_03_gb300 import ssm as s
    return s


def inputs(lens, channels, width, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(x=r(sum(lens), channels).to(BF), weight=r(channels, width), bias=r(channels),
                past=r(len(lens), width - 1, channels).to(BF))


def cu_of(lens):
    at = [0]
    for m in lens:
        at.append(at[-1] + m)
    return i32(at)


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [2], [3], [5], [16], [17], [1, 1, 1], [0, 4, 0, 0, 33, 1], [2, 0, 15, 100]])
@pytest.mark.parametrize("channels", [8, 1016, 1032])
def test_sizes(ssm, width, lens, channels):
    i = inputs(lens, channels, width, seed=width)
    state = torch.full_like(i["past"], 7.0)
    out = ssm.short_conv(i["x"], i["weight"], cu_of(lens), bias=i["bias"], state_in=i["past"], state_out=state)
    y, e, s = ref.conv(i["x"], i["weight"], lens, i["bias"], "silu", i["past"])
    ref.check(out, y, e)
    assert torch.equal(state.double(), s)


@pytest.mark.parametrize("lens", [[700, 1, 3000, 0, 25, 900], [20000]])
def test_many_tokens(ssm, lens):
    """Tiles of several tokens, cut wherever the sequences begin."""
    channels = 2048
    i = inputs(lens, channels, 4, seed=5)
    state = torch.full_like(i["past"], 7.0)
    out = ssm.short_conv(i["x"], i["weight"], cu_of(lens), bias=i["bias"], state_in=i["past"], state_out=state)
    y, e, s = ref.conv(i["x"], i["weight"], lens, i["bias"], "silu", i["past"])
    ref.check(out, y, e)
    assert torch.equal(state.double(), s)


@pytest.mark.parametrize("n,channels", [(1, 64), (37, 520), (700, 8192)])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_one_token_each(ssm, n, channels, act):
    i = inputs([1] * n, channels, 4, seed=n)
    want = ref.conv(i["x"], i["weight"], [1] * n, None, act, i["past"])
    by_cu = ssm.short_conv(i["x"], i["weight"], cu_of([1] * n), act=act, state_in=i["past"])
    state = i["past"].clone()
    out = ssm.short_conv(i["x"], i["weight"], act=act, state_in=state, state_out=state)      # in place
    ref.check(out, want[0], want[1])
    assert torch.equal(out, by_cu) and torch.equal(state.double(), want[2])


@pytest.mark.parametrize("lens", [[1, 2, 3, 40, 0], [3000, 1, 5000, 0, 200]])
def test_in_place_beginnings_and_pieces(ssm, lens):
    """States updated in place, kept apart, or not given; and a prompt in pieces gives what it gives in one."""
    i = inputs(lens, 1024, 4, seed=2)
    cu = cu_of(lens)
    apart = torch.empty_like(i["past"])
    want = ssm.short_conv(i["x"], i["weight"], cu, state_in=i["past"], state_out=apart)
    state = i["past"].clone()
    assert torch.equal(ssm.short_conv(i["x"], i["weight"], cu, state_in=state, state_out=state), want)
    assert torch.equal(state, apart)
    fresh = torch.full_like(apart, 7.0)
    begin = ssm.short_conv(i["x"], i["weight"], cu, state_out=fresh)
    zero = torch.zeros_like(apart)
    kept = torch.empty_like(apart)
    assert torch.equal(begin, ssm.short_conv(i["x"], i["weight"], cu, state_in=zero, state_out=kept))
    assert torch.equal(fresh, kept)
    assert torch.equal(ssm.short_conv(i["x"], i["weight"], cu), begin)
    # every sequence in two pieces
    first = [m // 3 for m in lens]
    at = cu.tolist()
    rows = [torch.cat([torch.arange(at[k], at[k] + f) for k, f in enumerate(first)]),
            torch.cat([torch.arange(at[k] + f, at[k + 1]) for k, f in enumerate(first)])]
    state = i["past"].clone()
    out = torch.empty_like(want)
    for r, part in zip(rows, (first, [m - f for m, f in zip(lens, first)])):
        r = r.cuda()
        out[r] = ssm.short_conv(i["x"][r], i["weight"], cu_of(part), state_in=state, state_out=state)
    assert torch.equal(out, want) and torch.equal(state, apart)


@pytest.mark.parametrize("width", [2, 3, 4])
@pytest.mark.parametrize("longest,channels", [(6, 1024), (40, 4096), (300, 8192)])
def test_in_place_wherever_sequences_begin(ssm, width, longest, channels):
    """Many sequences, so that they begin at every distance from where the work is cut: a state that is overwritten must have been
    read by all who need it."""
    gen = torch.Generator().manual_seed(width)
    lens = torch.randint(0, longest, (4000 if longest < 300 else 150,), generator=gen).tolist()
    i = inputs(lens, channels, width, seed=longest)
    cu = cu_of(lens)
    y, e, s = ref.conv(i["x"][:, :64].contiguous(), i["weight"][:64], lens, None, "silu", i["past"][:, :, :64])
    for _ in range(4):
        state = i["past"].clone()
        out = ssm.short_conv(i["x"], i["weight"], cu, state_in=state, state_out=state)
        ref.check(out[:, :64], y, e)
        assert torch.equal(state[:, :, :64].double(), s)


def test_slices_slots_and_untouched_rows(ssm):
    """x as a slice of a projection, states in slots of a larger pool, rows that no sequence holds."""
    lens, C = [30, 1, 7], 256
    g = torch.Generator(device="cuda").manual_seed(3)
    proj = torch.randn(50, 3 * C, generator=g, device="cuda").to(BF)
    x = proj[:, C:2 * C]
    w = torch.randn(C, 4, generator=g, device="cuda")
    pool = torch.randn(9, 3, C, generator=g, device="cuda").to(BF)
    slots = [5, 0, 8]
    out = torch.full((50, C), 3.0, dtype=BF, device="cuda")
    new = torch.full_like(pool, 4.0)
    cu = i32([4, 34, 35, 42])                 # rows 0 .. 3 and 42 .. 49 belong to nobody
    ssm.short_conv(x, w, cu, state_in=pool, state_out=new, slots=i32(slots), out=out)
    y, e, s = ref.conv(x[4:42], w, lens, None, "silu", pool[slots])
    ref.check(out[4:42], y, e)
    assert (out[:4] == 3).all() and (out[42:] == 3).all()
    assert torch.equal(new[slots].double(), s)
    rest = [k for k in range(9) if k not in slots]
    assert (new[rest] == 4).all()


@pytest.mark.parametrize("lens", [[30, 5, 9], [4000, 3000, 5000], [3, 0, 2]])
def test_a_slot_outside_the_pool(ssm, lens):
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    i = inputs(lens, 1024, 4, seed=4)
    out, new = torch.full_like(i["x"], 3.0), torch.full_like(i["past"], 4.0)
    ssm.short_conv(i["x"], i["weight"], cu_of(lens), state_in=i["past"], state_out=new, slots=i32([0, 3, 2]), out=out)
    assert gdn.device_error() == 6
    y, e, s = ref.conv(i["x"], i["weight"], lens, None, "silu", i["past"])
    a, b = lens[0], lens[0] + lens[1]
    ref.check(out[:a], y[:a], e[:a])
    ref.check(out[b:], y[b:], e[b:])
    assert (out[a:b] == 3).all() and (new[1] == 4).all()
    assert torch.equal(new[[0, 2]].double(), s[[0, 2]])


def test_not_finite_inputs_stay_with_their_channel_and_taps(ssm):
    i = inputs([40], 16, 4, seed=6)
    i["x"][10, 3], i["x"][20, 5] = float("inf"), float("nan")
    out = ssm.short_conv(i["x"], i["weight"], cu_of([40]), act="none")
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[10:14, 3], want[20:24, 5] = True, True
    assert torch.equal(bad, want)


def test_no_sequences_and_no_tokens(ssm):
    w = torch.randn(64, 4, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    assert ssm.short_conv(x, w).shape == (0, 64)
    past, new = torch.randn(3, 3, 64, device="cuda").to(BF), torch.zeros(3, 3, 64, dtype=BF, device="cuda")
    assert ssm.short_conv(x, w, i32([0, 0, 0, 0]), state_in=past, state_out=new).shape == (0, 64)
    assert torch.equal(past, new)


def test_beyond_32_bit_offsets(ssm):
    """300000 tokens of 8192 channels: 2.5e9 elements; the last rows, and those around 2^31 elements."""
    T, C = 300_000, 8192
    x = torch.zeros(T, C, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(8)
    w = torch.randn(C, 4, generator=g, device="cuda")
    spots = [(2 ** 31 // C - 40, 80), (T - 64, 64)]
    for at, m in spots:
        x[at:at + m] = torch.randn(m, C, generator=g, device="cuda").to(BF)
    state = torch.empty(1, 3, C, dtype=BF, device="cuda")
    out = ssm.short_conv(x, w, i32([0, T]), state_out=state)
    for at, m in spots:
        y, e, _ = ref.conv(x[at - 3:at + m], w, [m + 3], None, "silu", None)
        ref.check(out[at:at + m], y[3:], e[3:])
    assert torch.equal(state[0], x[-3:])


def test_streams_and_graphs(ssm):
    """On another stream, and captured: a replay sees the buffers' present contents and goes on from the state."""
    i = inputs([1] * 6, 512, 4, seed=9)
    state, x, out = i["past"].clone(), i["x"].clone(), torch.empty_like(i["x"])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    ssm.short_conv(x, i["weight"], state_in=i["past"], out=out, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    want = ref.conv(x, i["weight"], [1] * 6, None, "silu", i["past"])
    ref.check(out, want[0], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.short_conv(x, i["weight"], state_in=state, state_out=state, out=out)
    past = state.clone()
    for step in range(3):
        x.copy_(torch.randn(6, 512, device="cuda").to(BF))
        graph.replay()
        y, e, s = ref.conv(x, i["weight"], [1] * 6, None, "silu", past)
        ref.check(out, y, e)
        assert torch.equal(state.double(), s)
        past = state.clone()
