"""gdn_ssm_scan against the plain 64-bit form: prompts in one piece and in several, single tokens, states."""
import pytest
import torch

import layer_helpers as ref
from layer_helpers import BF, F32, i32

pytestmark = pytest.mark.gpu
JOINED = 4096          # no piece of a scan is longer


@pytest.fixture(scope="module")
def ssm():
    from gated_deltanet_linear_03_gb300 import ssm as s
    return s


def inputs(lens, channels, n_state, groups=1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    T = sum(lens)
    return dict(x=r(T, channels).to(BF), dt=r(T, channels).to(BF), z=(2 * r(T, channels)).to(BF), b=r(T, groups, n_state).to(BF),
                c=r(T, groups, n_state).to(BF), a=-torch.exp(1.5 * r(channels, n_state)), d=r(channels), bias=-3 + 1.5 * r(channels),
                past=r(len(lens), channels, n_state))


def cu_of(lens):
    at = [0]
    for m in lens:
        at.append(at[-1] + m)
    return i32(at)


def both(ssm, i, lens, cu="given", max_len=None, out_dtype=F32, past=True, **kw):
    state = torch.full_like(i["past"], 7.0)
    out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens) if cu else None, d=i["d"], z=i["z"], dt_bias=i["bias"],
                   state_in=i["past"] if past else None, state_out=state, max_len=max(lens) if max_len is None else max_len,
                   out_dtype=out_dtype, **kw)
    y, e, h, he = ref.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], lens, i["d"], i["z"], i["bias"],
                           past=i["past"] if past else None, joined=JOINED if max(lens) > 512 else 0)
    ref.check(out, y, e)
    ref.check(state, h, he)
    return out, state


@pytest.mark.parametrize("n_state", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,channels,groups", [([1], 8, 1), ([2], 16, 2), ([31, 1, 0, 33], 40, 1), ([64], 48, 3), ([5, 0, 200], 136, 1)])
def test_sizes(ssm, n_state, lens, channels, groups):
    both(ssm, inputs(lens, channels, n_state, groups, seed=n_state), lens)


@pytest.mark.parametrize("n_state,channels,lens", [(16, 64, [3000]), (16, 1024, [1500, 1, 700, 0, 2500]), (32, 40, [1, 1999, 3, 600]),
                                                   (64, 96, [2600]), (128, 24, [513, 40, 1300])])
@pytest.mark.parametrize("past", [False, True])
def test_long_sequences(ssm, n_state, channels, lens, past):
    """Few channels and many tokens: in pieces that are joined, wherever the sequences begin in them."""
    both(ssm, inputs(lens, channels, n_state, seed=len(lens)), lens, past=past)


@pytest.mark.parametrize("n,channels,groups", [(1, 8, 1), (1, 4096, 1), (37, 264, 3), (130, 1024, 2)])
@pytest.mark.parametrize("n_state", [16, 64, 128])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_one_token_each(ssm, n, channels, groups, n_state, out_dtype):
    i = inputs([1] * n, channels, n_state, groups, seed=n)
    out, state = both(ssm, i, [1] * n, cu=None, out_dtype=out_dtype)
    again, kept = both(ssm, i, [1] * n, out_dtype=out_dtype)
    assert torch.equal(out, again) and torch.equal(state, kept)


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("bias,softplus", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("lens", [[70, 3], [1, 1], [900, 40]])
def test_options(ssm, skip, gate, bias, softplus, lens):
    i = inputs(lens, 72, 16, seed=3)
    if not softplus:                 # the widths themselves: positive
        i["dt"], i["bias"] = (0.05 * i["dt"].float().abs()).to(BF), i["bias"].abs() * 0.01
    kw = dict(d=i["d"] if skip else None, z=i["z"] if gate else None, dt_bias=i["bias"] if bias else None)
    state = torch.empty_like(i["past"])
    out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), dt_softplus=softplus, state_in=i["past"], state_out=state,
                   max_len=max(lens), **kw)
    y, e, h, he = ref.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], lens, kw["d"], kw["z"], kw["dt_bias"], softplus, i["past"],
                           joined=JOINED if max(lens) > 512 else 0)
    ref.check(out, y, e)
    ref.check(state, h, he)


@pytest.mark.parametrize("lens", [[3, 70, 0, 40], [1800, 3, 900, 0]])
@pytest.mark.parametrize("max_len", [0, 1, 50, 10 ** 6])
def test_whatever_the_host_says_of_the_lengths(ssm, lens, max_len):
    both(ssm, inputs(lens, 48, 16, seed=7), lens, max_len=max_len)


@pytest.mark.parametrize("lens,channels", [([3, 70, 0, 40], 48), ([2500, 3, 1200, 0], 64)])
def test_in_place_beginnings_and_pieces(ssm, lens, channels):
    i = inputs(lens, channels, 16, seed=8)
    args = (i["x"], i["dt"], i["a"], i["b"], i["c"])
    kw = dict(d=i["d"], z=i["z"], dt_bias=i["bias"], max_len=max(lens), out_dtype=F32)
    apart = torch.empty_like(i["past"])
    want = ssm.scan(*args, cu_of(lens), state_in=i["past"], state_out=apart, **kw)
    state = i["past"].clone()
    assert torch.equal(ssm.scan(*args, cu_of(lens), state_in=state, state_out=state, **kw), want)
    assert torch.equal(state, apart)
    zero = torch.zeros_like(apart)
    begin = ssm.scan(*args, cu_of(lens), state_in=zero, **kw)
    assert torch.equal(ssm.scan(*args, cu_of(lens), **kw), begin)
    # in two pieces: other roundings where pieces are joined elsewhere, so against the plain form
    first = [m // 3 for m in lens]
    at = cu_of(lens).tolist()
    rows = [torch.cat([torch.arange(at[k], at[k] + f) for k, f in enumerate(first)]).cuda(),
            torch.cat([torch.arange(at[k] + f, at[k + 1]) for k, f in enumerate(first)]).cuda()]
    state, out = i["past"].clone(), torch.empty_like(want)
    for r, part in zip(rows, (first, [m - f for m, f in zip(lens, first)])):
        out[r] = ssm.scan(*(i[k][r] if k != "a" else i["a"] for k in ("x", "dt", "a", "b", "c")), cu_of(part), d=i["d"], z=i["z"][r],
                          dt_bias=i["bias"], state_in=state, state_out=state, max_len=max(part), out_dtype=F32)
    y, e, h, he = ref.scan(*args, lens, i["d"], i["z"], i["bias"], past=i["past"], joined=JOINED if max(lens) > 512 else 0)
    ref.check(out, y, e)
    ref.check(state, h, he)


@pytest.mark.parametrize("lens,channels", [([30, 1, 7], 64), ([900, 1, 1100], 32)])
def test_slices_slots_and_untouched_rows(ssm, lens, channels):
    g = torch.Generator(device="cuda").manual_seed(11)
    C, N, T = channels, 16, sum(lens)
    proj = torch.randn(T + 9, 3 * C, generator=g, device="cuda").to(BF)
    x, dt, z = proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:]
    bc = torch.randn(T + 9, 40 + 2 * N, generator=g, device="cuda").to(BF)
    b, c = bc[:, 40:40 + N].unsqueeze(1), bc[:, 40 + N:].unsqueeze(1)
    a = -torch.exp(torch.randn(C, N, generator=g, device="cuda"))
    pool = torch.randn(9, C, N, generator=g, device="cuda")
    slots, new = [5, 0, 8], torch.full((9, C, N), 4.0, device="cuda")
    cu = [4]
    for m in lens:
        cu.append(cu[-1] + m)
    out = torch.full((T + 9, C), 3.0, device="cuda")
    ssm.scan(x, dt, a, b, c, i32(cu), z=z, state_in=pool, state_out=new, slots=i32(slots), max_len=max(lens), out=out)
    rows = slice(4, 4 + T)
    y, e, h, he = ref.scan(x[rows], dt[rows], a, b[rows], c[rows], lens, None, z[rows], None, past=pool[slots],
                           joined=JOINED if max(lens) > 512 else 0)
    ref.check(out[rows], y, e)
    ref.check(new[slots], h, he)
    assert (out[:4] == 3).all() and (out[4 + T:] == 3).all()
    assert (new[[k for k in range(9) if k not in slots]] == 4).all()


@pytest.mark.parametrize("lens", [[30, 5, 9], [2000, 1500, 900], [1, 1, 1], [700, 0, 900]])
def test_a_slot_outside_the_pool(ssm, lens):
    from gated_deltanet_linear_03_gb300 import gdn
    assert gdn.device_error() == 0
    i = inputs(lens, 64, 16, seed=12)
    out, new = torch.full((sum(lens), 64), 3.0, device="cuda"), torch.full_like(i["past"], 4.0)
    ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), state_in=i["past"], state_out=new, slots=i32([0, 3, 2]),
             max_len=max(lens), out=out)
    assert gdn.device_error() == 6
    y, e, h, he = ref.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], lens, past=i["past"], joined=JOINED if max(lens) > 512 else 0)
    p, q = lens[0], lens[0] + lens[1]
    ref.check(out[:p], y[:p], e[:p])
    ref.check(out[q:], y[q:], e[q:])
    ref.check(new[[0, 2]], h[[0, 2]], he[[0, 2]])
    assert (out[p:q] == 3).all() and (new[1] == 4).all()


def test_a_sequence_that_is_not_finite_spoils_no_other(ssm):
    """Sequences next to one another in one CTA's tokens: states are set anew at every beginning."""
    for lens in ([40, 50, 60], [1000, 700, 900]):
        i = inputs(lens, 32, 16, seed=13)
        clean = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), max_len=max(lens))
        i["x"][lens[0] + 7, 3] = float("nan")
        i["x"][lens[0] + 9, 5] = float("inf")
        out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu_of(lens), max_len=max(lens))
        a, b = lens[0], lens[0] + lens[1]
        assert torch.equal(out[:a], clean[:a]) and torch.equal(out[b:], clean[b:])
        keep = [k for k in range(32) if k not in (3, 5)]
        assert torch.equal(out[a:b][:, keep], clean[a:b][:, keep])
        assert torch.isnan(out[a + 7:b, 3]).all() and not torch.isfinite(out[a + 9:b, 5]).any()


@pytest.mark.parametrize("lens", [[100], [1], [1200]])
def test_strong_and_absent_decay(ssm, lens):
    """Widths from almost nothing to tens, a of zero and of -1000: decays of 1 and of 0."""
    i = inputs(lens, 16, 16, seed=14)
    i["a"][:, 0], i["a"][:, 1] = 0.0, -1000.0
    i["bias"][:4], i["bias"][4:8] = -20.0, 30.0
    both(ssm, i, lens)


def test_no_sequences_and_no_tokens(ssm):
    i = inputs([0, 0], 64, 16)
    new = torch.zeros_like(i["past"])
    out = ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], i32([0, 0, 0]), state_in=i["past"], state_out=new)
    assert out.shape == (0, 64) and torch.equal(new, i["past"])
    assert ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"]).shape == (0, 64)


def test_beyond_32_bit_offsets(ssm):
    """600000 tokens of 4096 channels, 2.5e9 elements: with decays that forget within a few tokens, its last rows are
    those of their own last thousand tokens."""
    T, C, last = 600_000, 4096, 700
    g = torch.Generator(device="cuda").manual_seed(15)
    x = torch.empty(T, C, dtype=BF, device="cuda").normal_(generator=g)
    dt = torch.full((1, C), 1.0, dtype=BF, device="cuda").expand(T, C).contiguous()
    b = torch.randn(T, 1, 16, generator=g, device="cuda").to(BF)
    a = torch.full((C, 16), -1.0, device="cuda")
    state = torch.empty(1, C, 16, device="cuda")
    out = ssm.scan(x, dt, a, b, b, i32([0, T]), state_out=state, max_len=T)
    y, e, h, he = ref.scan(x[-last:], dt[-last:], a, b[-last:], b[-last:], [last], joined=JOINED)
    ref.check(out[-50:], y[-50:], e[-50:] + 1e-30)
    ref.check(state, h, he)


def test_streams_graphs_and_two_calls_at_once(ssm):
    lens = [1500, 40, 900]
    i = inputs(lens, 128, 16, seed=16)
    args, cu = (i["x"], i["dt"], i["a"], i["b"], i["c"]), cu_of(lens)
    want = ssm.scan(*args, cu, max_len=max(lens))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(want) for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, o in zip(streams, outs):
            ssm.scan(*args, cu, max_len=max(lens), out=o, stream=s)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
    # two graphs, each with a prompt and a token behind it
    state = [torch.zeros(3, 128, 16, device="cuda") for _ in range(2)]
    tok = inputs([1, 1, 1], 128, 16, seed=17)
    graphs, ys = [], []
    for h in state:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ssm.scan(*args, cu, max_len=max(lens), state_out=h)
            ys.append(ssm.scan(tok["x"], tok["dt"], i["a"], tok["b"], tok["c"], state_in=h, state_out=h))
        graphs.append(graph)
    for graph in (*graphs, *graphs):
        graph.replay()
    h = torch.zeros(3, 128, 16, device="cuda")
    ssm.scan(*args, cu, max_len=max(lens), state_out=h)
    y = ssm.scan(tok["x"], tok["dt"], i["a"], tok["b"], tok["c"], state_in=h, state_out=h)
    for got, kept in zip(ys, state):
        assert torch.equal(got, y) and torch.equal(kept, h)
