"""The cases that the recurrent layer's other operators are measured on, and their plain forms.

Four calls stand behind the cases, those that a token meets between the norm and the residual sum besides the
recurrence and attention:

  ssm.short_conv    the short causal convolution in front of a recurrence, per channel, with its activation; the last
                    inputs of every sequence are its state
  ssm.scan          the selective state space scan: a diagonal recurrence whose step width, input and output vectors
                    come from the token, with its skip and gate
  linear.q4_linear  a projection by weights of 4 bits with a scale (and an offset) for each group of inputs
  linear.q4_gated   the first half of a gated feed-forward block by two such matrices: act(x gate) * (x up)

``run`` computes the plain form in 32-bit torch operations, or, with ``own`` set, calls the package.

Sizes: the hybrid model's linear layers (16 query/key and 32 value heads of 128: 8192 convolved channels, 12352
outputs of the input projection with its gates) and generic ones; from one token to tens of thousands.
"""
import math

import torch

own = False


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one generated token through the convolution of q, k and v of one linear layer: latency
        dict(name="conv_1_token", op="conv", n=1, lens="1", channels=8192, width=4, act="silu", bias=False, past=True),
        # the same layer for packed prompts that go on after earlier pieces
        dict(name="conv_prompts", op="conv", n=5, lens="log 300 9000", channels=8192, width=4, act="silu", bias=True, past=True),
        # one generated token of one conversation
        dict(name="scan_1_token", op="scan", n=1, lens="1", channels=4096, states=16, groups=1, gate=True, skip=True, past=True),
        # one token each for a batch of conversations: every state is read and written
        dict(name="scan_batch", op="scan", n=61, lens="1", channels=4096, states=16, groups=1, gate=True, skip=True, past=True),
        # a whole prompt
        dict(name="scan_prompt", op="scan", n=1, lens="8192", channels=4096, states=16, groups=1, gate=True, skip=True, past=False),
        # packed prompts of odd lengths, larger states, several groups of channels with their own vectors
        dict(name="scan_ragged", op="scan", n=7, lens="log 60 4000", channels=1536, states=64, groups=4, gate=True, skip=True, past=True),
        # a long document through a narrow layer: few channels, many steps
        dict(name="scan_long", op="scan", n=1, lens="40000", channels=1024, states=16, groups=1, gate=False, skip=True, past=False),
        # the input projection of a linear layer, one token
        dict(name="matvec_1_token", op="linear", rows=1, n_out=12352, k=2048, group=64, offsets=True, out="bf16"),
        # scores over a vocabulary, one token
        dict(name="matvec_vocabulary", op="linear", rows=1, n_out=131071, k=2048, group=64, offsets=True, out="f32"),
        # one token each for a batch of conversations
        dict(name="matvec_batch", op="linear", rows=33, n_out=4096, k=4096, group=128, offsets=False, out="bf16"),
        # the feed-forward block of one token
        dict(name="gated_1_token", op="gated", rows=1, n_out=5632, k=2048, group=64, offsets=True, act="silu"),
        # the feed-forward block of a piece of a prompt
        dict(name="gated_piece", op="gated", rows=509, n_out=6000, k=2048, group=64, offsets=True, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "linear", "linear", "gated"])
    if op in ("linear", "gated"):
        group = rng.choice([64, 128])
        k = group * _log_int(rng, 4, 8192 // group)
        rows = _log_int(rng, 1, 512)
        n_out = _log_int(rng, 100, max(200, min(40_000, 12_000_000_000 // (rows * k * (2 if op == "gated" else 1)))))
        c = dict(op=op, rows=rows, n_out=n_out, k=k, group=group, offsets=rng.random() < 0.6)
        if op == "gated":
            return dict(c, act=rng.choice(["silu", "gelu"]))
        return dict(c, out=rng.choice(["bf16", "bf16", "f32"]))
    tokens = rng.random() < 0.4
    if op == "conv":
        channels = 8 * _log_int(rng, 32, 1536)
        n = _log_int(rng, 1, 128) if tokens else rng.randint(1, 12)
        longest = 100_000_000 // (channels * n)
        return dict(op="conv", n=n, lens="1" if tokens else "log 1 %d" % max(2, min(30_000, longest)), channels=channels,
                    width=rng.choice([2, 3, 4, 4]), act=rng.choice(["silu", "silu", "none"]), bias=rng.random() < 0.5,
                    past=rng.random() < 0.7)
    states = rng.choice([16, 16, 32, 64, 128])
    groups = rng.choice([1, 1, 2, 4])
    channels = 8 * groups * _log_int(rng, 16, 512 // groups)
    n = _log_int(rng, 1, 128) if tokens else rng.randint(1, 8)
    longest = 500_000_000 // (channels * states * n)
    return dict(op="scan", n=n, lens="1" if tokens else "log 1 %d" % max(2, min(40_000, longest)), channels=channels,
                states=states, groups=groups, gate=rng.random() < 0.7, skip=rng.random() < 0.8, past=rng.random() < 0.7)


def _lengths(case):
    """'40': 40 for every sequence; 'log a b': spread over [a, b], evenly over the logarithm, in a mixed order, odd and even."""
    text, n = case["lens"], case["n"]
    if not text.startswith("log"):
        return [int(text)] * n
    _, lo, hi = text.split()
    lo, hi = float(lo), float(hi)
    at = [((i * 7 + 3) % n + 0.5) / n if n % 7 else (i + 0.5) / n for i in range(n)]
    return [max(1, int(lo * (hi / lo) ** x)) for x in at]


def work(case):
    if case["op"] in ("linear", "gated"):
        m, n, k, two = case["rows"], case["n_out"], case["k"], 2 if case["op"] == "gated" else 1
        weights = two * n * (k // 2 + k // case["group"] * (4 if case["offsets"] else 2))
        out = 4 if case.get("out") == "f32" else 2
        return {"bytes": weights + 2 * m * k + out * m * n, "flops": 2.0 * two * m * n * k}
    n, C, T = case["n"], case["channels"], sum(_lengths(case))
    if case["op"] == "conv":
        state = n * (case["width"] - 1) * C * 2
        return {"bytes": 4 * T * C + state * (2 if case["past"] else 1) + C * 4 * (case["width"] + case["bias"]),
                "flops": 2.0 * T * C * case["width"]}
    N, G = case["states"], case["groups"]
    state = n * C * N * 4
    per = 2 * C * (3 + case["gate"]) + 4 * G * N
    return {"bytes": T * per + state * (2 if case["past"] else 1) + 4 * C * N, "flops": T * C * (7.0 * N + 10)}


# ---------------------------------------------------------------------------------------------------- inputs
def _quantised(g, n_out, k, group, offsets):
    """A random matrix in 4 bits: codes [n_out, k / 2], the even input in the low half, and scales (and offsets) [n_out, k / group]."""
    bf = torch.bfloat16
    w = torch.randn(n_out, k // group, group, generator=g, device="cuda") * k ** -0.5
    if offsets:
        lo, hi = w.amin(dim=-1), w.amax(dim=-1)
        scale, offset = ((hi - lo) / 15).to(bf), lo.to(bf)
        code = (w - offset.float()[..., None]) / scale.float()[..., None]
    else:
        scale, offset = (w.abs().amax(dim=-1) / 7.5).to(bf), None
        code = w / scale.float()[..., None] + 8
    code = code.round_().clamp_(0, 15).to(torch.uint8).view(n_out, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale, offset


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    bf = torch.bfloat16

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] in ("linear", "gated"):
        m, n, k = case["rows"], case["n_out"], case["k"]
        # activations after a norm: a few inputs much larger than the rest
        x = rand(m, k) * torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 20.0, 1.0)
        names = ("w",) if case["op"] == "linear" else ("gate", "up")
        return dict(case=case, x=x.to(bf), **{name: _quantised(g, n, k, case["group"], case["offsets"]) for name in names})
    n, C, lens = case["n"], case["channels"], _lengths(case)
    T = sum(lens)
    cu = [0]
    for m in lens:
        cu.append(cu[-1] + m)
    s = dict(case=case, T=T, longest=max(lens), cu=torch.tensor(cu, dtype=torch.int32, device="cuda"), x=rand(T, C).to(bf))
    if case["op"] == "conv":
        s["weight"] = rand(C, case["width"]) * case["width"] ** -0.5
        s["bias"] = 0.1 * rand(C) if case["bias"] else None
        s["past"] = rand(n, case["width"] - 1, C).to(bf) if case["past"] else None
        s["state"] = torch.zeros(n, case["width"] - 1, C, dtype=bf, device="cuda")
        return s
    N, G = case["states"], case["groups"]
    # step widths between 0.001 and 0.1 when the token adds nothing, decays of 1 .. N
    width = torch.exp(math.log(1e-3) + math.log(100.0) * torch.rand(C, generator=g, device="cuda"))
    s["dt_bias"] = width + torch.log(-torch.expm1(-width))
    s["dt"] = rand(T, C).to(bf)
    s["a"] = (-torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(0.1 * rand(C, N))).contiguous()
    bc = rand(T, 2, G, N).to(bf)                       # both come out of one projection
    s["b"], s["c"] = bc[:, 0], bc[:, 1]
    s["d"] = 1 + 0.1 * rand(C) if case["skip"] else None
    s["z"] = rand(T, C).to(bf) if case["gate"] else None
    s["past"] = 0.3 * rand(n, C, N) if case["past"] else None
    s["state"] = torch.zeros(n, C, N, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if op == "conv":
        return _conv_own(state) if own else _conv_plain(state)
    if op == "scan":
        return _scan_own(state) if own else _scan_plain(state)
    if op == "linear":
        return _linear_own(state) if own else _linear_plain(state)
    return _gated_own(state) if own else _gated_plain(state)


def _conv_own(s):
    from gated_deltanet_linear_03_gb300 import ssm
    c = s["case"]
    out = ssm.short_conv(s["x"], s["weight"], None if c["lens"] == "1" else s["cu"], bias=s["bias"], act=c["act"],
                         state_in=s["past"], state_out=s["state"])
    return dict(out=out, state=s["state"])


def _scan_own(s):
    from gated_deltanet_linear_03_gb300 import ssm
    c = s["case"]
    out = ssm.scan(s["x"], s["dt"], s["a"], s["b"], s["c"], None if c["lens"] == "1" else s["cu"], d=s["d"], z=s["z"],
                   dt_bias=s["dt_bias"], state_in=s["past"], state_out=s["state"], max_len=s["longest"])
    return dict(out=out, state=s["state"])


def _linear_own(s):
    from gated_deltanet_linear_03_gb300 import linear
    return linear.q4_linear(s["x"], linear.Q4(*s["w"]), out_dtype=torch.float32 if s["case"]["out"] == "f32" else torch.bfloat16)


def _gated_own(s):
    from gated_deltanet_linear_03_gb300 import linear
    return linear.q4_gated(s["x"], linear.Q4(*s["gate"]), linear.Q4(*s["up"]), act=s["case"]["act"])


def _places(s):
    """Of every token: its sequence, and its place there."""
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(s["case"]["n"], device="cuda"), cu[1:] - cu[:-1], output_size=s["T"])
    return seq, torch.arange(s["T"], device="cuda") - cu[seq]


def _conv_plain(s):
    c, T, cu = s["case"], s["T"], s["cu"].long()
    n, w, C = c["n"], c["width"], c["channels"]
    seq, at = _places(s)
    past = s["past"].float() if c["past"] else torch.zeros(n, w - 1, C, device="cuda")
    x = s["x"].float()
    y = x * s["weight"][:, w - 1]
    for back in range(1, w):
        inside = at >= back
        before = torch.where(inside[:, None], x[(torch.arange(T, device="cuda") - back).clamp_min(0)],
                             past[seq, (w - 1 - back + at).clamp(0, w - 2)])
        y = y + before * s["weight"][:, w - 1 - back]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    # the last w - 1 inputs of every sequence, those from before its first token among them
    back = torch.arange(w - 1, 0, -1, device="cuda")
    place = (cu[1:] - cu[:-1])[:, None] - back
    state = torch.where((place >= 0)[..., None], x[(cu[:-1, None] + place).clamp(0, T - 1)],
                        past[torch.arange(n, device="cuda")[:, None], (place + w - 1).clamp(0, w - 2)])
    return dict(out=y.to(torch.bfloat16), state=state.to(torch.bfloat16))


def _scan_plain(s):
    c, T, cu = s["case"], s["T"], s["cu"].long()
    C, N, G = c["channels"], c["states"], c["groups"]
    v = s["dt"].float() + s["dt_bias"]
    step = v.clamp_min(0) + torch.log1p(torch.exp(-v.abs()))
    x = s["x"].float()
    b, cc = (t.float()[:, :, None].expand(T, G, C // G, N).reshape(T, C, N) for t in (s["b"], s["c"]))
    decay = torch.exp(step[..., None] * s["a"])
    h = (step * x)[..., None] * b
    if c["past"]:
        h[cu[:-1]] += decay[cu[:-1]] * s["past"]
    if s["longest"] > 1:
        # h_t = decay_t h_{t-1} + h_t by doubling: after each round an entry stands for twice as many tokens; a sequence's
        # first token keeps nothing of what is before it
        decay[cu[:-1]] = 0
        reach = 1
        while reach < s["longest"]:
            h[reach:] += decay[reach:] * h[:-reach].clone()
            decay[reach:] *= decay[:-reach].clone()
            reach *= 2
    y = (h * cc).sum(dim=-1)
    if s["d"] is not None:
        y = y + s["d"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z / (1 + torch.exp(-z))
    return dict(out=y.to(torch.bfloat16), state=h[cu[1:] - 1])


def _values(w, group):
    """The matrix [n_out, k] that codes, scales and offsets stand for, in 32 bits."""
    codes, scale, offset = w
    q = torch.stack([codes & 15, codes >> 4], dim=-1).view(codes.shape[0], -1, group).float()
    if offset is None:
        return ((q - 8) * scale.float()[..., None]).flatten(1)
    return (q * scale.float()[..., None] + offset.float()[..., None]).flatten(1)


def _linear_plain(s):
    y = torch.matmul(s["x"].float(), _values(s["w"], s["case"]["group"]).T)
    return y if s["case"]["out"] == "f32" else y.to(torch.bfloat16)


def _gated_plain(s):
    group = s["case"]["group"]
    a = torch.matmul(s["x"].float(), _values(s["gate"], group).T)
    b = torch.matmul(s["x"].float(), _values(s["up"], group).T)
    if s["case"]["act"] == "silu":
        a = a / (1 + torch.exp(-a))
    else:
        a = 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    return (a * b).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _conv_exact, "scan": _scan_exact, "linear": _linear_exact, "gated": _gated_exact}[case["op"]](s)


def _conv_exact(s):
    c, outs, states = s["case"], [], []
    w = c["width"]
    for i, m in enumerate(_lengths(c)):
        lo = int(s["cu"][i])
        before = s["past"][i].double() if c["past"] else torch.zeros(w - 1, c["channels"], dtype=torch.float64, device="cuda")
        line = torch.cat([before, s["x"][lo:lo + m].double()])
        y = torch.einsum("tcw,cw->tc", line.unfold(0, w, 1), s["weight"].double())
        if s["bias"] is not None:
            y += s["bias"].double()
        outs.append(y * torch.sigmoid(y) if c["act"] == "silu" else y)
        states.append(line[m:])
    return dict(out=torch.cat(outs), state=torch.stack(states))


def _scan_exact(s):
    c = s["case"]
    C, N, G = c["channels"], c["states"], c["groups"]
    f64 = torch.float64
    a, lens, cu = s["a"].double(), _lengths(c), s["cu"].tolist()
    h = s["past"].double().clone() if c["past"] else torch.zeros(c["n"], C, N, dtype=f64, device="cuda")
    out = torch.empty(s["T"], C, dtype=f64, device="cuda")
    # token by token, all sequences that are still running at once, the longest first
    order = sorted(range(c["n"]), key=lambda i: -lens[i])
    start = torch.tensor([cu[i] for i in order], device="cuda")
    h = h[torch.tensor(order, device="cuda")]
    for t in range(max(lens)):
        live = sum(lens[i] > t for i in order)
        row = start[:live] + t
        step = torch.nn.functional.softplus(s["dt"][row].double() + s["dt_bias"].double(), threshold=1e9)
        x = s["x"][row].double()
        b, cc = (m[row].double().repeat_interleave(C // G, dim=1) for m in (s["b"], s["c"]))
        h[:live] = torch.exp(step[..., None] * a) * h[:live] + (step * x)[..., None] * b
        out[row] = torch.einsum("icn,icn->ic", h[:live], cc)
    if s["d"] is not None:
        out += s["d"].double() * s["x"].double()
    if s["z"] is not None:
        z = s["z"].double()
        out *= z * torch.sigmoid(z)
    state = torch.empty_like(h)
    state[torch.tensor(order, device="cuda")] = h
    return dict(out=out, state=state)


def _product(x, w, group):
    """x [m, k] by a quantised matrix: the codes' products group by group, then scales and offsets."""
    codes, scale, offset = w
    m, k = x.shape
    x = x.double().view(m, k // group, group)
    y = torch.empty(m, codes.shape[0], dtype=torch.float64, device="cuda")
    for lo in range(0, codes.shape[0], 8192):
        part = codes[lo:lo + 8192].to(torch.int64)
        q = torch.empty(part.shape[0], k, dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = part % 16, part // 16
        q = q.view(-1, k // group, group)
        q = (q if offset is not None else q - 8) * scale[lo:lo + 8192].double()[..., None]
        y[:, lo:lo + 8192] = x.flatten(1) @ q.flatten(1).T
        if offset is not None:
            y[:, lo:lo + 8192] += x.sum(dim=-1) @ offset[lo:lo + 8192].double().T
    return y


def _linear_exact(s):
    return _product(s["x"], s["w"], s["case"]["group"])


def _gated_exact(s):
    a, b = (_product(s["x"], s[name], s["case"]["group"]) for name in ("gate", "up"))
    if s["case"]["act"] == "silu":
        return a * torch.sigmoid(a) * b
    return torch.nn.functional.gelu(a, approximate="tanh") * b
