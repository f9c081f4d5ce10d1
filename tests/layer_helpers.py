"""64-bit plain forms of the short convolution, the selective scan and the 4-bit products, each with a bound on what 32-bit
arithmetic may be off by.  They run where their inputs are."""
import math

import torch

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def i32(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def conv(x, weight, lens, bias=None, act="silu", past=None):
    """(y, bound, new states) of packed sequences; past: [n, width - 1, channels] or None.

    Bound: a sum of width products and a bias, each rounded once more: (width + 2) 2^-24 < 2^-21 of the sum of magnitudes,
    carried on by an activation whose slope is below 1.1, and an exponential and a quotient (2^-20 of the result)."""
    n, w = len(lens), weight.shape[1]
    ys, es, states, at = [], [], [], 0
    for i in range(n):
        before = past[i].double() if past is not None else torch.zeros(w - 1, x.shape[1], dtype=F64, device=x.device)
        line = torch.cat([before, x[at:at + lens[i]].double()])
        at += lens[i]
        win = line.unfold(0, w, 1)[:lens[i]] if lens[i] else line.new_zeros(0, x.shape[1], w)
        y = (win * weight.double()).sum(-1)
        e = (win * weight.double()).abs().sum(-1)
        if bias is not None:
            y, e = y + bias.double(), e + bias.double().abs()
        if act == "silu":
            y = y * torch.sigmoid(y)
        ys.append(y)
        es.append(1.1 * 2.0 ** -21 * e + 2.0 ** -20 * y.abs())
        states.append(line[lens[i]:])
    return torch.cat(ys), torch.cat(es), torch.stack(states) if n else None


def scan(x, dt, a, b, c, lens, d=None, z=None, dt_bias=None, softplus=True, past=None, joined=0):
    """(y, its bound, new states, their bound).

    Bound.  The step width has a relative error below 2^-21 (an exponential, a logarithm, a sum), the decay e^(D a) of
    2^-21 (1 + |D a|) (its argument's and the exponential's), the new term D x B of 2^-20; they add up as the states do.
    A scan in pieces carries the state over up to `joined` tokens by one exponential of a sum of as many widths,
    rounded as often: at most joined 2^-24 |a S| e^(a S) <= joined 2^-25 of the largest state.  y: a product and a sum
    of n_state terms, 2^-20 of their magnitudes, the skip, and the gate (2^-20)."""
    n, (T, C), N, G = len(lens), x.shape, a.shape[1], b.shape[1]
    a, dev = a.double(), x.device
    h = past.double().clone() if past is not None else torch.zeros(n, C, N, dtype=F64, device=dev)
    big, err, top = h.abs(), torch.zeros_like(h), h.abs()
    y, ye = torch.zeros(T, C, dtype=F64, device=dev), torch.zeros(T, C, dtype=F64, device=dev)
    start, at = [], 0
    for m in lens:
        start.append(at)
        at += m
    for t in range(max(lens, default=0)):
        live = torch.tensor([i for i in range(n) if lens[i] > t], device=dev)
        row = torch.tensor([start[i] + t for i in live.tolist()], device=dev)
        w = dt[row].double() + (dt_bias.double() if dt_bias is not None else 0)
        if softplus:
            w = torch.nn.functional.softplus(w, threshold=1e9)
        xv = x[row].double()
        bv, cv = (m[row].double().repeat_interleave(C // G, dim=1) for m in (b, c))
        arg = w[..., None] * a
        decay, new = torch.exp(arg), (w * xv)[..., None] * bv
        e = decay * err[live] + 2.0 ** -21 * (1 + arg.abs()) * decay * big[live] + 2.0 ** -20 * new.abs()
        h[live] = decay * h[live] + new
        big[live] = decay * big[live] + new.abs()
        err[live] = e
        top[live] = torch.maximum(top[live], big[live])
        e = e + joined * 2.0 ** -25 * top[live]
        v = (h[live] * cv).sum(-1)
        ve = (e * cv.abs()).sum(-1) + 2.0 ** -20 * (big[live] * cv.abs()).sum(-1)
        if d is not None:
            v = v + d.double() * xv
            ve = ve + 2.0 ** -22 * (d.double() * xv).abs()
        if z is not None:
            s = z[row].double() * torch.sigmoid(z[row].double())
            v, ve = v * s, ve * s.abs() * (1 + 2.0 ** -19) + 2.0 ** -20 * (v * s).abs()
        y[row], ye[row] = v, ve + 2.0 ** -23 * v.abs()
    return y, ye, h, err + joined * 2.0 ** -25 * top + 2.0 ** -23 * h.abs()


def q4_values(w):
    codes, scales, offsets = w
    n = codes.shape[0]
    q = torch.stack([codes % 16, codes // 16], dim=-1).view(n, scales.shape[1], -1).double()
    s = scales.double()[..., None]
    return ((q - 8) * s if offsets is None else q * s + offsets.double()[..., None]).flatten(1)


def q4_product(x, w, rounded=None):
    """(y, bound): products exact, their sums in 32 bits.  A group of 64 is summed by four matrix instructions, each an
    aligned sum that may cut what is below 2^-23 of its largest term, then scaled and added; the offset's part likewise:
    (16 + 4 groups of 64) 2^-23 of the sum of the magnitudes that are added, among which, rounded=False (few rows and bf16
    outputs), are the 128 that every code carries along.  rounded=True (many), weights rounded to fp16: 2^-11 of each, and 2^-19
    of the row's largest 15 |scale| + |offset|; inputs below 2^-40 of their row's largest may be lost."""
    codes, scales, offsets = w
    n, half = codes.shape
    k, groups = 2 * half, scales.shape[1]
    q = torch.stack([codes % 16, codes // 16], dim=-1).view(n, k).double()
    s = scales.double().repeat_interleave(k // groups, dim=1).abs()
    o = 8 * s if offsets is None else offsets.double().repeat_interleave(k // groups, dim=1).abs()
    v, mag = q4_values(w), x.double().abs()
    carried = 0 if rounded is None else 128 * s
    bound = (16 + 4 * (k // 64)) * 2.0 ** -23 * (mag @ (q * s + o + 2 * carried).T)
    if rounded:
        top = (15 * s + (0 if offsets is None else o)).amax(dim=1)
        bound = bound + 2.0 ** -11 * (mag @ v.abs().T) + 2.0 ** -19 * mag.sum(-1, keepdim=True) * top
        bound = bound + 2.0 ** -40 * mag.amax(-1, keepdim=True) * v.abs().sum(-1)
    return x.double() @ v.T, bound


def gated(x, gate, up, act, rounded=None):
    """(y, bound) of act(x gate) * (x up): slopes of both activations are below 1.13; the exponential and the quotient are good to
    2^-20, or to 2^-18 in the form for outputs in bf16 (its argument, below 64, is rounded: 64 log2 e 2^-24 log 2)."""
    (a, ea), (b, eb) = q4_product(x, gate, rounded), q4_product(x, up, rounded)
    f = a * torch.sigmoid(a) if act == "silu" else 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    y = f * b
    return y, 1.13 * ea * (b.abs() + eb) + f.abs() * eb + 2.0 ** (-20 if rounded is None else -18) * y.abs() + 2.0 ** -20 * (a.abs() * b.abs()).clamp_max(1e-6)


def check(got, want, bound):
    """got: bf16 or fp32, rounded once."""
    half = 2.0 ** -8 if got.dtype is BF else 2.0 ** -24
    off = (got.double().to(want.device) - want).abs()
    allowed = bound + half * (want.abs() + bound) + 1e-37
    assert torch.isfinite(got).all()
    assert (off <= allowed).all(), f"off by up to {float((off / allowed).max()):.3g} of what is allowed"
