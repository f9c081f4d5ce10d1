"""Plain 64-bit forms of the cache, attention and block-norm operators, written from their formulas, for the tests."""
import math
from dataclasses import dataclass

import torch

BLOCK = 16
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
FLOOR = 2.0 ** -60


def rotate(x, pos, cos, sin, interleaved):
    """x [T, h, d] (any type), pos [T]: rotated in 64 bits."""
    x = x.double().clone()
    if cos is None or cos.shape[1] == 0:
        return x
    half = cos.shape[1]
    c, s = cos.double()[pos][:, None], sin.double()[pos][:, None]
    ia = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def quantise(x, dtype):
    """Blocks x [..., 16, d] (bf16 values) to (codes, scales), in 32 bits as the definition is."""
    x = x.float()
    amax = x.abs().amax(dim=(-1, -2)).clamp_min(FLOOR)
    y = x * (torch.tensor(QMAX[dtype]) / amax)[..., None, None]
    codes = torch.round(y).clamp(-127, 127).to(torch.int8) if dtype == torch.int8 else y.clamp(-448, 448).to(dtype)
    return codes, amax / QMAX[dtype]


@dataclass
class Cache:
    """A pool on the CPU: pages in no order, one slot a sequence."""
    table: torch.Tensor
    k_pages: torch.Tensor
    v_pages: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor

    def on(self, dev):
        return Cache(*[getattr(self, f).to(dev) for f in ("table", "k_pages", "v_pages", "k_scales", "v_scales")])

    @property
    def args(self):
        return self.k_pages, self.v_pages, self.k_scales, self.v_scales

    def values(self, which, n, upto):
        """Tokens 0 .. upto of sequence n in 64 bits [upto, hkv, d]."""
        pages, scales = (self.k_pages, self.k_scales) if which == "k" else (self.v_pages, self.v_scales)
        hkv, page, d = pages.shape[1:]
        out = torch.zeros(upto, hkv, d, dtype=torch.float64)
        for j in range(upto):
            p = int(self.table[n, j // page])
            out[j] = pages[p, :, j % page].to(torch.float64) * scales[p, :, j % page // BLOCK, None].double()
        return out


def make_table(lens, page, gen, spare=3, bad=None):
    """A table with pages in random order; entries no token reaches are `bad` (default: another sequence's page)."""
    need = [max(0, -(-x // page)) for x in lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(need + [1]) + 1), 0 if bad is None else bad, dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    return table, n_pages


def make_cache(lens, hkv, d, page, dtype, seed, spread=0.5, bad=None):
    """A filled pool; rows past a sequence's end are zero codes."""
    gen = torch.Generator().manual_seed(seed)
    table, n_pages = make_table(lens, page, gen, bad=bad)
    out = []
    for _ in range(2):
        x = torch.randn(n_pages, hkv, page // BLOCK, BLOCK, d, generator=gen)
        x = x * torch.exp(spread * torch.randn(n_pages, hkv, page // BLOCK, 1, 1, generator=gen))
        codes, scales = quantise(x.to(torch.bfloat16), dtype)
        codes = codes.view(torch.int8).view(n_pages, hkv, page, d).clone()
        for i, length in enumerate(lens):
            if length % page:
                codes[int(table[i, length // page]), :, length % page:] = 0
        out.append((codes.view(dtype), scales.contiguous()))
    return Cache(table, out[0][0], out[1][0], out[0][1], out[1][1])


def attend(q, cache, cu, lens, window=0, sinks=0, sm_scale=None):
    """(outputs, bounds on their error) in 64 bits: the bound is the one that the kernels' number formats give,

    a weight's relative error: 2^-11 (fp16) + 2 delta, delta the error of the score in fp32: 2^-23 d sum |q_i k_i| scale
    (sequential worst case of d additions; the products are exact) + 2^-19 (exponentials and the logarithm of the
    scale); a weight below fp16's normal range has the absolute error 2^-25 of the largest weighted scale."""
    T, hq, d = q.shape
    hkv = cache.k_pages.shape[1]
    group = hq // hkv
    scale = 1 / math.sqrt(d) if sm_scale is None else sm_scale
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    tol = torch.zeros(T, hq, d, dtype=torch.float64)
    qmax = QMAX[cache.k_pages.dtype]
    for n, L in enumerate(lens):
        m = cu[n + 1] - cu[n]
        if m == 0 or L == 0:
            continue
        k, v = cache.values("k", n, L), cache.values("v", n, L)
        page = cache.k_pages.shape[2]
        j = torch.arange(L)
        vs = cache.v_scales.double()[cache.table[n].long()[j // page], :, j % page // BLOCK]       # [L, hkv]
        pos = L - m + torch.arange(m)
        seen = j[None] <= pos[:, None]
        if window:
            seen &= (j[None] > pos[:, None] - window) | (j[None] < sinks)
        for h in range(hq):
            x = q[cu[n]:cu[n + 1], h].double()
            s = (x @ k[:, h // group].T) * scale
            s_abs = (x.abs() @ k[:, h // group].abs().T) * abs(scale)
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(dim=1, keepdim=True).clamp_min(-1e300)
            e = torch.exp(s - top)
            w = e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)
            o = w @ v[:, h // group]
            delta = 2.0 ** -23 * d * s_abs.masked_fill(~seen, 0).amax(dim=1, keepdim=True) + 2.0 ** -19
            a = w @ v[:, h // group].abs()
            small = (w * vs[:, h // group]).amax(dim=1, keepdim=True) * (2.0 ** -25 * qmax) * seen.sum(dim=1, keepdim=True)
            out[cu[n]:cu[n + 1], h] = o
            tol[cu[n]:cu[n + 1], h] = a * (2.0 ** -11 + 2 * delta) + small + 1e-30
    return out, tol


def block_norm(x, residual, pre, post=None, gate=None, act="sigmoid", scale=1.0, eps=1e-6):
    y = x.double()
    if post is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * post.double()
    if gate is not None:
        g = gate.double()
        y = y * torch.sigmoid(g) * (g if act == "silu" else 1)
    add = (scale.double() if isinstance(scale, torch.Tensor) else scale) * y
    r = residual.double() + add
    return r, r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps) * pre.double(), add.abs()
