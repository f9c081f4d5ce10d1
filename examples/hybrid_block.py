"""Serving a small hybrid stack: a Gated DeltaNet layer and an attention layer with an 8-bit paged cache, for ragged
prompts and then one token a sequence at a time.

    python examples/hybrid_block.py [--tokens 24] [--format int8|e4m3] [--complete]

Every layer is: block_norm (the norm before the layer, fused with the gated residual sum after the one before),
projections, then gdn.prefill / gdn.decode_step or attn.kv_append + attn.attend.  The complete stack holds its weights in
4 bits (linear.q4_linear), has a short convolution in front of the recurrence (ssm.short_conv), and two more layers: a
selective state space layer (ssm.scan behind a convolution of its own) and a gated feed-forward block (linear.q4_gated).
Weights are random.  The run compares decoding with a prefill of the same tokens in one piece.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_deltanet_linear_03_gb300 import attn, gdn, linear, norm, ssm  # noqa: E402

DIM, HK, HV, DK = 512, 2, 4, 128             # the linear layer: query/key heads, value heads, head size
HQ, HKV, D, ROT = 8, 2, 64, 32               # the attention layer: query heads, key/value heads, head size, rotated part
PAGE, MAX_LEN = 32, 1024
INNER, STATES, RANK, FF = 1024, 16, 64, 1024  # the state space layer: channels, states, inputs of its step widths; the feed-forward block
CONV = 4                                     # taps of the convolutions


class Hybrid:
    """The stack's weights, and the state of ``n_seqs`` sequences: a recurrent state, cache pages, lengths."""

    def __init__(self, n_seqs, cache_dtype=torch.int8, seed=0, device="cuda", complete=False):
        gen = torch.Generator().manual_seed(seed)

        def matrix(rows, cols):
            w = torch.randn(rows, cols, generator=gen) * rows ** -0.5
            return linear.Q4(*(t.to(device) for t in linear.quantize(w.T))) if complete else w.to(torch.bfloat16).to(device)

        self.complete = complete
        self.w_gdn = matrix(DIM, 2 * HK * DK + HV * DK + 2 * HV)     # q, k, v, decay and beta inputs
        self.w_attn = matrix(DIM, (HQ + 2 * HKV) * D)                # q, k, v
        self.w_out = [matrix(HV * DK, DIM), matrix(HQ * D, DIM)]
        self.w_gate = [matrix(DIM, DIM) for _ in range(2)]
        self.pre = [torch.ones(DIM, device=device) for _ in range(3)]
        self.post = [torch.ones(DIM, device=device) for _ in range(2)]
        self.gdn_norm = torch.ones(DK, device=device)
        self.decay, self.bias = torch.full((HV,), 0.1, device=device), torch.zeros(HV, device=device)
        angle = torch.arange(MAX_LEN)[:, None] * 10000.0 ** (-torch.arange(ROT // 2) * 2.0 / ROT)
        self.cos, self.sin = angle.cos().float().to(device), angle.sin().float().to(device)

        per_seq = MAX_LEN // PAGE
        self.n, self.device = n_seqs, device
        self.state = torch.zeros(n_seqs, HV, DK, DK, device=device)
        self.cache = attn.alloc_cache(n_seqs * per_seq, HKV, PAGE, D, n_seqs, cache_dtype, device)
        self.table = torch.randperm(n_seqs * per_seq, generator=gen).to(torch.int32).view(n_seqs, per_seq).to(device)
        self.lens = [0] * n_seqs
        if not complete:
            return

        def taps(channels):
            return (torch.randn(channels, CONV, generator=gen) * CONV ** -0.5).to(device)

        qkv = 2 * HK * DK + HV * DK
        self.conv = [taps(qkv), taps(INNER)]                          # in front of the recurrence, and of the scan
        self.conv_state = [torch.zeros(n_seqs, CONV - 1, c, dtype=torch.bfloat16, device=device) for c in (qkv, INNER)]
        self.w_in = matrix(DIM, 2 * INNER)                            # the scan's inputs and its gate
        self.w_x = matrix(INNER, RANK + 2 * STATES)                   # what the step widths, B and C come from
        self.w_dt, self.w_y = matrix(RANK, INNER), matrix(INNER, DIM)
        self.a = -torch.arange(1.0, STATES + 1, device=device).repeat(INNER, 1)
        self.dt_bias, self.skip = torch.full((INNER,), -3.0, device=device), torch.ones(INNER, device=device)
        self.ssm_state = torch.zeros(n_seqs, INNER, STATES, device=device)
        self.ff_gate, self.ff_up, self.ff_down = matrix(DIM, FF), matrix(DIM, FF), matrix(FF, DIM)
        self.more = [torch.ones(DIM, device=device) for _ in range(4)]

    def _i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device=self.device)

    def _mul(self, x, w):
        return linear.q4_linear(x, w) if self.complete else x @ w

    def _conv(self, i, x, cu):
        return ssm.short_conv(x, self.conv[i], cu, state_in=self.conv_state[i], state_out=self.conv_state[i])

    def forward(self, x, new):
        """The next ``new[n]`` tokens of every sequence, packed in ``x`` (bf16 [sum(new), DIM]).  One token of each takes the
        decode kernels."""
        T = x.shape[0]
        cu_host = [0]
        for m in new:
            cu_host.append(cu_host[-1] + m)
        cu, past = self._i32(cu_host), self._i32(self.lens)
        self.lens = [a + b for a, b in zip(self.lens, new)]
        kv_lens = self._i32(self.lens)

        residual, h = norm.block_norm(x, torch.zeros(T, DIM, device=self.device), self.pre[0])

        tokens = None if all(m == 1 for m in new) else cu     # (one token each needs no table of where sequences begin)
        p = self._mul(h, self.w_gdn)
        qkv, a, b = p.split([2 * HK * DK + HV * DK, HV, HV], dim=1)
        if self.complete:
            qkv = self._conv(0, qkv, tokens)                  # read where the projection left it
        q, k, v = qkv.split([HK * DK, HK * DK, HV * DK], dim=1)
        q, k, v = (t.reshape(T, -1, DK).contiguous() for t in (q, k, v))
        args = (q, k, v, a.float().contiguous(), b.float().contiguous())
        opts = dict(qk_norm=True, q_scale=DK ** -0.5, norm_weight=self.gdn_norm, gate_scale=self.decay, gate_bias=self.bias)
        if all(m == 1 for m in new):
            y = gdn.decode_step(self.state, *args, **opts)
        else:
            y, _ = gdn.prefill(*args, cu, init_state=self.state, final_state=self.state, cu_seqlens_host=cu_host, **opts)
        residual, h = norm.block_norm(self._mul(y.reshape(T, -1), self.w_out[0]), residual, self.pre[1], post_weight=self.post[0],
                                      gate=self._mul(h, self.w_gate[0]), gate_act="silu")

        p = self._mul(h, self.w_attn).view(T, HQ + 2 * HKV, D)       # q, k and v are read where the projection left them
        q, k, v = p.split([HQ, HKV, HKV], dim=1)
        q, _ = attn.kv_append(k, v, self.cos, self.sin, cu, past, self.table, *self.cache, q=q)
        y = attn.attend(q, *self.cache[:4], self.table, cu, kv_lens, max_q_len=max(new), max_kv_len=max(self.lens))
        residual, h = norm.block_norm(self._mul(y.view(T, -1), self.w_out[1]), residual, self.pre[2], post_weight=self.post[1],
                                      gate=self._mul(h, self.w_gate[1]))
        return self._state_space_and_feed_forward(residual, h, tokens, max(new)) if self.complete else h

    def _state_space_and_feed_forward(self, residual, h, cu, longest):
        x, z = linear.q4_linear(h, self.w_in).split([INNER, INNER], dim=1)
        x = self._conv(1, x, cu)
        p = linear.q4_linear(x, self.w_x)
        b, c = (p[:, at:at + STATES].unsqueeze(1) for at in (RANK, RANK + STATES))
        dt = linear.q4_linear(p[:, :RANK], self.w_dt)
        y = ssm.scan(x, dt, self.a, b, c, cu, d=self.skip, z=z, dt_bias=self.dt_bias, state_in=self.ssm_state,
                     state_out=self.ssm_state, max_len=longest)
        residual, h = norm.block_norm(linear.q4_linear(y, self.w_y), residual, self.more[0], post_weight=self.more[1])
        y = linear.q4_linear(linear.q4_gated(h, self.ff_gate, self.ff_up), self.ff_down)
        return norm.block_norm(y, residual, self.more[2], post_weight=self.more[3])[1]


def run(tokens=24, cache_dtype=torch.int8, prompts=(200, 37, 1, 64), complete=False):
    """Decoded outputs [tokens, n, DIM], and the same rows of a prefill of everything at once."""
    n = len(prompts)
    gen = torch.Generator().manual_seed(1)
    xs = [torch.randn(m + tokens, DIM, generator=gen).to(torch.bfloat16).cuda() for m in prompts]

    served = Hybrid(n, cache_dtype, complete=complete)
    served.forward(torch.cat([x[:m] for x, m in zip(xs, prompts)]), list(prompts))
    decoded = torch.stack([served.forward(torch.stack([x[m + t] for x, m in zip(xs, prompts)]), [1] * n)
                           for t in range(tokens)])

    whole = Hybrid(n, cache_dtype, complete=complete).forward(torch.cat(xs), [m + tokens for m in prompts])
    at, rows = 0, []
    for m in prompts:
        rows.append(whole[at + m:at + m + tokens])
        at += m + tokens
    return decoded.float(), torch.stack(rows, dim=1).float()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--format", choices=["int8", "e4m3"], default="int8")
    ap.add_argument("--complete", action="store_true", help="4-bit weights, short convolutions, a state space and a feed-forward layer")
    a = ap.parse_args()
    decoded, whole = run(a.tokens, torch.int8 if a.format == "int8" else torch.float8_e4m3fn, complete=a.complete)
    rel = ((decoded - whole).square().mean() / whole.square().mean()).sqrt().item()
    print(f"{a.tokens} tokens of {decoded.shape[1]} sequences, {a.format} cache: decode and prefill differ by {rel:.4f} (RMS, relative)")


if __name__ == "__main__":
    main()
