"""The norms around a block, fused with its gate, scale and residual sum (include/gdn.h: gdn_block_norm).

    from gated_deltanet_linear_03_gb300 import norm
    residual, h = norm.block_norm(x, residual, pre_weight, post_weight=w, gate=g, scale=0.5)
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from .attn import _contiguous, _device, _launch
from .gdn import DTYPE, load_library

GATE_ACT = {"sigmoid": 0, "silu": 1}


def block_norm(x: torch.Tensor, residual: torch.Tensor, pre_weight: torch.Tensor, *,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
               gate_act: str = "sigmoid", scale: Union[float, torch.Tensor] = 1.0, eps: float = 1e-6,
               residual_out: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Run ``gdn_block_norm`` on rows of the last dimension.  Returns ``(residual_out, out)``:

        y = rmsnorm(x) * post_weight     (x itself without post_weight)
        residual_out = residual + scale * y * gate_act(gate)
        out = rmsnorm(residual_out) * pre_weight

    ``x`` and ``gate`` bf16, ``residual`` bf16 or fp32 (its type is ``residual_out``'s), weights fp32 [dim];
    ``scale`` is a number or fp32 [dim].  ``residual_out`` may be ``residual``, ``out`` may be ``x`` or ``gate``."""
    lib = load_library()
    dev = _device(x, "x")
    nd, shape = x.dim(), x.shape
    if nd < 1:
        raise ValueError("x must have a last dimension to normalise over")
    dim = shape[-1]
    xp = _contiguous("x", x, torch.bfloat16, nd, dev)
    if residual.dtype not in DTYPE:
        raise ValueError(f"residual must be bf16 or fp32, got {residual.dtype}")
    rp = _contiguous("residual", residual, residual.dtype, nd, dev)
    pre = _contiguous("pre_weight", pre_weight, torch.float32, 1, dev)
    gp = _contiguous("gate", gate, torch.bfloat16, nd, dev) if gate is not None else 0
    post = _contiguous("post_weight", post_weight, torch.float32, 1, dev) if post_weight is not None else 0
    sw, number = 0, 1.0
    if isinstance(scale, torch.Tensor):
        sw = _contiguous("scale", scale, torch.float32, 1, dev)
    else:
        number = float(scale)
    for name, t in (("pre_weight", pre_weight), ("post_weight", post_weight), ("scale", scale if sw else None)):
        if t is not None and t.shape[0] != dim:
            raise ValueError(f"{name} must have {dim} entries")
    if gate_act not in GATE_ACT:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACT)}")
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    if out is None:
        out = torch.empty_like(x)
    ro = _contiguous("residual_out", residual_out, residual.dtype, nd, dev)
    op = _contiguous("out", out, torch.bfloat16, nd, dev)
    if residual.shape != shape or residual_out.shape != shape or out.shape != shape or (gate is not None and gate.shape != shape):
        raise ValueError("x, gate, residual and the outputs must have one shape")
    rows = x.numel() // dim if dim else 0
    _launch(lib.gdn_block_norm, "gdn_block_norm", dev, stream, rows, dim, xp, gp, GATE_ACT[gate_act], rp,
            DTYPE[residual.dtype], post, pre, sw, number, float(eps), ro, op)
    return residual_out, out
