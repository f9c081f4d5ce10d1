"""The norms around a block, fused with its gate, scale and residual sum (include/gdn.h: gdn_block_norm).

    from gated_deltanet_linear_03_gb300 import norm
    residual, h = norm.block_norm(x, residual, pre_weight, post_weight=w, gate=g, scale=0.5)
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from .attn import _contiguous, _device, _empty, _int32, _launch
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
    bf16, f32 = torch.bfloat16, torch.float32
    res = residual.dtype
    res_code = DTYPE.get(res)
    if res_code is None:
        raise ValueError(f"residual must be bf16 or fp32, got {res}")
    if residual.shape != shape or (gate is not None and gate.shape != shape) or \
            (residual_out is not None and residual_out.shape != shape) or (out is not None and out.shape != shape):
        raise ValueError("x, gate, residual and the outputs must have one shape")
    scaled = isinstance(scale, torch.Tensor)
    if pre_weight.size(0) != dim or (post_weight is not None and post_weight.size(0) != dim) or (scaled and scale.size(0) != dim):
        raise ValueError(f"pre_weight, post_weight and a scale per channel must have {dim} entries")
    act = GATE_ACT.get(gate_act)
    if act is None:
        raise ValueError(f"gate_act must be one of {sorted(GATE_ACT)}")
    xp, rp = _contiguous("x", x, bf16, nd, dev), _contiguous("residual", residual, res, nd, dev)
    if residual_out is None:
        residual_out = _empty(stream, shape, res, x.device)
        rop = residual_out.data_ptr()
    else:
        rop = _contiguous("residual_out", residual_out, res, nd, dev)
    if out is None:
        out = _empty(stream, shape, bf16, x.device)
        op = out.data_ptr()
    else:
        op = _contiguous("out", out, bf16, nd, dev)
    _launch(lib.gdn_block_norm, "gdn_block_norm", dev, stream, _int32(x.numel() // dim) if dim else 0, dim, xp,
            0 if gate is None else _contiguous("gate", gate, bf16, nd, dev), act, rp, res_code,
            0 if post_weight is None else _contiguous("post_weight", post_weight, f32, 1, dev),
            _contiguous("pre_weight", pre_weight, f32, 1, dev), _contiguous("scale", scale, f32, 1, dev) if scaled else 0,
            1.0 if scaled else scale, eps, rop, op)
    return residual_out, out
