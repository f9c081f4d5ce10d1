"""Products with weights of 4 bits (include/gdn.h: gdn_q4_linear, gdn_q4_gated).

    from gated_deltanet_linear_03_gb300 import linear
    w = linear.quantize(weight)                       # once, when the weights are loaded
    y = linear.q4_linear(x, w)                        # x weight^T
    h = linear.q4_gated(x, gate, up, act="silu")      # silu(x gate^T) * (x up^T), the first half of a feed-forward block

Argument marshalling only, like :mod:`gdn`: the products run in ``libgdn.so``, there is no CPU fallback, and a call only
enqueues work on the current stream of the tensors' device (or ``stream``).
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from .attn import _contiguous, _device, _empty, _int32, _launch, _refuse
from .gdn import DTYPE, GDN_OK, GdnError, fast_calls, load_library

FFN_ACT = {"silu": 0, "gelu": 1}
_BF16, _U8 = torch.bfloat16, torch.uint8


class Q4(NamedTuple):
    """A matrix [n_out, k] in 4 bits: ``scales * codes + offsets``, or ``scales * (codes - 8)`` without offsets.

    ``codes``: uint8 [n_out, k / 2], inputs 2i and 2i + 1 in the low and the high half of byte i; ``scales`` and
    ``offsets``: bf16 [n_out, k / group] for groups of 64 or 128 inputs."""
    codes: torch.Tensor
    scales: torch.Tensor
    offsets: Optional[torch.Tensor] = None


def quantize(weight: torch.Tensor, group: int = 64, offsets: bool = True) -> Q4:
    """``weight`` [n_out, k] (any float type, any device) in 4 bits, each value to the nearest that its group's bf16 scale
    (and offset) can give.  With ``offsets`` a group's codes span its smallest to its largest value, otherwise its largest
    magnitude, to both sides of zero."""
    if weight.dim() != 2 or group not in (64, 128) or weight.size(1) % group:
        raise ValueError("weight must be [n_out, k] with k a multiple of group, 64 or 128")
    n_out, k = weight.shape
    w = weight.float().contiguous().view(n_out, k // group, group)
    if offsets:
        lo, hi = w.amin(dim=-1), w.amax(dim=-1)
        scale, offset = ((hi - lo) / 15).to(_BF16), lo.to(_BF16)
        code = w - offset.float()[..., None]
    else:
        scale, offset = (w.abs().amax(dim=-1) / 7.5).to(_BF16), None
        code = w.clone()
    s = scale.float()[..., None]
    code = torch.where(s > 0, code / s, 0)
    code = (code if offsets else code + 8).round_().clamp_(0, 15).to(_U8).view(n_out, k)
    return Q4(code[:, 0::2] | (code[:, 1::2] << 4), scale, offset)


def values(w: Q4) -> torch.Tensor:
    """The matrix that ``w`` stands for, fp32 [n_out, k]."""
    n_out, half = w.codes.shape
    group = 2 * half // w.scales.size(1)
    q = torch.stack([w.codes & 15, w.codes >> 4], dim=-1).view(n_out, -1, group).float()
    s = w.scales.float()[..., None]
    return ((q - 8) * s if w.offsets is None else q * s + w.offsets.float()[..., None]).flatten(1)


# Calls in which nothing is wrong go by csrc/fast_calls.cpp, which checks the same; what follows makes the others, or says what is
# wrong with them.
def _matrix(name: str, w: Q4, k: int, index: int):
    """(codes, scales, offsets addresses, n_out, group) of a matrix whose inputs are ``k``."""
    codes, scales, offsets = w
    cp = _contiguous(name + ".codes", codes, _U8, 2, index)
    sp = _contiguous(name + ".scales", scales, _BF16, 2, index)
    n_out, half = codes.shape
    rows, groups = shape = scales.shape
    if 2 * half != k or rows != n_out or groups == 0 or k % groups:
        raise ValueError(f"{name} must have codes [n_out, {k // 2}] and scales [n_out, {k} / group], "
                         f"got {tuple(codes.shape)} and {tuple(shape)}")
    op = 0
    if offsets is not None:
        op = _contiguous(name + ".offsets", offsets, _BF16, 2, index)
        if offsets.shape != shape:
            raise ValueError(f"{name}.offsets must have the shape of its scales")
    return cp, sp, op, n_out, k // groups


def _rows(x: torch.Tensor, index: int):
    """(row stride, rows, k) of activations bf16 [..., k]: contiguous, or 2-d with contiguous rows."""
    shape = x.shape
    if x.dtype is not _BF16 or not shape:
        _refuse("x", x, _BF16, 2, index)
    k = shape[-1]
    if len(shape) == 2:
        if x.is_contiguous():
            return k, shape[0], k
        if x.stride(1) == 1:
            return x.stride(0), shape[0], k
    elif x.is_contiguous():
        return k, x.numel() // k if k else 0, k
    raise ValueError("x must be contiguous, or 2-d with contiguous rows")


def _output(x, n_out, out, out_dtype, index, stream):
    shape = (*x.shape[:-1], n_out)
    if out is None:
        code = DTYPE.get(out_dtype)
        if code is None:
            raise ValueError("out_dtype must be bf16 or fp32")
        return _empty(stream, shape, out_dtype, x.device), code
    code = DTYPE.get(out.dtype)
    if code is None or out.shape != shape:
        raise ValueError(f"out must be {shape}, in bf16 or fp32")
    _contiguous("out", out, out.dtype, len(shape), index)
    return out, code


@functools.lru_cache(maxsize=4096)
def workspace_size(rows: int, n_out: int, k: int, group: int, out_dtype=torch.bfloat16) -> int:
    """Bytes of workspace that :func:`q4_linear` and :func:`q4_gated` need for this problem (``gdn_q4_workspace_size``)."""
    st = ctypes.c_int(0)
    need = load_library().gdn_q4_workspace_size(_int32(rows), n_out, k, group, DTYPE[out_dtype], st)
    if st.value != GDN_OK:
        raise GdnError(st.value, "gdn_q4_workspace_size")
    return int(need)


def _workspace(workspace, rows, n_out, k, group, out, index, stream):
    """(address, bytes, what keeps the memory alive)."""
    if workspace is not None:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    else:
        need = workspace_size(rows, n_out, k, group, out.dtype)
        if need == 0:
            return 0, 0, None
        workspace = _empty(stream, need, _U8, out.device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def q4_linear(x: torch.Tensor, w: Q4, *, out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
              workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Run ``gdn_q4_linear``: ``x`` (bf16 [..., k]) times the transpose of ``w``: [..., n_out] in bf16 or fp32."""
    if stream is None and workspace is None:
        done = fast_calls().q4_linear(x, w, 0, out, DTYPE.get(out_dtype, -1))
        if done is not None:
            return done
    lib = load_library()
    dev = _device(x, "x")
    stride, rows, k = _rows(x, dev)
    cp, sp, fp, n_out, group = _matrix("w", w, k, dev)
    out, code = _output(x, n_out, out, out_dtype, dev, stream)
    wsp, ws_bytes, _keep = _workspace(workspace, rows, n_out, k, group, out, dev, stream)
    _launch(lib.gdn_q4_linear, "gdn_q4_linear", dev, stream, _int32(rows), n_out, k, group, x.data_ptr(), stride, cp, sp, fp,
            out.data_ptr(), code, wsp, ws_bytes)
    return out


def q4_gated(x: torch.Tensor, gate: Q4, up: Q4, *, act: str = "silu", out: Optional[torch.Tensor] = None,
             out_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Run ``gdn_q4_gated``: ``act(x gate^T) * (x up^T)`` for two matrices of one shape ([n_out, k], one group size, offsets
    in both or neither); ``act`` is "silu" or "gelu" (its tanh form)."""
    if stream is None and workspace is None:
        done = fast_calls().q4_gated(x, gate, up, FFN_ACT.get(act, -1), out, DTYPE.get(out_dtype, -1))
        if done is not None:
            return done
    lib = load_library()
    dev = _device(x, "x")
    stride, rows, k = _rows(x, dev)
    gc, gs, go, n_out, group = _matrix("gate", gate, k, dev)
    uc, us, uo, n_up, up_group = _matrix("up", up, k, dev)
    if n_up != n_out or up_group != group or (go == 0) != (uo == 0):
        raise ValueError("gate and up must have one shape and one kind of groups")
    act_code = FFN_ACT.get(act)
    if act_code is None:
        raise ValueError(f"act must be one of {sorted(FFN_ACT)}")
    out, code = _output(x, n_out, out, out_dtype, dev, stream)
    wsp, ws_bytes, _keep = _workspace(workspace, rows, n_out, k, group, out, dev, stream)
    _launch(lib.gdn_q4_gated, "gdn_q4_gated", dev, stream, _int32(rows), n_out, k, group, x.data_ptr(), stride, gc, gs, go,
            uc, us, uo, act_code, out.data_ptr(), code, wsp, ws_bytes)
    return out
