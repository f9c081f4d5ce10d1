"""The short causal convolution and the selective state space scan (include/gdn.h: gdn_short_conv, gdn_ssm_scan).

    from gated_deltanet_linear_03_gb300 import ssm
    x = ssm.short_conv(x, weight, cu_seqlens, state_in=conv_state, state_out=conv_state)          # prompts, packed
    y = ssm.scan(x, dt, a, b, c, cu_seqlens, d=d, z=z, dt_bias=bias, state_in=h, state_out=h)
    x = ssm.short_conv(x, weight, state_in=conv_state, state_out=conv_state)                      # one token a sequence

Argument marshalling only, like :mod:`gdn`: the kernels run in ``libgdn.so``, there is no CPU fallback, and a call only
enqueues work on the current stream of the tensors' device (or ``stream``).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from .attn import _contiguous, _device, _empty, _int32, _launch, _refuse
from .gdn import DTYPE, GDN_OK, GdnError, load_library

CONV_ACT = {"none": 0, "silu": 1}
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _rows(name: str, t: torch.Tensor, tokens: int, width: int, index: int) -> Tuple[int, int]:
    """Address and row stride of a bf16 [tokens, width] tensor whose rows are contiguous."""
    if t.dtype is not _BF16 or t.get_device() != index or t.dim() != 2:
        _refuse(name, t, _BF16, 2, index)
    if t.shape != (tokens, width):
        raise ValueError(f"{name} must be [{tokens}, {width}], got {tuple(t.shape)}")
    stride = t.stride()
    if stride[1] != 1 and width > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.data_ptr(), stride[0] if tokens > 1 else width       # (a single row's stride says nothing)


def _sequences(cu_seqlens, tokens, state_in, state_out, slots, entry, dtype, index):
    """(n_seqs, cu address, state addresses, slots address, n_slots) of a call."""
    cu = sl = si = so = n_slots = 0
    if cu_seqlens is None:
        n = tokens
    else:
        cu = _contiguous("cu_seqlens", cu_seqlens, _I32, 1, index)
        n = cu_seqlens.size(0) - 1
    ndim = len(entry) + 1
    if state_in is not None:
        si = _contiguous("state_in", state_in, dtype, ndim, index)
        n_slots = state_in.size(0)
        if state_in.shape[1:] != entry:
            raise ValueError(f"state_in must be [slots, {', '.join(map(str, entry))}]")
    if state_out is not None:
        so = si if state_out is state_in else _contiguous("state_out", state_out, dtype, ndim, index)
        if state_out.shape[1:] != entry:
            raise ValueError(f"state_out must be [slots, {', '.join(map(str, entry))}]")
        if state_in is not None and state_out.size(0) != n_slots:
            raise ValueError("state_in and state_out must have the same slots")
        n_slots = state_out.size(0)
    if slots is not None:
        sl = _contiguous("slots", slots, _I32, 1, index)
        if slots.size(0) != n:
            raise ValueError("slots must name one slot for each sequence")
    return n, cu, si, so, sl, n_slots


def _parameter(name: str, t: Optional[torch.Tensor], channels: int, index: int) -> int:
    """The address of an optional fp32 [channels] tensor."""
    if t is None:
        return 0
    p = _contiguous(name, t, _F32, 1, index)
    if t.size(0) != channels:
        raise ValueError(f"{name} must have {channels} entries")
    return p


def short_conv(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None, *,
               bias: Optional[torch.Tensor] = None, act: str = "silu", state_in: Optional[torch.Tensor] = None,
               state_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Run ``gdn_short_conv``: the causal convolution of every channel with its 2 to 4 taps, and its activation
    (``act``: "silu" or "none").  Returns bf16 [T, channels].

    ``x``: bf16 [T, channels], rows contiguous (it may be a slice of a projection).  ``weight``: fp32 [channels, width],
    the last tap on the token itself; ``bias``: fp32 [channels].  ``cu_seqlens``: int32 [n + 1], or None for one token a
    sequence.  ``state_in`` / ``state_out``: bf16 [slots, width - 1, channels], the inputs before the call's tokens and
    those before the next call's; None for sequences that begin, or are not continued.  They may be the same tensor."""
    lib = load_library()
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [tokens, channels]")
    T, channels = x.shape
    xp, stride = _rows("x", x, T, channels, dev)
    wp = _contiguous("weight", weight, _F32, 2, dev)
    if weight.size(0) != channels:
        raise ValueError(f"weight must be [{channels}, width]")
    width = weight.size(1)
    code = CONV_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(CONV_ACT)}")
    n, cu, si, so, sl, n_slots = _sequences(cu_seqlens, T, state_in, state_out, slots, (width - 1, channels), _BF16, dev)
    bp = _parameter("bias", bias, channels, dev)
    if out is None:
        out = _empty(stream, (T, channels), _BF16, x.device)
        op = out.data_ptr()
    else:
        op = _contiguous("out", out, _BF16, 2, dev)
        if out.shape != (T, channels):
            raise ValueError("out must have the shape of x")
    _launch(lib.gdn_short_conv, "gdn_short_conv", dev, stream, n, T, channels, width, xp, stride, wp, bp, code, cu, si, so,
            sl, n_slots, op)
    return out


@functools.lru_cache(maxsize=4096)
def scan_workspace_size(n_seqs: int, total_tokens: int, channels: int, n_state: int, groups: int, max_len: int = 0) -> int:
    """Bytes of workspace that :func:`scan` needs for this problem (``gdn_ssm_scan_workspace_size``)."""
    st = ctypes.c_int(0)
    need = load_library().gdn_ssm_scan_workspace_size(*map(_int32, (n_seqs, total_tokens, channels, n_state, groups, max_len)), st)
    if st.value != GDN_OK:
        raise GdnError(st.value, "gdn_ssm_scan_workspace_size")
    return int(need)


def _vectors(name: str, t: torch.Tensor, shape, index: int) -> Tuple[int, int]:
    """Address and token stride of a bf16 [tokens, groups, n_state] tensor whose tokens' rows are contiguous."""
    if t.dtype is not _BF16 or t.get_device() != index or t.dim() != 3:
        _refuse(name, t, _BF16, 3, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    stride = t.stride()
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name}: a token's vectors must be contiguous")
    return t.data_ptr(), stride[0] if shape[0] > 1 else shape[1] * shape[2]


def scan(x: torch.Tensor, dt: torch.Tensor, a: torch.Tensor, b: torch.Tensor, c: torch.Tensor,
         cu_seqlens: Optional[torch.Tensor] = None, *, d: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
         dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True, state_in: Optional[torch.Tensor] = None,
         state_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None, max_len: int = 0,
         out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """Run ``gdn_ssm_scan``: ``h = exp(D a) h + D x b``, ``y = (h . c + d x) silu(z)`` with the step width
    ``D = softplus(dt + dt_bias)`` (``dt + dt_bias`` without ``dt_softplus``).  Returns [T, channels].

    ``x``, ``dt``, ``z``: bf16 [T, channels]; ``b``, ``c``: bf16 [T, groups, n_state]; all may be slices of projections.
    ``a``: fp32 [channels, n_state]; ``d``, ``dt_bias``: fp32 [channels].  ``cu_seqlens``: int32 [n + 1], or None for one
    token a sequence.  ``state_in`` / ``state_out``: fp32 [slots, channels, n_state], None for sequences that begin, or
    are not continued; they may be the same tensor.  ``max_len``: the longest sequence as far as the host knows; it
    chooses the kernel, nothing else."""
    lib = load_library()
    dev = _device(x, "x")
    if x.dim() != 2 or b.dim() != 3:
        raise ValueError("x must be [tokens, channels] and b [tokens, groups, n_state]")
    T, channels = x.shape
    groups, n_state = b.size(1), b.size(2)
    xp, x_stride = _rows("x", x, T, channels, dev)
    dp, d_stride = _rows("dt", dt, T, channels, dev)
    zp, z_stride = (0, 0) if z is None else _rows("z", z, T, channels, dev)
    shape = (T, groups, n_state)
    bp, b_stride = _vectors("b", b, shape, dev)
    cp, c_stride = _vectors("c", c, shape, dev)
    ap = _contiguous("a", a, _F32, 2, dev)
    if a.shape != (channels, n_state):
        raise ValueError(f"a must be [{channels}, {n_state}]")
    n, cu, si, so, sl, n_slots = _sequences(cu_seqlens, T, state_in, state_out, slots, (channels, n_state), _F32, dev)
    skip, bias = _parameter("d", d, channels, dev), _parameter("dt_bias", dt_bias, channels, dev)
    if out is None:
        if out_dtype not in DTYPE:
            raise ValueError("out_dtype must be bf16 or fp32")
        out = _empty(stream, (T, channels), out_dtype, x.device)
        op = out.data_ptr()
    else:
        out_dtype = out.dtype
        op = _contiguous("out", out, out_dtype, 2, dev)
        if out_dtype not in DTYPE or out.shape != (T, channels):
            raise ValueError("out must have the shape of x, in bf16 or fp32")
    max_len = 1 if cu_seqlens is None else min(_int32(max_len), T)
    if workspace is None:
        ws_bytes = 0 if max_len == 1 else scan_workspace_size(n, T, channels, n_state, groups, max_len)
        wsp = 0
        if ws_bytes:
            workspace = _empty(stream, ws_bytes, torch.uint8, x.device)
            wsp = workspace.data_ptr()
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    else:
        ws_bytes, wsp = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _launch(lib.gdn_ssm_scan, "gdn_ssm_scan", dev, stream, n, T, channels, n_state, groups, xp, x_stride, dp, d_stride, ap,
            bp, b_stride, cp, c_stride, skip, zp, z_stride, bias, int(bool(dt_softplus)), cu, max_len, si, so, sl, n_slots, op,
            DTYPE[out_dtype], wsp, ws_bytes)
    return out
