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
from typing import Optional

import torch

from .attn import _contiguous, _device, _empty, _int32, _launch, _refuse
from .gdn import DTYPE, GDN_OK, GdnError, fast_calls, load_library

CONV_ACT = {"none": 0, "silu": 1}
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


# Calls in which nothing is wrong go by csrc/fast_calls.cpp, which checks the same; what follows makes the others, or says what is
# wrong with them.
def _rows(name: str, t: torch.Tensor, shape, index: int) -> int:
    """The row stride of a bf16 [tokens, width] tensor whose rows are contiguous; ``shape`` is what it must be."""
    if t.dtype is not _BF16 or t.get_device() != index or t.dim() != 2:
        _refuse(name, t, _BF16, 2, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1]                       # (a single row's stride says nothing)
    stride = t.stride()
    if stride[1] != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return stride[0]


def _states(state_in, state_out, d0: int, d1: int, dtype, index: int):
    """(addresses of both, slots) of states [slots, d0, d1]."""
    si = so = n_slots = 0
    if state_in is not None:
        si = _contiguous("state_in", state_in, dtype, 3, index)
        n_slots, e0, e1 = state_in.shape
        if e0 != d0 or e1 != d1:
            raise ValueError(f"state_in must be [slots, {d0}, {d1}], got {tuple(state_in.shape)}")
        if state_out is state_in:
            return si, si, n_slots
    if state_out is not None:
        so = _contiguous("state_out", state_out, dtype, 3, index)
        slots, e0, e1 = state_out.shape
        if e0 != d0 or e1 != d1 or (si and slots != n_slots):
            raise ValueError(f"state_out must be [slots, {d0}, {d1}] with as many slots as state_in, got {tuple(state_out.shape)}")
        n_slots = slots
    return si, so, n_slots


def _packing(cu_seqlens, slots, tokens: int, index: int):
    """(sequences, address of cu_seqlens, address of slots)."""
    cu = sl = 0
    n = tokens
    if cu_seqlens is not None:
        cu = _contiguous("cu_seqlens", cu_seqlens, _I32, 1, index)
        n = cu_seqlens.shape[0] - 1
    if slots is not None:
        sl = _contiguous("slots", slots, _I32, 1, index)
        if slots.shape[0] != n:
            raise ValueError("slots must name one slot for each sequence")
    return n, cu, sl


def _parameter(name: str, t: torch.Tensor, channels: int, index: int) -> int:
    """The address of an fp32 [channels] tensor."""
    if t.dtype is _F32 and t.get_device() == index and t.is_contiguous() and t.shape == (channels,):
        return t.data_ptr()
    _refuse(name, t, _F32, 1, index) if t.dim() != 1 or t.shape[0] == channels else None
    raise ValueError(f"{name} must have {channels} entries")


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
    if stream is None:
        done = fast_calls().short_conv(x, weight, cu_seqlens, bias, CONV_ACT.get(act, -1), state_in, state_out, slots, out)
        if done is not None:
            return done
    lib = load_library()
    dev = _device(x, "x")
    shape = x.shape
    stride = _rows("x", x, shape, dev)
    T, channels = shape
    wp = _contiguous("weight", weight, _F32, 2, dev)
    rows, width = weight.shape
    if rows != channels:
        raise ValueError(f"weight must be [{channels}, width]")
    code = CONV_ACT.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(CONV_ACT)}")
    n, cu, sl = (T, 0, 0) if cu_seqlens is None and slots is None else _packing(cu_seqlens, slots, T, dev)
    si, so, n_slots = _states(state_in, state_out, width - 1, channels, _BF16, dev)
    bp = 0 if bias is None else _parameter("bias", bias, channels, dev)
    if out is None:
        out = _empty(stream, shape, _BF16, x.device)
    elif out.dtype is not _BF16 or out.get_device() != dev or not out.is_contiguous() or out.shape != shape:
        _contiguous("out", out, _BF16, 2, dev)
        raise ValueError("out must have the shape of x")
    _launch(lib.gdn_short_conv, "gdn_short_conv", dev, stream, n, T, channels, width, x.data_ptr(), stride, wp, bp, code, cu, si,
            so, sl, n_slots, out.data_ptr())
    return out


def scan_workspace_size(n_seqs: int, total_tokens: int, channels: int, n_state: int, groups: int, max_len: int = 0) -> int:
    """Bytes of workspace that :func:`scan` needs for this problem on the current device
    (``gdn_ssm_scan_workspace_size``), by whose multiprocessors the scan is divided."""
    return _workspace_size(torch.cuda.current_device() if torch.cuda.is_available() else -1, n_seqs, total_tokens, channels, n_state,
                           groups, max_len)


@functools.lru_cache(maxsize=4096)
def _workspace_size(index: int, *sizes: int) -> int:
    """:func:`scan_workspace_size` on CUDA device ``index`` (-1: there is none)."""
    st = ctypes.c_int(0)
    size = load_library().gdn_ssm_scan_workspace_size
    if index < 0 or torch._C._cuda_getDevice() == index:
        need = size(*map(_int32, sizes), st)
    else:
        with torch.cuda.device(index):
            need = size(*map(_int32, sizes), st)
    if st.value != GDN_OK:
        raise GdnError(st.value, "gdn_ssm_scan_workspace_size")
    return int(need)


def _vectors(name: str, t: torch.Tensor, shape, index: int) -> int:
    """The token stride of a bf16 [tokens, groups, n_state] tensor whose tokens' vectors are contiguous."""
    if t.dtype is not _BF16 or t.get_device() != index or t.dim() != 3:
        _refuse(name, t, _BF16, 3, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[1] * shape[2]
    stride = t.stride()
    if stride[2] != 1 or (shape[1] > 1 and stride[1] != shape[2]):
        raise ValueError(f"{name}: a token's vectors must be contiguous")
    return stride[0] if shape[0] > 1 else shape[1] * shape[2]


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
    if stream is None and workspace is None:
        done = fast_calls().scan(x, dt, a, b, c, cu_seqlens, d, z, dt_bias, dt_softplus, state_in, state_out, slots, max_len, out,
                                 DTYPE.get(out_dtype, -1))
        if done is not None:
            return done
    lib = load_library()
    dev = _device(x, "x")
    shape, vectors = x.shape, b.shape
    x_stride = _rows("x", x, shape, dev)
    d_stride = _rows("dt", dt, shape, dev)
    b_stride = _vectors("b", b, vectors, dev)
    c_stride = _vectors("c", c, vectors, dev)
    T, channels = shape
    tokens, groups, n_state = vectors
    if tokens != T:
        raise ValueError("x and b must have the same tokens")
    zp = z_stride = 0
    if z is not None:
        z_stride = _rows("z", z, shape, dev)
        zp = z.data_ptr()
    ap = _contiguous("a", a, _F32, 2, dev)
    if a.shape != (channels, n_state):
        raise ValueError(f"a must be [{channels}, {n_state}]")
    skip = 0 if d is None else _parameter("d", d, channels, dev)
    bias = 0 if dt_bias is None else _parameter("dt_bias", dt_bias, channels, dev)
    si, so, n_slots = _states(state_in, state_out, channels, n_state, _F32, dev)
    if out is not None:
        out_dtype = out.dtype
        _contiguous("out", out, out_dtype, 2, dev)
    out_code = DTYPE.get(out_dtype)
    if out_code is None or (out is not None and out.shape != shape):
        raise ValueError("out must have the shape of x, in bf16 or fp32")
    if out is None:
        out = _empty(stream, shape, out_dtype, x.device)
    wsp = ws_bytes = 0
    if cu_seqlens is None:
        n, cu, sl = (T, 0, 0) if slots is None else _packing(None, slots, T, dev)
        max_len = 1
    else:
        n, cu, sl = _packing(cu_seqlens, slots, T, dev)
        max_len = min(_int32(max_len), T)
        if workspace is None:
            ws_bytes = _workspace_size(dev, n, T, channels, n_state, groups, max_len)
            if ws_bytes:
                workspace = _empty(stream, ws_bytes, torch.uint8, x.device)
                wsp = workspace.data_ptr()
    if workspace is not None and not wsp:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
        ws_bytes, wsp = workspace.numel() * workspace.element_size(), workspace.data_ptr()
    _launch(lib.gdn_ssm_scan, "gdn_ssm_scan", dev, stream, n, T, channels, n_state, groups, x.data_ptr(), x_stride, dt.data_ptr(),
            d_stride, ap, b.data_ptr(), b_stride, c.data_ptr(), c_stride, skip, zp, z_stride, bias, 1 if dt_softplus else 0, cu,
            max_len, si, so, sl, n_slots, out.data_ptr(), out_code, wsp, ws_bytes)
    return out
