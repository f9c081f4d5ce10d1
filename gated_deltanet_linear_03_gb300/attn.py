"""The 8-bit paged key/value cache and attention over it (include/gdn.h: gdn_kv_append, gdn_kv_read, gdn_attend).

    from gated_deltanet_linear_03_gb300 import attn
    cache = attn.alloc_cache(n_pages, hkv, page_size, d, n_slots)            # pages, scales, open blocks
    q, _ = attn.kv_append(k, v, cos, sin, cu_seqlens, past_lens, block_table, *cache, q=q, open_out=cache[-1])
    out = attn.attend(q, *cache[:4], block_table, cu_seqlens, kv_lens, max_q_len=..., max_kv_len=...)

Argument marshalling only, like :mod:`gdn`: the kernels run in ``libgdn.so``, there is no CPU fallback, and a
call only enqueues work on the current stream of the tensors' device (or ``stream``).
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from .gdn import DTYPE, GDN_OK, GdnError, load_library

KV_BLOCK = 16                                             # tokens that share a scale
FORMAT = {torch.int8: 0, torch.float8_e4m3fn: 1}


# These calls are made for every layer of every generated token, where the host's time counts as much as the GPU's, so the
# checks are written for the case that nothing is wrong; `_refuse` finds out what was.
def _contiguous(name: str, t: torch.Tensor, dtype, ndim: int, index: int) -> int:
    """The address of a contiguous tensor of this type on CUDA device ``index``."""
    if t.dtype is dtype and t.get_device() == index and t.dim() == ndim and t.is_contiguous():
        return t.data_ptr()
    _refuse(name, t, dtype, ndim, index)


def _refuse(name, t, dtype, ndim, index):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be a contiguous {ndim}-d tensor")


def _device(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    return index


def _int32(x: int) -> int:
    """``x`` for a C int: a value beyond its range becomes the range's end, or -1, which the library judges as it would ``x``
    (ctypes alone would pass its low 32 bits)."""
    return x if -1 <= x <= 0x7fffffff else 0x7fffffff if x > 0 else -1


def _launch(fn, name, index, stream, *args):
    """Call ``fn(*args, stream)`` with the tensors' device current."""
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st != GDN_OK:
        raise GdnError(st, name)


def _empty(stream, shape, dtype, device) -> torch.Tensor:
    """Memory for what a call writes, from the pool of the stream that it runs on: memory of another stream could still be
    in use there, or be given away there while the call runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _token_rows(name: str, t: torch.Tensor, heads: int, d: int, index: int) -> Tuple[int, int]:
    """Address and token stride of a bf16 [T, heads, d] tensor whose head vectors are contiguous."""
    if t.dtype is not torch.bfloat16 or t.get_device() != index or t.dim() != 3:
        _refuse(name, t, torch.bfloat16, 3, index)
    shape, stride = t.shape, t.stride()
    if shape[1] != heads or shape[2] != d:
        raise ValueError(f"{name} must be [tokens, {heads}, {d}], got {tuple(shape)}")
    if stride[2] != 1 or (heads > 1 and stride[1] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * d       # (a single token's stride says nothing)


def _pool(k_pages, v_pages, k_scales, v_scales, block_table, index):
    """Checked (addresses, (table address, max_pages, n_pages, page_size, format), hkv, d) of a cache."""
    dtype = k_pages.dtype
    fmt = FORMAT.get(dtype)
    if fmt is None:
        raise ValueError(f"k_pages must be int8 or float8_e4m3fn, got {dtype}")
    addresses = (_contiguous("k_pages", k_pages, dtype, 4, index), _contiguous("v_pages", v_pages, dtype, 4, index),
                 _contiguous("k_scales", k_scales, torch.float32, 3, index),
                 _contiguous("v_scales", v_scales, torch.float32, 3, index))
    table = _contiguous("block_table", block_table, torch.int32, 2, index)
    shape = k_pages.shape
    n_pages, hkv, page, d = shape
    if v_pages.shape != shape:
        raise ValueError("v_pages must have the shape of k_pages")
    scales = k_scales.shape
    if scales != (n_pages, hkv, page // KV_BLOCK) or v_scales.shape != scales:
        raise ValueError(f"k_scales and v_scales must be {(n_pages, hkv, page // KV_BLOCK)}")
    return addresses, (table, block_table.size(1), n_pages, page, fmt), hkv, d


def alloc_cache(n_pages: int, hkv: int, page_size: int, d: int, n_slots: int, dtype=torch.int8, device="cuda"):
    """An empty cache: ``(k_pages, v_pages, k_scales, v_scales, open_blocks)`` in the layouts of include/gdn.h."""
    pages = [torch.zeros(n_pages, hkv, page_size, d, dtype=torch.int8, device=device).view(dtype) for _ in range(2)]
    scales = [torch.zeros(n_pages, hkv, page_size // KV_BLOCK, dtype=torch.float32, device=device) for _ in range(2)]
    return (*pages, *scales, torch.zeros(n_slots, 2, hkv, KV_BLOCK, d, dtype=torch.bfloat16, device=device))


def kv_append(k: torch.Tensor, v: torch.Tensor, cos: Optional[torch.Tensor], sin: Optional[torch.Tensor],
              cu_seqlens: torch.Tensor, past_lens: torch.Tensor, block_table: torch.Tensor, k_pages: torch.Tensor,
              v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor, open_in: torch.Tensor, *,
              open_out: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None, interleaved: bool = False,
              stream=None) -> Tuple[Optional[torch.Tensor], torch.Tensor]:
    """Run ``gdn_kv_append``: rotate ``k`` (and ``q``) to positions ``past_lens[n], past_lens[n] + 1, ...`` and put
    ``k`` and ``v`` into the cache (updated in place).  Returns ``(rotated q or None, open_out)``.

    ``k``, ``v``, ``q`` are bf16 [T, heads, d]; they may be slices of one projection (head vectors contiguous, any
    token stride that is a multiple of 8).  ``cos`` / ``sin``: fp32 [positions, rot / 2], or None for no rotation.
    ``open_in`` (bf16 [slots, 2, hkv, 16, d]) holds each sequence's unfinished block; ``open_out`` defaults to
    updating it in place.  ``q_out`` may be ``q``."""
    lib = load_library()
    dev = _device(k, "k")
    pages, pool, hkv, d = _pool(k_pages, v_pages, k_scales, v_scales, block_table, dev)
    T = k.size(0)
    kp, k_stride = _token_rows("k", k, hkv, d, dev)
    vp, v_stride = _token_rows("v", v, hkv, d, dev)
    if v.size(0) != T:
        raise ValueError("k and v must have the same tokens")
    cu = _contiguous("cu_seqlens", cu_seqlens, torch.int32, 1, dev)
    past = _contiguous("past_lens", past_lens, torch.int32, 1, dev)
    n = past_lens.size(0)
    if cu_seqlens.size(0) != n + 1 or block_table.size(0) != n:
        raise ValueError("cu_seqlens, past_lens and block_table must describe the same sequences")
    rot = positions = cp = sp = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        cp = _contiguous("cos", cos, torch.float32, 2, dev)
        sp = _contiguous("sin", sin, torch.float32, 2, dev)
        positions, half = cos.shape
        if sin.shape != (positions, half):
            raise ValueError("cos and sin must have the same shape")
        rot = 2 * half
    oo = op = _contiguous("open_in", open_in, torch.bfloat16, 5, dev)
    n_slots = open_in.size(0)
    opened = (n_slots, 2, hkv, KV_BLOCK, d)
    if open_in.shape != opened:
        raise ValueError(f"open_in must be [slots, 2, {hkv}, {KV_BLOCK}, {d}]")
    if open_out is None:
        open_out = open_in
    else:
        oo = _contiguous("open_out", open_out, torch.bfloat16, 5, dev)
        if open_out.shape != opened:
            raise ValueError("open_out must have the shape of open_in")
    sl = 0
    if slots is not None:
        sl = _contiguous("slots", slots, torch.int32, 1, dev)
        if slots.size(0) != n:
            raise ValueError("slots must name one slot for each sequence")
    hq = qp = q_stride = qo = 0
    if q is not None:
        hq = q.size(1) if q.dim() == 3 else 0
        qp, q_stride = _token_rows("q", q, hq, d, dev)
        if q.size(0) != T:
            raise ValueError("q and k must have the same tokens")
        if q_out is None:
            q_out = _empty(stream, (T, hq, d), torch.bfloat16, q.device)
            qo = q_out.data_ptr()
        else:
            qo = _contiguous("q_out", q_out, torch.bfloat16, 3, dev)
            if q_out.shape != (T, hq, d):
                raise ValueError("q_out must have the shape of q")
        if T == 0:
            qp = qo = 0
    elif q_out is not None:
        raise ValueError("q_out without q")
    _launch(lib.gdn_kv_append, "gdn_kv_append", dev, stream, n, T, hq, hkv, d, rot, qp, q_stride, kp, k_stride, vp,
            v_stride, cp, sp, positions, int(bool(interleaved)), cu, past, *pool, *pages, op, oo, sl,
            n_slots, qo)
    return q_out, open_out


def kv_read(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
            block_table: torch.Tensor, cu_tokens: torch.Tensor, total_tokens: int, *, out_dtype=torch.bfloat16,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Run ``gdn_kv_read``: the values of the first ``cu_tokens[n + 1] - cu_tokens[n]`` tokens of every sequence,
    packed: ``(k, v)``, each [total_tokens, hkv, d].  ``total_tokens`` is ``cu_tokens``'s last entry, known on the
    host."""
    lib = load_library()
    dev = _device(k_pages, "k_pages")
    pages, pool, hkv, d = _pool(k_pages, v_pages, k_scales, v_scales, block_table, dev)
    cu = _contiguous("cu_tokens", cu_tokens, torch.int32, 1, dev)
    n = cu_tokens.size(0) - 1
    if block_table.size(0) != n:
        raise ValueError("cu_tokens and block_table must describe the same sequences")
    out_code = DTYPE.get(out_dtype)
    if out_code is None:
        raise ValueError("out_dtype must be bf16 or fp32")
    shape, device = (total_tokens, hkv, d), k_pages.device
    k, v = _empty(stream, shape, out_dtype, device), _empty(stream, shape, out_dtype, device)
    _launch(lib.gdn_kv_read, "gdn_kv_read", dev, stream, n, total_tokens, hkv, d, cu, *pool, *pages, k.data_ptr(),
            v.data_ptr(), out_code)
    return k, v


@functools.lru_cache(maxsize=4096)
def attend_workspace_size(n_seqs: int, total_tokens: int, hq: int, hkv: int, d: int, max_q_len: int,
                          max_kv_len: int) -> int:
    """Bytes of workspace that :func:`attend` needs for this problem (``gdn_attend_workspace_size``)."""
    st = ctypes.c_int(0)
    sizes = map(_int32, (n_seqs, total_tokens, hq, hkv, d, max_q_len, max_kv_len))
    need = load_library().gdn_attend_workspace_size(*sizes, st)
    if st.value != GDN_OK:
        raise GdnError(st.value, "gdn_attend_workspace_size")
    return int(need)


def attend(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
           v_scales: torch.Tensor, block_table: torch.Tensor, cu_seqlens: torch.Tensor, kv_lens: torch.Tensor, *,
           max_q_len: int, max_kv_len: int, sm_scale: Optional[float] = None, window: int = 0, sinks: int = 0,
           out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16, workspace: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """Run ``gdn_attend``: causal attention of the queries ``q`` (bf16 [T, hq, d], rotated) over the cache, which
    already holds their own keys and values.  ``kv_lens`` (int32 [n]) counts each sequence's cached tokens;
    ``max_q_len`` and ``max_kv_len`` bound the device values.  With ``window`` a query sees the last ``window``
    tokens (its own included) and the first ``sinks``.  ``sm_scale`` defaults to 1 / sqrt(d)."""
    lib = load_library()
    dev = _device(q, "q")
    pages, pool, hkv, d = _pool(k_pages, v_pages, k_scales, v_scales, block_table, dev)
    qp = _contiguous("q", q, torch.bfloat16, 3, dev)
    shape = q.shape
    T, hq, width = shape
    if width != d:
        raise ValueError(f"q must be [tokens, heads, {d}], got {tuple(shape)}")
    cu = _contiguous("cu_seqlens", cu_seqlens, torch.int32, 1, dev)
    lens = _contiguous("kv_lens", kv_lens, torch.int32, 1, dev)
    n = kv_lens.size(0)
    if cu_seqlens.size(0) != n + 1 or block_table.size(0) != n:
        raise ValueError("cu_seqlens, kv_lens and block_table must describe the same sequences")
    if out is not None:
        out_dtype = out.dtype
        op = _contiguous("out", out, out_dtype, 3, dev)
    out_code = DTYPE.get(out_dtype)
    if out_code is None or (out is not None and out.shape != shape):
        raise ValueError("out must have the shape of q, in bf16 or fp32")
    if out is None:
        out = _empty(stream, shape, out_dtype, q.device)
        op = out.data_ptr()
    if max_q_len > T:
        max_q_len = T
    if workspace is None:
        ws_bytes = attend_workspace_size(n, T, hq, hkv, d, max_q_len, max_kv_len)
        workspace = _empty(stream, ws_bytes, torch.uint8, q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    else:
        ws_bytes = workspace.numel() * workspace.element_size()
    table, max_pages, n_pages, page, fmt = pool
    _launch(lib.gdn_attend, "gdn_attend", dev, stream, n, T, hq, hkv, d, qp, *pages, table, max_pages, n_pages, page,
            fmt, cu, lens, _int32(max_q_len), _int32(max_kv_len), 1.0 / math.sqrt(d) if sm_scale is None else sm_scale,
            _int32(window), _int32(sinks), op, out_code, workspace.data_ptr(), ws_bytes)
    return out
