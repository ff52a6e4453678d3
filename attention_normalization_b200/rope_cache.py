"""Headwise QK-Norm with the position rotation, its gradient, the append to a
paged cache and attention over the 4-bit cache: marshalling for the entry
points of the same names in ``include/qknorm.h``, where layouts, padding rules
and errors are stated.

Rows are 2-D views as everywhere in this package.  ``cos_sin`` is the fp32
table ``[table_rows, rotary_dim]`` (cosines, then sines, of each position),
``positions`` and ``slots`` are int64 ``[T]``.  The calls record nothing for
autograd and refuse operands that it would have to follow: a training step calls
them in the ``forward`` of a ``torch.autograd.Function`` (or under
``torch.no_grad()``) and ``qknorm_headwise_rope_backward`` in its ``backward``.  A
step of serving:

    q = qknorm_rope_append_kv4(q, k, v, gamma_q, gamma_k, cos_sin, positions, cache, slots)
    o = qknorm_kv4_attention(q, cache, block_table, seq_lens, max_seq_len=longest)
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _DTYPES, _clib, _on, _raw_current_stream, _rows, _stream_handle, _used_on, capi, gamma_dtype

# These calls are short on the GPU, so what they look at on the host is kept
# small: each operand once, its device as a number, what is made here not at all.

_Tensor = torch.Tensor
_GAMMA = {dt: gamma_dtype(dt) for dt in _DTYPES}
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, where, index, stream, *args):
    """`fn(*args, stream)` with device `index` current."""
    if stream is None and _raw_current_stream is not None and index == _current_device():
        st = fn(*args, _raw_current_stream(index))
    else:
        dev = torch.device("cuda", index)
        with _on(dev):
            st = fn(*args, _stream_handle(stream, dev))
    if st:
        _clib.check(st, where)


def _first(t, name):
    """(T, width, row stride, device number, type) of the rows that the call's
    other operands have to go with."""
    T, W, s = _rows(t, name)
    return T, W, s, t.get_device(), t.dtype


def _like(t, name, index, dt):
    """(T, width, row stride) of the rows `t`, on device `index` and of type `dt`."""
    if not isinstance(t, _Tensor) or t.dtype is not dt or t.get_device() != index:
        raise ValueError(f"{name} must be a tensor on cuda:{index} with dtype {dt}")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D [T, width]")
    T, W = shape
    s0, s1 = t.stride()
    if s1 != 1 and T > 0 and W > 1:
        raise ValueError(f"{name} rows must be unit-stride along the width")
    return T, W, (s0 if T > 1 else max(s0, W))


def _match(t, name, index, dt, T, W, stride=None):
    """Row stride of the [T, W] rows `t`, which has to be `stride` where that is given."""
    To, Wo, s = _like(t, name, index, dt)
    if To != T or Wo != W:
        raise ValueError(f"{name} must be [{T}, {W}]")
    if stride is not None and s != stride and T > 1:
        raise ValueError(f"{name} must match its input's row stride")
    return s


def _flat(t, name, n, dtype, index):
    """Pointer of a contiguous tensor of `n` elements."""
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.get_device() != index or t.numel() != n \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of {n} elements on cuda:{index}")
    return t.data_ptr()


def _int32(**sizes):
    """Refuses sizes that the library's 32-bit arguments cannot hold: ctypes would cut them off."""
    for name, n in sizes.items():
        if not -1 << 31 <= n < 1 << 31:
            raise ValueError(f"{name} = {n} must be below 2**31")


def _table(cos_sin, index):
    if not isinstance(cos_sin, _Tensor) or cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index \
            or len(cos_sin.shape) != 2 or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be a contiguous float32 CUDA tensor [table_rows, rotary_dim] on cuda:{index}")
    P, rot = cos_sin.shape
    return cos_sin.data_ptr(), P, rot


def _heads(width, head_dim, name):
    if head_dim < 1 or width % head_dim:
        raise ValueError(f"{name}: the row width must be a whole number of heads of head_dim elements")
    return width // head_dim


_grad_enabled = torch.is_grad_enabled


def _untracked(where, *tensors):
    """Refuses tensors whose gradient autograd follows: outputs would lose it silently."""
    for t in tensors:
        if isinstance(t, _Tensor) and t.requires_grad:
            raise ValueError(f"{where} records nothing for autograd and an operand requires a gradient: call it under "
                             "torch.no_grad() or in the forward of a torch.autograd.Function")


def qknorm_headwise_rope(q_in: torch.Tensor, k_in: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor,
                         head_dim: int, cos_sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6, *,
                         interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Headwise QK-Norm and position rotation of every Q and K head in one
    launch; returns ``(q_out, k_out)``.  ``interleaved`` rotates the pairs
    ``(2i, 2i + 1)`` instead of ``(i, i + rotary_dim / 2)``."""
    if _grad_enabled():
        _untracked("qknorm_headwise_rope", q_in, k_in, gamma_q, gamma_k, cos_sin)
    T, Wq, sq, dev, dt = _first(q_in, "q_in")
    Tk, Wk, sk = _like(k_in, "k_in", dev, dt)
    if T != Tk:
        raise ValueError("q_in and k_in must have the same number of tokens")
    table, P, rot = _table(cos_sin, dev)
    pos = _flat(positions, "positions", T, torch.int64, dev)
    gdt = _GAMMA[dt]
    gq, gk = _flat(gamma_q, "gamma_q", head_dim, gdt, dev), _flat(gamma_k, "gamma_k", head_dim, gdt, dev)
    if q_out is None:
        q_out = q_in.new_empty_strided((T, Wq), (sq, 1))
        _used_on(stream, q_out)
    else:
        _match(q_out, "q_out", dev, dt, T, Wq, sq)
    if k_out is None:
        k_out = k_in.new_empty_strided((T, Wk), (sk, 1))
        _used_on(stream, k_out)
    else:
        _match(k_out, "k_out", dev, dt, T, Wk, sk)
    _call(capi().qknorm_headwise_rope, "qknorm_headwise_rope", dev, stream,
          q_in.data_ptr(), q_out.data_ptr(), gq, sq, _heads(Wq, head_dim, "q_in"), k_in.data_ptr(), k_out.data_ptr(),
          gk, sk, _heads(Wk, head_dim, "k_in"), T, head_dim, table, P, rot, 1 if interleaved else 0, pos, eps,
          _DTYPES[dt])
    return q_out, k_out


def rope_backward_workspace_bytes(T: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    """Workspace ``qknorm_headwise_rope_backward`` needs."""
    _int32(q_heads=q_heads, k_heads=k_heads, head_dim=head_dim)
    n = capi().qknorm_headwise_rope_backward_workspace_bytes(T, q_heads, k_heads, head_dim)
    if n < 0:
        raise ValueError("invalid sizes for the gradient's workspace")
    return n


def _workspace(workspace, dev):
    """Pointer and bytes of a caller's workspace."""
    if not isinstance(workspace, _Tensor) or workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def qknorm_headwise_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q_in: torch.Tensor, k_in: torch.Tensor,
                                  gamma_q: torch.Tensor, gamma_k: torch.Tensor, head_dim: int, cos_sin: torch.Tensor,
                                  positions: torch.Tensor, eps: float = 1e-6, *, interleaved: bool = False, dq_in=None,
                                  dk_in=None, dgamma_q=None, dgamma_k=None, workspace=None, stream=None):
    """Gradient of ``qknorm_headwise_rope``: ``dq_out`` and ``dk_out`` are the
    gradients of its outputs, ``q_in`` and ``k_in`` the rows it read.  Returns
    ``(dq_in, dk_in, dgamma_q, dgamma_k)``, the last two fp32 ``[head_dim]``
    summed over tokens and heads (overwritten, not accumulated)."""
    if _grad_enabled():  # a gradient of this gradient
        _untracked("qknorm_headwise_rope_backward", dq_out, dk_out)
    T, Wq, sq, dev, dt = _first(q_in, "q_in")
    Tk, Wk, sk = _like(k_in, "k_in", dev, dt)
    if T != Tk:
        raise ValueError("q_in and k_in must have the same number of tokens")
    hq, hk = _heads(Wq, head_dim, "q_in"), _heads(Wk, head_dim, "k_in")
    table, P, rot = _table(cos_sin, dev)
    pos = _flat(positions, "positions", T, torch.int64, dev)
    gdt, f32 = _GAMMA[dt], torch.float32
    gq, gk = _flat(gamma_q, "gamma_q", head_dim, gdt, dev), _flat(gamma_k, "gamma_k", head_dim, gdt, dev)
    dqs, dks = _match(dq_out, "dq_out", dev, dt, T, Wq), _match(dk_out, "dk_out", dev, dt, T, Wk)
    made = []
    if dq_in is None:
        made.append(dq_in := q_in.new_empty((T, Wq)))
        dqi = Wq
    else:
        dqi = _match(dq_in, "dq_in", dev, dt, T, Wq)
    if dk_in is None:
        made.append(dk_in := k_in.new_empty((T, Wk)))
        dki = Wk
    else:
        dki = _match(dk_in, "dk_in", dev, dt, T, Wk)
    if dgamma_q is None and dgamma_k is None:
        dgamma_q, dgamma_k = made_g = cos_sin.new_empty((2, head_dim)).unbind(0)
        made += made_g
    elif dgamma_q is None:
        made.append(dgamma_q := cos_sin.new_empty((head_dim,)))
    elif dgamma_k is None:
        made.append(dgamma_k := cos_sin.new_empty((head_dim,)))
    pgq, pgk = _flat(dgamma_q, "dgamma_q", head_dim, f32, dev), _flat(dgamma_k, "dgamma_k", head_dim, f32, dev)
    lib = capi()
    if workspace is None:
        need = lib.qknorm_headwise_rope_backward_workspace_bytes(T, hq, hk, head_dim)
        made.append(workspace := cos_sin.new_empty((max(need, 16) // 4,)))
        ws, ws_bytes = workspace.data_ptr(), max(need, 16)
    else:
        ws, ws_bytes = _workspace(workspace, dev)
    _used_on(stream, *made)
    _call(lib.qknorm_headwise_rope_backward, "qknorm_headwise_rope_backward", dev, stream,
          q_in.data_ptr(), sq, dq_out.data_ptr(), dqs, dq_in.data_ptr(), dqi, gq, pgq, hq,
          k_in.data_ptr(), sk, dk_out.data_ptr(), dks, dk_in.data_ptr(), dki, gk, pgk, hk,
          T, head_dim, table, P, rot, 1 if interleaved else 0, pos, eps, ws, ws_bytes, _DTYPES[dt])
    return dq_in, dk_in, dgamma_q, dgamma_k


# --------------------------------------------------------------------------- paged caches

_Strides = ctypes.c_int64 * 3


def _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out, interleaved, stream):
    """The arguments the two append calls share, the query output, T, kv heads, the device and the type."""
    T, Wk, sk, dev, dt = _first(k_in, "k_in")
    sv = _match(v_in, "v_in", dev, dt, T, Wk)
    hk = _heads(Wk, head_dim, "k_in")
    table, P, rot = _table(cos_sin, dev)
    pos = _flat(positions, "positions", T, torch.int64, dev)
    if (gamma_k is None) != (gamma_q is None) and q_in is not None:
        raise ValueError("gamma_q and gamma_k: both (norm and rotation) or neither (rotation only)")
    gdt = _GAMMA[dt]
    gq = None if gamma_q is None else _flat(gamma_q, "gamma_q", head_dim, gdt, dev)
    gk = None if gamma_k is None else _flat(gamma_k, "gamma_k", head_dim, gdt, dev)
    if q_in is None:
        qp, qo, sq, hq, q_out = None, None, 0, 0, None
    else:
        Tq, Wq, sq = _like(q_in, "q_in", dev, dt)
        if Tq != T:
            raise ValueError("q_in and k_in must have the same number of tokens")
        hq = _heads(Wq, head_dim, "q_in")
        if q_out is None:
            q_out = q_in.new_empty_strided((T, Wq), (sq, 1))
            _used_on(stream, q_out)
        else:
            _match(q_out, "q_out", dev, dt, T, Wq, sq)
        qp, qo = q_in.data_ptr(), q_out.data_ptr()
    args = (qp, qo, gq, sq, hq, k_in.data_ptr(), gk, sk, v_in.data_ptr(), sv, hk, T, head_dim, table, P, rot,
            1 if interleaved else 0, pos)
    return args, q_out, T, hk, dev, dt


def qknorm_rope_append(q_in, k_in: torch.Tensor, v_in: torch.Tensor, gamma_q, gamma_k, head_dim: int,
                       cos_sin: torch.Tensor, positions: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       slots: torch.Tensor, eps: float = 1e-6, *, interleaved: bool = False, q_out=None, stream=None):
    """Headwise norm and rotation of Q and K rows, the keys and values going to
    the paged caches; returns ``q_out``.

    ``k_cache`` and ``v_cache`` are indexed ``[page, token, head, dim]`` with any
    strides but the last (a heads-first cache is passed as
    ``cache.transpose(1, 2)``); token t goes to page ``slots[t] // page_size``,
    place ``slots[t] % page_size``, and nowhere where that lies outside the
    cache.  ``gamma_q`` and ``gamma_k`` of ``None`` leave the norm out, ``q_in``
    of ``None`` the Q rows."""
    if _grad_enabled():
        _untracked("qknorm_rope_append", q_in, k_in, v_in, gamma_q, gamma_k, cos_sin)
    args, q_out, T, hk, dev, dt = _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out,
                                               interleaved, stream)
    pages = k_cache.shape[:2]
    strides = []
    for c, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if not isinstance(c, _Tensor) or c.dtype is not dt or c.get_device() != dev:
            raise ValueError(f"{name} must be a tensor on cuda:{dev} with dtype {dt}")
        shape, stride = c.shape, c.stride()
        if len(shape) != 4 or shape[2] != hk or shape[3] != head_dim or (head_dim > 1 and stride[3] != 1):
            raise ValueError(f"{name} must be [pages, page_size, {hk}, {head_dim}] with unit stride along the last")
        if shape[:2] != pages:
            raise ValueError("k_cache and v_cache must have the same pages")
        strides.append(_Strides(stride[0], stride[1], stride[2]))
    s = _flat(slots, "slots", T, torch.int64, dev)
    _call(capi().qknorm_rope_append, "qknorm_rope_append", dev, stream, *args, k_cache.data_ptr(), strides[0],
          v_cache.data_ptr(), strides[1], *pages, s, eps, _DTYPES[dt])
    return q_out


class Kv4Cache(NamedTuple):
    """A 4-bit paged cache: codes ``[pages, kv_heads, page_size, head_dim / 2]``
    uint8 and scales ``[pages, kv_heads, page_size, head_dim / 64]`` float16 of
    the keys, then of the values.  Any tuple of four such tensors will do."""
    k_codes: torch.Tensor
    k_scales: torch.Tensor
    v_codes: torch.Tensor
    v_scales: torch.Tensor


def kv4_cache(num_pages: int, page_size: int, kv_heads: int, head_dim: int, device) -> Kv4Cache:
    """An empty 4-bit cache (every element zero)."""
    if head_dim not in (64, 128, 256) or page_size < 1 or page_size % 16:
        raise ValueError("the 4-bit cache takes head_dim 64, 128 or 256 and a page_size that is a multiple of 16")

    def codes():
        return torch.full((num_pages, kv_heads, page_size, head_dim // 2), 0x88, dtype=torch.uint8, device=device)

    def scales():
        return torch.zeros((num_pages, kv_heads, page_size, head_dim // 64), dtype=torch.float16, device=device)
    return Kv4Cache(codes(), scales(), codes(), scales())


def _kv4_args(cache, dev):
    """The cache's pointers and ``(num_pages, page_size, kv_heads, head_dim)``."""
    kc, ks, vc, vs = cache
    pages, hk, ps, half = shape = kc.shape
    n = pages * hk * ps
    ptrs = (_flat(kc, "k_codes", n * half, torch.uint8, dev), _flat(ks, "k_scales", n * half // 32, torch.float16, dev),
            _flat(vc, "v_codes", n * half, torch.uint8, dev), _flat(vs, "v_scales", n * half // 32, torch.float16, dev))
    if vc.shape != shape or ks.shape != vs.shape or ks.shape != (pages, hk, ps, half // 32):
        raise ValueError("the cache's codes must be [pages, kv_heads, page_size, head_dim / 2] and its scales "
                         "[pages, kv_heads, page_size, head_dim / 64]")
    return ptrs, (pages, ps, hk, 2 * half)


def qknorm_rope_append_kv4(q_in, k_in: torch.Tensor, v_in: torch.Tensor, gamma_q, gamma_k, cos_sin: torch.Tensor,
                           positions: torch.Tensor, cache, slots: torch.Tensor, eps: float = 1e-6, *,
                           interleaved: bool = False, q_out=None, stream=None):
    """``qknorm_rope_append`` into a 4-bit cache (``kv4_cache``); returns ``q_out``."""
    if _grad_enabled():
        _untracked("qknorm_rope_append_kv4", q_in, k_in, v_in, gamma_q, gamma_k, cos_sin)
    if not isinstance(k_in, _Tensor) or not k_in.is_cuda:
        raise ValueError("k_in must be a CUDA tensor (this library has no CPU path)")
    ptrs, (pages, ps, heads, head_dim) = _kv4_args(cache, k_in.get_device())
    args, q_out, T, hk, dev, dt = _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out,
                                               interleaved, stream)
    if hk != heads:
        raise ValueError(f"k_in has {hk} heads, the cache {heads}")
    s = _flat(slots, "slots", T, torch.int64, dev)
    _call(capi().qknorm_rope_append_kv4, "qknorm_rope_append_kv4", dev, stream, *args, *ptrs, pages, ps, s, eps,
          _DTYPES[dt])
    return q_out


def qknorm_kv4_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, *, k_out=None, v_out=None,
                    stream=None):
    """The cached tokens at ``slots`` as K and V rows ``[n, kv_heads * head_dim]``
    of ``dtype`` (zeros for a slot outside the cache)."""
    if not isinstance(slots, _Tensor) or not slots.is_cuda:
        raise ValueError("slots must be a CUDA tensor (this library has no CPU path)")
    dev, n = slots.get_device(), slots.numel()
    ptrs, (pages, ps, hk, d) = _kv4_args(cache, dev)
    if dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError(f"dtype {dtype} unsupported (float32, bfloat16, float16)")
    s = _flat(slots, "slots", n, torch.int64, dev)
    W = hk * d
    made = []
    if k_out is None:
        made.append(k_out := slots.new_empty((n, W), dtype=dtype))
        sk = W
    else:
        sk = _match(k_out, "k_out", dev, dtype, n, W)
    if v_out is None:
        made.append(v_out := slots.new_empty((n, W), dtype=dtype))
        sv = W
    else:
        sv = _match(v_out, "v_out", dev, dtype, n, W)
    _used_on(stream, *made)
    _call(capi().qknorm_kv4_read, "qknorm_kv4_read", dev, stream, *ptrs, pages, ps, hk, d, s, n, k_out.data_ptr(), sk,
          v_out.data_ptr(), sv, _DTYPES[dtype])
    return k_out, v_out


def kv4_attention_workspace_bytes(T: int, batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int,
                                  max_seq_len: int) -> int:
    """Workspace that serves every ``qknorm_kv4_attention`` with these heads and
    at most this batch, ``max_q_len`` and ``max_seq_len``."""
    _int32(batch=batch, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, max_q_len=max_q_len, max_seq_len=max_seq_len)
    n = capi().qknorm_kv4_attention_workspace_bytes(T, batch, q_heads, kv_heads, head_dim, max_q_len, max_seq_len)
    if n < 0:
        raise ValueError("invalid sizes for the attention's workspace")
    return n


def qknorm_kv4_attention(q: torch.Tensor, cache, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                         max_seq_len: int, q_start=None, max_q_len: int = 1, softmax_scale: float | None = None,
                         window: int = 0, out=None, lse=None, return_lse: bool = False, workspace=None, stream=None):
    """Causal attention of the rows of ``q`` ``[T, q_heads * head_dim]`` over
    the 4-bit cache; returns ``out``, or ``(out, lse)`` with ``return_lse``.

    ``block_table`` int32 ``[B, max_pages]``, ``seq_lens`` int32 ``[B]`` (the
    rows' own tokens counted), ``q_start`` int32 ``[B + 1]`` or ``None`` for one
    row per sequence.  ``max_seq_len`` and ``max_q_len`` are bounds the host
    knows (longer sequences are cut there).  ``window`` > 0 limits a row to that
    many last tokens.  Rows of no sequence are left as they were in ``out`` and
    ``lse`` (unspecified where these are made here)."""
    if _grad_enabled():
        _untracked("qknorm_kv4_attention", q)
    if (max_seq_len | max_q_len | window) >> 31:
        _int32(max_seq_len=max_seq_len, max_q_len=max_q_len, window=window)
    T, W, sq, dev, dt = _first(q, "q")
    ptrs, (pages, ps, hk, d) = _kv4_args(cache, dev)
    hq = _heads(W, d, "q")
    if not isinstance(block_table, torch.Tensor) or len(block_table.shape) != 2:
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    i32 = torch.int32
    bt = _flat(block_table, "block_table", B * max_pages, i32, dev)
    sl = _flat(seq_lens, "seq_lens", B, i32, dev)
    qs = None if q_start is None else _flat(q_start, "q_start", B + 1, i32, dev)
    made = []
    if out is None:
        made.append(out := q.new_empty((T, W)))
        so = W
    else:
        so = _match(out, "out", dev, dt, T, W)
    if lse is not None:
        lp = _flat(lse, "lse", T * hq, torch.float32, dev)
    elif return_lse:
        made.append(lse := q.new_empty((T, hq), dtype=torch.float32))
        lp = lse.data_ptr()
    else:
        lp = None
    lib = capi()
    if workspace is None:
        need = lib.qknorm_kv4_attention_workspace_bytes(T, B, hq, hk, d, max_q_len, max_seq_len)
        if need > 0:
            made.append(workspace := block_table.new_empty((need // 4,)))
            ws, ws_bytes = workspace.data_ptr(), need
        else:
            ws, ws_bytes = None, 0
    else:
        ws, ws_bytes = _workspace(workspace, dev)
    _used_on(stream, *made)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
    _call(lib.qknorm_kv4_attention, "qknorm_kv4_attention", dev, stream, q.data_ptr(), sq, out.data_ptr(), so, lp, hq,
          *ptrs, pages, ps, hk, d, bt, max_pages, sl, qs, T, B, max_q_len, max_seq_len, window, scale, ws, ws_bytes,
          _DTYPES[dt])
    return (out, lse) if return_lse else out
