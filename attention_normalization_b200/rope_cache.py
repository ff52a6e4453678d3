"""Headwise QK-Norm with the position rotation, its gradient, the append to a
paged cache and attention over the 4-bit cache: marshalling for the entry
points of the same names in ``include/qknorm.h``, where layouts, padding rules
and errors are stated.

Rows are 2-D views as everywhere in this package.  ``cos_sin`` is the fp32
table ``[table_rows, rotary_dim]`` (cosines, then sines, of each position),
``positions`` and ``slots`` are int64 ``[T]``.  A step of serving:

    q = qknorm_rope_append_kv4(q, k, v, gamma_q, gamma_k, cos_sin, positions, cache, slots)
    o = qknorm_kv4_attention(q, cache, block_table, seq_lens, max_seq_len=longest)
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple

import torch

from . import _DTYPES, _clib, _on, _out_like, _rows, _same, _stream_handle, _vec, capi, gamma_dtype


def _ints(t, name, n, dtype, device):
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == device and t.dtype == dtype and t.is_contiguous()
            and t.numel() == n):
        raise ValueError(f"{name} must be a contiguous CUDA {dtype} tensor of {n} elements on {device}")
    return t.data_ptr()


def _table(cos_sin, positions, T, device):
    if not (isinstance(cos_sin, torch.Tensor) and cos_sin.is_cuda and cos_sin.device == device
            and cos_sin.dtype == torch.float32 and cos_sin.dim() == 2 and cos_sin.is_contiguous()):
        raise ValueError(f"cos_sin must be a contiguous float32 CUDA tensor [table_rows, rotary_dim] on {device}")
    return [cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1]], _ints(positions, "positions", T, torch.int64, device)


def _heads(width, head_dim, name):
    if head_dim < 1 or width % head_dim:
        raise ValueError(f"{name}: the row width must be a whole number of heads of head_dim elements")
    return width // head_dim


def _rows_like(t, name, like, shape):
    """Stride of `t`, rows of `shape` on the device and of the type of `like`."""
    _same(like.device, like.dtype, t, name)
    To, W, s = _rows(t, name)
    if (To, W) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}")
    return s


def _used_on(stream, *tensors):
    """Tensors allocated here on the current stream but used on `stream`: the
    allocator must not hand them out again before that stream is done."""
    if isinstance(stream, torch.cuda.Stream):
        for t in tensors:
            t.record_stream(stream)


def _out_rows(out, name, like, shape, stride, stream):
    if out is None:
        out = _out_like(like, stride)
        _used_on(stream, out)
        return out
    if _rows_like(out, name, like, shape) != stride and shape[0] > 1:
        raise ValueError(f"{name} must match its input's shape and row stride")
    return out


def qknorm_headwise_rope(q_in: torch.Tensor, k_in: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor,
                         head_dim: int, cos_sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6, *,
                         interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Headwise QK-Norm and position rotation of every Q and K head in one
    launch; returns ``(q_out, k_out)``.  ``interleaved`` rotates the pairs
    ``(2i, 2i + 1)`` instead of ``(i, i + rotary_dim / 2)``."""
    T, Wq, sq = _rows(q_in, "q_in")
    Tk, Wk, sk = _rows(k_in, "k_in")
    if T != Tk:
        raise ValueError("q_in and k_in must have the same number of tokens")
    dev, dt = q_in.device, q_in.dtype
    _same(dev, dt, k_in, "k_in")
    hq, hk = _heads(Wq, head_dim, "q_in"), _heads(Wk, head_dim, "k_in")
    table, pos = _table(cos_sin, positions, T, dev)
    q_out = _out_rows(q_out, "q_out", q_in, (T, Wq), sq, stream)
    k_out = _out_rows(k_out, "k_out", k_in, (T, Wk), sk, stream)
    gdt = gamma_dtype(dt)
    with _on(dev):
        st = capi().qknorm_headwise_rope(
            q_in.data_ptr(), q_out.data_ptr(), _vec(gamma_q, "gamma_q", head_dim, gdt, dev), sq, hq,
            k_in.data_ptr(), k_out.data_ptr(), _vec(gamma_k, "gamma_k", head_dim, gdt, dev), sk, hk, T, head_dim,
            *table, int(interleaved), pos, float(eps), _DTYPES[dt], _stream_handle(stream, dev))
    _clib.check(st, "qknorm_headwise_rope")
    return q_out, k_out


def rope_backward_workspace_bytes(T: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    """Workspace ``qknorm_headwise_rope_backward`` needs."""
    n = capi().qknorm_headwise_rope_backward_workspace_bytes(T, q_heads, k_heads, head_dim)
    if n < 0:
        raise ValueError("invalid sizes for the gradient's workspace")
    return n


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty((max(need, 16),), dtype=torch.uint8, device=dev)
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.device == dev
            and workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {dev}")
    return workspace


def qknorm_headwise_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q_in: torch.Tensor, k_in: torch.Tensor,
                                  gamma_q: torch.Tensor, gamma_k: torch.Tensor, head_dim: int, cos_sin: torch.Tensor,
                                  positions: torch.Tensor, eps: float = 1e-6, *, interleaved: bool = False, dq_in=None,
                                  dk_in=None, dgamma_q=None, dgamma_k=None, workspace=None, stream=None):
    """Gradient of ``qknorm_headwise_rope``: ``dq_out`` and ``dk_out`` are the
    gradients of its outputs, ``q_in`` and ``k_in`` the rows it read.  Returns
    ``(dq_in, dk_in, dgamma_q, dgamma_k)``, the last two fp32 ``[head_dim]``
    summed over tokens and heads (overwritten, not accumulated)."""
    T, Wq, sq = _rows(q_in, "q_in")
    Tk, Wk, sk = _rows(k_in, "k_in")
    if T != Tk:
        raise ValueError("q_in and k_in must have the same number of tokens")
    dev, dt = q_in.device, q_in.dtype
    _same(dev, dt, k_in, "k_in")
    hq, hk = _heads(Wq, head_dim, "q_in"), _heads(Wk, head_dim, "k_in")
    table, pos = _table(cos_sin, positions, T, dev)
    dqs, dks = _rows_like(dq_out, "dq_out", q_in, (T, Wq)), _rows_like(dk_out, "dk_out", k_in, (T, Wk))
    fresh = []
    if dq_in is None:
        fresh.append(dq_in := torch.empty((T, Wq), dtype=dt, device=dev))
    if dk_in is None:
        fresh.append(dk_in := torch.empty((T, Wk), dtype=dt, device=dev))
    dqi, dki = _rows_like(dq_in, "dq_in", q_in, (T, Wq)), _rows_like(dk_in, "dk_in", k_in, (T, Wk))
    if dgamma_q is None:
        fresh.append(dgamma_q := torch.empty((head_dim,), dtype=torch.float32, device=dev))
    if dgamma_k is None:
        fresh.append(dgamma_k := torch.empty((head_dim,), dtype=torch.float32, device=dev))
    need = capi().qknorm_headwise_rope_backward_workspace_bytes(T, hq, hk, head_dim)
    if workspace is None:
        fresh.append(workspace := _workspace(None, need, dev))
    workspace = _workspace(workspace, need, dev)
    _used_on(stream, *fresh)
    gdt = gamma_dtype(dt)
    f32 = torch.float32
    with _on(dev):
        st = capi().qknorm_headwise_rope_backward(
            q_in.data_ptr(), sq, dq_out.data_ptr(), dqs, dq_in.data_ptr(), dqi,
            _vec(gamma_q, "gamma_q", head_dim, gdt, dev), _vec(dgamma_q, "dgamma_q", head_dim, f32, dev), hq,
            k_in.data_ptr(), sk, dk_out.data_ptr(), dks, dk_in.data_ptr(), dki,
            _vec(gamma_k, "gamma_k", head_dim, gdt, dev), _vec(dgamma_k, "dgamma_k", head_dim, f32, dev), hk,
            T, head_dim, *table, int(interleaved), pos, float(eps), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _DTYPES[dt], _stream_handle(stream, dev))
    _clib.check(st, "qknorm_headwise_rope_backward")
    return dq_in, dk_in, dgamma_q, dgamma_k


# --------------------------------------------------------------------------- paged caches

def _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out, interleaved, stream):
    """The arguments the two append calls share, the query output and T, kv heads."""
    T, Wk, sk = _rows(k_in, "k_in")
    dev, dt = k_in.device, k_in.dtype
    sv = _rows_like(v_in, "v_in", k_in, (T, Wk))
    hk = _heads(Wk, head_dim, "k_in")
    table, pos = _table(cos_sin, positions, T, dev)
    gdt = gamma_dtype(dt)
    if (gamma_k is None) != (gamma_q is None) and q_in is not None:
        raise ValueError("gamma_q and gamma_k: both (norm and rotation) or neither (rotation only)")
    gq, gk = (None if g is None else _vec(g, name, head_dim, gdt, dev)
              for g, name in ((gamma_q, "gamma_q"), (gamma_k, "gamma_k")))
    if q_in is None:
        qp, qo, sq, hq = None, None, 0, 0
    else:
        _same(dev, dt, q_in, "q_in")
        Tq, Wq, sq = _rows(q_in, "q_in")
        if Tq != T:
            raise ValueError("q_in and k_in must have the same number of tokens")
        hq = _heads(Wq, head_dim, "q_in")
        q_out = _out_rows(q_out, "q_out", q_in, (T, Wq), sq, stream)
        qp, qo = q_in.data_ptr(), q_out.data_ptr()
    args = [qp, qo, gq, sq, hq, k_in.data_ptr(), gk, sk, v_in.data_ptr(), sv, hk, T, head_dim, *table,
            int(interleaved), pos]
    return args, q_out if q_in is not None else None, T, hk


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
    args, q_out, T, hk = _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out,
                                      interleaved, stream)
    dev = k_in.device
    shapes, strides = [], []
    for c, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _same(dev, k_in.dtype, c, name)
        if c.dim() != 4 or tuple(c.shape[2:]) != (hk, head_dim) or (head_dim > 1 and c.stride(3) != 1):
            raise ValueError(f"{name} must be [pages, page_size, {hk}, {head_dim}] with unit stride along the last")
        shapes.append((c.shape[0], c.shape[1]))
        strides.append((ctypes.c_int64 * 3)(*c.stride()[:3]))
    if shapes[0] != shapes[1]:
        raise ValueError("k_cache and v_cache must have the same pages")
    s = _ints(slots, "slots", T, torch.int64, dev)
    with _on(dev):
        st = capi().qknorm_rope_append(*args, k_cache.data_ptr(), strides[0], v_cache.data_ptr(), strides[1],
                                       *shapes[0], s, float(eps), _DTYPES[k_in.dtype], _stream_handle(stream, dev))
    _clib.check(st, "qknorm_rope_append")
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
    for t, name, dt in ((kc, "k_codes", torch.uint8), (ks, "k_scales", torch.float16), (vc, "v_codes", torch.uint8),
                        (vs, "v_scales", torch.float16)):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.device == dev and t.dtype == dt and t.dim() == 4
                and t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous 4-D CUDA {dt} tensor on {dev}")
    pages, hk, ps, half = kc.shape
    if vc.shape != kc.shape or ks.shape != vs.shape or tuple(ks.shape) != (pages, hk, ps, half * 2 // 64):
        raise ValueError("the cache's codes must be [pages, kv_heads, page_size, head_dim / 2] and its scales "
                         "[pages, kv_heads, page_size, head_dim / 64]")
    return [t.data_ptr() for t in (kc, ks, vc, vs)], (pages, ps, hk, 2 * half)


def qknorm_rope_append_kv4(q_in, k_in: torch.Tensor, v_in: torch.Tensor, gamma_q, gamma_k, cos_sin: torch.Tensor,
                           positions: torch.Tensor, cache, slots: torch.Tensor, eps: float = 1e-6, *,
                           interleaved: bool = False, q_out=None, stream=None):
    """``qknorm_rope_append`` into a 4-bit cache (``kv4_cache``); returns ``q_out``."""
    dev = k_in.device
    ptrs, (pages, ps, heads, head_dim) = _kv4_args(cache, dev)
    args, q_out, T, hk = _append_rows(q_in, k_in, v_in, gamma_q, gamma_k, head_dim, cos_sin, positions, q_out,
                                      interleaved, stream)
    if hk != heads:
        raise ValueError(f"k_in has {hk} heads, the cache {heads}")
    s = _ints(slots, "slots", T, torch.int64, dev)
    with _on(dev):
        st = capi().qknorm_rope_append_kv4(*args, *ptrs, pages, ps, s, float(eps), _DTYPES[k_in.dtype],
                                           _stream_handle(stream, dev))
    _clib.check(st, "qknorm_rope_append_kv4")
    return q_out


def qknorm_kv4_read(cache, slots: torch.Tensor, dtype: torch.dtype = torch.bfloat16, *, k_out=None, v_out=None,
                    stream=None):
    """The cached tokens at ``slots`` as K and V rows ``[n, kv_heads * head_dim]``
    of ``dtype`` (zeros for a slot outside the cache)."""
    dev = slots.device
    ptrs, (pages, ps, hk, d) = _kv4_args(cache, dev)
    if dtype not in (torch.float32, torch.bfloat16, torch.float16):
        raise TypeError(f"dtype {dtype} unsupported (float32, bfloat16, float16)")
    n = slots.numel()
    s = _ints(slots, "slots", n, torch.int64, dev)
    fresh = []
    if k_out is None:
        fresh.append(k_out := torch.empty((n, hk * d), dtype=dtype, device=dev))
    if v_out is None:
        fresh.append(v_out := torch.empty((n, hk * d), dtype=dtype, device=dev))
    _used_on(stream, *fresh)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _same(dev, dtype, t, name)
    (Tk, Wk, sk), (Tv, Wv, sv) = _rows(k_out, "k_out"), _rows(v_out, "v_out")
    if (Tk, Wk) != (n, hk * d) or (Tv, Wv) != (n, hk * d):
        raise ValueError(f"k_out and v_out must be [{n}, {hk * d}]")
    with _on(dev):
        st = capi().qknorm_kv4_read(*ptrs, pages, ps, hk, d, s, n, k_out.data_ptr(), sk, v_out.data_ptr(), sv,
                                    _DTYPES[dtype], _stream_handle(stream, dev))
    _clib.check(st, "qknorm_kv4_read")
    return k_out, v_out


def kv4_attention_workspace_bytes(T: int, batch: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int,
                                  max_seq_len: int) -> int:
    """Workspace ``qknorm_kv4_attention`` needs for these bounds."""
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
    T, W, sq = _rows(q, "q")
    dev, dt = q.device, q.dtype
    ptrs, (pages, ps, hk, d) = _kv4_args(cache, dev)
    hq = _heads(W, d, "q")
    if not (isinstance(block_table, torch.Tensor) and block_table.dim() == 2):
        raise ValueError("block_table must be [B, max_pages]")
    B, max_pages = block_table.shape
    bt = _ints(block_table, "block_table", B * max_pages, torch.int32, dev)
    sl = _ints(seq_lens, "seq_lens", B, torch.int32, dev)
    qs = None if q_start is None else _ints(q_start, "q_start", B + 1, torch.int32, dev)
    fresh = []
    if out is None:
        fresh.append(out := torch.empty((T, W), dtype=dt, device=dev))
    so = _rows_like(out, "out", q, (T, W))
    if lse is None and return_lse:
        fresh.append(lse := torch.empty((T, hq), dtype=torch.float32, device=dev))
    lp = None if lse is None else _vec(lse, "lse", T * hq, torch.float32, dev)
    need = capi().qknorm_kv4_attention_workspace_bytes(T, B, hq, hk, d, int(max_q_len), int(max_seq_len))
    if workspace is None:
        fresh.append(workspace := _workspace(None, need, dev))
    workspace = _workspace(workspace, need, dev)
    _used_on(stream, *fresh)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else float(softmax_scale)
    with _on(dev):
        st = capi().qknorm_kv4_attention(q.data_ptr(), sq, out.data_ptr(), so, lp, hq, *ptrs, pages, ps, hk, d, bt,
                                         max_pages, sl, qs, T, B, int(max_q_len), int(max_seq_len), int(window), scale,
                                         workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                         _DTYPES[dt], _stream_handle(stream, dev))
    _clib.check(st, "qknorm_kv4_attention")
    return (out, lse) if return_lse else out
