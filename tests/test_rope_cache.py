"""Headwise QK-Norm with rotation, its gradient, the paged append, the 4-bit
cache and attention over it, against the formulas in 64 bits.

Tolerances are counted from the arithmetic.  u = 2^-24 is fp32's half step.  A
head's squared sum is a sum of at most 64 terms in sequence and 5 tree levels, so
r is off by less than 2^-19 relative with the reciprocal root's 2 ulp, and so is
a normalized element n.  A rotated element a cos - b sin is then within
2^-18 (|a| + |b|) of the exact one, and rounding to the output type adds half a
step of that type (relative, or half the smallest subnormal)."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import attention_normalization_b200 as qk
from attention_normalization_b200 import _clib
from attention_normalization_b200 import build as qbuild

DEV = "cuda:0"
BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF_STEP = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24, E4M3: 2.0 ** -4}
HALF_TINY = {BF16: 0.0, F16: 2.0 ** -25, F32: 0.0, E4M3: 2.0 ** -10}
EPS = 1e-6


def f64(t):
    return t.detach().cpu().to(torch.float64)


def table(P, rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    a = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * i / max(rot, 1))[None]
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(n, cs, rot, inter, transposed=False):
    """R(pos) (or its transpose) on n [T, h, D] in 64 bits, and |a| + |b| of each element's pair."""
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if transposed:
        s = -s
    ia = torch.arange(0, rot, 2) if inter else torch.arange(rot // 2)
    ib = ia + 1 if inter else ia + rot // 2
    y, mag = n.clone(), n.abs()
    a, b = n[..., ia], n[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def forward(x, gamma, D, cs, pos, inter, eps=EPS):
    """The operator in 64 bits: y [T, h, D] and the magnitude that errors scale with."""
    T = x.shape[0]
    n = f64(x).reshape(T, -1, D)
    eps = float(np.float32(eps))
    if gamma is not None:
        n = n / (n.square().mean(-1, keepdim=True) + eps).sqrt() * f64(gamma)
    rot, P = cs.shape[1], cs.shape[0]
    ok = (pos >= 0) & (pos < P)
    rows = cs.double()[pos.clamp(0, max(P - 1, 0))] if P else torch.zeros((T, rot), dtype=torch.float64)
    y, mag = rotate(n, rows, rot, inter)
    y[pos < 0] = 0.0
    mag[pos < 0] = 0.0
    y[pos >= P] = math.nan
    assert ok.shape == pos.shape
    return y, mag


def check(got, want, mag, dtype, rel=2.0 ** -18):
    got, want, mag = f64(got).reshape(-1), want.reshape(-1), mag.reshape(-1)
    assert torch.equal(got.isnan(), want.isnan())
    if dtype == E4M3:
        want = want.clamp(-448, 448)
    tol = HALF_STEP[dtype] * (want.abs() + rel * mag) + HALF_TINY[dtype] + rel * mag
    off = (got - want).abs() - tol
    worst = torch.nan_to_num(off, nan=-1.0).max() if off.numel() else torch.tensor(-1.0)
    assert worst <= 0, f"{int((off > 0).sum())} of {off.numel()} elements off, by up to {float(worst):.3g}"


def gamma_of(D, dtype, g):
    return (1 + 0.1 * torch.randn(D, generator=g)).to(BF16 if dtype == E4M3 else dtype)


def rows_of(T, W, dtype, g, pad=0, shift=0):
    """[T, W] rows, padded by `pad` columns and starting `shift` elements into the buffer; sentinels around."""
    buf = torch.full((T * (W + pad) + shift + pad,), 5.0)
    view = buf[shift:shift + T * (W + pad)].view(T, W + pad)
    view[:, :W] = torch.randn((T, W), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    dev = buf.to(dtype).to(DEV)
    return dev, dev[shift:shift + T * (W + pad)].view(T, W + pad)[:, :W]


SHAPES = [  # T, q heads, k heads, D, rotary, interleaved, pad, shift
    (1, 1, 1, 64, 64, False, 0, 0),
    (1, 40, 8, 128, 128, False, 0, 0),
    (5, 3, 2, 128, 64, False, 32, 0),
    (7, 4, 1, 96, 96, True, 0, 0),
    (33, 8, 2, 80, 80, False, 16, 0),
    (9, 2, 2, 256, 128, True, 0, 0),
    (4, 5, 3, 192, 96, False, 0, 0),
    (3, 2, 1, 512, 512, False, 0, 0),
    (3, 2, 1, 1024, 256, True, 0, 0),
    (6, 3, 1, 128, 0, False, 0, 0),
    (11, 2, 3, 7, 6, False, 1, 1),
    (2, 3, 1, 1, 0, False, 0, 0),
    (17, 2, 2, 128, 128, False, 3, 5),
    (8, 2, 1, 64, 2, True, 0, 0),
    (300, 6, 2, 64, 64, False, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32, E4M3])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,pad,shift", SHAPES)
def test_norm_and_rotation(T, hq, hk, D, rot, inter, pad, shift, dtype):
    g = torch.Generator().manual_seed(T * 1000 + D)
    qb, q = rows_of(T, hq * D, dtype, g, pad, shift)
    kb, k = rows_of(T, hk * D, dtype, g, pad, shift)
    gq, gk = gamma_of(D, dtype, g), gamma_of(D, dtype, g)
    P = 37
    cs, pos = table(P, rot), torch.randint(-3, P + 3, (T,), generator=g)
    args = (gq.to(DEV), gk.to(DEV), D, cs.to(DEV), pos.to(DEV))
    before = qb.clone()
    qo, ko = qk.qknorm_headwise_rope(q, k, *args, EPS, interleaved=inter)
    assert torch.equal(qb.view(torch.uint8), before.view(torch.uint8))
    for got, x, gm in ((qo, q, gq), (ko, k, gk)):
        check(got, *forward(x, gm, D, cs, pos, inter), dtype)
    qi, ki = qk.qknorm_headwise_rope(q, k, *args, EPS, interleaved=inter, q_out=q, k_out=k)  # in place
    for a, b in ((qi, qo), (ki, ko)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    if pad:  # columns between the rows
        assert bool((qb[shift:shift + T * (hq * D + pad)].view(T, -1)[:, hq * D:].float() == 5).all())


@pytest.mark.gpu
def test_zero_tokens():
    e = torch.empty((0, 128), dtype=BF16, device=DEV)
    one = torch.ones(128, dtype=BF16, device=DEV)
    cs, none = table(4, 128).to(DEV), torch.empty(0, dtype=torch.int64, device=DEV)
    q, k = qk.qknorm_headwise_rope(e, e.clone(), one, one, 128, cs, none)
    assert q.shape == (0, 128) and k.shape == (0, 128)
    _, _, dgq, dgk = qk.qknorm_headwise_rope_backward(e, e, e.clone(), e.clone(), one, one, 128, cs, none)
    assert not dgq.any() and not dgk.any()


# --------------------------------------------------------------------------- gradient

def gradient(x, dy, gamma, D, cs, pos, inter, eps=EPS):
    """dx [T, h, D], dgamma [D] in 64 bits, and the magnitudes that errors scale with."""
    T = x.shape[0]
    eps = float(np.float32(eps))
    v, gm = f64(x).reshape(T, -1, D), f64(gamma)
    P, rot = cs.shape
    u, mag = rotate(f64(dy).reshape(T, -1, D), cs.double()[pos.clamp(0, P - 1)], rot, inter, transposed=True)
    pad = pos < 0
    r = 1 / (v.square().mean(-1, keepdim=True) + eps).sqrt()
    c = r.square() * (u * gm * v).mean(-1, keepdim=True)
    c_mag = r.square() * (mag * gm.abs() * v.abs()).mean(-1, keepdim=True)
    dx = r * (u * gm - v * c)
    dx_mag = r * (mag * gm.abs() + v.abs() * c_mag)
    dg, dg_mag = u * v * r, mag * v.abs() * r
    for t in (dx, dx_mag, dg, dg_mag):
        t[pad] = 0.0
    return dx, dx_mag, dg.sum((0, 1)), dg_mag.sum((0, 1))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,pad,shift", SHAPES)
def test_gradient(T, hq, hk, D, rot, inter, pad, shift, dtype):
    g = torch.Generator().manual_seed(T * 77 + D)
    _, q = rows_of(T, hq * D, dtype, g, pad, shift)
    _, k = rows_of(T, hk * D, dtype, g, 0, shift)
    dqb, dq = rows_of(T, hq * D, dtype, g, 2 * pad, shift)
    _, dk = rows_of(T, hk * D, dtype, g, pad, shift)
    gq, gk = gamma_of(D, dtype, g), gamma_of(D, dtype, g)
    P = 29
    cs, pos = table(P, rot), torch.randint(-2, P, (T,), generator=g)
    args = (gq.to(DEV), gk.to(DEV), D, cs.to(DEV), pos.to(DEV))
    out = qk.qknorm_headwise_rope_backward(dq, dk, q, k, *args, EPS, interleaved=inter)
    again = qk.qknorm_headwise_rope_backward(dq, dk, q, k, *args, EPS, interleaved=inter)
    for a, b in zip(out, again):
        assert torch.equal(a, b)
    for got, dg, x, dy, gm in ((out[0], out[2], q, dq, gq), (out[1], out[3], k, dk, gk)):
        dx, dx_mag, want, mag = gradient(x, dy, gm, D, cs, pos, inter)
        # u carries 2^-22 of |a| + |b|, r and M 2^-18: dx within 2^-16 of its terms
        check(got, dx, dx_mag, dtype, rel=2.0 ** -16)
        # a sum over all tokens and heads: at most `rows` additions in sequence
        rows = T * max(hq, hk)
        assert bool(((f64(dg) - want).abs() <= (2.0 ** -17 + rows * 2.0 ** -24) * mag + 1e-30).all())
    # dx over dy, and over x
    keep = (out[0].clone(), out[1].clone())
    q2, dq2 = q.clone(), dq
    got = qk.qknorm_headwise_rope_backward(dq2, dk, q, k, *args, EPS, interleaved=inter, dq_in=dq2, dk_in=k)
    assert torch.equal(got[0], keep[0]) and torch.equal(got[1], keep[1]) and torch.equal(q, q2)
    if pad:
        assert bool((dqb[shift:shift + T * (hq * D + 2 * pad)].view(T, -1)[:, hq * D:].float() == 5).all())


@pytest.mark.gpu
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (96, 48, True), (10, 6, False)])
def test_gradient_against_differences(D, rot, inter):
    """Central differences of the fp32 forward pass along random directions.
    With a step h the difference quotient of L = <w, y> is off by h^2 |L'''| / 6
    and by the forward's rounding over 2h: y is within 2^-18 of |n| <= a few, so
    <w, y> is off by about 2^-18 sqrt(T h D) / h.  With h = 2^-6 both stay below
    2^-10 sqrt(T h D) for inputs of unit size."""
    g = torch.Generator().manual_seed(D)
    T, hq, hk = 3, 2, 1
    x = [torch.randn((T, h * D), generator=g) for h in (hq, hk)]
    gm = [1 + 0.1 * torch.randn(D, generator=g) for _ in range(2)]
    w = [torch.randn((T, h * D), generator=g) for h in (hq, hk)]
    dx = [torch.randn((T, h * D), generator=g) for h in (hq, hk)]
    dgm = [torch.randn(D, generator=g) for _ in range(2)]
    cs, pos = table(64, rot), torch.tensor([5, 63, 0])

    def loss(s):
        y = qk.qknorm_headwise_rope(*[(a + s * b).to(DEV) for a, b in zip(x, dx)],
                                    *[(a + s * b).to(DEV) for a, b in zip(gm, dgm)], D, cs.to(DEV), pos.to(DEV), EPS,
                                    interleaved=inter)
        return sum(float((f64(a) * f64(b)).sum()) for a, b in zip(y, w))
    h = 2.0 ** -6
    slope = (loss(h) - loss(-h)) / (2 * h)
    out = qk.qknorm_headwise_rope_backward(*[t.to(DEV) for t in (*w, *x, *gm)], D, cs.to(DEV), pos.to(DEV), EPS,
                                           interleaved=inter)
    want = sum(float((f64(a) * f64(b)).sum()) for a, b in zip(out, (*dx, *dgm)))
    # |L'''| along a unit-size direction: (r |dx|)^3-like terms of each element, a few tens per element at most
    bound = (2.0 ** -18 / h + 40 * h * h / 6) * math.sqrt(T * (hq + hk) * D) * 4
    assert abs(slope - want) <= bound, (slope, want, bound)


@pytest.mark.gpu
def test_gradient_of_a_position_past_the_table_is_nan():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn((2, 128), generator=g).to(DEV) for _ in range(2))
    one = torch.ones(64, device=DEV)
    cs = table(4, 64).to(DEV)
    out = qk.qknorm_headwise_rope_backward(dy, dy, x, x, one, one, 64, cs, torch.tensor([3, 4], device=DEV))
    assert not out[0][0].isnan().any() and out[0][1].isnan().all() and out[2].isnan().all()


# --------------------------------------------------------------------------- append

def slots_of(T, pages, ps, g, holes=True):
    s = torch.randperm(pages * ps, generator=g)[:T]
    if holes and T > 2:
        s[1] = -1
        s[T - 1] = pages * ps  # past the cache
    return s


LAYOUTS = ["tokens first", "heads first", "pages of both", "padded"]


def caches_of(layout, pages, ps, hk, D, dtype, g):
    """(buffer, k_cache, v_cache): the caches indexed [page, token, head, dim]."""
    if layout == "tokens first":
        buf = torch.randn((2, pages, ps, hk, D), generator=g)
    elif layout == "heads first":
        buf = torch.randn((2, pages, hk, ps, D), generator=g)
    elif layout == "pages of both":
        buf = torch.randn((pages, 2, ps, hk, D), generator=g)
    else:
        buf = torch.randn((2, pages, ps, hk + 1, D + 3), generator=g)
    buf = buf.to(dtype).to(DEV)
    if layout == "tokens first":
        return buf, buf[0], buf[1]
    if layout == "heads first":
        return buf, buf[0].transpose(1, 2), buf[1].transpose(1, 2)
    if layout == "pages of both":
        return buf, buf[:, 0], buf[:, 1]
    return buf, buf[0][:, :, :hk, :D], buf[1][:, :, :hk, :D]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32, E4M3])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,ps", [
    (1, 4, 2, 128, 128, False, True, 16), (37, 6, 2, 64, 64, False, True, 5), (20, 0, 3, 128, 64, True, True, 1),
    (9, 2, 1, 96, 96, False, False, 7), (5, 3, 1, 10, 4, True, True, 3), (130, 8, 4, 128, 128, False, True, 32)])
def test_append(T, hq, hk, D, rot, inter, norm, ps, layout, dtype):
    g = torch.Generator().manual_seed(T + D)
    W = (hq + 2 * hk) * D
    _, x = rows_of(T, W, dtype, g)
    q, k, v = x[:, :hq * D] if hq else None, x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:]
    gq, gk = (gamma_of(D, dtype, g), gamma_of(D, dtype, g)) if norm else (None, None)
    P = 50
    cs, pos = table(P, rot), torch.randint(-1, P + 1, (T,), generator=g)
    pages = T // ps + 4
    slots = slots_of(T, pages, ps, g)
    buf, kc, vc = caches_of(layout, pages, ps, hk, D, dtype, g)
    before = buf.clone()
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo = qk.qknorm_rope_append(q, k, v, to(gq), to(gk), D, to(cs), to(pos), kc, vc, to(slots), EPS, interleaved=inter)
    if hq:
        check(qo, *forward(q, gq, D, cs, pos, inter), dtype)
    else:
        assert qo is None
    held = (slots >= 0) & (slots < pages * ps)
    page, off = slots[held] // ps, slots[held] % ps
    y, mag = forward(k, gk, D, cs, pos, inter)
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[buf.element_size()]
    check(kc.cpu().view(bits)[page, off].view(dtype), y[held], mag[held], dtype)
    assert torch.equal(vc.cpu().view(bits)[page, off], v.cpu().view(bits).reshape(T, hk, D)[held])
    # every bit that no slot names is as it was
    b = caches_of(layout, pages, ps, hk, D, dtype, torch.Generator().manual_seed(0))
    b[0].copy_(before)
    for c in (kc, vc, *b[1:]):
        c.view(bits)[page.to(DEV), off.to(DEV)] = 0
    assert torch.equal(buf.view(bits), b[0].view(bits))


def quantise(y):
    """numpy, 64 bits: y [..., D] -> codes (with 8 added), scales as fp16."""
    y = np.asarray(y).reshape(*y.shape[:-1], -1, 64)
    with np.errstate(all="ignore"):
        s = np.minimum(np.abs(y).max(-1) / 7, 65504.0).astype(np.float16)
        bad = ~np.isfinite(y).all(-1)
        s[bad] = np.nan
        w = s.astype(np.float64)[..., None]
        c = np.where(w > 0, np.clip(np.rint(y / w), -7, 7), 0.0)
        c[bad] = 0
    return (c + 8).astype(np.uint8).reshape(*y.shape[:-2], -1), s


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def special_rows(x, D):
    """Rows of zeros, ties, tiny and huge values, an infinity and a NaN, as far as there are rows."""
    rows = [lambda r: r.zero_(), lambda r: r.copy_((torch.arange(r.numel()) % 15 - 7) * 0.5),
            lambda r: r.mul_(1e-7), lambda r: r.mul_(1e4), lambda r: r[:1].fill_(math.inf), lambda r: r[-1:].fill_(math.nan),
            lambda r: r.copy_((torch.arange(r.numel()) % 2) * 7.0)]
    for i, f in enumerate(rows):
        if i + 3 < x.shape[0]:
            f(x[i + 3])
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm,ps,shift", [
    (1, 4, 2, 128, 128, False, True, 16, 0), (37, 6, 2, 64, 64, False, True, 16, 0), (20, 0, 3, 128, 64, True, True, 48, 0),
    (33, 2, 1, 256, 256, False, False, 32, 0), (21, 3, 1, 256, 128, True, True, 16, 0), (40, 2, 2, 128, 0, False, False, 16, 0),
    (23, 1, 2, 128, 128, False, True, 16, 3), (600, 4, 4, 128, 128, False, True, 64, 0), (15, 1, 1, 64, 6, False, True, 16, 0)])
def test_append_kv4(T, hq, hk, D, rot, inter, norm, ps, shift, dtype):
    g = torch.Generator().manual_seed(T + D + rot)
    W = (hq + 2 * hk) * D
    x = special_rows(torch.randn((T, W), generator=g) * torch.exp(torch.randn((T, 1), generator=g)), D).to(dtype)
    buf = torch.zeros(T * W + shift, dtype=dtype)
    buf[shift:] = x.reshape(-1)
    x = buf.to(DEV)[shift:].view(T, W)
    q, k, v = x[:, :hq * D] if hq else None, x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:]
    gq, gk = (gamma_of(D, dtype, g), gamma_of(D, dtype, g)) if norm else (None, None)
    P = 50
    cs, pos = table(P, rot), torch.randint(-1, P + 1, (T,), generator=g)
    pages = T // ps + 3
    slots = slots_of(T, pages, ps, g)
    cache = qk.kv4_cache(pages, ps, hk, D, DEV)
    for t in cache:
        t.copy_(torch.randint(0, 100, t.shape, generator=g).to(t.dtype))
    before = [t.cpu().clone() for t in cache]
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo = qk.qknorm_rope_append_kv4(q, k, v, to(gq), to(gk), to(cs), to(pos), cache, to(slots), EPS, interleaved=inter)
    finite = torch.isfinite(f64(x)).all(-1)
    if hq:
        y, mag = forward(q, gq, D, cs, pos, inter)
        check(qo.cpu()[finite], y[finite], mag[finite], dtype)
    held = (slots >= 0) & (slots < pages * ps)
    page, off = slots[held] // ps, slots[held] % ps
    yk, yv = forward(k, gk, D, cs, pos, inter)[0], f64(v).reshape(T, hk, D)
    for y, codes, scales, c0, s0 in ((yk, cache[0], cache[1], before[0], before[1]), (yv, cache[2], cache[3], before[2], before[3])):
        c, s = quantise(y[held].numpy())
        want_c = unpack(c0)
        want_c[page, :, off] = torch.from_numpy(c)
        want_s = s0.clone()
        want_s[page, :, off] = torch.from_numpy(s)
        got_s = scales.cpu()
        assert torch.equal(got_s.isnan(), want_s.isnan())
        assert torch.equal(torch.nan_to_num(got_s), torch.nan_to_num(want_s))
        assert torch.equal(unpack(codes.cpu()), want_c)
    for out_dtype in (BF16, F16, F32):
        kr, vr = qk.qknorm_kv4_read(cache, to(slots), out_dtype)
        for got, codes, scales in ((kr, cache[0], cache[1]), (vr, cache[2], cache[3])):
            val = (unpack(codes.cpu()).double() - 8) * scales.cpu().double().repeat_interleave(64, -1)
            want = torch.zeros((T, hk, D), dtype=torch.float64)
            want[held] = val[page, :, off]
            want = want.float().to(out_dtype).reshape(T, -1)  # code * scale is exact in fp32
            assert torch.equal(torch.nan_to_num(got.cpu()), torch.nan_to_num(want))
            assert torch.equal(got.cpu().isnan(), want.isnan())


# --------------------------------------------------------------------------- attention

def attention(q, cache, block_table, seq_lens, q_start, max_q, max_len, window, scale):
    """64 bits: out [T, hq, D], lse [T, hq], the tolerance of out and of lse; None rows stay NaN (of no sequence)."""
    kc, ks, vc, vs = (t.cpu() for t in cache)
    pages, hk, ps, half = kc.shape
    D = 2 * half
    T, hq = q.shape[0], q.shape[1] // D
    val = lambda c, s: (unpack(c).double() - 8) * s.double().repeat_interleave(64, -1)  # noqa: E731
    K, V = val(kc, ks), val(vc, vs)
    Q = f64(q).reshape(T, hq, D)
    out, lse = torch.full((T, hq, D), math.nan, dtype=torch.float64), torch.full((T, hq), math.nan, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    named = torch.zeros(T, dtype=torch.bool)
    for b in range(block_table.shape[0]):
        r0, r1 = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        r1 = min(r1, r0 + max_q, T)
        L = max(0, min(int(seq_lens[b]), max_len, block_table.shape[1] * ps))
        t = torch.arange(L)
        page = block_table[b].long()[t // ps] if L else t
        there = (page >= 0) & (page < pages)
        page = page.clamp(0, max(pages - 1, 0))
        k, v = (x[page, :, t % ps] if pages else torch.zeros((L, hk, D), dtype=torch.float64) for x in (K, V))  # [L, hk, D]
        for i in range(r1 - r0):
            pos = L - (r1 - r0) + i
            keep = there & (t <= pos)
            if window:
                keep &= t > pos - window
            row = r0 + i
            named[row] = True
            out[row], lse[row] = 0.0, -math.inf
            if not keep.any():
                continue
            kk, vv = (x[keep].repeat_interleave(hq // hk, 1) for x in (k, v))  # [n, hq, D]
            s = torch.einsum("hd,nhd->hn", Q[row], kk) * scale
            p = torch.softmax(s, -1)
            out[row] = torch.einsum("hn,nhd->hd", p, vv)
            lse[row] = torch.logsumexp(s, -1)
            # scores: products exact in fp32, summed with D * 2^-24 of the terms, and the reciprocal steps of
            # scale and exponent; weights rounded to fp16 (2^-11) or flushed below 2^-28 of the largest
            ds = (torch.einsum("hd,nhd->hn", Q[row].abs(), kk.abs()) * abs(scale)).amax(-1) * (D + 8) * 2.0 ** -24 \
                + s.abs().amax(-1) * 2.0 ** -22 + 2.0 ** -20
            A = torch.einsum("hn,nhd->hd", p, vv.abs())
            tol[row] = (2.0 ** -11 + 2 * ds[:, None]) * A + 2.0 ** -28 * vv.abs().sum(0) * p.amax(-1, keepdim=True)
            ltol[row] = 2 * ds + lse[row].abs() * 2.0 ** -23 + 2.0 ** -20
    return out, lse, tol, ltol, named


def random_cache(pages, ps, hk, D, g):
    cache = qk.kv4_cache(pages, ps, hk, D, DEV)
    for i in (0, 2):
        cache[i].copy_(torch.randint(0, 256, cache[i].shape, generator=g).to(torch.uint8))
        cache[i + 1].copy_((torch.exp(torch.randn(cache[i + 1].shape, generator=g)) * 0.15).half())
    return cache


def run_attention(q, cache, bt, lens, q_start, max_q, max_len, window, scale=None, **kw):
    D = cache[0].shape[3] * 2
    T, hq = q.shape[0], q.shape[1] // D
    out = torch.full((T, hq * D), 3.0, dtype=q.dtype, device=DEV)
    lse = torch.full((T, hq), 3.0, device=DEV)
    qk.qknorm_kv4_attention(q, cache, bt.to(DEV), lens.to(DEV), max_seq_len=max_len, q_start=None if q_start is None else q_start.to(DEV),
                            max_q_len=max_q, window=window, softmax_scale=scale, out=out, lse=lse, **kw)
    return out, lse


def check_attention(q, cache, bt, lens, q_start, max_q, max_len, window=0, scale=None):
    D = cache[0].shape[3] * 2
    got, lse = run_attention(q, cache, bt, lens, q_start, max_q, max_len, window, scale)
    want, wl, tol, ltol, named = attention(q, cache, bt, lens, q_start, max_q, max_len, window,
                                           1 / math.sqrt(D) if scale is None else scale)
    o, l = f64(got).reshape(want.shape), f64(lse)
    assert bool((o[~named] == 3).all()) and bool((l[~named] == 3).all()), "rows of no sequence were written"
    o, l, want, wl, tol, ltol = (x[named] for x in (o, l, want, wl, tol, ltol))
    assert torch.equal(o.isnan(), want.isnan()) and torch.equal(l.isnan(), wl.isnan())
    assert torch.equal(l == -math.inf, wl == -math.inf)
    full = HALF_STEP[q.dtype] * (want.abs() + tol) + HALF_TINY[q.dtype] + tol
    off = torch.nan_to_num((o - want).abs() - full, nan=-1.0)
    assert off.numel() == 0 or off.max() <= 0, f"{int((off > 0).sum())} of {off.numel()}, by {float(off.max()):.3g}"
    seen = wl.isfinite()
    assert bool(((l - wl).abs()[seen] <= ltol[seen]).all())
    return got, lse


def tables(lens, ps, pages, g, extra=2):
    per = [-(-max(int(n), 0) // ps) for n in lens]
    order = torch.randperm(pages, generator=g)
    bt = torch.full((len(lens), max(per, default=0) + extra), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        bt[b, :n] = order[at:at + n].int()
        at += n
    return bt


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hk,ps,lens,window", [
    (1, 1, 16, [1], 0), (8, 8, 16, [0, 5, 16, 17], 0), (6, 2, 32, [100, 31, 32, 33, 1], 0), (16, 2, 16, [300, 7], 50),
    (40, 8, 64, [513], 0), (16, 1, 48, [129, 64, 0, 200], 1), (3, 1, 16, [700], 128), (20, 1, 16, [95, 40], 0)])
def test_attention_of_one_token_each(hq, hk, ps, lens, window, D, dtype):
    g = torch.Generator().manual_seed(hq * 100 + D)
    pages = sum(-(-n // ps) for n in lens) + 2
    cache = random_cache(pages, ps, hk, D, g)
    q = torch.randn((len(lens) + 1, hq * D), generator=g).to(dtype).to(DEV)
    check_attention(q, cache, tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32), None, 1, max(lens), window)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (BF16, 256)])
@pytest.mark.parametrize("hq,hk,ps,lens,qn,window", [
    (8, 2, 16, [40, 9, 100], [3, 9, 0], 0), (4, 4, 32, [65, 64], [33, 1], 0), (16, 2, 16, [200, 3], [17, 5], 40),
    (5, 1, 48, [160], [150], 0), (2, 1, 16, [31, 0, 70], [31, 2, 8], 7)])
def test_attention_of_chunks(hq, hk, ps, lens, qn, window, dtype, D):
    g = torch.Generator().manual_seed(sum(lens) + D)
    pages = sum(-(-n // ps) for n in lens) + 1
    cache = random_cache(pages, ps, hk, D, g)
    q_start = torch.tensor([0, *np.cumsum(qn)], dtype=torch.int32)
    q = torch.randn((int(q_start[-1]) + 3, hq * D), generator=g).to(dtype).to(DEV)
    check_attention(q, cache, tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32), q_start, max(qn), max(lens), window)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hk,D,L,window", [(8, 1, 128, 20011, 0), (2, 2, 64, 9000, 0), (16, 2, 256, 5003, 3000), (40, 8, 128, 33000, 0)])
def test_attention_over_a_long_cache(hq, hk, D, L, window):
    g = torch.Generator().manual_seed(L)
    ps, lens = 64, [L, 70]
    pages = sum(-(-n // ps) for n in lens) + 1
    cache = random_cache(pages, ps, hk, D, g)
    q = torch.randn((2, hq * D), generator=g).to(BF16).to(DEV)
    bt, sl = tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32)
    got, lse = check_attention(q, cache, bt, sl, None, 1, L, window)
    again, lse2 = run_attention(q, cache, bt, sl, None, 1, L, window)
    assert torch.equal(got, again) and torch.equal(lse, lse2)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hk,D,dtype,rows,window", [(8, 4, 128, BF16, 1, 0), (16, 2, 64, F16, 3, 0), (6, 3, 256, BF16, 2, 700)])
def test_attention_of_many_uneven_sequences(hq, hk, D, dtype, rows, window):
    """Enough tokens to be cut into shares, which then begin and end inside
    sequences, in ones without tokens and in ones without rows."""
    g = torch.Generator().manual_seed(D + rows)
    ps, B = 32, 23
    lens = [int(x) for x in torch.randint(0, 1500, (B,), generator=g)]
    lens[0], lens[5], lens[6], lens[22] = 2900, 0, 1, 0
    qn = [rows] * B
    if rows > 1:
        qn[3] = qn[22] = 0
        qn[7] = 1
    pages = sum(-(-n // ps) for n in lens)
    cache = random_cache(pages, ps, hk, D, g)
    q_start = torch.tensor([0, *np.cumsum(qn)], dtype=torch.int32)
    q = torch.randn((int(q_start[-1]) + 1, hq * D), generator=g).to(dtype).to(DEV)
    check_attention(q, cache, tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32),
                    None if rows == 1 else q_start, rows, 3000, window)


@pytest.mark.gpu
def test_attention_to_a_token_whose_values_are_zeros():
    """All weight on a token with zero values, hundreds of powers of two above
    the others, wherever it comes: zeros, and its score as lse."""
    g = torch.Generator().manual_seed(12)
    hq, hk, D, ps, L = 4, 1, 128, 16, 1100
    for zero in (0, 40, 700, L - 1):
        cache = random_cache(70, ps, hk, D, g)
        bt = torch.arange(70, dtype=torch.int32).view(1, 70)
        q = torch.randn((1, hq * D), generator=g).to(BF16).to(DEV)
        page, off = zero // ps, zero % ps
        cache[1][page, 0, off] = 200.0
        # codes of the query's signs: a large positive score for head 0
        sign = (q[0, :D].float() >= 0).cpu()
        c = torch.where(sign, 15, 1).to(torch.uint8)
        cache[0][page, 0, off] = (c[0::2] | (c[1::2] << 4)).to(DEV)
        cache[2][page, 0, off] = 0x88
        cache[3][page, 0, off] = 0.0
        out, lse = check_attention(q, cache, bt, torch.tensor([L], dtype=torch.int32), None, 1, L)
        assert not out[0, :D].any() and float(lse[0, 0]) > 1000


@pytest.mark.gpu
def test_caches_past_four_gigabytes():
    """The last cells of caches whose offsets do not fit 32 bits."""
    g = torch.Generator().manual_seed(13)
    hq, hk, D, ps = 8, 8, 256, 16
    T, pages = 3, 70000  # 4.6 GB of bfloat16 each
    x = torch.randn((T, (hq + 2 * hk) * D), generator=g).to(BF16).to(DEV)
    q, k, v = x[:, :hq * D], x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:]
    gm, cs, pos = gamma_of(D, BF16, g), table(8, D), torch.tensor([1, 2, 3])
    slots = torch.tensor([pages * ps - 1, 5, (pages - 2) * ps + 3])
    kc, vc = (torch.empty((pages, ps, hk, D), dtype=BF16, device=DEV) for _ in range(2))
    qk.qknorm_rope_append(q, k, v, gm.to(DEV), gm.to(DEV), D, cs.to(DEV), pos.to(DEV), kc, vc, slots.to(DEV), EPS)
    y, mag = forward(k, gm, D, cs, pos, False)
    at = (slots.to(DEV) // ps, slots.to(DEV) % ps)
    check(kc[at], y, mag, BF16)
    assert torch.equal(vc[at].reshape(T, -1), v)
    del kc, vc
    pages = 270000  # 4.4 GB of codes each
    cache = tuple(torch.empty(s, dtype=t, device=DEV) for _ in range(2) for s, t in (
        ((pages, hk, ps, D // 2), torch.uint8), ((pages, hk, ps, D // 64), torch.float16)))
    slots = torch.arange(T) + (pages - 1) * ps
    q_out = qk.qknorm_rope_append_kv4(q, k, v, gm.to(DEV), gm.to(DEV), cs.to(DEV), pos.to(DEV), cache, slots.to(DEV), EPS)
    kr, vr = qk.qknorm_kv4_read(cache, slots.to(DEV), F32)
    for got, want in ((kr, y), (vr, f64(v).reshape(T, hk, D))):
        c, s = quantise(want.numpy())
        value = (torch.from_numpy(c).double() - 8) * torch.from_numpy(s).double().repeat_interleave(64, -1)
        assert torch.equal(got.cpu().double(), value.reshape(T, -1))
    small = tuple(t[-1:].clone() for t in cache)
    lens, one = torch.tensor([T], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV)
    outs = [qk.qknorm_kv4_attention(q_out, c, torch.tensor([[p]], dtype=torch.int32, device=DEV), lens, max_seq_len=16,
                                    q_start=one, max_q_len=T) for c, p in ((cache, pages - 1), (small, 0))]
    assert torch.equal(*outs)


@pytest.mark.gpu
def test_calls_at_once_on_two_streams():
    """Two long attentions and a gradient on streams of their own, their
    workspaces made for each call, equal to the same calls alone."""
    g = torch.Generator().manual_seed(14)
    hq, hk, D, ps, L = 8, 2, 128, 64, 9000
    pages = -(-L // ps)
    bt, lens = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1), torch.tensor([L], dtype=torch.int32, device=DEV)
    caches = [random_cache(pages, ps, hk, D, g) for _ in range(2)]
    qs = [torch.randn((1, hq * D), generator=g).to(BF16).to(DEV) for _ in range(2)]
    x, dy = (torch.randn((700, hq * D), generator=g).to(BF16).to(DEV) for _ in range(2))
    gm, cs, pos = gamma_of(D, BF16, g).to(DEV), table(700, D).to(DEV), torch.arange(700, device=DEV)

    def calls(streams):
        out = [qk.qknorm_kv4_attention(q, c, bt, lens, max_seq_len=L, stream=s) for q, c, s in zip(qs, caches, streams)]
        return [*out, *qk.qknorm_headwise_rope_backward(dy, dy, x, x, gm, gm, D, cs, pos, stream=streams[2])]
    alone = calls([None] * 3)
    torch.cuda.synchronize()
    for _ in range(5):
        streams = [torch.cuda.Stream() for _ in range(3)]
        for a, b in zip(calls(streams), alone):
            torch.cuda.synchronize()
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_attention_ignores_what_is_masked_and_missing():
    """NaN and infinite scales behind the length, before the window and on pages
    that are not in the table; page numbers outside the cache count as absent."""
    g = torch.Generator().manual_seed(5)
    hq, hk, D, ps = 8, 2, 128, 16
    cache = random_cache(9, ps, hk, D, g)
    bt = torch.tensor([[2, 7, 1, 5], [3, -1, 9, 6], [8, 2 ** 31 - 1, -2 ** 31, 0]], dtype=torch.int32)
    lens = torch.tensor([37, 64, 40], dtype=torch.int32)
    for i in (1, 3):
        cache[i][1, :, 37 - 32:] = math.nan   # behind sequence 0's length
        cache[i][5] = math.inf
        cache[i][0, :, 8:] = math.nan         # behind sequence 2's length
        cache[i][4] = math.nan                # on no table
    q = torch.randn((3, hq * D), generator=g).to(BF16).to(DEV)
    check_attention(q, cache, bt, lens, None, 1, 64)
    cache[1][2, :, :5] = math.nan             # before sequence 0's window of 32
    cache[3][2, :, :5] = math.nan
    check_attention(q, cache, bt, lens, None, 1, 64, window=32)
    none = torch.full((3, 4), -1, dtype=torch.int32)
    check_attention(q, cache, none, lens, None, 1, 64)


@pytest.mark.gpu
def test_attention_extremes():
    """Large and tiny queries and scales, a NaN query row, a NaN value group: each stays where it belongs."""
    g = torch.Generator().manual_seed(6)
    hq, hk, D, ps = 4, 1, 128, 16
    cache = random_cache(8, ps, hk, D, g)
    bt, lens = torch.arange(8, dtype=torch.int32).view(2, 4), torch.tensor([50, 64], dtype=torch.int32)
    for size in (1e-30, 1e-6, 30.0):
        q = (torch.randn((2, hq * D), generator=g) * size).to(BF16).to(DEV)
        check_attention(q, cache, bt, lens, None, 1, 64, scale=None if size < 10 else 0.01)
    check_attention(q, cache, bt, lens, None, 1, 64, scale=0.0)
    cache[3][:, :, ::3] *= 2.0 ** -12          # value scales far apart
    cache[3][3, :, 5] = 60000.0
    q = torch.randn((2, hq * D), generator=g).to(F16).to(DEV)
    check_attention(q, cache, bt, lens, None, 1, 64)
    cache[3].zero_()                           # every value zero: zeros, and the sums stay
    out, lse = check_attention(q, cache, bt, lens, None, 1, 64)
    assert not out.any() and bool(lse.isfinite().all())
    cache[3].fill_(0.25)
    q[0, D] = math.nan                         # head 1 of row 0
    out, lse = run_attention(q, cache, bt, lens, None, 1, 64, 0)
    o = out.view(2, hq, D)
    assert o[0, 1].isnan().all() and lse[0, 1].isnan() and not o[0, [0, 2, 3]].isnan().any() and not o[1].isnan().any()
    q[0, D] = 0.0
    cache[3][2, 0, 3, 1] = math.nan            # dims 64.. of one value of sequence 0
    out, _ = run_attention(q, cache, bt, lens, None, 1, 64, 0)
    o = out.view(2, hq, D)
    assert o[0, :, 64:].isnan().all() and not o[0, :, :64].isnan().any() and not o[1].isnan().any()
    cache[1][2, 0, 3, 0] = math.nan            # a key's scale: every row of sequence 0
    out, _ = run_attention(q, cache, bt, lens, None, 1, 64, 0)
    assert out[0].isnan().all() and not out[1].isnan().any()


@pytest.mark.gpu
def test_attention_keeps_to_its_bounds():
    """Row ranges and lengths that lie outside the buffers are cut, not followed."""
    g = torch.Generator().manual_seed(7)
    hq, hk, D, ps = 2, 1, 64, 16
    cache = random_cache(4, ps, hk, D, g)
    bt = torch.arange(4, dtype=torch.int32).view(1, 4)
    q = torch.randn((3, hq * D), generator=g).to(BF16).to(DEV)
    for q_start, L, max_q, max_len in (([0, 9], 64, 9, 64), ([-5, 2], 64, 9, 64), ([2, 1], 64, 4, 64), ([7, 9], 64, 4, 64),
                                       ([0, 3], 2 ** 31 - 1, 3, 64), ([0, 3], -7, 3, 64), ([0, 3], 64, 3, 20)):
        out, lse = run_attention(q, cache, bt, torch.tensor([L], dtype=torch.int32), torch.tensor(q_start, dtype=torch.int32),
                                 max_q, max_len, 0)
        assert bool(out.isfinite().all())
        if q_start == [0, 3]:
            check_attention(q, cache, bt, torch.tensor([L], dtype=torch.int32), torch.tensor(q_start, dtype=torch.int32), max_q, max_len)


@pytest.mark.gpu
def test_attention_strided_rows_and_side_stream():
    g = torch.Generator().manual_seed(8)
    hq, hk, D, ps = 8, 2, 128, 16
    cache = random_cache(40, ps, hk, D, g)
    lens = torch.tensor([300, 200], dtype=torch.int32)
    bt = tables(lens, ps, 40, g)
    buf = torch.randn((2, hq * D + 10), generator=g).to(BF16).to(DEV)
    for shift in (0, 1):
        q = buf[:, shift:shift + hq * D]
        want, _ = run_attention(q.contiguous(), cache, bt, lens, None, 1, 300, 0)
        out = torch.full((2, hq * D + 6), 9.0, dtype=BF16, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        qk.qknorm_kv4_attention(q, cache, bt.to(DEV), lens.to(DEV), max_seq_len=300, out=out[:, 3:3 + hq * D], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(out[:, 3:3 + hq * D], want)
        assert bool((out[:, :3] == 9).all()) and bool((out[:, 3 + hq * D:] == 9).all())


# --------------------------------------------------------------------------- together

@pytest.mark.gpu
def test_a_prompt_then_tokens_captured():
    """Projection rows -> append (norm, rotation, 4 bits) -> attention: a prompt
    as one chunk, then decode steps replayed from one graph, against the same
    steps called one by one, and the attention against 64 bits."""
    g = torch.Generator().manual_seed(9)
    hq, hk, D, ps, n, steps = 8, 2, 128, 16, 45, 5
    W = (hq + 2 * hk) * D
    gq, gk = gamma_of(D, BF16, g).to(DEV), gamma_of(D, BF16, g).to(DEV)
    cs = table(128, D).to(DEV)
    w = (torch.randn((W, 256), generator=g) / 16).to(BF16).to(DEV)
    hidden = torch.randn((n + steps, 256), generator=g).to(BF16).to(DEV)
    rows, _, _ = qk.qknorm_qkv_gemm_stats(hidden, w, hq * D, hk * D, hk * D)

    def split(r):
        return r[:, :hq * D], r[:, hq * D:(hq + hk) * D], r[:, (hq + hk) * D:]
    bt = torch.tensor([[3, 0, 5, 2, 1]], dtype=torch.int32, device=DEV)

    def slot(t):
        return bt[0].long()[t // ps] * ps + t % ps

    def prompt(cache):
        t = torch.arange(n, device=DEV)
        q = qk.qknorm_rope_append_kv4(*split(rows[:n]), gq, gk, cs, t, cache, slot(t), EPS)
        return q, qk.qknorm_kv4_attention(q, cache, bt, torch.tensor([n], dtype=torch.int32, device=DEV), max_seq_len=ps * 5,
                                          q_start=torch.tensor([0, n], dtype=torch.int32, device=DEV), max_q_len=n)

    eager = qk.kv4_cache(6, ps, hk, D, DEV)
    q, out = prompt(eager)
    check_attention(q.contiguous(), eager, bt.cpu(), torch.tensor([n], dtype=torch.int32), torch.tensor([0, n], dtype=torch.int32), n, ps * 5)
    want = []
    for i in range(steps):
        t = torch.tensor([n + i], device=DEV)
        q = qk.qknorm_rope_append_kv4(*split(rows[n + i:n + i + 1]), gq, gk, cs, t, eager, slot(t), EPS)
        want.append(qk.qknorm_kv4_attention(q, eager, bt, (t + 1).int(), max_seq_len=ps * 5))
        if i == 0:
            check_attention(q.contiguous(), eager, bt.cpu(), torch.tensor([n + 1], dtype=torch.int32), None, 1, ps * 5)

    cache = qk.kv4_cache(6, ps, hk, D, DEV)
    assert torch.equal(prompt(cache)[1], out)
    x, t = rows[n:n + 1].clone(), torch.tensor([n], device=DEV)
    s1, len1 = slot(t), (t + 1).int()

    def step():
        q = qk.qknorm_rope_append_kv4(*split(x), gq, gk, cs, t, cache, s1, EPS)
        return qk.qknorm_kv4_attention(q, cache, bt, len1, max_seq_len=ps * 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(steps):
        x.copy_(rows[n + i:n + i + 1])
        t.fill_(n + i)
        s1.copy_(slot(t))
        len1.fill_(n + i + 1)
        graph.replay()
        assert torch.equal(got, want[i]), i
    for a, b in zip(cache, eager):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_training_step_captured():
    """Forward and gradient in one graph, replayed on new inputs, equal to eager calls."""
    g = torch.Generator().manual_seed(10)
    T, hq, hk, D = 50, 4, 2, 128
    cs, pos = table(64, D).to(DEV), torch.arange(T, device=DEV)
    gq, gk = gamma_of(D, BF16, g).to(DEV), gamma_of(D, BF16, g).to(DEV)
    x, dy = (torch.randn((T, (hq + hk) * D), generator=g).to(BF16).to(DEV) for _ in range(2))

    def step():
        q, k, dq, dk = x[:, :hq * D], x[:, hq * D:], dy[:, :hq * D], dy[:, hq * D:]
        y = qk.qknorm_headwise_rope(q, k, gq, gk, D, cs, pos)
        return (*y, *qk.qknorm_headwise_rope_backward(dq, dk, q, k, gq, gk, D, cs, pos))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(2):
        x.mul_(-0.7)
        dy.add_(0.25)
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a.contiguous(), b.contiguous())


# --------------------------------------------------------------------------- refusals (no GPU)

OK, INVALID, UNSUPPORTED, CUDA = 0, 1, 3, 4
BASE = 1 << 32


@pytest.fixture(scope="module")
def lib():
    qbuild.build(quiet=True)
    return _clib.load()


def at(i):
    return BASE + (i << 30)


def rope_args(**kw):
    a = dict(q_in=at(0), q_out=at(1), gq=at(2), qs=4096, hq=32, k_in=at(3), k_out=at(4), gk=at(5), ks=1024, hk=8, T=64,
             D=128, cs=at(6), P=4096, rot=128, inter=0, pos=at(7), eps=1e-6, dtype=1, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, CUDA), ({"q_out": at(0), "k_out": at(3)}, CUDA), ({"T": 0, "q_in": 0, "pos": 0}, OK),
    ({"rot": 0, "cs": 0}, CUDA), ({"P": 0, "cs": 0}, CUDA),
    ({"rot": 127}, INVALID), ({"rot": 130}, INVALID), ({"rot": -2}, INVALID), ({"P": -1}, INVALID), ({"pos": 0}, INVALID),
    ({"pos": at(7) + 4}, INVALID), ({"cs": at(6) + 2}, INVALID), ({"cs": 0}, INVALID), ({"hq": 0}, INVALID), ({"hk": -1}, INVALID),
    ({"D": 0}, INVALID), ({"D": 2048, "qs": 1 << 17, "ks": 1 << 17}, UNSUPPORTED), ({"qs": 4095}, INVALID), ({"ks": 1023}, INVALID),
    ({"T": -1}, INVALID), ({"T": 1 << 30}, INVALID), ({"eps": -1.0}, INVALID), ({"eps": float("nan")}, INVALID),
    ({"dtype": 9}, INVALID), ({"dtype": -1}, INVALID), ({"gq": 0}, INVALID), ({"gk": at(5) + 1}, INVALID), ({"q_in": 0}, INVALID),
    ({"q_in": at(0) + 1}, INVALID), ({"q_out": at(0) + 16}, INVALID), ({"q_out": at(3)}, INVALID), ({"k_out": at(1)}, INVALID),
    ({"k_out": at(7)}, INVALID), ({"q_out": at(6) + 1024}, INVALID), ({"q_out": at(2)}, INVALID)])
def test_rope_refusals(lib, kw, status):
    st = lib.qknorm_headwise_rope(*rope_args(**kw))
    if torch.cuda.is_available() and status == CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    assert st == status, lib.qknorm_last_error()


def grad_args(**kw):
    a = dict(q=at(0), qs=4096, dq=at(1), dqs=4096, dqi=at(2), dqis=4096, gq=at(3), dgq=at(4), hq=32, k=at(5), ks=1024, dk=at(6),
             dks=1024, dki=at(7), dkis=1024, gk=at(8), dgk=at(9), hk=8, T=64, D=128, cs=at(10), P=4096, rot=128, inter=0,
             pos=at(11), eps=1e-6, ws=at(12), wb=1 << 24, dtype=1, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, CUDA), ({"dqi": at(1), "dki": at(5)}, CUDA), ({"dtype": 3}, UNSUPPORTED), ({"wb": 100}, INVALID), ({"ws": 0}, INVALID),
    ({"ws": at(12) + 2}, INVALID), ({"dgq": 0}, INVALID), ({"dgk": at(4)}, INVALID), ({"dgk": at(9) + 1}, INVALID),
    ({"dqi": at(6)}, INVALID), ({"dqi": at(1) + 16}, INVALID), ({"dqi": at(0), "dqis": 8192}, INVALID), ({"ws": at(2)}, INVALID),
    ({"dqs": 100}, INVALID), ({"dq": 0}, INVALID), ({"gq": 0}, INVALID), ({"rot": 3}, INVALID), ({"dgq": at(3)}, INVALID)])
def test_gradient_refusals(lib, kw, status):
    if torch.cuda.is_available() and status == CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    assert lib.qknorm_headwise_rope_backward(*grad_args(**kw)) == status, lib.qknorm_last_error()


def test_gradient_workspace(lib):
    f = lib.qknorm_headwise_rope_backward_workspace_bytes
    assert f(0, 32, 8, 128) == 0
    assert f(1, 1, 1, 128) == 2 * 2 * 128 * 4
    assert f(100000, 32, 8, 128) == 592 * 2 * 128 * 4
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0), (1, 1, 1, 1025), (1 << 31, 1, 1, 1)):
        assert f(*bad) == -1
    with pytest.raises(ValueError):
        qk.rope_backward_workspace_bytes(-1, 1, 1, 1)


def append_args(cache, **kw):
    a = dict(q_in=at(0), q_out=at(1), gq=at(2), qs=6144, hq=32, k=at(3), gk=at(4), ks=1024, v=at(5), vs=1024, hk=8, T=64, D=128,
             cs=at(6), P=4096, rot=128, inter=0, pos=at(7), **cache, slots=at(12), eps=1e-6, dtype=1, stream=None)
    a.update(kw)
    return list(a.values())


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


PAGES = dict(kc=at(8), kst=strides(16384, 1024, 128), vc=at(9), vst=strides(16384, 1024, 128), n=100, ps=16)
PAGES4 = dict(kc=at(8), ksc=at(9), vc=at(10), vsc=at(11), n=100, ps=16)


@pytest.mark.parametrize("kw,status", [
    ({}, CUDA), ({"hq": 0, "q_in": 0, "q_out": 0, "gq": 0}, CUDA), ({"gq": 0, "gk": 0}, CUDA), ({"T": 0}, OK),
    ({"kst": strides(16384, 128, 2048), "vst": strides(16384, 128, 2048)}, CUDA),
    ({"vc": at(8) + 16384 * 2, "kst": strides(32768, 1024, 128), "vst": strides(32768, 1024, 128)}, CUDA),
    ({"kst": strides(1024, 102400, 128), "vst": strides(1024, 102400, 128)}, CUDA),  # pages innermost
    ({"n": 0, "kc": 0, "vc": 0}, CUDA),
    ({"gq": 0}, INVALID), ({"gk": 0}, INVALID), ({"slots": 0}, INVALID), ({"slots": at(12) + 1}, INVALID), ({"n": -1}, INVALID),
    ({"ps": 0}, INVALID), ({"n": 1 << 50}, INVALID), ({"kc": 0}, INVALID), ({"kst": None}, INVALID),
    ({"kst": strides(16384, 1024, 127)}, INVALID), ({"kst": strides(16383, 1024, 128)}, INVALID),
    ({"vst": strides(-16384, 1024, 128)}, INVALID), ({"vst": strides(0, 1024, 128)}, INVALID), ({"kst": strides(1 << 61, 1024, 128)}, INVALID),
    ({"vc": at(8) + 4096}, INVALID), ({"kc": at(3)}, INVALID), ({"vc": at(1)}, INVALID), ({"kc": at(12)}, INVALID), ({"kc": at(8) + 1}, INVALID),
    ({"hk": 0}, INVALID), ({"hq": -1}, INVALID), ({"vs": 1000}, INVALID), ({"v": 0}, INVALID), ({"q_out": at(5)}, INVALID)])
def test_append_refusals(lib, kw, status):
    if torch.cuda.is_available() and status == CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    assert lib.qknorm_rope_append(*append_args(PAGES, **kw)) == status, lib.qknorm_last_error()


@pytest.mark.parametrize("kw,status", [
    ({}, CUDA), ({"T": 0}, OK), ({"dtype": 3}, UNSUPPORTED), ({"ps": 24}, UNSUPPORTED), ({"D": 96}, UNSUPPORTED), ({"D": 96, "rot": 96}, UNSUPPORTED),
    ({"ps": 0}, INVALID), ({"n": -1}, INVALID), ({"kc": 0}, INVALID), ({"vsc": at(11) + 8}, INVALID), ({"ksc": at(8)}, INVALID),
    ({"vc": at(8) + 16}, INVALID), ({"vsc": at(5)}, INVALID), ({"kc": at(7)}, INVALID), ({"n": 1 << 58}, INVALID), ({"gk": 0}, INVALID)])
def test_append_kv4_refusals(lib, kw, status):
    if torch.cuda.is_available() and status == CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    if kw.get("D") == 96:
        kw = {"rot": 64, **kw}
    assert lib.qknorm_rope_append_kv4(*append_args(PAGES4, **kw)) == status, lib.qknorm_last_error()


def attn_args(**kw):
    a = dict(q=at(0), qs=4096, out=at(1), os=4096, lse=at(2), hq=32, kc=at(3), ks=at(4), vc=at(5), vs=at(6), n=100, ps=16, hk=8,
             D=128, bt=at(7), mp=64, sl=at(8), qst=0, T=64, B=64, mq=1, ml=1024, win=0, scale=0.1, ws=at(9), wb=1 << 29, dtype=1,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,status", [
    ({}, CUDA), ({"T": 0, "B": 0}, OK), ({"lse": 0}, CUDA), ({"qst": at(10), "mq": 7}, CUDA), ({"n": 0, "kc": 0, "ks": 0, "vc": 0, "vs": 0}, CUDA),
    ({"dtype": 0}, UNSUPPORTED), ({"dtype": 3}, UNSUPPORTED), ({"dtype": 5}, INVALID), ({"D": 96}, UNSUPPORTED), ({"ps": 8}, UNSUPPORTED),
    ({"hq": 30}, INVALID), ({"hq": 0}, INVALID), ({"scale": float("nan")}, INVALID), ({"scale": float("inf")}, INVALID), ({"win": -1}, INVALID),
    ({"mq": 0}, INVALID), ({"mq": 2}, INVALID), ({"T": 63}, INVALID), ({"ml": -1}, INVALID), ({"mp": -1}, INVALID), ({"q": 0}, INVALID),
    ({"bt": 0}, INVALID), ({"sl": 0}, INVALID), ({"sl": at(8) + 2}, INVALID), ({"qs": 4095}, INVALID), ({"os": 10}, INVALID),
    ({"q": at(0) + 1}, INVALID), ({"kc": at(3) + 8}, INVALID), ({"out": at(0)}, INVALID), ({"lse": at(1)}, INVALID), ({"out": at(5)}, INVALID),
    ({"T": 1 << 28}, INVALID), ({"B": 70000, "T": 70000}, UNSUPPORTED), ({"vs": 0}, INVALID)])
def test_attention_refusals(lib, kw, status):
    if torch.cuda.is_available() and status == CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    assert lib.qknorm_kv4_attention(*attn_args(**kw)) == status, lib.qknorm_last_error()


def test_wrappers_refuse_host_tensors():
    x, one, cs = torch.zeros((2, 128)), torch.ones(64), table(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_headwise_rope(x, x, one, one, 64, cs, torch.zeros(2, dtype=torch.int64))
    cache = qk.kv4_cache(2, 16, 1, 128, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_kv4_read(cache, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_rope_append_kv4(None, x, x, one, one, cs, torch.zeros(2, dtype=torch.int64), cache,
                                  torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        qk.qknorm_kv4_attention(x.bfloat16(), cache, torch.zeros((2, 1), dtype=torch.int32),
                                torch.zeros(2, dtype=torch.int32), max_seq_len=16)
    with pytest.raises(ValueError):
        qk.kv4_cache(2, 8, 1, 128, "cpu")
    with pytest.raises(ValueError):
        qk.kv4_cache(2, 16, 1, 96, "cpu")
