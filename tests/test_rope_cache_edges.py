"""Corners of the rotation, paged-cache and 4-bit attention calls: values at the
ends of the number range, sizes at which a kernel's loops go round more than
once, bounds at the ends of their types, streams given as handles.  The formulas
in 64 bits and their tolerances are test_rope_cache.py's."""
from __future__ import annotations

import pytest
import torch

import attention_normalization_b200 as qk
import test_rope_cache as rc
from test_rope_cache import BF16, DEV, EPS, F16, F32


# --------------------------------------------------------------------------- 4-bit append

@pytest.mark.gpu
@pytest.mark.parametrize("dtype,shift", [(BF16, 0), (F32, 0), (BF16, 3)])
@pytest.mark.parametrize("D,rot,inter", [(64, 64, False), (128, 64, True), (256, 256, False)])
@pytest.mark.parametrize("eps,sizes", [
    (EPS, (3e18, 1e19, 1e25, 1e30)),             # the squared sum passes fp32's largest number, x does not
    (0.0, (1e-22, 1e-24, 1e-30, 1e-38, 1e18)),   # and its smallest, with nothing added to it
    (1e-38, (1e-19, 1e-25))])
def test_append_kv4_of_keys_whose_squared_sum_leaves_fp32(eps, sizes, D, rot, inter, dtype, shift):
    """Codes and scales are the formula's in 64 bits there too, whichever kernel
    takes the rows (shift: the element-wise one)."""
    g = torch.Generator().manual_seed(D + len(sizes))
    hk, ps = 2, 16
    T = 3 * len(sizes)
    x = torch.randn((T, 2 * hk * D), generator=g) * torch.tensor(sizes).repeat(3)[:, None]
    buf = torch.zeros(T * 2 * hk * D + shift)
    buf[shift:] = x.reshape(-1)
    x = buf.to(dtype).to(DEV)[shift:].view(T, 2 * hk * D)
    k, v = x[:, :hk * D], x[:, hk * D:]
    gm, cs, pos = rc.gamma_of(D, dtype, g), rc.table(40, rot), torch.randint(0, 40, (T,), generator=g)
    cache = qk.kv4_cache(2, ps, hk, D, DEV)
    slots = torch.arange(T)
    qk.qknorm_rope_append_kv4(None, k, v, None, gm.to(DEV), cs.to(DEV), pos.to(DEV), cache, slots.to(DEV), eps,
                              interleaved=inter)
    y = rc.forward(k, gm, D, cs, pos, inter, eps)[0]
    for want, codes, scales in ((y, *cache[:2]), (rc.f64(v).reshape(T, hk, D), *cache[2:])):
        c, s = rc.quantise(want.numpy())
        assert torch.equal(scales.cpu()[slots // ps, :, slots % ps], torch.from_numpy(s))
        assert torch.equal(rc.unpack(codes.cpu())[slots // ps, :, slots % ps], torch.from_numpy(c))
