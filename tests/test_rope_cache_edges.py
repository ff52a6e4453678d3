"""Corners of the rotation, paged-cache and 4-bit attention calls: values at the
ends of the number range, sizes at which a kernel's loops go round more than
once, bounds at the ends of their types, streams given as handles.  The formulas
in 64 bits and their tolerances are test_rope_cache.py's."""
from __future__ import annotations

import math

import pytest
import torch

import attention_normalization_b200 as qk
import test_rope_cache as rc
from attention_normalization_b200 import _clib, rope_cache
from attention_normalization_b200 import build as qbuild
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


# --------------------------------------------------------------------------- streams

def test_tensors_made_for_a_raw_stream_handle_are_recorded(monkeypatch):
    """What a call allocates and drops is kept by the allocator until a stream
    given as an integer is done with it, as for a torch stream."""
    made = []

    class External:
        def __init__(self, handle, device):
            made.append((handle, device))

    class Held:
        def __init__(self):
            self.streams = []

        def get_device(self):
            return 3

        def record_stream(self, s):
            self.streams.append(s)
    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    a, b = Held(), Held()
    rope_cache._used_on(0x7F00, a, b)
    assert made == [(0x7F00, 3)] and len(a.streams) == len(b.streams) == 1
    assert isinstance(a.streams[0], External) and a.streams[0] is b.streams[0]
    rope_cache._used_on(0, a)
    assert a.streams[1] == ("default", 3)
    rope_cache._used_on(None, a)
    rope_cache._used_on(0x7F00)
    assert len(a.streams) == 2 and len(made) == 1


@pytest.mark.gpu
def test_workspaces_of_calls_on_a_raw_stream_handle():
    """Attention over a split cache and a gradient on a stream given as an
    integer that is still busy, while the current stream allocates and fills
    buffers of the sizes of the workspaces that the calls have dropped."""
    g = torch.Generator().manual_seed(15)
    hq, hk, D, ps, L, T = 8, 2, 128, 64, 9000, 700
    pages = -(-L // ps)
    bt, lens = torch.arange(pages, dtype=torch.int32, device=DEV).view(1, -1), torch.tensor([L], dtype=torch.int32, device=DEV)
    cache = rc.random_cache(pages, ps, hk, D, g)
    q = torch.randn((1, hq * D), generator=g).to(BF16).to(DEV)
    x, dy = (torch.randn((T, hq * D), generator=g).to(BF16).to(DEV) for _ in range(2))
    gm, cs, pos = rc.gamma_of(D, BF16, g).to(DEV), rc.table(T, D).to(DEV), torch.arange(T, device=DEV)
    sizes = [qk.kv4_attention_workspace_bytes(1, 1, hq, hk, D, 1, L), qk.rope_backward_workspace_bytes(T, hq, hq, D)]
    assert min(sizes) > 0
    big = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)

    def calls(stream):
        return [qk.qknorm_kv4_attention(q, cache, bt, lens, max_seq_len=L, stream=stream),
                *qk.qknorm_headwise_rope_backward(dy, dy, x, x, gm, gm, D, cs, pos, stream=stream)]
    alone = calls(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(8):
                big.zero_()  # keeps the stream busy until the buffers below are filled
        got = calls(side.cuda_stream)
        fill = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert torch.equal(a, b)
        del fill


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True])
def test_workspace_of_a_projection_on_another_stream(raw):
    """The partial sums that the projection makes room for and drops, on a busy
    stream, while the current stream allocates and fills buffers of their size."""
    g = torch.Generator().manual_seed(16)
    T, Dm, Hq, Hk = 512, 256, 512, 256
    x = torch.randn((T, Dm), generator=g).to(BF16).to(DEV)
    w = (torch.randn((Hq + 2 * Hk, Dm), generator=g) / 16).to(BF16).to(DEV)
    gq, gk = rc.gamma_of(Hq, BF16, g).to(DEV), rc.gamma_of(Hk, BF16, g).to(DEV)
    n = qk.qkv_workspace_bytes(T, Hq, Hk)
    assert n > 0
    big = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    alone = qk.qknorm_qkv_projection(x, w, gq, gk, Hq, Hk, Hk)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            for _ in range(8):
                big.zero_()
        got = qk.qknorm_qkv_projection(x, w, gq, gk, Hq, Hk, Hk, stream=side.cuda_stream if raw else side)
        fill = [torch.empty(n, dtype=torch.uint8, device=DEV).fill_(0xFF) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, alone)
        del fill


# --------------------------------------------------------------------------- attention

@pytest.mark.gpu
@pytest.mark.parametrize("rows,D,scales,n,octaves,strong", [
    (1, 128, (64.0, 2.0 ** -14), 1020, 8.3, (0, 32, 64, 96)),     # one CTA, a strong token for each of its warps
    (1, 128, (2.0 ** -14, 64.0), 1020, 8.3, (0, 32, 64, 96)),
    (4, 128, (2.0 ** -14, 64.0), 1016, 8.3, (0, 32, 64, 96)),     # 16 query rows
    (1, 256, (2.0 ** -4, 2.0 ** -14, 16.0, 2.0 ** -9), 1020, 8.3, (0, 32, 64, 96)),
    (1, 128, (1.0, 2.0 ** -13), 131072, 18.2, (0,)),              # cut into shares; the tail is 30% of the weight
    (4, 128, (2.0 ** -10, 8.0), 30000, 13.62, (20000,)),
    (1, 256, (2.0 ** -4, 2.0 ** -13, 16.0, 2.0 ** -9), 30000, 13.62, (29999,)),
    (1, 64, (0.5,), 30000, 13.62, (0,))])
def test_attention_of_groups_whose_value_scales_are_far_apart(rows, D, scales, n, octaves, strong):
    """A few strong tokens and a long tail, `octaves` powers of two below them, of
    equal weights and positive values, so that rounding errors of the weights do
    not cancel: every group of dims keeps its tail, whatever the other groups'
    scales are.  Heads at other multiples of the scores come along.  The
    tolerance counts 2^-11 of each product and 2^-28 of the row's largest for what
    lies further below."""
    g = torch.Generator().manual_seed(n + D)
    ps, hq = 64, 4
    L = n + rows
    pages = -(-L // ps)
    cache = qk.kv4_cache(pages, ps, 1, D, DEV)
    for t in strong:                                 # codes of 7; the other keys are zeros
        cache[0][t // ps, 0, t % ps] = 0xFF
        cache[1][t // ps, 0, t % ps] = octaves * math.log(2.0) / (7 * math.sqrt(D))
    cache[2].copy_(torch.randint(9, 16, cache[2].shape, generator=g) | torch.randint(9, 16, cache[2].shape, generator=g) << 4)
    cache[3].copy_(torch.tensor(scales))
    q = torch.tensor([1.0, 0.5, -1.0, 0.9375]).repeat_interleave(D).repeat(rows, 1).to(BF16).to(DEV)
    rc.check_attention(q, cache, torch.arange(pages, dtype=torch.int32).view(1, -1), torch.tensor([L], dtype=torch.int32),
                       torch.tensor([0, rows], dtype=torch.int32), rows, L)


@pytest.fixture(scope="module")
def lib():
    qbuild.build(quiet=True)
    return _clib.load()


HEADS = [(32, 8, 128), (8, 8, 64), (32, 8, 64), (6, 2, 256), (20, 1, 128)]


@pytest.mark.parametrize("hq,hk,D", HEADS)
def test_attention_workspace_grows_with_every_bound(lib, hq, hk, D):
    f = lib.qknorm_kv4_attention_workspace_bytes
    batches, q_lens, lens = (0, 1, 2, 7, 37, 64, 110, 111, 400, 5000), (1, 2, 3, 8, 9, 50, 400), (0, 1024, 1025, 2048, 2049, 4096, 100000, 1 << 30)
    size = {(b, n, s): f(1, b, hq, hk, D, n, s) for b in batches for n in q_lens for s in lens}
    assert min(size.values()) == 0 and 0 < max(size.values()) < 32 << 20
    for i, b in enumerate(batches):
        for j, n in enumerate(q_lens):
            for k, s in enumerate(lens):
                for key in ((batches[max(i - 1, 0)], n, s), (b, q_lens[max(j - 1, 0)], s), (b, n, lens[max(k - 1, 0)])):
                    assert size[key] <= size[b, n, s], (key, (b, n, s))


@pytest.mark.parametrize("hq,hk,D", HEADS)
@pytest.mark.parametrize("most", [(120, 1), (120, 5), (5000, 2)])
def test_attention_workspace_of_the_largest_call_serves_smaller_ones(lib, most, hq, hk, D):
    """The call's own check, on addresses that nothing reads: it goes on to the
    launch, which fails for want of a device."""
    if torch.cuda.is_available():
        pytest.skip("an accepted call with made-up addresses is not launched")
    B, n, s = *most, 4096
    bytes_ = lib.qknorm_kv4_attention_workspace_bytes(B * n, B, hq, hk, D, n, s)
    for b in (1, 2, 3, 11, 56, 64, 110, 111, B):
        for m in range(1, n + 1):
            for t in (s, 2048, 1500, 16):
                st = lib.qknorm_kv4_attention(*rc.attn_args(
                    q=rc.at(0), qs=hq * D, out=rc.at(1), os=hq * D, lse=0, hq=hq, hk=hk, D=D, qst=rc.at(10), T=b * m, B=b, mq=m,
                    ml=t, wb=bytes_))
                assert st == rc.CUDA, (b, m, t, lib.qknorm_last_error())


@pytest.mark.gpu
def test_one_workspace_for_every_batch():
    g = torch.Generator().manual_seed(17)
    hq, hk, D, ps, L, most = 16, 8, 128, 64, 1500, 120
    pages = -(-L // ps)
    cache = rc.random_cache(pages, ps, hk, D, g)
    bt = torch.randint(0, pages, (most, pages), generator=g).int().to(DEV)
    lens = torch.randint(1, L + 1, (most,), generator=g).int().to(DEV)
    q = torch.randn((most, hq * D), generator=g).to(BF16).to(DEV)
    held = torch.empty(qk.kv4_attention_workspace_bytes(most, most, hq, hk, D, 1, L), dtype=torch.uint8, device=DEV)
    for B in (1, 5, 40, 56, most):
        args = (q[:B], cache, bt[:B], lens[:B])
        assert torch.equal(qk.qknorm_kv4_attention(*args, max_seq_len=L, workspace=held),
                           qk.qknorm_kv4_attention(*args, max_seq_len=L))


@pytest.mark.gpu
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 21, 20, 19, 1])
@pytest.mark.parametrize("hq,hk,rows,L", [(4, 2, 30, 20), (16, 1, 30, 20), (2, 2, 1, 20), (8, 1, 3, 1)])
def test_attention_windows_as_long_as_the_sequence_and_longer(hq, hk, rows, L, window):
    """With more rows than cached tokens too, whose first rows lie before the sequence."""
    g = torch.Generator().manual_seed(rows + hq)
    cache = rc.random_cache(3, 16, hk, 128, g)
    q = torch.randn((rows, hq * 128), generator=g).to(BF16).to(DEV)
    rc.check_attention(q, cache, torch.tensor([[2, 0]], dtype=torch.int32), torch.tensor([L], dtype=torch.int32),
                       torch.tensor([0, rows], dtype=torch.int32), rows, 32, window)


@pytest.mark.parametrize("kw,status", [
    ({"ml": 2 ** 31 - 1}, rc.CUDA), ({"mp": 2 ** 31 - 1}, rc.CUDA), ({"ml": 2 ** 31 - 2 ** 21, "mp": 2 ** 27}, rc.CUDA),
    ({"ml": 2 ** 31 - 2 ** 21 + 1, "mp": 2 ** 27}, rc.UNSUPPORTED), ({"win": 2 ** 31 - 1}, rc.CUDA)])
def test_attention_bounds_at_the_ends_of_their_type(lib, kw, status):
    if torch.cuda.is_available() and status == rc.CUDA:
        pytest.skip("an accepted call with made-up addresses is not launched")
    # one sequence: its page table of 2^31 entries stays below the next address
    st = lib.qknorm_kv4_attention(*rc.attn_args(**{"T": 1, "B": 1, "bt": 1 << 44, **kw}))
    assert st == status, lib.qknorm_last_error()


# --------------------------------------------------------------------------- autograd

def test_operands_that_autograd_follows_are_refused():
    """Every call that would drop a gradient says so (the operands' devices are looked at later)."""
    x, one, cs = torch.zeros((2, 128)), torch.ones(64), rc.table(4, 64)
    pos, cache = torch.zeros(2, dtype=torch.int64), qk.kv4_cache(2, 16, 2, 64, "cpu")
    bt, lens, pages = torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, dtype=torch.int32), torch.zeros((2, 16, 2, 64))
    calls = [(lambda q, k, v, gq, gk: qk.qknorm_headwise_rope(q, k, gq, gk, 64, cs, pos), (0, 1, 3, 4)),
             (lambda q, k, v, gq, gk: qk.qknorm_headwise_rope_backward(q, k, x, x, gq, gk, 64, cs, pos), (0, 1)),
             (lambda q, k, v, gq, gk: qk.qknorm_rope_append(q, k, v, gq, gk, 64, cs, pos, pages, pages.clone(), pos), range(5)),
             (lambda q, k, v, gq, gk: qk.qknorm_rope_append_kv4(q, k, v, gq, gk, cs, pos, cache, pos), range(5)),
             (lambda q, k, v, gq, gk: qk.qknorm_kv4_attention(q, cache, bt, lens, max_seq_len=16), (0,))]
    for call, tracked in calls:
        for i in tracked:
            args = [x.clone(), x.clone(), x.clone(), one.clone(), one.clone()]
            args[i].requires_grad_()
            with pytest.raises(ValueError, match="autograd"):
                call(*args)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(*args)


@pytest.mark.gpu
def test_a_training_step_in_an_autograd_function():
    """Forward and gradient in a torch.autograd.Function as a user writes it,
    against autograd through the formula in 64 bits; grads that come as an
    expanded scalar are made rows first, gammas get their own type back."""
    g = torch.Generator().manual_seed(18)
    T, hq, hk, D = 21, 4, 2, 64
    cs, pos = rc.table(40, D), torch.randint(0, 40, (T,), generator=g)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, gq, gk):
            ctx.save_for_backward(q, k, gq, gk)
            return qk.qknorm_headwise_rope(q, k, gq, gk, D, cs.to(DEV), pos.to(DEV))

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dq, dk):
            q, k, gq, gk = ctx.saved_tensors
            dq, dk, dgq, dgk = qk.qknorm_headwise_rope_backward(dq.contiguous(), dk.contiguous(), q, k, gq, gk, D, cs.to(DEV),
                                                                pos.to(DEV))
            return dq, dk, dgq.to(gq.dtype), dgk.to(gk.dtype)
    leaves = [torch.randn((T, h * D), generator=g).to(DEV).requires_grad_() for h in (hq, hk)]
    leaves += [rc.gamma_of(D, F32, g).to(DEV).requires_grad_() for _ in range(2)]
    w = torch.randn((T, hq * D), generator=g).to(DEV)
    q, k = Rope.apply(*leaves)
    ((q * w).sum() + k.sum()).backward()
    for x, dy, gm, dx, dg in ((leaves[0], w, leaves[2], leaves[0].grad, leaves[2].grad),
                              (leaves[1], torch.ones_like(leaves[1]), leaves[3], leaves[1].grad, leaves[3].grad)):
        want, mag, want_g, mag_g = rc.gradient(x, dy, gm, D, cs, pos, False)
        rc.check(dx, want, mag, F32, rel=2.0 ** -16)
        assert bool(((rc.f64(dg) - want_g).abs() <= (2.0 ** -17 + T * hq * 2.0 ** -24) * mag_g + 1e-30).all())


# --------------------------------------------------------------------------- sizes at which the kernels' loops go round
#
# The vector kernels take several lots of a token's heads in one warp from 24
# warps' rows per SM on (14208 rows of 128 dims of bf16, twice that of 64 dims),
# the gradient's CTAs take tokens in turn from 2368 warps' on.  Head counts leave
# a remainder in the last lot.

LARGE = [  # T, q heads, k heads, D, rotary, interleaved, pad, shift
    (3001, 13, 5, 128, 128, False, 0, 0),
    (3001, 13, 5, 128, 64, True, 16, 0),
    (2503, 19, 3, 64, 64, False, 0, 0),
    (3001, 11, 3, 96, 96, True, 0, 0),
    (2003, 7, 3, 256, 128, False, 0, 0),
    (1501, 13, 5, 128, 128, False, 0, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32, rc.E4M3])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,pad,shift", LARGE)
def test_rotation_of_many_rows(T, hq, hk, D, rot, inter, pad, shift, dtype):
    g = torch.Generator().manual_seed(T + D)
    _, q = rc.rows_of(T, hq * D, dtype, g, pad, shift)
    _, k = rc.rows_of(T, hk * D, dtype, g, pad, shift)
    gq, gk = rc.gamma_of(D, dtype, g), rc.gamma_of(D, dtype, g)
    P = 997
    cs, pos = rc.table(P, rot), torch.randint(-40, P + 40, (T,), generator=g)
    args = (gq.to(DEV), gk.to(DEV), D, cs.to(DEV), pos.to(DEV), EPS)
    qo, ko = qk.qknorm_headwise_rope(q, k, *args, interleaved=inter)
    for got, x, gm in ((qo, q, gq), (ko, k, gk)):
        rc.check(got, *rc.forward(x, gm, D, cs, pos, inter), dtype)
    for a, b in zip(qk.qknorm_headwise_rope(q, k, *args, interleaved=inter, q_out=q, k_out=k), (qo, ko)):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,pad,shift", [*LARGE, (9000, 40, 8, 128, 128, False, 0, 0), (20011, 5, 2, 64, 32, True, 0, 0)])
def test_gradient_of_many_rows(T, hq, hk, D, rot, inter, pad, shift, dtype):
    g = torch.Generator().manual_seed(T + D)
    (_, q), (_, k), (_, dq), (_, dk) = (rc.rows_of(T, h * D, dtype, g, p, shift) for h, p in ((hq, pad), (hk, 0), (hq, 2 * pad), (hk, pad)))
    gq, gk = rc.gamma_of(D, dtype, g), rc.gamma_of(D, dtype, g)
    P = 997
    cs, pos = rc.table(P, rot), torch.randint(-40, P, (T,), generator=g)
    args = (gq.to(DEV), gk.to(DEV), D, cs.to(DEV), pos.to(DEV), EPS)
    out = qk.qknorm_headwise_rope_backward(dq, dk, q, k, *args, interleaved=inter)
    for got, dg, x, dy, gm in ((out[0], out[2], q, dq, gq), (out[1], out[3], k, dk, gk)):
        dx, dx_mag, want, mag = rc.gradient(x, dy, gm, D, cs, pos, inter)
        rc.check(got, dx, dx_mag, dtype, rel=2.0 ** -16)
        # dgamma: 2368 warps; a lane adds T * heads / 2368 products at most and one lot more of each item it takes
        # (under 200 here), then 5 + 8 + 19 + 32 sums in fixed order
        assert T * max(hq, hk) / 2368 < 160
        assert bool(((rc.f64(dg) - want).abs() <= (2.0 ** -17 + 264 * 2.0 ** -24) * mag + 1e-30).all())
    again = qk.qknorm_headwise_rope_backward(dq, dk, q, k, *args, interleaved=inter)
    inside = qk.qknorm_headwise_rope_backward(dq, dk, q.clone(), k.clone(), *args, interleaved=inter, dq_in=dq, dk_in=dk)
    for a, b, c in zip(out, again, inside):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["tokens first", "heads first"])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm", [
    (3001, 13, 5, 128, 128, False, True), (2503, 19, 11, 64, 64, True, False), (3001, 0, 7, 128, 64, False, True)])
def test_append_of_many_rows(T, hq, hk, D, rot, inter, norm, layout, dtype):
    g = torch.Generator().manual_seed(T + D)
    ps = 32
    W = (hq + 2 * hk) * D
    _, x = rc.rows_of(T, W, dtype, g)
    q, k, v = x[:, :hq * D] if hq else None, x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:]
    gq, gk = (rc.gamma_of(D, dtype, g), rc.gamma_of(D, dtype, g)) if norm else (None, None)
    P = 997
    cs, pos = rc.table(P, rot), torch.randint(-40, P + 40, (T,), generator=g)
    pages = T // ps + 4
    slots = rc.slots_of(T, pages, ps, g)
    buf, kc, vc = rc.caches_of(layout, pages, ps, hk, D, dtype, g)
    bits = {2: torch.int16, 4: torch.int32}[buf.element_size()]
    want_v = vc.cpu()
    kept = kc.cpu()
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo = qk.qknorm_rope_append(q, k, v, to(gq), to(gk), D, to(cs), to(pos), kc, vc, to(slots), EPS, interleaved=inter)
    if hq:
        rc.check(qo, *rc.forward(q, gq, D, cs, pos, inter), dtype)
    held = (slots >= 0) & (slots < pages * ps)
    at = (slots[held] // ps, slots[held] % ps)
    y, mag = rc.forward(k, gk, D, cs, pos, inter)
    rc.check(kc.cpu()[at], y[held], mag[held], dtype)
    want_v[at] = v.cpu().reshape(T, hk, D)[held]
    assert torch.equal(vc.cpu().contiguous().view(bits), want_v.contiguous().view(bits))
    other = torch.ones((pages, ps), dtype=torch.bool)
    other[at] = False
    assert torch.equal(kc.cpu()[other].view(bits), kept[other].view(bits))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter,norm", [
    (3001, 13, 5, 128, 128, False, True), (1501, 2, 21, 128, 64, True, True), (3001, 0, 19, 64, 64, False, True),
    (2003, 3, 9, 256, 256, False, False)])
def test_append_kv4_of_many_rows(T, hq, hk, D, rot, inter, norm, dtype):
    """Codes and scales to the last one, at sizes where some keys lie next to a border."""
    g = torch.Generator().manual_seed(T + D)
    ps = 32
    W = (hq + 2 * hk) * D
    _, x = rc.rows_of(T, W, dtype, g)
    q, k, v = x[:, :hq * D] if hq else None, x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:]
    gq, gk = (rc.gamma_of(D, dtype, g), rc.gamma_of(D, dtype, g)) if norm else (None, None)
    P = 997
    cs, pos = rc.table(P, rot), torch.randint(-40, P + 40, (T,), generator=g)
    pages = T // ps + 4
    slots = rc.slots_of(T, pages, ps, g)
    cache = qk.kv4_cache(pages, ps, hk, D, DEV)
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    qo = qk.qknorm_rope_append_kv4(q, k, v, to(gq), to(gk), to(cs), to(pos), cache, to(slots), EPS, interleaved=inter)
    if hq:
        rc.check(qo, *rc.forward(q, gq, D, cs, pos, inter), dtype)
    held = (slots >= 0) & (slots < pages * ps)
    page, off = slots[held] // ps, slots[held] % ps
    for y, codes, scales in ((rc.forward(k, gk, D, cs, pos, inter)[0], *cache[:2]), (rc.f64(v).reshape(T, hk, D), *cache[2:])):
        c, s = rc.quantise(y[held].numpy())
        want_c, want_s = torch.full(codes.shape[:-1] + (D,), 8, dtype=torch.uint8), torch.zeros(scales.shape, dtype=torch.float16)
        want_c[page, :, off], want_s[page, :, off] = torch.from_numpy(c), torch.from_numpy(s)
        assert torch.equal(rc.unpack(codes.cpu()), want_c)
        assert torch.equal(scales.cpu().view(torch.int16)[~want_s.isnan()], want_s.view(torch.int16)[~want_s.isnan()])
        assert torch.equal(scales.cpu().isnan(), want_s.isnan())


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16), (256, BF16)])
@pytest.mark.parametrize("hq,hk,qn,lens,window,sharp", [
    (8, 2, [4, 4], [5000, 4999], 0, 1.0), (8, 2, [5, 0, 2], [3000, 2500, 1700], 0, 8.0), (6, 2, [9, 6], [4100, 1100], 900, 1.0),
    (2, 1, [11], [9001], 0, 8.0), (20, 1, [1, 2], [2100, 4000], 0, 1.0)])
def test_attention_of_chunks_over_long_caches(hq, hk, qn, lens, window, sharp, D, dtype):
    """Several query tiles a sequence, cut into shares; with sharp scores the
    references move on the way."""
    g = torch.Generator().manual_seed(sum(lens) + D)
    ps = 32
    pages = sum(-(-n // ps) for n in lens) + 1
    cache = rc.random_cache(pages, ps, hk, D, g)
    q_start = torch.tensor([0] + qn).cumsum(0).int()
    q = torch.randn((int(q_start[-1]) + 1, hq * D), generator=g).to(dtype).to(DEV)
    args = (q, cache, rc.tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32), q_start, max(qn), max(lens), window)
    assert qk.kv4_attention_workspace_bytes(q.shape[0], len(qn), hq, hk, D, max(qn), max(lens)) > 0
    got, lse = rc.check_attention(*args, scale=sharp / math.sqrt(D))
    again, lse2 = rc.run_attention(*args, scale=sharp / math.sqrt(D))
    assert torch.equal(got, again) and torch.equal(lse, lse2)


# --------------------------------------------------------------------------- sizes past 32 bits

@pytest.mark.parametrize("size", [2 ** 31, 2 ** 32, 2 ** 32 + 16, 2 ** 40, -2 ** 32 + 16])
def test_bounds_past_32_bits_are_refused_not_cut_off(size):
    """2^32 as "no bound" would otherwise arrive as 0 and cut every sequence there."""
    x, cache = torch.zeros((1, 128), dtype=BF16), qk.kv4_cache(1, 16, 1, 128, "cpu")
    bt, lens = torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    for kw in ({"max_seq_len": size}, {"max_seq_len": 16, "max_q_len": size}, {"max_seq_len": 16, "window": size}):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qk.qknorm_kv4_attention(x, cache, bt, lens, **kw)
    for i in range(1, 7):
        args = [1, 1, 8, 8, 128, 1, 16]
        args[i] = size
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qk.kv4_attention_workspace_bytes(*args)
    for i in range(1, 4):
        args = [1, 8, 8, 128]
        args[i] = size
        with pytest.raises(ValueError, match="2\\*\\*31"):
            qk.rope_backward_workspace_bytes(*args)


# --------------------------------------------------------------------------- whole units or shares

def needs_workspace(lib, **kw):
    """Whether the call cuts its units into shares: it then refuses an absent workspace."""
    st = lib.qknorm_kv4_attention(*rc.attn_args(**{"qs": 1 << 13, "os": 1 << 13, "lse": 0, "qst": rc.at(10), "ws": 0, "wb": 0,
                                                   "mp": 1 << 17, **kw}))
    assert st in (rc.CUDA, rc.INVALID), lib.qknorm_last_error()
    return st == rc.INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call with made-up addresses is not launched")
def test_units_are_as_long_as_their_window(lib):
    long = dict(T=64, B=64, mq=1, ml=32768)
    assert needs_workspace(lib, **long)
    assert not needs_workspace(lib, **long, win=512)
    assert needs_workspace(lib, **{**long, "B": 4, "T": 4}, win=2048)
    assert not needs_workspace(lib, **{**long, "B": 4, "T": 4}, win=1024)
    assert not needs_workspace(lib, **{**long, "B": 4, "T": 4, "ml": 1024}, win=4096)


@pytest.mark.gpu
@pytest.mark.parametrize("D,hq,hk,rows,window", [(128, 8, 2, 1, 500), (64, 8, 8, 1, 17), (256, 4, 1, 3, 300), (128, 16, 2, 5, 1000)])
def test_attention_in_a_window_of_a_long_cache(D, hq, hk, rows, window):
    g = torch.Generator().manual_seed(D + window)
    ps, lens, qn = 32, [6000, 40, 2777], [rows, rows, 1]
    pages = sum(-(-n // ps) for n in lens) + 1
    cache = rc.random_cache(pages, ps, hk, D, g)
    q_start = torch.tensor([0] + qn).cumsum(0).int()
    q = torch.randn((int(q_start[-1]), hq * D), generator=g).to(BF16).to(DEV)
    rc.check_attention(q, cache, rc.tables(lens, ps, pages, g), torch.tensor(lens, dtype=torch.int32), q_start, rows, 6000, window)


@pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call with made-up addresses is not launched")
@pytest.mark.parametrize("D,B,rows,L,shares", [
    (128, 64, 1, 4096, True), (128, 64, 1, 2048, False), (128, 4, 1, 2048, True), (128, 4, 1, 1024, False), (128, 128, 1, 4096, False),
    (64, 64, 1, 4096, True), (64, 16, 1, 4096, True), (64, 16, 1, 2048, False), (64, 128, 1, 4096, False),
    (256, 16, 1, 2048, True), (256, 64, 1, 1024, False), (256, 4, 1, 1024, False),
    (128, 64, 4, 4096, False), (128, 16, 8, 4096, True), (64, 64, 4, 4096, False), (64, 16, 8, 2048, False),
    (128, 1, 200, 4096, False), (128, 16, 9, 8192, True), (64, 64, 4, 8192, True)])
def test_units_are_cut_where_that_was_faster(lib, D, B, rows, L, shares):
    """The rule's two sides at sizes where both were measured (the comment beside it)."""
    assert needs_workspace(lib, D=D, B=B, T=B * rows, mq=rows, ml=L) == shares


# --------------------------------------------------------------------------- in place on packed rows

@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("T,hq,hk,D,rot,inter", [(1, 4, 2, 128, 128, False), (50, 6, 2, 64, 32, True), (3001, 13, 5, 128, 128, False)])
def test_append_with_its_q_rows_in_place(T, hq, hk, D, rot, inter, shift):
    """Q's columns of packed rows turned where they are, K's and V's beside them read."""
    g = torch.Generator().manual_seed(T + D)
    ps, W = 16, (hq + 2 * hk) * D
    pages = T // ps + 4
    buf, _ = rc.rows_of(T, W, BF16, g, 16, shift)
    gm, cs = rc.gamma_of(D, BF16, g).to(DEV), rc.table(64, rot).to(DEV)
    pos, slots = torch.randint(-2, 66, (T,), generator=g).to(DEV), rc.slots_of(T, pages, ps, g).to(DEV)
    caches = [[torch.zeros((pages, ps, hk, D), dtype=BF16, device=DEV) for _ in range(2)] for _ in range(2)]
    four = [qk.kv4_cache(pages, ps, hk, D, DEV) for _ in range(2)]

    def rows():  # at the same alignment each time: the element-wise kernel sums in another order
        r = buf.clone()[shift:shift + T * (W + 16)].view(T, W + 16)
        return r[:, :hq * D], r[:, hq * D:(hq + hk) * D], r[:, (hq + hk) * D:W]
    now, now4, kept = rows(), rows(), rows()
    apart = qk.qknorm_rope_append(*kept, gm, gm, D, cs, pos, *caches[0], slots, interleaved=inter)
    inside = qk.qknorm_rope_append(*now, gm, gm, D, cs, pos, *caches[1], slots, interleaved=inter, q_out=now[0])
    apart4 = qk.qknorm_rope_append_kv4(*kept, gm, gm, cs, pos, four[0], slots, interleaved=inter)
    inside4 = qk.qknorm_rope_append_kv4(*now4, gm, gm, cs, pos, four[1], slots, interleaved=inter, q_out=now4[0])
    assert inside is now[0] and inside4 is now4[0]
    for a, b in ((apart, inside), (apart4, inside4), *zip(caches[0], caches[1]), *zip(four[0], four[1]), *zip(now[1:], kept[1:]),
                 *zip(now4[1:], kept[1:])):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# --------------------------------------------------------------------------- captured, repeated indices

@pytest.mark.gpu
def test_two_captured_attentions_on_one_workspace():
    """Cut into shares, two graphs replayed in turn on one buffer, with other
    lengths and queries each time, against eager calls."""
    g = torch.Generator().manual_seed(19)
    hq, hk, D, ps, L, B = 8, 2, 128, 64, 9000, 3
    pages = -(-L // ps)
    cache = rc.random_cache(pages, ps, hk, D, g)
    bt = torch.stack([torch.randperm(pages, generator=g) for _ in range(B)]).int().to(DEV)
    held = torch.empty(qk.kv4_attention_workspace_bytes(B, B, hq, hk, D, 1, L), dtype=torch.uint8, device=DEV)
    assert held.numel() > 0
    q, lens = [torch.zeros((B, hq * D), dtype=BF16, device=DEV) for _ in range(2)], [torch.ones(B, dtype=torch.int32, device=DEV) for _ in range(2)]

    def call(i, **kw):
        return qk.qknorm_kv4_attention(q[i], cache, bt, lens[i], max_seq_len=L, return_lse=True, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(0, workspace=held)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for i in range(2):
        with torch.cuda.graph(graphs[i]):
            outs.append(call(i, workspace=held))
    for _ in range(3):
        for i in range(2):
            q[i].copy_(torch.randn((B, hq * D), generator=g))
            lens[i].copy_(torch.randint(0, L + 1, (B,), generator=g))
        graphs[0].replay()
        graphs[1].replay()
        for i in range(2):
            for a, b in zip(outs[i], call(i)):
                assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [100, 3000])
def test_attention_to_the_same_page_over_and_over(L):
    g = torch.Generator().manual_seed(L)
    cache = rc.random_cache(3, 32, 2, 128, g)
    bt = torch.randint(0, 3, (2, -(-L // 32)), generator=g).int()
    q = torch.randn((2, 4 * 128), generator=g).to(BF16).to(DEV)
    rc.check_attention(q, cache, bt, torch.tensor([L, L - 31], dtype=torch.int32), None, 1, L)


@pytest.mark.gpu
def test_tokens_on_the_same_slot_disturb_no_other_cell():
    g = torch.Generator().manual_seed(20)
    T, hk, D, ps = 64, 2, 128, 16
    x = torch.randn((T, 2 * hk * D), generator=g).to(BF16).to(DEV)
    k, v, gm, cs = x[:, :hk * D], x[:, hk * D:], rc.gamma_of(D, BF16, g).to(DEV), rc.table(T, D).to(DEV)
    pos, once = torch.arange(T, device=DEV), torch.randperm(T + ps, generator=g)[:T]
    twice = once.clone()
    twice[::8] = int(once[0])
    held = [qk.kv4_cache(T // ps + 1, ps, hk, D, DEV) for _ in range(2)]
    for cache, slots in zip(held, (once, twice)):
        qk.qknorm_rope_append_kv4(None, k, v, None, gm, cs, pos, cache, slots.to(DEV))
    alone = torch.ones(T, dtype=torch.bool)
    alone[::8] = False
    at = once[alone]
    for a, b in zip(*held):
        assert torch.equal(a.cpu()[at // ps, :, at % ps], b.cpu()[at // ps, :, at % ps])
    other = torch.tensor([s for s in range(T + ps) if s not in twice.tolist()])
    assert not held[1][1].cpu()[other // ps, :, other % ps].any()
