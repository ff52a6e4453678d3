"""The serving and training operators around headwise QK-Norm that are measured:
the norm with the position rotation in the same pass and its gradient, the
append to a paged cache (element types and 4 bits), and attention over the
4-bit cache.

A case's ``op`` names the operator.  Where ``own`` is false ``run`` computes it
with elementary torch operations; where it is true it calls this framework.

4-bit cache: a head's vector is split into groups of 64; a group has one fp16
scale s = fp16(max |y| / 7) and codes clamp(rint(y / s), -7, 7), stored as
code + 8 in a nibble, element 2i in the low and 2i + 1 in the high nibble of
byte i.  Pages are [page][kv head][token][...].
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
_ESZ = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
_EPS = 1e-6
_GROUP = 64
_DEV = "cuda"


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the headwise batch of the benchmark (32 + 8 heads of 128, 4096 tokens) on packed rows, rotated
        {"name": "rope prompt bf16", "op": "rope", "T": 4096, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "packed": True},
        # one decoded token of the decode width (40 heads of 128): latency
        {"name": "rope token bf16", "op": "rope", "T": 1, "hq": 40, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "packed": True},
        # E4M3 activations, an odd number of tokens, partial rotation of adjacent pairs
        {"name": "rope ragged e4m3", "op": "rope", "T": 1537, "hq": 16, "hk": 16, "d": 128, "rot": 64,
         "inter": True, "dtype": "e4m3", "packed": False},
        # a training step's gradient at the largest token count of the shard-decomposed case
        {"name": "rope grad bf16", "op": "rope_grad", "T": 16384, "hq": 40, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "packed": True},
        # a small fp32 model: heads of 96, rotation of 64 of them, odd token count
        {"name": "rope grad odd f32", "op": "rope_grad", "T": 777, "hq": 12, "hk": 4, "d": 96, "rot": 64,
         "inter": True, "dtype": "f32", "packed": False},
        # a decode step of 256 sequences into a 16-token paged cache
        {"name": "append tokens bf16", "op": "append", "T": 256, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "page": 16, "norm": True, "heads_first": False, "decode": True},
        # a prompt whose rows the projection has normalised already: rotation only, heads-first pages
        {"name": "append prompt f16", "op": "append", "T": 5001, "hq": 32, "hk": 8, "d": 64, "rot": 64,
         "inter": False, "dtype": "f16", "page": 64, "norm": False, "heads_first": True, "decode": False},
        # a decode step into the 4-bit cache, read back
        {"name": "append 4-bit tokens", "op": "append4", "T": 64, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "page": 32, "norm": True, "decode": True},
        # a prompt into the 4-bit cache, read back
        {"name": "append 4-bit prompt", "op": "append4", "T": 4096, "hq": 32, "hk": 8, "d": 128, "rot": 128,
         "inter": False, "dtype": "bf16", "page": 16, "norm": True, "decode": False},
        # one decoded token for each of 64 sequences of up to 4096 tokens
        {"name": "attend batch bf16", "op": "attend4", "B": 64, "q_len": 1, "max_len": 4096, "hq": 32, "hk": 8,
         "d": 128, "dtype": "bf16", "page": 16, "window": 0},
        # one sequence with a long cache: the split over its length carries it
        {"name": "attend long bf16", "op": "attend4", "B": 1, "q_len": 1, "max_len": 131072, "hq": 40, "hk": 8,
         "d": 128, "dtype": "bf16", "page": 64, "window": 0},
        # chunks of prompts over what is cached, in a window
        {"name": "attend chunk f16", "op": "attend4", "B": 4, "q_len": 509, "max_len": 4096, "hq": 32, "hk": 8,
         "d": 128, "dtype": "f16", "page": 32, "window": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_grad", "append", "append4", "attend4"])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "attend4":
        d = rng.choice([64, 128, 256])
        B = _log(rng, 1, 48)
        q_len = rng.choice([1, 1, 1, rng.randint(2, 9), rng.randint(10, 300)])
        if q_len > 9:
            B = min(B, max(1, 16384 // (hq * d)))
        most = min(65536 if q_len <= 9 else 4096, 131072 * 128 // (B * d))
        max_len = max(q_len, _log(rng, 16, most))
        return {"op": op, "B": B, "q_len": q_len, "max_len": max_len, "hq": hq, "hk": hk, "d": d,
                "dtype": rng.choice(["bf16", "f16"]), "page": rng.choice([16, 32, 64, 128]),
                "window": rng.choice([0, 0, max(1, max_len // 3)])}
    d = rng.choice([64, 128, 256]) if op == "append4" else rng.choice([32, 64, 80, 96, 128, 192, 256])
    rot = rng.choice([d, d, d // 2])
    rot -= rot % 2
    case = {"op": op, "T": 0, "hq": hq, "hk": hk, "d": d, "rot": rot, "inter": rng.random() < 0.4}
    case["dtype"] = rng.choice({"rope": ["bf16", "f16", "f32", "e4m3"], "rope_grad": ["bf16", "f16", "f32"],
                                "append": ["bf16", "f16", "f32"], "append4": ["bf16", "f16"]}[op])
    case["T"] = _log(rng, 1, min(8192, 128_000_000 // ((hq + 2 * hk) * d * _ESZ[case["dtype"]])))
    if op in ("rope", "rope_grad"):
        case["packed"] = rng.random() < 0.5
        return case
    case["page"] = rng.choice([16, 32, 64, 128])
    case["norm"] = rng.random() < 0.7
    case["decode"] = case["T"] <= 512 and rng.random() < 0.5
    if op == "append":
        case["heads_first"] = rng.random() < 0.5
    return case


def _lens(case):
    """Cached tokens of each sequence: spread over a quarter to all of max_len,
    the first the longest, never below the query tokens."""
    top = case["max_len"]
    return [max(case["q_len"], top - int(0.75 * top * ((0.6180339887 * b) % 1.0))) for b in range(case["B"])]


# --------------------------------------------------------------------------- inputs

def _table(P, rot):
    """[P, rot] fp32: the cosines, then the sines, of pos / 10000^(2i / rot)."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=_DEV)
    a = torch.arange(P, dtype=torch.float64, device=_DEV)[:, None] * torch.pow(10000.0, -2.0 * i / rot)[None, :]
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()


def _rows(case, seed, names):
    """The activations of `names` (with their widths), each row scaled by its
    token's exp(U(ln 0.1, ln 10)), packed side by side or in buffers of their own."""
    g = torch.Generator(device=_DEV).manual_seed(seed)
    T, dt = case["T"], _DT[case["dtype"]]
    s = torch.exp(math.log(0.1) + torch.rand((T, 1), generator=g, device=_DEV) * math.log(100.0))
    width = sum(w for _, w in names)
    x = (torch.randn((T, width), generator=g, device=_DEV) * s).to(dt)
    out, c = {}, 0
    for name, w in names:
        out[name] = x[:, c:c + w] if case.get("packed", True) else x[:, c:c + w].contiguous()
        c += w
    return out, g


def _gamma(case, g):
    gdt = torch.bfloat16 if case["dtype"] == "e4m3" else _DT[case["dtype"]]
    return (1.0 + 0.1 * torch.randn((case["d"],), generator=g, device=_DEV)).to(gdt)


def prepare(case, seed):
    return {"rope": _prepare_rope, "rope_grad": _prepare_rope, "append": _prepare_append, "append4": _prepare_append,
            "attend4": _prepare_attend}[case["op"]](case, seed)


def _prepare_rope(case, seed):
    T, d = case["T"], case["d"]
    wide = [("q", case["hq"] * d), ("k", case["hk"] * d)]
    st, g = _rows(case, seed, wide)
    st["gamma_q"], st["gamma_k"] = _gamma(case, g), _gamma(case, g)
    start = int(torch.randint(0, 2048, (1,), generator=g, device=_DEV))
    st["positions"] = torch.arange(start, start + T, device=_DEV)
    st["table"] = _table(start + T + 5, case["rot"])
    if case["op"] == "rope_grad":
        for name, w in wide:
            st["d" + name] = torch.randn((T, w), generator=g, device=_DEV).to(_DT[case["dtype"]])
    st["case"] = case
    return st


def _prepare_append(case, seed):
    T, d, hk, ps = case["T"], case["d"], case["hk"], case["page"]
    st, g = _rows(case, seed, [("q", case["hq"] * d), ("k", hk * d), ("v", hk * d)])
    st["gamma_q"], st["gamma_k"] = (_gamma(case, g), _gamma(case, g)) if case["norm"] else (None, None)
    if case["decode"]:  # each sequence's next token, on a page of its own
        pages = T + 7
        st["positions"] = torch.randint(0, 4096, (T,), generator=g, device=_DEV)
        page = torch.randperm(pages, generator=g, device=_DEV)[:T]
        st["slots"] = page * ps + st["positions"] % ps
        P = 4096
    else:  # one prompt on scattered pages
        n = -(-T // ps)
        pages = n + 7
        t = torch.arange(T, device=_DEV)
        st["positions"] = t
        st["slots"] = torch.randperm(pages, generator=g, device=_DEV)[t // ps] * ps + t % ps
        P = T
    st["table"] = _table(P, case["rot"])
    if case["op"] == "append":
        shape = (pages, hk, ps, d) if case["heads_first"] else (pages, ps, hk, d)
        for name in ("k_cache", "v_cache"):
            c = torch.randn(shape, generator=g, device=_DEV).to(_DT[case["dtype"]])
            st[name] = c.transpose(1, 2) if case["heads_first"] else c  # indexed [page, token, head, dim]
    else:
        st["cache"] = _empty_cache(pages, ps, hk, d)
    st["case"] = case
    return st


def _empty_cache(pages, ps, hk, d):
    """Codes and scales of the keys, then of the values: all zeros."""
    return tuple(t for _ in range(2) for t in (
        torch.full((pages, hk, ps, d // 2), 0x88, dtype=torch.uint8, device=_DEV),
        torch.zeros((pages, hk, ps, d // _GROUP), dtype=torch.float16, device=_DEV)))


def _prepare_attend(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)
    B, d, hk, ps = case["B"], case["d"], case["hk"], case["page"]
    lens = _lens(case)
    per = [-(-n // ps) for n in lens]
    pages, most = sum(per) + 3, max(per)
    cache = _empty_cache(pages, ps, hk, d)
    # keys of unit mean square (normalised), values of spread scales, quantised as the append does
    for codes, scales, spread in ((*cache[:2], False), (*cache[2:], True)):
        step = max(1, (1 << 26) // (hk * ps * d))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            y = torch.randn((n, hk, ps, d // _GROUP, _GROUP), generator=g, device=_DEV)
            if spread:
                y *= torch.exp(math.log(0.1) + torch.rand((n, hk, ps, 1, 1), generator=g, device=_DEV) * math.log(100.0))
            s = (y.abs().amax(-1) / 7).to(torch.float16)
            c = (torch.round(y / s.float()[..., None]).clamp(-7, 7) + 8).to(torch.uint8).view(n, hk, ps, d // 2, 2)
            scales[p:p + n] = s
            codes[p:p + n] = c[..., 0] | (c[..., 1] << 4)
    order = torch.randperm(pages, generator=g, device=_DEV).to(torch.int32)
    table = torch.full((B, most), -1, dtype=torch.int32, device=_DEV)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    q = torch.randn((B * case["q_len"], case["hq"] * d), generator=g, device=_DEV).to(_DT[case["dtype"]])
    return {"case": case, "q": q, "cache": cache, "block_table": table, "max_len": max(lens),
            "seq_lens": torch.tensor(lens, dtype=torch.int32, device=_DEV),
            "q_start": torch.arange(B + 1, dtype=torch.int32, device=_DEV) * case["q_len"]}


# --------------------------------------------------------------------------- one pass

def run(state):
    return {"rope": _run_rope, "rope_grad": _run_rope_grad, "append": _run_append, "append4": _run_append4,
            "attend4": _run_attend}[state["case"]["op"]](state)


def _plain_rotate(n, case, table, positions):
    """R(pos) applied to n [T, heads, d] (the type of n)."""
    rot = case["rot"]
    cs = table[positions].to(n.dtype)[:, None, :]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if case["inter"]:
        a, b = n[..., 0:rot:2], n[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    else:
        a, b = n[..., :rot // 2], n[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    return torch.cat([turned, n[..., rot:]], dim=-1)


def _plain_norm_rope(x, gamma, case, table, positions, wide=torch.float32):
    T, d = x.shape[0], case["d"]
    n = x.to(wide).reshape(T, -1, d)
    if gamma is not None:
        n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + _EPS) * gamma.to(wide)
    return _plain_rotate(n, case, table, positions)


def _round(y, dt):
    """`y` rounded once to `dt` (E4M3 saturates at its largest value)."""
    return y.clamp(-448.0, 448.0).to(dt) if dt == torch.float8_e4m3fn else y.to(dt)


def _run_rope(st):
    case = st["case"]
    if own:
        import attention_normalization_b200 as qk
        q, k = qk.qknorm_headwise_rope(st["q"], st["k"], st["gamma_q"], st["gamma_k"], case["d"], st["table"],
                                       st["positions"], _EPS, interleaved=case["inter"])
        return {"q": q, "k": k}
    return {x: _round(_plain_norm_rope(st[x], st["gamma_" + x], case, st["table"], st["positions"]).flatten(1),
                      st[x].dtype) for x in ("q", "k")}


def _run_rope_grad(st):
    case = st["case"]
    if own:
        import attention_normalization_b200 as qk
        dq, dk, gq, gk = qk.qknorm_headwise_rope_backward(
            st["dq"], st["dk"], st["q"], st["k"], st["gamma_q"], st["gamma_k"], case["d"], st["table"],
            st["positions"], _EPS, interleaved=case["inter"])
        return {"dq": dq, "dk": dk, "dgamma_q": gq, "dgamma_k": gk}
    out = {}
    back = st["table"].clone()
    back[:, case["rot"] // 2:] *= -1  # the transposed rotation
    for x in ("q", "k"):
        T = case["T"]
        v, gamma = st[x].float().reshape(T, -1, case["d"]), st["gamma_" + x].float()
        r = torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS)
        z = v * r
        dn = _plain_rotate(st["d" + x].float().reshape(T, -1, case["d"]), case, back, st["positions"])
        out["dgamma_" + x] = (dn * z).sum(dim=(0, 1), dtype=torch.float64).float()
        dz = dn * gamma
        out["d" + x] = (r * (dz - z * (dz * z).mean(-1, keepdim=True))).flatten(1).to(st[x].dtype)
    return out


def _run_append(st):
    case = st["case"]
    if own:
        import attention_normalization_b200 as qk
        q = qk.qknorm_rope_append(st["q"], st["k"], st["v"], st["gamma_q"], st["gamma_k"], case["d"], st["table"],
                                  st["positions"], st["k_cache"], st["v_cache"], st["slots"], _EPS,
                                  interleaved=case["inter"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    dt = st["q"].dtype
    q = _plain_norm_rope(st["q"], st["gamma_q"], case, st["table"], st["positions"]).flatten(1).to(dt)
    k = _plain_norm_rope(st["k"], st["gamma_k"], case, st["table"], st["positions"]).to(dt)
    page, off = st["slots"] // case["page"], st["slots"] % case["page"]
    st["k_cache"][page, off] = k
    st["v_cache"][page, off] = st["v"].reshape(k.shape)
    return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_half(a):
    """The fp64 values a >= 0 rounded once to fp16 (a cast through fp32 would
    round twice), saturated."""
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-14) - 10)
    return (torch.round(a / step) * step).clamp(max=65504.0).to(torch.float16)


def _plain_quantise(y, d):
    """fp64 [T, heads, d] -> bytes [T, heads, d / 2], scales [T, heads, d / 64]."""
    y = y.unflatten(-1, (d // _GROUP, _GROUP))
    s = _plain_half(y.abs().amax(-1) / 7)
    w = s.double()[..., None]
    c = torch.where(w > 0, torch.round(y / w).clamp(-7, 7), torch.zeros_like(y)).flatten(-2)
    c = (c + 8).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _plain_values(codes, scales):
    """Bytes [..., d / 2] and scales [..., d / 64] -> fp32 [..., d]."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float() - 8
    return (c.unflatten(-1, (-1, _GROUP)) * scales.float()[..., None]).flatten(-2)


def _run_append4(st):
    case, cache = st["case"], st["cache"]
    if own:
        import attention_normalization_b200 as qk
        q = qk.qknorm_rope_append_kv4(st["q"], st["k"], st["v"], st["gamma_q"], st["gamma_k"], st["table"],
                                      st["positions"], cache, st["slots"], _EPS, interleaved=case["inter"])
        k, v = qk.qknorm_kv4_read(cache, st["slots"], q.dtype)
        return {"q": q, "k": k, "v": v, "k_scales": cache[1], "v_scales": cache[3]}
    d, dt = case["d"], st["q"].dtype
    q = _plain_norm_rope(st["q"], st["gamma_q"], case, st["table"], st["positions"]).flatten(1).to(dt)
    # in 64 bits: a key next to the border of two codes
    k = _plain_norm_rope(st["k"], st["gamma_k"], case, st["table"], st["positions"], torch.float64)
    v = st["v"].double().reshape(k.shape)
    page, off = st["slots"] // case["page"], st["slots"] % case["page"]
    out = {"q": q}
    for name, y, codes, scales in (("k", k, *cache[:2]), ("v", v, *cache[2:])):
        c, s = _plain_quantise(y, d)
        codes[page, :, off], scales[page, :, off] = c, s
        out[name] = _plain_values(codes[page, :, off], scales[page, :, off]).flatten(1).to(dt)
        out[name + "_scales"] = scales
    return out


def _run_attend(st):
    case, cache = st["case"], st["cache"]
    if own:
        import attention_normalization_b200 as qk
        out, lse = qk.qknorm_kv4_attention(st["q"], cache, st["block_table"], st["seq_lens"], max_seq_len=st["max_len"],
                                           q_start=st["q_start"], max_q_len=case["q_len"], window=case["window"],
                                           return_lse=True)
        return {"out": out, "lse": lse}
    B, n, hq, hk, d = case["B"], case["q_len"], case["hq"], case["hk"], case["d"]
    page = st["block_table"].long().clamp(min=0)  # [B, pages]; what lies past a sequence's length is masked

    def cached(codes, scales):  # [B, hk, pages * page size, d]
        return _plain_values(codes[page].transpose(1, 2).flatten(2, 3), scales[page].transpose(1, 2).flatten(2, 3))

    q = st["q"].float().view(B, n, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(B, hk, -1, d)  # row = head, token
    s = (q @ cached(*cache[:2]).transpose(-1, -2) / math.sqrt(d)).view(B, hk, hq // hk, n, -1)
    token = torch.arange(s.shape[-1], device=_DEV)
    at = (st["seq_lens"][:, None] - n + torch.arange(n, device=_DEV))[:, None, None, :, None]  # each query's position
    hidden = token > at
    if case["window"]:
        hidden = hidden | (token <= at - case["window"])
    s = s.masked_fill(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    z = p.sum(-1, keepdim=True)
    v = cached(*cache[2:])
    o = ((p / z).reshape(B, hk, -1, v.shape[2]) @ v).view(B, hk, hq // hk, n, d)
    lse = (m + torch.log(z)).squeeze(-1)
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(B * n, hq * d).to(st["q"].dtype),
            "lse": lse.permute(0, 3, 1, 2).reshape(B * n, hq)}


# --------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    esz, d = _ESZ.get(case["dtype"], 2), case["d"]
    if case["op"] == "attend4":
        lens, n, w = _lens(case), case["q_len"], case["window"]
        seen = [min(L, w + n - 1) if w else L for L in lens]
        pairs = sum(min(L - n + i + 1, w) if w else L - n + i + 1 for L in lens for i in range(n))
        rows = case["B"] * n * case["hq"]
        return {"bytes": sum(seen) * case["hk"] * 2 * (d // 2 + 2 * (d // _GROUP)) + 2 * rows * d * esz + 4 * rows,
                "flops": 4 * pairs * case["hq"] * d}
    T = case["T"]
    q, k = T * case["hq"] * d * esz, T * case["hk"] * d * esz
    table = T * (case["rot"] * 4 + 8)
    if case["op"] == "rope":
        return {"bytes": 2 * (q + k) + table, "flops": 8 * (q + k) // esz}
    if case["op"] == "rope_grad":
        return {"bytes": 3 * (q + k) + table + 8 * d, "flops": 20 * (q + k) // esz}
    if case["op"] == "append":
        return {"bytes": 2 * (q + 2 * k) + table + 8 * T, "flops": 8 * (q + k) // esz}
    cached = T * case["hk"] * (d // 2 + 2 * (d // _GROUP))
    # q in and out, k and v in, the cache written, then read and the rows written
    return {"bytes": 2 * q + 2 * k + 2 * cached + (2 * cached + 2 * k) + table + 8 * T, "flops": 12 * (q + 2 * k) // esz}


# --------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend4":
        return _exact_attend(case, st)
    T, d, rot = case["T"], case["d"], case["rot"]
    cs = st["table"].double()[st["positions"]]
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]  # cos + i sin

    def rotate(n, w):
        n = n.clone()
        if case["inter"]:
            first, second = slice(0, rot, 2), slice(1, rot, 2)
        else:
            first, second = slice(0, rot // 2), slice(rot // 2, rot)
        c = torch.complex(n[..., first].contiguous(), n[..., second].contiguous()) * w
        n[..., first], n[..., second] = c.real, c.imag
        return n

    def heads(x):
        return x.double().reshape(T, -1, d)

    def forward(x, gamma):
        n = heads(x)
        if gamma is not None:
            n = gamma.double() * n / ((n * n).sum(-1, keepdim=True) / d + _EPS).sqrt()
        return rotate(n, turn)

    if case["op"] == "rope_grad":
        out = {}
        for x in ("q", "k"):
            v, gamma = heads(st[x]), st["gamma_" + x].double()
            rms = ((v * v).sum(-1, keepdim=True) / d + _EPS).sqrt()
            u = rotate(heads(st["d" + x]), turn.conj())
            out["dgamma_" + x] = (u * v / rms).sum((0, 1))
            u = u * gamma
            out["d" + x] = (u / rms - v * (u * v).sum(-1, keepdim=True) / (d * rms ** 3)).reshape(T, -1)
        return out
    q = forward(st["q"], st["gamma_q"]).reshape(T, -1)
    if case["dtype"] == "e4m3":
        q = q.clamp(-448, 448)
    if case["op"] == "rope":
        k = forward(st["k"], st["gamma_k"]).reshape(T, -1)
        return {"q": q, "k": k.clamp(-448, 448) if case["dtype"] == "e4m3" else k}
    k, v = forward(st["k"], st["gamma_k"]), heads(st["v"])
    page, off = st["slots"] // case["page"], st["slots"] % case["page"]
    if case["op"] == "append":
        caches = []
        for c, y in ((st["k_cache"], k), (st["v_cache"], v)):
            c = c.double()
            c[page, off] = y
            caches.append(c)
        return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}
    import numpy as np
    out = {"q": q}
    for name, y, held in (("k", k, st["cache"][1]), ("v", v, st["cache"][3])):
        y = y.reshape(T, case["hk"], -1, _GROUP).cpu().numpy()
        s = np.minimum(np.abs(y).max(-1) / 7, 65504.0).astype(np.float16).astype(np.float64)  # numpy rounds once
        c = np.clip(np.rint(np.divide(y, s[..., None], out=np.zeros_like(y), where=s[..., None] > 0)), -7, 7)
        out[name] = torch.from_numpy((c * s[..., None]).reshape(T, -1))
        scales = held.double().cpu()
        scales[page.cpu(), :, off.cpu()] = torch.from_numpy(s)
        out[name + "_scales"] = scales
    return out


def _exact_attend(case, st):
    """Sequence by sequence, over the tokens that it has."""
    n, hq, hk, d, ps = case["q_len"], case["hq"], case["hk"], case["d"], case["page"]
    cache, out, lse = st["cache"], [], []
    for b, L in enumerate(_lens(case)):
        page = st["block_table"][b, :-(-L // ps)].long()

        def tokens(codes, scales):  # [hk, L, d]
            c = codes[page].permute(1, 0, 2, 3).reshape(hk, -1, d // 2)[:, :L].to(torch.int64)
            v = torch.empty((hk, L, d), dtype=torch.float64, device=c.device)
            v[..., 0::2], v[..., 1::2] = (c % 16 - 8).double(), (c // 16 - 8).double()
            s = scales[page].permute(1, 0, 2, 3).reshape(hk, -1, d // _GROUP)[:, :L].double()
            return v * s.repeat_interleave(_GROUP, dim=-1)

        K, V = tokens(*cache[:2]), tokens(*cache[2:])
        q = st["q"][b * n:(b + 1) * n].double().reshape(n, hk, hq // hk, d)
        s = torch.einsum("nhgd,hld->hgnl", q, K) * d ** -0.5
        at = torch.arange(L - n, L, device=s.device)[:, None]
        t = torch.arange(L, device=s.device)[None, :]
        keep = t <= at
        if case["window"]:
            keep &= t > at - case["window"]
        s = torch.where(keep, s, torch.full_like(s, -math.inf))
        lse.append(torch.logsumexp(s, -1).permute(2, 0, 1).reshape(n, hq))
        out.append(torch.einsum("hgnl,hld->nhgd", torch.softmax(s, -1), V).reshape(n, hq * d))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
