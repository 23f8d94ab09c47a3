"""Measured cases of the operators around the routed experts: routing by
scores, RMSNorm with the residual's addition, microscaled quantisation, and
the product of 4-bit microscaled weights with 8-bit microscaled tokens.

``run`` computes a case in plain torch operations, or (``own``) through the
library's entry points.  Both read the same buffers; packed weights are in the
layout that ``include/gale.h`` documents.
"""
from __future__ import annotations

import math

import torch

own = False

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
DTYPES = {"f32": F32, "bf16": BF16, "f16": F16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the router of one decoded token: 256 experts, six picked, as the layer benchmark routes
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 256, "k": 6, "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "group_top": 2, "renorm": True, "scale": 2.5, "masked": 0, "dtype": "f32"},
        # the router of a prompt of 4096 tokens
        {"name": "route_prompt", "op": "route", "tokens": 4096, "experts": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "group_top": 2, "renorm": True, "scale": 2.5, "masked": 0,
         "dtype": "f32"},
        # the router of many packed prompts, plain softmax scores in 16 bits (equal logits are frequent)
        {"name": "route_many", "op": "route", "tokens": 65536, "experts": 256, "k": 6, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "group_top": 1, "renorm": True, "scale": 1.0, "masked": 0,
         "dtype": "bf16"},
        # the norm before a layer, one decoded token
        {"name": "norm_token", "op": "norm", "tokens": 1, "cols": 4096, "dtype": "bf16", "residual": True,
         "out": "bf16"},
        # the same for a prompt of 4096 tokens
        {"name": "norm_prompt", "op": "norm", "tokens": 4096, "cols": 4096, "dtype": "bf16", "residual": True,
         "out": "bf16"},
        # odd sizes in 32 bits, no residual (a final norm)
        {"name": "norm_odd", "op": "norm", "tokens": 10007, "cols": 5001, "dtype": "f32", "residual": False,
         "out": "f32"},
        # a load-time quantisation of a large non-expert matrix, and the values it stands for
        {"name": "quantize_large", "op": "quantize", "rows": 65536, "cols": 4096, "dtype": "f32"},
        # a small one of odd sizes
        {"name": "quantize_odd", "op": "quantize", "rows": 2050, "cols": 1001, "dtype": "bf16"},
        # the output head for one token: tokens to 8 bits, then the product
        {"name": "product_token", "op": "product", "tokens": 1, "rows": 65536, "cols": 4096, "norm": False,
         "dtype": "bf16", "out": "f32"},
        # norm and a shared projection for a decoded batch of eight
        {"name": "product_batch", "op": "product", "tokens": 8, "rows": 2048, "cols": 4096, "norm": True,
         "dtype": "bf16", "out": "bf16"},
        # norm and projection of a ragged chunk, sizes that fill no tile
        {"name": "product_ragged", "op": "product", "tokens": 1000, "rows": 5000, "cols": 4000, "norm": True,
         "dtype": "bf16", "out": "bf16"},
        # a prompt of 4096 tokens through a wide projection
        {"name": "product_prompt", "op": "product", "tokens": 4096, "rows": 16384, "cols": 4096, "norm": False,
         "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "norm", "norm", "quantize", "product", "product", "product"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log(rng, 8, 512 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        experts = groups * size
        masked = rng.choice([0, 0, 0, experts // 8])
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "k": rng.randint(1, min(16, keep * size)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.6, "groups": groups,
                "keep": keep, "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 1.5, 2.5]), "masked": masked, "dtype": rng.choice(["f32", "bf16", "f16"])}
    if op == "norm":
        cols = _log(rng, 64, 8192)
        tokens = min(_log(rng, 1, 16384), (1 << 26) // cols)
        dtype = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "tokens": tokens, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.7,
                "out": rng.choice([dtype, "bf16", "f32"])}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 16, 16384), "cols": _log(rng, 64, 8192),
                "dtype": rng.choice(["f32", "bf16", "f16"])}
    rows, cols = _log(rng, 64, 16384), _log(rng, 64, 8192)
    tokens = max(1, min(_log(rng, 1, 8192), (1 << 38) // (rows * cols)))
    return {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "norm": rng.random() < 0.5,
            "dtype": rng.choice(["bf16", "f16", "f32"]), "out": rng.choice(["f32", "bf16", "f16"])}


def work(case):
    op = case["op"]
    if op == "route":
        n = case["tokens"] * case["experts"]
        return {"bytes": n * SIZE[case["dtype"]] + 8 * case["tokens"] * case["k"] + 4 * case["experts"],
                "flops": 8 * n}
    if op == "norm":
        n = case["tokens"] * case["cols"]
        b = SIZE[case["dtype"]] * (3 if case["residual"] else 1) + SIZE[case["out"]]
        return {"bytes": n * b + 4 * case["cols"], "flops": 5 * n}
    if op == "quantize":  # the matrix in; the packed codes and scales out and in; the values out
        n = case["rows"] * case["cols"]
        return {"bytes": int(n * (SIZE[case["dtype"]] + 2 * (0.5 + 1 / 32) + 2)), "flops": 4 * n}
    t, r, c = case["tokens"], case["rows"], case["cols"]
    x = t * c * SIZE[case["dtype"]] * (3 if case["norm"] else 1)
    return {"bytes": int(r * c * (0.5 + 1 / 32) + x + t * r * SIZE[case["out"]]), "flops": 2 * t * r * c}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _up(n, m):
    return (n + m - 1) // m * m


def _sizes4(rows, cols):
    """Bytes of the packed weights: code section, start of the scales, total."""
    rp, cp = _up(rows, 128), _up(cols, 128)
    codes = rp * cp // 2
    return rp, cp, codes, _up(_up(codes, 256) + rp * cp // 32, 256)


def _scale_exponent(amax, top_mantissa, top_exponent):
    """The smallest k with amax <= 2^k * top_mantissa * 2^top_exponent, in [-127, 127]; -127 for zero."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    k = e - 1 - top_exponent + (m * 2 > top_mantissa).to(e.dtype)
    return torch.where(amax > 0, k.clamp(-127, 127), torch.full_like(k, -127))


def _power(k):
    """2^k in 32 bits, k in [-126, 127], by its bits: exact on every device."""
    return ((k.to(torch.int32) + 127) << 23).view(F32)


def _times_power(x, k):
    """x * 2^k (k an int tensor); in two factors, since 2^k alone may leave the range of 32 bits."""
    half = torch.div(k, 2, rounding_mode="floor")
    return x * _power(half) * _power(k - half)


def _pad_cols(x, to):
    return torch.nn.functional.pad(x, (0, to - x.shape[-1])) if x.shape[-1] < to else x


def _codes4(v):
    """e2m1 codes of values in [-6, 6], round to nearest even: steps of 0.5 to 2, 1 to 4, 2 to 6."""
    a = v.abs()
    c = torch.where(a <= 2, torch.round(a * 2), torch.where(a <= 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    return c.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)


def _pack4(w):
    """A [rows, cols] matrix as packed bytes of the library's MXFP4 layout."""
    rows, cols = w.shape
    rp, cp, codes, total = _sizes4(rows, cols)
    buf = torch.zeros(total, dtype=torch.uint8, device="cuda")
    q = buf[:codes].view(rp // 128, cp // 128, 128, 64)
    at = _up(codes, 256)
    s = buf[at:at + rp * cp // 32].view(rp // 128, cp // 128, 32, 4, 4)
    for r0 in range(0, rows, 8192):  # in slices, for the memory of the temporaries
        part = _pad_cols(w[r0:r0 + 8192].float(), cp)
        n = part.shape[0]
        part = torch.nn.functional.pad(part, (0, 0, 0, _up(n, 128) - n))
        b = part.view(part.shape[0], cp // 32, 32)
        k = _scale_exponent(b.abs().amax(-1), 1.5, 2)
        c = _codes4(_times_power(b, -k[..., None])).view(-1, 128, cp // 128, 128).permute(0, 2, 1, 3)
        t0 = r0 // 128
        t1 = t0 + c.shape[0]
        q[t0:t1] = c[..., 0::2] | (c[..., 1::2] << 4)
        s[t0:t1] = (k + 127).to(torch.uint8).view(-1, 4, 32, cp // 128, 4).permute(0, 3, 2, 1, 4)
    return buf


def _tokens(g, tokens, cols, dtype):
    """Hidden states: unit normal values, some features twenty times as large."""
    x = torch.randn(tokens, cols, generator=g, device="cuda")
    big = torch.rand(cols, generator=g, device="cuda") < 0.005
    return (x * torch.where(big, 20.0, 1.0)).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "route":
        t, e = case["tokens"], case["experts"]
        logits = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
        if case["masked"]:  # experts that are not available
            logits[:, torch.randperm(e, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        st["bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
        st["ids"] = torch.empty(t, case["k"], dtype=torch.int32, device="cuda")
        st["gates"] = torch.empty(t, case["k"], device="cuda")
        return st
    if op == "quantize":
        w = torch.randn(case["rows"], case["cols"], generator=g, device="cuda") * 0.02
        st["w"] = w.to(DTYPES[case["dtype"]])
        st["packed"] = torch.empty(_sizes4(case["rows"], case["cols"])[3], dtype=torch.uint8, device="cuda")
        st["values"] = torch.empty(case["rows"], case["cols"], dtype=BF16, device="cuda")
        return st
    t, c, dtype = case["tokens"], case["cols"], DTYPES[case["dtype"]]
    st["x"] = _tokens(g, t, c, dtype)
    if op == "norm" or case["norm"]:
        residual = op == "product" or case["residual"]
        st["residual"] = (3 * _tokens(g, t, c, F32)).to(dtype) if residual else None
        st["weight"] = 1 + 0.1 * torch.randn(c, generator=g, device="cuda")
        st["sum"] = torch.empty(t, c, dtype=dtype, device="cuda") if residual else None
    if op == "norm":
        st["y"] = torch.empty(t, c, dtype=DTYPES[case["out"]], device="cuda")
        return st
    r = case["rows"]
    st["packed"] = _pack4(torch.randn(r, c, generator=g, device="cuda") * 0.02)
    st["y"] = torch.empty(t, r, dtype=DTYPES[case["out"]], device="cuda")
    # 8-bit tokens: codes [tokens][cols up to 128], then scales for whole groups of 128 tokens
    cp = _up(c, 128)
    st["x8"] = torch.empty(_up(_up(t * cp, 256) + _up(t, 128) * cp // 32, 256), dtype=torch.uint8, device="cuda")
    st["ws"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_route(st):
    # 64 bits: whole numbers are decided by these scores, and near ones must not tie
    c = st["case"]
    l = st["logits"].double()
    l = torch.where(torch.isnan(l), torch.full_like(l, -math.inf), l).clamp(max=torch.finfo(F32).max)
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True).clamp(min=-torch.finfo(F32).max))
        s = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    none = torch.isneginf(l)
    sel = s if st["bias"] is None else s + st["bias"].double()
    sel = torch.where(none, torch.full_like(s, -math.inf), sel)
    key = l if st["bias"] is None else sel
    n, groups = l.shape[0], c["groups"]
    if groups > 1:
        top = sel.view(n, groups, -1).sort(-1, descending=True).values[..., :c["group_top"]]
        score = torch.where(torch.isneginf(top), torch.zeros_like(top), top).sum(-1)
        score = torch.where(torch.isneginf(top[..., 0]), torch.full_like(score, -math.inf), score)
        kept = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["keep"]]
        out = torch.ones(n, groups, dtype=torch.bool, device=l.device).scatter(1, kept, False)
        out = out.repeat_interleave(l.shape[1] // groups, 1)
    else:
        out = torch.zeros_like(none)
    # experts outside the kept groups come after every other, the masked ones of kept groups included
    order = key.sort(dim=-1, descending=True, stable=True).indices
    back = out.gather(1, order).to(torch.uint8).sort(dim=-1, stable=True).indices[:, :c["k"]]
    ids = order.gather(1, back)
    g = s.gather(1, ids)
    if c["renorm"]:
        total = g.sum(-1, keepdim=True)
        g = torch.where(total > 0, g / total.clamp(min=1e-300), torch.zeros_like(g))
    return [ids.to(torch.int32), (g * c["scale"]).float()]


def _plain_norm(x, residual, weight, eps=1e-6):
    h = x.float() if residual is None else x.float() + residual.float()
    return h, h * torch.rsqrt(h.square().mean(-1, keepdim=True) + eps) * weight


def _plain_mx8(v):
    """v rounded to e4m3 codes with a power-of-two scale per 32 columns, as the values they stand for."""
    n = v.shape[1]
    b = _pad_cols(v, _up(n, 32)).view(v.shape[0], -1, 32)
    k = _scale_exponent(b.abs().amax(-1), 1.75, 8)[..., None]
    return _times_power(_times_power(b, -k).to(torch.float8_e4m3fn).float(), k).reshape(v.shape[0], -1)[:, :n]


def _plain_unpack4(packed, rows, cols):
    rp, cp, codes, _ = _sizes4(rows, cols)
    b = packed[:codes].view(rp // 128, cp // 128, 128, 64)
    q = torch.stack([b & 15, b >> 4], -1).view(rp // 128, cp // 128, 128, 128).permute(0, 2, 1, 3).reshape(rp, cp)
    a = (q & 7).float()
    a = torch.where(a <= 4, a * 0.5, torch.where(a <= 6, a - 2, a * 2 - 8))  # 0 .5 1 1.5 2 3 4 6
    a = torch.where(q >= 8, -a, a)
    at = _up(codes, 256)
    s = packed[at:at + rp * cp // 32].view(rp // 128, cp // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp // 32)
    v = _times_power(a.view(rp, cp // 32, 32), s.int()[..., None] - 127)
    return v.view(rp, cp)[:rows, :cols]


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        return _plain_route(st)
    if op == "norm":
        h, y = _plain_norm(st["x"], st["residual"], st["weight"])
        y = y.to(st["y"].dtype)
        return [y] if st["residual"] is None else [y, h.to(st["x"].dtype)]
    if op == "quantize":
        w = st["w"].float()
        rows, cols = w.shape
        b = _pad_cols(w, _up(cols, 32)).view(rows, -1, 32)
        k = _scale_exponent(b.abs().amax(-1), 1.5, 2)[..., None]
        q = _codes4(_times_power(b, -k))
        a = (q & 7).float()
        a = torch.where(a <= 4, a * 0.5, torch.where(a <= 6, a - 2, a * 2 - 8))
        return [_times_power(torch.where(q >= 8, -a, a), k).view(rows, -1)[:, :cols].to(BF16)]
    if case["norm"]:
        h, v = _plain_norm(st["x"], st["residual"], st["weight"])
    else:
        v = st["x"].float()
    y = _plain_mx8(v) @ _plain_unpack4(st["packed"], case["rows"], case["cols"]).t()
    y = y.to(st["y"].dtype)
    return [y, h.to(st["x"].dtype)] if case["norm"] else [y]


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------

def _own(st):
    import bit_expert_gemv_b200 as G

    case, op = st["case"], st["case"]["op"]
    if op == "route":
        G.gale_route_select(st["logits"], st["ids"], st["gates"], bias=st["bias"],
                            score=G.GALE_SCORE_SIGMOID if case["score"] == "sigmoid" else G.GALE_SCORE_SOFTMAX,
                            n_groups=case["groups"], keep_groups=case["keep"], group_top=case["group_top"],
                            renorm=case["renorm"], scale=case["scale"])
        return [st["ids"], st["gates"]]
    if op == "norm":
        G.gale_rmsnorm(st["x"], y=st["y"], residual=st["residual"], weight=st["weight"], sum_out=st["sum"], eps=1e-6)
        return [st["y"]] if st["residual"] is None else [st["y"], st["sum"]]
    if op == "quantize":
        G.gale_mx4_quantize(st["w"], st["packed"])
        G.gale_mx4_unpack(st["packed"], st["values"])
        return [st["values"]]
    if case["norm"]:
        G.gale_rmsnorm(st["x"], mx8=st["x8"], residual=st["residual"], weight=st["weight"], sum_out=st["sum"],
                       eps=1e-6)
    else:
        G.gale_mx8_quantize(st["x"], st["x8"])
    G.gale_mx_gemm(st["packed"], case["rows"], case["cols"], st["x8"], st["y"], st["ws"])
    return [st["y"], st["sum"]] if case["norm"] else [st["y"]]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _power64(k):
    return ((k.long() + 1023) << 52).view(torch.float64)


def _exact_round(v, grid, top):
    """Blocks of 32 in 64 bits: the values of the nearest grid points (ties to the even place), by search in the grid."""
    n = v.shape[1]
    b = _pad_cols(v, _up(n, 32)).view(v.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.ones_like(amax)) / top)).long()
    k = torch.where(amax > top * _power64(k), k + 1, k)
    k = torch.where((amax > 0) & (amax <= top * _power64(k - 1)), k - 1, k)
    unit = _power64(k.clamp(-127, 127))
    a = b.abs() / unit
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, len(grid) - 1)
    below, above = grid[hi - 1], grid[hi]
    up = (above - a < a - below) | ((above - a == a - below) & (hi % 2 == 0))
    r = torch.where(up, above, below) * unit
    return (torch.where(b < 0, -r, r)).view(v.shape[0], -1)[:, :n]


def _grid8():
    vals = [m * 2.0 ** -9 for m in range(8)]
    vals += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)]
    return torch.tensor(vals, dtype=torch.float64, device="cuda")


def _grid4():
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")


def _exact_weights(packed, rows, cols, first, last):
    """Rows first .. last - 1 of packed MXFP4 bytes in 64 bits, by each element's address."""
    cp = _up(cols, 128)
    nt = cp // 128
    r = torch.arange(first, last, device="cuda")[:, None]
    c = torch.arange(cols, device="cuda")[None, :]
    byte = ((r // 128) * nt + c // 128) * 8192 + (r % 128) * 64 + (c % 128) // 2
    q = (packed[byte] >> ((c % 2) * 4).to(torch.uint8)) & 15
    at = _up(_up(rows, 128) * cp // 2, 256)
    b = torch.arange(_up(cols, 32) // 32, device="cuda")[None, :]
    s = packed[at + ((r // 128) * nt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]
    sign = 1.0 - 2.0 * (q >> 3).double()
    unit = _power64(s.long() - 127)
    return sign * _grid4()[(q & 7).long()] * unit.repeat_interleave(32, 1)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        import numpy as np

        l = st["logits"].double().cpu().numpy()
        none = l == -np.inf
        with np.errstate(over="ignore"):
            if case["score"] == "sigmoid":
                s = 1 / (1 + np.exp(-l))
            else:
                s = np.exp(l - l.max(1, keepdims=True))
                s /= s.sum(1, keepdims=True)
        with_bias = s if st["bias"] is None else s + st["bias"].double().cpu().numpy()
        with_bias = np.where(none, -np.inf, with_bias)
        key = l if st["bias"] is None else with_bias
        n, e = l.shape
        out = np.zeros((n, e), dtype=bool)
        if case["groups"] > 1:
            top = np.partition(with_bias.reshape(n, case["groups"], -1), -case["group_top"], -1)
            top = top[..., -case["group_top"]:]
            score = np.where(np.isneginf(top), 0, top).sum(-1)
            score[np.isneginf(top.max(-1))] = -np.inf
            place = np.argsort(np.argsort(-score, 1, kind="stable"), 1, kind="stable")
            out = np.repeat(place >= case["keep"], e // case["groups"], 1)
        ids = np.lexsort((np.broadcast_to(np.arange(e), key.shape), -key, out), axis=1)[:, :case["k"]]
        g = np.take_along_axis(s, ids, 1)
        if case["renorm"]:
            g = g / g.sum(1, keepdims=True)
        return [ids.astype(np.int32), g * case["scale"]]
    if op == "quantize":
        return [torch.cat([_exact_round(p.double(), _grid4(), 6.0) for p in st["w"].split(8192)])]
    x = st["x"].double()
    h = None
    if op == "norm" or case["norm"]:
        h = x if st["residual"] is None else x + st["residual"].double()
        x = h / (h.pow(2).sum(-1, keepdim=True) / h.shape[1] + 1e-6).sqrt() * st["weight"].double()
        if op == "norm":
            return [x] if st["residual"] is None else [x, h]
    x = torch.cat([_exact_round(p, _grid8(), 448.0) for p in x.split(1024)])
    rows, cols = case["rows"], case["cols"]
    y = [x @ _exact_weights(st["packed"], rows, cols, r0, min(rows, r0 + 4096)).t() for r0 in range(0, rows, 4096)]
    return [torch.cat(y, 1), h] if case["norm"] else [torch.cat(y, 1)]
