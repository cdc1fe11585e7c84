"""The MXFP4 and mixture-of-experts operators over the range of calls they are made for: plain forms, inputs, exact values.

MXFP4: E2M1 codes, two a byte (low nibble first), and one power-of-two scale (E8M0 byte b, 2^(b - 127)) for each block of 32
values along a row. With a block's largest magnitude m the scale is 2^(floor(log2 m) - 2) ("floor") or the smallest 2^s with
m <= 6 * 2^s ("ceil"), at least 2^-127; the codes round x / scale to the nearest E2M1 value, ties to the even code, saturating
at 6. Kinds of case ("op"):

  quantize  a tensor to MXFP4 along its rows, its columns or both, returned as the values the codes stand for
  linear    y = deq(a) . deq(w)^T from MXFP4 operands, or from raw activations that the call quantizes first
  step      the three products of a training step, y = q(x) q(w)^T, dx = q(dy) q(w), dw = q(dy)^T q(x), each operand quantized
            along the axis that its product sums over
  route     a router: the top k of x . wr^T + bias for each token, and their softmax weights
  moe       a router and its experts, y = sum_k weight_k . down_e(silu(gate_e(x)) * up_e(x)), with 4-bit expert weights
"""
import math

import torch

own = False

_MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------


def listed():
    return [
        # the wide activations of a transformer block's second MLP product, one pass over 100 MB
        {"name": "quantize_wide", "op": "quantize", "rows": 4096, "cols": 12288, "dtype": "bf16", "rule": "floor", "orient": "rows"},
        # a gradient quantized along both axes: the row count ends inside a block of 32
        {"name": "quantize_both_ragged", "op": "quantize", "rows": 1003, "cols": 2080, "dtype": "f32", "rule": "ceil", "orient": "both"},
        # one token through a resident layer: the weights' bytes and the launch count
        {"name": "linear_token", "op": "linear", "m": 1, "n": 12288, "k": 4096, "out": "bf16", "raw": True},
        # a decode batch with fp32 logits-like output, its activations quantized already
        {"name": "linear_decode_f32", "op": "linear", "m": 33, "n": 6144, "k": 4096, "out": "f32", "raw": False},
        # a prompt or an image's latent tokens through a large layer
        {"name": "linear_prefill", "op": "linear", "m": 4096, "n": 12288, "k": 4096, "out": "bf16", "raw": False},
        # sizes that fill no tile, and rows of y that start off 16 bytes
        {"name": "linear_odd", "op": "linear", "m": 777, "n": 1001, "k": 2080, "out": "bf16", "raw": True},
        # a training step of one layer, a ragged batch of tokens
        {"name": "step", "op": "step", "m": 2000, "n": 4096, "k": 2048},
        # one token's routing: latency
        {"name": "route_token", "op": "route", "t": 1, "h": 4096, "e": 64, "k": 4, "masked": 0, "renorm": True},
        # a decode batch's routing, some experts shut off
        {"name": "route_batch", "op": "route", "t": 64, "h": 4096, "e": 128, "k": 8, "masked": 5, "renorm": False},
        # one token through a mixture-of-experts layer: six experts' weights are read, the others' are not
        {"name": "moe_token", "op": "moe", "t": 1, "h": 2048, "f": 1408, "e": 64, "k": 6, "fmt": "mxfp4"},
        # a decode batch on NVFP4 experts
        {"name": "moe_batch_nvfp4", "op": "moe", "t": 16, "h": 4096, "f": 1280, "e": 32, "k": 4, "fmt": "nvfp4"},
        # the largest batch the layer takes in one call: every expert's weights are read
        {"name": "moe_batch", "op": "moe", "t": 64, "h": 2048, "f": 1024, "e": 64, "k": 8, "fmt": "mxfp4"},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "step", "route", "moe", "moe"])
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 32, 12288, 32), "dtype": rng.choice(["bf16", "f32"]),
                "rule": rng.choice(["floor", "ceil"]), "orient": rng.choice(["rows", "cols", "both"])}
    if op == "linear":
        return {"op": op, "m": _log(rng, 1, 4096), "n": _log(rng, 8, 8192), "k": _log(rng, 32, 8192, 32),
                "out": rng.choice(["bf16", "f32"]), "raw": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "m": _log(rng, 32, 2048), "n": _log(rng, 32, 4096, 32), "k": _log(rng, 32, 4096, 32)}
    t, e = _log(rng, 1, 64), rng.choice([4, 8, 16, 40, 64, 96, 128])
    k = rng.randint(1, min(8, e))
    if op == "route":
        return {"op": op, "t": t, "h": _log(rng, 64, 8192, 32), "e": e, "k": k, "masked": rng.randint(0, e), "renorm": rng.random() < 0.5}
    e = min(e, 64)
    return {"op": op, "t": t, "h": _log(rng, 256, 2048, 32), "f": _log(rng, 128, 1024, 32), "e": e, "k": min(k, e),
            "fmt": rng.choice(["mxfp4", "nvfp4"])}


def _distinct(c):
    """Experts that the tokens of a case meet, if they are drawn evenly."""
    return c["e"] * (1.0 - (1.0 - c["k"] / c["e"]) ** c["t"])


def work(c):
    if c["op"] == "quantize":
        n, src = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        sides = 2 if c["orient"] == "both" else 1
        return {"bytes": n * (src + sides * (0.5 + 1 / 32 + 2)), "flops": 0}
    if c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m * (2 if c["raw"] else 17 / 32) + n * 17 / 32) * k + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if c["op"] == "step":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": 2 * (m * k + n * k + m * n) + 2 * m * n + 2 * m * k + 4 * n * k, "flops": 6 * m * n * k}
    if c["op"] == "route":
        t, h, e, k = c["t"], c["h"], c["e"], c["k"]
        return {"bytes": 2 * h * (t + e) + 4 * e + 8 * t * k, "flops": 2 * t * h * e}
    t, h, f, e, k = c["t"], c["h"], c["f"], c["e"], c["k"]
    bits = 0.5 + (1 / 32 if c["fmt"] == "mxfp4" else 1 / 16)
    return {"bytes": _distinct(c) * 3 * h * f * bits + 2 * h * (2 * t + e) + 8 * t * k, "flops": 6 * t * k * h * f + 2 * t * h * e}


# ---- plain form of the format ----------------------------------------------------------------


def _pow2(byte):
    """2^(byte - 127) as fp32 (byte 0 is the subnormal 2^-127)."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23).view(torch.float32)


def _blocks(x, rule):
    """Scale bytes [r, c / 32] and fp32 quotients [r, c / 32, 32] of an fp32 matrix."""
    v = x.reshape(x.shape[0], -1, 32)
    m = v.abs().amax(-1).contiguous().view(torch.int32)
    e = (m >> 23) - 2
    if rule == "ceil":
        e = e + ((m & 0x7FFFFF) > 0x400000).int()
    e = e.clamp(min=0)
    return e.to(torch.uint8), v * _pow2(254 - e)[..., None]


def _nibbles(q):
    """E2M1 codes (int32) of fp32 values, to nearest, ties to the even code, saturating."""
    a = q.abs()
    n = (a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int()
    n = n + (a > 2.5).int() + (a >= 3.5).int() + (a > 5.0).int()
    return n + 8 * torch.signbit(q).int()


def _table(device):
    """The two values of each code byte, [256, 2] fp32."""
    v = torch.tensor(_MAGNITUDES + tuple(-m for m in _MAGNITUDES), device=device)
    b = torch.arange(256, device=device)
    return torch.stack([v[b % 16], v[b // 16]], -1)


def _mx_values(x, rule):
    """fp32 values that the MXFP4 form of an fp32 matrix stands for."""
    e, q = _blocks(x, rule)
    n = _nibbles(q)
    mag = torch.tensor(_MAGNITUDES, device=x.device)[n & 7]
    return (torch.where(n >= 8, -mag, mag) * _pow2(e)[..., None]).reshape(x.shape)


def _mx_pack(x, rule="floor"):
    """Codes [r, c / 2] and scale bytes [r, c / 32] of a matrix."""
    e, q = _blocks(x.float(), rule)
    n = _nibbles(q).reshape(x.shape[0], -1, 2)
    return (n[..., 0] + 16 * n[..., 1]).to(torch.uint8), e


def _decode(codes, scales, block):
    """fp32 values of packed codes [..., c / 2] with fp32 block scales [..., c / block]."""
    v = _table(codes.device)[codes.int()].flatten(-2)
    return (v.unflatten(-1, (-1, block)) * scales[..., None]).flatten(-2)


def _swizzle(s):
    """Scale bytes [rows, blocks] in the tensor-core operand layout: zero-padded atoms of 128 rows x 4 blocks."""
    r, b = s.shape
    p = torch.zeros((r + 127) // 128 * 128, (b + 3) // 4 * 4, dtype=torch.uint8, device=s.device)
    p[:r, :b] = s
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _columns(x):
    """x^T with its rows (the columns of the result) padded with zeros to a whole block of 32."""
    return torch.nn.functional.pad(x.T, (0, -x.shape[0] % 32)).contiguous()


# ---- inputs ----------------------------------------------------------------------------------


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, cols, dtype=torch.bfloat16):
    """N(0, 1) with one channel in a thousand 20 times as large, as the activations of a transformer have them."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    x[:, torch.rand(cols, device="cuda", generator=g) < 1e-3] *= 20.0
    return x.to(dtype)


def _operand(x):
    codes, scales = _mx_pack(x)
    return {"codes": codes, "lin": scales, "swz": _swizzle(scales)}


def _experts(g, e, rows, cols, fmt):
    """Stacked expert weights N(0, 0.02^2) in 4 bits: codes [e, rows, cols / 2], block scales, and for NVFP4 a global scale each."""
    w = torch.randn(e * rows, cols, device="cuda", generator=g) * 0.02
    if fmt == "mxfp4":
        codes, scales = _mx_pack(w)
        return {"codes": codes.view(e, rows, -1), "scales": scales.view(e, rows, -1), "gs": None}
    v = w.view(e, rows, -1, 16)
    gs = v.abs().amax((1, 2, 3)) / 2688.0
    sb = (v.abs().amax(-1) / (6.0 * gs[:, None, None])).to(torch.float8_e4m3fn)
    n = _nibbles(v / (sb.float() * gs[:, None, None]).clamp(min=1e-30)[..., None]).view(e, rows, -1, 2)
    return {"codes": (n[..., 0] + 16 * n[..., 1]).to(torch.uint8), "scales": sb.view(torch.uint8), "gs": gs}


def prepare(c, seed):
    g = _rng(seed)
    s = dict(c)
    if c["op"] == "quantize":
        s["x"] = _activations(g, c["rows"], c["cols"], _TYPES[c["dtype"]])
    elif c["op"] == "linear":
        x = _activations(g, c["m"], c["k"])
        s["x"] = x if c["raw"] else _operand(x)
        s["w"] = _operand(torch.randn(c["n"], c["k"], device="cuda", generator=g) * 0.02)
    elif c["op"] == "step":
        s["x"] = _activations(g, c["m"], c["k"])
        s["w"] = (torch.randn(c["n"], c["k"], device="cuda", generator=g) * 0.02).bfloat16()
        s["dy"] = (torch.randn(c["m"], c["n"], device="cuda", generator=g) * 1e-3).bfloat16()
    else:
        s["x"] = _activations(g, c["t"], c["h"])
        s["wr"] = (torch.randn(c["e"], c["h"], device="cuda", generator=g) / math.sqrt(c["h"])).bfloat16()
        s["bias"] = 0.1 * torch.randn(c["e"], device="cuda", generator=g)
        if c["op"] == "route":
            s["bias"][torch.randperm(c["e"], device="cuda", generator=g)[: c["masked"]]] = -math.inf
        else:
            s["up"] = _experts(g, c["e"], 2 * c["f"], c["h"], c["fmt"])
            s["down"] = _experts(g, c["e"], c["h"], c["f"], c["fmt"])
    return s


# ---- one pass --------------------------------------------------------------------------------


def run(s):
    return _run_own(s) if own else _run_plain(s)


def _operand_values(o):
    return _decode(o["codes"], _pow2(o["lin"]), 32)


def _route_plain(s, renorm):
    # 64 bits: which of two experts comes first must not hang on the order of a sum
    z = s["x"].double() @ s["wr"].double().T + s["bias"].double()
    top, ids = torch.sort(z, dim=-1, descending=True, stable=True)
    top, ids = top[:, : s["k"]], ids[:, : s["k"]]
    live = top > -math.inf
    p = torch.exp(top - top[:, :1].clamp(min=-1e300))
    over = p.sum(-1, keepdim=True) if renorm else torch.exp(z - top[:, :1].clamp(min=-1e300)).sum(-1, keepdim=True)
    w = torch.where(live, p / over, torch.zeros_like(p)).float()
    return torch.where(live, ids, torch.full_like(ids, -1)).int(), w


def _expert_values(o, ids=None):
    """fp32 weights of all experts, or of those of the given slots."""
    take = (lambda t: t) if ids is None else (lambda t: t[ids])
    if o["gs"] is None:
        return _decode(take(o["codes"]), _pow2(take(o["scales"])), 32)
    scales = take(o["scales"]).view(torch.float8_e4m3fn).float()
    return _decode(take(o["codes"]), scales, 16) * take(o["gs"])[:, None, None]


def _moe_plain(s):
    ids, w = _route_plain(s, True)
    x, f = s["x"].float(), s["f"]
    if ids.numel() < s["e"]:  # fewer slots than experts: the slots' own weights
        slot = ids.reshape(-1).long()
        xs = x.repeat_interleave(s["k"], 0)[:, :, None]
        a = (_expert_values(s["up"], slot) @ xs)[..., 0]
        h = torch.nn.functional.silu(a[:, :f]) * a[:, f:]
        y = (_expert_values(s["down"], slot) @ h[:, :, None])[..., 0]
        y = (y.view(s["t"], s["k"], -1) * w[..., None]).sum(1)
    else:
        a = x @ _expert_values(s["up"]).transpose(1, 2)
        h = torch.nn.functional.silu(a[..., :f]) * a[..., f:]
        share = torch.zeros(s["t"], s["e"], device=x.device).scatter_(1, ids.long(), w)
        y = torch.einsum("eth,te->th", h @ _expert_values(s["down"]).transpose(1, 2), share)
    return {"ids": ids, "weights": w, "y": y.bfloat16()}


def _run_plain(s):
    if s["op"] == "quantize":
        x, out = s["x"].float(), {}
        if s["orient"] != "cols":
            out["rows"] = _mx_values(x, s["rule"]).bfloat16()  # two significant bits: exact in bf16
        if s["orient"] != "rows":
            out["cols"] = _mx_values(_columns(x), s["rule"]).bfloat16()
        return out
    if s["op"] == "linear":
        a = _mx_values(s["x"].float(), "floor") if s["raw"] else _operand_values(s["x"])
        return (a @ _operand_values(s["w"]).T).to(_TYPES[s["out"]])
    if s["op"] == "step":
        x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
        q = lambda v: _mx_values(v, "floor")  # noqa: E731
        y = q(x) @ q(w).T
        dx = q(dy) @ q(_columns(w)).T
        dw = q(_columns(dy)) @ q(_columns(x)).T
        return {"y": y.bfloat16(), "dx": dx.bfloat16(), "dw": dw}
    if s["op"] == "route":
        ids, w = _route_plain(s, s["renorm"])
        return {"ids": ids, "weights": w}
    return _moe_plain(s)


def _run_own(s):
    import nvfp4_block_scaled_14_b200 as nv
    if s["op"] == "quantize":
        q = nv.quantize_mxfp4(s["x"], scale_rule=s["rule"], orient=s["orient"], linear=True)
        q = dict(zip(("rows", "cols"), q)) if s["orient"] == "both" else {s["orient"]: q}
        return {side: nv.dequantize_mxfp4(v, torch.bfloat16) for side, v in q.items()}
    if s["op"] == "linear":
        w = nv.MXFP4Tensor(s["w"]["codes"], s["w"]["swz"], s["w"]["lin"], s["n"], s["k"])
        if s["raw"]:
            return nv.linear_dynamic_mxfp4(s["x"], w, out_dtype=_TYPES[s["out"]], resident_weights=True)
        a = nv.MXFP4Tensor(s["x"]["codes"], s["x"]["swz"], s["x"]["lin"], s["m"], s["k"])
        return nv.linear_mxfp4(a, w, out_dtype=_TYPES[s["out"]], resident_weights=True)
    if s["op"] == "step":
        x, xt = nv.quantize_mxfp4(s["x"], orient="both")
        w, wt = nv.quantize_mxfp4(s["w"], orient="both")
        dy, dyt = nv.quantize_mxfp4(s["dy"], orient="both")
        return {"y": nv.linear_mxfp4(x, w), "dx": nv.linear_mxfp4(dy, wt), "dw": nv.linear_mxfp4(dyt, xt, out_dtype=torch.float32)}
    renorm = s.get("renorm", True)
    ids, w = nv.moe_route(s["x"], s["wr"], s["k"], bias=s["bias"], renormalize=renorm)
    if s["op"] == "route":
        return {"ids": ids, "weights": w}
    up = nv.ExpertWeights(s["up"]["codes"], s["up"]["scales"], s["up"]["gs"])
    down = nv.ExpertWeights(s["down"]["codes"], s["down"]["scales"], s["down"]["gs"])
    return {"ids": ids, "weights": w, "y": nv.moe_experts(s["x"], ids, w, up, down)}


# ---- exact values ----------------------------------------------------------------------------


def _exact_e2m1(v):
    """Nearest E2M1 value of fp64 values: multiples of half the binade's unit, rounded half to even."""
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent.clamp(min=1) - 2)
    return (torch.round(v / step) * step).clamp(-6.0, 6.0)


def _exact_mx(x, rule):
    v = x.double().reshape(x.shape[0], -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    if rule == "floor":
        s = torch.frexp(top).exponent - 3
    else:
        mant, s = torch.frexp(top / 6.0)
        s = torch.where(mant == 0.5, s - 1, s)
    s = torch.where(top > 0, s, torch.full_like(s, -127)).clamp(min=-127)
    one = torch.ones_like(top)
    return (_exact_e2m1(v * torch.ldexp(one, -s)) * torch.ldexp(one, s)).reshape(x.shape)


def _exact_codes(codes, scale, block):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int16)
    e, m = (n >> 1) & 3, (n & 1).double()
    mag = torch.where(e == 0, 0.5 * m, torch.ldexp(1.0 + 0.5 * m, (e - 1).int()))
    return torch.where(n >= 8, -mag, mag) * scale.repeat_interleave(block, -1)


def _exact_operand(o):
    b = o["lin"].int()
    return _exact_codes(o["codes"], torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127), 32)


def _exact_expert(o, e):
    if o["gs"] is None:
        b = o["scales"][e].int()
        return _exact_codes(o["codes"][e], torch.ldexp(torch.ones_like(b, dtype=torch.float64), b - 127), 32)
    return _exact_codes(o["codes"][e], o["scales"][e].view(torch.float8_e4m3fn).double() * o["gs"][e].double(), 16)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "quantize":
        out = {}
        if c["orient"] != "cols":
            out["rows"] = _exact_mx(s["x"], c["rule"])
        if c["orient"] != "rows":
            out["cols"] = _exact_mx(_columns(s["x"]), c["rule"])
        return out
    if c["op"] == "linear":
        a = _exact_mx(s["x"], "floor") if c["raw"] else _exact_operand(s["x"])
        return a @ _exact_operand(s["w"]).T
    if c["op"] == "step":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        return {"y": _exact_mx(x, "floor") @ _exact_mx(w, "floor").T,
                "dx": _exact_mx(dy, "floor") @ _exact_mx(_columns(w), "floor").T,
                "dw": _exact_mx(_columns(dy), "floor") @ _exact_mx(_columns(x), "floor").T}
    z = (s["x"].double()[:, None, :] * s["wr"].double()[None]).sum(-1) + s["bias"].double()
    renorm = c["op"] == "moe" or c["renorm"]
    share = torch.zeros_like(z)
    left, weights = z.clone(), []
    for _ in range(c["k"]):  # the largest left, the lowest index of equal ones
        best = left.amax(-1, keepdim=True)
        at = (left == best).int().argmax(-1, keepdim=True)
        share.scatter_(1, at, (best > -math.inf).double())
        weights.append(at)
        left.scatter_(1, at, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.where(z > -math.inf, torch.exp(z - torch.where(top > -math.inf, top, 0.0)), 0.0)
    norm = (p * share if renorm else p).sum(-1, keepdim=True)
    share = torch.where(norm > 0, p * share / norm.clamp(min=1e-300), 0.0)
    out = {"ids": None, "weights": torch.cat([share.gather(1, at) for at in weights], 1)}
    # a slot past the last open expert has no weight; its index repeats, so it is told by order
    live = (z > -math.inf).sum(-1, keepdim=True) > torch.arange(c["k"], device=z.device)
    out["weights"] = torch.where(live, out["weights"], 0.0)
    if c["op"] == "route":
        return out
    x, f = s["x"].double(), c["f"]
    y = torch.zeros(c["t"], c["h"], dtype=torch.float64, device=x.device)
    for e in range(c["e"]):
        t = share[:, e].nonzero()[:, 0]
        if t.numel():
            a = x[t] @ _exact_expert(s["up"], e).T
            gate, up = a[:, :f], a[:, f:]
            y[t] += share[t, e, None] * ((gate / (1.0 + torch.exp(-gate)) * up) @ _exact_expert(s["down"], e).T)
    out["y"] = y
    return out
