"""What is measured of the operators around the projections of a quantized MLP:
the RMS norm that ends in 8- or 4-bit codes and its backward, the microscaled
4-bit quantizer, and the product of two 4-bit operands.

A case names an operator (``op``), its sizes and its formats:

  norm          h = bf16(x + residual); y = h / rms(h) * weight; codes of y
  norm_bwd      the gradients of that norm's input and weight
  quant         bf16 -> 4-bit codes and scales along the rows (and along the
                columns, transposed), read back as the values they stand for
  product       A (4 bit) x B (4 bit) transposed -> bf16
  linear        bf16 activations quantized, then the product with weights laid
                out before
  linear_bwd    both gradients of a linear layer: the incoming gradient is
                quantized along both axes, then multiplied with the transposed
                weight and the transposed activations kept from the forward

4-bit formats: "e8m0" (E2M1 codes, one power-of-two scale for 32 values) and
"e4m3" (E2M1 codes, one E4M3 scale for 16 values, times a scale per tensor).
Codes are packed two to a byte, the lower index in the low four bits; scales
lie in tiles of 128 rows x 4 groups, 512 bytes each: the scale of row r and
group g is byte (r % 32) * 16 + (r % 128) // 32 * 4 + g % 4 of its tile.
"""
import math

import torch

own = False

DEVICE = "cuda"


# ---- the cases --------------------------------------------------------------------

def _norm(name, rows, channels, codes, scales, group, residual, weight):
    return {"name": name, "op": "norm", "rows": rows, "channels": channels, "codes": codes,
            "scales": scales, "group": group, "residual": residual, "weight": weight}


def listed():
    return [
        # one token decoded: the norm before a projection, latency alone
        _norm("norm_1x7168_e4m3", 1, 7168, "e4m3", "fp32", 128, True, "bf16"),
        # a ragged batch of decoded tokens, straight to the 4-bit operand of the product
        _norm("norm_37x4096_e2m1", 37, 4096, "e2m1", "e8m0", 32, True, "bf16"),
        # one scale a token and INT8 codes, no residual, an odd number of rows
        _norm("norm_4099x1408_int8", 4099, 1408, "int8", "fp32", 0, False, "fp32"),
        # the benchmark's largest activation: a training or prefill step's norm
        _norm("norm_16384x7168_e4m3", 16384, 7168, "e4m3", "fp32", 128, True, "bf16"),
        # the backward of a short ragged step, and of a full one
        {"name": "norm_bwd_517x7168", "op": "norm_bwd", "rows": 517, "channels": 7168, "residual": True,
         "weight": "bf16"},
        {"name": "norm_bwd_16384x4096", "op": "norm_bwd", "rows": 16384, "channels": 4096,
         "residual": True, "weight": "fp32"},
        # activations of a few tokens; a training step's tensor quantized for all three products
        {"name": "quant_19x7168_e8m0", "op": "quant", "rows": 19, "channels": 7168, "scales": "e8m0",
         "columns": False},
        {"name": "quant_8192x4096_e4m3_both", "op": "quant", "rows": 8192, "channels": 4096,
         "scales": "e4m3", "columns": True},
        # one token against a layer's weights: bound by reading them
        {"name": "product_1x4096x7168_e4m3", "op": "product", "rows": 1, "outs": 4096, "channels": 7168,
         "scales": "e4m3"},
        # a ragged serving batch through a linear layer, quantizer included
        {"name": "linear_61x7168x4096_e8m0", "op": "linear", "rows": 61, "outs": 7168, "channels": 4096,
         "scales": "e8m0"},
        # prefill or a training forward: gate and up projections in one product
        {"name": "product_8192x14336x4096_e8m0", "op": "product", "rows": 8192, "outs": 14336,
         "channels": 4096, "scales": "e8m0"},
        # a training backward of a projection with a ragged token count
        {"name": "linear_bwd_4064x4096x2816_e4m3", "op": "linear_bwd", "rows": 4064, "outs": 4096,
         "channels": 2816, "scales": "e4m3"},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "norm_bwd", "norm_bwd", "quant", "quant", "product", "product",
                     "linear", "linear_bwd"])
    if op == "norm":
        codes = rng.choice(["int8", "e4m3", "e2m1"])
        scales = rng.choice(["e8m0", "e4m3"] if codes == "e2m1" else ["fp32", "e8m0"])
        group = {"e8m0": 32, "e4m3": 16}[scales] if codes == "e2m1" else rng.choice([0, 32, 64, 128, 256])
        return {"op": op, "rows": _log(rng, 1, 16384), "channels": _log(rng, 64, 7168, 32 if codes == "e2m1" else 16),
                "codes": codes, "scales": scales, "group": group, "residual": rng.random() < 0.7,
                "weight": rng.choice(["bf16", "fp32"])}
    if op == "norm_bwd":
        return {"op": op, "rows": _log(rng, 1, 16384), "channels": _log(rng, 64, 7168, 16),
                "residual": rng.random() < 0.7, "weight": rng.choice(["bf16", "fp32"])}
    scales = rng.choice(["e8m0", "e4m3"])
    if op == "quant":
        return {"op": op, "rows": _log(rng, 1, 8192), "channels": _log(rng, 32, 7168, 32), "scales": scales,
                "columns": rng.random() < 0.5}
    return {"op": op, "rows": _log(rng, 1, 4096 if op == "linear_bwd" else 8192),
            "outs": _log(rng, 64, 7168, 32 if op == "linear_bwd" else 1),
            "channels": _log(rng, 64, 7168, 32), "scales": scales}


# ---- inputs -----------------------------------------------------------------------

def _normal(gen, rows, channels, sigma=1.0, outliers=False):
    """bf16 activations; with outliers, a few channels an order of magnitude larger."""
    x = torch.randn(rows, channels, generator=gen, device=DEVICE) * sigma
    if outliers:
        big = torch.rand(channels, generator=gen, device=DEVICE) < 0.01
        x = torch.where(big, x * 12, x)
    return x.bfloat16()


def _scale_bytes(rows, channels, scales):
    groups = channels // _GROUP[scales]
    return -(-rows // 128), -(-groups // 4), 512


def _empty_fp4(rows, channels, scales):
    return (torch.empty(rows, channels // 2, dtype=torch.uint8, device=DEVICE),
            torch.empty(_scale_bytes(rows, channels, scales), dtype=_SCALE_DTYPE[scales], device=DEVICE))


def _up32(n):
    return -(-n // 32) * 32


def _global(x, scales):
    """The scale per tensor of the "e4m3" format: the tensor's largest value is then 448 * 6 of its units. Kept to
    eight bits, so that its products with scales and borders are exact in 32: bf16 values meet many exact ties."""
    return (x.float().abs().amax() / 2688).bfloat16().float().reshape(1) if scales == "e4m3" else None


def _pack(values, group_scales, scales):
    """(codes, scale tiles) of a plain quantization's E2M1 values and scales."""
    code = (values.abs() * 2).to(torch.int64)
    code = torch.where(code >= 8, (code + 16) // 4, torch.where(code >= 4, (code + 4) // 2, code))
    code = torch.where(code > 7, 7, code) | (torch.signbit(values).to(torch.int64) << 3)
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8)
    rows, groups = group_scales.shape
    tr, tg = -(-rows // 128), -(-groups // 4)
    full = torch.zeros(tr * 128, tg * 4, dtype=torch.uint8, device=DEVICE)
    full[:rows, :groups] = group_scales.to(_SCALE_DTYPE[scales]).view(torch.uint8)
    tiles = full.reshape(tr, 4, 32, tg, 4).permute(0, 3, 2, 1, 4).reshape(tr, tg, 512).contiguous()
    return packed, tiles.view(_SCALE_DTYPE[scales])


def _operand(x, scales):
    """A 4-bit operand as a program keeps it: codes, scale tiles, the scale per tensor."""
    g = _global(x, scales)
    values, s = _quant_fp4(x.float(), scales, g)
    return (*_pack(values, s, scales), g)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, rows, channels = case["op"], case["rows"], case["channels"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        w = 1 + 0.2 * torch.randn(channels, generator=gen, device=DEVICE)
        s["weight"] = w if case["weight"] == "fp32" else w.bfloat16()
    if op == "norm":
        s["x"] = _normal(gen, rows, channels, 0.7)
        s["residual"] = _normal(gen, rows, channels, 1.5, outliers=True) if case["residual"] else None
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["global"] = (torch.rand(1, generator=gen, device=DEVICE) + 0.5) * 2.0 ** -8 \
            if case["scales"] == "e4m3" else None
        if case["codes"] == "e2m1":
            s["q"], s["s"] = _empty_fp4(rows, channels, case["scales"])
            s["values"] = torch.empty_like(s["x"])
        else:
            groups = -(-channels // (case["group"] or channels))
            s["q"] = torch.empty(rows, channels, dtype=torch.int8 if case["codes"] == "int8" else torch.float8_e4m3fn,
                                 device=DEVICE)
            s["s"] = torch.empty(rows, groups, device=DEVICE,
                                 dtype=torch.float32 if case["scales"] == "fp32" else torch.float8_e8m0fnu)
    elif op == "norm_bwd":
        s["h"] = _normal(gen, rows, channels, 1.5, outliers=True)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + _EPS).float()
        s["grad_y"] = _normal(gen, rows, channels, 0.01)
        s["grad_h"] = _normal(gen, rows, channels, 0.02) if case["residual"] else None
        s["grad_x"] = torch.empty_like(s["h"])
        s["grad_weight"] = torch.empty(channels, device=DEVICE)
    elif op == "quant":
        s["x"] = _normal(gen, rows, channels, 1.0, outliers=True)
        s["global"] = _global(s["x"], case["scales"])
        s["out"] = _empty_fp4(rows, channels, case["scales"])
        s["values"] = torch.empty_like(s["x"])
        if case["columns"]:
            s["out"] += _empty_fp4(channels, _up32(rows), case["scales"])
            s["values_t"] = torch.empty(channels, _up32(rows), dtype=torch.bfloat16, device=DEVICE)
    else:
        outs, scales = case["outs"], case["scales"]
        x = _normal(gen, rows, channels, 1.0, outliers=True)
        w = _normal(gen, outs, channels, 0.02)
        if op == "linear_bwd":
            gy = _normal(gen, rows, outs, 0.01)
            pad = torch.zeros(_up32(rows) - rows, channels, dtype=torch.bfloat16, device=DEVICE)
            s["x_t"] = _operand(torch.cat([x, pad]).t().contiguous(), scales)
            s["w_t"] = _operand(w.t().contiguous(), scales)
            s["grad_y"], s["global"] = gy, _global(gy, scales)
            s["out"] = _empty_fp4(rows, outs, scales) + _empty_fp4(outs, _up32(rows), scales)
            s["grad_x"] = torch.empty_like(x)
            s["grad_w"] = torch.empty(outs, channels, device=DEVICE)
        else:
            s["w"] = _operand(w, scales)
            s["y"] = torch.empty(rows, outs, dtype=torch.bfloat16, device=DEVICE)
            if op == "product":
                s["x"] = _operand(x, scales)
            else:
                s["x"], s["global"] = x, _global(x, scales)
                s["out"] = _empty_fp4(rows, channels, scales)
    return s


# ---- the plain forms --------------------------------------------------------------

_EPS = 1e-6
_GROUP = {"e8m0": 32, "e4m3": 16}
_SCALE_DTYPE = {"e8m0": torch.float8_e8m0fnu, "e4m3": torch.float8_e4m3fn}
_QMAX = {"int8": 127.0, "e4m3": 448.0, "e2m1": 6.0}


def _pow2_ceil(t):
    """The smallest power of two not below t > 0, as E8M0 holds it."""
    m, e = torch.frexp(t)
    return torch.ldexp(torch.ones_like(t), torch.where(m == 0.5, e - 1, e).clamp(-126, 127))


def _e4m3(v):
    return v.clamp(-448, 448).to(torch.float8_e4m3fn)


def _e2m1(v):
    """Round to nearest, ties to even, onto 0, .5, 1, 1.5, 2, 3, 4, 6; larger ones to 6."""
    a = v.abs().clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _quant_fp4(x, scales, g):
    """(E2M1 values, scales of the groups) of fp32 rows, both as numbers."""
    rows, channels = x.shape
    v = x.reshape(rows, -1, _GROUP[scales])
    amax = v.abs().amax(2)
    if scales == "e8m0":
        s = _pow2_ceil(amax / torch.full_like(amax, 6))     # a quotient, not a product with fl32(1 / 6)
        unit = s = torch.where(amax > 0, s, 1.0)
    else:
        s = _e4m3(amax / (6 * g)).float().clamp(min=2.0 ** -9)
        s = torch.where(amax > 0, s, 1.0)
        unit = s * g
    return _e2m1(v / unit.unsqueeze(2)).reshape(rows, channels), s


def _expand(s, scales, g):
    unit = s if g is None else s * g
    return unit.repeat_interleave(_GROUP[scales], 1)


def _fake_quant(x, scales, g):
    values, s = _quant_fp4(x, scales, g)
    return values * _expand(s, scales, g)


def _unpack(codes, tiles, scales, g):
    """fp32 values of packed codes and scale tiles."""
    rows, channels = codes.shape[0], codes.shape[1] * 2
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEVICE)
    b = codes.int()
    v = table[torch.stack([b & 15, b >> 4], 2).reshape(rows, channels)]
    tr, tg, _ = tiles.shape
    s = tiles.float().reshape(tr, tg, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tr * 128, tg * 4)
    return v * _expand(s[:rows, :channels // _GROUP[scales]], scales, g)


def _plain_norm(s):
    case = s["case"]
    h = s["x"]
    if case["residual"]:
        h = (s["x"].float() + s["residual"].float()).bfloat16()
    f = h.float()
    y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + _EPS) * s["weight"].float()
    rows, channels = y.shape
    out = {"h": h} if case["residual"] else {}
    if case["codes"] == "e2m1":
        out["values"] = _fake_quant(y, case["scales"], s["global"]).bfloat16()
        return out
    group = case["group"] or channels
    pad = -channels % group
    v = torch.nn.functional.pad(y, (0, pad)).reshape(rows, -1, group)
    amax = v.abs().amax(2)
    sc = amax / _QMAX[case["codes"]]
    if case["scales"] == "e8m0":
        sc = _pow2_ceil(sc)
    sc = torch.where(amax > 0, sc, 1.0)
    v = (v * (1 / sc).unsqueeze(2)).reshape(rows, -1)[:, :channels]
    out["q"] = torch.round(v).bfloat16() if case["codes"] == "int8" else _e4m3(v)
    out["s"] = sc if case["scales"] == "fp32" else sc.to(torch.float8_e8m0fnu)
    return out


def _plain_norm_bwd(s):
    h, gy, rstd = s["h"].float(), s["grad_y"].float(), s["rstd"].unsqueeze(1)
    n = h * rstd
    gn = gy * s["weight"].float()
    gx = rstd * (gn - n * (gn * n).mean(1, keepdim=True))
    if s["case"]["residual"]:
        gx = gx + s["grad_h"].float()
    return {"grad_x": gx.bfloat16(), "grad_weight": (gy * n).sum(0)}


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_bwd":
        return _plain_norm_bwd(s)
    scales = case["scales"]
    if op == "quant":
        x = s["x"].float()
        out = {"values": _fake_quant(x, scales, s["global"]).bfloat16()}
        if case["columns"]:
            x = torch.nn.functional.pad(x, (0, 0, 0, _up32(case["rows"]) - case["rows"])).t().contiguous()
            out["values_t"] = _fake_quant(x, scales, s["global"]).bfloat16()
        return out
    if op == "product":
        return _unpack(*s["x"][:2], scales, s["x"][2]).matmul(_unpack(*s["w"][:2], scales, s["w"][2]).t()).bfloat16()
    if op == "linear":
        return _fake_quant(s["x"].float(), scales, s["global"]).matmul(
            _unpack(*s["w"][:2], scales, s["w"][2]).t()).bfloat16()
    gy = s["grad_y"].float()
    gx = _fake_quant(gy, scales, s["global"]).matmul(_unpack(*s["w_t"][:2], scales, s["w_t"][2]).t())
    gy = torch.nn.functional.pad(gy, (0, 0, 0, _up32(case["rows"]) - case["rows"])).t().contiguous()
    gw = _fake_quant(gy, scales, s["global"]).matmul(_unpack(*s["x_t"][:2], scales, s["x_t"][2]).t())
    return {"grad_x": gx.bfloat16(), "grad_w": gw}


# ---- the framework's operators ----------------------------------------------------

def _own(s):
    import swiglu_backward_int8_b200 as sdq
    case = s["case"]
    op = case["op"]
    if op == "norm":
        sdq.rmsnorm_quant(s["x"], s["weight"], s["residual"], eps=_EPS, group_size=case["group"],
                          codes=case["codes"], scales=case["scales"], q=s["q"], s=s["s"], h=s["h"],
                          global_scale=s["global"])
        out = {"h": s["h"]} if case["residual"] else {}
        if case["codes"] == "e2m1":
            out["values"] = sdq.dequantize_fp4(s["q"], s["s"], global_scale=s["global"], out=s["values"])
            return out
        out["q"] = s["q"].bfloat16() if case["codes"] == "int8" else s["q"]
        out["s"] = s["s"]
        return out
    if op == "norm_bwd":
        sdq.rmsnorm_backward(s["grad_y"], s["h"], s["weight"], s["rstd"], s["grad_h"], grad_x=s["grad_x"],
                             grad_weight=s["grad_weight"])
        return {"grad_x": s["grad_x"], "grad_weight": s["grad_weight"]}
    if op == "quant":
        o = s["out"]
        sdq.quantize_fp4(s["x"], scales=case["scales"], axis="both" if case["columns"] else "rows", q=o[0], s=o[1],
                         q_t=o[2] if case["columns"] else None, s_t=o[3] if case["columns"] else None,
                         global_scale=s["global"])
        out = {"values": sdq.dequantize_fp4(o[0], o[1], global_scale=s["global"], out=s["values"])}
        if case["columns"]:
            out["values_t"] = sdq.dequantize_fp4(o[2], o[3], global_scale=s["global"], out=s["values_t"])
        return out
    if op == "product":
        (a, a_s, a_g), (b, b_s, b_g) = s["x"], s["w"]
        return sdq.matmul_fp4(a, a_s, b, b_s, a_global=a_g, b_global=b_g, out=s["y"])
    if op == "linear":
        (q, qs), (b, b_s, b_g) = s["out"], s["w"]
        sdq.quantize_fp4(s["x"], scales=case["scales"], q=q, s=qs, global_scale=s["global"])
        return sdq.matmul_fp4(q, qs, b, b_s, a_global=s["global"], b_global=b_g, out=s["y"])
    q, qs, q_t, qs_t = s["out"]
    sdq.quantize_fp4(s["grad_y"], scales=case["scales"], axis="both", q=q, s=qs, q_t=q_t, s_t=qs_t,
                     global_scale=s["global"])
    (w, w_s, w_g), (x, x_s, x_g) = s["w_t"], s["x_t"]
    return {"grad_x": sdq.matmul_fp4(q, qs, w, w_s, a_global=s["global"], b_global=w_g, out=s["grad_x"]),
            "grad_w": sdq.matmul_fp4(q_t, qs_t, x, x_s, a_global=s["global"], b_global=x_g, out=s["grad_w"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---- what a pass cannot do without ------------------------------------------------

def _fp4_bytes(rows, channels, scales):
    return rows * channels // 2 + rows * channels // _GROUP[scales]


def work(case):
    op, m, k = case["op"], case["rows"], case["channels"]
    if op == "norm":
        w = k * (4 if case["weight"] == "fp32" else 2)
        read = m * k * (4 if case["residual"] else 2) + w
        write = m * k * 2 if case["residual"] else 0
        if case["codes"] == "e2m1":     # codes and scales written, read back, their values written
            write += 2 * _fp4_bytes(m, k, case["scales"]) + 2 * m * k
        else:
            groups = -(-k // (case["group"] or k))
            write += m * k + m * groups * (4 if case["scales"] == "fp32" else 1)
            if case["codes"] == "int8":     # the codes as numbers of a wider type
                write += 3 * m * k
        return {"bytes": read + write, "flops": 8 * m * k}
    if op == "norm_bwd":
        w = k * (4 if case["weight"] == "fp32" else 2)
        return {"bytes": m * k * (8 if case["residual"] else 6) + 4 * m + w + 4 * k, "flops": 12 * m * k}
    if op == "quant":
        b = 2 * m * k + 2 * _fp4_bytes(m, k, case["scales"]) + 2 * m * k
        if case["columns"]:
            b += 2 * _fp4_bytes(k, _up32(m), case["scales"]) + 2 * _up32(m) * k
        return {"bytes": b, "flops": 6 * m * k * (2 if case["columns"] else 1)}
    n = case["outs"]
    if op == "product":
        return {"bytes": _fp4_bytes(m, k, case["scales"]) + _fp4_bytes(n, k, case["scales"]) + 2 * m * n,
                "flops": 2 * m * n * k}
    if op == "linear":
        return {"bytes": 2 * m * k + 2 * _fp4_bytes(m, k, case["scales"]) + _fp4_bytes(n, k, case["scales"]) + 2 * m * n,
                "flops": 2 * m * n * k}
    mp = _up32(m)
    b = 2 * m * n + 2 * _fp4_bytes(m, n, case["scales"]) + 2 * _fp4_bytes(n, mp, case["scales"])
    b += _fp4_bytes(k, n, case["scales"]) + _fp4_bytes(k, mp, case["scales"]) + 2 * m * k + 4 * n * k
    return {"bytes": b, "flops": 4 * m * n * k}


# ---- the definitions in 64 bits -----------------------------------------------------

def _x_e2m1(v):
    """Nearest of the eight magnitudes by comparison with the midpoints; ties go to the even code."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEVICE)
    mids = (grid[1:] + grid[:-1]) / 2
    a = v.abs()
    lo, hi = torch.bucketize(a, mids), torch.bucketize(a, mids, right=True)
    return torch.where(v < 0, -1.0, 1.0) * grid[torch.where(lo % 2 == 0, lo, hi)]


def _x_e4m3(v):
    """Nearest E4M3 number by its spacing: 2^(e - 3), no finer than 2^-9."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _x_pow2(v):
    e = torch.ceil(torch.log2(v.clamp(min=2.0 ** -200)))
    e = torch.where(torch.exp2(e - 1) >= v, e - 1, e)
    return torch.exp2(torch.where(torch.exp2(e) < v, e + 1, e).clamp(-127, 127))


def _x_fp4(x, scales, g):
    """Rows of 64-bit numbers quantized and read back."""
    n = 32 if scales == "e8m0" else 16
    v = x.reshape(-1, n)
    top = v.abs().max(1, keepdim=True).values
    if scales == "e8m0":
        unit = _x_pow2(top / 6)
    else:
        g = g.double()
        unit = _x_e4m3(top / (6 * g)).clamp(min=2.0 ** -9) * g
    unit = torch.where(top > 0, unit, 1.0)
    return (_x_e2m1(v / unit) * unit).reshape(x.shape)


def _x_operand(codes, tiles, g):
    """Codes from their bits (sign, two exponent bits, one of mantissa), scales by gathering from the tiles."""
    rows, half = codes.shape
    c = torch.stack([codes % 16, codes // 16], 2).reshape(rows, 2 * half).long()
    mant, expo, sign = c % 2, c // 2 % 4, c // 8
    v = torch.where(expo == 0, mant * 0.5, (1 + mant * 0.5).double() * torch.exp2((expo - 1).double()))
    v = torch.where(sign == 1, -v, v)
    n = 32 if tiles.dtype == torch.float8_e8m0fnu else 16
    r = torch.arange(rows, device=DEVICE).unsqueeze(1)
    k = torch.arange(2 * half // n, device=DEVICE).unsqueeze(0)
    at = (r // 128 * tiles.shape[1] + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4
    b = tiles.view(torch.uint8).reshape(-1)[at].long()
    if n == 32:
        s = torch.exp2((b - 127).double())
    else:
        s = torch.where(b // 8 == 0, (b % 8).double() * 2.0 ** -9,
                        (1 + (b % 8).double() / 8) * torch.exp2((b // 8 - 7).double()))
    v = (v.reshape(rows, -1, n) * s.unsqueeze(2)).reshape(rows, 2 * half)
    return v if g is None else v * g.double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        out = {}
        if case["residual"]:
            x = x + s["residual"].double()
            out["h"] = x
            x = x.float().bfloat16().double()
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + _EPS) * s["weight"].double()
        if case["codes"] == "e2m1":
            out["values"] = _x_fp4(y, case["scales"], s["global"])
            return out
        group = case["group"] or case["channels"]
        q, sc = [], []
        for part in y.split(group, 1):
            top = part.abs().max(1, keepdim=True).values
            unit = top / {"int8": 127, "e4m3": 448}[case["codes"]]
            if case["scales"] == "e8m0":
                unit = _x_pow2(unit)
            unit = torch.where(top > 0, unit, 1.0)
            q.append(torch.round(part / unit) if case["codes"] == "int8" else _x_e4m3(part / unit))
            sc.append(unit)
        out["q"], out["s"] = torch.cat(q, 1), torch.cat(sc, 1)
        return out
    if op == "norm_bwd":
        h, gy, w, r = s["h"].double(), s["grad_y"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        dot = (gy * w * h).sum(1, keepdim=True)
        gx = gy * w * r - h * (r ** 3 * dot / h.shape[1])
        if case["residual"]:
            gx = gx + s["grad_h"].double()
        return {"grad_x": gx, "grad_weight": torch.einsum("mk,mk,m->k", gy, h, r[:, 0])}
    scales = case["scales"]
    if op == "quant":
        x = s["x"].double()
        out = {"values": _x_fp4(x, scales, s["global"])}
        if case["columns"]:
            full = torch.zeros(_up32(case["rows"]), case["channels"], dtype=torch.float64, device=DEVICE)
            full[:case["rows"]] = x
            out["values_t"] = _x_fp4(full.t().contiguous(), scales, s["global"])
        return out
    if op == "product":
        return _x_operand(*s["x"]) @ _x_operand(*s["w"]).t()
    if op == "linear":
        return _x_fp4(s["x"].double(), scales, s["global"]) @ _x_operand(*s["w"]).t()
    gy = torch.zeros(_up32(case["rows"]), case["outs"], dtype=torch.float64, device=DEVICE)
    gy[:case["rows"]] = s["grad_y"].double()
    return {"grad_x": _x_fp4(s["grad_y"].double(), scales, s["global"]) @ _x_operand(*s["w_t"]).t(),
            "grad_w": _x_fp4(gy.t().contiguous(), scales, s["global"]) @ _x_operand(*s["x_t"]).t()}
