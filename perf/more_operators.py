"""What the operators of the gated, dropout-regularised residual block are measured on.

Five operators around the FP8 linear layer: the gated product (both projections,
the activation and their product), its data gradient, layer norm that casts its
output to fp8 (with the residual's addition in front), its backward pass, and
dropout from a counter-based generator whose mask is never stored, added to the
residual stream.  ``run`` computes a case either with the library (``own``) or
in elementary torch operations in fp32.
"""
import math

import torch

own = False

E4M3, E5M2 = 0, 1
FMAX = {E4M3: 448.0, E5M2: 57344.0}
CODE = {E4M3: torch.float8_e4m3fn, E5M2: torch.float8_e5m2}
EPS = 1e-5


# ------------------------------------------------------------------- cases --

def gated(name, m, n, k, recipe="block", act="silu", bias=False, aux=False):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "recipe": recipe, "act": act, "bias": bias,
            "aux": aux}


def dgrad(name, m, n, k, recipe="block", act="silu"):
    return {"name": name, "op": "dgrad", "m": m, "n": n, "k": k, "recipe": recipe, "act": act}


def norm(name, rows, cols, recipe="block", both=False, residual=True, beta=True):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "recipe": recipe, "both": both,
            "residual": residual, "beta": beta}


def back(name, rows, cols, skip=True, beta=True):
    return {"name": name, "op": "back", "rows": rows, "cols": cols, "skip": skip, "beta": beta}


def drop(name, rows, cols, p=0.1, residual=True):
    return {"name": name, "op": "drop", "rows": rows, "cols": cols, "p": p, "residual": residual}


def listed():
    return [
        # one new token of a decode step through both up projections: one read of their weights
        gated("gated token", 1, 14336, 4096),
        # a prompt of odd length with biases and the GELU gate, one scale per tensor
        gated("gated prompt", 1001, 7168, 2048, recipe="tensor", act="gelu", bias=True),
        # the training step's tokens, both pre-activations kept for the backward pass
        gated("gated train", 8192, 14336, 4096, aux=True),
        # a short fine-tuning batch on MXFP8 operands
        dgrad("dgrad short", 1000, 2048, 1024, recipe="mx", act="gelu"),
        # the training step's gradient through the down projection and the gate
        dgrad("dgrad train", 8192, 14336, 4096),
        # one new token of a decode step: the norm in front of the up projections
        norm("norm token", 1, 4096, recipe="tensor"),
        # a prompt of odd length, MXFP8 operands, a norm without bias
        norm("norm prompt", 777, 7168, recipe="mx", beta=False),
        # the training step's tokens: row codes for the forward product and column codes for the weight gradient
        norm("norm train", 8192, 4096, both=True),
        # a short fine-tuning batch without a residual branch beside the norm
        back("back short", 1000, 2048, skip=False),
        # a long training batch, with the gradient of the residual branch added
        back("back long", 16384, 7168),
        # the gradient of a small ragged batch through the mask
        drop("drop short", 129, 1001, p=0.25, residual=False),
        # the training step's tokens on their way into the residual stream
        drop("drop train", 8192, 4096),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated", "dgrad", "dgrad", "norm", "norm", "back", "drop"))
    recipe = rng.choice(("block", "mx", "tensor"))
    act = rng.choice(("silu", "gelu"))
    yes = lambda: rng.random() < 0.5  # noqa: E731
    if op in ("gated", "dgrad"):
        n, k = 128 * spread(rng, 1, 112), 128 * spread(rng, 1, 112)
        m = spread(rng, 1, min(8192, 2 ** 38 // (n * k)))
        c = gated("", m, n, k, recipe, act, yes(), yes()) if op == "gated" else dgrad("", m, n, k, recipe, act)
    elif op == "norm":
        cols = 128 * spread(rng, 1, 64)
        most = min(16384, 8192 * 4096 // cols)
        if yes():
            c = norm("", 128 * spread(rng, 1, most // 128), cols, recipe, True, yes(), yes())
        else:
            c = norm("", spread(rng, 1, most), cols, recipe, False, yes(), yes())
    elif op == "back":
        cols = 8 * spread(rng, 8, 1024)
        c = back("", spread(rng, 1, min(32768, 8192 * 4096 // cols)), cols, yes(), yes())
    else:
        cols = spread(rng, 64, 8192)
        c = drop("", spread(rng, 1, min(32768, 8192 * 4096 // cols)), cols, rng.choice((0.05, 0.1, 0.25, 0.5)), yes())
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs --

def normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std)


def activations(g, rows, cols):
    """Rows of a residual stream: off centre, a few channels stand out, and one row in a batch holds nothing (a padded
    token)."""
    x = normal(g, rows, cols).add_(normal(g, rows, 1, std=0.5))
    x[:, torch.randint(0, cols, (max(1, cols // 256),), generator=g, device="cuda")] *= 16.0
    if rows > 4:
        x[rows // 3] = 0.0
    return x.bfloat16()


def atoms(e):
    """Power-of-two exponents [rows][K/32] -> the scale bytes in the library's order (rows beyond the matrix hold 127)."""
    rows, n = e.shape
    groups = 2 * -(-rows // 256)
    b = torch.full((groups * 128, n), 127, dtype=torch.uint8, device=e.device)
    b[:rows] = (e + 127).to(torch.uint8)
    return b.view(groups, 4, 32, n // 4, 4).permute(3, 0, 2, 1, 4).reshape(-1)


def exponents(sf, rows, k):
    """The inverse of ``atoms``."""
    groups = 2 * -(-rows // 256)
    b = sf.view(k // 128, groups, 32, 4, 4).permute(1, 3, 2, 0, 4).reshape(groups * 128, k // 32)
    return b[:rows].to(torch.int32) - 127


def mx_exponent(amax, fmt):
    """The smallest e with amax <= FMAX 2^e (0 for a block of zeros)."""
    m, e = torch.frexp(amax)
    e = e - (9 if fmt == E4M3 else 16) + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))


def encode(v, fmt):
    return v.clamp(-FMAX[fmt], FMAX[fmt]).to(CODE[fmt])


def inverse(amax, fmt):
    """(factor before the cast, scale after it) of the block and tensor rules."""
    inv = FMAX[fmt] / amax
    ok = (amax > 0) & torch.isfinite(inv)
    return torch.where(ok, inv, torch.ones_like(inv)), torch.where(ok, amax / FMAX[fmt], torch.ones_like(amax))


def cast(y, fmt, recipe, amax=None):
    """fp32 [rows][k] -> codes, and the scales as the library lays them out ([K/128][rows], bytes, or one)."""
    rows, k = y.shape
    if recipe == "block":
        b = y.view(rows, k // 128, 128)
        inv, scale = inverse(b.abs().amax(2), fmt)
        return encode((b * inv[:, :, None]).view(rows, k), fmt), scale.t()
    if recipe == "mx":
        b = y.view(rows, k // 32, 32)
        e = mx_exponent(b.abs().amax(2), fmt)
        return encode(torch.ldexp(b, -e[:, :, None]).view(rows, k), fmt), atoms(e).view(torch.float8_e8m0fnu)
    inv, scale = inverse(amax, fmt)
    return encode(y * inv, fmt), scale


def operand(y, fmt, recipe):
    """What a cast left in hand: codes (bytes) and scales with the leading dimension that the library wants."""
    rows, k = y.shape
    codes, scale = cast(y, fmt, recipe, y.abs().amax().view(1))
    if recipe == "block":
        pad = torch.ones((k // 128, -(-rows // 4) * 4), device="cuda")
        pad[:, :rows] = scale
        scale = pad
    elif recipe == "mx":
        scale = scale.view(torch.uint8)
    return codes.view(torch.uint8).contiguous(), scale.contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = operand(normal(g, m, k), E4M3, case["recipe"])
        # gate rows, then up rows: both projections are one operand
        s["b"], s["sb"] = operand(normal(g, 2 * n, k, std=1.0 / math.sqrt(k)), E4M3, case["recipe"])
        s["bias"] = normal(g, 2 * n, std=0.1).bfloat16() if case["bias"] else None
        s["out"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        s["aux"] = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda") if case["aux"] else None
    elif case["op"] == "dgrad":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = operand(normal(g, m, k, std=1e-2), E5M2, case["recipe"])
        s["b"], s["sb"] = operand(normal(g, n, k, std=1.0 / math.sqrt(k)), E4M3, case["recipe"])
        s["z"] = normal(g, m, 2 * n).bfloat16()
        s["out"] = torch.empty((m, 2 * n), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"] = activations(g, rows, cols)
        s["residual"] = activations(g, rows, cols) if case["residual"] else None
        s["gamma"] = (1.0 + normal(g, cols, std=0.2)).bfloat16()
        s["beta"] = normal(g, cols, std=0.2).bfloat16() if case["beta"] else None
        if case["recipe"] == "tensor":
            s["amax"] = torch.rand(1, generator=g, device="cuda") * 8.0 + 8.0  # the largest of earlier steps
    elif case["op"] == "back":
        rows, cols = case["rows"], case["cols"]
        s["h"] = activations(g, rows, cols)
        s["gamma"] = (1.0 + normal(g, cols, std=0.2)).bfloat16()
        h = s["h"].double()
        mean = h.mean(1)
        s["mean"], s["rstd"] = mean.float(), torch.rsqrt((h - mean[:, None]).square().mean(1) + EPS).float()
        s["dy"] = normal(g, rows, cols, std=1e-2).bfloat16()
        s["skip"] = normal(g, rows, cols, std=1e-2).bfloat16() if case["skip"] else None
    else:
        rows, cols = case["rows"], case["cols"]
        s["x"] = normal(g, rows, cols).bfloat16()
        s["residual"] = activations(g, rows, cols) if case["residual"] else None
        # a run's seed, the place of this dropout in the model, and the step, which a captured step counts on the device
        s["seed"], s["site"] = (seed * 0x9E3779B97F4A7C15 + 1) % 2 ** 64, 5
        s["step"] = torch.randint(0, 2 ** 40, (1,), generator=g, device="cuda")
        s["out"] = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    if own:
        keep(s)
    return s


def keep(s):
    """The outputs and workspaces that a training or serving loop allocates once."""
    import fp8_linear_layer_gb300 as fp8
    case = s["case"]
    if case["op"] == "norm":
        s["norm"] = {"block": fp8.empty_layernorm, "mx": fp8.empty_mx_layernorm,
                     "tensor": fp8.empty_tensor_layernorm}[case["recipe"]](
                         case["rows"], case["cols"], E4M3, cols_too=case["both"], residual=case["residual"])
    elif case["op"] == "back":
        s["dx"] = torch.empty_like(s["dy"])
        s["dgamma"] = torch.empty(case["cols"], device="cuda")
        s["dbeta"] = torch.empty(case["cols"], device="cuda") if case["beta"] else None
        s["work"] = fp8.layernorm_workspace(case["rows"], case["cols"])


# --------------------------------------------------------------- operators --

def run(s):
    case = s["case"]
    return (OWN if own else PLAIN)[case["op"]](s, case)


def operands(fp8, s, case, fmt):
    kind = {"block": fp8.Fp8Tensor, "mx": fp8.Fp8MxTensor, "tensor": fp8.Fp8TensorScaled}[case["recipe"]]
    return kind(s["a"], s["sa"], fmt), kind(s["b"], s["sb"], E4M3)


def own_gated(s, case):
    import fp8_linear_layer_gb300 as fp8
    call = {"block": fp8.gemm_gated, "mx": fp8.mx_gemm_gated, "tensor": fp8.tensor_gemm_gated}[case["recipe"]]
    out, aux = call(*operands(fp8, s, case, E4M3), s["bias"],
                    fp8.ACT_SILU if case["act"] == "silu" else fp8.ACT_GELU, out=s["out"], aux=s["aux"])
    return [out, aux] if case["aux"] else [out]


def own_dgrad(s, case):
    import fp8_linear_layer_gb300 as fp8
    call = {"block": fp8.gemm_gated_dgrad, "mx": fp8.mx_gemm_gated_dgrad,
            "tensor": fp8.tensor_gemm_gated_dgrad}[case["recipe"]]
    return [call(*operands(fp8, s, case, E5M2), s["z"], fp8.ACT_SILU if case["act"] == "silu" else fp8.ACT_GELU,
                 out=s["out"])]


def values(codes, scale, fmt, recipe):
    rows, k = codes.shape
    v = codes.view(CODE[fmt]).float()
    if recipe == "block":
        return (v.view(rows, k // 128, 128) * scale[:, :rows].t()[:, :, None]).view(rows, k)
    if recipe == "mx":
        return torch.ldexp(v.view(rows, k // 32, 32), exponents(scale, rows, k)[:, :, None]).view(rows, k)
    return v * scale


def activate(z, act):
    """(act(z), act'(z))"""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return z * p, p * (1.0 + z * (1.0 - p))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def plain_gated(s, case):
    z = values(s["a"], s["sa"], E4M3, case["recipe"]) @ values(s["b"], s["sb"], E4M3, case["recipe"]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    n = case["n"]
    y = activate(z[:, :n], case["act"])[0] * z[:, n:]
    return [y.bfloat16(), z.bfloat16()] if case["aux"] else [y.bfloat16()]


def plain_dgrad(s, case):
    d = values(s["a"], s["sa"], E5M2, case["recipe"]) @ values(s["b"], s["sb"], E4M3, case["recipe"]).t()
    n = case["n"]
    z = s["z"].float()
    y, slope = activate(z[:, :n], case["act"])
    return [torch.cat((d * z[:, n:] * slope, d * y), 1).bfloat16()]


def as_codes(t, recipe, rows):
    """An operand's codes and scales as the values that they stand for (views: nothing is computed)."""
    q = t.q.view(CODE[t.fmt])
    return (q, t.scale[:, :rows]) if recipe == "block" else (q, t.sf.view(torch.float8_e8m0fnu)) if recipe == "mx" \
        else (q, t.scale)


def own_norm(s, case):
    import fp8_linear_layer_gb300 as fp8
    recipe = case["recipe"]
    if recipe == "tensor":
        r = fp8.tensor_layernorm_quantize(s["x"], s["gamma"], s["beta"], EPS, E4M3, s["amax"], residual=s["residual"],
                                          out=s["norm"])
    else:
        call = fp8.layernorm_quantize if recipe == "block" else fp8.mx_layernorm_quantize
        r = call(s["x"], s["gamma"], s["beta"], EPS, E4M3, residual=s["residual"], out=s["norm"])
    out = {"mean": r.mean, "rstd": r.rstd, "rows": as_codes(r.rows, recipe, case["rows"])}
    if case["residual"]:
        out["h"] = r.h
    if case["both"]:
        out["cols"] = as_codes(r.cols, recipe, case["cols"])
    if recipe == "tensor":
        out["amax"] = r.amax
    return out


def plain_norm(s, case):
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).bfloat16()
    hf = h.float()
    mean = hf.mean(1)
    c = hf - mean[:, None]
    rstd = torch.rsqrt(c.square().mean(1) + EPS)
    y = c * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    recipe, amax = case["recipe"], s.get("amax")
    out = {"mean": mean, "rstd": rstd, "rows": cast(y, E4M3, recipe, amax)}
    if case["residual"]:
        out["h"] = h
    if case["both"]:
        out["cols"] = cast(y.t().contiguous(), E4M3, recipe, amax)
    if recipe == "tensor":
        out["amax"] = y.abs().amax().view(1)
    return out


def own_back(s, case):
    import fp8_linear_layer_gb300 as fp8
    dx, dgamma, dbeta = fp8.layernorm_backward(s["dy"], s["h"], s["gamma"], s["mean"], s["rstd"],
                                               residual_grad=s["skip"], out=s["dx"], dgamma=s["dgamma"],
                                               dbeta=s["dbeta"], bias=case["beta"], workspace=s["work"])
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta} if case["beta"] else {"dx": dx, "dgamma": dgamma}


def plain_back(s, case):
    dy, xhat = s["dy"].float(), (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    d = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (d - d.mean(1, keepdim=True) - xhat * (d * xhat).mean(1, keepdim=True))
    if s["skip"] is not None:
        dx = dx + s["skip"].float()
    out = {"dx": dx.bfloat16(), "dgamma": (dy * xhat).sum(0)}
    if case["beta"]:
        out["dbeta"] = dy.sum(0)
    return out


# The mask: word i % 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
# 2011) with the seed's halves as key and the counter (i / 4, site, step's halves), for element i of the matrix by rows.
# An element whose word is below p 2^32 is dropped.

def words(n, seed, site, step):
    low = 0xFFFFFFFF
    c = [torch.arange(-(-n // 4), device="cuda"), torch.full((1,), site, device="cuda"), step & low, (step >> 32) & low]
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64 bits, of which the sign bit is the highest
        c = [((b >> 32) & low) ^ c[1] ^ k0, b & low, ((a >> 32) & low) ^ c[3] ^ k1, a & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, 1).view(-1)[:n]


def own_drop(s, case):
    import fp8_linear_layer_gb300 as fp8
    return fp8.dropout(s["x"], case["p"], s["seed"], s["site"], s["step"], residual=s["residual"], out=s["out"])


def plain_drop(s, case):
    rows, cols = case["rows"], case["cols"]
    kept = words(rows * cols, s["seed"], s["site"], s["step"]).view(rows, cols) >= int(case["p"] * 2 ** 32)
    y = torch.where(kept, s["x"].float() * (1.0 / (1.0 - case["p"])), torch.zeros((), device="cuda"))
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.bfloat16()


OWN = {"gated": own_gated, "dgrad": own_dgrad, "norm": own_norm, "back": own_back, "drop": own_drop}
PLAIN = {"gated": plain_gated, "dgrad": plain_dgrad, "norm": plain_norm, "back": plain_back, "drop": plain_drop}


# -------------------------------------------------------------------- work --

def scale_bytes(rows, k, recipe):
    return 4 if recipe == "tensor" else rows * k // 32  # 4 bytes for 128 codes, or 1 for 32


def work(case):
    if case["op"] == "gated":
        m, n, k = case["m"], case["n"], case["k"]
        moved = (m + 2 * n) * k + scale_bytes(m, k, case["recipe"]) + scale_bytes(2 * n, k, case["recipe"])
        return {"bytes": moved + 2 * m * n * (3 if case["aux"] else 1) + (4 * n if case["bias"] else 0),
                "flops": 4 * m * n * k}
    if case["op"] == "dgrad":
        m, n, k = case["m"], case["n"], case["k"]
        moved = (m + n) * k + scale_bytes(m, k, case["recipe"]) + scale_bytes(n, k, case["recipe"])
        return {"bytes": moved + 8 * m * n, "flops": 2 * m * n * k}
    n = case["rows"] * case["cols"]
    if case["op"] == "norm":
        sides = 2 if case["both"] else 1
        moved = n * (2 + (4 if case["residual"] else 0) + sides) + sides * scale_bytes(
            case["rows"], case["cols"], case["recipe"])
        return {"bytes": moved + 8 * case["rows"] + (4 if case["beta"] else 2) * case["cols"], "flops": 10 * n}
    if case["op"] == "back":
        return {"bytes": n * (8 if case["skip"] else 6) + 8 * case["rows"] + (10 if case["beta"] else 6) * case["cols"],
                "flops": 14 * n}
    return {"bytes": n * (6 if case["residual"] else 4), "flops": 3 * n}


# ------------------------------------------------------------------- exact --

def nearest(v, fmt):
    """The nearest values of an fp8 format, saturating, from the format's definition (ties to even)."""
    bits, low = (3, -6) if fmt == E4M3 else (2, -14)
    _, e = torch.frexp(v.abs())
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=low) - bits)
    return (torch.round(v / step) * step).clamp(-FMAX[fmt], FMAX[fmt])


def exact_cast(y, recipe, amax):
    """Codes' values and scales of y [rows][k] in 64 bits."""
    rows, k = y.shape
    if recipe == "tensor":
        scale = amax / 448.0
        return nearest(y / scale, E4M3), scale
    width = 128 if recipe == "block" else 32
    top = torch.stack([c.abs().amax(1) for c in y.split(width, 1)], 1)
    if recipe == "block":
        scale = torch.where(top > 0, top / 448.0, torch.ones_like(top))
        return nearest(y / scale.repeat_interleave(width, 1), E4M3), scale.t().contiguous()
    e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 448.0)) / 448.0))
    q = nearest(y / torch.exp2(e).repeat_interleave(width, 1), E4M3)
    groups = 2 * ((rows + 255) // 256)
    sf = torch.ones((k // 128) * groups * 512, dtype=torch.float64, device=y.device)
    r = torch.arange(rows, device=y.device)[:, None]
    j = torch.arange(k // 32, device=y.device)[None, :]
    sf[((j // 4) * groups + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4] = torch.exp2(e)
    return q, sf


def exact_values(codes, scale, fmt, recipe):
    """An operand's entries in 64 bits, the codes taken apart by their bits."""
    bits, bias = (3, 7) if fmt == E4M3 else (2, 15)
    c = torch.arange(256, device=codes.device)
    m, e = (c & ((1 << bits) - 1)).double(), (c >> bits) & ((1 << (7 - bits)) - 1)
    v = torch.where(e > 0, (1.0 + m / (1 << bits)) * torch.exp2((e - bias).double()),
                    m / (1 << bits) * 2.0 ** (1 - bias)) * (1.0 - 2.0 * (c >> 7).double())
    v = v[codes.long()]
    rows, k = codes.shape
    if recipe == "tensor":
        return v * scale.double()
    if recipe == "block":
        return v * scale[:, :rows].double().t().repeat_interleave(128, 1)
    groups = 2 * ((rows + 255) // 256)
    r = torch.arange(rows, device=codes.device)[:, None]
    j = torch.arange(k // 32, device=codes.device)[None, :]
    e = scale[((j // 4) * groups + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4].double() - 127.0
    return v * torch.exp2(e).repeat_interleave(32, 1)


def exact_gate(z, act):
    """(act(z), act'(z)) in 64 bits, both as forms of the logistic function and its argument's slope."""
    c = 2.0 * math.sqrt(2.0 / math.pi)
    u, du = (z, 1.0) if act == "silu" else (c * z + c * 0.044715 * z ** 3, c + 3.0 * c * 0.044715 * z ** 2)
    up, down = 1.0 / (1.0 + torch.exp(-u)), 1.0 / (1.0 + torch.exp(u))
    return z * up, up + z * du * up * down


def exact_words(n, seed, site, step):
    """The generator's words, its products in halves of 16 bits."""
    low, half = 2 ** 32, 2 ** 16

    def high_low(m, v):
        p0, p1 = (m % half) * v, (m // half) * v  # m v = p0 + p1 2^16, each below 2^48
        return (p1 + p0 // half) // half, ((p1 % half) * half + p0) % low

    i = torch.arange(n, device="cuda")
    x = [i[::4] // 4, torch.full_like(i[::4], site), torch.full_like(i[::4], step % low),
         torch.full_like(i[::4], step // low)]
    for r in range(10):
        key = (seed % low + r * 0x9E3779B9) % low, (seed // low + r * 0xBB67AE85) % low
        (h0, l0), (h1, l1) = high_low(0xD2511F53, x[0]), high_low(0xCD9E8D57, x[2])
        x = [h1 ^ x[1] ^ key[0], l1, h0 ^ x[3] ^ key[1], l0]
    out = torch.empty(len(x[0]) * 4, dtype=torch.int64, device="cuda")
    for j in range(4):
        out[j::4] = x[j]
    return out[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("gated", "dgrad"):
        fmt = E4M3 if case["op"] == "gated" else E5M2
        z = exact_values(s["a"], s["sa"], fmt, case["recipe"]) @ exact_values(
            s["b"], s["sb"], E4M3, case["recipe"]).t()
        n = case["n"]
        if case["op"] == "dgrad":
            g, u = s["z"].double().split(n, 1)
            y, slope = exact_gate(g, case["act"])
            out = torch.empty((case["m"], 2 * n), dtype=torch.float64, device="cuda")
            out[:, :n] = z * slope * u
            out[:, n:] = z * y
            return [out]
        if s["bias"] is not None:
            z += s["bias"].double()
        y = exact_gate(z[:, :n], case["act"])[0] * z[:, n:]
        return [y, z] if case["aux"] else [y]
    if case["op"] == "norm":
        h = s["x"].double() if s["residual"] is None else (s["x"].double() + s["residual"].double()).bfloat16().double()
        mean = h.sum(1) / case["cols"]
        c = h - mean[:, None]
        rstd = 1.0 / torch.sqrt((c * c).sum(1) / case["cols"] + EPS)
        y = s["gamma"].double() * c * rstd[:, None]
        if s["beta"] is not None:
            y += s["beta"].double()
        amax = s["amax"].double() if case["recipe"] == "tensor" else None
        out = {"mean": mean, "rstd": rstd, "rows": exact_cast(y, case["recipe"], amax)}
        if case["residual"]:
            out["h"] = h
        if case["both"]:
            out["cols"] = exact_cast(y.t(), case["recipe"], amax)
        if case["recipe"] == "tensor":
            out["amax"] = y.abs().max().view(1)
        return out
    if case["op"] == "back":
        # through the norm as a function of h: y = gamma (h - m) r + beta, with the m and r that the forward pass kept
        dy, c, r = s["dy"].double(), s["h"].double() - s["mean"].double()[:, None], s["rstd"].double()[:, None]
        out = {"dgamma": (dy * c * r).sum(0)}
        if case["beta"]:
            out["dbeta"] = dy.sum(0)
        dy *= s["gamma"].double()
        dx = (dy - dy.sum(1, keepdim=True) / case["cols"]) * r - c * r ** 3 * ((dy * c).sum(1, keepdim=True)
                                                                                 / case["cols"])
        if s["skip"] is not None:
            dx += s["skip"].double()
        return {"dx": dx, **out}
    rows, cols = case["rows"], case["cols"]
    dropped = exact_words(rows * cols, s["seed"], s["site"], int(s["step"])).view(rows, cols) < math.floor(
        case["p"] * 2.0 ** 32)
    y = (s["x"].double() / (1.0 - case["p"])).masked_fill(dropped, 0.0)
    return y if s["residual"] is None else y + s["residual"].double()
