"""The 8-bit operators of the DoRA layer, as cases to measure.

Serving: ``rms_norm_i8`` (residual addition, root-mean-square norm, int8 codes
with one scale a token; ``norm`` false: the codes of the rows as they are) makes
the input of ``linear_i8`` (int8 product with a scale for each token and each
channel, the adapter's branch and the magnitude beside it).

Training: ``compose_fwd`` and ``fused_linear`` keep z = (base - b) + s * lora,
all that the backward needs of the two activations, as int8 codes with a scale
for every 128 columns of a token; ``compose_bwd`` reads them.

Codes are the nearest integers (ties to even) of 127 * v / max|v|; outputs give
the values codes * scale.  ``run`` computes the plain form in elementary torch
operations, or, where ``own`` is true, makes the library's calls.
"""

from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
BLOCK = 128  # columns that share a scale in a checkpoint


def listed():
    return [
        # one decoded token before a projection: a launch's latency
        {"name": "norm_token", "op": "rms_norm_i8", "tokens": 1, "d": 8192, "dtype": "bf16", "norm": True,
         "residual": True, "want_y": False},
        # a prompt; the bf16 rows go to the adapter's branch
        {"name": "norm_prompt", "op": "rms_norm_i8", "tokens": 8192, "d": 8192, "dtype": "bf16", "norm": True,
         "residual": True, "want_y": True},
        # one decoded token through the 8192 x 8192 module at rank 384
        {"name": "i8_token", "op": "linear_i8", "tokens": 1, "d_in": 8192, "d_out": 8192, "r": 384, "bias": False},
        # an odd batch of decoded tokens through the MLP up-projection of a ~32B decoder
        {"name": "i8_batch", "op": "linear_i8", "tokens": 33, "d_in": 5120, "d_out": 27648, "r": 384, "bias": True},
        # a ragged prompt through a layer without an adapter
        {"name": "i8_plain", "op": "linear_i8", "tokens": 1000, "d_in": 4096, "d_out": 4096, "r": 0, "bias": True},
        # a long prompt through the 8192 x 8192 module
        {"name": "i8_prompt", "op": "linear_i8", "tokens": 8192, "d_in": 8192, "d_out": 8192, "r": 384,
         "bias": False},
        # a small fp32 module with a bias and an odd width
        {"name": "ckpt_fwd_f32", "op": "compose_fwd", "tokens": 257, "d_out": 4099, "dtype": "f32", "bias": True},
        # a training step's tokens through the 8192 x 8192 module
        {"name": "ckpt_fwd", "op": "compose_fwd", "tokens": 8192, "d_out": 8192, "dtype": "bf16", "bias": False},
        {"name": "ckpt_bwd_f32", "op": "compose_bwd", "tokens": 257, "d_out": 4099, "dtype": "f32"},
        {"name": "ckpt_bwd", "op": "compose_bwd", "tokens": 8192, "d_out": 8192, "dtype": "bf16"},
        # the 4096 x 4096 module at rank 64 with a bias, a ragged batch
        {"name": "fused_small", "op": "fused_linear", "tokens": 1000, "d_in": 4096, "d_out": 4096, "r": 64,
         "bias": True},
        # the 8192 x 8192 module at rank 384, a training step's tokens
        {"name": "fused_large", "op": "fused_linear", "tokens": 8192, "d_in": 8192, "d_out": 8192, "r": 384,
         "bias": False},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["rms_norm_i8", "linear_i8", "linear_i8", "compose_fwd", "compose_bwd", "fused_linear"])
    s = rng.choice([0.5, 2.0, 0.35])
    if op == "rms_norm_i8":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return {"op": op, "tokens": _log(rng, 1, 4096), "d": _log(rng, 512, 8192, 8 if dtype == "bf16" else 1),
                "dtype": dtype, "norm": rng.random() < 0.75, "residual": rng.random() < 0.5,
                "want_y": rng.random() < 0.5}
    if op == "linear_i8":
        return {"op": op, "tokens": _log(rng, 1, 8192), "d_in": _log(rng, 512, 8192, 16),
                "d_out": _log(rng, 512, 8192, 8), "r": rng.choice([0, _log(rng, 8, 384, 8)]),
                "bias": rng.random() < 0.5, "s": s}
    if op in ("compose_fwd", "compose_bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        case = {"op": op, "tokens": _log(rng, 1, 8192 if dtype == "bf16" else 4096),
                "d_out": _log(rng, 512, 8192, 8 if dtype == "bf16" else 1), "dtype": dtype, "s": s}
        if op == "compose_fwd":
            case["bias"] = rng.random() < 0.5
        return case
    return {"op": op, "tokens": _log(rng, 64, 8192), "d_in": _log(rng, 512, 8192, 8),
            "d_out": _log(rng, 512, 8192, 8), "r": _log(rng, 8, 384, 8), "bias": rng.random() < 0.5, "s": s}


# ------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda")

    def uniform(self, *shape):
        return torch.rand(*shape, generator=self.g, device="cuda")


def _codes(v, block):
    """(codes as floats [rows, blocks, block], scale [rows, blocks]) of fp32 rows, the last block padded with zeros."""
    rows, cols = v.shape
    blocks = -(-cols // block)
    v = torch.nn.functional.pad(v, (0, blocks * block - cols)).view(rows, blocks, block)
    top = v.abs().amax(dim=2)
    ratio = v.double() * 127.0 / torch.where(top > 0, top, torch.ones_like(top)).double().unsqueeze(2)
    return ratio.round(), top / 127.0


def _values(codes, scale, cols):
    rows = codes.shape[0]
    return (codes.float() * scale.unsqueeze(2)).reshape(rows, -1)[:, :cols]


def _activations(d, tokens, width):
    """Rows as a layer sees them: some channels are much larger than the others, and so are some tokens."""
    return d.normal(tokens, width) * torch.exp(0.5 * d.normal(width)) * torch.exp(0.3 * d.normal(tokens, 1))


def _module(d, d_in, d_out, r):
    """W, A and B of an adapted module."""
    w = (0.015 * d.normal(d_out, d_in)).to(torch.bfloat16)
    a = ((2.0 * d.uniform(r, d_in) - 1.0) / math.sqrt(d_in)).to(torch.bfloat16)
    b = (0.002 * d.normal(d_out, r)).to(torch.bfloat16)
    return w, a, b


def _magnitudes(d, w, a, b, s):
    """The magnitude m around the base weight's row norm, and n = ||W + s B A||."""
    m = w.norm(dim=1) * (1.0 + 5e-4 * d.normal(w.shape[0]))
    return m, (w + s * (b.float() @ a.float())).norm(dim=1)


def prepare(case, seed):
    d = _Draws(seed)
    op, dt = case["op"], _dtype(case)
    st = {"case": case, "s": case.get("s", 0.5)}
    if op == "rms_norm_i8":
        st["x"] = _activations(d, case["tokens"], case["d"]).to(dt)
        st["residual"] = _activations(d, case["tokens"], case["d"]).to(dt) if case["residual"] else None
        st["weight"] = (1.0 + 0.2 * d.normal(case["d"])).to(dt)
    elif op == "linear_i8":
        w, a, b = _module(d, case["d_in"], case["d_out"], case["r"])
        x = _activations(d, case["tokens"], case["d_in"]).to(dt)
        xq, xs = _codes(x.float(), case["d_in"])
        wq, ws = _codes(w.float(), case["d_in"])
        st["m"], st["n"] = _magnitudes(d, wq[:, 0].float() * ws, a, b, st["s"])
        st["x_q"], st["x_scale"] = xq[:, 0].to(torch.int8), xs[:, 0].contiguous()
        st["w_q"], st["w_scale"] = wq[:, 0].to(torch.int8), ws[:, 0].contiguous()
        st["x"], st["a"], st["b"] = x, a, b
        st["bias"] = (0.1 * d.normal(case["d_out"])).to(dt) if case["bias"] else None
    elif op == "fused_linear":
        w, a, b = _module(d, case["d_in"], case["d_out"], case["r"])
        st["m"], st["n"] = _magnitudes(d, w.float(), a, b, st["s"])
        st["x"] = _activations(d, case["tokens"], case["d_in"]).to(dt)
        st["w"], st["a"], st["b"] = w, a, b
        st["bias"] = (0.1 * d.normal(case["d_out"])).to(dt) if case["bias"] else None
    else:
        tokens, width = case["tokens"], case["d_out"]
        base = _activations(d, tokens, width).to(dt)
        lora = (0.1 * _activations(d, tokens, width)).to(dt)
        st["m"] = 1.5 + 0.1 * d.normal(width)
        st["n"] = st["m"] / (1.0 + 5e-4 * d.normal(width))
        if op == "compose_fwd":
            st["base"], st["lora"] = base, lora
            st["bias"] = (0.1 * d.normal(width)).to(dt) if case["bias"] else None
        else:  # what a forward has kept
            codes, scale = _codes(base.float() + st["s"] * lora.float(), BLOCK)
            st["z8"] = codes.reshape(tokens, -1)[:, :width].to(torch.int8).contiguous()
            st["z_scale"] = scale.contiguous()
            st["dy"] = d.normal(tokens, width).to(dt)
    return st


# --------------------------------------------------------------------- run
def run(st):
    op = st["case"]["op"]
    return globals()[("_own_" if own else "_plain_") + op](st)


def _plain_rms_norm_i8(st):
    x, dt = st["x"], st["x"].dtype
    out = {}
    h = x
    if st["residual"] is not None:
        h = out["h"] = (x.float() + st["residual"].float()).to(dt)
    hf = h.float()
    if st["case"]["norm"]:
        v = hf * st["weight"].float()
        rstd = torch.rsqrt(hf.square().mean(dim=1, keepdim=True) + EPS)
        if st["case"]["want_y"]:
            out["y"] = (v * rstd).to(dt)
    else:
        v, rstd = hf, torch.ones_like(hf[:, :1])
    codes, scale = _codes(v, v.shape[1])
    scale = scale * rstd
    out["value"], out["scale"] = _values(codes, scale, v.shape[1]).to(dt), scale[:, 0]
    return out


def _own_rms_norm_i8(st):
    from factored_weight_norm_b200 import dora as D

    out = {}
    if st["case"]["norm"]:
        q, scale, h, y = D.dora_rms_norm_i8(st["x"], st["weight"], EPS, residual=st["residual"],
                                            want_y=st["case"]["want_y"])
        if y is not None:
            out["y"] = y
    else:
        q, scale, h = D.dora_quantize_rows_i8(st["x"], residual=st["residual"])
    if h is not None:
        out["h"] = h
    out["value"], out["scale"] = D.dora_dequantize_i8(q, scale, dtype=st["x"].dtype), scale
    return out


def _plain_linear_i8(st):
    z = st["x_q"].float() @ st["w_q"].float().t() * st["x_scale"].unsqueeze(1) * st["w_scale"]
    if st["case"]["r"]:
        z = z + st["s"] * (st["x"].float() @ st["a"].float().t() @ st["b"].float().t())
    y = z * (st["m"] / st["n"])
    if st["bias"] is not None:
        y = y + st["bias"].float()
    return y.to(torch.bfloat16)


def _own_linear_i8(st):
    from factored_weight_norm_b200 import dora as D

    if st["case"]["r"]:
        return D.dora_linear_i8_fwd(st["x_q"], st["x_scale"], st["w_q"], st["w_scale"], x=st["x"], A=st["a"],
                                    B=st["b"], m=st["m"], n=st["n"], s=st["s"], bias=st["bias"])
    return D.dora_linear_i8_fwd(st["x_q"], st["x_scale"], st["w_q"], st["w_scale"], m=st["m"], n=st["n"],
                                bias=st["bias"])


def _kept(z, dt):
    codes, scale = _codes(z, BLOCK)
    return _values(codes, scale, z.shape[1]).to(dt), scale


def _plain_compose_fwd(st):
    base, lora, m, n, dt = st["base"].float(), st["lora"].float(), st["m"], st["n"], st["base"].dtype
    inner = base if st["bias"] is None else base - st["bias"].float()
    y = base + ((m - n) / n * inner + m / n * st["s"] * lora)
    z, scale = _kept(inner + st["s"] * lora, dt)
    return {"y": y.to(dt), "z": z, "z_scale": scale}


def _own_compose_fwd(st):
    from factored_weight_norm_b200 import dora as D

    y, z8, scale = D.dora_compose_fwd_ckpt8(st["base"], st["lora"], st["m"], st["n"], st["s"], bias=st["bias"])
    return {"y": y, "z": D.dora_dequantize_i8(z8, scale, dtype=y.dtype), "z_scale": scale}


def _plain_compose_bwd(st):
    dy, n = st["dy"].float(), st["n"]
    z = st["z8"].float() * st["z_scale"].repeat_interleave(BLOCK, dim=1)[:, :dy.shape[1]]
    d_base = dy * (st["m"] / n)
    return {"d_base": d_base.to(st["dy"].dtype), "d_lora": (st["s"] * d_base).to(st["dy"].dtype),
            "d_m": (dy * z).sum(dim=0) / n}


def _own_compose_bwd(st):
    from factored_weight_norm_b200 import dora as D

    d_base, d_lora, d_m = D.dora_compose_bwd_ckpt8(st["dy"], st["z8"], st["z_scale"], st["m"], st["n"], st["s"])
    return {"d_base": d_base, "d_lora": d_lora, "d_m": d_m}


def _plain_fused_linear(st):
    x = st["x"].float()
    z = x @ st["w"].float().t() + st["s"] * (x @ st["a"].float().t() @ st["b"].float().t())
    y = z * (st["m"] / st["n"])
    if st["bias"] is not None:
        y = y + st["bias"].float()
    kept, scale = _kept(z, torch.bfloat16)
    return {"y": y.to(torch.bfloat16), "z": kept, "z_scale": scale}


def _own_fused_linear(st):
    from factored_weight_norm_b200 import dora as D

    y, z8, scale = D.dora_fused_linear_fwd_ckpt8(st["x"], st["w"], st["a"], st["b"], st["m"], st["n"], st["s"],
                                                 bias=st["bias"])
    return {"y": y, "z": D.dora_dequantize_i8(z8, scale, dtype=y.dtype), "z_scale": scale}


# -------------------------------------------------------------------- work
def work(case):
    op, t = case["op"], case["tokens"]
    e = 4 if case.get("dtype") == "f32" else 2
    if op == "rms_norm_i8":
        y = case["norm"] and case["want_y"]
        size = t * case["d"]
        # x, residual, h, y and the values; the weight; the scales
        return {"bytes": size * e * (2 + 2 * case["residual"] + y) + case["d"] * e * case["norm"] + 4 * t,
                "flops": 6 * size}
    if op in ("linear_i8", "fused_linear"):
        d_in, d_out, r = case["d_in"], case["d_out"], case["r"]
        flops = 2 * t * (d_in * d_out + r * (d_in + d_out))
        sides = 2 * r * (d_in + d_out) + 8 * d_out + 2 * d_out * case["bias"]
        if op == "linear_i8":
            rows = t * (d_in + 4 + (2 * d_in if r else 0))
            return {"bytes": rows + d_out * (d_in + 4) + sides + 2 * t * d_out, "flops": flops}
        return {"bytes": 2 * t * d_in + 2 * d_in * d_out + sides + t * (4 * d_out + 4 * -(-d_out // BLOCK)),
                "flops": flops}
    width = case["d_out"]
    size, scales = t * width, 4 * t * -(-width // BLOCK)
    if op == "compose_fwd":  # base, lora; y, the values
        return {"bytes": 4 * e * size + scales + 8 * width + e * width * case["bias"], "flops": 9 * size}
    return {"bytes": (3 * e + 1) * size + scales + 12 * width, "flops": 5 * size}  # dy, z8; d_base, d_lora


# ------------------------------------------------------------------- exact
def _nearest(v, width):
    """The values that 8 bits keep of fp64 rows, and their scales: each stretch of `width` columns by itself."""
    short = -v.shape[1] % width
    parts = torch.cat([v, v.new_zeros(v.shape[0], short)], dim=1).unflatten(1, (-1, width))
    top = parts.abs().max(dim=2, keepdim=True).values
    unit = top / 127
    kept = torch.where(top > 0, torch.round(127 * parts / top), 0 * parts) * unit
    return kept.flatten(1)[:, : v.shape[1]], unit[:, :, 0]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    if op == "rms_norm_i8":
        out, h = {}, f["x"]
        if case["residual"]:
            out["h"] = f["x"] + f["residual"]
            h = out["h"].to(st["x"].dtype).double()  # the norm is of the rows as they are stored
        scaled = h
        if case["norm"]:
            scaled = h / (h.pow(2).mean(dim=1) + EPS).sqrt().unsqueeze(1) * f["weight"]
            if case["want_y"]:
                out["y"] = scaled
        if case["norm"]:  # the codes do not depend on the row's norm: take them before it rounds
            kept, unit = _nearest(h * f["weight"], case["d"])
            root = (h.pow(2).mean(dim=1, keepdim=True) + EPS).sqrt()
            out["value"], out["scale"] = kept / root, (unit / root)[:, 0]
        else:
            out["value"], unit = _nearest(scaled, case["d"])
            out["scale"] = unit[:, 0]
        return out
    g = f["m"] / f["n"]
    if op == "linear_i8":
        z = torch.einsum("ti,oi->to", f["x_q"], f["w_q"]) * torch.outer(f["x_scale"], f["w_scale"])
        if case["r"]:
            z += f["s"] * torch.einsum("tr,or->to", torch.einsum("ti,ri->tr", f["x"], f["a"]), f["b"])
        return g * z + (f["bias"] if case["bias"] else 0.0)
    if op == "fused_linear":
        z = torch.einsum("ti,oi->to", f["x"], f["w"] + f["s"] * torch.einsum("or,ri->oi", f["b"], f["a"]))
        kept, unit = _nearest(z, BLOCK)
        return {"y": g * z + (f["bias"] if case["bias"] else 0.0), "z": kept, "z_scale": unit}
    if op == "compose_fwd":
        shift = f["bias"] if case["bias"] else 0.0
        z = f["base"] - shift + f["s"] * f["lora"]
        kept, unit = _nearest(z, BLOCK)
        return {"y": g * z + shift, "z": kept, "z_scale": unit}
    column = torch.arange(case["d_out"], device=f["dy"].device) // BLOCK
    z = f["z8"] * f["z_scale"][:, column]
    return {"d_base": g * f["dy"], "d_lora": f["s"] * g * f["dy"], "d_m": torch.einsum("to,to->o", f["dy"], z) / f["n"]}
