"""Operators of a decoder layer in 8-bit integers, as they are measured: the norm with the residual's
addition and an output in 8 bits, the quantisation of rows, the product of 8-bit integers, and the gated
pair of projections with its activation.

``run`` computes them in their plain form (elementary torch operations in fp32) or, with ``own`` set,
through the library's entry points. ``exact`` is the definition in fp64.

A row in 8 bits is codes q (int8, -127 .. 127) and one fp32 scale s; an element stands for q * s:
s = max |v| / 127, q = round(v * 127 / max |v|), half to even.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}

# ------------------------------------------------------------------------------------- cases
# norm: `tokens` rows of `width`, x of type `x`, the residual of type `residual` ("" for none);
# `out` names the outputs: "q" (8 bits with scales), "y" (x's type) or both.
# quantize: `tokens` rows of `width` of type `x`.
# linear: `tokens` rows of `width` codes through an [outs][width] weight, result of type `y`;
# gated: through two of them and the activation `act`.


def _norm(name, tokens, width, x="bf16", residual="bf16", out="q"):
    return {"name": name, "kind": "norm", "tokens": tokens, "width": width, "x": x, "residual": residual, "out": out}


def _quant(name, tokens, width, x="bf16"):
    return {"name": name, "kind": "quantize", "tokens": tokens, "width": width, "x": x}


def _linear(name, tokens, width, outs, y="bf16"):
    return {"name": name, "kind": "linear", "tokens": tokens, "width": width, "outs": outs, "y": y}


def _gated(name, tokens, width, outs, y="bf16", act="silu"):
    return {"name": name, "kind": "gated", "tokens": tokens, "width": width, "outs": outs, "y": y, "act": act}


def listed():
    return [
        # one user's token before the 4096-wide block's projections: latency
        _norm("norm_one_token", 1, 4096),
        # prompts of the 8192-wide block, an odd number of tokens, the residual stream in fp32
        _norm("norm_prompts_12289", 12289, 8192, residual="f32"),
        # the gate's outputs of the mixed serving step (64 decode tokens, a chunk of 1024), for the down projection
        _quant("quantize_step_1088", 1088, 11008),
        # a down projection's weight, one scale an output channel: when a model is loaded
        _quant("quantize_weight", 4096, 14336, x="f32"),
        # one user's token through the o projection: latency and 17 MB of weights
        _linear("linear_one_token", 1, 4096, 4096),
        # a batch of 16 through the 8192-wide block's down projection: 235 MB of weights
        _linear("linear_batch_16", 16, 28672, 8192),
        # a prefill chunk through q, k and v side by side (32 + 2 x 8 heads of 128)
        _linear("linear_chunk_320", 320, 4096, 6144),
        # a prompt through the 4096-wide block's down projection
        _linear("linear_prompt_2048", 2048, 14336, 4096),
        # one user's token through gate and up of the 4096-wide block
        _gated("gated_one_token", 1, 4096, 14336),
        # an odd batch, just past what single tokens take
        _gated("gated_batch_61", 61, 4096, 11008),
        # the mixed serving step
        _gated("gated_step_1088", 1088, 4096, 11008),
        # a prompt through gate and up of the 8192-wide block: bound by the tensor cores
        _gated("gated_prompt_4096", 4096, 8192, 28672),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


WIDTHS = [4096, 4096, 8192, 11008, 14336, 2048, 1024, 28672]


def draw(rng):
    kind = rng.choice(["norm", "norm", "quantize", "linear", "linear", "linear", "gated", "gated", "gated"])
    if kind in ("norm", "quantize"):
        width = rng.choice(WIDTHS) if rng.random() < 0.6 else _log(rng, 16, 30000)
        tokens = _log(rng, 1, min(40000, 12289 * 8192 // width))
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        if kind == "quantize":
            c = _quant("", tokens, width, x)
        else:
            c = _norm("", tokens, width, x, rng.choice([x, x, "f32", ""]), rng.choice(["q", "q", "y", "qy"]))
    else:
        width = rng.choice(WIDTHS) if rng.random() < 0.6 else 16 * _log(rng, 2, 1200)
        n = 2 if kind == "gated" else 1
        room = (8192 * 2 * 28672) // (n * width)  # as many weights as the largest listed case
        outs = min(room, rng.choice(WIDTHS) if rng.random() < 0.6 else _log(rng, 8, 30000))
        tokens = _log(rng, 1, max(1, min(6000, 4096 * 8192 * 2 * 28672 // (n * width * outs))))
        y = rng.choice(["bf16", "bf16", "bf16", "f16", "f32"])
        c = (_linear("", tokens, width, outs, y) if kind == "linear" else
             _gated("", tokens, width, outs, y, rng.choice(["silu", "silu", "gelu"])))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------- inputs
def _activations(g, tokens, width):
    """fp32 rows with a few channels that are much larger than the others, as activations have them."""
    x = torch.randn(tokens, width, generator=g, device="cuda")
    big = torch.rand(width, generator=g, device="cuda") < 0.01
    return x.mul_(torch.where(big, 12.0, 1.0))


def _codes(g, rows, width, spread):
    """Codes and scales of rows of normal values: what a quantiser has left of weights or activations."""
    q = torch.empty(rows, width, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    step = max(1, (1 << 27) // width)
    for i in range(0, rows, step):
        v = torch.randn(min(rows, i + step) - i, width, generator=g, device="cuda") * spread
        a = v.abs().amax(1, keepdim=True)
        q[i:i + step], s[i:i + step] = (v * (127.0 / a)).round_().to(torch.int8), a[:, 0] / 127.0
    return q, s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)
    tokens, width = c["tokens"], c["width"]
    s = {"case": dict(c)}
    new = dict(device="cuda")
    if c["kind"] in ("norm", "quantize"):
        t = TYPES[c["x"]]
        s["x"] = _activations(g, tokens, width).to(t)
        if c["kind"] == "norm":
            s["weight"] = (1.0 + 0.1 * torch.randn(width, generator=g, device="cuda")).to(t)
            s["eps"] = 1e-5
            if c["residual"]:
                s["residual"] = (2.0 * torch.randn(tokens, width, generator=g, device="cuda")).to(TYPES[c["residual"]])
                s["residual_out"] = torch.empty_like(s["residual"])
            if "y" in c["out"]:
                s["y"] = torch.empty(tokens, width, dtype=t, **new)
        if c["kind"] == "quantize" or "q" in c["out"]:
            s["q"] = torch.empty(tokens, width, dtype=torch.int8, **new)
            s["scales"] = torch.empty(tokens, **new)
            s["values"] = torch.empty(tokens, width, dtype=torch.bfloat16, **new)
        return s
    x = _activations(g, tokens, width)
    a = x.abs().amax(1, keepdim=True)
    s["x"], s["x_scales"] = (x * (127.0 / a)).round().to(torch.int8), (a[:, 0] / 127.0).contiguous()
    # weights of a size that keeps the outputs near one
    s["w"], s["w_scales"] = _codes(g, c["outs"], width, width ** -0.5)
    if c["kind"] == "gated":
        s["up"], s["up_scales"] = _codes(g, c["outs"], width, width ** -0.5)
    s["y"] = torch.empty(tokens, c["outs"], dtype=TYPES[c["y"]], **new)
    if own:  # the handle, made once when a model is loaded
        from quantized_linear_error_gb300 import spear
        up = dict(up=s["up"], up_scales=s["up_scales"], activation=c["act"]) if c["kind"] == "gated" else {}
        s["layer"] = spear.SpearW8Linear(s["w"], s["w_scales"], max_tokens=tokens, **up)
    return s


# ------------------------------------------------------------------------------------- plain forms
def _quantise(v):
    a = v.abs().amax(1, keepdim=True)
    return torch.round(v * (127.0 / a)), a / 127.0


def _norm_plain(s):
    h, outs = s["x"].float(), []
    if "residual" in s:
        h = h + s["residual"].float()
        outs.append(h.to(s["residual"].dtype))
    v = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    if "y" in s:
        outs.append(v.to(s["x"].dtype))
    if "q" in s:
        q, scale = _quantise(v)
        outs += [scale[:, 0], (q * scale).bfloat16()]
    return outs


def _product(x, x_scales, w, w_scales):
    return (x.float() @ w.float().t()) * x_scales[:, None] * w_scales


def run(state):
    s, c = state, state["case"]
    if own:
        from quantized_linear_error_gb300 import spear
        if c["kind"] in ("linear", "gated"):
            return s["layer"].forward(s["x"], s["x_scales"], s["y"])
        outs = []
        if c["kind"] == "quantize":
            spear.quantize_rows(s["x"], s["q"], s["scales"])
        else:
            spear.rms_norm(s["x"], s["weight"], s["eps"], s.get("residual"), s.get("residual_out"), s.get("y"),
                           s.get("q"), s.get("scales"))
            outs = [s[k] for k in ("residual_out", "y") if k in s]
        if "q" in s:  # what the codes stand for
            outs += [s["scales"], spear.dequantize_rows(s["q"], s["scales"], s["values"])]
        return outs
    if c["kind"] == "norm":
        return _norm_plain(s)
    if c["kind"] == "quantize":
        q, scale = _quantise(s["x"].float())
        return [scale[:, 0], (q * scale).bfloat16()]
    y = _product(s["x"], s["x_scales"], s["w"], s["w_scales"])
    if c["kind"] == "gated":
        if c["act"] == "silu":
            y = y / (1.0 + torch.exp(-y))
        else:
            y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
        y = y * _product(s["x"], s["x_scales"], s["up"], s["up_scales"])
    return y.to(TYPES[c["y"]])


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    t, k = c["tokens"], c["width"]
    if c["kind"] in ("norm", "quantize"):
        # codes and scales out, and what they stand for (bf16) read back from them
        held = t * (k * (1 + 2) + 4)
        if c["kind"] == "quantize":
            return {"bytes": t * k * BYTES[c["x"]] + held, "flops": 5 * t * k}
        b = t * k * BYTES[c["x"]] + k * BYTES[c["x"]]
        b += 2 * t * k * BYTES[c["residual"]] if c["residual"] else 0
        b += t * k * BYTES[c["x"]] if "y" in c["out"] else 0
        return {"bytes": b + (held if "q" in c["out"] else 0), "flops": t * k * (9 if "q" in c["out"] else 5)}
    n = c["outs"] * (2 if c["kind"] == "gated" else 1)
    return {"bytes": n * (k + 4) + t * (k + 4) + t * c["outs"] * BYTES[c["y"]], "flops": 2 * t * n * k}


# ------------------------------------------------------------------------------------- definition in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case

    def held(v):
        top = v.abs().max(1, keepdim=True).values
        scale = top / 127
        return [scale.squeeze(1), (v / scale).round().clamp(-127, 127) * scale]

    if c["kind"] == "quantize":
        return held(s["x"].double())
    if c["kind"] == "norm":
        h, outs = s["x"].double(), []
        if c["residual"]:
            h = h + s["residual"].double()
            outs.append(h)
        rms = (h.square().sum(1, keepdim=True) / c["width"] + s["eps"]).sqrt()
        v = h / rms * s["weight"].double()
        if "y" in c["out"]:
            outs.append(v)
        return outs + (held(v) if "q" in c["out"] else [])
    x = s["x"].double() * s["x_scales"].double()[:, None]
    out = torch.empty(c["tokens"], c["outs"], dtype=torch.float64, device="cuda")
    step = max(1, (1 << 27) // c["width"])
    for i in range(0, c["outs"], step):  # weights expanded to 64 bits a part at a time

        def through(codes, scales):
            return torch.einsum("mk,nk->mn", x, codes[i:i + step].double() * scales[i:i + step].double()[:, None])

        y = through(s["w"], s["w_scales"])
        if c["kind"] == "gated":
            if c["act"] == "silu":
                y = y * torch.sigmoid(y)
            else:
                y = y * (0.5 + 0.5 * torch.tanh((2 / math.pi) ** 0.5 * (y + 0.044715 * y ** 3)))
            y = y * through(s["up"], s["up_scales"])
        out[:, i:i + step] = y
    return out
