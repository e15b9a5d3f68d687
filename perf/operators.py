"""The operators of a training block's dense part, as cases to measure.

A feed-forward block of a sharded training step runs, between the all-gather of
its parameters and the reduce-scatter of their gradients: the residual stream's
RMS norm, two linear layers with bias, activation and residual, and the same
backward, with what the backward pass needs kept in 8 bits.  Every case is one
call of that chain.  ``run`` computes it in elementary torch operations in 32
bits (``own`` false) or through fsdp_layout_aware_gb300 (``own`` true).

8-bit checkpoints: blocks of 32 along a row, a power-of-two scale (one byte,
exponent + 127) and e4m3 codes.  They are returned as the values they stand
for, in bf16, which holds them exactly.
"""

import math

import torch

own = False

EPS = 1e-5
BLOCK = 32
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTS = ("none", "relu", "gelu", "gelu_erf", "silu")
GELU_A = math.sqrt(2.0 / math.pi)
GELU_B = 0.044715

# Widths are those of the framework's workloads (synth/configs.py): 8192 and
# 28672, 5120 and 13824, 2048 and 768, and the uneven group's odd sizes.
# 8192 tokens is a rank's share of a long-context batch.


def listed():
    return [
        # One decoding step's norm: a single row, where only latency counts.
        {"name": "norm, one token", "op": "norm", "rows": 1, "cols": 8192, "dtype": "bf16", "residual": True, "keep": False},
        # A rank's batch through a wide block's norm, the output also kept in 8 bits.
        {"name": "norm, long, kept", "op": "norm", "rows": 16384, "cols": 8192, "dtype": "bf16", "residual": True,
         "keep": True},
        # The backward pass of a norm whose input was kept in 8 bits, the stream's own gradient added.
        {"name": "norm grad, checkpoint", "op": "norm_grad", "rows": 8192, "cols": 5120, "dtype": "bf16",
         "residual": True, "keep": True},
        # A short, odd fp32 batch (evaluation, fine-tuning).
        {"name": "norm grad, ragged", "op": "norm_grad", "rows": 97, "cols": 2047, "dtype": "fp32", "residual": False,
         "keep": False},
        # An activation written as a checkpoint and read back: a whole FFN's inner activation.
        {"name": "checkpoint, long", "op": "store", "rows": 8192, "cols": 13824, "dtype": "bf16"},
        # The activation's gradient from a checkpoint of odd rows.
        {"name": "checkpoint grad, ragged", "op": "load", "rows": 4093, "cols": 4095, "dtype": "bf16", "act": "silu"},
        # One token through a wide block's up projection: the weights are read once.
        {"name": "linear, one token", "op": "linear", "rows": 1, "inner": 8192, "outer": 28672, "act": "silu",
         "bias": True, "residual": True, "keep": "no"},
        # An FFN's up projection in training: bias, gelu, the pre-activation kept in 8 bits.
        {"name": "linear, FFN up, kept", "op": "linear", "rows": 8192, "inner": 5120, "outer": 13824, "act": "gelu",
         "bias": True, "residual": False, "keep": "mx8"},
        # The down projection's input gradient, through the kept pre-activation's derivative.
        {"name": "input grad, FFN down", "op": "grad_input", "rows": 8192, "outer": 5120, "inner": 13824, "act": "gelu",
         "keep": "mx8"},
        # Odd everything: no row starts on a 16-byte boundary.
        {"name": "input grad, ragged", "op": "grad_input", "rows": 1021, "outer": 4095, "inner": 2047, "act": "none",
         "keep": "no"},
        # One expert's share of tokens: a small weight, a long sum.
        {"name": "weight grad, expert", "op": "grad_weight", "rows": 4093, "outer": 768, "inner": 2048, "bias": False,
         "keep": "no"},
        # The largest: a wide block's up projection, its input kept in 8 bits.
        {"name": "weight grad, wide, kept", "op": "grad_weight", "rows": 8192, "outer": 28672, "inner": 8192,
         "bias": True, "keep": "mx8"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of them whole multiples of 64, as real widths are, where that fits."""
    n = _log_int(rng, lo, hi)
    n = max(lo, n // 64 * 64) if n >= 64 and rng.random() < 0.5 else n
    return n - 1 if n == 3072 else n  # a width that no workload of the framework has


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "store", "load", "linear", "linear", "grad_input", "grad_weight"])
    c = {"op": op}
    if op in ("norm", "norm_grad", "store", "load"):
        c["rows"] = _log_int(rng, 1, 16384)
        c["cols"] = _size(rng, 64, 13824 if op in ("store", "load") else 8192)
        c["dtype"] = rng.choice(["bf16", "fp32"])
        if op in ("norm", "norm_grad"):
            c["residual"] = rng.random() < 0.5
            c["keep"] = rng.random() < 0.5
        if op == "load":
            c["act"] = rng.choice(ACTS[1:])
        return c
    c["rows"] = _log_int(rng, 1, 16384)
    c["outer"] = _size(rng, 64, 28672)
    c["inner"] = _size(rng, 64, 28672)
    most = 8192 * 28672 * 8192
    while c["rows"] * c["outer"] * c["inner"] > most:  # no more than the largest listed case
        k = max(("rows", "outer", "inner"), key=lambda n: c[n])
        c[k] = (c[k] + 1) // 2
    if op == "linear":
        c.update(act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                 keep=rng.choice(["no", "bf16", "mx8"]))
    elif op == "grad_input":
        c.update(act=rng.choice(ACTS), keep=rng.choice(["bf16", "mx8"]))
        if c["act"] == "none":
            c["keep"] = "no"
    else:
        c.update(bias=rng.random() < 0.5, keep=rng.choice(["no", "mx8"]))
    return c


# ---------------------------------------------------------------- inputs

def _two_to(e):
    """2^e in fp32 for -127 <= e <= 127, from its bits: a power function may be a rounding off."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).int().view(torch.float32)


def _quantise(v):
    """Codes and scale bytes of fp32 values (rows, cols)."""
    rows, cols = v.shape
    blocks = -(-cols // BLOCK)
    v = torch.nn.functional.pad(v, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    a = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2)
    m, x = torch.frexp(a)  # a = m * 2^x with m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(a > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, -127)).clamp_(min=-127)
    codes = (v * _two_to(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes.view(rows, blocks * BLOCK)[:, :cols].contiguous().view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """fp32 values of codes and scale bytes."""
    cols = codes.shape[1]
    s = _two_to(scales.int() - 127)
    return codes.view(torch.float8_e4m3fn).float() * s.repeat_interleave(BLOCK, 1)[:, :cols]


def _activations(g, rows, cols, dtype):
    """Normal values with a few loud channels, as a residual stream has them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    loud = torch.randint(0, cols, (max(1, cols // 256),), generator=g, device="cuda")
    x[:, loud] *= 20.0
    return x.to(dtype)


def _gradients(g, rows, cols, dtype):
    return (torch.randn(rows, cols, generator=g, device="cuda") * 1e-3).to(dtype)


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    op, rows = case["op"], case["rows"]
    bf = torch.bfloat16
    s = {"case": dict(case)}

    def empty(r, c, dtype):
        return torch.empty(r, c, dtype=dtype, device="cuda")

    if op in ("norm", "norm_grad", "store", "load"):
        cols, t = case["cols"], TYPES[case["dtype"]]
        if op in ("norm", "norm_grad"):
            s["w"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(t)
        if op == "norm":
            s["x"] = _activations(g, rows, cols, t)
            s["r"] = _activations(g, rows, cols, t) if case["residual"] else None
            s["h"] = empty(rows, cols, t) if case["residual"] else None
            s["y"] = empty(rows, cols, t)
            s["rstd"] = torch.empty(rows, device="cuda")
            if case["keep"]:
                s["codes"] = empty(rows, cols, torch.uint8)
                s["scales"] = empty(rows, -(-cols // BLOCK), torch.uint8)
                s["y8"] = empty(rows, cols, bf)
        elif op == "norm_grad":
            h = _activations(g, rows, cols, t)
            s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
            if case["keep"]:
                s["codes"], s["scales"] = _quantise(h.float())
            else:
                s["h"] = h
            s["dy"] = _gradients(g, rows, cols, t)
            s["dres"] = _gradients(g, rows, cols, t) if case["residual"] else None
            s["dx"] = empty(rows, cols, t)
            s["dw"] = torch.empty(cols, dtype=t, device="cuda")
        elif op == "store":
            s["x"] = _activations(g, rows, cols, t)
            s["codes"] = empty(rows, cols, torch.uint8)
            s["scales"] = empty(rows, -(-cols // BLOCK), torch.uint8)
            s["v"] = empty(rows, cols, bf)
        else:
            s["codes"], s["scales"] = _quantise(_activations(g, rows, cols, bf).float())
            s["g"] = _gradients(g, rows, cols, t)
            s["out"] = empty(rows, cols, t)
        return s
    inner, outer = case["inner"], case["outer"]
    if op == "linear":
        s["x"] = torch.randn(rows, inner, generator=g, device="cuda").to(bf)
        s["w"] = (torch.randn(outer, inner, generator=g, device="cuda") / math.sqrt(inner)).to(bf)
        s["b"] = (0.1 * torch.randn(outer, generator=g, device="cuda")).to(bf) if case["bias"] else None
        s["r"] = _activations(g, rows, outer, bf) if case["residual"] else None
        s["y"] = empty(rows, outer, bf)
        if case["keep"] == "bf16":
            s["z"] = empty(rows, outer, bf)
        elif case["keep"] == "mx8":
            s["codes"] = empty(rows, outer, torch.uint8)
            s["scales"] = empty(rows, -(-outer // BLOCK), torch.uint8)
            s["z"] = empty(rows, outer, bf)
    elif op == "grad_input":
        s["dy"] = _gradients(g, rows, outer, bf)
        s["w"] = (torch.randn(outer, inner, generator=g, device="cuda") / math.sqrt(inner)).to(bf)
        if case["keep"] != "no":
            z = torch.randn(rows, inner, generator=g, device="cuda").to(bf)
            if case["keep"] == "mx8":
                s["codes"], s["scales"] = _quantise(z.float())
            else:
                s["z"] = z
        s["dx"] = empty(rows, inner, bf)
    else:
        s["dy"] = _gradients(g, rows, outer, bf)
        x = torch.randn(rows, inner, generator=g, device="cuda").to(bf)
        if case["keep"] == "mx8":
            s["codes"], s["scales"] = _quantise(x.float())
        else:
            s["x"] = x
        s["dw"] = empty(outer, inner, bf)
        s["db"] = torch.empty(outer, dtype=bf, device="cuda") if case["bias"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0.0)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    if name == "gelu_erf":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1.0 + torch.tanh(GELU_A * (z + GELU_B * z * z * z)))


def _act_grad(name, z):
    if name == "relu":
        return (z > 0.0).to(z.dtype)
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if name == "gelu_erf":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    t = torch.tanh(GELU_A * (z + GELU_B * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * GELU_A * (1.0 + 3.0 * GELU_B * z * z)


def _plain(s):
    c = s["case"]
    op = c["op"]
    bf = torch.bfloat16
    if op == "norm":
        t = s["x"].dtype
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        y = h * rstd[:, None] * s["w"].float()
        out = {"y": y.to(t), "rstd": rstd}
        if s["r"] is not None:
            out["h"] = h.to(t)
        if c["keep"]:
            out["y8"] = _values(*_quantise(y)).to(bf)
        return out
    if op == "norm_grad":
        t = s["dy"].dtype
        h = _values(s["codes"], s["scales"]) if c["keep"] else s["h"].float()
        n = h * s["rstd"][:, None]
        dy = s["dy"].float()
        g = dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - n * (g * n).mean(1, keepdim=True))
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return {"dx": dx.to(t), "dw": (dy * n).sum(0).to(t)}
    if op == "store":
        return _values(*_quantise(s["x"].float())).to(bf)
    if op == "load":
        return (s["g"].float() * _act_grad(c["act"], _values(s["codes"], s["scales"]))).to(s["g"].dtype)
    if op == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(c["act"], z)
        if s["r"] is not None:
            y = y + s["r"].float()
        out = {"y": y.to(bf)}
        if c["keep"] == "bf16":
            out["z"] = z.to(bf)
        elif c["keep"] == "mx8":
            out["z"] = _values(*_quantise(z)).to(bf)
        return out
    if op == "grad_input":
        dx = s["dy"].float() @ s["w"].float()
        if c["act"] != "none":
            dx = dx * _act_grad(c["act"], _values(s["codes"], s["scales"]) if c["keep"] == "mx8" else s["z"].float())
        return {"dx": dx.to(bf)}
    x = _values(s["codes"], s["scales"]) if c["keep"] == "mx8" else s["x"].float()
    dy = s["dy"].float()
    out = {"dw": (dy.t() @ x).to(bf)}
    if c["bias"]:
        out["db"] = dy.sum(0).to(bf)
    return out


# ---------------------------------------------------------------- the framework's

def _framework(s):
    import fsdp_layout_aware_gb300 as tide
    c = s["case"]
    op = c["op"]
    kept = tide.Checkpoint8(s["codes"], s["scales"]) if "codes" in s else None
    if op == "norm":
        tide.tide_rms_norm(s["x"], s["w"], EPS, y=s["y"], residual=s["r"], h=s["h"], rstd=s["rstd"], y8=kept)
        out = {"y": s["y"], "rstd": s["rstd"]}
        if s["r"] is not None:
            out["h"] = s["h"]
        if c["keep"]:
            tide.tide_checkpoint_load(kept, s["y8"])
            out["y8"] = s["y8"]
        return out
    if op == "norm_grad":
        tide.tide_rms_norm_backward(s["dy"], kept if c["keep"] else s["h"], s["w"], s["rstd"], s["dx"], dweight=s["dw"],
                                    dres=s["dres"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "store":
        tide.tide_checkpoint_store(s["x"], kept)
        tide.tide_checkpoint_load(kept, s["v"])
        return s["v"]
    if op == "load":
        tide.tide_checkpoint_load(kept, s["out"], act=c["act"], grad=s["g"])
        return s["out"]
    if op == "linear":
        z = kept if c["keep"] == "mx8" else s["z"] if c["keep"] == "bf16" else None
        tide.tide_linear(s["x"], s["w"], s["y"], bias=s["b"], act=c["act"], residual=s["r"], z=z)
        out = {"y": s["y"]}
        if c["keep"] == "mx8":
            tide.tide_checkpoint_load(kept, s["z"])
        if c["keep"] != "no":
            out["z"] = s["z"]
        return out
    if op == "grad_input":
        z = kept if c["keep"] == "mx8" else s["z"] if c["keep"] == "bf16" else None
        tide.tide_linear_grad_input(s["dy"], s["w"], s["dx"], act=c["act"], z=z)
        return {"dx": s["dx"]}
    tide.tide_linear_grad_weight(s["dy"], kept if c["keep"] == "mx8" else s["x"], s["dw"], db=s["db"])
    out = {"dw": s["dw"]}
    if c["bias"]:
        out["db"] = s["db"]
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- floors

def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("norm", "norm_grad", "store", "load"):
        cols = case["cols"]
        n, b = rows * cols, 2 if case["dtype"] == "bf16" else 4
        kept = n + rows * -(-cols // BLOCK)
        if op == "norm":
            bytes_ = n * b * (4 if case["residual"] else 2) + cols * b + rows * 4 + (2 * n if case["keep"] else 0)
            return {"bytes": bytes_, "flops": 6 * n}
        if op == "norm_grad":
            bytes_ = n * b * (3 if case["residual"] else 2) + (kept if case["keep"] else n * b) + 2 * cols * b + rows * 4
            return {"bytes": bytes_, "flops": 10 * n}
        if op == "store":
            return {"bytes": n * (b + 2), "flops": 3 * n}
        return {"bytes": kept + 2 * n * b, "flops": 10 * n}
    inner, outer = case["inner"], case["outer"]
    flops = 2 * rows * inner * outer
    bytes_ = 2 * (rows * inner + inner * outer + rows * outer)

    def kept(cols):
        return rows * cols + rows * -(-cols // BLOCK)

    if op == "linear":
        bytes_ += 2 * outer if case["bias"] else 0
        bytes_ += 2 * rows * outer if case["residual"] else 0
        bytes_ += 2 * rows * outer if case["keep"] != "no" else 0
    elif op == "grad_input":
        bytes_ += kept(inner) if case["keep"] == "mx8" else 2 * rows * inner if case["keep"] == "bf16" else 0
    else:
        bytes_ += kept(inner) - 2 * rows * inner if case["keep"] == "mx8" else 0
        bytes_ += 2 * outer if case["bias"] else 0
    return {"bytes": bytes_, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def _power64(e):
    """2^e in fp64 for whole numbers e held in fp64."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decode64(codes, scales):
    """Values of checkpoint bytes, from the bits of the format."""
    c = codes.long()
    sign = 1.0 - 2.0 * (c >> 7).double()
    ex, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex > 0, (1.0 + man / 8.0) * _power64((ex - 7).double()), man * 2.0 ** -9)
    mag = torch.where((c & 127) == 127, torch.full_like(mag, math.nan), mag)
    s = _power64(scales.double() - 127.0)
    col = torch.arange(codes.shape[1], device=codes.device) // BLOCK
    return sign * mag * s[:, col]


def _nearest64(v):
    """What an 8-bit checkpoint of 64-bit values stands for."""
    rows, cols = v.shape
    col = torch.arange(cols, device=v.device) // BLOCK
    blocks = -(-cols // BLOCK)
    a = torch.zeros(rows, blocks, dtype=torch.float64, device=v.device)
    a.scatter_reduce_(1, col.expand(rows, cols), v.abs(), "amax")
    e = torch.ceil(torch.log2(torch.clamp(a, min=1e-300) / 448.0))
    e = torch.where(a > 448.0 * _power64(e), e + 1, e)
    e = torch.where(a <= 448.0 * _power64(e - 1), e - 1, e)
    s = _power64(torch.clamp(e, min=-127.0))[:, col]
    q = v / s
    step = _power64(torch.clamp(torch.floor(torch.log2(torch.clamp(q.abs(), min=1e-300))), min=-6.0) - 3.0)
    return torch.round(q / step) * step * s


def _act64(name, z, grad):
    z = z.double()
    if name == "none":
        return torch.ones_like(z) if grad else z
    if name == "relu":
        return torch.where(z > 0, torch.ones_like(z) if grad else z, torch.zeros_like(z))
    if name == "silu":
        p = torch.sigmoid(z)
        return p + z * p * (1 - p) if grad else z * p
    if name == "gelu_erf":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi) if grad else z * cdf
    p = torch.sigmoid(2 * GELU_A * (z + GELU_B * z ** 3))
    return p + z * p * (1 - p) * 2 * GELU_A * (1 + 3 * GELU_B * z ** 2) if grad else z * p


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.dtype in (torch.bfloat16, torch.float32) else v)
         for k, v in s.items()}
    kept_in = op in ("norm_grad", "load", "grad_input", "grad_weight") and "codes" in s
    kept = _decode64(s["codes"], s["scales"]) if kept_in else None
    if op == "norm":
        h = d["x"] if d["r"] is None else d["x"] + d["r"]
        rstd = (h.square().sum(1) / h.shape[1] + EPS) ** -0.5
        y = h * rstd.unsqueeze(1) * d["w"]
        out = {"y": y, "rstd": rstd}
        if d["r"] is not None:
            out["h"] = h
        if case["keep"]:  # what is kept, not its nearest code: where a value lies between two codes, either is right
            out["y8"] = y
        return out
    if op == "norm_grad":
        n = (kept if kept_in else d["h"]) * d["rstd"].unsqueeze(1)
        g = d["dy"] * d["w"]
        dx = (g - n * torch.einsum("tc,tc->t", g, n).unsqueeze(1) / g.shape[1]) * d["rstd"].unsqueeze(1)
        return {"dx": dx if d["dres"] is None else dx + d["dres"], "dw": torch.einsum("tc,tc->c", d["dy"], n)}
    if op == "store":
        return _nearest64(d["x"])
    if op == "load":
        return d["g"] * _act64(case["act"], kept, True)
    if op == "linear":
        z = torch.einsum("ti,oi->to", d["x"], d["w"])
        z = z if d["b"] is None else z + d["b"]
        y = _act64(case["act"], z, False)
        out = {"y": y if d["r"] is None else y + d["r"]}
        if case["keep"] != "no":
            out["z"] = z  # for 8 bits as for y8 above
        return out
    if op == "grad_input":
        dx = torch.einsum("to,oi->ti", d["dy"], d["w"])
        return {"dx": dx * _act64(case["act"], kept if kept_in else d["z"], True) if case["act"] != "none" else dx}
    out = {"dw": torch.einsum("to,ti->oi", d["dy"], kept if kept_in else d["x"])}
    if case["bias"]:
        out["db"] = torch.einsum("to->o", d["dy"])
    return out
