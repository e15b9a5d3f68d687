"""The operators at the two ends of a language model's training step, as cases to measure.

Around the blocks of a sharded training step stand the token embedding, the log
probabilities of the batch's tokens (the loss), the gradients of both, and,
once the gradients are reduced, their global norm and the clipping by it.
Every case is one such step.  ``run`` computes it in elementary torch
operations in 32 bits (``own`` false) or through fsdp_layout_aware_gb300
(``own`` true).

  embedding     out[t] = scale * weight[token t]; a token outside the vocabulary
                (padding) gives zeros, and adds to no gradient
  its gradient  dweight[v] = scale * sum of dy[t] over the t with token v, for every v
  log probs     z = scale * logits; lse = log sum exp z; logp = z[target] - lse, 0 for a
                target outside the vocabulary; entropy = -sum p log p; the `top`
                largest logits' tokens (ties: the lowest) and log probabilities
  its gradient  dlogits = scale * (dlogp * (onehot - p) - dentropy * p * (log p + entropy))
  norm, clip    norm = the square root of the sum of all tensors' squares;
                out = x * min(1, most / (norm + eps))

A row of logits that are all -inf has lse and log probabilities -inf, entropy
0 and no gradient.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
INDEX = {"i32": torch.int32, "i64": torch.int64}
CLIP_EPS = 1e-6
GAP = 8  # elements between the tensors of a list that share a buffer, at least

# Widths are those of the framework's workloads (synth/configs.py): 8192, 5120, 2048, and the uneven group's odd sizes;
# vocabularies of 32000 and 131072 and odd ones are generic.  The wide block's shards are its 351,288,320 parameters
# over 64 ranks, 5,488,880 each; 391 tensors are an expert layer's.


def listed():
    return [
        # One decoding step's lookup: a single row, where only latency counts.
        {"name": "embed, one token", "op": "embed", "tokens": 1, "vocab": 32000, "cols": 8192, "dtype": "bf16",
         "index": "i64", "scale": 1.0, "pad": 0.0, "hot": 0.0},
        # A rank's batch of long sequences into a wide model, rows scaled by the root of the width.
        {"name": "embed, long", "op": "embed", "tokens": 16384, "vocab": 131072, "cols": 8192, "dtype": "bf16",
         "index": "i64", "scale": 90.50966799187809, "pad": 0.0, "hot": 0.0},
        # The same batch's gradient: a dense one, as the reduce-scatter reads it.
        {"name": "embed grad, long", "op": "embed_grad", "tokens": 16384, "vocab": 131072, "cols": 8192, "dtype": "bf16",
         "index": "i64", "scale": 90.50966799187809, "pad": 0.0, "hot": 0.0},
        # Fine-tuning of a small vocabulary on padded sequences, one separator token in a third of the places, odd rows.
        {"name": "embed grad, ragged, padded", "op": "embed_grad", "tokens": 4093, "vocab": 4999, "cols": 4095,
         "dtype": "fp32", "index": "i32", "scale": 1.0, "pad": 0.3, "hot": 0.3},
        # One generated token's log probability, entropy and 20 alternatives.
        {"name": "log probs, one token", "op": "log_probs", "rows": 1, "vocab": 131072, "dtype": "bf16", "index": "i64",
         "scale": 1.0, "entropy": True, "top": 20, "masked": False, "ignored": 0.0},
        # Scoring of whole sequences with alternatives, as distillation and evaluation ask for them.
        {"name": "log probs, long, top", "op": "log_probs", "rows": 4096, "vocab": 131072, "dtype": "bf16", "index": "i64",
         "scale": 1.0, "entropy": True, "top": 20, "masked": False, "ignored": 0.05},
        # Constrained decoding at a temperature: most tokens masked out, an odd fp32 vocabulary.
        {"name": "log probs, ragged, masked", "op": "log_probs", "rows": 1021, "vocab": 50001, "dtype": "fp32",
         "index": "i32", "scale": 1.4285714285714286, "entropy": False, "top": 5, "masked": True, "ignored": 0.1},
        # The largest: the loss's gradient for a rank's batch, an entropy term with it.
        {"name": "log probs grad, long", "op": "log_probs_grad", "rows": 8192, "vocab": 131072, "dtype": "bf16",
         "index": "i64", "scale": 1.0, "entropy": True, "masked": False, "ignored": 0.05},
        # A short, odd batch: no row starts where the one before it did within a 16-byte word.
        {"name": "log probs grad, ragged", "op": "log_probs_grad", "rows": 97, "vocab": 4999, "dtype": "bf16",
         "index": "i32", "scale": 1.0, "entropy": False, "masked": True, "ignored": 0.3},
        # The norm of a small adapter's gradients.
        {"name": "norm, small", "op": "norm", "tensors": 12, "total": 98304, "dtype": "bf16", "even": True},
        # A wide block's reduced shards on all of 64 ranks: norm, then clipping.
        {"name": "clip, a group's shards", "op": "clip", "tensors": 64, "total": 351288320, "dtype": "fp32", "even": True,
         "most": 0.5},
        # An expert layer's tensors of all sizes and alignments, some bf16 and some fp32.
        {"name": "clip, ragged", "op": "clip", "tensors": 391, "total": 20000003, "dtype": "both", "even": False,
         "most": 0.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; half of them whole multiples of 64, as real widths are, where that fits."""
    n = _log_int(rng, lo, hi)
    return max(lo, n // 64 * 64) if n >= 64 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "log_probs", "log_probs", "log_probs_grad", "norm", "clip"])
    c = {"op": op}
    if op in ("embed", "embed_grad"):
        c["tokens"] = _log_int(rng, 1, 32768)
        c["vocab"] = _size(rng, 64, 131072)
        c["cols"] = _size(rng, 64, 8192)
        c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        c["index"] = rng.choice(["i32", "i64"])
        c["scale"] = rng.choice([1.0, math.sqrt(c["cols"])])
        c["pad"] = rng.choice([0.0, 0.0, 0.1, 0.5])
        c["hot"] = rng.choice([0.0, 0.0, 0.1, 0.4])
        return c
    if op in ("log_probs", "log_probs_grad"):
        c["rows"] = _log_int(rng, 1, 8192)
        c["vocab"] = _size(rng, 64, 131072)
        c["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
        while c["rows"] * c["vocab"] > 1 << (29 if op == "log_probs" else 30) - (c["dtype"] == "fp32"):
            c["rows"] = (c["rows"] + 1) // 2
        c["index"] = rng.choice(["i32", "i64"])
        c["scale"] = rng.choice([1.0, 1.0, 1.25, 0.7])
        c["entropy"] = rng.random() < 0.5
        c["masked"] = rng.random() < 0.25
        c["ignored"] = rng.choice([0.0, 0.05, 0.4])
        if op == "log_probs":
            c["top"] = rng.choice([0, 0, 1, 5, 20])
        return c
    c["tensors"] = _log_int(rng, 1, 2000)
    c["dtype"] = rng.choice(["bf16", "fp32", "both"])
    c["total"] = max(c["tensors"], _log_int(rng, 1000, 340000000))
    c["even"] = rng.random() < 0.5
    if op == "clip":
        c["most"] = rng.choice([0.1, 1.0, 1000000.0])
    return c


# ---------------------------------------------------------------- inputs

def _spread(case):
    """[(type, first element in its buffer, elements)] of a list of tensors, and the buffers' lengths: the case's alone.
    Even lists are equal tensors on 128-byte boundaries, others of sizes over a factor of a thousand at odd places."""
    n, total = case["tensors"], case["total"]
    if case["even"]:
        sizes = [max(1, total // n)] * n
    else:
        u = [math.exp(6.9 * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(n)]
        rest, whole, sizes = max(0, total - n), sum(u), []
        for v in u:
            sizes.append(1 + int(rest * (v / whole)))
    places, ends = [], {"bf16": 0, "fp32": 0}
    for i, k in enumerate(sizes):
        t = case["dtype"] if case["dtype"] != "both" else ("bf16", "fp32")[i % 2]
        at = ends[t] + (i % 5 if not case["even"] else 0)
        places.append((t, at, k))
        ends[t] = -(-(at + k + GAP) // 64) * 64 if case["even"] else at + k + GAP
    return places, ends


def _tokens(case, g):
    """Token ids, the low ones frequent (the r-th about 1/r of the first), `hot` of them one id, `pad` of them -1."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(vocab + 1)).long() - 1).clamp_(0, vocab - 1)
    t = torch.where(torch.rand(n, generator=g, device="cuda") < case["hot"], vocab // 3, t)
    t = torch.where(torch.rand(n, generator=g, device="cuda") < case["pad"], -1, t)
    return t.to(INDEX[case["index"]])


def _logits(case, g, targets):
    """A model's logits: the target far up in two rows of three; where masked, a tenth of the tokens is allowed (the target
    among them) and, of four rows and more, one allows none."""
    rows, vocab = case["rows"], case["vocab"]
    z = torch.randn(rows, vocab, generator=g, device="cuda") * 2.5
    at = targets.long().clamp(0, vocab - 1)[:, None]
    z.scatter_add_(1, at, torch.where(torch.rand(rows, 1, generator=g, device="cuda") < 0.67, 9.0, 0.0))
    if case["masked"]:
        shut = torch.rand(rows, vocab, generator=g, device="cuda") < 0.9
        shut.scatter_(1, at, False)
        if rows >= 4:
            shut[1] = True
        z.masked_fill_(shut, -math.inf)
    return z.to(TYPES[case["dtype"]])


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    if op in ("embed", "embed_grad"):
        n, vocab, cols, t = case["tokens"], case["vocab"], case["cols"], TYPES[case["dtype"]]
        s["tokens"] = _tokens(case, g)
        if op == "embed":
            s["w"] = empty(vocab, cols, dtype=t).normal_(0.0, 0.02, generator=g)
            s["out"] = empty(n, cols, dtype=t)
        else:
            s["dy"] = empty(n, cols, dtype=t).normal_(0.0, 1e-3, generator=g)
            s["dw"] = empty(vocab, cols, dtype=t)
    elif op in ("log_probs", "log_probs_grad"):
        rows, vocab, t = case["rows"], case["vocab"], TYPES[case["dtype"]]
        targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        s["logits"] = _logits(case, g, targets)
        targets = torch.where(torch.rand(rows, generator=g, device="cuda") < case["ignored"], -1, targets)
        s["targets"] = targets.to(INDEX[case["index"]])
        if op == "log_probs":
            s["logp"], s["lse"] = empty(rows), empty(rows)
            s["entropy"] = empty(rows) if case["entropy"] else None
            if case["top"]:
                s["top_logp"], s["top_tokens"] = empty(rows, case["top"]), empty(rows, case["top"], dtype=torch.int32)
        else:
            s["lse"], log_s, m = _lse(s["logits"], case["scale"])
            s["dlogp"] = torch.randn(rows, generator=g, device="cuda") / rows
            if case["entropy"]:
                s["entropy"] = _entropy(s["logits"], case["scale"], log_s, m)
                s["dentropy"] = torch.randn(rows, generator=g, device="cuda") * (0.01 / rows)
            s["dlogits"] = empty(rows, vocab, dtype=t)
    else:
        places, ends = _spread(case)
        s["flat"], s["out"] = {}, {}
        for t, n in ends.items():
            if n:
                s["flat"][t] = torch.zeros(n, dtype=TYPES[t], device="cuda")
                s["out"][t] = torch.zeros(n, dtype=TYPES[t], device="cuda")
        s["grads"] = [s["flat"][t][at:at + k] for t, at, k in places]
        s["outs"] = [s["out"][t][at:at + k] for t, at, k in places]
        for x in s["grads"]:
            x.normal_(0.0, 1e-3, generator=g)
        s["norm"] = empty(1)
    return s


# ---------------------------------------------------------------- plain forms

def _lse(logits, scale):
    """(lse, log of the sum over the largest's, the largest with 0 for an empty row's)."""
    z = logits.float() * scale
    m = z.amax(1)
    lone = torch.where(m == -math.inf, 0.0, m)
    log_s = torch.log(torch.exp(z - lone[:, None]).sum(1))
    return lone + log_s, log_s, lone


def _entropy(logits, scale, log_s, m):
    d = logits.float() * scale - m[:, None]
    e = torch.exp(d)
    h = log_s - torch.where(e > 0, e * d, 0.0).sum(1) / torch.exp(log_s)
    return torch.where(log_s == -math.inf, 0.0, h)


def _top(logits, k):
    """Tokens of the k largest logits of each row, ties by the lowest token: the largest of whole numbers made of both."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7fffffff), bits)  # as the values, in whole numbers
    vocab = logits.shape[1]
    tokens = torch.arange(vocab, device=logits.device)
    return (order * (1 << 31) + ((1 << 31) - 1 - tokens)).topk(k, 1).indices


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "embed":
        t = s["tokens"].long()
        here = (t >= 0) & (t < c["vocab"])
        rows = s["w"][t.clamp(0, c["vocab"] - 1)].float() * c["scale"]
        return torch.where(here[:, None], rows, 0.0).to(s["w"].dtype)
    if op == "embed_grad":
        t = s["tokens"].long()
        here = (t >= 0) & (t < c["vocab"])
        dw = torch.zeros(c["vocab"], c["cols"], device="cuda")
        dw.index_add_(0, t[here], s["dy"][here].float())
        return (dw * c["scale"]).to(s["dy"].dtype)
    if op == "log_probs":
        z, t = s["logits"], s["targets"].long()
        here = (t >= 0) & (t < c["vocab"])
        lse, log_s, m = _lse(z, c["scale"])
        empty = lse == -math.inf

        def log_p(tokens):
            p = z.gather(1, tokens).float() * c["scale"] - m[:, None] - log_s[:, None]
            return torch.where(empty[:, None], -math.inf, p)

        logp = log_p(t.clamp(0, c["vocab"] - 1)[:, None])[:, 0]
        out = {"logp": torch.where(here, logp, 0.0), "lse": lse}
        if c["entropy"]:
            out["entropy"] = _entropy(z, c["scale"], log_s, m)
        if c["top"]:
            top = _top(z, c["top"])
            out["top_tokens"], out["top_logp"] = top.int(), log_p(top)
        return out
    if op == "log_probs_grad":
        t = s["targets"].long()
        here = (t >= 0) & (t < c["vocab"])
        lse = torch.where(s["lse"] == -math.inf, math.inf, s["lse"])[:, None]  # an empty row's p are 0
        d = s["logits"].float() * c["scale"] - lse
        p = torch.exp(d)
        g = torch.where(here & (s["lse"] != -math.inf), s["dlogp"], 0.0)[:, None]
        dz = -p * g
        if c["entropy"]:
            dz -= s["dentropy"][:, None] * torch.where(p > 0, p * (d + s["entropy"][:, None]), 0.0)
        dz.scatter_add_(1, t.clamp(0, c["vocab"] - 1)[:, None], g)
        return (dz * c["scale"]).to(s["logits"].dtype)
    norm = torch.cat([x.float() for x in s["grads"]]).square().sum(dtype=torch.float64).sqrt()
    out = {"norm": norm.float().reshape(1)}
    if op == "clip":
        by = torch.clamp(c["most"] / (norm + CLIP_EPS), max=1.0).float()
        out["clipped"] = {t: (x.float() * by).to(x.dtype) for t, x in s["flat"].items()}
    return out


# ---------------------------------------------------------------- the framework's

def _framework(s):
    import fsdp_layout_aware_gb300 as tide
    c = s["case"]
    op = c["op"]
    if op == "embed":
        tide.tide_embedding(s["tokens"], s["w"], s["out"], scale=c["scale"])
        return s["out"]
    if op == "embed_grad":
        tide.tide_embedding_backward(s["tokens"], s["dy"], s["dw"], scale=c["scale"])
        return s["dw"]
    if op == "log_probs":
        top = (s["top_logp"], s["top_tokens"]) if c["top"] else None
        tide.tide_log_probs(s["logits"], s["targets"], s["logp"], lse=s["lse"], entropy=s["entropy"], top=top,
                            scale=c["scale"])
        out = {"logp": s["logp"], "lse": s["lse"]}
        if c["entropy"]:
            out["entropy"] = s["entropy"]
        if c["top"]:
            out["top_logp"], out["top_tokens"] = top
        return out
    if op == "log_probs_grad":
        tide.tide_log_probs_backward(s["logits"], s["lse"], s["dlogits"], targets=s["targets"], dlogp=s["dlogp"],
                                     entropy=s.get("entropy"), dentropy=s.get("dentropy"), scale=c["scale"])
        return s["dlogits"]
    if "list" not in s:  # a program keeps its lists of tensors, like its pointer arrays
        s["list"] = tide.TensorList(s["grads"])
        s["out_list"] = tide.TensorList(s["outs"])
    tide.tide_grad_norm(s["list"], s["norm"])
    out = {"norm": s["norm"]}
    if op == "clip":
        tide.tide_grad_clip(s["list"], s["norm"], c["most"], eps=CLIP_EPS, out=s["out_list"])
        out["clipped"] = s["out"]
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------- floors

def _rows_used(case):
    """How many rows of the vocabulary the tokens are expected to name."""
    n, vocab = case["tokens"], case["vocab"]
    r = torch.arange(1, vocab + 1, dtype=torch.float64)
    p = torch.log((r + 1) / r) / math.log(vocab + 1) * (1 - case["hot"])
    p[vocab // 3] += case["hot"]
    return float((1 - torch.exp(n * torch.log1p(-p * (1 - case["pad"])))).sum())


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        n, cols, b = case["tokens"], case["cols"], 2 if case["dtype"] == "bf16" else 4
        index = n * (4 if case["index"] == "i32" else 8)
        if op == "embed":
            return {"bytes": index + (_rows_used(case) + n) * cols * b, "flops": n * cols}
        return {"bytes": index + (n * (1 - case["pad"]) + case["vocab"]) * cols * b, "flops": n * cols}
    if op in ("log_probs", "log_probs_grad"):
        n, b = case["rows"] * case["vocab"], 2 if case["dtype"] == "bf16" else 4
        row = 4 + 4 + (4 if case["index"] == "i32" else 8)
        if op == "log_probs":
            row += (4 if case["entropy"] else 0) + 8 * case["top"]
            return {"bytes": n * b + case["rows"] * row, "flops": 5 * n}
        return {"bytes": 2 * n * b + case["rows"] * (row + (8 if case["entropy"] else 0)), "flops": 6 * n}
    places, _ = _spread(case)
    bytes_ = sum(k * (2 if t == "bf16" else 4) for t, _, k in places)
    n = sum(k for _, _, k in places)
    return {"bytes": bytes_ * (2 if op == "clip" else 1) + 4, "flops": n * (3 if op == "clip" else 2)}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        vocab, t = case["vocab"], s["tokens"].long()
        named = ((t >= 0) & (t < vocab)).double().unsqueeze(1) * case["scale"]
        if op == "embed":
            return s["w"].double().index_select(0, t % vocab) * named
        order = torch.argsort(t, stable=True)
        dy = s["dy"].double().mul_(named)
        dw = torch.zeros(vocab, case["cols"], dtype=torch.float64, device="cuda")
        dw.index_put_(((t % vocab)[order],), dy[order], accumulate=True)
        return dw
    if op in ("log_probs", "log_probs_grad"):
        vocab, t = case["vocab"], s["targets"].long()
        named = (t >= 0) & (t < vocab)
        logs = torch.log_softmax(s["logits"].double().mul_(case["scale"]), 1)
        logs.masked_fill_((s["logits"] == -math.inf).all(1, keepdim=True), -math.inf)
        if op == "log_probs":
            z = s["logits"].double().mul_(case["scale"])
            out = {"logp": torch.where(named, logs[torch.arange(len(t), device="cuda"), t % vocab], 0.0),
                   "lse": torch.logsumexp(z, 1)}
            del z
            if case["entropy"]:
                out["entropy"] = -torch.special.xlogy(logs.exp(), logs.exp()).sum(1)
            if case["top"]:
                top = [torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
                       for x in s["logits"].split(512)]
                out["top_tokens"] = torch.cat(top).int()
                out["top_logp"] = logs.gather(1, torch.cat(top))
            return out
        # From the kept lse and entropy, which are inputs.
        lse = s["lse"].double().unsqueeze(1)
        logs = s["logits"].double().mul_(case["scale"]).sub_(lse).masked_fill_(lse == -math.inf, -math.inf)
        p = logs.exp()
        g = s["dlogp"].double() * named * (s["lse"] > -math.inf)
        onehot = torch.zeros_like(p)
        onehot[torch.arange(len(t), device="cuda"), t % vocab] = 1.0
        dz = onehot.sub_(p).mul_(g.unsqueeze(1))
        if case["entropy"]:
            h = s["entropy"].double().unsqueeze(1)
            dz -= (torch.special.xlogy(p, p) + p * h) * s["dentropy"].double().unsqueeze(1)
        return dz.mul_(case["scale"])
    squares = torch.stack([torch.dot(x.double(), x.double()) for x in s["grads"]])
    norm = torch.sqrt(squares.sum())
    out = {"norm": norm.reshape(1)}
    if op == "clip":
        by = min(1.0, case["most"] / (norm.item() + CLIP_EPS))
        out["clipped"] = {t: x.double() * by for t, x in s["flat"].items()}
    return out
