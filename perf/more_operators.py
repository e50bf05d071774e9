"""What a training step of these layers needs around the layer and the head,
measured: the embedding's lookup and its gradient, the normalisation before
the activation quantizer with its backward, and the AdamW update of every
weight.

  normalisation   mean = center * sum x / k, d = x - mean,
                  rstd = 1 / sqrt(sum d^2 / k + eps), both from sums in 64 bits;
                  y = ((d rstd) w) + b, every step one rounding to 32 bits.
                  With the quantizer: gamma = max |y| of the row,
                  xq = clamp(rint(y / (max(gamma, 1e-5) / 128)), -127, 127)
  its backward    xh = (x - mean) rstd, g = dy w,
                  dx = rstd (g - center * mean(g) - xh mean(g xh)),
                  dw = sum_t dy xh, db = sum_t dy
  embedding       out[t] = scale table[id[t]]; a negative id gives zeros
  its backward    dtable[v] = scale sum over t with id[t] = v of dout[t],
                  alone or added to what dtable holds (a tied head's gradient)
  AdamW           m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2,
                  w = w (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps),
                  every step one rounding to 32 bits.  BF16 masters carry the
                  low 16 bits of the 32-bit weight beside them.  States in 8
                  bits are e4m3 times a scale for each 256 values: m rounded
                  to nearest, sqrt(v) by a hash of its place and the step.

Where `own` is false, `run` is the plain form: elementary torch operations.
Where it is true, `run` makes the calls of this repository's package.
"""

import math
import random

import torch

own = False

EPS_NORM = 1e-5
ADAM = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1)
MOST_BYTES = {"norm_fwd": 6.0e8, "norm_bwd": 6.0e8, "embed_fwd": 9.0e8, "embed_bwd": 2.0e9, "adamw": 5.0e9}
KINDS = tuple(MOST_BYTES)


def listed():
    """Widths and feed-forward sizes are those of the transformer blocks this
    repository works on (256, 1536, 3200, 5120); vocabularies as in its output head."""
    return [
        # decode: one token on its way into a layer, normalised and quantized
        dict(name="norm_quant_1tok", kind="norm_fwd", tokens=1, k=3200, x="float32", y="float32", quant=True,
             center=False, bias=False),
        # a training step's forward: the quantized input, and what the layer's backward reads
        dict(name="norm_quant_block", kind="norm_fwd", tokens=4096, k=5120, x="bfloat16", y="float32", quant=True,
             center=True, bias=True),
        # odd sizes: rows that no vector load fits
        dict(name="norm_bwd_ragged", kind="norm_bwd", tokens=777, k=1541, x="float16", y="float16", center=True,
             bias=True),
        # the gradient of a layer's input (32 bits) on its way back into the residual stream
        dict(name="norm_bwd_block", kind="norm_bwd", tokens=8192, k=5120, x="bfloat16", y="float32", center=True,
             bias=True),
        # a few prompts' next tokens
        dict(name="embed_fwd_few", kind="embed_fwd", tokens=37, vocab=32003, k=1536, table="bfloat16", out="float32",
             gone=0.0, scale=1.0),
        # a training batch
        dict(name="embed_fwd_block", kind="embed_fwd", tokens=16384, vocab=128256, k=5120, table="bfloat16",
             out="bfloat16", gone=0.02, scale=2.0),
        # odd sizes, padded batch
        dict(name="embed_bwd_ragged", kind="embed_bwd", tokens=777, vocab=50257, k=1541, table="float16",
             out="float16", gone=0.25, scale=1.0, add=False),
        # a table of its own: the whole gradient is written
        dict(name="embed_bwd_block", kind="embed_bwd", tokens=65536, vocab=32000, k=3200, table="bfloat16",
             out="bfloat16", gone=0.02, scale=1.0, add=False),
        # tied to the head, whose gradient is there already
        dict(name="embed_bwd_tied", kind="embed_bwd", tokens=16384, vocab=128256, k=5120, table="bfloat16",
             out="float32", gone=0.02, scale=2.0, add=True),
        # a unit-sized model: many small tensors
        dict(name="adamw_unit", kind="adamw", blocks=4, width=256, ffn=704, bits=32, w="bfloat16", low=True,
             g="float32", schedule=False),
        # a block's masters and norms, states in 32 bits
        dict(name="adamw_block", kind="adamw", blocks=1, width=3200, ffn=8640, bits=32, w="bfloat16", low=True,
             g="float32", schedule=False),
        # a larger block, states in 8 bits, the step's factors on the GPU (a clipped gradient)
        dict(name="adamw8_block", kind="adamw", blocks=1, width=5120, ffn=13824, bits=8, w="bfloat16", low=True,
             g="float32", schedule=True),
    ]


SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}


def _shapes(case):
    """A transformer block's seven matrices and two norm weights, `blocks` times over."""
    w, f = case["width"], case["ffn"]
    return ([(w, w)] * 4 + [(f, w)] * 2 + [(w, f)] + [(w,)] * 2) * case["blocks"]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(KINDS)
    half = rng.choice(("bfloat16", "bfloat16", "float16"))
    if kind.startswith("norm"):
        x = rng.choice((half, half, "float32"))
        case = dict(kind=kind, tokens=log_uniform(1, 16384), k=log_uniform(64, 16384), x=x,
                    y=rng.choice((x, "float32")), center=rng.random() < 0.7, bias=rng.random() < 0.5)
        if kind == "norm_fwd":
            case["quant"] = rng.random() < 0.5
            if case["quant"]:
                case["k"] = max(64, case["k"] // 64 * 64)
    elif kind.startswith("embed"):
        table = rng.choice((half, half, "float32"))
        case = dict(kind=kind, tokens=log_uniform(1, 65536), vocab=log_uniform(500, 128256), k=log_uniform(8, 8192),
                    table=table, out=rng.choice((table, "float32")), gone=rng.choice((0.0, 0.02, 0.5)),
                    scale=rng.choice((1.0, 2.0)))
        if rng.random() < 0.5:
            case["k"] = max(8, case["k"] // 8 * 8)
        if kind == "embed_bwd":
            case["add"] = rng.random() < 0.5
    else:
        width = log_uniform(64, 5120)
        case = dict(kind=kind, blocks=log_uniform(1, 8), width=width, ffn=log_uniform(64, 13824),
                    bits=rng.choice((8, 32)), w=rng.choice(("bfloat16", "bfloat16", "float16", "float32")),
                    g=rng.choice(("float32", "bfloat16")), schedule=rng.random() < 0.5)
        case["low"] = case["w"] == "bfloat16" and rng.random() < 0.8
    while work(case)["bytes"] > MOST_BYTES[kind]:
        for f in ("tokens", "blocks", "vocab", "ffn"):
            if case.get(f, 1) > 1:
                case[f] = case[f] // 2
    return case


def work(case):
    kind = case["kind"]
    if kind.startswith("norm"):
        t, k, x, y = case["tokens"], case["k"], SIZE[case["x"]], SIZE[case["y"]]
        if kind == "norm_fwd":
            return {"bytes": t * k * (x + y + (1 if case["quant"] else 0)) + 8 * k + 12 * t, "flops": 8 * t * k}
        return {"bytes": t * k * (2 * x + y) + 12 * k + 8 * t, "flops": 13 * t * k}
    if kind.startswith("embed"):
        # distinct ids of `tokens` draws with the weights 1 / (rank + 3): the expected number
        t, v, k = case["tokens"] * (1.0 - case["gone"]), case["vocab"], case["k"]
        norm = math.log((v + 3.0) / 3.0)
        rows, r = 0.0, 1.0
        while r <= v:                                              # by stretches of ranks, each 2% longer than the last
            n = min(max(1.0, 0.02 * r), v + 1 - r)
            rows -= n * math.expm1(-t / ((r + n / 2 + 2.0) * norm))
            r += n
        table, out = SIZE[case["table"]], SIZE[case["out"]]
        if kind == "embed_fwd":
            return {"bytes": int(rows * k * table + case["tokens"] * (k * out + 8)), "flops": int(t * k)}
        moved = 2 * rows if case["add"] else v
        return {"bytes": int(moved * k * table + t * k * out + 8 * case["tokens"]), "flops": int(t * k)}
    n = sum(math.prod(s) for s in _shapes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / 256
    return {"bytes": int(n * (2 * SIZE[case["w"]] + (4 if case["low"] else 0) + SIZE[case["g"]] + state)),
            "flops": 15 * n}


# ------------------------------------------------------------------ inputs

def _ids(case, g):
    """Token ids as text has them: the id of rank r about 1 / (r + 3) as often, ranks scattered over the
    vocabulary, a share of the batch padding."""
    t, v = case["tokens"], case["vocab"]
    u = torch.rand(t, generator=g, device="cuda", dtype=torch.float64)
    rank = (3.0 * (((v + 3.0) / 3.0) ** u - 1.0)).long().clamp(0, v - 1)
    ids = torch.randperm(v, generator=g, device="cuda")[rank]
    return torch.where(torch.rand(t, generator=g, device="cuda") < case["gone"], torch.full_like(ids, -1), ids)


def _weights(case, shapes, normal, g):
    """Weights, gradients and states of many tensors, each a piece of one buffer of its kind (the buffers), and
    the pieces of every tensor (each)."""
    starts, total = [], 0
    for shape in shapes:
        starts.append(total)
        total += -(-math.prod(shape) // 256) * 256
    real = torch.zeros(total, device="cuda")                       # 1 where a tensor is, 0 in the gaps between them
    w32 = torch.zeros(total, device="cuda")
    matrix = len(shapes[0]) == 2
    for shape, at in zip(shapes, starts):
        n = math.prod(shape)
        real[at:at + n] = 1.0
        # norm weights are held in 32 bits and do not decay
        w32[at:at + n] = normal(n) / math.sqrt(shape[-1]) if matrix else 1.0 + 0.1 * normal(n)
    size = real * 1e-3 * torch.exp(normal(total))                  # of each value's gradients
    f = {}
    if case["low"]:
        bits = w32.view(torch.int32)
        high = (bits + 0x8000) >> 16
        f["w"] = high.to(torch.int16).view(torch.bfloat16)
        f["w_low"] = (bits - (high << 16)).to(torch.int16)
    else:
        f["w"] = w32.to(getattr(torch, case["w"]))
    f["g"] = (size * normal(total)).to(getattr(torch, case["g"]))
    m, root = 0.3 * size * normal(total), 0.1 * size * (0.5 + torch.rand(total, generator=g, device="cuda"))
    if case["bits"] == 32:
        f["m"], f["v"] = m, root * root
    else:
        for name, x in (("m", m), ("v", root)):
            x = x.view(-1, 256)
            scale = (x.abs().amax(dim=1) * (1.0 / 448.0)).clamp(min=2.0 ** -126)
            f[name] = (x / scale[:, None]).clamp(-448, 448).view(-1).to(torch.float8_e4m3fn)
            f[name + "_scale"] = scale
    each = [{name: x[at // 256:-(-(at + math.prod(shape)) // 256)] if name.endswith("scale")
             else x[at:at + math.prod(shape)] for name, x in f.items()} for shape, at in zip(shapes, starts)]
    for e in each:
        e["weight_decay"] = ADAM["weight_decay"] if matrix else 0.0
    return dict(buffers=f, each=each, weight_decay=each[0]["weight_decay"])


def prepare(case, seed):
    """Activations with a few strong channels, as a residual stream has them; weights of a trained norm;
    gradients of a mean over the tokens; optimizer states as after some steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = case["kind"]
    s = dict(case=case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if kind.startswith("norm"):
        t, k = case["tokens"], case["k"]
        strong = torch.where(torch.rand(k, generator=g, device="cuda") < 0.01, 8.0, 1.0)
        x = (normal(t, k) * strong + 0.3 * normal(t, 1)) * torch.exp(0.5 * normal(t, 1))
        s["x"] = x.to(getattr(torch, case["x"]))
        s["w"] = 1.0 + 0.2 * normal(k)
        s["b"] = 0.1 * normal(k) if case["bias"] else None
        if kind == "norm_bwd":
            scale = 64.0 if case["y"] == "float16" else 1.0        # loss scaling, as 16-bit training uses it
            s["dy"] = (normal(t, k) * (scale / math.sqrt(k))).to(getattr(torch, case["y"]))
            s["mean"], s["rstd"], _ = _statistics(s["x"], case["center"])
    elif kind.startswith("embed"):
        s["ids"] = _ids(case, g)
        dtype = getattr(torch, case["table"])
        if kind == "embed_fwd":
            s["table"] = (normal(case["vocab"], case["k"]) / math.sqrt(case["k"])).to(dtype)
        else:
            s["dout"] = (0.05 * normal(case["tokens"], case["k"])).to(getattr(torch, case["out"]))
            if case["add"]:
                s["dtable"] = (0.05 * normal(case["vocab"], case["k"])).to(dtype)
    else:
        s["step"], shapes = 9, _shapes(case)
        s["matrices"] = _weights(case, [x for x in shapes if len(x) == 2], normal, g)
        s["vectors"] = _weights(dict(case, w="float32", low=False, g="float32", bits=32),
                                [x for x in shapes if len(x) == 1], normal, g)
        s["tensors"] = s["matrices"]["each"] + s["vectors"]["each"]
        if case["schedule"]:
            # lr, 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t), the gradients' factor (clipping), the step
            s["schedule"] = torch.tensor([ADAM["lr"], 1.0 / (1.0 - ADAM["beta1"] ** 10),
                                          1.0 / math.sqrt(1.0 - ADAM["beta2"] ** 10), 0.37, 10.0], device="cuda")
    return s


# ------------------------------------------------------------------ the plain form

def _statistics(x, center):
    """mean, rstd (rounded to 32 bits) and x less its mean, from sums in 64 bits."""
    x = x.double()
    mean = x.mean(dim=1, keepdim=True) * (1.0 if center else 0.0)
    var = (x - mean).square().mean(dim=1, keepdim=True)
    return mean.float()[:, 0], (1.0 / (var + EPS_NORM).sqrt()).float()[:, 0], (x - mean).float()


def _norm(s):
    case = s["case"]
    mean, rstd, d = _statistics(s["x"], case["center"])
    y = d * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    out = y.to(getattr(torch, case["y"]))
    if not case["quant"]:
        return out, mean, rstd
    gamma = y.abs().amax(dim=1)
    step = gamma.clamp(min=1e-5) / 128.0
    xq = torch.round(y / step[:, None]).clamp(-127, 127).to(torch.int8)
    return xq, gamma, out, mean, rstd


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"]
    c1 = g.mean(dim=1, keepdim=True) * (1.0 if s["case"]["center"] else 0.0)
    c2 = (g * xh).mean(dim=1, keepdim=True)
    dx = (s["rstd"][:, None] * (g - c1 - xh * c2)).to(s["x"].dtype)
    return dx, (dy * xh).sum(dim=0), dy.sum(dim=0) if s["b"] is not None else None


def _embed(s):
    ids = s["ids"]
    rows = s["table"][ids.clamp(min=0)].float() * s["case"]["scale"]
    return torch.where(ids[:, None] >= 0, rows, torch.zeros_like(rows)).to(getattr(torch, s["case"]["out"]))


def _embed_backward(s):
    case, ids = s["case"], s["ids"]
    dtype = getattr(torch, case["table"])
    dout = torch.where(ids[:, None] >= 0, s["dout"].float(), torch.zeros((), device="cuda"))
    total = torch.zeros(case["vocab"], case["k"], device="cuda").index_add_(0, ids.clamp(min=0), dout) * case["scale"]
    if not case["add"]:
        return total.to(dtype)
    s["dtable"].copy_((s["dtable"].float() + total).to(dtype))
    return s["dtable"]


def _dither(n, seed):
    """16 bits for each of n values: halves of a hash (two rounds of multiply and xor-shift) of the pair's number."""
    h = (torch.arange((n + 1) // 2, device="cuda") * 0x9E3779B9 + seed) & 0xFFFFFFFF
    h = h ^ (h >> 16)
    h = (h * 0x7FEB352D) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 0x846CA68B) & 0xFFFFFFFF
    h = h ^ (h >> 16)
    return torch.stack((h & 0xFFFF, h >> 16), dim=1).view(-1)[:n].int()


def _blocks(x):
    """x in blocks of 256, each with its scale: (values / scale, scales)."""
    b = torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)
    scale = (b.abs().amax(dim=1) * (1.0 / 448.0)).clamp(min=2.0 ** -126)
    return (b * (1.0 / scale)[:, None]).view(-1)[:x.numel()], scale


def _held(codes, scale):
    return codes.float() * scale.repeat_interleave(256)[:codes.numel()]


def _adamw_one(e, lr, bias1, bias2, factor, seed):
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    w = e["w"].float()
    if "w_low" in e:
        w = ((e["w"].view(torch.int16).int() << 16) + e["w_low"].int()).view(torch.float32)
    small = "m_scale" in e
    m = _held(e["m"], e["m_scale"]) if small else e["m"]
    v = _held(e["v"], e["v_scale"]).square() if small else e["v"]
    g = e["g"].float() * factor
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    root = v.sqrt()
    w = w * (1.0 - lr * e["weight_decay"]) - (m / (root * bias2 + ADAM["eps"])) * (lr * bias1)
    if "w_low" in e:
        bits = w.view(torch.int32)
        high = (bits + 0x8000) >> 16
        e["w"].copy_(high.to(torch.int16).view(torch.bfloat16))
        e["w_low"].copy_((bits - (high << 16)).to(torch.int16))
    else:
        e["w"].copy_(w.to(e["w"].dtype))
    if not small:
        e["m"].copy_(m)
        e["v"].copy_(v)
        return
    t, scale = _blocks(m)
    e["m_scale"].copy_(scale)
    e["m"].copy_(t.to(torch.float8_e4m3fn))
    t, scale = _blocks(root)
    e["v_scale"].copy_(scale)
    least = torch.where(t < 2.0 ** -6, 2.0 ** -6, 0.0)
    t = (((t + least).view(torch.int32) + (_dither(t.numel(), seed) << 4)) & -0x100000).view(torch.float32) - least
    t = torch.where(root > 0, t.clamp(2.0 ** -9, 448.0), torch.zeros_like(t))
    e["v"].copy_(t.to(torch.float8_e4m3fn))


def _adamw_outputs(s):
    """Every buffer that a step changes."""
    return [{name: x for name, x in s[k]["buffers"].items() if name != "g"} for k in ("matrices", "vectors")]


def _adamw(s):
    if "schedule" in s:
        f = s["schedule"]
        lr, bias1, bias2, factor, seed = f[0], f[1], f[2], f[3], f[4].long()
    else:
        t = s["step"]
        lr, factor, seed = torch.tensor(ADAM["lr"]), 1.0, t
        bias1 = torch.tensor(1.0 / (1.0 - ADAM["beta1"] ** t))
        bias2 = torch.tensor(1.0 / math.sqrt(1.0 - ADAM["beta2"] ** t))
    [_adamw_one(e, lr, bias1, bias2, factor, seed) for e in s["tensors"]]


# ------------------------------------------------------------------ one pass

def run(state):
    s, case = state, state["case"]
    kind = case["kind"]
    if kind == "adamw":
        s["step"] += 1
        if own:
            from sparse_linear_layers_absmean_amd import sbl
            if "items" not in s:                                   # the list that a program makes once
                s["items"] = sbl.AdamWItems(s["tensors"])
            sbl.sbl_adamw_batch(s["items"], ADAM["lr"], ADAM["beta1"], ADAM["beta2"], ADAM["eps"], s["step"],
                                schedule=s.get("schedule"))
        else:
            _adamw(s)
        return _adamw_outputs(s)
    if not own:
        return {"norm_fwd": _norm, "norm_bwd": _norm_backward, "embed_fwd": _embed, "embed_bwd": _embed_backward}[kind](s)
    from sparse_linear_layers_absmean_amd import sbl
    if kind == "norm_fwd":
        call = sbl.norm_quant if case["quant"] else sbl.norm
        return call(s["x"], s["w"], s["b"], eps=EPS_NORM, center=case["center"], dtype=getattr(torch, case["y"]))
    if kind == "norm_bwd":
        return sbl.norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], want_bias=case["bias"],
                                 center=case["center"])
    if kind == "embed_fwd":
        return sbl.embed(s["ids"], s["table"], scale=case["scale"], dtype=getattr(torch, case["out"]))
    if case["add"]:
        return sbl.embed_backward(s["ids"], s["dout"], case["vocab"], scale=case["scale"], add_to=s["dtable"])
    return sbl.embed_backward(s["ids"], s["dout"], case["vocab"], scale=case["scale"],
                              dtype=getattr(torch, case["table"]))


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_norm(s):
    case = s["case"]
    x = s["x"].double()
    k = x.shape[1]
    mean = torch.mv(x, torch.full((k,), 1.0 / k, dtype=torch.float64, device="cuda")) if case["center"] \
        else torch.zeros(x.shape[0], dtype=torch.float64, device="cuda")
    if case["kind"] == "norm_fwd":
        var = torch.linalg.vector_norm(x - mean[:, None], dim=1).square() / k
        rstd = torch.rsqrt(var + EPS_NORM)
        y = torch.addcmul(torch.zeros((), dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double(),
                          (x - mean[:, None]) * rstd[:, None], s["w"].double())
        if not case["quant"]:
            return y, mean, rstd
        return None, torch.linalg.vector_norm(y, ord=math.inf, dim=1), y, mean, rstd
    # the gradient from the Jacobian of (x - mean) rstd, row by row: (I - (center 1 1^T + xh xh^T) / k) rstd
    dy, rstd = s["dy"].double(), s["rstd"].double()
    xh = (x - s["mean"].double()[:, None]) * rstd[:, None]
    g = dy * s["w"].double()
    dx = g - xh * (torch.einsum("tk,tk->t", g, xh) / k)[:, None]
    if case["center"]:
        dx -= g.sum(dim=1, keepdim=True) / k
    ones = torch.ones(dy.shape[0], dtype=torch.float64, device="cuda")
    return dx * rstd[:, None], torch.mv((dy * xh).t(), ones), torch.mv(dy.t(), ones) if case["bias"] else None


def _exact_embed(s):
    case, ids = s["case"], s["ids"]
    here = torch.nonzero(ids >= 0)[:, 0]
    if case["kind"] == "embed_fwd":
        out = torch.zeros(ids.numel(), case["k"], dtype=torch.float64, device="cuda")
        out[here] = s["table"].double()[ids[here]] * case["scale"]
        return out
    total = s["dtable"].double() if case["add"] else torch.zeros(case["vocab"], case["k"], dtype=torch.float64,
                                                                 device="cuda")
    return total.index_put_((ids[here],), s["dout"][here].double() * case["scale"], accumulate=True)


def _exact_adamw(s):
    """From the sums that m and v are, divided as they are written in the formula; codes and low bits have no
    value of their own here."""
    t = s["step"] + 1
    lr, c1, c2, factor = ADAM["lr"], 1.0 - ADAM["beta1"] ** t, 1.0 - ADAM["beta2"] ** t, 1.0
    if "schedule" in s:
        lr, c1, c2, factor = (float(x) for x in s["schedule"][:4].double())
        c1, c2 = 1.0 / c1, c2 ** -2
    out = []
    for group in (s["matrices"], s["vectors"]):
        e = group["buffers"]
        small = "m_scale" in e
        m, v = e["m"].double(), e["v"].double()
        if small:
            m, v = ((x.view(-1, 256) * e[scale].double()[:, None]).view(-1) for x, scale in
                    ((m, "m_scale"), (v, "v_scale")))
            v = v * v
        g = e["g"].double() * factor
        m = torch.lerp(g, m, ADAM["beta1"])
        v = torch.lerp(g * g, v, ADAM["beta2"])
        w = e["w"].double()
        if "w_low" in e:
            w = ((e["w"].view(torch.int16).int() << 16) + e["w_low"].int()).view(torch.float32).double()
        w = w - lr * group["weight_decay"] * w - lr * (m / c1) / ((v / c2).sqrt() + ADAM["eps"])
        new = dict(w=w, w_low=None, m=m, v=v)
        if small:
            new.update(m=None, v=None, m_scale=m.view(-1, 256).abs().amax(dim=1) / 448.0,
                       v_scale=v.sqrt().view(-1, 256).amax(dim=1) / 448.0)
        out.append({name: new[name] for name in e if name != "g"})
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"n": _exact_norm, "e": _exact_embed, "a": _exact_adamw}[case["kind"][0]](s)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(12)]:
        print(c, work(c))
