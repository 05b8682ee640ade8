"""What is measured of the training operators around the loss: the embedding of (noisy) token ids and its gradient, the
norm before the output head with its backward pass, and activations kept in 8 bits between the two passes.

`own` False computes each operator in its plain form (elementary torch operations in fp32, rounded once at the end);
`own` True makes the calls of diffusion_lm_loss_b200 that a training program makes."""
import math

import torch

own = False

BLOCK = 128          # columns that share one scale of an 8-bit activation
TINY = 2.0 ** -100   # blocks whose largest magnitude is below it are held as zeros


def listed():
    return [
        # the smallest training batch (2 sequences of 64, vocabulary 1,024): launch latency
        dict(name="embed_fwd_t128", op="embed_fwd", tokens=128, d=256, vocab=1024, masked=0.5, pads=0.0, scale=1.0),
        # LLaDA-like packed batch, half of the tokens masked
        dict(name="embed_fwd_t16384", op="embed_fwd", tokens=16384, d=4096, vocab=126464, masked=0.5, pads=0.0, scale=1.0),
        # its gradient: the smallest batch
        dict(name="embed_bwd_t128", op="embed_bwd", tokens=128, d=256, vocab=1024, masked=0.5, pads=0.0, scale=1.0, grad="bf16"),
        # the packed batch: the mask id's row sums some 8,000 tokens, most other rows none or one
        dict(name="embed_bwd_t16384", op="embed_bwd", tokens=16384, d=4096, vocab=126464, masked=0.5, pads=0.0, scale=1.0, grad="bf16"),
        # uniform noise (no mask id), padded, scaled embeddings, odd width, gradient kept in fp32
        dict(name="embed_bwd_t5000_d1001", op="embed_bwd", tokens=5000, d=1001, vocab=32768, masked=0.0, pads=0.2, scale=31.625, grad="f32"),
        # the last norm on one token's state: launch latency
        dict(name="norm_fwd_r1", op="norm_fwd", rows=1, d=4096, kind="rms", bias=False, param="bf16", offset=0.0),
        # the last norm of the packed batch
        dict(name="norm_fwd_r16384", op="norm_fwd", rows=16384, d=4096, kind="layer", bias=True, param="bf16", offset=0.0),
        dict(name="norm_bwd_r16384", op="norm_bwd", rows=16384, d=4096, kind="layer", bias=True, param="bf16", offset=0.0, grad="f32"),
        # odd width, fp32 parameters, weights stored as w - 1
        dict(name="norm_bwd_r777_d1003", op="norm_bwd", rows=777, d=1003, kind="rms", bias=False, param="f32", offset=1.0, grad="f32"),
        # a norm whose input is kept in 8 bits between forward and backward (canvas plus prefix of 4 sequences)
        dict(name="norm_kept8_r6144", op="norm_kept8", rows=6144, d=4096, kind="layer", bias=True, param="bf16", offset=0.0, grad="f32", fmt="int8"),
        # an activation packed in the forward pass and unpacked in the backward pass
        dict(name="act8_r16384", op="act8", rows=16384, d=4096, fmt="int8"),
        # odd width, few rows
        dict(name="act8_r130_d1001", op="act8", rows=130, d=1001, fmt="e4m3"),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi=8192):
    """A row width: a multiple of 8 in three cases of four, any number in the fourth."""
    d = _between(rng, 64, hi)
    return d if rng.random() < 0.25 else max(64, d // 8 * 8)


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "norm_fwd", "norm_bwd", "norm_kept8", "act8"])
    if op.startswith("embed"):
        d = _width(rng, 4096)
        vocab = _between(rng, 500, min(262144, 126464 * 4096 // d // (1 if op == "embed_fwd" else 2)))
        case = dict(op=op, tokens=_between(rng, 1, 16384), d=d, vocab=vocab, masked=rng.choice([0.0, rng.uniform(0.05, 0.95)]),
                    pads=rng.choice([0.0, rng.uniform(0.02, 0.6)]), scale=rng.choice([1.0, math.sqrt(d)]))
        if op == "embed_bwd":
            case["grad"] = rng.choice(["bf16", "f32"])
        return case
    d = _width(rng)
    case = dict(op=op, rows=_between(rng, 1, min(32768, 2 ** 26 // d)), d=d)
    if op != "act8":
        case.update(kind=rng.choice(["layer", "rms"]), bias=rng.random() < 0.5, param=rng.choice(["bf16", "f32"]),
                    offset=rng.choice([0.0, 1.0]))
        if op != "norm_fwd":
            case["grad"] = rng.choice(["bf16", "f32"])
    if op in ("act8", "norm_kept8"):
        case["fmt"] = rng.choice(["int8", "e4m3"])
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000 + seed)
    c = dict(case)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    if c["op"].startswith("embed"):
        t, v = c["tokens"], c["vocab"]
        ids = torch.randint(0, v - 1, (t,), generator=gen, device="cuda", dtype=torch.int32)
        ids = torch.where(uniform(t) < c["masked"], torch.full_like(ids, v - 1), ids)   # the last id is the mask id
        c["ids"] = ids
        c["pad"] = (uniform(t) < c["pads"]).to(torch.uint8) if c["pads"] > 0 else None
        if c["op"] == "embed_fwd":
            c["weight"] = normal(v, c["d"], std=0.02).to(torch.bfloat16)
        else:
            c["d_out"] = normal(t, c["d"], std=1e-2).to(torch.bfloat16)
        return c
    r, d = c["rows"], c["d"]
    # states of a residual stream: some channels much larger than the rest, a mean that is not zero
    channel = torch.exp(0.5 * normal(d)) * torch.where(uniform(d) < 0.01, 12.0, 1.0)
    c["x"] = (normal(r, d) * channel + 0.1).to(torch.bfloat16)
    if c["op"] == "act8":
        return c
    param = torch.bfloat16 if c["param"] == "bf16" else torch.float32
    c["weight"] = (1.0 - c["offset"] + normal(d, std=0.1)).to(param)
    c["bias_t"] = normal(d, std=0.1).to(param) if c["bias"] else None
    c["eps"] = 1e-5
    if c["op"] != "norm_fwd":
        c["d_y"] = normal(r, d, std=1e-2).to(torch.bfloat16)
    if c["op"] == "norm_bwd":     # what the forward pass left
        x = c["x"].double()
        mean = x.mean(1) if c["kind"] == "layer" else torch.zeros(r, device="cuda", dtype=torch.float64)
        var = (x - mean[:, None]).square().mean(1)
        c["mean"] = mean.float() if c["kind"] == "layer" else None
        c["rstd"] = (1.0 / torch.sqrt(var + c["eps"])).float()
    return c


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _blocks(x):
    """[rows, d] -> [rows, blocks, BLOCK] in fp32, zeros behind the row's end."""
    r, d = x.shape
    nb = (d + BLOCK - 1) // BLOCK
    out = torch.zeros((r, nb * BLOCK), dtype=torch.float32, device=x.device)
    out[:, :d] = x
    return out.view(r, nb, BLOCK)


def _plain_held8(x, fmt):
    """The fp32 values that the 8-bit form of x stands for."""
    b = _blocks(x)
    a = b.abs().amax(2, keepdim=True)
    top = torch.full_like(a, 127.0 if fmt == "int8" else 448.0)   # a tensor: a number's quotient is rounded twice
    zero = a < TINY
    inv = torch.where(zero, 0.0, top / a)
    q = (b * inv).round() if fmt == "int8" else (b * inv).to(torch.float8_e4m3fn).float()
    v = q * torch.where(zero, 0.0, a / top)
    return v.view(x.shape[0], -1)[:, :x.shape[1]]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1) if s["kind"] == "layer" else None
    xc = x - mean[:, None] if mean is not None else x
    rstd = 1.0 / torch.sqrt(xc.square().mean(1) + s["eps"])
    y = xc * rstd[:, None] * (s["weight"].float() + s["offset"])
    if s["bias_t"] is not None:
        y = y + s["bias_t"].float()
    return y.to(torch.bfloat16), mean, rstd


def _plain_norm_bwd(s, x, mean, rstd):
    dy = s["d_y"].float()
    xh = (x - mean[:, None] if mean is not None else x) * rstd[:, None]
    g = dy * (s["weight"].float() + s["offset"])
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(1, keepdim=True)
    out = {"d_x": (dx * rstd[:, None]).to(torch.bfloat16), "d_weight": (dy * xh).sum(0).to(_dtype(s["grad"]))}
    if s["bias_t"] is not None:
        out["d_bias"] = dy.sum(0).to(_dtype(s["grad"]))
    return out


def _plain(s):
    op = s["op"]
    if op == "embed_fwd":
        out = s["weight"][s["ids"].long()].float() * s["scale"]
        if s["pad"] is not None:
            out = out * (s["pad"] == 0)[:, None]
        return out.to(torch.bfloat16)
    if op == "embed_bwd":
        g = s["d_out"].float()
        if s["pad"] is not None:
            g = g * (s["pad"] == 0)[:, None]
        d_weight = torch.zeros((s["vocab"], s["d"]), dtype=torch.float32, device="cuda")
        d_weight.index_add_(0, s["ids"].long(), g)
        return (d_weight * s["scale"]).to(_dtype(s["grad"]))
    if op == "act8":
        return _plain_held8(s["x"], s["fmt"]).to(torch.bfloat16)
    if op == "norm_bwd":
        return _plain_norm_bwd(s, s["x"].float(), s["mean"], s["rstd"])
    y, mean, rstd = _plain_norm_fwd(s)
    out = {"y": y, "rstd": rstd}
    if mean is not None:
        out["mean"] = mean
    if op == "norm_kept8":
        out.update(_plain_norm_bwd(s, _plain_held8(s["x"], s["fmt"]), mean, rstd))
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import diffusion_lm_loss_b200 as dlm
    op = s["op"]
    if op == "embed_fwd":
        lay = dlm.make_layout(1, s["tokens"], None, s["pad"])
        return dlm.embed_fwd(lay, s["ids"], s["weight"], s["scale"])
    if op == "embed_bwd":
        lay = dlm.make_layout(1, s["tokens"], None, s["pad"])
        return dlm.embed_bwd(lay, s["ids"], s["d_out"], s["vocab"], s["scale"], grad_dtype=_dtype(s["grad"])).d_weight
    fmt = {"int8": dlm.PACK_INT8, "e4m3": dlm.PACK_E4M3}.get(s.get("fmt"), 0)
    if op == "act8":
        return dlm.unpack8(dlm.pack8(s["x"], fmt))
    kind = dlm.NORM_LAYER if s["kind"] == "layer" else dlm.NORM_RMS
    out = {}
    if op == "norm_bwd":
        held, mean, rstd = s["x"], s["mean"], s["rstd"]
    else:
        f = dlm.norm_fwd(s["x"], s["weight"], s["bias_t"], s["eps"], kind, s["offset"], pack=fmt)
        held, mean, rstd = f.packed, f.mean, f.rstd
        out = {"y": f.y, "rstd": f.rstd}
        if mean is not None:
            out["mean"] = mean
    if op != "norm_fwd":
        b = dlm.norm_bwd(s["d_y"], held, rstd, mean, s["weight"], kind, s["offset"], want_d_bias=s["bias"],
                         grad_dtype=_dtype(s["grad"]))
        out.update(d_x=b.d_x, d_weight=b.d_weight)
        if s["bias"]:
            out["d_bias"] = b.d_bias
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op, d = c["op"], c["d"]
    if op.startswith("embed"):
        t, v = c["tokens"], c["vocab"]
        live = t * (1.0 - c["pads"])
        plain_ids = live * (1.0 - c["masked"])
        rows = v * (1.0 - (1.0 - 1.0 / v) ** plain_ids) + (1.0 if c["masked"] > 0 else 0.0)   # distinct ids expected
        ids = 4 * t + (t if c["pads"] > 0 else 0)
        if op == "embed_fwd":
            return {"bytes": ids + 2 * d * rows + 2 * d * t, "flops": float(live * d)}
        return {"bytes": ids + 2 * d * live + (2 if c["grad"] == "bf16" else 4) * d * v, "flops": float(live * d)}
    n = c["rows"] * d
    scales = 4 * c["rows"] * ((d + BLOCK - 1) // BLOCK)
    if op == "act8":
        return {"bytes": 2 * (3 * n + scales), "flops": 4.0 * n}
    params = (2 if c["param"] == "bf16" else 4) * d
    both = 2 if c["bias"] else 1
    stats = (8 if c["kind"] == "layer" else 4) * c["rows"]
    fwd = 4 * n + params * both + stats
    if op == "norm_fwd":
        return {"bytes": fwd, "flops": 7.0 * n}
    bwd = 6 * n + stats + params + (2 if c["grad"] == "bf16" else 4) * d * both
    if op == "norm_bwd":
        return {"bytes": bwd, "flops": 12.0 * n}
    return {"bytes": fwd + n + scales + bwd - n + scales, "flops": 21.0 * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_held8(x, fmt):
    x = x.double()
    r, d = x.shape
    col = torch.arange(d, device=x.device) // BLOCK
    nb = int(col[-1]) + 1
    top = torch.zeros((r, nb), dtype=torch.float64, device=x.device)
    top.scatter_reduce_(1, col.expand(r, d), x.abs(), "amax")
    # which code an element gets is defined through the block's two factors in fp32 (each division and the product
    # rounded once): an element halfway between two codes goes where these send it
    most = 127.0 if fmt == "int8" else 448.0
    step = torch.where(top < TINY, torch.zeros_like(top), (top / most).float().double())[:, col]
    inv = torch.where(top < TINY, torch.zeros_like(top), (most / torch.clamp(top, min=TINY)).float().double())[:, col]
    u = (x * inv).float().double()
    if fmt == "int8":
        return torch.round(u) * step
    # 3 bits behind the leading one, exponents down to 2^-6, subnormal steps of 2^-9
    _, e = torch.frexp(u)
    ulp = torch.ldexp(torch.ones_like(u), torch.clamp(e - 1, min=-6) - 3)
    return torch.round(u / ulp) * ulp * step


def exact(case, seed):
    s = prepare(case, seed)
    op, d = s["op"], s["d"]
    if op.startswith("embed"):
        ids = s["ids"].long()
        keep = torch.ones_like(ids, dtype=torch.bool) if s["pad"] is None else s["pad"] == 0
        if op == "embed_fwd":
            out = torch.zeros((s["tokens"], d), dtype=torch.float64, device="cuda")
            out[keep] = s["weight"].double()[ids[keep]] * s["scale"]
            return out
        out = torch.zeros((s["vocab"], d), dtype=torch.float64, device="cuda")
        ids, g = ids[keep], s["d_out"][keep].double()
        if ids.numel():
            at = torch.argsort(ids)
            rows, counts = torch.unique_consecutive(ids[at], return_counts=True)
            ends = torch.cumsum(counts, 0)
            sums = torch.cumsum(g[at], 0)[ends - 1]
            sums[1:] -= sums[:-1].clone()
            out[rows] = sums * s["scale"]
        return out
    if op == "act8":
        return _exact_held8(s["x"], s["fmt"])
    x = s["x"].double()
    layer = s["kind"] == "layer"
    w = s["weight"].double() + s["offset"]
    out = {}
    if op == "norm_bwd":
        mean = s["mean"].double()[:, None] if layer else 0.0
        rstd = s["rstd"].double()[:, None]
    else:
        mean = torch.sum(x, 1, keepdim=True) / d if layer else 0.0
        rstd = (torch.sum((x - mean) ** 2, 1, keepdim=True) / d + s["eps"]) ** -0.5
        y = (x - mean) * rstd * w
        out = {"y": y if s["bias_t"] is None else y + s["bias_t"].double(), "rstd": rstd[:, 0]}
        if layer:
            out["mean"] = mean[:, 0]
    if op != "norm_fwd":
        held = x if op == "norm_bwd" else _exact_held8(s["x"], s["fmt"])
        dy = s["d_y"].double()
        xh = (held - mean) * rstd
        # the transposed Jacobian of y applied to dy: rstd * (I - 1 1^T / d - xh xh^T / d) (w * dy)
        g = w * dy
        dots = torch.einsum("rd,rd->r", g, xh)[:, None] / d
        ones = torch.einsum("rd->r", g)[:, None] / d if layer else 0.0
        out.update(d_x=rstd * (g - ones - xh * dots), d_weight=torch.einsum("rd,rd->d", dy, xh))
        if s["bias_t"] is not None:
            out["d_bias"] = dy.sum(0)
    return out
