"""Plain 64-bit forms of the embedding, the norm and the 8-bit activations, and
how far the kernels' fp32 arithmetic may be from them.

u = 2^-24 is fp32's half step, HALF[t] that of an output type.  A sum of terms
x_i whose longest chain of additions has n links is off by at most
n u sum|x_i| (first order)."""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BLOCK = 128
INT8, E4M3 = 1, 2


def embed(ids, weight, scale, pad=None):
    out = weight.double()[ids.long()] * scale
    return out if pad is None else out * (pad == 0)[:, None]


def embed_grad(ids, d_out, vocab, scale, pad=None):
    """(dW, sum of |terms|) in 64 bits."""
    keep = torch.ones_like(ids, dtype=torch.bool) if pad is None else pad == 0
    g = d_out.double()[keep] * scale
    i = ids.long()[keep]
    dw = torch.zeros((vocab, d_out.shape[1]), dtype=torch.float64, device=d_out.device)
    mag = dw.clone()
    return dw.index_add_(0, i, g), mag.index_add_(0, i, g.abs())


def embed_grad_bound(ids, dw, mag, dtype):
    """A row of n tokens: n - 1 additions at most in a chain, the scale's
    product, the output's rounding."""
    n = int(torch.bincount(ids.long()).max()) if ids.numel() else 0
    return (n + 2) * U * mag + HALF[dtype] * dw.abs() + 1e-40


def chain(d):
    """Longest chain of additions over a row: at most 32 elements in a lane,
    or one of every 512, five shuffles, 32 warps."""
    return max(32, -(-d // 512)) + 5 + 32


def norm(x, w, b, eps, rms, offset):
    """y, mean, rstd in 64 bits (w, b: None or [d])."""
    x = x.double()
    mean = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device) if rms else x.mean(1)
    rstd = ((x - mean[:, None]) ** 2).mean(1).add(eps).rsqrt()
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * (w.double() + offset)
    if b is not None:
        y = y + b.double()
    return y, mean, rstd


def norm_bounds(x, w, b, eps, rms, offset):
    """Bounds of |error| of bf16 y, of mean and of rstd (relative).

    mean: chain u mean|x|.  Centred squares: 3 roundings each, chain more in
    their sum, and the mean's error adds its square: rstd is off by half of
    that relative to var + eps, and by 4 u of its own (rsqrtf, the sum with
    eps, the product with 1/d)."""
    xd = x.double()
    y, mean, rstd = norm(x, w, b, eps, rms, offset)
    L = chain(x.shape[1])
    dm = torch.zeros_like(mean) if rms else (L + 2) * U * xd.abs().mean(1)
    dr = (L + 3) * U / 2 + 4 * U + dm ** 2 * rstd ** 2 / 2
    wf = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if w is None else (w.double() + offset).abs()
    xc = (xd - mean[:, None]).abs()
    core = wf * rstd[:, None] * (dm[:, None] + xc * (dr[:, None] + 5 * U))
    bb = 0.0 if b is None else b.double().abs()
    fp32 = core + 2 * U * (wf * rstd[:, None] * xc + bb)
    return fp32 * 1.01 + HALF[torch.bfloat16] * y.abs() * 1.01 + 1e-40, dm + 1e-40, dr


def norm_grad(dy, x, mean, rstd, w, rms, offset):
    """dx, dw, db in 64 bits from given statistics."""
    dy, x = dy.double(), x.double()
    xh = (x - (0.0 if rms else mean.double()[:, None])) * rstd.double()[:, None]
    g = dy if w is None else dy * (w.double() + offset)
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if not rms:
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd.double()[:, None], (dy * xh).sum(0), dy.sum(0)


def norm_grad_bounds(dy, x, mean, rstd, w, rms, offset, dtype):
    """Bounds for bf16 dx and dw, db of `dtype`.  xh carries 2 roundings, g 2,
    the row sums `chain` more, the last line 4; dw, db: a chain of at most
    `rows` additions over products with 3 roundings."""
    dx, dw, db = norm_grad(dy, x, mean, rstd, w, rms, offset)
    dy, x = dy.double(), x.double()
    r = rstd.double()[:, None]
    xh = ((x - (0.0 if rms else mean.double()[:, None])) * r).abs()
    g = (dy if w is None else dy * (w.double() + offset)).abs()
    L = chain(x.shape[1])
    m1 = 0.0 if rms else g.mean(1, keepdim=True)
    bdx = r * U * (L + 16) * (g + m1 + xh * (g * xh).mean(1, keepdim=True))
    n = x.shape[0] + 8
    bdw = n * U * (dy.abs() * xh).sum(0)
    bdb = n * U * dy.abs().sum(0)
    h = HALF[dtype]
    return (bdx * 1.01 + HALF[torch.bfloat16] * dx.abs() * 1.01 + 1e-40, bdw * 1.01 + h * dw.abs() * 1.01 + 1e-40,
            bdb * 1.01 + h * db.abs() * 1.01 + 1e-40)


def pack(x, fmt):
    """(codes as uint8, scale) of the 8-bit form, on the CPU: every step is
    one IEEE fp32 operation, so both are defined bit for bit."""
    x = x.detach().cpu().float()
    r, d = x.shape
    nb = -(-d // BLOCK)
    top = torch.tensor(127.0 if fmt == INT8 else 448.0)
    b = torch.zeros((r, nb * BLOCK))
    b[:, :d] = x
    b = b.view(r, nb, BLOCK)
    a = b.abs().amax(2)
    a = torch.where(torch.isnan(b).any(2), torch.tensor(float("nan")), a)
    ok = (a >= 2.0 ** -100) & (a < float("inf"))
    safe = torch.where(ok, a, torch.ones_like(a))
    inv = torch.where(ok, top.expand_as(a) / safe, torch.zeros_like(a))
    scale = torch.where(ok, safe / top.expand_as(a), torch.zeros_like(a))
    scale = torch.where(a < 2.0 ** -100, torch.zeros_like(a), torch.where(ok, scale, torch.full_like(a, float("nan"))))
    u = torch.where(ok[:, :, None], b, torch.zeros_like(b)) * inv[:, :, None]
    u = u.view(r, -1)[:, :d]
    if fmt == INT8:
        return torch.round(u).to(torch.int8).view(torch.uint8), scale
    return u.to(torch.float8_e4m3fn).view(torch.uint8), scale


def held(q, scale, fmt, dtype=torch.float32):
    """The values of codes and factors: code * scale, rounded to fp32
    (unpack8), or in 64 bits, where it is exact (norm_bwd)."""
    v = (q.view(torch.int8) if fmt == INT8 else q.view(torch.float8_e4m3fn)).float().to(dtype)
    d = q.shape[1]
    return v * scale.to(dtype).repeat_interleave(BLOCK, 1)[:, :d]


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got - want).abs()
    bad = ~(err <= bound)
    if bool(bad.any()):
        k = int((err / bound).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst at {k}: got "
                             f"{got.reshape(-1)[k].item()!r}, want {want.reshape(-1)[k].item()!r}, bound "
                             f"{bound.expand_as(want).reshape(-1)[k].item()!r}")


# --------------------------------------------------------------------------
# Bounds by the additions that a term really goes through, in place of all of
# its row's or column's (the bounds above): for long rows only these see a
# single lost or doubled term.
# --------------------------------------------------------------------------
def embed_links(n, tokens):
    """Additions on the way of a term in a table row of n tokens (n: a tensor),
    the most over the kernels: 32 in a chunk (of 8 to 32 tokens); a warp's share
    of the row's chunks, of which there are n / 8 + 2 at most, and 16 warps.  Calls
    of up to 1,024 tokens may take one launch: an eighth of the row's part of
    the list, and 8 warps."""
    long = 32 + torch.ceil((n / 8 + 2) / 16) + 16
    if tokens <= 1024:
        long = torch.maximum(long, torch.full_like(n, 128 + 8))
    return torch.minimum(n, long)


def embed_grad_tight(ids, dw, mag, dtype, pad=None):
    """embed_links additions, the scale's product, one more addition where the
    sums are added to a gradient, the output's rounding."""
    kept = ids.long() if pad is None else ids.long()[pad == 0]
    n = torch.bincount(kept, minlength=dw.shape[0]).double()[:, None]
    return ((embed_links(n, ids.numel()) + 2) * U * mag + HALF[dtype] * dw.abs()) * 1.01 + 1e-40


def norm_links(rows):
    """Additions on the way of a term of dw or db: the rows of a group (144 CTAs
    at least where there are that many rows; two rows in the single-CTA calls),
    up to 16 groups of a CTA, 148 partial rows in 16 shares of up to 10, and
    the 16 shares."""
    return max(2, -(-rows // 144)) + 16 + 10 + 16


def norm_grad_tight(dy, x, mean, rstd, w, rms, offset, dtype):
    """norm_grad_bounds with norm_links additions: xh has 2 roundings, its
    product with dy one."""
    dx, dw, db = norm_grad(dy, x, mean, rstd, w, rms, offset)
    bx, _, _ = norm_grad_bounds(dy, x, mean, rstd, w, rms, offset, dtype)
    dy, x = dy.double(), x.double()
    xh = ((x - (0.0 if rms else mean.double()[:, None])) * rstd.double()[:, None]).abs()
    n = (norm_links(x.shape[0]) + 3) * U
    h = HALF[dtype]
    return (bx, (n * (dy.abs() * xh).sum(0) + h * dw.abs()) * 1.01 + 1e-40,
            (n * dy.abs().sum(0) + h * db.abs()) * 1.01 + 1e-40)


# --------------------------------------------------------------------------
# Inputs whose sums are exact in fp32 in any order: small integers (times powers
# of two), of which 2^24 units are never reached.  A term lost or counted twice
# shows whatever the length.
# --------------------------------------------------------------------------
def integers(shape, top, g, device, zero=False):
    """Whole numbers -top..top, zero left out unless asked for."""
    v = torch.randint(1, top + 1, shape, generator=g, device=device)
    v = torch.where(torch.rand(shape, generator=g, device=device) < 0.5, -v, v)
    if zero:
        v = torch.where(torch.rand(shape, generator=g, device=device) < 0.2, torch.zeros_like(v), v)
    return v


def exact_norm_inputs(r, d, fmt, g, device):
    """dy, x (bf16), held (64 bits), q, scale, mean, rstd: dy xh are multiples of
    1/8 below 4 x (8 + 3) / 2 = 22, so 176 units: 95,000 rows stay below 2^24."""
    x = integers((r, d), 8, g, device, zero=True).to(torch.bfloat16)
    dy = integers((r, d), 4, g, device).to(torch.bfloat16)
    mean = integers((r,), 3, g, device, zero=True).float()
    rstd = 2.0 ** -torch.randint(1, 3 if fmt == 0 else 2, (r,), generator=g, device=device).float()
    if fmt == 0:
        return dy, x, x.double(), None, None, mean, rstd
    codes = x.to(torch.int8).view(torch.uint8) if fmt == INT8 else x.float().to(torch.float8_e4m3fn).view(torch.uint8)
    scale = 2.0 ** -torch.randint(0, 3, (r, -(-d // BLOCK)), generator=g, device=device).float()
    return dy, None, held(codes, scale, fmt, torch.float64), codes, scale, mean, rstd
