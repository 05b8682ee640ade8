"""Long sums on the GPU: table gradients of rows of up to 20,000 tokens and
parameter gradients over up to 21,312 rows, on whole numbers, whose sums are
exact in any order, and on real values within the bounds of the additions that
a term really goes through; kernels with several rows to a group or CTA."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

dlm = pytest.importorskip("diffusion_lm_loss_b200")
bf16, f32 = torch.bfloat16, torch.float32
LAYER, RMS = 0, 1


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dlm.lib()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _placed(t, shift):
    """t's values in rows that start `shift` elements behind a 16-byte border."""
    buf = torch.zeros(t.numel() + shift + 8, dtype=t.dtype, device=t.device)
    v = buf[shift:shift + t.numel()].view(t.shape)
    v.copy_(t)
    return v


def _ids(kind, t, vocab, g):
    if kind == "one":
        return torch.full((t,), vocab // 2, dtype=torch.int32, device="cuda")
    if kind == "words":                     # the r-th most frequent with a share of 1 / r
        p = 1.0 / torch.arange(1, vocab + 1, device="cuda")
        return torch.multinomial(p / p.sum(), t, replacement=True, generator=g).int()
    if kind == "runs":                      # just under, just as many and just more tokens than 1 to 20 chunks
        runs = [c * n + e for c in (8, 16, 32) for n in (1, 2, 7, 8, 9, 10, 17, 20) for e in (-1, 0, 1)]
        ids = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), torch.tensor(runs, device="cuda")).int()
        return ids[torch.randperm(ids.numel(), generator=g, device="cuda")].contiguous()
    ids = torch.randint(0, vocab, (t,), generator=g, device="cuda", dtype=torch.int32)
    hit = torch.rand(t, generator=g, device="cuda") < 0.5
    return torch.where(hit, torch.full_like(ids, vocab - 1), ids)


# chunks of 8 tokens, of 16 and of 32 (t / 32 x tiles of 256 columns at least 2,368: the last six), aligned and not;
# one launch; "runs" has 12,432 tokens
TABLES = [(20000, 1000, 40, "one"), (20000, 1000, 41, "one"), (1000, 50, 512, "masked"), (1024, 50, 500, "words"),
          (1024, 20, 33, "one"), (4097, 1024, 136, "words"), (12432, 400, 264, "runs"), (12432, 400, 1001, "runs"),
          (40000, 70, 264, "masked"), (16384, 1000, 1032, "masked"), (16384, 1000, 1033, "words"),
          (12432, 400, 1544, "runs"), (12432, 400, 1601, "runs"), (12432, 90000, 1544, "words")]


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("t,vocab,d,kind", TABLES)
def test_table_gradients_of_whole_numbers_are_exact(t, vocab, d, kind, dtype):
    g = _gen(t + d)
    ids = _ids(kind, t, vocab, g)
    dy = ref.integers((ids.numel(), d), 8, g, "cuda").to(bf16)
    lay = dlm.make_layout(1, ids.numel())
    dw, mag = ref.embed_grad(ids, dy, vocab, 2.0)
    got = dlm.embed_bwd(lay, ids, dy, vocab, 2.0, grad_dtype=dtype)
    assert got.device_status() == 0 and torch.equal(got.d_weight, dw.to(dtype))
    old = ref.integers((vocab, d), 100, g, "cuda").to(dtype)
    acc = old.clone()
    dlm.embed_bwd(lay, ids, dy, vocab, 2.0, d_weight=acc, accumulate=True)
    want = torch.where((mag.sum(1) > 0)[:, None], (old.double() + dw).to(dtype), old)
    assert torch.equal(acc, want)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("t,vocab,d,kind", TABLES)
def test_table_gradients_within_their_additions(t, vocab, d, kind, dtype):
    g = _gen(t * d)
    ids = _ids(kind, t, vocab, g)
    pad = (torch.rand(ids.numel(), generator=g, device="cuda") < 0.1).to(torch.uint8)
    dy = torch.randn((ids.numel(), d), generator=g, device="cuda").to(bf16)
    lay = dlm.make_layout(1, ids.numel(), None, pad)
    dw, mag = ref.embed_grad(ids, dy, vocab, 5.5, pad)
    got = dlm.embed_bwd(lay, ids, dy, vocab, 5.5, grad_dtype=dtype).d_weight
    ref.assert_within(got, dw, ref.embed_grad_tight(ids, dw, mag, dtype, pad))
    old = torch.randn((vocab, d), generator=g, device="cuda").to(dtype)
    acc = old.clone()
    dlm.embed_bwd(lay, ids, dy, vocab, 5.5, d_weight=acc, accumulate=True)
    there = mag.sum(1) > 0
    want = old.double() + dw
    bound = ref.embed_grad_tight(ids, want, mag + old.double().abs(), dtype, pad)
    ref.assert_within(acc[there], want[there], bound[there])
    assert torch.equal(acc[~there], old[~there])


# one piece a lane, two with several groups, two rows at a time (9 to 12 warps), one group of 13 to 16, wider than
# a group holds; on the 16-byte borders, in step with one another off them, out of step (the last column)
ROWS = [(21312, 256, 0), (20665, 264, 0), (3100, 4096, 0), (900, 4608, 0), (900, 5120, 0), (900, 6144, 0), (900, 6152, 0),
        (900, 8192, 0), (20001, 250, 0), (1500, 2001, 0), (900, 5001, 0), (700, 8001, 0), (600, 8200, 0), (600, 9001, 0),
        (9001, 64, 1), (5000, 1000, 1), (700, 7001, 1)]


def _backward(dy, x, packed, mean, rstd, w, kind, bias, **kw):
    return dlm.norm_bwd(dy, x if packed is None else packed, rstd, mean if kind == LAYER else None, w, kind,
                        want_d_weight=True, want_d_bias=bias, grad_dtype=f32, **kw)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("kind,bias", [(LAYER, True), (LAYER, False), (RMS, True), (RMS, False)])
@pytest.mark.parametrize("r,d,shift", ROWS)
def test_parameter_gradients_of_whole_numbers_are_exact(r, d, shift, kind, bias, fmt):
    g = _gen(r + d + fmt)
    dy, x, held, q, s, mean, rstd = ref.exact_norm_inputs(r, d, fmt, g, "cuda")
    w = torch.randn(d, generator=g, device="cuda")
    packed = None if fmt == 0 else dlm.Packed8(q, s, fmt)
    dys, xs = _placed(dy, shift), None if x is None else _placed(x, shift)
    got = _backward(dys, xs, packed, mean, rstd, w, kind, bias)
    dx, dw, db = ref.norm_grad(dy, held, mean, rstd, w, kind == RMS, 0.0)
    assert torch.equal(got.d_weight.double(), dw)
    assert torch.equal(got.d_bias.double(), db) if bias else got.d_bias is None
    bx, _, _ = ref.norm_grad_bounds(dy, held, mean, rstd, w, kind == RMS, 0.0, f32)
    ref.assert_within(got.d_x, dx, bx, "d_x")
    old = ref.integers((2, d), 100, g, "cuda").float()
    acc = old.clone()
    more = _backward(dys, xs, packed, mean, rstd, w, kind, bias, d_weight=acc[0], d_bias=acc[1] if bias else None,
                     accumulate=True)
    assert torch.equal(more.d_x, got.d_x) and torch.equal(acc[0].double(), old[0].double() + dw)
    assert torch.equal(acc[1].double(), old[1].double() + (db if bias else 0))


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("kind,bias", [(LAYER, True), (RMS, True), (RMS, False)])
@pytest.mark.parametrize("r,d,shift", ROWS)
def test_forward_and_backward_of_many_rows(r, d, shift, kind, bias, fmt):
    """The way a program runs them: what the forward pass keeps goes into the
    backward pass, several rows to a group or CTA in both."""
    g = _gen(r * d + fmt)
    x = (torch.randn((r, d), generator=g, device="cuda") * 2 + 3).to(bf16)
    w, b = 1 + 0.3 * torch.randn(d, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda")
    dy = torch.randn((r, d), generator=g, device="cuda").to(bf16)
    rms = kind == RMS
    xs = _placed(x, shift)
    out = dlm.norm_fwd(xs, w, b if bias else None, 1e-5, kind, pack=fmt)
    y, mean, rstd = ref.norm(x, w, b if bias else None, 1e-5, rms, 0.0)
    by, bm, br = ref.norm_bounds(x, w, b if bias else None, 1e-5, rms, 0.0)
    ref.assert_within(out.y, y, by, "y")
    ref.assert_within(out.rstd, rstd, rstd * br, "rstd")
    if not rms:
        ref.assert_within(out.mean, mean, bm, "mean")
    held = x
    if fmt:
        codes, scale = ref.pack(x, fmt)
        assert torch.equal(out.packed.q.cpu(), codes) and torch.equal(out.packed.scale.cpu(), scale)
        held = ref.held(codes.cuda(), scale.cuda(), fmt, torch.float64)
    got = _backward(_placed(dy, shift), xs, out.packed, out.mean, out.rstd, w, kind, bias)
    dx, dw, db = ref.norm_grad(dy, held, out.mean, out.rstd, w, rms, 0.0)
    bx, bw, bb = ref.norm_grad_tight(dy, held, out.mean, out.rstd, w, rms, 0.0, f32)
    ref.assert_within(got.d_x, dx, bx, "d_x")
    ref.assert_within(got.d_weight, dw, bw, "d_weight")
    if bias:
        ref.assert_within(got.d_bias, db, bb, "d_bias")


@pytest.mark.parametrize("kind", [LAYER, RMS])
@pytest.mark.parametrize("d", [9001, 33001])
def test_wide_rows_of_one_cta_stay_apart(d, kind):
    """Rows that one CTA takes in turn: 592 apart forward, 148 backward."""
    r = 1200 if d < 10000 else 620
    g = _gen(d)
    x = torch.randn((r, d), generator=g, device="cuda").to(bf16)
    dy = torch.randn((r, d), generator=g, device="cuda").to(bf16)
    clean = dlm.norm_fwd(x, kind=kind)
    want = dlm.norm_bwd(dy, x, clean.rstd, clean.mean, kind=kind)
    rows = torch.tensor([0, 5, 148 * 2 + 5, r - 1], device="cuda")
    bad = x.clone()
    bad[rows[::2], d - 1] = float("nan")
    bad[rows[1::2], 0] = float("inf")
    good = torch.ones(r, dtype=torch.bool, device="cuda")
    good[rows] = False
    out = dlm.norm_fwd(bad, kind=kind)
    assert torch.equal(out.y[good], clean.y[good]) and torch.equal(out.rstd[good], clean.rstd[good])
    assert bool(torch.isnan(out.y[rows[::2]]).all())
    got = dlm.norm_bwd(dy, bad, out.rstd, out.mean, kind=kind)
    assert torch.equal(got.d_x[good], want.d_x[good]) and bool(torch.isnan(got.d_x[rows[::2]]).all())
