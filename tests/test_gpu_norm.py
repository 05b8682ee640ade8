"""Layer norm and RMS norm on the GPU, forward and backward, against 64-bit
forms with bounds counted from the roundings: widths around the kernels'
splits, strides and alignment, parameter and gradient types, the 8-bit
checkpoint, rows with NaN, constant rows, streams and graphs, autograd."""
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


def _make(r, d, param, offset, seed, shift=3.0):
    g = _gen(seed)
    x = (torch.randn((r, d), generator=g, device="cuda") * 2 + shift).to(bf16)
    w = (1 - offset + 0.3 * torch.randn(d, generator=g, device="cuda")).to(param)
    b = (0.5 * torch.randn(d, generator=g, device="cuda")).to(param)
    dy = torch.randn((r, d), generator=g, device="cuda").to(bf16)
    return x, w, b, dy


def _placed(t, ld, shift=0):
    r, d = t.shape
    buf = torch.full((r * ld + shift + 8,), 7.0, dtype=t.dtype, device=t.device)
    v = buf[shift:shift + r * ld].view(r, ld)[:, :d]
    v.copy_(t)
    return v


def _check_fwd(out, x, w, b, eps, rms, offset):
    y, mean, rstd = ref.norm(x, w, b, eps, rms, offset)
    by, bm, br = ref.norm_bounds(x, w, b, eps, rms, offset)
    ref.assert_within(out.rstd, rstd, rstd * br, "rstd")
    if rms:
        assert out.mean is None
    else:
        ref.assert_within(out.mean, mean, bm, "mean")
    ref.assert_within(out.y, y, by, "y")


def _check_bwd(got, dy, x, mean, rstd, w, rms, offset, dtype, weight=True, bias=True):
    dx, dw, db = ref.norm_grad(dy, x, mean, rstd, w, rms, offset)
    bx, bw, bb = ref.norm_grad_bounds(dy, x, mean, rstd, w, rms, offset, dtype)
    ref.assert_within(got.d_x, dx, bx, "d_x")
    assert (got.d_weight is not None) == weight and (got.d_bias is not None) == bias
    if weight:
        assert got.d_weight.dtype == dtype
        ref.assert_within(got.d_weight, dw, bw, "d_weight")
    if bias:
        ref.assert_within(got.d_bias, db, bb, "d_bias")


WIDTHS = [1, 7, 8, 64, 129, 256, 264, 520, 1003, 1024, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 8193, 16384, 32776, 40000]


@pytest.mark.parametrize("kind", [LAYER, RMS])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_and_backward_widths(d, kind):
    r = 5 if d > 1000 else 37
    param, offset = (f32, 1.0) if d % 3 == 0 else (bf16, 0.0)
    x, w, b, dy = _make(r, d, param, offset, d)
    out = dlm.norm_fwd(x, w, b, 1e-5, kind, offset)
    _check_fwd(out, x, w, b, 1e-5, kind == RMS, offset)
    dtype = f32 if d % 2 else bf16
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, kind, offset, want_d_bias=True, grad_dtype=dtype)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, kind == RMS, offset, dtype)
    again = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, kind, offset, want_d_bias=True, grad_dtype=dtype,
                         workspace=got.workspace.fill_(0xA5))
    assert torch.equal(again.d_x, got.d_x) and torch.equal(again.d_weight, got.d_weight)
    assert torch.equal(again.d_bias, got.d_bias)


@pytest.mark.parametrize("r", [1, 2, 3, 147, 149, 297, 600, 3001])
@pytest.mark.parametrize("d", [40, 512, 1001])
def test_row_counts(r, d):
    x, w, b, dy = _make(r, d, bf16, 0.0, r)
    out = dlm.norm_fwd(x, w, b)
    _check_fwd(out, x, w, b, 1e-5, False, 0.0)
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_bias=True, grad_dtype=f32)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, f32)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d", [256, 264, 512, 520, 1288, 2560, 3336, 4104, 4608, 5120, 6144, 6152, 7168])
def test_many_rows_either_side_of_the_split_rules(d, fmt):
    """One, two and three pieces a lane, every number of warps up to 8, and
    widths that fill the last warp or leave most of it without work; one row
    short of and past the size from which the rings take over."""
    for r in (-(-148 * 4608 * 8 // d) - 1, -(-148 * 4608 * 8 // d) + 41):
        x, w, b, dy = _make(r, d, bf16, 0.0, d + fmt)
        kind = RMS if d % 3 == 1 else LAYER
        out = dlm.norm_fwd(x, w, b, 1e-5, kind, pack=fmt)
        _check_fwd(out, x, w, b, 1e-5, kind == RMS, 0.0)
        if fmt:
            q, s = ref.pack(x, fmt)
            assert torch.equal(out.packed.q.cpu(), q) and torch.equal(out.packed.scale.cpu(), s)
        # backward, an odd and an even number of rows for each group
        for n in (r, 148 * 3 + 1, 148 * 2, 2, 1):
            got = dlm.norm_bwd(dy[:n], x[:n], out.rstd[:n], None if kind == RMS else out.mean[:n], w, kind,
                               want_d_bias=kind == LAYER, grad_dtype=f32)
            _check_bwd(got, dy[:n], x[:n], None if kind == RMS else out.mean[:n], out.rstd[:n], w, kind == RMS, 0.0, f32,
                       bias=kind == LAYER)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d", [65, 500, 1501, 2001, 3003, 5001, 8100])
def test_many_rows_off_the_16_byte_borders(d, fmt):
    """Rows in step with one another but not with the borders, several to a
    group of warps, whose rows must keep one phase."""
    r = 1300 if d > 1000 else 5000
    x, w, b, dy = _make(r, d, f32 if d % 2 else bf16, 0.0, d + fmt)
    x[r // 2] = float("inf")                  # a neighbour's infinities stay out
    out = dlm.norm_fwd(x, w, b, pack=fmt)
    ok = torch.ones(r, dtype=torch.bool, device="cuda")
    ok[r // 2] = False
    sub = dlm.NormOut(out.y[ok], out.mean[ok], out.rstd[ok], None)
    _check_fwd(sub, x[ok], w, b, 1e-5, False, 0.0)
    x[r // 2] = 1.0
    out = dlm.norm_fwd(x, w, b, pack=fmt)
    got = dlm.norm_bwd(dy, out.packed if fmt else x, out.rstd, out.mean, w, want_d_bias=True, grad_dtype=f32)
    held = ref.held(*ref.pack(x, fmt), fmt, torch.float64).cuda() if fmt else x
    _check_bwd(got, dy, held, out.mean, out.rstd, w, False, 0.0, f32)


@pytest.mark.parametrize("fmt", [0, 1, 2])
@pytest.mark.parametrize("d", [1, 8, 65, 129, 256, 264, 500, 1003, 2048, 2056, 4096, 4104, 5001, 5120, 6144, 6152, 8192])
@pytest.mark.parametrize("r", [1, 2, 30, 150, 1301])
def test_rms_without_a_bias(r, d, fmt):
    x, w, _, dy = _make(r, d, f32 if d % 2 else bf16, 0.0, d + r + fmt, shift=0.5)
    out = dlm.norm_fwd(x, w, None, 1e-6, RMS, pack=fmt)
    _check_fwd(out, x, w, None, 1e-6, True, 0.0)
    got = dlm.norm_bwd(dy, out.packed if fmt else x, out.rstd, None, w, RMS, grad_dtype=f32)
    held = ref.held(*ref.pack(x, fmt), fmt, torch.float64).cuda() if fmt else x
    _check_bwd(got, dy, held, None, out.rstd, w, True, 0.0, f32, bias=False)
    old = torch.randn(d, device="cuda")
    acc = dlm.norm_bwd(dy, out.packed if fmt else x, out.rstd, None, w, RMS, d_weight=old.clone(), accumulate=True)
    assert torch.equal(acc.d_x, got.d_x) and torch.equal(acc.d_weight, old + got.d_weight)


@pytest.mark.parametrize("d,ld", [(1000, 1003), (1001, 1001), (264, 264), (77, 85)])
@pytest.mark.parametrize("shift", [0, 1, 8])
@pytest.mark.parametrize("r", [1, 2, 400])
def test_rows_in_and_out_of_step(r, d, ld, shift):
    """x, y, dy, dx in one stride (in step), and y, dx in another (out of step)."""
    x, w, b, dy = _make(r, d, f32, 0.0, ld + shift + r)
    for other in (ld, ld + 1):
        xs, dys = _placed(x, ld, shift), _placed(dy, ld, shift)
        y, dx = _placed(x * 0, other, shift), _placed(x * 0, other, shift)
        out = dlm.norm_fwd(xs, w, b, out=dlm.NormOut(y, torch.empty(r, device="cuda"), torch.empty(r, device="cuda"), None))
        _check_fwd(out, x, w, b, 1e-5, False, 0.0)
        got = dlm.norm_bwd(dys, xs, out.rstd, out.mean, w, want_d_bias=True, d_x=dx, grad_dtype=f32)
        _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, f32)
        for v in (y, dx):
            v.fill_(7.0)
            assert bool((v._base == 7.0).all()), "wrote outside its columns"


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("r,d", [(1, 4096), (2, 4096), (4, 4096), (5, 4096), (7, 1001), (16, 256), (32, 256), (33, 256)])
def test_accumulate_with_few_rows(r, d, dtype):
    """One CTA that writes the gradients itself, and the first size with two
    launches, both ways of writing."""
    x, w, b, dy = _make(r, d, bf16, 0.0, r)
    out = dlm.norm_fwd(x, w, b)
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_bias=True, grad_dtype=dtype)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, dtype)
    old = torch.randn(d, device="cuda").to(dtype)
    dw, db = old.clone(), old.clone()
    dlm.norm_bwd(dy, x, out.rstd, out.mean, w, d_weight=dw, d_bias=db, accumulate=True)
    _, ew, eb = ref.norm_grad(dy, x, out.mean, out.rstd, w, False, 0.0)
    _, bw, bb = ref.norm_grad_bounds(dy, x, out.mean, out.rstd, w, False, 0.0, f32)
    for g, e, bound in ((dw, ew, bw), (db, eb, bb)):
        want = old.double() + e
        # the sum's own error, one fp32 addition, the output's rounding
        ref.assert_within(g, want, bound + 1.01 * (ref.HALF[dtype] * want.abs() + ref.U * (want.abs() + bound)))


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("kind", [LAYER, RMS])
@pytest.mark.parametrize("r,d", [(3, 8), (37, 200), (9, 1001), (150, 4096), (300, 520), (5, 8200), (2, 40000), (2, 9001)])
def test_checkpoint_in_8_bits(r, d, kind, fmt):
    x, w, b, dy = _make(r, d, f32, 0.0, d + fmt)
    out = dlm.norm_fwd(x, w, b, 1e-6, kind, pack=fmt)
    plain = dlm.norm_fwd(x, w, b, 1e-6, kind)
    assert torch.equal(out.y, plain.y) and torch.equal(out.rstd, plain.rstd)
    apart = dlm.pack8(x, fmt)
    assert torch.equal(out.packed.q, apart.q) and torch.equal(out.packed.scale, apart.scale)
    q, s = ref.pack(x, fmt)
    held = ref.held(q, s, fmt, torch.float64).cuda()
    got = dlm.norm_bwd(dy, out.packed, out.rstd, out.mean, w, kind, want_d_bias=True)
    # x is the held value code * scale, unrounded by definition
    _check_bwd(got, dy, held, out.mean, out.rstd, w, kind == RMS, 0.0, f32)


@pytest.mark.parametrize("ld,shift", [(264, 0), (257, 0), (256, 1), (256, 4), (264, 8)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_strides_and_alignment(ld, shift, fmt):
    r, d = 23, 256
    x, w, b, dy = _make(r, d, bf16, 0.0, ld + shift)
    xs, dys = _placed(x, ld, shift), _placed(dy, ld, shift)
    y, dx = _placed(x * 0, ld, shift), _placed(x * 0, ld, shift)
    want = dlm.norm_fwd(x, w, b, pack=fmt)
    pk = dlm._empty_packed(r, d, fmt, x.device) if fmt else None
    out = dlm.norm_fwd(xs, w, b, pack=fmt, out=dlm.NormOut(y, torch.empty(r, device="cuda"), torch.empty(r, device="cuda"), pk))
    assert out.y.data_ptr() == y.data_ptr()
    _check_fwd(out, x, w, b, 1e-5, False, 0.0)
    if fmt:
        assert torch.equal(out.packed.q, want.packed.q) and torch.equal(out.packed.scale, want.packed.scale)
    got = dlm.norm_bwd(dys, out.packed if fmt else xs, out.rstd, out.mean, w, want_d_bias=True, d_x=dx, grad_dtype=f32)
    held = ref.held(*ref.pack(x, fmt), fmt, torch.float64).cuda() if fmt else x
    _check_bwd(got, dy, held, out.mean, out.rstd, w, False, 0.0, f32)
    for v in (y, dx):
        v.fill_(7.0)
        assert bool((v._base == 7.0).all()), "wrote outside its columns"


@pytest.mark.parametrize("shift", [1, 2])
def test_parameters_not_on_16_byte_borders(shift):
    x, w, b, dy = _make(9, 512, f32, 0.0, 1)
    ws = torch.zeros(512 + shift, device="cuda")[shift:]
    bs = torch.zeros(512 + shift, device="cuda")[shift:]
    ws.copy_(w), bs.copy_(b)
    out = dlm.norm_fwd(x, ws, bs)
    _check_fwd(out, x, w, b, 1e-5, False, 0.0)
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, ws, want_d_bias=True)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, f32)


@pytest.mark.parametrize("d", [256, 1003, 9001])
def test_optional_parameters_and_gradients(d):
    x, w, b, dy = _make(30, d, bf16, 0.0, d)
    for ww, bb in ((None, None), (w, None), (None, b)):
        out = dlm.norm_fwd(x, ww, bb, weight_offset=1.0)       # the offset belongs to a weight
        _check_fwd(out, x, ww, bb, 1e-5, False, 1.0)
        got = dlm.norm_bwd(dy, x, out.rstd, out.mean, ww, weight_offset=1.0)
        _check_bwd(got, dy, x, out.mean, out.rstd, ww, False, 1.0, bf16, weight=ww is not None, bias=False)
    only_b = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_weight=False, want_d_bias=True)
    _check_bwd(only_b, dy, x, out.mean, out.rstd, w, False, 0.0, bf16, weight=False)
    none = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_weight=False)
    _check_bwd(none, dy, x, out.mean, out.rstd, w, False, 0.0, bf16, weight=False, bias=False)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_accumulate_and_no_rows(dtype):
    x, w, b, dy = _make(100, 136, bf16, 0.0, 5)
    out = dlm.norm_fwd(x, w, b)
    fresh = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_bias=True, grad_dtype=f32)
    old = torch.randn(136, device="cuda").to(dtype)
    dw, db = old.clone(), old.clone()
    dlm.norm_bwd(dy, x, out.rstd, out.mean, w, d_weight=dw, d_bias=db, accumulate=True)
    for got, add in ((dw, fresh.d_weight), (db, fresh.d_bias)):
        want = old.double() + add.double()
        ref.assert_within(got, want, ref.HALF[dtype] * want.abs() + ref.U * (old.double().abs() + add.double().abs()))
    empty = dlm.norm_bwd(dy[:0], x[:0], out.rstd[:0], out.mean[:0], w, want_d_bias=True, grad_dtype=dtype)
    assert not empty.d_weight.any() and not empty.d_bias.any() and empty.d_x.shape == (0, 136)
    dlm.norm_bwd(dy[:0], x[:0], out.rstd[:0], out.mean[:0], w, d_weight=dw, accumulate=True)
    assert torch.equal(dw, (old.float() + fresh.d_weight).to(dtype)) or dtype == f32
    assert dlm.norm_fwd(x[:0], w, b).y.shape == (0, 136)


def test_a_mean_far_from_zero_and_constant_rows():
    """Centred squares: a mean of 300 times the deviation costs no more than
    the inputs' own rounding; a constant row is all bias."""
    x, w, b, dy = _make(20, 4096, f32, 0.0, 8, shift=600.0)
    x[3] = 5.0
    out = dlm.norm_fwd(x, w, b)
    _check_fwd(out, x, w, b, 1e-5, False, 0.0)
    assert torch.equal(out.y[3], b.to(bf16)) and out.mean[3] == 5.0
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, w, want_d_bias=True)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, f32)


@pytest.mark.parametrize("d", [512, 1001, 9000])
def test_nan_and_infinity_stay_in_their_row(d):
    x, w, b, dy = _make(12, d, bf16, 0.0, 9)
    x[4, 7] = float("nan")
    x[6, 1] = float("inf")
    out = dlm.norm_fwd(x, w, b, pack=dlm.PACK_INT8)
    good = torch.ones(12, dtype=torch.bool, device="cuda")
    good[4] = good[6] = False
    assert bool(torch.isfinite(out.y[good]).all())
    assert bool(torch.isnan(out.y[4]).all()) and bool(torch.isnan(out.rstd[4]))
    got = dlm.norm_bwd(dy, x, out.rstd, out.mean, w)
    assert bool(torch.isfinite(got.d_x[good]).all()) and bool(torch.isnan(got.d_x[4]).all())


@pytest.mark.parametrize("kind", [LAYER, RMS])
@pytest.mark.parametrize("d", [256, 1024, 4096, 5001, 5120, 6144, 8192])
def test_nan_and_infinity_stay_in_their_row_of_many(d, kind):
    """Rows that share a turn, an exchange of sums and a chunk of memory with
    one that is not finite."""
    r = -(-148 * 4608 * 8 // d) + 5
    x, w, _, dy = _make(r, d, bf16, 0.0, 9)
    rows = torch.tensor([0, 148, 149, 296, r // 2, r - 1], device="cuda")
    clean = dlm.norm_fwd(x, w, None, kind=kind)
    want = dlm.norm_bwd(dy, x, clean.rstd, clean.mean, w, kind)
    bad = x.clone()
    bad[rows[::2], d - 1] = float("nan")
    bad[rows[1::2], 0] = float("inf")
    good = torch.ones(r, dtype=torch.bool, device="cuda")
    good[rows] = False
    out = dlm.norm_fwd(bad, w, None, kind=kind)
    assert torch.equal(out.y[good], clean.y[good]) and torch.equal(out.rstd[good], clean.rstd[good])
    assert bool(torch.isnan(out.y[rows[::2]]).all())
    got = dlm.norm_bwd(dy, bad, out.rstd, out.mean, w, kind)
    assert torch.equal(got.d_x[good], want.d_x[good])
    assert bool(torch.isnan(got.d_x[rows[::2]]).all()) and bool(torch.isnan(got.d_weight[d - 1]))


def test_rows_past_two_to_the_31_elements():
    ld = 2 ** 30 + 8
    buf = torch.zeros(2 * ld + 512, dtype=bf16, device="cuda")
    x, w, b, dy = _make(3, 512, bf16, 0.0, 2)
    v = torch.as_strided(buf, (3, 512), (ld, 1))
    v.copy_(x)
    out = dlm.norm_fwd(v, w, b)
    _check_fwd(out, x, w, b, 1e-5, False, 0.0)
    got = dlm.norm_bwd(dy, v, out.rstd, out.mean, w, d_x=None, want_d_bias=True)
    _check_bwd(got, dy, x, out.mean, out.rstd, w, False, 0.0, bf16)
    dlm.norm_bwd(dy, x, out.rstd, out.mean, w, d_x=v)
    assert torch.equal(v, got.d_x)


def test_streams_and_graph():
    g = [_make(700, 1000, bf16, 0.0, k) for k in range(2)]

    def step(x, w, b, dy):
        o = dlm.norm_fwd(x, w, b, pack=dlm.PACK_INT8)
        n = dlm.norm_bwd(dy, o.packed, o.rstd, o.mean, w, want_d_bias=True)
        return o.y, n.d_x, n.d_weight, n.d_bias

    want = [step(*a) for a in g]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = step(*g[k])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    static = [t.clone() for t in g[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*static)
    for k in (1, 0):
        for s, t in zip(static, g[k]):
            s.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[k]))


@pytest.mark.parametrize("keep8", [0, 1, 2])
@pytest.mark.parametrize("kind", [LAYER, RMS])
def test_autograd(kind, keep8):
    x, w, b, dy = _make(50, 264, bf16, 0.0, 11)
    bias = b if kind == LAYER else None
    out = dlm.norm_fwd(x, w, bias, 1e-6, kind, pack=keep8)
    want = dlm.norm_bwd(dy, out.packed if keep8 else x, out.rstd, out.mean, w, kind, want_d_bias=bias is not None)
    xs, ws = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    bs = None if bias is None else b.clone().requires_grad_(True)
    y = dlm.norm(xs, ws, bs, 1e-6, kind, keep8=keep8)
    assert torch.equal(y, out.y)
    y.backward(dy, retain_graph=True)
    assert torch.equal(xs.grad, want.d_x) and torch.equal(ws.grad, want.d_weight)
    if bs is not None:
        assert torch.equal(bs.grad, want.d_bias)
    xs.grad = None
    (y * 1.0).sum().backward()                       # an expanded upstream gradient
    ones = dlm.norm_bwd(torch.ones_like(dy), out.packed if keep8 else x, out.rstd, out.mean, w, kind)
    assert torch.equal(xs.grad, ones.d_x)
    # frozen parameters; a bias without a weight
    xs.grad = ws.grad = None
    dlm.norm(xs, w, None, 1e-6, kind, keep8=keep8).backward(dy)
    assert torch.equal(xs.grad, want.d_x) and w.grad is None
    only = b.clone().requires_grad_(True)
    dlm.norm(x, None, only, 1e-6, kind, keep8=keep8).backward(dy)
    ref.assert_within(only.grad, dy.double().sum(0), ref.HALF[bf16] * dy.double().sum(0).abs() * 1.01 +
                      58 * ref.U * dy.double().abs().sum(0))


def test_autograd_refuses_an_input_changed_in_place():
    x, w, b, dy = _make(8, 64, bf16, 0.0, 12)
    z = x.clone().requires_grad_(True) * 1.0
    y = dlm.norm(z, w, b)
    z.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy)
