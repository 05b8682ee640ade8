"""Embedding, norm and 8-bit activations without a GPU: what the library and
the binding refuse, valid calls that reach the device check, CUDA failures
turned into status codes, and the 64-bit forms that the GPU tests compare with,
themselves held to central differences and to the 8-bit format's own
definition."""
import ctypes
import weakref

import pytest
import torch

import diffusion_lm_loss_b200 as dlm
import train_ref as ref
from diffusion_lm_loss_b200 import build as dlm_build
from test_host_failures import _a_device_may_be_usable, _fails_at

bf16, f32 = torch.bfloat16, torch.float32
INVALID, TOO_SMALL = 1, 3


@pytest.fixture(scope="module")
def L():
    dlm_build.build()
    return dlm.lib()


# --------------------------------------------------------------------------
# the C ABI
# --------------------------------------------------------------------------
def test_embed_rejections(L):
    lay = dlm.Layout(2, 32, 64, None, None)
    p = ctypes.byref(lay)

    def fwd(layout=p, ids=16, w=16, ld_w=64, vocab=100, d=64, scale=1.0, out=16, ld_out=64):
        return L.dlm_embed_fwd(layout, ids, w, ld_w, vocab, d, scale, out, ld_out, None, None)
    for kw in (dict(layout=None), dict(layout=ctypes.byref(dlm.Layout(2, 32, 65, None, None))), dict(vocab=0), dict(d=0),
               dict(d=-8), dict(ld_w=63), dict(ld_out=63), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(ids=None), dict(w=None), dict(out=None)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(layout=ctypes.byref(dlm.Layout(2, 0, 0, None, None)), ids=None) == 0           # no tokens

    need = L.dlm_embed_bwd_workspace_size(p, 64, 100)
    assert need >= 256 + 101 * 4 + 64 * 8

    def bwd(layout=p, ids=16, dy=16, ld=64, vocab=100, d=64, scale=1.0, gt=0, acc=0, dw=16, ld_dw=64, ws=256, n=need):
        return L.dlm_embed_bwd(layout, ids, dy, ld, vocab, d, scale, gt, acc, dw, ld_dw, ws, n, None)
    for kw in (dict(layout=None), dict(vocab=0), dict(d=0), dict(ld=63), dict(ld_dw=63), dict(scale=float("nan")),
               dict(gt=2), dict(gt=-1), dict(acc=2), dict(ids=None), dict(dy=None), dict(dw=None), dict(ws=None),
               dict(ws=128)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(n=need - 1) == TOO_SMALL
    for bad in ((None, 64, 100), (p, 0, 100), (p, 64, 0), (p, 64, 2 ** 31 - 1), (p, 2 ** 31 - 1, 100)):
        assert L.dlm_embed_bwd_workspace_size(*bad) == 0
    # more blocks than a launch can have
    huge = dlm.Layout(1, 0, 2 ** 31 - 1, 16, None)
    assert L.dlm_embed_bwd(ctypes.byref(huge), 16, 16, 10 ** 6, 100, 10 ** 6, 1.0, 0, 0, 16, 10 ** 6, 256, 2 ** 62,
                           None) == INVALID


def test_pack_rejections(L):
    def pack(x=16, rows=4, cols=128, ld=128, fmt=1, q=16, s=16):
        return L.dlm_pack8(x, rows, cols, ld, fmt, q, s, None)

    def unpack(q=16, s=16, rows=4, cols=128, fmt=1, out=16, ld=128):
        return L.dlm_unpack8(q, s, rows, cols, fmt, out, ld, None)
    for kw in (dict(rows=-1), dict(cols=-1), dict(ld=127), dict(fmt=0), dict(fmt=3), dict(q=None), dict(s=None),
               dict(cols=2 ** 31 - 2, ld=2 ** 31)):
        assert pack(**kw) == INVALID, kw
        assert unpack(**kw) == INVALID, kw
    assert pack(x=None) == INVALID and unpack(out=None) == INVALID
    assert pack(rows=0, x=None) == 0 and pack(cols=0, q=None) == 0
    assert unpack(rows=0, q=None) == 0 and unpack(cols=0, out=None) == 0


def test_norm_rejections(L):
    def fwd(x=16, rows=4, d=64, ld=64, w=16, b=16, pt=0, kind=0, eps=1e-5, off=0.0, y=16, ld_y=64, mean=16, rstd=16,
            fmt=0, q=None, qs=None):
        return L.dlm_norm_fwd(x, rows, d, ld, w, b, pt, kind, eps, off, y, ld_y, mean, rstd, fmt, q, qs, None)
    nan, inf = float("nan"), float("inf")
    for kw in (dict(rows=-1), dict(rows=2 ** 31), dict(d=0), dict(ld=63), dict(ld_y=63), dict(kind=2), dict(pt=2),
               dict(eps=-1e-9), dict(eps=nan), dict(eps=inf), dict(off=nan), dict(off=inf), dict(fmt=3), dict(fmt=-1),
               dict(x=None), dict(y=None), dict(rstd=None), dict(mean=None), dict(fmt=1), dict(fmt=1, q=16),
               dict(fmt=2, qs=16)):
        assert fwd(**kw) == INVALID, kw
    assert fwd(rows=0, x=None) == 0

    need = L.dlm_norm_bwd_workspace_size(4, 64)
    assert need > 0

    def bwd(dy=16, ld_dy=64, x=16, ld_x=64, fmt=0, q=None, qs=None, mean=16, rstd=16, w=16, pt=0, kind=0, off=0.0,
            rows=4, d=64, dx=16, ld_dx=64, gt=0, acc=0, dw=16, db=16, ws=256, n=need):
        return L.dlm_norm_bwd(dy, ld_dy, x, ld_x, fmt, q, qs, mean, rstd, w, pt, kind, off, rows, d, dx, ld_dx, gt, acc,
                              dw, db, ws, n, None)
    for kw in (dict(rows=2 ** 31), dict(dy=None), dict(ld_dy=63), dict(x=None), dict(ld_x=63), dict(fmt=3), dict(fmt=1, q=16),
               dict(fmt=1, qs=16), dict(mean=None), dict(rstd=None), dict(pt=2), dict(kind=-1), dict(off=nan),
               dict(rows=-1), dict(d=0), dict(dx=None), dict(ld_dx=63), dict(gt=2), dict(acc=2), dict(ws=None),
               dict(ws=100)):
        assert bwd(**kw) == INVALID, kw
    assert bwd(n=need - 1) == TOO_SMALL
    assert L.dlm_norm_bwd_workspace_size(-1, 64) == 0 and L.dlm_norm_bwd_workspace_size(4, 0) == 0


def test_norm_workspace_holds_its_partial_rows(L):
    """The workspace grows with the rows up to what is resident at once, and
    never past it."""
    for d in (1, 64, 1000, 4096, 8192, 8193, 40000):
        sizes = [L.dlm_norm_bwd_workspace_size(r, d) for r in (0, 1, 100, 1000, 10 ** 5, 10 ** 9)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[-1] <= 148 * 64 * 2 * 4 * (d + 64)
        assert all(s % 256 == 0 and s > 0 for s in sizes)


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------
def _cpu_only(fn):
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        fn()


def test_embed_arguments():
    lay = dlm.make_layout(2, 8)
    w = torch.zeros(50, 24, dtype=bf16)
    ids = torch.zeros(16, dtype=torch.int32)
    dy = torch.zeros(16, 24, dtype=bf16)
    with pytest.raises(ValueError, match="ids: needs at least 16"):
        dlm.embed_fwd(lay, ids[:15], w)
    with pytest.raises(TypeError, match="ids"):
        dlm.embed_fwd(lay, ids.long(), w)
    with pytest.raises(TypeError, match="weight"):
        dlm.embed_fwd(lay, ids, w.float())
    with pytest.raises(ValueError, match="unit column stride"):
        dlm.embed_fwd(lay, ids, torch.zeros(24, 50, dtype=bf16).t())
    with pytest.raises(ValueError, match="rows overlap"):
        dlm.embed_fwd(lay, ids, w[:1].expand(50, 24))
    with pytest.raises(ValueError, match="vocab, d_model"):
        dlm.embed_fwd(lay, ids, w[0])
    with pytest.raises(ValueError, match="out: needs at least 16 rows"):
        dlm.embed_fwd(lay, ids, w, out=dy[:9])
    with pytest.raises(ValueError, match="out: must have 24 columns"):
        dlm.embed_fwd(lay, ids, w, out=torch.zeros(16, 32, dtype=bf16))
    with pytest.raises(ValueError, match="dev_status"):
        dlm.embed_fwd(lay, ids, w, dev_status=torch.zeros(1))
    _cpu_only(lambda: dlm.embed_fwd(lay, ids, w))
    with pytest.raises(ValueError, match="d_out: needs at least 16 rows"):
        dlm.embed_bwd(lay, ids, dy[:15], 50)
    with pytest.raises(ValueError, match="accumulate needs d_weight"):
        dlm.embed_bwd(lay, ids, dy, 50, accumulate=True)
    with pytest.raises(TypeError, match="d_weight"):
        dlm.embed_bwd(lay, ids, dy, 50, d_weight=w.half())
    with pytest.raises(ValueError, match="d_weight: needs at least 51 rows"):
        dlm.embed_bwd(lay, ids, dy, 51, d_weight=w)
    with pytest.raises(TypeError, match="grad_dtype"):
        dlm.embed_bwd(lay, ids, dy, 50, grad_dtype=torch.float16)
    with pytest.raises(TypeError, match="workspace"):
        dlm.embed_bwd(lay, ids, dy, 50, workspace=torch.zeros(10))
    with pytest.raises(ValueError, match="at least one column"):
        dlm.embed_bwd(lay, ids, dy[:, :0], 50)
    _cpu_only(lambda: dlm.embed_bwd(lay, ids, dy, 50))


def test_pack_arguments():
    x = torch.zeros(4, 200, dtype=bf16)
    with pytest.raises(ValueError, match="format"):
        dlm.pack8(x, 0)
    with pytest.raises(TypeError, match="x"):
        dlm.pack8(x.float())
    with pytest.raises(ValueError, match="2-D"):
        dlm.pack8(x[0])
    p = dlm.Packed8(torch.zeros(4, 200, dtype=torch.uint8), torch.zeros(4, 2), dlm.PACK_INT8)
    with pytest.raises(ValueError, match="another format"):
        dlm.pack8(x, dlm.PACK_E4M3, out=p)
    with pytest.raises(ValueError, match="out: q"):
        dlm.pack8(x[:, :100], out=p)
    with pytest.raises(ValueError, match="packed: q"):
        dlm.unpack8(dlm.Packed8(p.q, torch.zeros(4, 1), 1))
    with pytest.raises(ValueError, match="packed: format"):
        dlm.unpack8(dlm.Packed8(p.q, p.scale, 7))
    with pytest.raises(ValueError, match="contiguous"):
        dlm.unpack8(dlm.Packed8(torch.zeros(4, 300, dtype=torch.uint8)[:, :200], p.scale, 1))
    with pytest.raises(ValueError, match="out: must have 200 columns"):
        dlm.unpack8(p, out=torch.zeros(4, 208, dtype=bf16))
    _cpu_only(lambda: dlm.pack8(x))
    _cpu_only(lambda: dlm.unpack8(p))


def test_norm_arguments():
    x = torch.zeros(6, 72, dtype=bf16)
    w, b = torch.zeros(72), torch.zeros(72)
    r = torch.zeros(6)
    with pytest.raises(TypeError, match="one type"):
        dlm.norm_fwd(x, w, b.to(bf16))
    with pytest.raises(ValueError, match="weight: needs at least 72"):
        dlm.norm_fwd(x, w[:71])
    with pytest.raises(ValueError, match="bias: must have shape"):
        dlm.norm_fwd(x, w, torch.zeros(1, 72))
    with pytest.raises(TypeError, match="weight"):
        dlm.norm_fwd(x, w.half())
    with pytest.raises(ValueError, match="pack"):
        dlm.norm_fwd(x, pack=5)
    with pytest.raises(ValueError, match="out.mean: required"):
        dlm.norm_fwd(x, out=dlm.NormOut(x.clone(), None, r, None))
    with pytest.raises(ValueError, match="out.packed"):
        dlm.norm_fwd(x, pack=1, out=dlm.NormOut(x.clone(), r, r.clone(), None))
    _cpu_only(lambda: dlm.norm_fwd(x, w, b))
    with pytest.raises(ValueError, match="mean: required"):
        dlm.norm_bwd(x, x, r, None, w)
    with pytest.raises(ValueError, match="rstd: needs at least 6"):
        dlm.norm_bwd(x, x, r[:5], r, w)
    with pytest.raises(ValueError, match="x: must have 72 columns"):
        dlm.norm_bwd(x, torch.zeros(6, 80, dtype=bf16), r, r, w)
    with pytest.raises(ValueError, match="rows overlap"):
        dlm.norm_bwd(x[:1].expand(6, 72), x, r, r, w)
    with pytest.raises(ValueError, match="x: q"):
        dlm.norm_bwd(x, dlm.Packed8(torch.zeros(6, 64, dtype=torch.uint8), torch.zeros(6, 1), 1), r, r, w)
    with pytest.raises(ValueError, match="accumulate needs"):
        dlm.norm_bwd(x, x, r, r, w, accumulate=True)
    with pytest.raises(ValueError, match="d_bias: must have shape"):
        dlm.norm_bwd(x, x, r, r, w, d_bias=torch.zeros(71))
    with pytest.raises(TypeError, match="d_bias: expected"):
        dlm.norm_bwd(x, x, r, r, w, d_weight=w, d_bias=b.to(bf16))
    with pytest.raises(ValueError, match="d_x: needs at least 6 rows"):
        dlm.norm_bwd(x, x, r, r, w, d_x=x[:3])
    _cpu_only(lambda: dlm.norm_bwd(x, x, r, r, w))


def test_an_expanded_or_transposed_gradient_becomes_rows():
    for t in (torch.ones(1).expand(3, 4), torch.zeros(4, 3).t(), torch.zeros(1, 4).expand(3, 4)):
        r = dlm._as_rows(t)
        assert r.is_contiguous() and torch.equal(r, t)
    t = torch.zeros(3, 8)[:, :4]
    assert dlm._as_rows(t) is t


def test_valid_calls_pass_host_checks(L, monkeypatch):
    if _a_device_may_be_usable():
        pytest.skip("the calls below carry CPU pointers")
    monkeypatch.setattr(dlm, "_on_cuda", lambda **kw: None)
    monkeypatch.setattr(dlm, "_stream", lambda: None)
    lay = dlm.make_layout(2, 8)
    ids = torch.zeros(16, dtype=torch.int32)
    w = torch.zeros(50, 24, dtype=bf16)
    x = torch.zeros(16, 32, dtype=bf16)[:, :24]
    r = torch.zeros(16)
    p = dlm._empty_packed(16, 24, 2, "cpu")
    for fn in (lambda: dlm.embed_fwd(lay, ids, w, 2.0, out=x), lambda: dlm.embed_bwd(lay, ids, x, 50),
               lambda: dlm.embed_bwd(lay, ids, x, 50, d_weight=w, accumulate=True),
               lambda: dlm.pack8(x), lambda: dlm.unpack8(p, out=x), lambda: dlm.norm_fwd(x, w[0], pack=2),
               lambda: dlm.norm_fwd(x, kind=dlm.NORM_RMS), lambda: dlm.norm_bwd(x, p, r, r, w[0], want_d_bias=True),
               lambda: dlm.norm_bwd(x, x, r, kind=dlm.NORM_RMS, d_weight=r[:0].new_zeros(24), accumulate=True)):
        with pytest.raises(dlm.DlmError) as e:
            fn()
        assert e.value.code in (2, 4), e.value                 # stopped at the device check, nothing earlier


def test_cuda_failures_are_reported(L):
    if _a_device_may_be_usable():
        pytest.skip("a CUDA device may be usable here: the hook must not run with fake pointers")
    lay = dlm.Layout(2, 32, 64, None, None)
    p = ctypes.byref(lay)
    ws = 1 << 20
    assert L.dlm_test_skip_device_check(1) == 0
    try:
        for _ in range(2):
            _fails_at(L, L.dlm_embed_fwd(p, 256, 512, 64, 100, 64, 1.0, 1024, 64, None, None), "k_embed_fwd launch")
            n = L.dlm_embed_bwd_workspace_size(p, 64, 100)
            _fails_at(L, L.dlm_embed_bwd(p, 256, 512, 64, 100, 64, 1.0, 0, 0, 1024, 64, ws, n, None), "k_embed_small launch")
            big = 1 << 22                                       # a table too large for the single launch
            n = L.dlm_embed_bwd_workspace_size(p, 64, big)
            _fails_at(L, L.dlm_embed_bwd(p, 256, 512, 64, big, 64, 1.0, 0, 0, 1024, 64, ws, n, None), "k_embed_sort")
            _fails_at(L, L.dlm_pack8(256, 4, 128, 128, 1, 512, 1024, None), "k_pack8 launch")
            _fails_at(L, L.dlm_unpack8(256, 512, 4, 128, 2, 1024, 128, None), "k_unpack8 launch")
            for d, step in ((64, "k_norm_fwd launch"), (40001, "k_norm_fwd_wide launch")):
                _fails_at(L, L.dlm_norm_fwd(256, 4, d, d, None, None, 0, 0, 1e-5, 0.0, 512, d, 1024, 2048, 0, None,
                                            None, None), step)
            for d, step in ((64, "k_norm_bwd launch"), (40001, "k_norm_bwd_wide launch")):
                n = L.dlm_norm_bwd_workspace_size(4, d)
                _fails_at(L, L.dlm_norm_bwd(256, d, 512, d, 0, None, None, 768, 1024, None, 0, 0, 0.0, 4, d, 2048, d,
                                            0, 0, 4096, None, ws, n, None), step)
            n = L.dlm_norm_bwd_workspace_size(0, 64)
            _fails_at(L, L.dlm_norm_bwd(None, 64, None, 64, 0, None, None, None, None, None, 0, 0, 0.0, 0, 64, None,
                                        64, 0, 0, 4096, None, ws, n, None), "k_norm_join launch")
    finally:
        assert L.dlm_test_skip_device_check(0) == 0


# --------------------------------------------------------------------------
# the 64-bit forms
# --------------------------------------------------------------------------
@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradient_is_the_difference_quotient(rms):
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn((4, 9), generator=g, dtype=torch.float64) for _ in range(2))
    w, b = (torch.randn(9, generator=g, dtype=torch.float64) for _ in range(2))
    _, mean, rstd = ref.norm(x, w, b, 1e-3, rms, 1.0)
    dx, dw, db = ref.norm_grad(dy, x, mean, rstd, w, rms, 1.0)

    def loss(x_, w_, b_):
        return float((ref.norm(x_, w_, b_, 1e-3, rms, 1.0)[0] * dy).sum())
    h = 1e-5
    for t, grad in ((x, dx), (w, dw), (b, db)):
        flat = t.view(-1)
        for k in range(flat.numel()):
            keep = flat[k].item()
            flat[k] = keep + h
            up = loss(x, w, b)
            flat[k] = keep - h
            down = loss(x, w, b)
            flat[k] = keep
            assert abs((up - down) / (2 * h) - grad.reshape(-1)[k].item()) < 1e-7


def test_embedding_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(2)
    w, dy = torch.randn((5, 3), generator=g, dtype=torch.float64), torch.randn((7, 3), generator=g, dtype=torch.float64)
    ids = torch.tensor([1, 4, 1, 0, 1, 4, 2], dtype=torch.int32)
    pad = torch.tensor([0, 0, 1, 0, 0, 0, 0], dtype=torch.uint8)
    dw, mag = ref.embed_grad(ids, dy, 5, 3.0, pad)
    for k in range(15):
        e = torch.zeros(15, dtype=torch.float64)
        e[k] = 1.0
        # the embedding is linear: the quotient is exact for any step
        want = float((ref.embed(ids, e.view(5, 3), 3.0, pad) * dy).sum())
        assert abs(want - dw.view(-1)[k].item()) < 1e-14 and mag.view(-1)[k] >= abs(want) - 1e-14
    assert not dw[3].any()


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_8_bit_form_takes_the_nearest_code(fmt):
    """Against all codes of the format: none is nearer to x / scale than the
    one taken, but for the rounding of x * inv."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn((3, 200), generator=g) * 5).to(bf16)
    q, s = ref.pack(x, fmt)
    held = ref.held(q, s, fmt).double()
    every = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    v = (every.view(torch.int8).double() if fmt == ref.INT8 else every.view(torch.float8_e4m3fn).double())
    v = v[torch.isfinite(v)]
    step = s.double().repeat_interleave(128, 1)[:, :200]
    best = (x.double()[:, :, None] - v * step[:, :, None]).abs().amin(2)
    assert bool(((x.double() - held).abs() <= best + step * 2.0 ** -14).all())
    top = 127 if fmt == ref.INT8 else 448
    for k in range(2):                                          # a block's largest element is its end code
        blk = x[:, 128 * k:128 * k + 128].float().abs()
        at = blk.argmax(1)
        assert torch.allclose(held[:, 128 * k:128 * k + 128].abs().gather(1, at[:, None])[:, 0],
                              s[:, k].double() * top, rtol=2.0 ** -20)


def test_bounds_refuse_planted_mistakes():
    """The GPU tests' bounds, on the CPU, against mistakes in the oracle: a
    dropped token, a missing term of dx, the variance about zero, a bias left
    out, a scale used twice."""
    g = torch.Generator().manual_seed(4)
    x = (torch.randn((20, 264), generator=g) + 1).to(bf16)
    dy = torch.randn((20, 264), generator=g).to(bf16)
    w, b = torch.randn(264, generator=g), torch.randn(264, generator=g)
    y, mean, rstd = ref.norm(x, w, b, 1e-5, False, 0.0)
    by, _, _ = ref.norm_bounds(x, w, b, 1e-5, False, 0.0)
    ref.assert_within(y.to(bf16), y, by)

    def refused(got, want, bound):
        with pytest.raises(AssertionError):
            ref.assert_within(got, want, bound)
    refused(ref.norm(x, w, b, 1e-5, True, 0.0)[0].to(bf16), y, by)
    refused(ref.norm(x, w, None, 1e-5, False, 0.0)[0].to(bf16), y, by)
    refused((y * (1 + 2.0 ** -6)).to(bf16), y, by)
    dx, dw, db = ref.norm_grad(dy, x, mean, rstd, w, False, 0.0)
    bx, bw, bb = ref.norm_grad_bounds(dy, x, mean, rstd, w, False, 0.0, f32)
    ref.assert_within(dx.to(bf16), dx, bx)
    ref.assert_within(dw.float(), dw, bw)
    refused(ref.norm_grad(dy, x, mean, rstd, w, True, 0.0)[0].to(bf16), dx, bx)
    part = ref.norm_grad(dy[1:], x[1:], mean[1:], rstd[1:], w, False, 0.0)
    refused(part[1].float(), dw, bw)
    refused(part[2].float(), db, bb)
    ids = torch.randint(0, 9, (20,), generator=g, dtype=torch.int32)
    de, mag = ref.embed_grad(ids, dy, 9, 2.0)
    be = ref.embed_grad_bound(ids, de, mag, bf16)
    ref.assert_within(de.to(bf16), de, be)
    refused(ref.embed_grad(ids[1:], dy[1:], 9, 2.0)[0].to(bf16), de, be)
    refused(ref.embed_grad(ids, dy, 9, 4.0)[0].to(bf16), de, be)


def test_no_second_workspace_is_asked_for_while_one_is_held(monkeypatch):
    """The buffers are several GB for the fused head: one request for it, and
    for the others never two buffers alive at once, whatever the allocator
    returns."""
    empty, alive, asked, most = torch.empty, [], [], []

    def off_border(n, *stride, **kw):
        n = n[0] if stride else n                    # empty_strided((n,), (1,)) or empty(n)
        buf = empty(n + 8192, **kw)
        at = (-buf.data_ptr()) % 4096 + 16           # on a 16-byte border only
        buf = buf[at:at + n]
        alive.append(weakref.ref(buf))
        asked.append(n)
        most.append(sum(r() is not None for r in alive[:-1]))
        return buf
    monkeypatch.setattr(torch, "empty", off_border)
    monkeypatch.setattr(torch, "empty_strided", off_border)
    for align, requests in ((1024, 1), (256, 2)):
        alive.clear(), asked.clear(), most.clear()
        ws = dlm._aligned_workspace(5000, "cpu", align)
        assert ws.numel() == 5000 and ws.data_ptr() % align == 0
        assert len(asked) == requests and max(most) == 0


def test_widths_that_would_pass_32_bits_are_refused(L):
    """Both passes count columns in 32 bits, in steps of up to 1,024."""
    lay = dlm.Layout(1, 4, 4, None, None)
    p = ctypes.byref(lay)
    for d in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 1024):
        assert L.dlm_embed_fwd(p, 16, 16, d, 4, d, 1.0, 16, d, None, None) == INVALID
        assert L.dlm_embed_bwd_workspace_size(p, d, 4) == 0
        assert L.dlm_embed_bwd(p, 16, 16, d, 4, d, 1.0, 0, 0, 16, d, 256, 2 ** 62, None) == INVALID
        assert L.dlm_norm_bwd_workspace_size(4, d) == 0
