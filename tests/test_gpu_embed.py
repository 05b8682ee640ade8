"""Embedding and its gradient on the GPU against 64-bit forms: sizes and
strides around the kernels' tiles and chunks, ids that all agree or never do,
pads, ids outside the table, the accumulate option, streams and graphs."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

dlm = pytest.importorskip("diffusion_lm_loss_b200")
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dlm.lib()


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype=bf16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _placed(t, ld, shift=0):
    """t's values in rows of stride ld that start `shift` elements into a buffer."""
    r, d = t.shape
    buf = torch.full((r * ld + shift + 8,), 7.0, dtype=t.dtype, device=t.device)
    v = buf[shift:shift + r * ld].view(r, ld)[:, :d]
    v.copy_(t)
    return v


def _ids(kind, t, vocab, g):
    if kind == "one":                       # every token the same id
        return torch.full((t,), vocab // 2, dtype=torch.int32, device="cuda")
    if kind == "last":
        return torch.full((t,), vocab - 1, dtype=torch.int32, device="cuda")
    ids = torch.randint(0, vocab, (t,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "masked":                    # absorbing noise: half of the tokens the mask id
        hit = torch.rand(t, generator=g, device="cuda") < 0.5
        ids = torch.where(hit, torch.full_like(ids, vocab - 1), ids)
    if kind == "runs":                      # rows of 20 to 70 tokens: they cross chunk borders in every way
        ids = (torch.arange(t, device="cuda", dtype=torch.int32) * 7919 // 45) % vocab
    return ids.contiguous()


@pytest.mark.parametrize("t,vocab,d,ldw,ldo,shift", [
    (1, 1, 1, 1, 1, 0), (1, 5, 8, 8, 8, 0), (5, 7, 1001, 1001, 1001, 0), (130, 1024, 256, 256, 256, 0),
    (64, 333, 1000, 1008, 1016, 0), (64, 333, 1000, 1001, 1003, 0), (33, 100, 4096, 4096, 4096, 1),
    (257, 5000, 4104, 4104, 4104, 0), (700, 50, 24, 24, 24, 0), (9, 30, 1023, 1023, 1025, 0), (9, 30, 1025, 1027, 1025, 3),
    (40, 30, 2047, 2047, 2047, 0), (40, 30, 2049, 2051, 2050, 5), (6, 7, 1024, 1024, 1024, 7), (6, 7, 263, 265, 270, 2)])
@pytest.mark.parametrize("scale", [1.0, 31.625])
def test_forward(t, vocab, d, ldw, ldo, shift, scale):
    g = _gen(t + d)
    w = _placed(_randn((vocab, d), g), ldw, shift)
    ids = _ids("rand", t, vocab, g)
    pad = (torch.rand(t, generator=g, device="cuda") < 0.3).to(torch.uint8) if t > 1 else None
    lay = dlm.make_layout(1, t, None, pad)
    if pad is not None:
        ids = torch.where(pad == 1, torch.full_like(ids, -100), ids)     # the ids of pads are not looked at
    out = _placed(torch.full((t, d), 3.0, dtype=bf16, device="cuda"), ldo, shift)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = dlm.embed_fwd(lay, ids, w, scale, out=out, dev_status=status)
    want = ref.embed(ids.clamp(min=0), w, scale, pad)
    assert got.data_ptr() == out.data_ptr() and status.item() == 0
    # one fp32 product and one rounding; exact for scale 1
    ref.assert_within(got, want, want.abs() * (0.0 if scale == 1.0 else 2.0 ** -8 + 2.0 ** -22))
    fresh = dlm.embed_fwd(lay, ids, w, scale)
    assert torch.equal(fresh.view(torch.int16), got.contiguous().view(torch.int16))
    base = out._base if out._base is not None else out
    rest = torch.as_strided(base, (base.numel(),), (1,)).clone()
    torch.as_strided(rest, (t, d), (ldo, 1), shift).fill_(7.0)
    assert bool((rest == 7.0).all()), "wrote outside its columns"


def test_forward_bad_ids_give_zero_rows_and_a_status_bit():
    g = _gen(1)
    w = _randn((10, 64), g)
    ids = torch.tensor([3, 10, -1, 9, 2147483647, -2147483648], dtype=torch.int32, device="cuda")
    lay = dlm.make_layout(1, 6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dlm.embed_fwd(lay, ids, w, dev_status=status)
    assert status.item() == dlm.DEV_BAD_TOKEN_ID
    want = torch.stack([w[3], w[3] * 0, w[3] * 0, w[9], w[3] * 0, w[3] * 0])
    assert torch.equal(out, want)
    assert torch.equal(dlm.embed_fwd(lay, ids, w), want)                 # nobody asked: no status


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("t,vocab,d,kind", [
    (1, 1, 1, "one"), (1, 64, 8, "rand"), (31, 40, 16, "one"), (32, 40, 16, "one"), (33, 40, 16, "one"),
    (64, 40, 8, "last"), (65, 40, 264, "one"), (130, 1024, 256, "masked"), (1000, 2, 72, "rand"),
    (1000, 131, 1000, "runs"), (4097, 1024, 136, "masked"), (5000, 300, 33, "masked"), (777, 5000, 1001, "rand"),
    (3000, 262144, 8, "masked"), (3000, 300001, 8, "rand"), (20000, 1000, 40, "one"), (100, 20, 9000, "runs"),
    # either side of the single launch's limits (tokens, bytes of the table), and tables whose zeros take every path
    (1024, 500, 512, "masked"), (1025, 500, 512, "masked"), (1024, 500, 512, "one"), (600, 9000, 1000, "runs"),
    (600, 9000, 1001, "runs"), (1, 40000, 1001, "rand"), (50, 3000, 9000, "masked"), (2000, 3000, 1500, "runs"),
    (33, 1000003, 9, "rand"), (40000, 70, 264, "masked")])
def test_gradient(t, vocab, d, kind, dtype):
    g = _gen(t + vocab + d)
    ids = _ids(kind, t, vocab, g)
    dy = _randn((t, d), g)
    lay = dlm.make_layout(1, t)
    scale = 1.0 if d % 3 else 5.5
    out = dlm.embed_bwd(lay, ids, dy, vocab, scale, grad_dtype=dtype)
    assert out.device_status() == 0 and out.d_weight.dtype == dtype
    dw, mag = ref.embed_grad(ids, dy, vocab, scale)
    ref.assert_within(out.d_weight, dw, ref.embed_grad_bound(ids, dw, mag, dtype))
    # the same bits again, in a workspace and a gradient that held something else
    dirty = torch.full_like(out.workspace, 0xA5)
    ws = dlm._aligned_workspace(dirty.numel(), "cuda", 256).copy_(dirty)
    again = dlm.embed_bwd(lay, ids, dy, vocab, scale, d_weight=torch.full_like(out.d_weight, float("nan")),
                          workspace=ws)
    assert torch.equal(again.d_weight, out.d_weight)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("t,vocab,d,ld,ldw,shift", [(200, 64, 40, 48, 56, 0), (200, 64, 40, 41, 43, 0), (97, 33, 128, 128, 128, 1),
                                                    (500, 40, 1001, 1001, 1001, 0), (300, 20011, 520, 528, 536, 0),
                                                    (1500, 20011, 521, 523, 525, 1), (300, 60000, 40, 40, 40, 0)])
def test_gradient_pads_strides_and_accumulate(t, vocab, d, ld, ldw, shift, dtype):
    g = _gen(d + ld)
    ids = _ids("masked", t, vocab, g)
    ids[ids == 5] = 6                                                     # no token has id 5
    pad = (torch.rand(t, generator=g, device="cuda") < 0.4).to(torch.uint8)
    dy = _placed(_randn((t, d), g), ld, shift)
    dy[pad == 1] = float("nan")                                           # rows of pads are not read
    lay = dlm.make_layout(1, t, None, pad)
    ids = torch.where(pad == 1, torch.full_like(ids, -100), ids)
    clean = torch.where((pad == 1)[:, None], torch.zeros_like(dy), dy)
    dw, mag = ref.embed_grad(ids.clamp(min=0), clean, vocab, 2.0, pad)
    buf = _placed(torch.full((vocab, d), float("nan"), dtype=dtype, device="cuda"), ldw, shift)
    out = dlm.embed_bwd(lay, ids, dy, vocab, 2.0, d_weight=buf)
    assert out.device_status() == 0
    ref.assert_within(buf, dw, ref.embed_grad_bound(ids.clamp(min=0), dw, mag, dtype))
    # added to what is there; rows without tokens are left alone, NaN and all
    old = _randn((vocab, d), g, dtype)
    old[5] = float("nan")
    acc = _placed(old, ldw, shift)
    base = acc._base
    dlm.embed_bwd(lay, ids, dy, vocab, 2.0, d_weight=acc, accumulate=True)
    touched = mag.abs().sum(1) > 0
    assert not touched[5] and bool(torch.isnan(acc[5]).all())
    bits = torch.int16 if dtype == bf16 else torch.int32
    assert torch.equal(acc[~touched].view(bits), old[~touched].view(bits))
    want = old.double() + dw
    # one more fp32 addition before the rounding
    bound = ref.embed_grad_bound(ids.clamp(min=0), want, mag + old.double().abs(), dtype)
    ref.assert_within(acc[touched], want[touched], bound[touched])
    rest = torch.as_strided(base, (base.numel(),), (1,)).clone()
    torch.as_strided(rest, (vocab, d), (ldw, 1), shift).fill_(7.0)
    assert bool((rest == 7.0).all()), "wrote outside its columns"


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [264, 1001])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gradient_rows_over_few_and_many_chunks(d, dtype, accumulate):
    """Tokens drawn as words are, and rows of just under, just as many and just
    more tokens than 1 to 20 chunks of 8, 16 and 32 hold, side by side."""
    g = _gen(d)
    vocab = 400
    p = 1.0 / torch.arange(1, vocab + 1, device="cuda")
    words = torch.multinomial(p / p.sum(), 3000, replacement=True, generator=g).int()
    runs = [c * n + e for c in (8, 16, 32) for n in (1, 2, 7, 8, 9, 10, 17, 20) for e in (-1, 0, 1)]
    rows = torch.repeat_interleave(torch.arange(len(runs), device="cuda"), torch.tensor(runs, device="cuda")).int()
    for ids in (words, rows[torch.randperm(rows.numel(), generator=g, device="cuda")]):
        dy = _randn((ids.numel(), d), g)
        lay = dlm.make_layout(1, ids.numel())
        dw, mag = ref.embed_grad(ids, dy, vocab, 3.0)
        old = _randn((vocab, d), g, dtype) if accumulate else torch.full((vocab, d), float("nan"), dtype=dtype, device="cuda")
        got = old.clone()
        dlm.embed_bwd(lay, ids, dy, vocab, 3.0, d_weight=got, accumulate=accumulate)
        if accumulate:
            untouched = mag.abs().sum(1) == 0
            assert torch.equal(got[untouched], old[untouched])
            dw, mag = old.double() + dw, mag + old.double().abs()
            bound = ref.embed_grad_bound(ids, dw, mag, dtype)
            ref.assert_within(got[~untouched], dw[~untouched], bound[~untouched])
        else:
            ref.assert_within(got, dw, ref.embed_grad_bound(ids, dw, mag, dtype))
        again = old.clone()
        dlm.embed_bwd(lay, ids, dy, vocab, 3.0, d_weight=again, accumulate=accumulate)
        assert torch.equal(again, got)


def test_gradient_no_tokens_all_pads_bad_ids():
    g = _gen(3)
    dy = _randn((6, 64), g)
    none = dlm.embed_bwd(dlm.make_layout(1, 0), torch.empty(0, dtype=torch.int32, device="cuda"), dy[:0], 9)
    assert none.device_status() == 0 and none.d_weight.shape == (9, 64) and not none.d_weight.any()
    keep = torch.full((9, 64), 2.0, device="cuda")
    dlm.embed_bwd(dlm.make_layout(1, 0), torch.empty(0, dtype=torch.int32, device="cuda"), dy[:0], 9, d_weight=keep,
                  accumulate=True)
    assert bool((keep == 2.0).all())
    pad = torch.ones(6, dtype=torch.uint8, device="cuda")
    bad = torch.tensor([3, 9, -1, 8, 2147483647, -2147483648], dtype=torch.int32, device="cuda")
    out = dlm.embed_bwd(dlm.make_layout(1, 6, None, pad), bad, dy, 9)
    assert out.device_status() == 0 and not out.d_weight.any()
    out = dlm.embed_bwd(dlm.make_layout(1, 6), bad, dy, 9, grad_dtype=f32)
    assert out.device_status() == dlm.DEV_BAD_TOKEN_ID
    want = torch.zeros((9, 64), device="cuda")
    want[3], want[8] = dy[0].float(), dy[3].float()
    assert torch.equal(out.d_weight, want)
    # the same through the three launches of a large table
    big = dlm.embed_bwd(dlm.make_layout(1, 6), torch.tensor([3, 40000, -1, 8, 2147483647, 39999], dtype=torch.int32, device="cuda"),
                        _randn((6, 512), g), 40000, grad_dtype=f32)
    assert big.device_status() == dlm.DEV_BAD_TOKEN_ID
    assert big.d_weight.any(1).nonzero()[:, 0].tolist() == [3, 8, 39999]
    empty = dlm.embed_bwd(dlm.make_layout(1, 0), torch.empty(0, dtype=torch.int32, device="cuda"), _randn((0, 512), g), 40000,
                          d_weight=big.d_weight.fill_(float("nan")), workspace=big.workspace)
    assert empty.device_status() == 0 and not empty.d_weight.any()
    # the next call on the same workspace reports itself only
    ok = dlm.embed_bwd(dlm.make_layout(1, 1), bad[:1], dy[:1], 9, workspace=out.workspace)
    assert ok.device_status() == 0


def test_infinities_and_nan_stay_in_their_row():
    g = _gen(4)
    ids = _ids("masked", 300, 50, g)
    dy = _randn((300, 72), g)
    where = int(ids[17])
    dy[17, 3], dy[17, 4] = float("inf"), float("nan")
    out = dlm.embed_bwd(dlm.make_layout(1, 300), ids, dy, 50).d_weight
    other = torch.ones(50, dtype=torch.bool, device="cuda")
    other[where] = False
    assert bool(torch.isfinite(out[other]).all())
    assert torch.isinf(out[where, 3]) and torch.isnan(out[where, 4]) and bool(torch.isfinite(out[where, 5:]).all())


def test_rows_past_two_to_the_31_elements():
    """A table of 2.2e9 elements: its last rows' offsets pass 32 bits."""
    V, D = 540000, 4096
    g = _gen(5)
    w = torch.zeros((V, D), dtype=bf16, device="cuda")
    ids = torch.tensor([0, V - 1, V - 2, V - 1, 530001], dtype=torch.int32, device="cuda")
    w[ids.long().unique()] = _randn((4, D), g)
    lay = dlm.make_layout(1, 5)
    assert torch.equal(dlm.embed_fwd(lay, ids, w), w[ids.long()])
    dy = _randn((5, D), g)
    w.fill_(3.0)
    dlm.embed_bwd(lay, ids, dy, V, d_weight=w)
    nz = (w != 0).any(1).nonzero()[:, 0]
    assert nz.tolist() == sorted(set(ids.tolist()))
    assert torch.equal(w[0], dy[0]) and torch.equal(w[V - 2], dy[2])
    assert torch.equal(w[V - 1], (dy[1].float() + dy[3].float()).to(bf16))


def test_two_streams_and_a_captured_graph():
    g = _gen(6)
    t, V, D = 3000, 2000, 512
    ids = [_ids("masked", t, V, g) for _ in range(2)]
    dy = [_randn((t, D), g) for _ in range(2)]
    w = _randn((V, D), g)
    lay = dlm.make_layout(1, t)
    want = [dlm.embed_bwd(lay, ids[k], dy[k], V).d_weight for k in range(2)]
    wf = [dlm.embed_fwd(lay, ids[k], w, 2.0) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = (dlm.embed_bwd(lay, ids[k], dy[k], V).d_weight, dlm.embed_fwd(lay, ids[k], w, 2.0))
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(got[k][0], want[k]) and torch.equal(got[k][1], wf[k])
    # captured once, replayed on other data in the same buffers
    sid, sdy = ids[0].clone(), dy[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dlm.embed_bwd(lay, sid, sdy, V)
        fwd = dlm.embed_fwd(lay, sid, w, 2.0)
    for k in (0, 1, 0):
        sid.copy_(ids[k])
        sdy.copy_(dy[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.d_weight, want[k]) and torch.equal(fwd, wf[k])


def test_autograd():
    g = _gen(7)
    t, V, D = 500, 300, 64
    ids = _ids("masked", t, V, g)
    lay = dlm.make_layout(1, t)
    w = _randn((V, D), g).requires_grad_(True)
    y = dlm.embed(lay, ids, w, 8.0)
    assert torch.equal(y, dlm.embed_fwd(lay, ids, w.detach(), 8.0))
    dy = _randn((t, D), g)
    y.backward(dy, retain_graph=True)
    want = dlm.embed_bwd(lay, ids, dy, V, 8.0).d_weight
    assert torch.equal(w.grad, want)
    w.grad = None
    y.sum().backward()                       # an expanded gradient
    dw, mag = ref.embed_grad(ids, torch.ones_like(dy), V, 8.0)
    ref.assert_within(w.grad, dw, ref.embed_grad_bound(ids, dw, mag, bf16))
    assert not dlm.embed(lay, ids, w.detach()).requires_grad
