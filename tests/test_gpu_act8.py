"""Activations in 8 bits on the GPU: codes and factors bit for bit against
their definition, values exact, blocks of zeros, tiny values, infinities and
NaN, strides, alignment, streams and graphs."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

dlm = pytest.importorskip("diffusion_lm_loss_b200")
bf16 = torch.bfloat16
FORMATS = [1, 2]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dlm.lib()


def _x(r, d, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((r, d), generator=g, device="cuda")
    return (x * torch.exp2(torch.randint(-20, 20, (r, d), generator=g, device="cuda") * 0.2)).to(bf16)


def _same(a, b):
    """Equal values, NaN equal to NaN."""
    return bool(((a == b) | (torch.isnan(a.float()) & torch.isnan(b.float()))).all())


def _check_packed(p, x, fmt):
    q, s = ref.pack(x, fmt)
    assert _same(p.scale.cpu(), s)
    if fmt == ref.INT8:
        assert torch.equal(p.q.cpu(), q)
    else:
        assert torch.equal(p.q.cpu().view(torch.float8_e4m3fn).float(), q.view(torch.float8_e4m3fn).float())
    v = dlm.unpack8(p)
    assert v.dtype == bf16 and _same(v.cpu(), ref.held(q, s, fmt).to(bf16))
    return v


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("r,d", [(1, 1), (1, 8), (3, 127), (3, 128), (3, 129), (5, 136), (130, 1001), (2, 4096), (37, 520),
                                 (1000, 256), (1, 70000), (4099, 24), (50, 1023), (50, 1025),
                                 (33, 2047), (33, 2049), (17, 7), (200, 5001)])
def test_pack_and_unpack(r, d, fmt):
    x = _x(r, d, r + d)
    v = _check_packed(dlm.pack8(x, fmt), x, fmt)
    # half a step of the block's factor (int8), or of the value (e4m3: 2^-4, 2^-10 of the factor below 2^-6 of it),
    # and the rounding to bf16
    a = x.float().abs()
    top = torch.stack([b.amax(1) for b in a.split(128, 1)], 1).repeat_interleave(128, 1)[:, :d].double()
    err = (v.double() - x.double()).abs()
    half = top / 127 / 2 if fmt == ref.INT8 else torch.maximum(x.double().abs() * 2.0 ** -4, top / 448 * 2.0 ** -10)
    assert bool((err <= half * (1 + 2.0 ** -20) + (x.double().abs() + half) * 2.0 ** -8).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_blocks(fmt):
    d = 128 * 10
    x = _x(2, d, 9)
    x[0, :128] = 0.0
    x[0, 128:256] *= 0
    x[0, 130] = 2.0 ** -100                   # the smallest magnitude that is held
    x[0, 256:384] = 2.0 ** -101               # a block below it
    x[0, 384:512] *= 0
    x[0, 400] = 1e-40                         # subnormal
    x[0, 512 + 5] = float("inf")
    x[0, 640 + 127] = float("nan")
    x[0, 768 + 1], x[0, 768 + 2] = float("-inf"), float("nan")
    x[0, 896 + 3] = 3.3895313892515355e38     # the largest bf16
    x[0, 1024:1152] = -0.0
    x[1, 0] = float("-inf")
    p = dlm.pack8(x, fmt)
    v = _check_packed(p, x, fmt)
    nan = torch.isnan(v).view(2, 10, 128)
    want = torch.zeros((2, 10), dtype=torch.bool, device="cuda")
    want[0, 4] = want[0, 5] = want[0, 6] = want[1, 0] = True
    assert torch.equal(nan.all(2), want) and torch.equal(nan.any(2), want)
    assert not v[0, :128].any() and not v[0, 256:512].any()
    assert v[0, 130] == x[0, 130] or fmt == ref.INT8
    # the same through rows that are not on 16-byte borders
    y = torch.zeros((2, d + 1), dtype=bf16, device="cuda")[:, 1:]
    y.copy_(x)
    py = dlm.pack8(y, fmt)
    assert torch.equal(py.q, p.q) and _same(py.scale, p.scale)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,ld,shift", [(256, 264, 0), (256, 257, 0), (1000, 1000, 4), (129, 136, 8),
                                         (1030, 1031, 1), (1024, 1024, 3), (2050, 2053, 6)])
def test_strides(d, ld, shift, fmt):
    x = _x(19, d, d)
    buf = torch.zeros(19 * ld + shift, dtype=bf16, device="cuda")
    v = buf[shift:].view(19, ld)[:, :d]
    v.copy_(x)
    p = dlm.pack8(v, fmt)
    _check_packed(p, x, fmt)
    out = torch.full((19 * ld + shift,), 7.0, dtype=bf16, device="cuda")
    o = out[shift:].view(19, ld)[:, :d]
    dlm.unpack8(p, out=o)
    assert torch.equal(o, dlm.unpack8(p))
    o.fill_(7.0)
    assert bool((out == 7.0).all()), "wrote outside its columns"
    again = dlm.Packed8(torch.empty_like(p.q), torch.empty_like(p.scale), fmt)
    assert dlm.pack8(v, fmt, out=again) is again and torch.equal(again.q, p.q)


def test_empty():
    for shape in ((0, 128), (4, 0)):
        p = dlm.pack8(torch.empty(shape, dtype=bf16, device="cuda"))
        assert dlm.unpack8(p).shape == shape


def test_rows_past_two_to_the_31_elements():
    ld = 2 ** 30 + 8
    buf = torch.zeros(2 * ld + 512, dtype=bf16, device="cuda")
    v = torch.as_strided(buf, (3, 512), (ld, 1))
    x = _x(3, 512, 3)
    v.copy_(x)
    p = dlm.pack8(v)
    _check_packed(p, x, dlm.PACK_INT8)
    v.zero_()
    dlm.unpack8(p, out=v)
    assert torch.equal(v, dlm.unpack8(p))


def test_streams_and_graph():
    xs = [_x(300, 1000, k) for k in range(2)]
    want = [dlm.unpack8(dlm.pack8(x)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k] = dlm.unpack8(dlm.pack8(xs[k]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = dlm.unpack8(dlm.pack8(x))
    for k in (1, 0):
        x.copy_(xs[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])
