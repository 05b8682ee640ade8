"""The bounds and exact inputs of the GPU tests of long sums, on the CPU: one
token or row lost or counted twice among 20,000 is seen, and plain fp32 sums in
the kernels' order stay within the bounds."""
import pytest
import torch

import train_ref as ref

bf16, f32 = torch.bfloat16, torch.float32


def _refused(got, want, bound):
    with pytest.raises(AssertionError):
        ref.assert_within(got, want, bound)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("t,vocab,d", [(20000, 1000, 40), (40000, 70, 264)])
def test_one_token_of_a_long_row_is_seen(t, vocab, d, dtype):
    g = torch.Generator().manual_seed(t)
    half = t // 2 if vocab == 70 else 0
    ids = torch.randint(0, vocab, (t,), generator=g, dtype=torch.int32)
    ids[half:] = vocab - 1
    dy = torch.randn((t, d), generator=g).to(bf16)
    dw, mag = ref.embed_grad(ids, dy, vocab, 5.5)
    bound = ref.embed_grad_tight(ids, dw, mag, dtype)
    ref.assert_within(dw.to(dtype), dw, bound)
    k = t - 7                                                # a token of the long row
    lost = torch.arange(t) != k
    _refused(ref.embed_grad(ids[lost], dy[lost], vocab, 5.5)[0].to(dtype), dw, bound)
    twice = torch.cat([torch.arange(t), torch.tensor([k])])
    _refused(ref.embed_grad(ids[twice], dy[twice], vocab, 5.5)[0].to(dtype), dw, bound)
    # whole numbers: equality in fp32
    dy = ref.integers((t, d), 8, g, "cpu").to(bf16)
    exact = ref.embed_grad(ids, dy, vocab, 2.0)[0]
    assert torch.equal(exact.float().double(), exact) and float(exact.abs().max()) < 2 ** 24
    assert not torch.equal(ref.embed_grad(ids[lost], dy[lost], vocab, 2.0)[0], exact)


def test_sums_in_the_kernels_order_stay_within_the_bounds():
    """Chunks of 32 tokens, their sums in 16 shares, in fp32: each step rounded."""
    g = torch.Generator().manual_seed(1)
    t, d = 20000, 64
    ids, dy = torch.zeros(t, dtype=torch.int32), torch.randn((t, d), generator=g).to(bf16)
    dw, mag = ref.embed_grad(ids, dy, 1, 5.5)

    def in_turn(rows):
        acc = torch.zeros_like(rows[0])
        for r in rows:
            acc = acc + r
        return acc
    chunks = torch.stack([in_turn(list(dy.float()[k:k + 32])) for k in range(0, t, 32)])
    shares = [in_turn(list(chunks[k:k + 40])) for k in range(0, len(chunks), 40)]
    got = in_turn(shares)[None] * 5.5
    ref.assert_within(got, dw, ref.embed_grad_tight(ids, dw, mag, f32))


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("r,d", [(21312, 256), (20665, 264)])
def test_one_row_of_many_is_seen(r, d, rms):
    g = torch.Generator().manual_seed(r)
    x = (torch.randn((r, d), generator=g) * 2 + 3).to(bf16)
    dy, w = torch.randn((r, d), generator=g).to(bf16), torch.randn(d, generator=g)
    _, mean, rstd = ref.norm(x, w, None, 1e-5, rms, 0.0)
    mean, rstd = mean.float(), rstd.float()
    _, dw, db = ref.norm_grad(dy, x, mean, rstd, w, rms, 0.0)
    _, bw, bb = ref.norm_grad_tight(dy, x, mean, rstd, w, rms, 0.0, f32)
    ref.assert_within(dw.float(), dw, bw)
    ref.assert_within(db.float(), db, bb)
    keep = torch.arange(r) != 148
    _, lw, lb = ref.norm_grad(dy[keep], x[keep], mean[keep], rstd[keep], w, rms, 0.0)
    _refused(lw.float(), dw, bw)
    _refused(lb.float(), db, bb)


@pytest.mark.parametrize("fmt", [0, ref.INT8, ref.E4M3])
@pytest.mark.parametrize("rms", [False, True])
def test_whole_numbers_sum_exactly(fmt, rms):
    g = torch.Generator().manual_seed(fmt)
    r, d = 20665, 200
    dy, _, held, _, _, mean, rstd = ref.exact_norm_inputs(r, d, fmt, g, "cpu")
    _, dw, db = ref.norm_grad(dy, held, mean, rstd, None, rms, 0.0)
    xh = (held - (0 if rms else mean.double()[:, None])) * rstd.double()[:, None]
    # every partial sum is a multiple of 1/8 below 2^21, in whatever order
    terms = dy.double() * xh * 8
    assert torch.equal(terms, terms.round()) and float(terms.abs().sum(0).max()) < 2 ** 24
    assert torch.equal(dw.float().double(), dw) and torch.equal(db.float().double(), db)
    keep = torch.arange(r) != 1234
    _, lw, lb = ref.norm_grad(dy[keep], held[keep], mean[keep], rstd[keep], None, rms, 0.0)
    assert not torch.equal(lw, dw) and not torch.equal(lb, db)
