"""One training step's ends together, as a program runs them: corrupted ids ->
embedding -> norm (its input kept in 8 bits) -> head and loss -> backward to the
norm's input and parameters and to the tied table.  Every stage against its
64-bit form on the values that it was given, and the autograd functions
against the direct calls bit for bit."""
import pytest
import torch

import train_ref as ref

pytestmark = pytest.mark.gpu

dlm = pytest.importorskip("diffusion_lm_loss_b200")
bf16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dlm.lib()


@pytest.mark.parametrize("keep8", [0, 1, 2])
def test_one_step_with_a_tied_table(keep8):
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    T, D, V, mask = 600, 256, 2048, 2047
    cu = torch.tensor([0, 100, 350, 600], dtype=torch.int32, device="cuda")
    pad = torch.zeros(T, dtype=torch.uint8, device="cuda")
    pad[340:350] = 1
    lay = dlm.make_layout(3, 0, cu, pad, n_tokens=T)
    clean = torch.randint(0, mask, (T,), generator=g, device="cuda", dtype=torch.int32)
    table = (0.1 * torch.randn((V, D), generator=g, device="cuda")).to(bf16)
    w = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(bf16)
    b = (0.1 * torch.randn(D, generator=g, device="cuda")).to(bf16)
    t, p = dlm.sample_t(3, 3)
    noisy, corrupted = dlm.corrupt(lay, clean, p, dlm.ABSORBING, mask, V, 3)
    scale = D ** 0.5

    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = dlm.embed_fwd(lay, noisy, table, scale, dev_status=status)
    want = ref.embed(noisy, table, scale, pad)
    ref.assert_within(x, want, want.abs() * (2.0 ** -8 + 2.0 ** -22), "embedding")
    n = dlm.norm_fwd(x, w, b, pack=keep8)
    y, _, _ = ref.norm(x, w, b, 1e-5, False, 0.0)
    ref.assert_within(n.y, y, ref.norm_bounds(x, w, b, 1e-5, False, 0.0)[0], "norm")
    head = dlm.linear_loss_fwd_bwd(lay, n.y, table, clean, corrupted, p)
    kept = n.packed if keep8 else x
    nb = dlm.norm_bwd(head.d_hidden, kept, n.rstd, n.mean, w, want_d_bias=True)
    held = ref.held(n.packed.q, n.packed.scale, keep8, torch.float64) if keep8 else x
    dx, dw, db = ref.norm_grad(head.d_hidden, held, n.mean, n.rstd, w, False, 0.0)
    bx, bw, bb = ref.norm_grad_bounds(head.d_hidden, held, n.mean, n.rstd, w, False, 0.0, bf16)
    ref.assert_within(nb.d_x, dx, bx, "d_x")
    ref.assert_within(nb.d_weight, dw, bw, "d_weight")
    ref.assert_within(nb.d_bias, db, bb, "d_bias")
    # the table's gradient: the head's, plus the embedding's, in one tensor
    total = head.d_weight.clone()
    eb = dlm.embed_bwd(lay, noisy, nb.d_x, V, scale, d_weight=total, accumulate=True)
    assert status.item() == 0 and head.device_status() == 0 and eb.device_status() == 0
    demb, mag = ref.embed_grad(noisy, nb.d_x, V, scale, pad)
    sum_ = head.d_weight.double() + demb
    ref.assert_within(total, sum_, ref.embed_grad_bound(noisy, sum_, mag + head.d_weight.double().abs(), bf16), "table")

    # the same step through autograd
    e1 = table.clone().requires_grad_(True)
    e2 = table.clone().requires_grad_(True)
    ws, bs = w.clone().requires_grad_(True), b.clone().requires_grad_(True)
    h = dlm.norm(dlm.embed(lay, noisy, e1, scale), ws, bs, keep8=keep8)
    loss = dlm.linear_diffusion_loss(lay, h, e2, clean, corrupted, p)
    loss.backward()
    assert loss.item() == head.loss.item()
    assert torch.equal(ws.grad, nb.d_weight) and torch.equal(bs.grad, nb.d_bias)
    assert torch.equal(e2.grad, head.d_weight)
    assert torch.equal(e1.grad, dlm.embed_bwd(lay, noisy, nb.d_x, V, scale).d_weight)
