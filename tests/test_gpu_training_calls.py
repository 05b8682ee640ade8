"""The embedding, norm and 8-bit calls on the GPU where the other files do not
look: calls without rows, results and masks used again, evaluation."""
import pytest
import torch

pytestmark = pytest.mark.gpu

dlm = pytest.importorskip("diffusion_lm_loss_b200")
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dlm.lib()


def _bits(t):
    return t.view(torch.int16 if t.dtype == bf16 else torch.int32)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("d", [136, 1001, 9001])
def test_no_rows_leave_the_gradients_they_would_add_to(d, dtype):
    none, stat = torch.zeros((0, d), dtype=bf16, device="cuda"), torch.zeros(0, device="cuda")
    dw = torch.randn(d, device="cuda").to(dtype)
    dw[::3], dw[1] = -0.0, float("nan")
    db = -dw
    want = dw.clone(), db.clone()
    dlm.norm_bwd(none, none, stat, stat, d_weight=dw, d_bias=db, accumulate=True)
    dlm.norm_bwd(none, none, stat, stat, d_weight=dw, accumulate=True)
    assert torch.equal(_bits(dw), _bits(want[0])) and torch.equal(_bits(db), _bits(want[1]))
    fresh = dlm.norm_bwd(none, none, stat, stat, d_weight=dw, d_bias=db)
    assert not _bits(fresh.d_weight).any() and not _bits(fresh.d_bias).any()


def test_a_reused_norm_result_reports_this_call_alone():
    a, b = (torch.randn((9, 264), device="cuda").to(bf16) for _ in range(2))
    first = dlm.norm_fwd(a, pack=dlm.PACK_INT8)
    second = dlm.norm_fwd(b, out=first)
    want = dlm.norm_fwd(b)
    assert second.packed is None and second.y.data_ptr() == first.y.data_ptr()
    assert torch.equal(second.y, want.y) and torch.equal(second.mean, want.mean) and torch.equal(second.rstd, want.rstd)
    rms = dlm.norm_fwd(b, kind=dlm.NORM_RMS, out=second)
    assert rms.mean is None and torch.equal(rms.y, dlm.norm_fwd(b, kind=dlm.NORM_RMS).y)


def test_embed_under_autograd_refuses_a_changed_mask_and_shows_bad_ids():
    pad = torch.zeros(6, dtype=torch.uint8, device="cuda")
    pad[2] = 1
    ids = torch.tensor([3, 1, -100, 3, 40, 0], dtype=torch.int32, device="cuda")
    lay = dlm.make_layout(1, 6, None, pad)
    w = torch.randn((9, 64), device="cuda").to(bf16).requires_grad_(True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = dlm.embed(lay, ids, w, dev_status=status)
    assert status.item() == dlm.DEV_BAD_TOKEN_ID                   # 40; the pad's id is not looked at
    y.sum().backward()
    assert w.grad[:, 0].tolist() == [1, 1, 0, 2, 0, 0, 0, 0, 0]
    status.zero_()
    ids[4] = 4
    y = dlm.embed(lay, ids, w, dev_status=status)
    assert status.item() == 0
    pad.fill_(0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_evaluation_allocates_no_8_bit_form():
    x = torch.randn((4096, 1024), device="cuda").to(bf16)
    w = torch.ones(1024, device="cuda", dtype=bf16, requires_grad=True)

    def peak():
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        y = dlm.norm(x, w, keep8=dlm.PACK_INT8)
        return torch.cuda.max_memory_allocated() - before, y
    kept, y = peak()
    with torch.no_grad():
        bare, z = peak()
    assert torch.equal(y, z) and not z.requires_grad
    assert kept - bare >= x.numel() and bare < x.numel() * 2 + (1 << 20)


def test_a_table_of_almost_two_to_the_31_rows():
    """The most rows that the gradient takes."""
    V = 2 ** 31 - 2
    ids = torch.tensor([0, V - 1, 5, V - 1, 2 ** 30, V - 2], dtype=torch.int32, device="cuda")
    lay = dlm.make_layout(1, 6)
    dy = torch.tensor([1, 2, 3, 4, 5, 6], device="cuda").to(bf16)[:, None]
    w = torch.full((V, 1), 9.0, dtype=bf16, device="cuda")
    out = dlm.embed_bwd(lay, ids, dy, V, d_weight=w)
    assert out.device_status() == 0 and int(torch.count_nonzero(w)) == 5
    rows = torch.tensor([0, V - 1, 5, 2 ** 30, V - 2], device="cuda")
    assert w[rows, 0].tolist() == [1, 6, 3, 5, 6]
    assert dlm.embed_fwd(lay, ids, w)[:, 0].tolist() == [1, 6, 3, 6, 5, 6]
    dlm.embed_bwd(lay, ids, dy, V, d_weight=w, accumulate=True, workspace=out.workspace)
    assert w[rows, 0].tolist() == [2, 12, 6, 10, 12] and int(torch.count_nonzero(w)) == 5
