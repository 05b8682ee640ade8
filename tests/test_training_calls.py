"""What the binding of the embedding, norm and 8-bit calls hands to the library
and returns to its caller, without a GPU: the library call is replaced by a
recorder, the rest runs as it is."""
import ctypes

import pytest
import torch

import diffusion_lm_loss_b200 as dlm
from diffusion_lm_loss_b200 import build as dlm_build
from test_host_failures import _a_device_may_be_usable

bf16 = torch.bfloat16


@pytest.fixture
def calls(monkeypatch):
    """(name, arguments) of each library call, which does nothing."""
    made = []
    monkeypatch.setattr(dlm, "_on_cuda", lambda **kw: None)
    monkeypatch.setattr(dlm, "_all_on", lambda *a: True)
    monkeypatch.setattr(dlm, "_call", lambda dev, name, *args: made.append((name, args)))
    return made


def test_a_reused_norm_result_reports_this_call_alone(calls):
    x = torch.zeros(4, 200, dtype=bf16)
    first = dlm.norm_fwd(x, pack=dlm.PACK_INT8)
    buffers = first.y, first.mean, first.rstd, first.packed
    plain = dlm.norm_fwd(x, out=first)
    assert plain.packed is None, "the codes of the call before"
    assert plain.y is buffers[0] and plain.mean is buffers[1] and plain.rstd is buffers[2]
    rms = dlm.norm_fwd(x, kind=dlm.NORM_RMS, out=dlm.NormOut(*buffers))
    assert rms.mean is None and rms.packed is None, "the means of the call before"
    again = dlm.norm_fwd(x, pack=dlm.PACK_INT8, out=dlm.NormOut(*buffers))
    assert again.packed is buffers[3] and again.mean is buffers[1]


@pytest.fixture
def plain_embedding(monkeypatch):
    """embed over plain CPU forms of its two calls."""
    def fwd(layout, ids, weight, scale=1.0, out=None, dev_status=None):
        pad = dlm._pad_mask(layout)
        y = weight[ids.long().clamp(0, weight.shape[0] - 1)] * scale
        return y if pad is None else y * (pad == 0)[:, None]

    def bwd(layout, ids, d_out, vocab, scale=1.0, **kw):
        pad = dlm._pad_mask(layout)
        assert layout.pad_mask == (None if pad is None else pad.data_ptr())
        keep = d_out if pad is None else d_out * (pad == 0)[:, None]
        dw = torch.zeros(vocab, d_out.shape[1]).index_add_(0, ids.long(), keep.float() * scale)
        return dlm.EmbedGrad(dw.to(bf16), torch.empty(0, dtype=torch.uint8))
    monkeypatch.setattr(dlm, "_on_cuda", lambda **kw: None)
    monkeypatch.setattr(dlm, "embed_fwd", fwd)
    monkeypatch.setattr(dlm, "embed_bwd", bwd)


def _embedding_inputs():
    pad = torch.tensor([0, 1, 0, 0, 0, 1], dtype=torch.uint8)
    ids = torch.tensor([1, 2, 1, 0, 4, 4], dtype=torch.int32)
    w = torch.ones(5, 3, dtype=bf16, requires_grad=True)
    return pad, ids, w, dlm.make_layout(1, 6, None, pad)


def test_a_pad_mask_changed_before_backward_is_refused(plain_embedding):
    pad, ids, w, lay = _embedding_inputs()
    y = dlm.embed(lay, ids, w)
    pad.zero_()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    for lay in (lay, dlm.make_layout(1, 6)):                 # a mask left alone, and none
        w.grad = None
        dlm.embed(lay, ids, w).sum().backward()
        assert w.grad[:, 0].tolist() == [1, 2, 1, 0, 2]


def test_backward_takes_the_pad_mask_that_was_saved(plain_embedding):
    """Saved-tensor hooks (here: copies) may hand back another tensor."""
    pad, ids, w, lay = _embedding_inputs()
    with torch.autograd.graph.saved_tensors_hooks(lambda t: t.clone(), lambda t: t):
        y = dlm.embed(lay, ids, w)
    pad.zero_()
    y.sum().backward()
    assert w.grad[:, 0].tolist() == [1, 2, 0, 0, 1]


def test_embed_hands_its_status_word_to_the_forward_call(calls):
    ids, w = torch.zeros(6, dtype=torch.int32), torch.zeros(5, 3, dtype=bf16, requires_grad=True)
    lay = dlm.make_layout(1, 6)
    status = torch.zeros(1, dtype=torch.int32)
    dlm.embed(lay, ids, w, 2.0, dev_status=status)
    dlm.embed(lay, ids, w, 2.0)
    assert [name for name, _ in calls] == ["dlm_embed_fwd"] * 2
    assert [args[-1] for _, args in calls] == [status.data_ptr(), None]
    with pytest.raises(ValueError, match="dev_status"):
        dlm.embed(lay, ids, w, dev_status=torch.zeros(1))


def test_norm_keeps_nothing_in_8_bits_where_no_gradient_is_recorded(calls):
    x = torch.zeros(4, 200, dtype=bf16)
    w = torch.zeros(200, dtype=bf16, requires_grad=True)

    def formats():
        out = [args[-3] for name, args in calls if name == "dlm_norm_fwd"]
        calls.clear()
        return out
    dlm.norm(x, w, keep8=dlm.PACK_INT8)
    with torch.no_grad():
        dlm.norm(x, w, keep8=dlm.PACK_INT8)
    with torch.inference_mode():
        dlm.norm(x, w, keep8=dlm.PACK_E4M3)
    dlm.norm(x, w.detach(), keep8=dlm.PACK_INT8)
    with torch.no_grad(), torch.enable_grad():
        dlm.norm(x, w, keep8=dlm.PACK_E4M3)
    assert formats() == [dlm.PACK_INT8, 0, 0, 0, dlm.PACK_E4M3]
    for off in (False, True):                                # refused all the same
        with torch.set_grad_enabled(not off), pytest.raises(ValueError, match="keep8"):
            dlm.norm(x, w, keep8=5)


def test_device_status_reads_on_the_workspace_s_own_device(monkeypatch):
    """The call that wrote the word ran on its tensors' device and on that
    device's stream: the reading has to wait for that stream."""
    current, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, current[0] = current[0], self.dev

        def __exit__(self, *exc):
            current[0] = self.before

    class Workspace:
        def get_device(self):
            return 1

        def data_ptr(self):
            return 4096

    class Lib:
        @staticmethod
        def dlm_get_device_status(ws, word, stream):
            seen.append((ws, stream))
            word._obj.value = 5
            return 0
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(dlm, "_stream", lambda: ("stream of", current[0]))
    monkeypatch.setattr(dlm, "_lib", Lib)
    assert dlm.device_status(Workspace()) == 5
    current[0] = 1
    assert dlm.device_status(Workspace()) == 5
    assert seen == [(4096, ("stream of", 1))] * 2


def test_sizes_past_32_bits_are_refused_and_not_cut_to_their_low_bits(calls):
    """The library counts columns and table rows in 32 bits, and ctypes cuts what
    does not fit: 2^32 + 256 columns would have come back as 256, the rest of the
    output never written.  (Shapes without memory: nothing is allocated.)"""
    def big(rows, cols, dtype=bf16):
        return torch.empty((rows, cols), dtype=dtype, device="meta")
    n = 2 ** 32 + 256
    ids, lay = torch.zeros(4, dtype=torch.int32), dlm.make_layout(1, 4)
    x, r = big(1, n), torch.zeros(1)
    p = dlm.Packed8(big(1, n, torch.uint8), big(1, n // 128, torch.float32), dlm.PACK_INT8)
    for size in (n, 2 ** 31):
        for fn in (lambda: dlm.embed_bwd_workspace_size(lay, size, 50), lambda: dlm.embed_bwd_workspace_size(lay, 8, size),
                   lambda: dlm.norm_bwd_workspace_size(4, size),
                   lambda: dlm.embed_bwd(lay, ids, torch.zeros(4, 8, dtype=bf16), size)):
            with pytest.raises(ValueError, match="32 bits"):
                fn()
    for fn in (lambda: dlm.embed_fwd(lay, ids, big(n, 2)), lambda: dlm.embed_fwd(lay, ids, big(3, n)),
               lambda: dlm.embed_bwd(lay, ids, big(4, n), 50), lambda: dlm.pack8(x), lambda: dlm.unpack8(p),
               lambda: dlm.norm_fwd(x), lambda: dlm.norm_bwd(x, p, r, r), lambda: dlm.norm_bwd(x, x, r, r)):
        with pytest.raises(ValueError, match="32 bits"):
            fn()
    assert not calls


def test_no_rows_to_accumulate_launch_nothing():
    """d_weight and d_bias are left as they are, bit for bit: adding zeros would
    turn -0 into 0.  (The device check is passed over, so that a launch would
    fail for want of a device.)"""
    if _a_device_may_be_usable():
        pytest.skip("a CUDA device may be usable here: the hook must not run with fake pointers")
    dlm_build.build()
    L = dlm.lib()
    assert L.dlm_test_skip_device_check(1) == 0
    try:
        n = L.dlm_norm_bwd_workspace_size(0, 64)

        def bwd(accumulate, dw, db):
            return L.dlm_norm_bwd(None, 64, None, 64, 0, None, None, None, None, None, 0, 0, 0.0, 0, 64, None, 64, 0,
                                  accumulate, dw, db, 1 << 20, n, None)
        assert bwd(1, 4096, 8192) == 0 and bwd(1, 4096, None) == 0 and bwd(0, None, None) == 0
        assert bwd(0, 4096, None) == 4                     # zeros are written: a launch
    finally:
        assert L.dlm_test_skip_device_check(0) == 0


def test_sizes_past_a_launch_s_blocks_have_no_workspace():
    """A workspace size of 0 for what the call would refuse, whatever the
    gradient's type and the accumulate option."""
    dlm_build.build()
    L = dlm.lib()

    def both(tokens, d, vocab):
        lay = ctypes.byref(dlm.Layout(1, 0, tokens, 16, None))
        codes = {L.dlm_embed_bwd(lay, 16, 16, d, vocab, d, 1.0, gt, acc, 16, d, 256, 2 ** 62, None)
                 for gt in (0, 1) for acc in (0, 1)}
        return L.dlm_embed_bwd_workspace_size(lay, d, vocab), codes
    for tokens, d, vocab in ((2 ** 31 - 1, 10 ** 6, 100), (1, 10 ** 6, 2 ** 31 - 2), (2 ** 31 - 1, 2 ** 17, 2 ** 20),
                             (100, 9000, 2 ** 31 - 2)):
        assert both(tokens, d, vocab) == (0, {1}), (tokens, d, vocab)
    if not _a_device_may_be_usable():
        for tokens, d, vocab in ((2 ** 31 - 1, 16, 100), (2 ** 20, 10 ** 6, 100), (100, 64, 2 ** 31 - 2)):
            size, codes = both(tokens, d, vocab)
            assert size > 0 and 1 not in codes and 3 not in codes, (tokens, d, vocab)
