"""What the binding of the embedding, norm and 8-bit calls hands to the library
and returns to its caller, without a GPU: the library call is replaced by a
recorder, the rest runs as it is."""
import pytest
import torch

import diffusion_lm_loss_b200 as dlm

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
