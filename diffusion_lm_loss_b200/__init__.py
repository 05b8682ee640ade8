"""Python binding of the B200 diffusion-LM noising-plus-loss library.

Argument marshalling only: every step runs in the CUDA kernels of
``libdlm.so`` (built from ``csrc/`` for sm_100a); torch provides device
memory and streams.  There is no CPU fallback -- importing this module
without the built library, or calling it on a non-sm_100 device, raises.

Two layers:
  * ``lib()``: the raw C ABI through ctypes, functions named as in
    ``include/dlm.h`` (``dlm_sample_t``, ``dlm_corrupt``,
    ``dlm_loss_fwd_bwd``, ``dlm_linear_loss_fwd_bwd``, ...);
  * tensor helpers with the same names minus the prefix (``sample_t``,
    ``corrupt``, ``loss_fwd_bwd``, ``linear_loss_fwd_bwd``,
    ``linear_loss_uniform_fwd_bwd``, ``decision_loss_fwd_bwd``, and next to the losses ``embed_fwd`` /
    ``embed_bwd``, ``norm_fwd`` / ``norm_bwd``, ``pack8`` / ``unpack8``) that check every tensor argument's
    dtype, size against the layout and device, allocate outputs and
    workspace with torch on the current device and call the ABI on the
    current torch stream;
  * ``torch.autograd.Function`` wrappers of the four losses
    (``diffusion_loss``, ``linear_diffusion_loss``,
    ``linear_uniform_loss``, ``decision_loss``): the forward runs the fused
    forward + backward call and keeps its gradients; the backward hands them
    over, multiplied by the upstream gradient in the library
    (``dlm_scale_bf16``, which does nothing when that gradient is 1); and of
    the embedding and the norm (``embed``, ``norm``, the norm's input kept in
    8 bits until its backward pass on request).
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdlm.so")

ABSORBING, UNIFORM = 0, 1
ALIGNED, SHIFTED = 0, 1
TIME_WEIGHT_NONE, TIME_WEIGHT_INV_ONE_MINUS_T = 0, 1
REDUCE_TOKEN_MEAN, REDUCE_EXAMPLE_MEAN = 0, 1

DEV_BAD_TOKEN_ID = 0x1
DEV_BAD_LAYOUT = 0x2
DEV_WAIT_TIMEOUT = 0x4
DEV_BAD_LABEL = 0x8

LABEL_HARD, LABEL_DIST, LABEL_SET = 0, 1, 2
LABEL_SOFTMAX_RESTRICTED, LABEL_SOFTMAX_FULL, LABEL_SOFTMAX_BOTH = 1, 2, 3
DECISION_MAX_ANSWERS = 128
DECISION_MAX_SLOTS = 65535

NORM_LAYER, NORM_RMS = 0, 1
PACK_NONE, PACK_INT8, PACK_E4M3 = 0, 1, 2
PACK_BLOCK = 128
# types of parameters and of their gradients (DLM_BF16, DLM_F32)
PARAM_DTYPES = {torch.bfloat16: 0, torch.float32: 1}

STATUS = {0: "DLM_OK", 1: "DLM_ERR_INVALID_ARGUMENT", 2: "DLM_ERR_UNSUPPORTED",
          3: "DLM_ERR_WORKSPACE_TOO_SMALL", 4: "DLM_ERR_CUDA"}

# every symbol include/dlm.h declares
EXPORTS = ("dlm_status_string", "dlm_last_cuda_error", "dlm_version", "dlm_sample_t", "dlm_corrupt",
           "dlm_loss_workspace_size", "dlm_loss_fwd_bwd", "dlm_loss_fwd_bwd_ex", "dlm_loss_fwd_bwd_static",
           "dlm_linear_loss_workspace_size",
           "dlm_linear_loss_fwd_bwd", "dlm_linear_loss_fwd_bwd_ex", "dlm_linear_loss_uniform_workspace_size",
           "dlm_linear_loss_uniform_fwd_bwd", "dlm_decision_workspace_size", "dlm_decision_loss_fwd_bwd",
           "dlm_scale_bf16", "dlm_get_device_status", "dlm_selftest_bounded_wait",
           "dlm_test_skip_device_check", "dlm_embed_fwd", "dlm_embed_bwd_workspace_size", "dlm_embed_bwd",
           "dlm_norm_fwd", "dlm_norm_bwd_workspace_size", "dlm_norm_bwd", "dlm_pack8", "dlm_unpack8")


class DlmError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str = ""):
        super().__init__(f"{where}: {STATUS.get(code, code)}" + (f" [{detail}]" if detail else ""))
        self.code = code


class LossOptions(ctypes.Structure):
    """dlm_loss_options_t: uniform-noise objective options."""
    _fields_ = [("struct_size", ctypes.c_uint32), ("time_weighting", ctypes.c_int32),
                ("weight_clip", ctypes.c_float), ("reduction", ctypes.c_int32),
                ("keep_unscored_rows", ctypes.c_int32)]

    def __init__(self, time_weighting=TIME_WEIGHT_NONE, weight_clip=0.0, reduction=REDUCE_TOKEN_MEAN,
                 keep_unscored_rows=0):
        super().__init__(ctypes.sizeof(LossOptions), time_weighting, weight_clip, reduction,
                         keep_unscored_rows)


class Layout(ctypes.Structure):
    """dlm_layout_t: n_units sequences of seq_len tokens (cu_seqlens NULL) or
    n_units packed documents (cu_seqlens [n_units+1] int32 on the device);
    pad_mask [n_tokens] uint8 on the device (1 = pad) or NULL."""
    _fields_ = [("n_units", ctypes.c_int32), ("seq_len", ctypes.c_int32),
                ("n_tokens", ctypes.c_int64), ("cu_seqlens", ctypes.c_void_p),
                ("pad_mask", ctypes.c_void_p)]


def make_layout(n_units: int, seq_len: int = 0, cu_seqlens: Optional[torch.Tensor] = None,
                pad_mask: Optional[torch.Tensor] = None, n_tokens: Optional[int] = None) -> Layout:
    """A dlm_layout_t over device tensors.  The layout holds references to
    cu_seqlens and pad_mask, whose device pointers it carries, so they stay
    allocated as long as the layout is in use."""
    if n_units < 0 or seq_len < 0 or (n_tokens is not None and n_tokens < 0):
        raise ValueError("n_units, seq_len and n_tokens must be non-negative")
    if cu_seqlens is not None:
        _check(cu_seqlens, torch.int32, "cu_seqlens", min_numel=n_units + 1)
        if n_tokens is None:
            raise ValueError("packed layouts need n_tokens (cu_seqlens lives on the device)")
        cu = cu_seqlens.data_ptr()
    else:
        cu = None
        n_tokens = n_units * seq_len if n_tokens is None else n_tokens
    pm = None
    if pad_mask is not None:
        _check(pad_mask, torch.uint8, "pad_mask", min_numel=n_tokens)
        pm = pad_mask.data_ptr()
    _on_cuda(cu_seqlens=cu_seqlens, pad_mask=pad_mask)
    lay = Layout(n_units, seq_len, n_tokens, cu, pm)
    lay._tensors = (cu_seqlens, pad_mask)
    return lay


_lib = None


def lib():
    """The loaded C ABI (ctypes), with argument and return types declared."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run python -m diffusion_lm_loss_b200.build "
                          "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u64, f32, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64,
                                  ctypes.c_float, ctypes.c_size_t)
    lp = ctypes.POINTER(Layout)
    L.dlm_status_string.restype = ctypes.c_char_p
    L.dlm_status_string.argtypes = [ctypes.c_int]
    L.dlm_last_cuda_error.restype = ctypes.c_char_p
    L.dlm_last_cuda_error.argtypes = []
    L.dlm_version.restype = ctypes.c_int
    L.dlm_version.argtypes = []
    L.dlm_sample_t.restype = ctypes.c_int
    L.dlm_sample_t.argtypes = [u64, i32, i32, f32, vp, vp, vp]
    L.dlm_corrupt.restype = ctypes.c_int
    L.dlm_corrupt.argtypes = [lp, vp, vp, i32, i32, i32, u64, vp, vp, vp, vp]
    L.dlm_loss_workspace_size.restype = sz
    L.dlm_loss_workspace_size.argtypes = [lp, lp]
    L.dlm_loss_fwd_bwd.restype = ctypes.c_int
    L.dlm_loss_fwd_bwd.argtypes = [lp, vp, i64, i32, vp, vp, vp, i32, i32, lp, vp, i64, vp, f32,
                                   f32, vp, vp, vp, vp, vp, sz, vp]
    L.dlm_loss_fwd_bwd_ex.restype = ctypes.c_int
    L.dlm_loss_fwd_bwd_ex.argtypes = [lp, vp, i64, i32, vp, vp, vp, i32, i32, lp, vp, i64, vp, f32,
                                      f32, ctypes.POINTER(LossOptions), vp, vp, vp, vp, vp, sz, vp]
    L.dlm_loss_fwd_bwd_static.restype = ctypes.c_int
    L.dlm_loss_fwd_bwd_static.argtypes = [lp, vp, i64, i32, vp, vp, vp, i32, i32, lp, vp, i64, vp, f32,
                                          f32, vp, vp, vp, vp, vp]
    L.dlm_linear_loss_workspace_size.restype = sz
    L.dlm_linear_loss_workspace_size.argtypes = [lp, i32, i32]
    L.dlm_linear_loss_fwd_bwd.restype = ctypes.c_int
    L.dlm_linear_loss_fwd_bwd.argtypes = [lp, vp, vp, i32, i32, vp, vp, vp, f32, vp, vp, vp, vp,
                                          vp, sz, vp]
    L.dlm_linear_loss_fwd_bwd_ex.restype = ctypes.c_int
    L.dlm_linear_loss_fwd_bwd_ex.argtypes = [lp, vp, vp, i32, i32, vp, vp, vp, i32, f32, vp, vp, vp, vp,
                                             vp, sz, vp]
    L.dlm_linear_loss_uniform_workspace_size.restype = sz
    L.dlm_linear_loss_uniform_workspace_size.argtypes = [lp, lp, i32, i32]
    L.dlm_linear_loss_uniform_fwd_bwd.restype = ctypes.c_int
    L.dlm_linear_loss_uniform_fwd_bwd.argtypes = [lp, vp, lp, vp, vp, vp, i32, i32, vp, i32, f32, f32,
                                                  vp, vp, vp, vp, vp, vp, sz, vp]
    L.dlm_decision_workspace_size.restype = sz
    L.dlm_decision_workspace_size.argtypes = [i32, i32]
    L.dlm_decision_loss_fwd_bwd.restype = ctypes.c_int
    L.dlm_decision_loss_fwd_bwd.argtypes = [i32, vp, i64, i64, i32, vp, vp, i64, vp, vp, vp, i32, f32, f32, f32, vp,
                                            vp, vp, i64, vp, sz, vp]
    L.dlm_scale_bf16.restype = ctypes.c_int
    L.dlm_scale_bf16.argtypes = [vp, i64, i64, i64, vp, vp]
    L.dlm_test_skip_device_check.restype = ctypes.c_int
    L.dlm_test_skip_device_check.argtypes = [i32]
    L.dlm_selftest_bounded_wait.restype = ctypes.c_int
    L.dlm_selftest_bounded_wait.argtypes = [u64, vp, vp]
    L.dlm_embed_fwd.restype = ctypes.c_int
    L.dlm_embed_fwd.argtypes = [lp, vp, vp, i64, i32, i32, f32, vp, i64, vp, vp]
    L.dlm_embed_bwd_workspace_size.restype = sz
    L.dlm_embed_bwd_workspace_size.argtypes = [lp, i32, i32]
    L.dlm_embed_bwd.restype = ctypes.c_int
    L.dlm_embed_bwd.argtypes = [lp, vp, vp, i64, i32, i32, f32, i32, i32, vp, i64, vp, sz, vp]
    L.dlm_norm_fwd.restype = ctypes.c_int
    L.dlm_norm_fwd.argtypes = [vp, i64, i32, i64, vp, vp, i32, i32, f32, f32, vp, i64, vp, vp, i32, vp, vp, vp]
    L.dlm_norm_bwd_workspace_size.restype = sz
    L.dlm_norm_bwd_workspace_size.argtypes = [i64, i32]
    L.dlm_norm_bwd.restype = ctypes.c_int
    L.dlm_norm_bwd.argtypes = [vp, i64, vp, i64, i32, vp, vp, vp, vp, vp, i32, i32, f32, i64, i32, vp, i64, i32, i32,
                               vp, vp, vp, sz, vp]
    L.dlm_pack8.restype = ctypes.c_int
    L.dlm_pack8.argtypes = [vp, i64, i32, i64, i32, vp, vp, vp]
    L.dlm_unpack8.restype = ctypes.c_int
    L.dlm_unpack8.argtypes = [vp, vp, i64, i32, i32, vp, i64, vp]
    L.dlm_get_device_status.restype = ctypes.c_int
    L.dlm_get_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    _lib = L
    return L


def _check(t: Optional[torch.Tensor], dtype, name: str, min_numel: Optional[int] = None,
           min_rows: Optional[int] = None, min_cols: Optional[int] = None):
    """A tensor argument before its pointer goes to the library: dtype and
    size (the C ABI sees only pointers, so a buffer shorter than the layout
    says would be read or written out of bounds on the device).  The device
    is checked afterwards, for all arguments of a call together (_on_cuda).
    min_numel: a contiguous buffer of at least that many elements; min_rows /
    min_cols: a 2-D tensor with unit column stride and at least that many rows
    / columns."""
    if t is None:
        raise ValueError(f"{name}: required")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if min_numel is not None:
        if not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if t.numel() < min_numel:
            raise ValueError(f"{name}: needs at least {min_numel} elements, has {t.numel()}")
    if min_rows is not None or min_cols is not None:
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name}: must be 2-D with unit column stride, got shape {tuple(t.shape)}")
        if min_rows is not None and t.shape[0] < min_rows:
            raise ValueError(f"{name}: needs at least {min_rows} rows, has {t.shape[0]}")
        if min_cols is not None and t.shape[1] < min_cols:
            raise ValueError(f"{name}: needs at least {min_cols} columns, has {t.shape[1]}")


def _on_cuda(**tensors):
    """Every tensor argument of a call (None = not given) on one CUDA device."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name}: must be a CUDA tensor (there is no CPU path)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name}: on {t.device}, the other arguments on {dev}")


def _like_rows(t: torch.Tensor, zero: bool = False) -> torch.Tensor:
    """A buffer with t's shape and strides (a gradient is written with the
    row stride of its input, which may be wider than the row)."""
    out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=t.device)
    return out.zero_() if zero else out


def _check_grad(g: Optional[torch.Tensor], like: torch.Tensor, name: str):
    """A caller-supplied gradient buffer: same dtype, shape and row stride as
    the input it is the gradient of."""
    _check(g, like.dtype, name)
    if tuple(g.shape) != tuple(like.shape) or (like.dim() == 2 and g.stride(0) != like.stride(0)):
        raise ValueError(f"{name}: must have the shape {tuple(like.shape)} and row stride "
                         f"{like.stride(0)} of its input")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream():
    """The current stream of the current device, as an address (the raw
    lookup: building torch.cuda.current_stream() costs 3 us a call)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ok(code: int, where: str):
    if code != 0:
        detail = lib().dlm_last_cuda_error().decode() if code == 4 else ""
        raise DlmError(code, where, detail)


def _call(dev: int, name: str, *args):
    """A library call on the current stream of CUDA device `dev`, which becomes
    the current device for it (-1: of the current one)."""
    fn = getattr(_lib or lib(), name)
    if dev >= 0 and dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            _ok(fn(*args, _stream()), name)
    else:
        _ok(fn(*args, _stream()), name)


def _check_out(loss: torch.Tensor, unit_loss: Optional[torch.Tensor], layout: Layout,
               workspace: torch.Tensor):
    """The scalar outputs and the workspace of a reused result object (the
    library itself checks the workspace's size against the call)."""
    _check(loss, torch.float32, "out.loss", min_numel=1)
    if unit_loss is not None:
        _check(unit_loss, torch.float32, "out.unit_loss", min_numel=layout.n_units)
    _check(workspace, torch.uint8, "out.workspace", min_numel=0)


def _bits(t: torch.Tensor) -> torch.Tensor:
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


# --------------------------------------------------------------------------
# tensor helpers
# --------------------------------------------------------------------------
def sample_t(seed: int, n_units: int, mode: int = ABSORBING, eps: float = 1e-3,
             device=None):
    """(t, p): float32 [n_units] on the current (or given) CUDA device."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    t = torch.empty(n_units, dtype=torch.float32, device=dev)
    p = torch.empty(n_units, dtype=torch.float32, device=dev)
    _ok(lib().dlm_sample_t(seed, n_units, mode, eps, _ptr(t), _ptr(p), _stream()), "dlm_sample_t")
    return t, p


def corrupt(layout: Layout, clean_ids: torch.Tensor, p: torch.Tensor, mode: int = ABSORBING,
            mask_id: int = 0, vocab: int = 0, seed: int = 0,
            dev_status: Optional[torch.Tensor] = None):
    """(noisy int32, corrupted uint8), same length as clean_ids."""
    _check(clean_ids, torch.int32, "clean_ids", min_numel=layout.n_tokens)
    _check(p, torch.float32, "p", min_numel=layout.n_units)
    if dev_status is not None and (dev_status.dtype not in (torch.int32, torch.uint32) or dev_status.numel() < 1):
        raise ValueError("dev_status: an int32 / uint32 tensor of at least one element")
    _on_cuda(clean_ids=clean_ids, p=p, dev_status=dev_status)
    noisy = torch.empty_like(clean_ids)
    corr = torch.empty(clean_ids.shape, dtype=torch.uint8, device=clean_ids.device)
    _ok(lib().dlm_corrupt(ctypes.byref(layout), _ptr(clean_ids), _ptr(p), mode, mask_id, vocab, seed,
                          _ptr(noisy), _ptr(corr), _ptr(dev_status), _stream()), "dlm_corrupt")
    return noisy, corr


@dataclass
class LossOut:
    loss: torch.Tensor            # float32 [1]
    unit_loss: torch.Tensor       # float32 [n_units]
    dlogits: torch.Tensor         # bf16, logits' shape
    enc_dlogits: Optional[torch.Tensor]
    workspace: torch.Tensor       # uint8; holds the device status word

    def device_status(self) -> int:
        return device_status(self.workspace)


def loss_workspace_size(layout: Layout, enc_layout: Optional[Layout] = None) -> int:
    return int(lib().dlm_loss_workspace_size(ctypes.byref(layout),
                                             ctypes.byref(enc_layout) if enc_layout else None))


def loss_fwd_bwd(layout: Layout, logits: torch.Tensor, vocab: int, clean_ids: torch.Tensor,
                 corrupted: Optional[torch.Tensor], p: Optional[torch.Tensor],
                 mode: int = ABSORBING, align: int = ALIGNED,
                 enc_layout: Optional[Layout] = None, enc_logits: Optional[torch.Tensor] = None,
                 enc_ids: Optional[torch.Tensor] = None, enc_ar_weight: float = 1.0,
                 grad_scale: float = 1.0, out: Optional[LossOut] = None,
                 options: Optional[LossOptions] = None) -> LossOut:
    """Weighted CE forward + backward (see dlm_loss_fwd_bwd).  logits: bf16
    [rows, ld] (2-D, row stride ld >= vocab).  Reuses the buffers of `out`
    when given (no allocation)."""
    T = layout.n_tokens
    _check(logits, torch.bfloat16, "logits", min_rows=T, min_cols=vocab)
    _check(clean_ids, torch.int32, "clean_ids", min_numel=T)
    if corrupted is not None or (mode == ABSORBING and T > 0):
        _check(corrupted, torch.uint8, "corrupted", min_numel=T)
    if p is not None:
        _check(p, torch.float32, "p", min_numel=layout.n_units)
    ld = logits.stride(0)
    enc_ld = 0
    if enc_logits is not None:
        if enc_layout is None:
            raise ValueError("enc_logits needs enc_layout")
        _check(enc_logits, torch.bfloat16, "enc_logits", min_rows=enc_layout.n_tokens, min_cols=vocab)
        _check(enc_ids, torch.int32, "enc_ids", min_numel=enc_layout.n_tokens)
        enc_ld = enc_logits.stride(0)
    if out is not None:
        _check_out(out.loss, out.unit_loss, layout, out.workspace)
        _check_grad(out.dlogits, logits, "out.dlogits")
        if enc_logits is not None:
            _check_grad(out.enc_dlogits, enc_logits, "out.enc_dlogits")
    o = out if out is not None else LossOut(None, None, None, None, None)
    _on_cuda(logits=logits, clean_ids=clean_ids, corrupted=corrupted, p=p, enc_logits=enc_logits,
             enc_ids=enc_ids, loss=o.loss, unit_loss=o.unit_loss, workspace=o.workspace, dlogits=o.dlogits,
             enc_dlogits=o.enc_dlogits if enc_logits is not None else None)
    dev = logits.device
    keep = options is not None and options.keep_unscored_rows
    if out is None:
        ws = _aligned_workspace(loss_workspace_size(layout, enc_layout), dev, 256)
        # rows the call leaves untouched must start as zeros
        out = LossOut(torch.empty(1, dtype=torch.float32, device=dev),
                      torch.empty(max(layout.n_units, 1), dtype=torch.float32, device=dev),
                      _like_rows(logits, keep),
                      _like_rows(enc_logits, keep) if enc_logits is not None else None, ws)
    if options is None:
        _ok(lib().dlm_loss_fwd_bwd(
            ctypes.byref(layout), _ptr(logits), ld, vocab, _ptr(clean_ids), _ptr(corrupted), _ptr(p),
            mode, align, ctypes.byref(enc_layout) if enc_layout is not None else None,
            _ptr(enc_logits), enc_ld, _ptr(enc_ids), enc_ar_weight, grad_scale, _ptr(out.loss),
            _ptr(out.unit_loss), _ptr(out.dlogits), _ptr(out.enc_dlogits), _ptr(out.workspace),
            out.workspace.numel(), _stream()), "dlm_loss_fwd_bwd")
    else:
        _ok(lib().dlm_loss_fwd_bwd_ex(
            ctypes.byref(layout), _ptr(logits), ld, vocab, _ptr(clean_ids), _ptr(corrupted), _ptr(p),
            mode, align, ctypes.byref(enc_layout) if enc_layout is not None else None,
            _ptr(enc_logits), enc_ld, _ptr(enc_ids), enc_ar_weight, grad_scale, ctypes.byref(options),
            _ptr(out.loss), _ptr(out.unit_loss), _ptr(out.dlogits), _ptr(out.enc_dlogits),
            _ptr(out.workspace), out.workspace.numel(), _stream()), "dlm_loss_fwd_bwd_ex")
    return out


@dataclass
class LinearOut:
    loss: torch.Tensor
    unit_loss: torch.Tensor
    d_hidden: torch.Tensor
    d_weight: Optional[torch.Tensor]
    workspace: torch.Tensor
    d_enc_hidden: Optional[torch.Tensor] = None

    def device_status(self) -> int:
        return device_status(self.workspace)


def _new(dev, dtype: torch.dtype, rows: int, cols: Optional[int] = None) -> torch.Tensor:
    """An uninitialised contiguous tensor [rows] or [rows, cols] on device
    `dev` (empty_strided: 0.8 us a tensor less than torch.empty, 0.4 less than
    new_empty)."""
    if cols is None:
        return torch.empty_strided((rows,), (1,), dtype=dtype, device=dev)
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _aligned_workspace(nbytes: int, device, align: int = 1024) -> torch.Tensor:
    """A uint8 workspace whose first byte is `align`-byte aligned (the loss
    needs 256, the fused head 1024; the caching allocator guarantees 512 and
    other allocators less): where that is not so by itself, a slice of a
    slightly larger buffer, which the slice keeps alive.  (Two buffers are never
    held at once, and one as large as the fused head's is asked for once.)"""
    if align <= 512:
        buf = torch.empty_strided((nbytes,), (1,), dtype=torch.uint8, device=device)
        if buf.data_ptr() % align == 0:
            return buf
        del buf
    buf = torch.empty(nbytes + align - 1, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % align
    return buf[off:off + nbytes]


def _check_head(layout: Layout, hidden: torch.Tensor, weight: torch.Tensor):
    """hidden [n_tokens, D] and weight [V, D], contiguous bf16; returns (T, D, V)."""
    T = layout.n_tokens
    _check(hidden, torch.bfloat16, "hidden", min_numel=0)
    _check(weight, torch.bfloat16, "weight", min_numel=0)
    if hidden.dim() != 2 or weight.dim() != 2 or hidden.shape[1] != weight.shape[1]:
        raise ValueError("hidden [tokens, d_model] and weight [vocab, d_model] must share d_model")
    if hidden.shape[0] < T:
        raise ValueError(f"hidden: needs at least {T} rows, has {hidden.shape[0]}")
    return T, int(hidden.shape[1]), int(weight.shape[0])


def linear_loss_workspace_size(layout: Layout, d_model: int, vocab: int) -> int:
    return int(lib().dlm_linear_loss_workspace_size(ctypes.byref(layout), d_model, vocab))


def linear_loss_fwd_bwd(layout: Layout, hidden: torch.Tensor, weight: torch.Tensor,
                        clean_ids: torch.Tensor, corrupted: torch.Tensor, p: torch.Tensor,
                        grad_scale: float = 1.0, want_d_weight: bool = True,
                        out: Optional[LinearOut] = None, align: int = ALIGNED) -> LinearOut:
    """Fused lm_head + absorbing loss (see dlm_linear_loss_fwd_bwd; align =
    SHIFTED goes through dlm_linear_loss_fwd_bwd_ex)."""
    T, D, V = _check_head(layout, hidden, weight)
    _check(clean_ids, torch.int32, "clean_ids", min_numel=T)
    _check(corrupted, torch.uint8, "corrupted", min_numel=T)
    _check(p, torch.float32, "p", min_numel=layout.n_units)
    if out is not None:
        _check_out(out.loss, out.unit_loss, layout, out.workspace)
        _check_grad(out.d_hidden, hidden, "out.d_hidden")
        if out.d_weight is not None:
            _check_grad(out.d_weight, weight, "out.d_weight")
    o = out if out is not None else LinearOut(None, None, None, None, None)
    _on_cuda(hidden=hidden, weight=weight, clean_ids=clean_ids, corrupted=corrupted, p=p, loss=o.loss,
             unit_loss=o.unit_loss, workspace=o.workspace, d_hidden=o.d_hidden, d_weight=o.d_weight)
    dev = hidden.device
    if out is None:
        ws = _aligned_workspace(linear_loss_workspace_size(layout, D, V), dev)
        out = LinearOut(torch.empty(1, dtype=torch.float32, device=dev),
                        torch.empty(max(layout.n_units, 1), dtype=torch.float32, device=dev),
                        torch.empty_like(hidden),
                        torch.empty_like(weight) if want_d_weight else None, ws)
    if align == ALIGNED:
        _ok(lib().dlm_linear_loss_fwd_bwd(
            ctypes.byref(layout), _ptr(hidden), _ptr(weight), D, V, _ptr(clean_ids), _ptr(corrupted),
            _ptr(p), grad_scale, _ptr(out.loss), _ptr(out.unit_loss), _ptr(out.d_hidden),
            _ptr(out.d_weight), _ptr(out.workspace), out.workspace.numel(), _stream()),
            "dlm_linear_loss_fwd_bwd")
    else:
        _ok(lib().dlm_linear_loss_fwd_bwd_ex(
            ctypes.byref(layout), _ptr(hidden), _ptr(weight), D, V, _ptr(clean_ids), _ptr(corrupted),
            _ptr(p), align, grad_scale, _ptr(out.loss), _ptr(out.unit_loss), _ptr(out.d_hidden),
            _ptr(out.d_weight), _ptr(out.workspace), out.workspace.numel(), _stream()),
            "dlm_linear_loss_fwd_bwd_ex")
    return out


def linear_loss_uniform_workspace_size(layout: Layout, enc_layout: Optional[Layout], d_model: int,
                                       vocab: int) -> int:
    enc = ctypes.byref(enc_layout) if enc_layout is not None else None
    return int(lib().dlm_linear_loss_uniform_workspace_size(ctypes.byref(layout), enc, d_model, vocab))


def linear_loss_uniform_fwd_bwd(layout: Layout, hidden: torch.Tensor, weight: torch.Tensor,
                                clean_ids: torch.Tensor, enc_layout: Optional[Layout] = None,
                                enc_hidden: Optional[torch.Tensor] = None,
                                enc_ids: Optional[torch.Tensor] = None, enc_ar_weight: float = 1.0,
                                align: int = ALIGNED, grad_scale: float = 1.0, want_d_weight: bool = True,
                                out: Optional[LinearOut] = None) -> LinearOut:
    """Fused lm_head + uniform-noise loss with the optional encoder
    next-token term (see dlm_linear_loss_uniform_fwd_bwd)."""
    T, D, V = _check_head(layout, hidden, weight)
    _check(clean_ids, torch.int32, "clean_ids", min_numel=T)
    if enc_layout is not None:
        Te = enc_layout.n_tokens
        _check(enc_hidden, torch.bfloat16, "enc_hidden", min_numel=Te * D)
        if enc_hidden.dim() != 2 or enc_hidden.shape[1] != D:
            raise ValueError("enc_hidden must be [enc_tokens, d_model]")
        _check(enc_ids, torch.int32, "enc_ids", min_numel=Te)
    if out is not None:
        _check_out(out.loss, out.unit_loss, layout, out.workspace)
        _check_grad(out.d_hidden, hidden, "out.d_hidden")
        if out.d_weight is not None:
            _check_grad(out.d_weight, weight, "out.d_weight")
        if enc_layout is not None:
            _check_grad(out.d_enc_hidden, enc_hidden, "out.d_enc_hidden")
    o = out if out is not None else LinearOut(None, None, None, None, None)
    _on_cuda(hidden=hidden, weight=weight, clean_ids=clean_ids, enc_hidden=enc_hidden, enc_ids=enc_ids,
             loss=o.loss, unit_loss=o.unit_loss, workspace=o.workspace, d_hidden=o.d_hidden,
             d_weight=o.d_weight, d_enc_hidden=o.d_enc_hidden if enc_layout is not None else None)
    dev = hidden.device
    if out is None:
        ws = _aligned_workspace(linear_loss_uniform_workspace_size(layout, enc_layout, D, V), dev)
        out = LinearOut(torch.empty(1, dtype=torch.float32, device=dev),
                        torch.empty(max(layout.n_units, 1), dtype=torch.float32, device=dev),
                        torch.empty_like(hidden),
                        torch.empty_like(weight) if want_d_weight else None, ws,
                        torch.empty_like(enc_hidden) if enc_layout is not None else None)
    enc = ctypes.byref(enc_layout) if enc_layout is not None else None
    _ok(lib().dlm_linear_loss_uniform_fwd_bwd(
        ctypes.byref(layout), _ptr(hidden), enc, _ptr(enc_hidden), _ptr(enc_ids), _ptr(weight), D, V,
        _ptr(clean_ids), align, enc_ar_weight, grad_scale, _ptr(out.loss), _ptr(out.unit_loss),
        _ptr(out.d_hidden), _ptr(out.d_enc_hidden), _ptr(out.d_weight), _ptr(out.workspace),
        out.workspace.numel(), _stream()),
        "dlm_linear_loss_uniform_fwd_bwd")
    return out


@dataclass
class DecisionOut:
    loss: torch.Tensor            # float32 [1]
    slot_loss: torch.Tensor       # float32 [n_slots]: each slot's share of the loss
    dlogits: torch.Tensor         # bf16 [n_slots, vocab]: row i = slot i
    workspace: torch.Tensor       # uint8; holds the device status word

    def device_status(self) -> int:
        return device_status(self.workspace)


def decision_workspace_size(n_slots: int, vocab: int) -> int:
    return int(lib().dlm_decision_workspace_size(n_slots, vocab))


def decision_loss_fwd_bwd(logits: torch.Tensor, vocab: int, cand_off: torch.Tensor, cand_ids: torch.Tensor,
                          label_kind: torch.Tensor, label_val: torch.Tensor,
                          slot_rows: Optional[torch.Tensor] = None,
                          label_softmax: int = LABEL_SOFTMAX_BOTH, brier_weight: float = 0.1,
                          hard_label_smoothing: float = 0.0, grad_scale: float = 1.0,
                          out: Optional[DecisionOut] = None) -> DecisionOut:
    """Typed-decision losses at label slots (see dlm_decision_loss_fwd_bwd).
    logits: bf16 [rows, ld]; slot i reads row slot_rows[i] (int64), or row i
    when slot_rows is None.  cand_off int32 [n_slots + 1]; cand_ids int32 and
    label_val float32 of the same length; label_kind int32 [n_slots].  Rows
    and offsets that leave these arrays (device data) are refused by the
    kernels (DEV_BAD_LAYOUT)."""
    n = int(cand_off.numel()) - 1
    if n < 0:
        raise ValueError("cand_off: needs n_slots + 1 entries")
    _check(cand_off, torch.int32, "cand_off", min_numel=n + 1)
    _check(label_kind, torch.int32, "label_kind", min_numel=n)
    _check(cand_ids, torch.int32, "cand_ids", min_numel=0)
    _check(label_val, torch.float32, "label_val", min_numel=cand_ids.numel())
    rows_needed = n
    if slot_rows is not None:
        _check(slot_rows, torch.int64, "slot_rows", min_numel=n)
        rows_needed = 1
    _check(logits, torch.bfloat16, "logits", min_rows=rows_needed if n > 0 else 0, min_cols=vocab)
    if out is not None:
        _check(out.loss, torch.float32, "out.loss", min_numel=1)
        _check(out.slot_loss, torch.float32, "out.slot_loss", min_numel=n)
        _check(out.dlogits, torch.bfloat16, "out.dlogits", min_rows=n, min_cols=vocab)
        _check(out.workspace, torch.uint8, "out.workspace", min_numel=0)
    o = out if out is not None else DecisionOut(None, None, None, None)
    _on_cuda(logits=logits, cand_off=cand_off, cand_ids=cand_ids, label_kind=label_kind, label_val=label_val,
             slot_rows=slot_rows, loss=o.loss, slot_loss=o.slot_loss, dlogits=o.dlogits, workspace=o.workspace)
    dev = logits.device
    if out is None:
        out = DecisionOut(torch.empty(1, dtype=torch.float32, device=dev),
                          torch.empty(max(n, 1), dtype=torch.float32, device=dev),
                          torch.empty((n, vocab), dtype=torch.bfloat16, device=dev),
                          _aligned_workspace(decision_workspace_size(n, vocab), dev, 256))
    _ok(lib().dlm_decision_loss_fwd_bwd(
        n, _ptr(logits), max(int(logits.shape[0]), 1), logits.stride(0), vocab, _ptr(slot_rows), _ptr(cand_off),
        int(cand_ids.numel()), _ptr(cand_ids),
        _ptr(label_kind), _ptr(label_val), label_softmax, brier_weight, hard_label_smoothing, grad_scale,
        _ptr(out.loss), _ptr(out.slot_loss), _ptr(out.dlogits), out.dlogits.stride(0), _ptr(out.workspace),
        out.workspace.numel(), _stream()), "dlm_decision_loss_fwd_bwd")
    return out


def device_status(workspace: torch.Tensor) -> int:
    """Device status word of a workspace (synchronises the current stream of
    its device)."""
    v = ctypes.c_uint32(0)
    _call(workspace.get_device(), "dlm_get_device_status", workspace.data_ptr(), ctypes.byref(v))
    return int(v.value)


# --------------------------------------------------------------------------
# embedding, norm, activations in 8 bits
# --------------------------------------------------------------------------
def _all_on(dev: int, *tensors) -> bool:
    """Whether these (None = not given) are on CUDA device `dev`: the quick
    form of _on_cuda, which words what is wrong where it is not so."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            return False
    return dev >= 0


def _check_rows(t: Optional[torch.Tensor], dtype, name: str, rows: int, cols: int) -> int:
    """A [rows, cols] argument with unit column stride (`rows`: at least so
    many); its row stride."""
    if t is not None and t.dtype is dtype and t.dim() == 2:     # the usual case, without a message to word
        (n, m), (ld, unit) = t.shape, t.stride()
        if n >= rows and m == cols and (unit == 1 or cols <= 1):
            if n <= 1:
                return cols
            if ld >= cols:
                return ld
    _check(t, dtype, name, min_rows=rows)
    if t.shape[1] != cols:
        raise ValueError(f"{name}: must have {cols} columns, has {t.shape[1]}")
    ld = t.stride(0) if t.shape[0] > 1 else cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap (row stride {ld}, {cols} columns)")
    return ld


def _in_32_bits(*sizes: int):
    """Sizes that the C ABI takes as int32 (ctypes would cut larger ones to
    their low bits)."""
    for n in sizes:
        if not -2 ** 31 <= n < 2 ** 31:
            raise ValueError(f"a size of {n}: columns and table rows are counted in 32 bits")


def _shape2(t: torch.Tensor, name: str):
    """(rows, columns) of a matrix."""
    if t.dim() != 2:
        raise ValueError(f"{name}: must be 2-D, got shape {tuple(t.shape)}")
    _in_32_bits(t.shape[1])
    return t.shape


def _as_rows(t: torch.Tensor) -> torch.Tensor:
    """An upstream gradient [rows, cols] as _check_rows wants it (an expanded
    or transposed one is copied)."""
    ok = t.shape[1] <= 1 or t.stride(1) == 1
    return t if ok and (t.shape[0] <= 1 or t.stride(0) >= t.shape[1]) else t.contiguous()


def _param_dtype(dtype, name: str) -> int:
    if dtype not in PARAM_DTYPES:
        raise TypeError(f"{name}: expected torch.bfloat16 or torch.float32, got {dtype}")
    return PARAM_DTYPES[dtype]


def _pad_mask(layout: Layout) -> Optional[torch.Tensor]:
    """The pad mask of a layout from make_layout."""
    return getattr(layout, "_tensors", (None, None))[1]


def embed_fwd(layout: Layout, ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              out: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * weight[ids] as bf16 [n_tokens, d_model] (see dlm_embed_fwd);
    rows of pads are zeros.  dev_status: an int32 / uint32 tensor that gets
    DEV_BAD_TOKEN_ID or'ed in when an id is outside the table."""
    T = layout.n_tokens
    _check(ids, torch.int32, "ids", min_numel=T)
    V, D = weight.shape if weight.dim() == 2 else (0, 0)
    if V < 1 or D < 1:
        raise ValueError("weight: [vocab, d_model]")
    _in_32_bits(V, D)
    ld_w = _check_rows(weight, torch.bfloat16, "weight", V, D)
    if dev_status is not None and (dev_status.dtype not in (torch.int32, torch.uint32) or dev_status.numel() < 1):
        raise ValueError("dev_status: an int32 / uint32 tensor of at least one element")
    ld_out = D if out is None else _check_rows(out, torch.bfloat16, "out", T, D)
    dev, pad = weight.get_device(), _pad_mask(layout)
    if not _all_on(dev, ids, out, dev_status, pad):
        _on_cuda(ids=ids, weight=weight, out=out, dev_status=dev_status, pad_mask=pad)
    if out is None:
        out = _new(weight.device, torch.bfloat16, T, D)
    _call(dev, "dlm_embed_fwd", ctypes.byref(layout), ids.data_ptr(), weight.data_ptr(), ld_w, V, D, scale,
          out.data_ptr(), ld_out, _ptr(dev_status))
    return out


@dataclass
class EmbedGrad:
    d_weight: torch.Tensor        # bf16 or float32 [vocab, d_model]
    workspace: torch.Tensor       # uint8; holds the device status word

    def device_status(self) -> int:
        return device_status(self.workspace)


def embed_bwd_workspace_size(layout: Layout, d_model: int, vocab: int) -> int:
    _in_32_bits(d_model, vocab)
    return int(lib().dlm_embed_bwd_workspace_size(ctypes.byref(layout), d_model, vocab))


def embed_bwd(layout: Layout, ids: torch.Tensor, d_out: torch.Tensor, vocab: int, scale: float = 1.0,
              grad_dtype: torch.dtype = torch.bfloat16, d_weight: Optional[torch.Tensor] = None,
              accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> EmbedGrad:
    """Gradient of embed_fwd's table (see dlm_embed_bwd), in a new tensor of
    grad_dtype or in `d_weight` (whose type then counts).  accumulate: added to
    what d_weight holds, e.g. the d_weight of a tied output head."""
    T = layout.n_tokens
    _check(ids, torch.int32, "ids", min_numel=T)
    D = d_out.shape[1] if d_out.dim() == 2 else 1
    if D < 1 or vocab < 1:
        raise ValueError("d_out and the table need at least one column and one row")
    _in_32_bits(D, vocab)
    ld = _check_rows(d_out, torch.bfloat16, "d_out", T, D)
    if accumulate and d_weight is None:
        raise ValueError("accumulate needs d_weight")
    if d_weight is not None:
        grad_dtype = d_weight.dtype
    gt = _param_dtype(grad_dtype, "grad_dtype" if d_weight is None else "d_weight")
    ld_dw = D if d_weight is None else _check_rows(d_weight, grad_dtype, "d_weight", vocab, D)
    if workspace is not None:
        _check(workspace, torch.uint8, "workspace", min_numel=0)
    dev, pad = d_out.get_device(), _pad_mask(layout)
    if not _all_on(dev, ids, d_weight, workspace, pad):
        _on_cuda(ids=ids, d_out=d_out, d_weight=d_weight, workspace=workspace, pad_mask=pad)
    if d_weight is None:
        d_weight = _new(d_out.device, grad_dtype, vocab, D)
    if workspace is None:
        workspace = _aligned_workspace(embed_bwd_workspace_size(layout, D, vocab), d_out.device, 256)
    _call(dev, "dlm_embed_bwd", ctypes.byref(layout), ids.data_ptr(), d_out.data_ptr(), ld, vocab, D, scale, gt,
          int(accumulate), d_weight.data_ptr(), ld_dw, workspace.data_ptr(), workspace.numel())
    return EmbedGrad(d_weight, workspace)


@dataclass
class Packed8:
    """An activation [rows, cols] in 8 bits (see dlm_pack8)."""
    q: torch.Tensor               # uint8 [rows, cols]: the codes' bytes
    scale: torch.Tensor           # float32 [rows, ceil(cols / PACK_BLOCK)]
    format: int                   # PACK_INT8 | PACK_E4M3

    @property
    def shape(self):
        return self.q.shape


def _empty_packed(rows: int, cols: int, fmt: int, dev) -> Packed8:
    return Packed8(_new(dev, torch.uint8, rows, cols), _new(dev, torch.float32, rows, -(-cols // PACK_BLOCK)), fmt)


def _check_packed(p: Packed8, rows: int, cols: int, name: str):
    if p.format not in (PACK_INT8, PACK_E4M3):
        raise ValueError(f"{name}: format must be PACK_INT8 or PACK_E4M3")
    _check(p.q, torch.uint8, f"{name}.q", min_numel=0)
    _check(p.scale, torch.float32, f"{name}.scale", min_numel=0)
    if tuple(p.q.shape) != (rows, cols) or tuple(p.scale.shape) != (rows, -(-cols // PACK_BLOCK)):
        raise ValueError(f"{name}: q [{rows}, {cols}] and scale [{rows}, {-(-cols // PACK_BLOCK)}], got "
                         f"{tuple(p.q.shape)} and {tuple(p.scale.shape)}")


def pack8(x: torch.Tensor, format: int = PACK_INT8, out: Optional[Packed8] = None) -> Packed8:
    """x (bf16 [rows, cols]) in 8 bits, one float factor per PACK_BLOCK
    columns (see dlm_pack8)."""
    rows, cols = _shape2(x, "x")
    ld = _check_rows(x, torch.bfloat16, "x", rows, cols)
    if out is not None:
        _check_packed(out, rows, cols, "out")
        if out.format != format:
            raise ValueError("out: has another format")
    elif format not in (PACK_INT8, PACK_E4M3):
        raise ValueError("format: PACK_INT8 or PACK_E4M3")
    dev = x.get_device()
    if not (_all_on(dev) if out is None else _all_on(dev, out.q, out.scale)):
        _on_cuda(x=x, q=out.q if out is not None else None, scale=out.scale if out is not None else None)
    if out is None:
        out = _empty_packed(rows, cols, format, x.device)
    _call(dev, "dlm_pack8", x.data_ptr(), rows, cols, ld, format, out.q.data_ptr(), out.scale.data_ptr())
    return out


def unpack8(packed: Packed8, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The bf16 values that pack8's (or norm_fwd's) codes stand for."""
    rows, cols = _shape2(packed.q, "packed.q")
    _check_packed(packed, rows, cols, "packed")
    ld = cols if out is None else _check_rows(out, torch.bfloat16, "out", rows, cols)
    dev = packed.q.get_device()
    if not _all_on(dev, packed.scale, out):
        _on_cuda(q=packed.q, scale=packed.scale, out=out)
    if out is None:
        out = _new(packed.q.device, torch.bfloat16, rows, cols)
    _call(dev, "dlm_unpack8", packed.q.data_ptr(), packed.scale.data_ptr(), rows, cols, packed.format, out.data_ptr(),
          ld)
    return out


@dataclass
class NormOut:
    y: torch.Tensor               # bf16 [rows, d_model]
    mean: Optional[torch.Tensor]  # float32 [rows] (None: RMS)
    rstd: torch.Tensor            # float32 [rows]
    packed: Optional[Packed8]     # x in 8 bits, when asked for


def _check_params(weight: Optional[torch.Tensor], bias: Optional[torch.Tensor], cols: int) -> int:
    """weight and bias [cols] of one type; its DLM_* number."""
    dtype = None
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is None:
            continue
        dt = _param_dtype(t.dtype, name)
        if t.dim() != 1 or t.numel() != cols or not t.is_contiguous():
            _check(t, t.dtype, name, min_numel=cols)
            raise ValueError(f"{name}: must have shape ({cols},), has {tuple(t.shape)}")
        if dtype is not None and dt != dtype:
            raise TypeError("weight and bias: must have one type")
        dtype = dt
    return 0 if dtype is None else dtype


def norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
             eps: float = 1e-5, kind: int = NORM_LAYER, weight_offset: float = 0.0, pack: int = PACK_NONE,
             out: Optional[NormOut] = None) -> NormOut:
    """Layer norm or RMS norm of the rows of x (bf16 [rows, d_model]; see
    dlm_norm_fwd).  pack: also x in 8 bits, which norm_bwd takes in x's place.
    Reuses the buffers of `out` when given; what comes back holds only what
    this call wrote."""
    rows, D = _shape2(x, "x")
    ld = _check_rows(x, torch.bfloat16, "x", rows, D)
    pt = _check_params(weight, bias, D)
    if pack not in (PACK_NONE, PACK_INT8, PACK_E4M3):
        raise ValueError("pack: PACK_NONE, PACK_INT8 or PACK_E4M3")
    layer = kind == NORM_LAYER
    ld_y, pk = D, None
    if out is not None:
        ld_y = _check_rows(out.y, torch.bfloat16, "out.y", rows, D)
        if layer:
            _check(out.mean, torch.float32, "out.mean", min_numel=rows)
        _check(out.rstd, torch.float32, "out.rstd", min_numel=rows)
        if pack != PACK_NONE:
            if out.packed is None or out.packed.format != pack:
                raise ValueError("out.packed: required, in the format asked for")
            pk = out.packed
            _check_packed(pk, rows, D, "out.packed")
        _on_cuda(x=x, weight=weight, bias=bias, y=out.y, mean=out.mean if layer else None, rstd=out.rstd,
                 q=pk.q if pk is not None else None, scale=pk.scale if pk is not None else None)
        out = NormOut(out.y, out.mean if layer else None, out.rstd, pk)
    else:
        if not _all_on(x.get_device(), weight, bias):
            _on_cuda(x=x, weight=weight, bias=bias)
        pk = _empty_packed(rows, D, pack, x.device) if pack != PACK_NONE else None
        out = NormOut(_new(x.device, torch.bfloat16, rows, D), _new(x.device, torch.float32, rows) if layer else None,
                      _new(x.device, torch.float32, rows), pk)
    _call(x.get_device(), "dlm_norm_fwd", x.data_ptr(), rows, D, ld, _ptr(weight), _ptr(bias), pt, kind, eps,
          weight_offset, out.y.data_ptr(), ld_y, out.mean.data_ptr() if layer else None, out.rstd.data_ptr(), pack,
          pk.q.data_ptr() if pk is not None else None, pk.scale.data_ptr() if pk is not None else None)
    return out


@dataclass
class NormGrad:
    d_x: torch.Tensor             # bf16 [rows, d_model]
    d_weight: Optional[torch.Tensor]
    d_bias: Optional[torch.Tensor]
    workspace: torch.Tensor       # uint8


@functools.lru_cache(maxsize=256)      # of the sizes alone
def norm_bwd_workspace_size(rows: int, d_model: int) -> int:
    _in_32_bits(d_model)
    return int(lib().dlm_norm_bwd_workspace_size(rows, d_model))


def norm_bwd(d_y: torch.Tensor, x, rstd: torch.Tensor, mean: Optional[torch.Tensor] = None,
             weight: Optional[torch.Tensor] = None, kind: int = NORM_LAYER, weight_offset: float = 0.0,
             want_d_weight: Optional[bool] = None, want_d_bias: bool = False,
             grad_dtype: Optional[torch.dtype] = None, d_weight: Optional[torch.Tensor] = None,
             d_bias: Optional[torch.Tensor] = None, accumulate: bool = False, d_x: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> NormGrad:
    """Backward pass of norm_fwd (see dlm_norm_bwd).  x: norm_fwd's input, or
    a Packed8 of it (norm_fwd's `packed`).  d_weight (by default when there is
    a weight) and d_bias (with want_d_bias) come in grad_dtype (by default the
    weight's type, else float32) or in the tensors given, which accumulate
    adds to."""
    rows, D = _shape2(d_y, "d_y")
    ld_dy = _check_rows(d_y, torch.bfloat16, "d_y", rows, D)
    pt = _check_params(weight, None, D)
    packed = isinstance(x, Packed8)
    if packed:
        _check_packed(x, rows, D, "x")
        xs, ld_x, fmt, q, qs = None, 0, x.format, x.q, x.scale
    else:
        ld_x = _check_rows(x, torch.bfloat16, "x", rows, D)
        xs, fmt, q, qs = x, PACK_NONE, None, None
    layer = kind == NORM_LAYER
    if layer:
        _check(mean, torch.float32, "mean", min_numel=rows)
    _check(rstd, torch.float32, "rstd", min_numel=rows)
    if want_d_weight is None:
        want_d_weight = weight is not None
    want_w, want_b = want_d_weight or d_weight is not None, want_d_bias or d_bias is not None
    if accumulate and (want_w and d_weight is None or want_b and d_bias is None):
        raise ValueError("accumulate needs d_weight and d_bias for the gradients asked for")
    for t, name in ((d_weight, "d_weight"), (d_bias, "d_bias")) if d_weight is not None or d_bias is not None else ():
        if t is not None:
            _param_dtype(t.dtype, name)
            _check(t, t.dtype, name, min_numel=0)
            if tuple(t.shape) != (D,):
                raise ValueError(f"{name}: must have shape ({D},), has {tuple(t.shape)}")
            if grad_dtype is not None and t.dtype != grad_dtype:
                raise TypeError(f"{name}: expected {grad_dtype}, got {t.dtype}")
            grad_dtype = t.dtype
    if grad_dtype is None:
        grad_dtype = weight.dtype if weight is not None else torch.float32
    gt = _param_dtype(grad_dtype, "grad_dtype")
    ld_dx = D if d_x is None else _check_rows(d_x, torch.bfloat16, "d_x", rows, D)
    if workspace is not None:
        _check(workspace, torch.uint8, "workspace", min_numel=0)
    dev = d_y.get_device()
    if not _all_on(dev, xs, q, qs, mean if layer else None, rstd, weight, d_x, d_weight, d_bias, workspace):
        _on_cuda(d_y=d_y, x=xs, q=q, scale=qs, mean=mean if layer else None, rstd=rstd, weight=weight, d_x=d_x,
                 d_weight=d_weight, d_bias=d_bias, workspace=workspace)
    if d_x is None:
        d_x = _new(d_y.device, torch.bfloat16, rows, D)
    if want_w and d_weight is None:
        d_weight = _new(d_y.device, grad_dtype, D)
    if want_b and d_bias is None:
        d_bias = _new(d_y.device, grad_dtype, D)
    if workspace is None:
        workspace = _aligned_workspace(norm_bwd_workspace_size(rows, D), d_y.device, 256)
    _call(dev, "dlm_norm_bwd", d_y.data_ptr(), ld_dy, _ptr(xs), ld_x, fmt, _ptr(q), _ptr(qs),
          mean.data_ptr() if layer else None, rstd.data_ptr(), _ptr(weight), pt, kind, weight_offset, rows, D,
          d_x.data_ptr(), ld_dx, gt, int(accumulate), _ptr(d_weight), _ptr(d_bias), workspace.data_ptr(),
          workspace.numel())
    return NormGrad(d_x, d_weight, d_bias, workspace)


# --------------------------------------------------------------------------
# autograd wrappers
# --------------------------------------------------------------------------
def scale_bf16_(x: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """x *= scale in place on the device (see dlm_scale_bf16); scale is a
    one-element float32 device tensor.  x: bf16, 1-D or 2-D with unit column
    stride."""
    _check(scale, torch.float32, "scale", min_numel=1)
    _check(x, torch.bfloat16, "x")
    x2 = x.view(1, -1) if x.dim() == 1 else x
    if x2.dim() != 2 or (x2.shape[1] > 1 and x2.stride(1) != 1):
        raise ValueError("x: 1-D contiguous or 2-D with unit column stride")
    _on_cuda(x=x, scale=scale)
    _ok(lib().dlm_scale_bf16(_ptr(x2), x2.shape[0], x2.shape[1], x2.stride(0) if x2.shape[0] > 1 else x2.shape[1],
                             _ptr(scale), _stream()), "dlm_scale_bf16")
    return x


def _upstream(grad: torch.Tensor) -> torch.Tensor:
    return grad.detach().reshape(1).to(torch.float32).contiguous()


class _DiffusionLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, enc_logits, layout, vocab, clean_ids, corrupted, p, mode, align, enc_layout,
                enc_ids, enc_ar_weight, options):
        out = loss_fwd_bwd(layout, logits, vocab, clean_ids, corrupted, p, mode, align, enc_layout=enc_layout,
                           enc_logits=enc_logits, enc_ids=enc_ids, enc_ar_weight=enc_ar_weight, options=options)
        ctx.grads = (out.dlogits, out.enc_dlogits)
        ctx.out = out
        return out.loss.view(())

    @staticmethod
    def backward(ctx, grad):
        g = _upstream(grad)
        d, de = ctx.grads
        ctx.grads = None
        scale_bf16_(d, g)
        if de is not None:
            scale_bf16_(de, g)
        return (d, de) + (None,) * 11


def diffusion_loss(layout: Layout, logits: torch.Tensor, vocab: int, clean_ids: torch.Tensor,
                   corrupted: Optional[torch.Tensor], p: Optional[torch.Tensor], mode: int = ABSORBING,
                   align: int = ALIGNED, enc_layout: Optional[Layout] = None,
                   enc_logits: Optional[torch.Tensor] = None, enc_ids: Optional[torch.Tensor] = None,
                   enc_ar_weight: float = 1.0, options: Optional[LossOptions] = None) -> torch.Tensor:
    """The loss of dlm_loss_fwd_bwd as a differentiable scalar of `logits`
    (and `enc_logits`).  The forward computes the gradient too and keeps it
    (memory of one logits tensor) until backward hands it to autograd.
    Logits are [rows, vocab] here (the gradient has their shape)."""
    for t, name in ((logits, "logits"), (enc_logits, "enc_logits")):
        if t is not None and (t.dim() != 2 or t.shape[1] != vocab):
            raise ValueError(f"{name}: [rows, vocab]")
    return _DiffusionLossFn.apply(logits, enc_logits, layout, vocab, clean_ids, corrupted, p, mode, align,
                                  enc_layout, enc_ids, enc_ar_weight, options)


class _LinearLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, layout, clean_ids, corrupted, p, align):
        out = linear_loss_fwd_bwd(layout, hidden, weight, clean_ids, corrupted, p,
                                  want_d_weight=weight.requires_grad, align=align)
        ctx.grads = (out.d_hidden, out.d_weight)
        ctx.out = out
        return out.loss.view(())

    @staticmethod
    def backward(ctx, grad):
        g = _upstream(grad)
        dh, dw = ctx.grads
        ctx.grads = None
        scale_bf16_(dh, g)
        if dw is not None:
            scale_bf16_(dw, g)
        return (dh, dw) + (None,) * 5


def linear_diffusion_loss(layout: Layout, hidden: torch.Tensor, weight: torch.Tensor, clean_ids: torch.Tensor,
                          corrupted: torch.Tensor, p: torch.Tensor, align: int = ALIGNED) -> torch.Tensor:
    """The loss of dlm_linear_loss_fwd_bwd as a differentiable scalar of
    `hidden` and `weight` (dW is skipped when weight does not require a
    gradient, e.g. a frozen head)."""
    return _LinearLossFn.apply(hidden, weight, layout, clean_ids, corrupted, p, align)


class _LinearUniformLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, enc_hidden, weight, layout, clean_ids, enc_layout, enc_ids, enc_ar_weight, align):
        out = linear_loss_uniform_fwd_bwd(layout, hidden, weight, clean_ids, enc_layout, enc_hidden, enc_ids,
                                          enc_ar_weight=enc_ar_weight, align=align,
                                          want_d_weight=weight.requires_grad)
        ctx.grads = (out.d_hidden, out.d_enc_hidden, out.d_weight)
        ctx.out = out
        return out.loss.view(())

    @staticmethod
    def backward(ctx, grad):
        g = _upstream(grad)
        grads = ctx.grads
        ctx.grads = None
        for t in grads:
            if t is not None:
                scale_bf16_(t, g)
        return grads + (None,) * 6


def linear_uniform_loss(layout: Layout, hidden: torch.Tensor, weight: torch.Tensor, clean_ids: torch.Tensor,
                        enc_layout: Optional[Layout] = None, enc_hidden: Optional[torch.Tensor] = None,
                        enc_ids: Optional[torch.Tensor] = None, enc_ar_weight: float = 1.0,
                        align: int = ALIGNED) -> torch.Tensor:
    """The loss of dlm_linear_loss_uniform_fwd_bwd as a differentiable
    scalar of `hidden`, `enc_hidden` and `weight`."""
    return _LinearUniformLossFn.apply(hidden, enc_hidden, weight, layout, clean_ids, enc_layout, enc_ids,
                                      enc_ar_weight, align)


class _DecisionLossFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, vocab, cand_off, cand_ids, label_kind, label_val, label_softmax, brier_weight,
                hard_label_smoothing):
        out = decision_loss_fwd_bwd(logits, vocab, cand_off, cand_ids, label_kind, label_val,
                                    label_softmax=label_softmax, brier_weight=brier_weight,
                                    hard_label_smoothing=hard_label_smoothing)
        ctx.grads = out.dlogits
        ctx.out = out
        return out.loss.view(())

    @staticmethod
    def backward(ctx, grad):
        d = ctx.grads
        ctx.grads = None
        scale_bf16_(d, _upstream(grad))
        return (d,) + (None,) * 8


def decision_loss(logits: torch.Tensor, vocab: int, cand_off: torch.Tensor, cand_ids: torch.Tensor,
                  label_kind: torch.Tensor, label_val: torch.Tensor, label_softmax: int = LABEL_SOFTMAX_BOTH,
                  brier_weight: float = 0.1, hard_label_smoothing: float = 0.0) -> torch.Tensor:
    """The typed-decision loss of dlm_decision_loss_fwd_bwd as a
    differentiable scalar of `logits` ([n_slots, vocab], one row per label
    slot)."""
    if logits.dim() != 2 or tuple(logits.shape) != (cand_off.numel() - 1, vocab):
        raise ValueError("logits: [n_slots, vocab], one row per label slot")
    return _DecisionLossFn.apply(logits, vocab, cand_off, cand_ids, label_kind, label_val, label_softmax,
                                 brier_weight, hard_label_smoothing)


class _EmbedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, layout, ids, scale, dev_status):
        ctx.save_for_backward(ids, _pad_mask(layout))         # both are read again, as they are now
        ctx.args = (layout, weight.shape[0], scale)
        return embed_fwd(layout, ids, weight, scale, dev_status=dev_status)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        ids, pad = ctx.saved_tensors
        layout, vocab, scale = ctx.args
        if pad is not None and pad.data_ptr() != layout.pad_mask:        # saved-tensor hooks gave another one back
            layout = make_layout(layout.n_units, layout.seq_len, layout._tensors[0], pad, layout.n_tokens)
        return (embed_bwd(layout, ids, _as_rows(grad), vocab, scale).d_weight,) + (None,) * 4


def embed(layout: Layout, ids: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
          dev_status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """embed_fwd as a differentiable function of `weight`; its gradient is
    dense, bf16 [vocab, d_model] (embed_bwd can add it to another one).
    dev_status as there: the one place where an id outside the table shows.
    To capture a whole backward pass in a CUDA graph, drop every earlier eager
    graph of the same parameters first (torch's own rule), or capture embed_bwd
    and norm_bwd, which have no such state."""
    return _EmbedFn.apply(weight, layout, ids, scale, dev_status)


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, kind, weight_offset, keep8):
        out = norm_fwd(x, weight, bias, eps, kind, weight_offset,
                       pack=keep8 if any(ctx.needs_input_grad[:3]) else PACK_NONE)
        p = out.packed
        ctx.args = (kind, weight_offset, keep8, None if bias is None else bias.dtype)
        ctx.save_for_backward(weight, out.mean, out.rstd, *((x, None) if p is None else (p.q, p.scale)))
        return out.y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        weight, mean, rstd, a, scale = ctx.saved_tensors
        kind, weight_offset, keep8, bias_dtype = ctx.args
        g = norm_bwd(_as_rows(grad), a if scale is None else Packed8(a, scale, keep8), rstd, mean, weight, kind,
                     weight_offset, want_d_weight=ctx.needs_input_grad[1], want_d_bias=ctx.needs_input_grad[2],
                     grad_dtype=bias_dtype if weight is None else weight.dtype)
        return (g.d_x, g.d_weight, g.d_bias) + (None,) * 4


def norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
         eps: float = 1e-5, kind: int = NORM_LAYER, weight_offset: float = 0.0,
         keep8: int = PACK_NONE) -> torch.Tensor:
    """norm_fwd as a differentiable function of `x`, `weight` and `bias`.
    keep8 = PACK_INT8 or PACK_E4M3: x is kept for the backward pass in 8 bits,
    written by the forward kernel, in place of x itself; the backward pass then
    takes those values for x (mean and rstd stay those of x)."""
    if keep8 not in (PACK_NONE, PACK_INT8, PACK_E4M3):
        raise ValueError("keep8: PACK_NONE, PACK_INT8 or PACK_E4M3")
    # under no_grad a parameter still says that it needs a gradient, and inside the function gradients are
    # always off: asked for here, so that no form is written that nobody reads
    return _NormFn.apply(x, weight, bias, eps, kind, weight_offset, keep8 if torch.is_grad_enabled() else PACK_NONE)
