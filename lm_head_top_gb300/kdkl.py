"""ctypes binding of libkdkl.so (the C ABI in include/kdkl.h).

Argument marshalling only: every step of the loss runs in the library's CUDA
kernels. PyTorch provides device memory (outputs and the workspace) and the
current stream. There is no CPU fallback: if the library is missing the calls
raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkdkl.so")

KD_OK = 0
STATUS_NAMES = {
    0: "KD_OK", 1: "KD_ERR_INVALID_ARG", 2: "KD_ERR_SHAPE", 3: "KD_ERR_ALIGNMENT",
    4: "KD_ERR_INDEX_RANGE", 5: "KD_ERR_WORKSPACE", 6: "KD_ERR_CUDA", 7: "KD_ERR_TIMEOUT",
    8: "KD_ERR_UNSUPPORTED",
}
KDKL_MAX_K = 512


class KDKLError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__("%s: %s" % (where, STATUS_NAMES.get(code, "status %d" % code)))


class kd_kl_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("V", ctypes.c_int64),
                ("K", ctypes.c_int32), ("temperature", ctypes.c_float), ("chunk", ctypes.c_int64)]


class kd_kl_options(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("scale_tau_sq", ctypes.c_int32),
                ("labels", ctypes.c_void_p)]


class kd_topk_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("V", ctypes.c_int64),
                ("K", ctypes.c_int32), ("reserved", ctypes.c_int32)]


KDKL_TOPK_MAX_K = 512


class kd_logprob_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("V", ctypes.c_int64),
                ("temperature", ctypes.c_float), ("dw_bf16", ctypes.c_int32),
                ("chunk", ctypes.c_int64)]


class kd_policy_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("S", ctypes.c_int64), ("clip_low", ctypes.c_double),
                ("clip_high", ctypes.c_double), ("dual_clip", ctypes.c_double),
                ("kl_coef", ctypes.c_double), ("norm", ctypes.c_double),
                ("reduction", ctypes.c_int32), ("advantage_per_sequence", ctypes.c_int32)]


class kd_pref_problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("P", ctypes.c_int64), ("beta", ctypes.c_double),
                ("label_smoothing", ctypes.c_double), ("margin", ctypes.c_double),
                ("kind", ctypes.c_int32), ("average", ctypes.c_int32), ("halves", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class kd_adamw_tensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n", ctypes.c_int64), ("decay", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class kd_adamw_options(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("grad_scale_dev", ctypes.c_void_p),
                ("grad_scale", ctypes.c_float), ("param_bf16", ctypes.c_int32),
                ("grad_bf16", ctypes.c_int32), ("state_8bit", ctypes.c_int32)]


KD_REDUCTIONS = {"token": 0, "sequence": 1, "sum": 2}
KD_PREF_KINDS = {"sigmoid": 0, "ipo": 1, "hinge": 2}
KD_ADAMW_BLOCK = 256  # elements that share one scale of an 8-bit state


class kd_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 32), ("launches", ctypes.c_int64),
                ("total_ms", ctypes.c_double)]


# name -> (restype, argtypes); every symbol include/kdkl.h declares.
_P = ctypes.c_void_p
_SIGS = {
    "kd_kl_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_kl_problem), ctypes.c_int]),
    "kd_kl_forward": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), _P, _P, _P, _P, _P, _P, _P, _P,
                                     _P, ctypes.c_size_t, _P]),
    "kd_kl_backward": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), _P, _P, _P, _P, _P, _P,
                                      ctypes.c_float, _P, _P, ctypes.c_int, _P, ctypes.c_size_t,
                                      _P]),
    "kd_kl_forward_ex": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), ctypes.POINTER(kd_kl_options),
                                        _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t,
                                        _P]),
    "kd_kl_backward_ex": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem),
                                         ctypes.POINTER(kd_kl_options), _P, _P, _P, _P, _P, _P, _P,
                                         ctypes.c_float, _P, _P, ctypes.c_int, _P, ctypes.c_size_t,
                                         _P]),
    "kd_kl_backward_reuse": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem),
                                            ctypes.POINTER(kd_kl_options), _P, _P, _P, _P, _P, _P,
                                            ctypes.c_size_t, ctypes.c_float, _P, _P, ctypes.c_int,
                                            _P, ctypes.c_size_t, _P]),
    "kd_kl_forward_noalloc": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), _P, _P, _P, _P, _P,
                                             _P, _P, _P, _P]),
    "kd_kl_noalloc_check_status": (ctypes.c_int, [_P]),
    "kd_rkl_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_kl_problem)]),
    "kd_rkl_forward": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), _P, _P, _P, _P, _P, _P, _P,
                                      _P, _P, ctypes.c_size_t, _P]),
    "kd_rkl_backward": (ctypes.c_int, [ctypes.POINTER(kd_kl_problem), _P, _P, _P, _P, _P, _P,
                                       ctypes.c_float, _P, _P, ctypes.c_int, _P, ctypes.c_size_t,
                                       _P]),
    "kd_lmhead_topk_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_topk_problem)]),
    "kd_lmhead_topk": (ctypes.c_int, [ctypes.POINTER(kd_topk_problem), _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "kd_logprob_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_logprob_problem),
                                                    ctypes.c_int]),
    "kd_logprob_forward": (ctypes.c_int, [ctypes.POINTER(kd_logprob_problem), _P, _P, _P, _P, _P,
                                          _P, _P, ctypes.c_size_t, _P]),
    "kd_logprob_backward": (ctypes.c_int, [ctypes.POINTER(kd_logprob_problem), _P, _P, _P, _P, _P,
                                           _P, _P, ctypes.c_int, _P, ctypes.c_size_t, _P]),
    "kd_policy_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_policy_problem)]),
    "kd_policy_loss": (ctypes.c_int, [ctypes.POINTER(kd_policy_problem), _P, _P, _P, _P, _P, _P,
                                      ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "kd_pref_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(kd_pref_problem)]),
    "kd_pref_loss": (ctypes.c_int, [ctypes.POINTER(kd_pref_problem), _P, _P, _P, _P,
                                    ctypes.c_float, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "kd_adamw_step": (ctypes.c_int, [ctypes.POINTER(kd_adamw_tensor), ctypes.c_int32,
                                     ctypes.POINTER(kd_adamw_options), _P]),
    "kd_kl_check_status": (ctypes.c_int, [_P, _P]),
    "kd_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kd_launch_count": (ctypes.c_int64, []),
    "kd_timing_begin": (ctypes.c_int, []),
    "kd_timing_end": (ctypes.c_int, [ctypes.POINTER(kd_kernel_time), ctypes.c_int,
                                     ctypes.POINTER(ctypes.c_int)]),
}

_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise RuntimeError("libkdkl.so not found at %s: build it with "
                               "`python -m lm_head_top_gb300.build`" % path)
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _problem(T, d, V, K, temperature, chunk) -> kd_kl_problem:
    return kd_kl_problem(int(T), int(d), int(V), int(K), float(temperature), int(chunk))


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))


def same_device(dev: torch.device, **tensors) -> None:
    """Every tensor given (None skipped) must live on ``dev``: the library runs
    on the current device with pointers as they are, so a tensor on another
    GPU would be read through the wrong device. Raises before anything runs."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, expected %s (the device of H)" % (name, t.device, dev))


def _out(t, name, dtype, shape, dev):
    """An output tensor passed in: right dtype, shape, contiguity and device."""
    if t is not None:
        _check(t, name, dtype, shape)
        same_device(dev, **{name: t})
    return t


def kd_status_string(code: int) -> str:
    return load().kd_status_string(int(code)).decode()


def kd_launch_count() -> int:
    return int(load().kd_launch_count())


def kd_kl_workspace_size(T, d, V, K, temperature=1.0, chunk=1024, which=0) -> int:
    p = _problem(T, d, V, K, temperature, chunk)
    return int(load().kd_kl_workspace_size(ctypes.byref(p), int(which)))


def _workspace(p: kd_kl_problem, which: int, device, workspace):
    need = int(load().kd_kl_workspace_size(ctypes.byref(p), which))
    if need == 0:
        raise KDKLError(2, "kd_kl_workspace_size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        _check(workspace, "workspace", torch.uint8, (workspace.numel(),))
        same_device(device, workspace=workspace)
    return workspace


def _call(fn_name: str, dev: torch.device, stream, *args):
    """Runs one library call with ``dev`` current (the library works on the
    current device and stream), raising KDKLError on a non-OK status."""
    if stream is not None and stream.device != dev:
        raise ValueError("stream is on %s, expected %s" % (stream.device, dev))
    with torch.cuda.device(dev):
        rc = getattr(load(), fn_name)(*args, _stream_ptr(stream))
    if rc != KD_OK:
        raise KDKLError(rc, fn_name)


def _teacher_args(H, W, topk_idx, topk_logit, mask):
    T, d = H.shape
    V = W.shape[0]
    K = topk_idx.shape[1]
    _check(H, "H", torch.bfloat16, (T, d))
    _check(W, "W", torch.bfloat16, (V, d))
    _check(topk_idx, "topk_idx", torch.int32, (T, K))
    _check(topk_logit, "topk_logit", torch.float32, (T, K))
    if mask is not None:
        _check(mask, "mask", torch.uint8, (T,))
    same_device(H.device, W=W, topk_idx=topk_idx, topk_logit=topk_logit, mask=mask)
    return T, d, V, K, H.device


def kd_kl_forward(H, W, topk_idx, topk_logit, mask=None, *, temperature=1.0, chunk=1024,
                  want_token_kl=False, loss=None, lse=None, token_kl=None, workspace=None,
                  stream=None):
    """Fused forward. Returns (loss [1] fp32, lse [T] fp32, token_kl [T] fp32 or None).
    The work is queued on ``stream`` (default: the current stream of H's device)."""
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    p = _problem(T, d, V, K, temperature, chunk)
    workspace = _workspace(p, 0, dev, workspace)
    loss = _out(loss, "loss", torch.float32, (1,), dev)
    lse = _out(lse, "lse", torch.float32, (T,), dev)
    token_kl = _out(token_kl, "token_kl", torch.float32, (T,), dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(T, dtype=torch.float32, device=dev) if lse is None else lse
    if want_token_kl and token_kl is None:
        token_kl = torch.empty(T, dtype=torch.float32, device=dev)
    _call("kd_kl_forward", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(topk_idx),
          _ptr(topk_logit), _ptr(mask), _ptr(loss), _ptr(lse), _ptr(token_kl), _ptr(workspace),
          workspace.numel())
    return loss, lse, token_kl


def _grad_outputs(dH, dW, T, V, d, accumulate_dW, dev):
    dH = _out(dH, "dH", torch.bfloat16, (T, d), dev)
    dW = _out(dW, "dW", torch.float32, (V, d), dev)
    dH = torch.empty((T, d), dtype=torch.bfloat16, device=dev) if dH is None else dH
    if dW is None:
        if accumulate_dW:
            raise ValueError("accumulate_dW needs an existing dW")
        dW = torch.empty((V, d), dtype=torch.float32, device=dev)
    return dH, dW


def kd_kl_backward(H, W, topk_idx, topk_logit, mask, lse, *, temperature=1.0, chunk=1024,
                   grad_loss=1.0, dH=None, dW=None, accumulate_dW=False, workspace=None,
                   fwd_workspace=None, stream=None):
    """Fused backward of grad_loss * loss. Returns (dH [T,d] bf16, dW [V,d] fp32).

    ``fwd_workspace``: the workspace the forward on these inputs used. The
    backward then reads the teacher rows that forward prepared instead of
    preparing them again (kd_kl_backward_reuse); topk_idx / topk_logit are
    only shape-checked."""
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    _check(lse, "lse", torch.float32, (T,))
    same_device(dev, lse=lse)
    p = _problem(T, d, V, K, temperature, chunk)
    dH, dW = _grad_outputs(dH, dW, T, V, d, accumulate_dW, dev)
    if fwd_workspace is not None:
        _check(fwd_workspace, "fwd_workspace", torch.uint8, (fwd_workspace.numel(),))
        same_device(dev, fwd_workspace=fwd_workspace)
        workspace = _workspace(p, 4, dev, workspace)
        _call("kd_kl_backward_reuse", dev, stream, ctypes.byref(p), None, _ptr(H), _ptr(W),
              _ptr(mask), _ptr(lse), None, _ptr(fwd_workspace), fwd_workspace.numel(),
              float(grad_loss), _ptr(dH), _ptr(dW), 1 if accumulate_dW else 0, _ptr(workspace),
              workspace.numel())
        return dH, dW
    workspace = _workspace(p, 1, dev, workspace)
    _call("kd_kl_backward", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(topk_idx),
          _ptr(topk_logit), _ptr(mask), _ptr(lse), float(grad_loss), _ptr(dH), _ptr(dW),
          1 if accumulate_dW else 0, _ptr(workspace), workspace.numel())
    return dH, dW


def _options(alpha, scale_tau_sq, labels, T, dev):
    if labels is not None:
        _check(labels, "labels", torch.int32, (T,))
        same_device(dev, labels=labels)
    return kd_kl_options(float(alpha), 1 if scale_tau_sq else 0,
                         None if labels is None else labels.data_ptr())


def kd_kl_forward_ex(H, W, topk_idx, topk_logit, mask=None, labels=None, *, temperature=1.0,
                     chunk=1024, alpha=1.0, scale_tau_sq=False, want_token_loss=False,
                     workspace=None, stream=None):
    """Mixed loss alpha*c*KL(tau) + (1-alpha)*CE(labels), c = tau^2 if scale_tau_sq.
    Returns (loss [1], lse [T] at tau, lse1 [T] at temperature 1, token_loss or None)."""
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    p = _problem(T, d, V, K, temperature, chunk)
    o = _options(alpha, scale_tau_sq, labels, T, dev)
    workspace = _workspace(p, 2, dev, workspace)
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    lse1 = torch.empty(T, dtype=torch.float32, device=dev)
    tok = torch.empty(T, dtype=torch.float32, device=dev) if want_token_loss else None
    _call("kd_kl_forward_ex", dev, stream, ctypes.byref(p), ctypes.byref(o), _ptr(H), _ptr(W),
          _ptr(topk_idx), _ptr(topk_logit), _ptr(mask), _ptr(loss), _ptr(lse), _ptr(lse1),
          _ptr(tok), _ptr(workspace), workspace.numel())
    return loss, lse, lse1, tok


def kd_kl_backward_ex(H, W, topk_idx, topk_logit, mask, labels, lse, lse1, *, temperature=1.0,
                      chunk=1024, alpha=1.0, scale_tau_sq=False, grad_loss=1.0, dH=None, dW=None,
                      accumulate_dW=False, workspace=None, fwd_workspace=None, stream=None):
    """Backward of grad_loss * kd_kl_forward_ex's loss. Returns (dH bf16, dW fp32).
    ``fwd_workspace`` as in kd_kl_backward."""
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    _check(lse, "lse", torch.float32, (T,))
    if lse1 is not None:
        _check(lse1, "lse1", torch.float32, (T,))
    same_device(dev, lse=lse, lse1=lse1)
    p = _problem(T, d, V, K, temperature, chunk)
    o = _options(alpha, scale_tau_sq, labels, T, dev)
    dH, dW = _grad_outputs(dH, dW, T, V, d, accumulate_dW, dev)
    if fwd_workspace is not None:
        _check(fwd_workspace, "fwd_workspace", torch.uint8, (fwd_workspace.numel(),))
        same_device(dev, fwd_workspace=fwd_workspace)
        workspace = _workspace(p, 4, dev, workspace)
        _call("kd_kl_backward_reuse", dev, stream, ctypes.byref(p), ctypes.byref(o), _ptr(H),
              _ptr(W), _ptr(mask), _ptr(lse), _ptr(lse1), _ptr(fwd_workspace),
              fwd_workspace.numel(), float(grad_loss), _ptr(dH), _ptr(dW),
              1 if accumulate_dW else 0, _ptr(workspace), workspace.numel())
        return dH, dW
    workspace = _workspace(p, 3, dev, workspace)
    _call("kd_kl_backward_ex", dev, stream, ctypes.byref(p), ctypes.byref(o), _ptr(H), _ptr(W),
          _ptr(topk_idx), _ptr(topk_logit), _ptr(mask), _ptr(lse), _ptr(lse1), float(grad_loss),
          _ptr(dH), _ptr(dW), 1 if accumulate_dW else 0, _ptr(workspace), workspace.numel())
    return dH, dW


def kd_kl_forward_noalloc(H, W, topk_idx, topk_logit, mask=None, *, temperature=1.0,
                          chunk=1024, want_token_kl=False, loss=None, lse=None, token_kl=None,
                          stream=None):
    """Forward for callers that cannot allocate a workspace: the library's own
    fixed scratch array is used instead (see kd_kl_forward_noalloc in kdkl.h).
    Outputs are allocated here only when not passed in."""
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    p = _problem(T, d, V, K, temperature, chunk)
    loss = _out(loss, "loss", torch.float32, (1,), dev)
    lse = _out(lse, "lse", torch.float32, (T,), dev)
    token_kl = _out(token_kl, "token_kl", torch.float32, (T,), dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(T, dtype=torch.float32, device=dev) if lse is None else lse
    if want_token_kl and token_kl is None:
        token_kl = torch.empty(T, dtype=torch.float32, device=dev)
    _call("kd_kl_forward_noalloc", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W),
          _ptr(topk_idx), _ptr(topk_logit), _ptr(mask), _ptr(loss), _ptr(lse), _ptr(token_kl))
    return loss, lse, token_kl


def kd_kl_noalloc_check_status(device=None, stream=None) -> int:
    """BLOCKING. Device-detected status of the latest kd_kl_forward_noalloc
    call on ``device`` (default: the current device)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    with torch.cuda.device(dev):
        return int(load().kd_kl_noalloc_check_status(_stream_ptr(stream)))


def kd_rkl_workspace_size(T, d, V, K, temperature=1.0) -> int:
    p = _problem(T, d, V, K, temperature, 1)
    return int(load().kd_rkl_workspace_size(ctypes.byref(p)))


def _rkl_args(H, W, topk_idx, topk_logit, mask, temperature, workspace):
    T, d, V, K, dev = _teacher_args(H, W, topk_idx, topk_logit, mask)
    p = _problem(T, d, V, K, temperature, 1)
    if workspace is None:
        need = int(load().kd_rkl_workspace_size(ctypes.byref(p)))
        if need == 0:
            raise KDKLError(2, "kd_rkl_workspace_size")
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", torch.uint8, (workspace.numel(),))
        same_device(dev, workspace=workspace)
    return p, workspace


def kd_rkl_forward(H, W, topk_idx, topk_logit, mask=None, *, temperature=1.0,
                   want_token_rkl=False, want_grad_z=False, loss=None, token_rkl=None, grad_z=None,
                   workspace=None, stream=None):
    """Reverse KL over the cached ids. Returns (loss [1] fp32, token_rkl [T] fp32 or None,
    grad_z [T,K] fp32 or None)."""
    p, workspace = _rkl_args(H, W, topk_idx, topk_logit, mask, temperature, workspace)
    dev = H.device
    T = H.shape[0]
    loss = _out(loss, "loss", torch.float32, (1,), dev)
    token_rkl = _out(token_rkl, "token_rkl", torch.float32, (T,), dev)
    grad_z = _out(grad_z, "grad_z", torch.float32, tuple(topk_idx.shape), dev)
    loss = torch.empty(1, dtype=torch.float32, device=dev) if loss is None else loss
    if want_token_rkl and token_rkl is None:
        token_rkl = torch.empty(T, dtype=torch.float32, device=dev)
    if want_grad_z and grad_z is None:
        grad_z = torch.empty(tuple(topk_idx.shape), dtype=torch.float32, device=dev)
    _call("kd_rkl_forward", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(topk_idx),
          _ptr(topk_logit), _ptr(mask), _ptr(loss), _ptr(token_rkl), _ptr(grad_z),
          _ptr(workspace), workspace.numel())
    return loss, token_rkl, grad_z


def kd_rkl_backward(H, W, topk_idx, topk_logit, mask=None, *, temperature=1.0, grad_z=None,
                    grad_loss=1.0, dH=None, dW=None, accumulate_dW=False, workspace=None,
                    stream=None):
    """Backward of grad_loss * reverse-KL loss. Returns (dH [T,d] bf16, dW [V,d] fp32).
    grad_z from kd_rkl_forward (same inputs) skips the logit recompute."""
    p, workspace = _rkl_args(H, W, topk_idx, topk_logit, mask, temperature, workspace)
    dev = H.device
    grad_z = _out(grad_z, "grad_z", torch.float32, tuple(topk_idx.shape), dev)
    T, d = H.shape
    dH, dW = _grad_outputs(dH, dW, T, W.shape[0], d, accumulate_dW, dev)
    _call("kd_rkl_backward", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(topk_idx),
          _ptr(topk_logit), _ptr(mask), _ptr(grad_z), float(grad_loss), _ptr(dH), _ptr(dW),
          1 if accumulate_dW else 0, _ptr(workspace), workspace.numel())
    return dH, dW


def kd_lmhead_topk_workspace_size(T, d, V, K) -> int:
    p = kd_topk_problem(int(T), int(d), int(V), int(K), 0)
    return int(load().kd_lmhead_topk_workspace_size(ctypes.byref(p)))


def kd_lmhead_topk(H, W, K, *, topk_idx=None, topk_logit=None, workspace=None, stream=None):
    """Offline teacher cache: the K largest logits of each row of H . W^T and
    their ids, per row by logit descending (ties: smaller id first).
    Returns (topk_idx [T,K] int32, topk_logit [T,K] fp32)."""
    T, d = H.shape
    V = W.shape[0]
    _check(H, "H", torch.bfloat16, (T, d))
    _check(W, "W", torch.bfloat16, (V, d))
    dev = H.device
    same_device(dev, W=W)
    p = kd_topk_problem(int(T), int(d), int(V), int(K), 0)
    need = int(load().kd_lmhead_topk_workspace_size(ctypes.byref(p)))
    if need == 0:
        raise KDKLError(2, "kd_lmhead_topk_workspace_size")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", torch.uint8, (workspace.numel(),))
        same_device(dev, workspace=workspace)
    topk_idx = _out(topk_idx, "topk_idx", torch.int32, (T, K), dev)
    topk_logit = _out(topk_logit, "topk_logit", torch.float32, (T, K), dev)
    if topk_idx is None:
        topk_idx = torch.empty((T, K), dtype=torch.int32, device=dev)
    if topk_logit is None:
        topk_logit = torch.empty((T, K), dtype=torch.float32, device=dev)
    _call("kd_lmhead_topk", dev, stream, ctypes.byref(p), _ptr(H), _ptr(W), _ptr(topk_idx),
          _ptr(topk_logit), _ptr(workspace), workspace.numel())
    return topk_idx, topk_logit


def _addr(t, name, dtype, shape, dev):
    """Address of an optional tensor argument after the checks of _check and
    same_device, in one expression when all is well: the calls below are short
    enough on the GPU for the host's part to count."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda
            and t.device == dev and t.is_contiguous()):
        _check(t, name, dtype, shape)
        same_device(dev, **{name: t})
    return t.data_ptr()


def _launch(fn_name, dev, stream, *args):
    """_call for addresses that are plain integers, without its context manager
    when ``dev`` is the current device already."""
    lib = _lib or load()
    if stream is not None and stream.device != dev:
        raise ValueError("stream is on %s, expected %s" % (stream.device, dev))
    raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        rc = getattr(lib, fn_name)(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = getattr(lib, fn_name)(*args, raw)
    if rc != KD_OK:
        raise KDKLError(rc, fn_name)


def _new(shape, dtype, dev, stream):
    """An output or workspace made here for a call on ``stream``: allocated as
    that stream's own memory, so that it is not handed to another stream's
    tensors while the call still runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _given_workspace(workspace, need, where, dev, stream):
    if need == 0:
        raise KDKLError(2, where)
    if workspace is None:
        return _new(need, torch.uint8, dev, stream)
    _addr(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    return workspace


def _outcome(t, name, dtype, shape, dev, stream):
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, dev, stream)
    _addr(t, name, dtype, shape, dev)
    return t


def kd_logprob_workspace_size(T, d, V, temperature=1.0, chunk=4096, which=0,
                              dW_dtype=torch.float32) -> int:
    p = kd_logprob_problem(int(T), int(d), int(V), float(temperature),
                           1 if dW_dtype == torch.bfloat16 else 0, int(chunk))
    return int(load().kd_logprob_workspace_size(ctypes.byref(p), int(which)))


def _logprob_args(H, W, ids):
    T, d = H.shape
    V = W.shape[0]
    dev = H.device
    return T, d, V, dev, (_addr(H, "H", torch.bfloat16, (T, d), dev),
                          _addr(W, "W", torch.bfloat16, (V, d), dev),
                          _addr(ids, "ids", torch.int32, (T,), dev))


def kd_logprob_forward(H, W, ids, mask=None, *, temperature=1.0, logp=None, lse=None,
                       workspace=None, stream=None):
    """Log-probability of ids[t] under softmax(H[t] . W^T / temperature), the logits
    never stored. Returns (logp [T] fp32, lse [T] fp32); masked tokens read 0."""
    T, d, V, dev, operands = _logprob_args(H, W, ids)
    counted = _addr(mask, "mask", torch.uint8, (T,), dev)
    p = kd_logprob_problem(T, d, V, float(temperature), 0, 1)
    workspace = _given_workspace(workspace, load().kd_logprob_workspace_size(ctypes.byref(p), 0),
                                 "kd_logprob_workspace_size", dev, stream)
    logp = _outcome(logp, "logp", torch.float32, (T,), dev, stream)
    lse = _outcome(lse, "lse", torch.float32, (T,), dev, stream)
    _launch("kd_logprob_forward", dev, stream, ctypes.byref(p), *operands, counted,
            logp.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel())
    return logp, lse


def kd_logprob_backward(H, W, ids, lse, grad_logp, *, temperature=1.0, chunk=4096, dH=None,
                        dW=None, dW_dtype=torch.float32, accumulate_dW=False, workspace=None,
                        stream=None):
    """Gradients of sum_t grad_logp[t] * logp[t]. Returns (dH [T,d] bf16, dW [V,d] in
    ``dW_dtype``: fp32, which may be added to, or bf16). Tokens whose gradient is
    zero are skipped. ``chunk`` bounds the workspace: chunk * V bf16 values of the
    gradient of the logits at a time, 1.6 GB at the default and V = 201,088. At 1024 it is
    a quarter of that and the call 3 % slower (6.77 and 6.59 ms for 3000 tokens)."""
    T, d, V, dev, operands = _logprob_args(H, W, ids)
    given = (_addr(lse, "lse", torch.float32, (T,), dev),
             _addr(grad_logp, "grad_logp", torch.float32, (T,), dev))
    if dW is not None:
        dW_dtype = dW.dtype
    if dW_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dW must be torch.float32 or torch.bfloat16, got %s" % dW_dtype)
    if accumulate_dW and dW is None:
        raise ValueError("accumulate_dW needs an existing dW")
    if accumulate_dW and dW_dtype == torch.bfloat16:
        raise ValueError("a bf16 dW is not accumulated: pass an fp32 one")
    p = kd_logprob_problem(T, d, V, float(temperature), 1 if dW_dtype == torch.bfloat16 else 0,
                           int(chunk))
    workspace = _given_workspace(workspace, load().kd_logprob_workspace_size(ctypes.byref(p), 1),
                                 "kd_logprob_workspace_size", dev, stream)
    dH = _outcome(dH, "dH", torch.bfloat16, (T, d), dev, stream)
    dW = _outcome(dW, "dW", dW_dtype, (V, d), dev, stream)
    _launch("kd_logprob_backward", dev, stream, ctypes.byref(p), *operands, *given, dH.data_ptr(),
            dW.data_ptr(), 1 if accumulate_dW else 0, workspace.data_ptr(), workspace.numel())
    return dH, dW


def kd_policy_loss(logp, old_logp, ref_logp, advantages, mask=None, cu_seqlens=None, *,
                   advantage_per_sequence=None, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
                   kl_coef=0.0, reduction="token", norm=1.0, grad_loss=1.0, want_grad=True,
                   loss=None, stats=None, grad_logp=None, workspace=None, stream=None):
    """Clipped policy loss with a KL term over packed sequences, and its gradient.

    logp, old_logp (None: ratio 1), ref_logp (None: no KL term, ``kl_coef`` 0): [T] fp32.
    advantages: [T], or one per sequence of ``cu_seqlens`` ([S+1] int32): told by
    their number, or by ``advantage_per_sequence``, which has to be given where there
    are as many sequences as tokens.
    reduction: "token" (mean over counted tokens), "sequence" (mean over the
    sequences of each one's mean) or "sum" (sum / ``norm``).
    Returns (loss [1], stats [3] = policy part, KL part, share of clipped tokens,
    grad_logp [T] = grad_loss * dloss/dlogp or None)."""
    T = logp.numel()
    dev = logp.device
    f32, flat = torch.float32, (T,)
    S = 0 if cu_seqlens is None else max(0, cu_seqlens.numel() - 1)
    if ref_logp is None and kl_coef != 0:
        raise ValueError("a KL term (kl_coef %r) needs ref_logp" % kl_coef)
    per_sequence = advantage_per_sequence
    if per_sequence is None:
        if S == T and S > 1 and cu_seqlens is not None:
            raise ValueError("%d sequences and as many tokens: advantage_per_sequence says which "
                             "of the two the advantages are for" % S)
        per_sequence = cu_seqlens is not None and advantages.numel() == S and S != T
    elif per_sequence and cu_seqlens is None:
        raise ValueError("advantages per sequence need cu_seqlens")
    if advantages.numel() != (S if per_sequence else T):
        raise ValueError("advantages has %d values, expected %d, one per %s"
                         % ((advantages.numel(),) + ((S, "sequence") if per_sequence
                                                     else (T, "token"))))
    given = (_addr(logp, "logp", f32, flat, dev), _addr(old_logp, "old_logp", f32, flat, dev),
             _addr(ref_logp, "ref_logp", f32, flat, dev),
             _addr(advantages, "advantages", f32, (S if per_sequence else T,), dev),
             _addr(mask, "mask", torch.uint8, flat, dev),
             _addr(cu_seqlens, "cu_seqlens", torch.int32, (S + 1,), dev))
    if reduction not in KD_REDUCTIONS:
        raise ValueError("reduction must be one of %s, got %r" % (sorted(KD_REDUCTIONS), reduction))
    p = kd_policy_problem(T, S, clip_low, clip_high, dual_clip, kl_coef, norm,
                          KD_REDUCTIONS[reduction], 1 if per_sequence else 0)
    need = load().kd_policy_workspace_size(ctypes.byref(p))
    workspace = _given_workspace(workspace, need or 256, "", dev, stream)  # 0: the call says why
    loss = _outcome(loss, "loss", f32, (1,), dev, stream)
    stats = _outcome(stats, "stats", f32, (3,), dev, stream)
    if want_grad or grad_logp is not None:
        grad_logp = _outcome(grad_logp, "grad_logp", f32, flat, dev, stream)
    _launch("kd_policy_loss", dev, stream, ctypes.byref(p), *given, grad_loss, loss.data_ptr(),
            stats.data_ptr(), None if grad_logp is None else grad_logp.data_ptr(),
            workspace.data_ptr(), workspace.numel())
    return loss, stats, grad_logp


def kd_pref_loss(logp, ref_logp, cu_seqlens, mask=None, *, beta=0.1, kind="sigmoid",
                 label_smoothing=0.0, margin=0.0, average=False, halves=False, grad_loss=1.0,
                 want_grad=True, loss=None, rewards=None, grad_logp=None, workspace=None,
                 stream=None):
    """Preference loss over pairs (chosen, rejected) of packed sequences, and its gradient.

    logp, ref_logp (None: no reference): [T] fp32; cu_seqlens: [2P+1] int32, sequences
    2i and 2i+1 forming pair i, or with ``halves`` i and P + i. ``average``: a
    sequence counts with the mean of its tokens' log ratios instead of their sum.
    Returns (loss [1], rewards [P,2], grad_logp [T] = grad_loss * dloss/dlogp or None)."""
    T = logp.numel()
    dev = logp.device
    f32, flat = torch.float32, (T,)
    n = cu_seqlens.numel()
    given = (_addr(logp, "logp", f32, flat, dev), _addr(ref_logp, "ref_logp", f32, flat, dev),
             _addr(mask, "mask", torch.uint8, flat, dev),
             _addr(cu_seqlens, "cu_seqlens", torch.int32, (n,), dev))
    if n % 2 != 1:
        raise ValueError("cu_seqlens holds 2 P + 1 offsets, got %d" % n)
    P = n // 2
    if kind not in KD_PREF_KINDS:
        raise ValueError("kind must be one of %s, got %r" % (sorted(KD_PREF_KINDS), kind))
    p = kd_pref_problem(T, P, beta, label_smoothing, margin, KD_PREF_KINDS[kind],
                        1 if average else 0, 1 if halves else 0, 0)
    need = load().kd_pref_workspace_size(ctypes.byref(p))
    workspace = _given_workspace(workspace, need or 256, "", dev, stream)  # 0: the call says why
    loss = _outcome(loss, "loss", f32, (1,), dev, stream)
    rewards = _outcome(rewards, "rewards", f32, (P, 2), dev, stream)
    if want_grad or grad_logp is not None:
        grad_logp = _outcome(grad_logp, "grad_logp", f32, flat, dev, stream)
    _launch("kd_pref_loss", dev, stream, ctypes.byref(p), *given, grad_loss, loss.data_ptr(),
            rewards.data_ptr(), None if grad_logp is None else grad_logp.data_ptr(),
            workspace.data_ptr(), workspace.numel())
    return loss, rewards, grad_logp


class KDAdamWTensors:
    """The tensors of an AdamW step, checked once: the host table that kd_adamw_step
    passes to the library, and the memory it points to (kept alive, not copied, also when
    a list or a tensor's data is exchanged). A step works on that memory: it does not
    notice that a gradient has been replaced since, and takes the old one."""

    def __init__(self, table, n, device, memory, param_bf16, grad_bf16, state_8bit):
        self.table, self.n, self.device, self.memory = table, n, device, memory
        self.param_bf16, self.grad_bf16, self.state_8bit = param_bf16, grad_bf16, state_8bit


def kd_adamw_tensors(params, grads, exp_avg, exp_avg_sq, *, copies=None, m_scales=None,
                     v_scales=None, decay=None) -> KDAdamWTensors:
    """The list of tensors for kd_adamw_step; make it again when a tensor is replaced (a
    step cannot notice: gradients are new tensors after ``zero_grad(set_to_none=True)``).

    params: fp32 or bf16; grads: fp32 or bf16. exp_avg / exp_avg_sq: fp32 (m and v), or
    torch.float8_e4m3fn (m and sqrt(v)) with ``m_scales`` / ``v_scales``: fp32, one for
    every 256 elements of a tensor (start from zeros, and ones for the scales).
    copies: bf16 tensors that receive the new parameters. decay: per tensor, whether
    weight decay applies (default: to all)."""
    n = len(params)
    lists = {"params": params, "grads": grads, "exp_avg": exp_avg, "exp_avg_sq": exp_avg_sq,
             "copies": copies, "m_scales": m_scales, "v_scales": v_scales}
    for name, ts in lists.items():
        if ts is not None and len(ts) != n:
            raise ValueError("%s has %d tensors, expected %d" % (name, len(ts), n))
    if decay is not None and len(decay) != n:
        raise ValueError("decay has %d values, expected %d" % (len(decay), n))
    if n == 0:
        return KDAdamWTensors((kd_adamw_tensor * 1)(), 0, None, [], 0, 0, 0)
    dev = params[0].device
    p_t, g_t, s_t = params[0].dtype, grads[0].dtype, exp_avg[0].dtype
    if p_t not in (torch.float32, torch.bfloat16):
        raise TypeError("params must be torch.float32 or torch.bfloat16, got %s" % p_t)
    if g_t not in (torch.float32, torch.bfloat16):
        raise TypeError("grads must be torch.float32 or torch.bfloat16, got %s" % g_t)
    if s_t not in (torch.float32, torch.float8_e4m3fn):
        raise TypeError("states must be torch.float32 or torch.float8_e4m3fn, got %s" % s_t)
    s8 = s_t == torch.float8_e4m3fn
    if s8 and (m_scales is None or v_scales is None):
        raise ValueError("8-bit states need m_scales and v_scales")
    table, memory = (kd_adamw_tensor * n)(), []
    columns = [c for c in (("param", "params", params, p_t), ("grad", "grads", grads, g_t),
                           ("exp_avg", "exp_avg", exp_avg, s_t),
                           ("exp_avg_sq", "exp_avg_sq", exp_avg_sq, s_t),
                           ("copy", "copies", copies, torch.bfloat16),
                           ("m_scale", "m_scales", m_scales if s8 else None, torch.float32),
                           ("v_scale", "v_scales", v_scales if s8 else None, torch.float32))
               if c[2] is not None]
    for i in range(n):
        shape, count = params[i].shape, params[i].numel()
        blocks = (count + KD_ADAMW_BLOCK - 1) // KD_ADAMW_BLOCK
        row = table[i]
        for field, name, ts, dtype in columns:
            t = ts[i]
            want = shape if field[1:] != "_scale" else (blocks,)
            if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == want
                    and t.device == dev and t.is_cuda and t.is_contiguous()):
                _check(t, "%s[%d]" % (name, i), dtype, want)
                raise ValueError("%s of tensor %d is on %s, expected %s" % (field, i, t.device, dev))
            setattr(row, field, t.data_ptr())
            memory.append(t.untyped_storage())
        row.n = count
        row.decay = 1 if decay is None or decay[i] else 0
    return KDAdamWTensors(table, n, dev, memory, 1 if p_t == torch.bfloat16 else 0,
                          1 if g_t == torch.bfloat16 else 0, 1 if s8 else 0)


def kd_adamw_step(tensors: KDAdamWTensors, *, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0,
                  step=1, grad_scale=1.0, grad_scale_dev=None, stream=None) -> None:
    """One AdamW step, in place, on the tensors of kd_adamw_tensors. ``step`` counts from 1.
    The gradients are multiplied by ``grad_scale`` and, if given, by the device scalar
    ``grad_scale_dev`` ([1] fp32, a clip coefficient)."""
    if not tensors.n:
        return
    o = kd_adamw_options(lr, betas[0], betas[1], eps, weight_decay, int(step),
                         _addr(grad_scale_dev, "grad_scale_dev", torch.float32, (1,),
                               tensors.device),
                         grad_scale, tensors.param_bf16, tensors.grad_bf16, tensors.state_8bit)
    _launch("kd_adamw_step", tensors.device, stream, tensors.table, tensors.n, ctypes.byref(o))


def kd_kl_check_status(workspace: torch.Tensor, stream=None) -> int:
    """BLOCKING. Device-detected status of the latest call that used ``workspace``."""
    with torch.cuda.device(workspace.device):
        return int(load().kd_kl_check_status(_ptr(workspace), _stream_ptr(stream)))


def kd_timing_begin() -> None:
    load().kd_timing_begin()


def kd_timing_end(max_entries: int = 32):
    """BLOCKING. Returns [(kernel name, launches, total ms)] since kd_timing_begin()."""
    arr = (kd_kernel_time * max_entries)()
    n = ctypes.c_int(0)
    rc = load().kd_timing_end(arr, max_entries, ctypes.byref(n))
    if rc != KD_OK:
        raise KDKLError(rc, "kd_timing_end")
    return [(arr[i].name.decode(), int(arr[i].launches), float(arr[i].total_ms))
            for i in range(min(n.value, max_entries))]
