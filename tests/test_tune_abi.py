"""Refusals of the tuning calls: argument errors come back synchronously, before
any device call, and the binding's own checks raise."""
import ctypes

import pytest
import torch

from lm_head_top_gb300 import kdkl

INVALID, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5
P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(kdkl.LIB_PATH):
        from lm_head_top_gb300 import build
        build.build()
    return kdkl.load()


def test_struct_layouts():
    assert ctypes.sizeof(kdkl.kd_logprob_problem) == 40
    assert ctypes.sizeof(kdkl.kd_policy_problem) == 64
    assert ctypes.sizeof(kdkl.kd_pref_problem) == 56
    assert ctypes.sizeof(kdkl.kd_adamw_tensor) == 72
    assert ctypes.sizeof(kdkl.kd_adamw_options) == 72


# ------------------------------------------------------------ log-probabilities

def _lp(lib, p, H=16, W=16, ids=16, out=64, ws=256, ws_bytes=BIG):
    return lib.kd_logprob_forward(ctypes.byref(p), P(H), P(W), P(ids), None, P(out), P(64), P(ws),
                                  ws_bytes, None)


def _lpb(lib, p, dH=4096, dW=8192, acc=0, grad=64, ws_bytes=BIG):
    return lib.kd_logprob_backward(ctypes.byref(p), P(16), P(16), P(16), P(64), P(grad), P(dH),
                                   P(dW), acc, P(256), ws_bytes, None)


@pytest.mark.parametrize("field,value,code", [
    ("d", 12, ALIGN), ("d", 0, SHAPE), ("V", 0, SHAPE), ("T", -1, SHAPE), ("T", 1 << 31, SHAPE),
    ("temperature", 0.0, INVALID), ("temperature", float("nan"), INVALID), ("chunk", 0, INVALID),
])
def test_logprob_problem_errors(lib, field, value, code):
    p = kdkl.kd_logprob_problem(10, 16, 100, 1.0, 0, 8)
    setattr(p, field, value)
    assert _lp(lib, p) == code and _lpb(lib, p) == code
    for which in (0, 1):
        assert lib.kd_logprob_workspace_size(ctypes.byref(p), which) == 0


def test_logprob_pointer_errors(lib):
    p = kdkl.kd_logprob_problem(10, 16, 100, 1.0, 0, 8)
    assert _lp(lib, p, ws=0) == WORKSPACE
    assert _lp(lib, p, H=0) == INVALID and _lp(lib, p, ids=0) == INVALID
    assert _lp(lib, p, out=0) == INVALID
    assert _lp(lib, p, H=8) == ALIGN and _lp(lib, p, ids=2) == ALIGN
    assert _lpb(lib, p, dW=0) == INVALID and _lpb(lib, p, grad=0) == INVALID
    assert _lpb(lib, p, dH=24) == ALIGN
    p.dw_bf16 = 1
    assert _lpb(lib, p, acc=1) == INVALID  # a bf16 dW is not accumulated
    assert lib.kd_logprob_workspace_size(ctypes.byref(p), 2) == 0


def test_logprob_workspace_is_linear_in_tokens(lib):
    for which in (0, 1):
        s = [kdkl.kd_logprob_workspace_size(T, 2880, 201088, 1.0, 1024, which)
             for T in (8192, 16384, 32768)]
        assert 0 < s[0] < s[1] < s[2] < 0.5 * 2 * 32768 * 201088


# ------------------------------------------------------------------ policy loss

def _policy(**kw):
    f = dict(T=10, S=0, clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, norm=1.0,
             reduction=0, advantage_per_sequence=0)
    f.update(kw)
    return kdkl.kd_policy_problem(*[f[n] for n, _ in kdkl.kd_policy_problem._fields_])


def _pl(lib, p, logp=64, ref=0, adv=64, cu=0, loss=64, ws=256, ws_bytes=BIG, g=1.0):
    return lib.kd_policy_loss(ctypes.byref(p), P(logp), None, P(ref), P(adv), None, P(cu), g,
                              P(loss), None, None, P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 31) - 4096), SHAPE), (dict(S=-1), SHAPE),
    (dict(clip_low=-0.1), INVALID), (dict(clip_low=1.5), INVALID),
    (dict(clip_high=-0.1), INVALID), (dict(clip_high=float("nan")), INVALID),
    (dict(dual_clip=0.5), INVALID), (dict(dual_clip=float("inf")), INVALID),
    (dict(kl_coef=float("inf")), INVALID), (dict(reduction=3), INVALID),
    (dict(reduction=2, norm=0.0), INVALID), (dict(reduction=1), SHAPE),
    (dict(advantage_per_sequence=1), SHAPE),
])
def test_policy_problem_errors(lib, kw, code):
    p = _policy(**kw)
    assert _pl(lib, p) == code
    assert lib.kd_policy_workspace_size(ctypes.byref(p)) == 0


def test_policy_pointer_errors(lib):
    p = _policy()
    need = lib.kd_policy_workspace_size(ctypes.byref(p))
    assert need > 0
    assert _pl(lib, p, ws=0) == WORKSPACE and _pl(lib, p, ws_bytes=need - 1) == WORKSPACE
    assert _pl(lib, p, logp=0) == INVALID and _pl(lib, p, adv=0) == INVALID
    assert _pl(lib, p, loss=0) == INVALID and _pl(lib, p, g=float("nan")) == INVALID
    assert _pl(lib, p, logp=66) == ALIGN and _pl(lib, p, ws=264) == ALIGN
    assert _pl(lib, _policy(kl_coef=0.1)) == INVALID          # a KL term without a reference
    assert _pl(lib, _policy(reduction=1, S=2)) == INVALID     # no cu_seqlens


# -------------------------------------------------------------- preference loss

def _pref(**kw):
    f = dict(T=10, P=1, beta=0.1, label_smoothing=0.0, margin=0.0, kind=0, average=0, halves=0,
             reserved=0)
    f.update(kw)
    return kdkl.kd_pref_problem(*[f[n] for n, _ in kdkl.kd_pref_problem._fields_])


def _pr(lib, p, logp=64, cu=64, loss=64, rewards=64, ws=256, ws_bytes=BIG, g=1.0):
    return lib.kd_pref_loss(ctypes.byref(p), P(logp), None, None, P(cu), g, P(loss), P(rewards),
                            None, P(ws), ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(T=(1 << 31) - 4096), SHAPE), (dict(P=0), SHAPE), (dict(P=-1), SHAPE),
    (dict(beta=0.0), INVALID), (dict(beta=float("inf")), INVALID),
    (dict(label_smoothing=1.0), INVALID), (dict(label_smoothing=-0.1), INVALID),
    (dict(margin=float("nan")), INVALID), (dict(kind=3), INVALID),
])
def test_pref_problem_errors(lib, kw, code):
    p = _pref(**kw)
    assert _pr(lib, p) == code
    assert lib.kd_pref_workspace_size(ctypes.byref(p)) == 0


def test_pref_pointer_errors(lib):
    p = _pref()
    need = lib.kd_pref_workspace_size(ctypes.byref(p))
    assert _pr(lib, p, ws=0) == WORKSPACE and _pr(lib, p, ws_bytes=need - 1) == WORKSPACE
    assert _pr(lib, p, logp=0) == INVALID and _pr(lib, p, cu=0) == INVALID
    assert _pr(lib, p, rewards=0) == INVALID and _pr(lib, p, g=float("inf")) == INVALID
    assert _pr(lib, p, cu=66) == ALIGN


# ------------------------------------------------------------------------ AdamW

def _adam(lib, t=None, n=1, **kw):
    f = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, grad_scale_dev=None,
             grad_scale=1.0, param_bf16=0, grad_bf16=0, state_8bit=0)
    f.update(kw)
    o = kdkl.kd_adamw_options(*[f[k] for k, _ in kdkl.kd_adamw_options._fields_])
    t = t if t is not None else kdkl.kd_adamw_tensor(64, 64, 64, 64, 0, 0, 0, 5, 1, 0)
    return lib.kd_adamw_step(ctypes.byref(t), n, ctypes.byref(o), None)


@pytest.mark.parametrize("kw", [
    dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(eps=-1.0),
    dict(eps=float("inf")), dict(weight_decay=float("inf")), dict(step=0), dict(n=-1),
    dict(grad_scale=float("nan")),
])
def test_adamw_option_errors(lib, kw):
    assert _adam(lib, **kw) == INVALID


def test_adamw_tensor_errors(lib):
    T = kdkl.kd_adamw_tensor
    assert _adam(lib, T(64, 64, 64, 64, 0, 0, 0, -1, 1, 0)) == SHAPE
    assert _adam(lib, T(0, 64, 64, 64, 0, 0, 0, 5, 1, 0)) == INVALID
    assert _adam(lib, T(64, 0, 64, 64, 0, 0, 0, 5, 1, 0)) == INVALID
    assert _adam(lib, T(66, 64, 64, 64, 0, 0, 0, 5, 1, 0)) == ALIGN
    assert _adam(lib, T(66, 66, 64, 64, 0, 0, 0, 5, 1, 0), param_bf16=1) == ALIGN  # fp32 gradients
    assert _adam(lib, T(64, 64, 64, 64, 0, 0, 0, 5, 1, 0), state_8bit=1) == INVALID  # no scales
    assert lib.kd_adamw_step(None, 0, None, None) == INVALID
    assert lib.kd_adamw_step(None, 1, ctypes.byref(kdkl.kd_adamw_options(
        1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, 1.0, 0, 0, 0)), None) == INVALID


# ----------------------------------------------------- the binding's own checks

def test_binding_refuses_host_tensors_and_wrong_types():
    T = 8
    f, i = torch.zeros(T), torch.zeros(T, dtype=torch.int32)
    H, W = torch.zeros(T, 16, dtype=torch.bfloat16), torch.zeros(9, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kdkl.kd_logprob_forward(H, W, i)                 # not on a GPU
    with pytest.raises(TypeError):
        kdkl.kd_logprob_forward(H.float(), W, i)
    with pytest.raises(ValueError):
        kdkl.kd_policy_loss(f, None, None, f)
    with pytest.raises(TypeError):
        kdkl.kd_policy_loss(f.double(), None, None, f)
    with pytest.raises(ValueError):
        kdkl.kd_pref_loss(f, None, i[:3])


def test_binding_refuses_uneven_adamw_lists():
    a = [torch.zeros(4), torch.zeros(4)]
    with pytest.raises(ValueError):
        kdkl.kd_adamw_tensors(a, a[:1], a, a)
    with pytest.raises(ValueError):
        kdkl.kd_adamw_tensors(a, a, a, a, decay=[True])
    with pytest.raises(TypeError):
        kdkl.kd_adamw_tensors([t.half() for t in a], a, a, a)
    s8 = [t.to(torch.float8_e4m3fn) for t in a]
    with pytest.raises(ValueError):
        kdkl.kd_adamw_tensors(a, a, s8, s8)              # no scales
    assert kdkl.kd_adamw_tensors([], [], [], []).n == 0
