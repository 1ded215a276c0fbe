"""Limits of the losses' arguments, refused synchronously before any device call: numbers
of sequences past what the kernels' 31-bit searches hold, and options that are finite in
64 bits but not in the 32 that the kernels compute with (an infinite weight would turn the
zero of a token that is not counted into a NaN)."""
import ctypes

import pytest

from lm_head_top_gb300 import kdkl
from tests.test_tune_abi import INVALID, SHAPE, WORKSPACE, _pl, _policy, _pr, _pref, lib  # noqa: F401


@pytest.mark.parametrize("S", [(1 << 30) + 1, (1 << 31) - 2])
def test_sequences_past_the_search(lib, S):  # noqa: F811
    p = _policy(S=S, reduction=1)
    assert lib.kd_policy_workspace_size(ctypes.byref(p)) == 0 and _pl(lib, p, cu=64) == SHAPE
    q = _pref(P=(S + 1) // 2)
    assert lib.kd_pref_workspace_size(ctypes.byref(q)) == 0 and _pr(lib, q) == SHAPE


def test_the_most_sequences(lib):  # noqa: F811
    assert lib.kd_policy_workspace_size(ctypes.byref(_policy(S=1 << 30, reduction=1))) > 4 << 30
    assert lib.kd_pref_workspace_size(ctypes.byref(_pref(P=1 << 29))) > 4 << 30


@pytest.mark.parametrize("kw", [dict(kl_coef=1e39), dict(kl_coef=-1e39),
                                dict(reduction=2, norm=1e-40)])
def test_policy_options_fit_32_bits(lib, kw):  # noqa: F811
    p = _policy(**kw)
    assert lib.kd_policy_workspace_size(ctypes.byref(p)) == 0
    assert _pl(lib, p, ref=64) == INVALID


def test_the_gradients_weight_fits_32_bits(lib):  # noqa: F811
    p = _policy(reduction=2, norm=1e-37)
    need = lib.kd_policy_workspace_size(ctypes.byref(p))
    assert _pl(lib, p, g=1e3) == INVALID
    assert _pl(lib, p, g=1.0, ws_bytes=need - 1) == WORKSPACE  # taken, up to the next check


@pytest.mark.parametrize("kw", [dict(beta=1e39), dict(beta=1e-46), dict(margin=-1e39),
                                dict(kind=1, beta=1e-39)])
def test_pref_options_fit_32_bits(lib, kw):  # noqa: F811
    p = _pref(**kw)
    assert lib.kd_pref_workspace_size(ctypes.byref(p)) == 0 and _pr(lib, p) == INVALID


def test_large_options_that_fit(lib):  # noqa: F811
    assert lib.kd_policy_workspace_size(ctypes.byref(_policy(kl_coef=1e38))) > 0
    assert lib.kd_policy_workspace_size(ctypes.byref(_policy(reduction=2, norm=1e-37))) > 0
    assert lib.kd_pref_workspace_size(ctypes.byref(_pref(beta=1e-37, kind=1))) > 0
