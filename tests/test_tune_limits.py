"""Limits of the losses' arguments, refused synchronously before any device call: numbers
of sequences past what the kernels' 31-bit searches hold."""
import ctypes

import pytest

from lm_head_top_gb300 import kdkl
from tests.test_tune_abi import SHAPE, _pl, _policy, _pr, _pref, lib  # noqa: F401


@pytest.mark.parametrize("S", [(1 << 30) + 1, (1 << 31) - 2])
def test_sequences_past_the_search(lib, S):  # noqa: F811
    p = _policy(S=S, reduction=1)
    assert lib.kd_policy_workspace_size(ctypes.byref(p)) == 0 and _pl(lib, p, cu=64) == SHAPE
    q = _pref(P=(S + 1) // 2)
    assert lib.kd_pref_workspace_size(ctypes.byref(q)) == 0 and _pr(lib, q) == SHAPE


def test_the_most_sequences(lib):  # noqa: F811
    assert lib.kd_policy_workspace_size(ctypes.byref(_policy(S=1 << 30, reduction=1))) > 4 << 30
    assert lib.kd_pref_workspace_size(ctypes.byref(_pref(P=1 << 29))) > 4 << 30
