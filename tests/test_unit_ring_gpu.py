"""The GEMM's units reach every role whichever way they are handed out: taken from
the launch's counter or round-robin, by CTA pairs or single CTAs, more units than
the ring has slots, units without K steps, fewer units than CTAs.

Round-robin changes no product and no order of sums: the results are the same bit
for bit. Single CTAs may cut the vocabulary into other splits: there the bounds of
the log-probabilities' own tests hold (a bf16 rounding of the logits' gradient and
one of the output, 2^-7 in the 2-norm; 1e-3 for logp)."""
import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot
from tests._helpers import LSE_ATOL, rel_l2
from tests.test_logprob_gpu import GRAD_TOL, _f64, _make

pytestmark = pytest.mark.gpu

# one tile of each product; more units than slots on every pair; a ragged K
SHAPES = [(1, 8, 9), (300, 200, 40_000), (700, 72, 60_001)]


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _run(kdkl, H, W, ids, mask, grad):
    logp, lse = kdkl.kd_logprob_forward(H, W, ids, mask)
    dH, dW = kdkl.kd_logprob_backward(H, W, ids, lse, grad)
    torch.cuda.synchronize()
    return logp, lse, dH, dW


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("counted", ["some", "none"])
def test_round_robin_same_bits(kdkl, monkeypatch, shape, counted):
    H, W, ids, mask, grad = (x.cuda() for x in _make(*shape, seed=3))
    if counted == "none":
        mask, grad = torch.zeros_like(mask), torch.zeros_like(grad)
    a = _run(kdkl, H, W, ids, mask, grad)
    monkeypatch.setenv("KDKL_STATIC_SCHED", "1")
    b = _run(kdkl, H, W, ids, mask, grad)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("static", [False, True])
def test_single_ctas(kdkl, monkeypatch, shape, static):
    H, W, ids, mask, grad = _make(*shape, seed=4, off=0.4 if shape[0] > 1 else 0.0)
    monkeypatch.setenv("KDKL_CTA_PAIR", "0")
    if static:
        monkeypatch.setenv("KDKL_STATIC_SCHED", "1")
    logp, lse, dH, dW = _run(kdkl, *(x.cuda() for x in (H, W, ids, mask, grad)))
    want, want_lse = ot.logprob_forward(_f64(H), _f64(W), ids.numpy(), mask.numpy(), 1.0)
    assert np.abs(logp.cpu().numpy() - want).max() <= LSE_ATOL
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= LSE_ATOL
    want_dH, want_dW = ot.logprob_backward(_f64(H), _f64(W), ids.numpy(),
                                           grad.numpy().astype(float), 1.0)
    assert rel_l2(dH.float().cpu().numpy(), want_dH) <= GRAD_TOL
    assert rel_l2(dW.cpu().numpy(), want_dW) <= GRAD_TOL
