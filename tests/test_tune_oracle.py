"""Pins of the oracle of the tuning calls: gradients against central
differences, the losses against closed special cases, e4m3 against torch."""
import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot

EPS = 1e-6


def _numeric(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        old = x[i]
        x[i] = old + EPS
        up = f()
        x[i] = old - EPS
        g[i] = (up - f()) / (2 * EPS)
        x[i] = old
    return g


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_logprob_gradients_match_differences(tau):
    r = np.random.default_rng(0)
    H, W = r.normal(size=(5, 6)), r.normal(size=(9, 6))
    ids, grad = r.integers(0, 9, 5), r.normal(size=5)
    grad[2] = 0.0
    f = lambda: float(ot.logprob_forward(H, W, ids, None, tau)[0] @ grad)  # noqa: E731
    dH, dW = ot.logprob_backward(H, W, ids, grad, tau)
    assert np.abs(dH - _numeric(f, H)).max() < 1e-8
    assert np.abs(dW - _numeric(f, W)).max() < 1e-8
    assert not dH[2].any()


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("dual", [0.0, 1.5])
def test_policy_gradient_matches_differences(reduction, dual):
    r = np.random.default_rng(1)
    T, cu = 40, np.array([0, 7, 7, 30, 40])
    logp, old, ref = (-r.random(T) * 3 for _ in range(3))
    adv, mask = r.normal(size=T), (r.random(T) < 0.7).astype(np.uint8)
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=dual, kl_coef=0.3, reduction=reduction,
              norm=11.0)
    loss, stats, grad, _ = ot.policy_loss(logp, old, ref, adv, mask, cu, **kw)
    num = _numeric(lambda: ot.policy_loss(logp, old, ref, adv, mask, cu, **kw)[0], logp)
    assert np.abs(grad - num).max() < 1e-7
    assert abs(loss - stats[0] - 0.3 * stats[1]) < 1e-12
    # the min / clip form of the surrogate
    ratio = np.exp(logp - old)
    s = np.minimum(ratio * adv, np.clip(ratio, 0.8, 1.3) * adv)
    if dual:
        s = np.where(adv < 0, np.maximum(s, dual * adv), s)
    w, _ = ot.policy_weights(mask, cu, T, reduction, 11.0)
    assert abs(stats[0] + (w * s).sum()) < 1e-12


@pytest.mark.parametrize("kind", ["sigmoid", "ipo", "hinge"])
@pytest.mark.parametrize("average,halves", [(False, False), (True, True)])
def test_pref_gradient_matches_differences(kind, average, halves):
    r = np.random.default_rng(2)
    T, cu = 33, np.array([0, 5, 12, 12, 20, 28, 33])
    logp, ref, mask = -r.random(T), -r.random(T), (r.random(T) < 0.8).astype(np.uint8)
    kw = dict(beta=0.7, kind=kind, label_smoothing=0.1, margin=0.2, average=average, halves=halves)
    _, _, grad = ot.pref_loss(logp, ref, mask, cu, **kw)
    num = _numeric(lambda: ot.pref_loss(logp, ref, mask, cu, **kw)[0], logp)
    assert np.abs(grad - num).max() < 1e-8


def test_pref_of_equal_policies_is_log_two():
    logp, cu = -np.arange(6.0), np.array([0, 3, 6])
    loss, rewards, _ = ot.pref_loss(logp, logp.copy(), None, cu, beta=0.3, kind="sigmoid",
                                    label_smoothing=0.0, margin=0.0, average=False, halves=False)
    assert abs(loss - np.log(2)) < 1e-12 and not rewards.any()


def test_adamw_first_step_moves_by_lr():
    p, m, v = ot.adamw(np.zeros(3), np.array([1e-3, -5.0, 0.0]), np.zeros(3), np.zeros(3), lr=0.1,
                       betas=(0.9, 0.999), eps=0.0 + 1e-30, weight_decay=0.0, step=1,
                       grad_scale=1.0)
    assert np.allclose(p, [-0.1, 0.1, 0.0])


def test_e4m3_matches_torch():
    x = np.concatenate([np.random.default_rng(3).normal(size=4000) * 100,
                        ot.e4m3_values()[:-1] + np.diff(ot.e4m3_values()) / 2,
                        np.array([0.0, -0.0, 463.0, 448.0, 2.0 ** -10, 2.0 ** -9])])
    x = x[np.abs(x) <= 463].astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(ot.to_e4m3(x.astype(np.float64)), got.astype(np.float64))
