"""The policy loss where a border or an input is at its end: clip ranges of zero.

The share of clipped tokens is a quotient of two whole numbers, rounded once: 2^-24."""
import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _cuda(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _ragged(T, S, r):
    """Offsets of S sequences, ends at odd places, some empty."""
    ends = np.sort(r.integers(0, T + 1, S - 1))
    return np.concatenate([[0], ends, [T]]).astype(np.int32)


@pytest.mark.parametrize("clip_low,clip_high", [(0.2, 0.0), (0.0, 0.3), (0.0, 0.0)])
@pytest.mark.parametrize("reduction,per_seq", [("token", False), ("token", True), ("sequence", True)])
@pytest.mark.parametrize("T,S", [(7, 3), (515, 40), (5003, 700), (2_600_003, 900)])
def test_clip_range_of_zero_counts_counted_tokens(kdkl, clip_low, clip_high, reduction, per_seq, T,
                                                  S):
    """Under the mask lie finite values whose ratio is past the border."""
    r = np.random.default_rng(T)
    logp = (-3 * r.random(T)).astype(np.float32)
    old = (logp + 0.3 * r.normal(size=T)).astype(np.float32)
    old[r.random(T) < 0.2] = logp[0]
    logp[old == logp[0]] = logp[0]  # ratios of exactly one
    mask = (r.random(T) >= 0.4).astype(np.uint8)
    off = mask == 0
    old[off] = logp[off] - np.where(r.random(off.sum()) < 0.5, 0.5, -0.5).astype(np.float32)
    cu = _ragged(T, S, r)
    adv = r.normal(size=S if per_seq else T).astype(np.float32)
    seq = np.searchsorted(cu[1:], np.arange(T), side="right")
    A = adv[seq] if per_seq else adv
    d = logp.astype(np.float64) - old.astype(np.float64)
    clipped = np.where(A >= 0, d > np.log1p(clip_high), d < np.log1p(-clip_low)) & ~off
    _, stats, grad = kdkl.kd_policy_loss(_cuda(logp), _cuda(old), None, _cuda(adv), _cuda(mask),
                                         _cuda(cu), clip_low=clip_low, clip_high=clip_high,
                                         reduction=reduction)
    assert abs(stats[2].item() - clipped.sum() / mask.sum()) <= 2.0 ** -24
    assert np.array_equal(grad.cpu().numpy() == 0, off | clipped)
    if T < 10_000:
        want = ot.policy_loss(logp.astype(np.float64), old.astype(np.float64), None,
                              adv.astype(np.float64), mask, cu, clip_low=clip_low,
                              clip_high=clip_high, dual_clip=0.0, kl_coef=0.0, reduction=reduction,
                              norm=1.0)
        assert abs(stats[2].item() - want[1][2]) <= 2.0 ** -24


@pytest.mark.parametrize("reduction", ["token", "sequence"])
@pytest.mark.parametrize("T", [2, 9, 700, 6001])
def test_as_many_sequences_as_tokens(kdkl, reduction, T):
    """Some sequences empty, others longer: either meaning of T advantages, told by the
    word. A token's gradient is the same product whichever array its advantage is from."""
    r = np.random.default_rng(T)
    logp = (-3 * r.random(T)).astype(np.float32)
    old = (logp + 0.3 * r.normal(size=T)).astype(np.float32)
    cu, adv = _ragged(T, T, r), r.normal(size=T).astype(np.float32)
    seq = np.searchsorted(cu[1:], np.arange(T), side="right")
    args = [_cuda(logp), _cuda(old), None]
    kw = dict(reduction=reduction)
    a = kdkl.kd_policy_loss(*args, _cuda(adv), None, _cuda(cu), advantage_per_sequence=True, **kw)
    b = kdkl.kd_policy_loss(*args, _cuda(adv[seq]), None, _cuda(cu), advantage_per_sequence=False,
                            **kw)
    c = kdkl.kd_policy_loss(*args, _cuda(adv), None, _cuda(cu), advantage_per_sequence=False, **kw)
    assert torch.equal(a[2], b[2]) and torch.equal(a[1], b[1]) and torch.equal(a[0], b[0])
    assert torch.equal(a[2], c[2]) == (seq == np.arange(T)).all()  # one token each: the same
