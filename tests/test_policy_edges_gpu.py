"""The policy and the preference loss where a border or an input is at its end: clip ranges of
zero and of one, advantages of zero, inputs left out in runs through shared memory, token
counts around the kernels' pieces.

What the kernels do: a lane takes 4 consecutive tokens, a warp 128 a step, a block has 16
warps; the policy loss takes up to 4,096 tokens in one block and counts masks of up to 32,768
in every block, the preference loss up to 8,192 tokens and 256 pairs in one block; runs of
four and more pieces (from some 2.5M tokens) come through shared memory. e^x is the
hardware's base-2 exponential (2 ulp) of a product rounded to fp32; sums are kept in two
floats. The bounds of test_policy_gpu hold with these too: an exponent below 4 rounded to
2^-24 of itself and 2 ulp are 8 * 2^-24 of a factor, of the 32 that they allow.

The share of clipped tokens is a quotient of two whole numbers, rounded once: 2^-24."""
import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot
from tests.test_policy_gpu import _policy_case, _policy_check, _pref_case, _pref_check

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


@pytest.mark.parametrize("T", [127, 128, 129, 511, 513, 4095, 4096, 4097, 8191, 8192, 8193, 32767,
                               32768, 32769])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
def test_policy_around_the_pieces(kdkl, T, reduction):
    _, _, got, want, mask = _policy_case(kdkl, T, 5, seed=T, reduction=reduction, dual_clip=1.5)
    _policy_check(got, want, T, w_sum=max(1.0, (mask != 0).sum() / 77.0))


@pytest.mark.parametrize("T,P", [(127, 2), (128, 2), (129, 2), (8191, 256), (8192, 256), (8192, 257),
                                 (8193, 3), (40_000, 600)])
@pytest.mark.parametrize("kind", ["sigmoid", "ipo", "hinge"])
def test_pref_around_the_pieces(kdkl, T, P, kind):
    _, f, got, want, arrays = _pref_case(kdkl, T, P, seed=T, kind=kind, halves=bool(P % 2))
    _pref_check(got, want, arrays, f)


@pytest.mark.parametrize("kl", [False, True])
def test_clip_low_of_one(kdkl, kl):
    """The lower border is minus infinity: no ratio is below it."""
    _, _, got, want, _ = _policy_case(kdkl, 5003, 20, clip_low=1.0, clip_high=0.1, use_ref=kl)
    _policy_check(got, want, 5003)
    old = torch.zeros(3, device="cuda")
    logp = torch.tensor([-200.0, float("-inf"), 0.0], device="cuda")
    loss, stats, grad = kdkl.kd_policy_loss(logp, old, None, torch.full((3,), -2.0, device="cuda"),
                                            clip_low=1.0)
    assert stats[2].item() == 0 and grad[:2].tolist() == [0.0, 0.0]
    assert abs(grad[2].item() - 2 / 3) <= 2.0 ** -22 and abs(loss.item() - 2 / 3) <= 2.0 ** -22


def test_advantage_of_zero_is_on_the_upper_side(kdkl):
    """Past the upper border it counts as clipped, below the lower one not; loss and
    gradient are zero either way."""
    d = torch.tensor([0.5, -0.5, 0.1, 0.0, 0.5, -0.5], device="cuda")
    adv = torch.tensor([0.0, 0.0, 0.0, -0.0, -0.0, -0.0], device="cuda")
    loss, stats, grad = kdkl.kd_policy_loss(d, torch.zeros(6, device="cuda"), None, adv,
                                            dual_clip=1.2)
    assert loss.item() == 0 and not grad.any()
    assert abs(stats[2].item() - 2 / 6) <= 2.0 ** -24


@pytest.mark.parametrize("use_old,use_ref,use_mask", [(False, True, True), (True, False, True),
                                                      (True, True, False), (False, False, False)])
@pytest.mark.parametrize("per_seq,reduction", [(True, "sequence"), (False, "token")])
def test_inputs_left_out_in_long_runs(kdkl, use_old, use_ref, use_mask, per_seq, reduction):
    """Through shared memory (aligned arrays) and without it: the same bits, and the
    definition in 64 bits."""
    T, S = 2_600_003, 60
    r = np.random.default_rng(1)
    lp = (-3 * r.random(T)).astype(np.float32)
    lo, lr = ((lp + s * r.normal(size=T)).astype(np.float32) for s in (0.3, 0.5))
    on = (r.random(T) >= 0.3).astype(np.uint8)
    cu, adv = _ragged(T, S, r), r.normal(size=S if per_seq else T).astype(np.float32)
    ins = [_cuda(lp), _cuda(lo) if use_old else None, _cuda(lr) if use_ref else None, _cuda(adv),
           _cuda(on) if use_mask else None, _cuda(cu)]
    kw = dict(clip_low=0.2, clip_high=0.3, kl_coef=0.1 if use_ref else 0.0, reduction=reduction,
              grad_loss=0.7)
    got = kdkl.kd_policy_loss(*ins, **kw)
    pad = torch.zeros(T + 1, device="cuda")
    pad[1:] = ins[0]
    for a, b in zip(got, kdkl.kd_policy_loss(pad[1:], *ins[1:], **kw)):
        assert torch.equal(a, b)
    on = ins[4] != 0 if use_mask else torch.ones(T, dtype=torch.bool, device="cuda")
    seq = torch.bucketize(torch.arange(T, device="cuda"), ins[5][1:].long(), right=True)
    p = ins[0].double()
    d = p - ins[1].double() if use_old else torch.zeros_like(p)
    x = ins[2].double() - p if use_ref else torch.zeros_like(p)
    A = ins[3].double()[seq] if per_seq else ins[3].double()
    ratio = d.exp()
    s = torch.minimum(ratio * A, ratio.clamp(0.8, 1.3) * A)
    n = torch.zeros(S, dtype=torch.double, device="cuda").index_add_(0, seq, on.double())
    w = (on / on.sum().double() if reduction == "token"
         else on / (n * (n > 0).sum()).clamp(min=1)[seq])
    grad = 0.7 * w * (torch.where(s == ratio * A, -s, 0.0) - kw["kl_coef"] * torch.expm1(x))
    U = 32 * 2.0 ** -24
    off = (got[2].double() - grad).abs()
    assert (off <= 4 * U * torch.maximum(grad.abs(), grad.abs().mean())).all()
    pg, kl = -(w * s).sum().item(), (w * (torch.expm1(x) - x)).sum().item()
    size = (w * s.abs()).sum().item() + abs(kl)
    assert abs(got[0].item() - pg - kw["kl_coef"] * kl) <= U * size
    clipped = ((s != ratio * A) & on).sum().item() / on.sum().item()
    assert abs(got[1][2].item() - clipped) <= 2.0 ** -24
