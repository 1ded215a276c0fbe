"""The clipped policy loss and the preference loss on the GPU against the fp64
oracle: token counts around the kernels' 8- and 2048-token pieces, ragged and
empty sequences, masks that leave sequences or everything out, garbage under
the mask, unaligned arrays, ratios next to the clip borders.

Tolerances. A gradient is a product of a few fp32 factors: expf (2 ulp) of a
difference whose rounding (2^-24 |d|, |d| < 4) scales the result, the KL term's
series, three more roundings: 32 * 2^-24 of its largest factor is ample.
Losses are sums of such terms, added exactly enough (fp64 across threads):
the same bound times the sum of the terms' magnitudes.

(Since this was written the kernels take 4 tokens a lane and 128 a warp's step, e^x is
the hardware's base-2 exponential of a product rounded to fp32, and sums are kept in two
floats: an exponent below 4 rounded to 2^-24 of itself and 2 ulp are 8 * 2^-24 of a
factor, within the 32. test_policy_edges_gpu has the sizes around those pieces.)"""
import math

import numpy as np
import pytest
import torch

import oracle.tune_oracle as ot

pytestmark = pytest.mark.gpu
U = 32 * 2.0 ** -24


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _cuda(x):
    return None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _cu(T, S, r):
    ends = np.sort(r.integers(0, T + 1, S - 1)) if S > 1 else np.zeros(0, dtype=np.int64)
    return np.concatenate([[0], ends, [T]]).astype(np.int32)


def _tokens(T, seed, garbage, off=0.3):
    r = np.random.default_rng(seed)
    logp = (-3 * r.random(T)).astype(np.float32)
    old = (logp + 0.3 * r.normal(size=T)).astype(np.float32)
    ref = (logp + 0.5 * r.normal(size=T)).astype(np.float32)
    mask = (r.random(T) >= off).astype(np.uint8)
    if garbage:
        logp[mask == 0], old[mask == 0], ref[mask == 0] = np.nan, np.inf, -np.inf
    return r, logp, old, ref, mask


def _f(x):
    return None if x is None else x.astype(np.float64)


def _policy_case(kdkl, T, S, seed=0, garbage=True, use_old=True, use_ref=True, use_mask=True,
                 per_seq=False, **kw):
    r, logp, old, ref, mask = _tokens(T, seed, garbage and use_mask)
    cu = _cu(T, S, r)
    adv = r.normal(size=S if per_seq else T).astype(np.float32)
    f = dict(clip_low=0.2, clip_high=0.3, dual_clip=0.0, kl_coef=0.1 if use_ref else 0.0,
             reduction="token", norm=77.0)
    f.update(kw)
    old, ref, mask = (old if use_old else None), (ref if use_ref else None), \
        (mask if use_mask else None)
    ins = [_cuda(x) for x in (logp, old, ref, adv, mask, cu)]
    loss, stats, grad = kdkl.kd_policy_loss(*ins, grad_loss=0.7, **f)
    # the oracle takes the parameters as the fp32 values that the call's inputs are
    r_loss, r_stats, r_grad, clipped = ot.policy_loss(_f(logp), _f(old), _f(ref), _f(adv), mask, cu,
                                                      **f)
    return ins, f, (loss, stats, grad), (r_loss, r_stats, 0.7 * r_grad, clipped), mask


def _policy_check(got, want, logp_T, w_sum=1.0):
    loss, stats, grad = (t.cpu().numpy().astype(np.float64) for t in got)
    r_loss, r_stats, r_grad, clipped = want
    # factors: |A| < 5, r < e^4, |e^x - 1| < 20
    assert np.array_equal(grad == 0, r_grad == 0)
    scale = np.maximum(np.abs(r_grad), np.abs(r_grad).mean() if r_grad.any() else 0)
    assert (np.abs(grad - r_grad) <= 4 * U * scale + 1e-12).all()
    assert abs(loss[0] - r_loss) <= U * 8 * w_sum
    assert np.abs(stats[:2] - r_stats[:2]).max() <= U * 8 * w_sum
    assert abs(stats[2] - r_stats[2]) <= 1e-6


@pytest.mark.parametrize("T", [1, 7, 8, 9, 255, 2047, 2048, 2049, 5003, 33001])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("per_seq", [False, True])
def test_policy(kdkl, T, reduction, per_seq):
    S = max(2, T // 61) if T > 8 else 2
    if per_seq and S == T:
        S += 1
    _, _, got, want, mask = _policy_case(kdkl, T, S, seed=T, reduction=reduction, per_seq=per_seq,
                                         dual_clip=1.5)
    _policy_check(got, want, T, w_sum=max(1.0, (mask != 0).sum() / 77.0))


@pytest.mark.parametrize("use_old,use_ref,use_mask", [(False, True, True), (True, False, True),
                                                      (True, True, False), (False, False, False)])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_optional_inputs(kdkl, use_old, use_ref, use_mask, reduction):
    for T, S in ((600, 5), (40000, 3)):
        _, _, got, want, _ = _policy_case(kdkl, T, S, use_old=use_old, use_ref=use_ref,
                                          use_mask=use_mask, reduction=reduction)
        _policy_check(got, want, T)


@pytest.mark.parametrize("T", [2_600_001, 2_600_003])
@pytest.mark.parametrize("per_seq,reduction", [(True, "sequence"), (False, "token"), (False, "sum")])
def test_policy_long_runs(kdkl, T, per_seq, reduction):
    """Runs of several pieces per warp, through shared memory and (unaligned arrays)
    without it: the same bits, and the definition in 64 bits by torch."""
    S = 700
    r, logp, old, ref, mask = _tokens(T, 7, True)
    cu = _cu(T, S, r)
    adv = r.normal(size=S if per_seq else T).astype(np.float32)
    ins = [_cuda(x) for x in (logp, old, ref, adv, mask, cu)]
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=1.5, kl_coef=0.1, reduction=reduction,
              norm=1e6, grad_loss=0.7)
    got = kdkl.kd_policy_loss(*ins, **kw)
    pad = torch.zeros(T + 1, device="cuda")
    pad[1:] = ins[0]
    plain = kdkl.kd_policy_loss(pad[1:], *ins[1:], **kw)
    for a, b in zip(got, plain):
        assert torch.equal(a, b)
    on = ins[4] != 0
    seq = torch.bucketize(torch.arange(T, device="cuda"), ins[5][1:].long(), right=True)
    lp, lo, lr = (torch.where(on, t.double(), 0.0) for t in ins[:3])
    A = ins[3].double()[seq] if per_seq else ins[3].double()
    d, x = lp - lo, lr - lp
    ratio = d.exp()
    s = torch.minimum(ratio * A, ratio.clamp(0.8, 1.3) * A)
    s = torch.where(A < 0, torch.maximum(s, 1.5 * A), s)
    n = torch.zeros(S, dtype=torch.double, device="cuda").index_add_(0, seq, on.double())
    w = {"token": on / on.sum().double(), "sum": on / 1e6,
         "sequence": on / (n * (n > 0).sum()).clamp(min=1)[seq]}[reduction]
    grad = 0.7 * w * (torch.where(s == ratio * A, -s, 0.0) - 0.1 * torch.expm1(x))
    off = (got[2].double() - grad).abs()
    assert (off <= 4 * U * torch.maximum(grad.abs(), grad.abs().mean())).all()
    pg, kl = -(w * s).sum().item(), (w * (torch.expm1(x) - x)).sum().item()
    size = (w * s.abs()).sum().item() + abs(kl)
    assert abs(got[0].item() - pg - 0.1 * kl) <= U * size
    assert abs(got[1][0].item() - pg) <= U * size and abs(got[1][1].item() - kl) <= U * size


@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_many_empty_sequences(kdkl, reduction):
    """More sequences than tokens in a block, most of them empty."""
    _, _, got, want, _ = _policy_case(kdkl, 3000, 9000, reduction=reduction, per_seq=True)
    _policy_check(got, want, 3000)


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("T", [900, 40000])
def test_policy_nothing_counted(kdkl, reduction, T):
    r, logp, old, ref, _ = _tokens(T, 0, False)
    logp[:] = np.nan
    zero = torch.zeros(T, dtype=torch.uint8, device="cuda")
    loss, stats, grad = kdkl.kd_policy_loss(_cuda(logp), _cuda(old), _cuda(ref), _cuda(old), zero,
                                            _cuda(_cu(T, 4, r)), kl_coef=0.1, reduction=reduction)
    assert loss.item() == 0 and not stats.any() and not grad.any()
    e = torch.zeros(0, device="cuda")
    loss, stats, grad = kdkl.kd_policy_loss(e, e, e, e, kl_coef=0.1)
    assert loss.item() == 0 and not stats.any() and grad.numel() == 0


def test_policy_borders_take_64_bits(kdkl):
    """logp - old_logp within a few steps of log(1 + clip), many times over: the
    clipped set is the exact one."""
    r = np.random.default_rng(5)
    T, hi, lo = 20000, 0.2, 0.2
    old = (-8 * r.random(T)).astype(np.float32)
    border = np.where(r.random(T) < 0.5, math.log1p(hi), math.log1p(-lo))
    logp = (old.astype(np.float64) + border).astype(np.float32)
    for _ in range(2):
        step = r.integers(0, 3, T)
        logp = np.where(step == 0, np.nextafter(logp, np.float32(9)),
                        np.where(step == 1, np.nextafter(logp, np.float32(-99)), logp))
    adv = r.normal(size=T).astype(np.float32)
    d = logp.astype(np.float64) - old.astype(np.float64)
    clipped = np.where(adv >= 0, d > math.log1p(hi), d < math.log1p(-lo))
    _, stats, grad = kdkl.kd_policy_loss(_cuda(logp), _cuda(old), None, _cuda(adv), clip_low=lo,
                                         clip_high=hi)
    assert np.array_equal(grad.cpu().numpy() == 0, clipped)
    assert abs(stats[2].item() - clipped.mean()) < 1e-7
    assert 0.05 < clipped.mean() < 0.95


def test_policy_kl_term_near_zero(kdkl):
    """e^x - 1 - x for |x| down to 2^-40 keeps its digits."""
    x = np.concatenate([2.0 ** -np.arange(0, 40), -2.0 ** -np.arange(0, 40), [1.5, -1.5, 3.0, -6.0]])
    ref = x.astype(np.float32)
    logp, adv = np.zeros_like(ref), np.zeros_like(ref)
    for i in range(len(x)):
        _, stats, grad = kdkl.kd_policy_loss(_cuda(logp[i:i + 1]), None, _cuda(ref[i:i + 1]),
                                             _cuda(adv[i:i + 1]), kl_coef=1.0)
        xi = float(ref[i])
        # k by its series where the subtraction loses digits in 64 bits too
        k = xi * xi / 2 * (1 + xi / 3 + xi * xi / 12) if abs(xi) < 1e-3 else math.expm1(xi) - xi
        assert abs(stats[1].item() - k) <= U * abs(k) * 4
        assert abs(grad.item() + math.expm1(xi)) <= U * abs(math.expm1(xi))


def test_policy_unaligned_views_and_reruns(kdkl):
    ins, f, got, _, _ = _policy_case(kdkl, 5003, 40, reduction="sequence")
    shifted = []
    for i, t in enumerate(ins):
        if i < 5:
            pad = torch.zeros(t.numel() + 3, dtype=t.dtype, device="cuda")
            pad[3:] = t
            t = pad[3:]
        shifted.append(t)
    again = kdkl.kd_policy_loss(*shifted, grad_loss=0.7, **f)
    rerun = kdkl.kd_policy_loss(*ins, grad_loss=0.7, **f)
    for a, b, c in zip(got, again, rerun):
        assert torch.equal(a, b) and torch.equal(a, c)
    loss, stats, none = kdkl.kd_policy_loss(*ins, grad_loss=0.7, want_grad=False, **f)
    assert none is None and torch.equal(loss, got[0]) and torch.equal(stats, got[1])


@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [1, 5, 10], [0, 5, 9], [0, -4, 10], [0, 99, 10]])
def test_bad_offsets_are_reported(kdkl, cu):
    x = torch.zeros(10, device="cuda")
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    S = len(cu) - 1
    adv = torch.zeros(S, device="cuda")
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    for reduction in ("token", "sequence"):
        kdkl.kd_policy_loss(x, None, None, adv, None, cu_t, reduction=reduction, workspace=ws)
        assert kdkl.kd_kl_check_status(ws) == 1
    if S % 2 == 0:
        kdkl.kd_pref_loss(x, None, cu_t, workspace=ws)
        assert kdkl.kd_kl_check_status(ws) == 1


# -------------------------------------------------------------- preference loss

def _pref_case(kdkl, T, P, seed=0, use_ref=True, use_mask=True, grad_loss=0.6, **kw):
    r, logp, _, ref, mask = _tokens(T, seed, use_mask)
    cu = _cu(T, 2 * P, r)
    f = dict(beta=0.1, kind="sigmoid", label_smoothing=0.0, margin=0.0, average=False, halves=False)
    f.update(kw)
    ref, mask = (ref if use_ref else None), (mask if use_mask else None)
    ins = [_cuda(x) for x in (logp, ref, cu, mask)]
    got = kdkl.kd_pref_loss(*ins, grad_loss=grad_loss, **f)
    want = ot.pref_loss(_f(logp), _f(ref), mask, cu, **f)
    return ins, f, got, (want[0], want[1], grad_loss * want[2]), (logp, ref, mask, cu)


def _pref_check(got, want, arrays, f):
    loss, rewards, grad = (t.cpu().numpy().astype(np.float64) for t in got)
    logp, ref, mask, cu = arrays
    # a sequence's sum: every log ratio rounded once and added in fp32 by eights, then in fp64
    # (by fours, then in two floats: fewer roundings than the bound below counts)
    on = np.ones(len(logp), bool) if mask is None else mask != 0
    gap = np.where(on, np.abs(logp.astype(np.float64)) + (0 if ref is None else np.abs(ref)), 0.0)
    gap = np.where(np.isfinite(gap), gap, 0.0)
    tot = np.array([gap[a:b].sum() for a, b in zip(cu, cu[1:])])
    off = 64 * 2.0 ** -24 * max(1.0, tot.max())     # of a sequence's sum
    beta = f["beta"]
    assert np.abs(rewards - want[1]).max() <= beta * off + 2.0 ** -23 * np.abs(want[1]).max()
    steep = {"sigmoid": beta, "hinge": beta, "ipo": 2 * (tot.max() * 2 + 1 / beta)}[f["kind"]]
    assert abs(loss[0] - want[0]) <= 2 * off * steep + 2.0 ** -23 * abs(want[0])
    curve = {"sigmoid": beta * beta, "hinge": 0.0, "ipo": 2.0}[f["kind"]]
    top = np.abs(want[2]).max()
    P = len(want[1])
    assert np.abs(grad - want[2]).max() <= 2 * off * curve / P + 2.0 ** -23 * top
    assert not grad[~on].any()


@pytest.mark.parametrize("T,P", [(2, 1), (7, 2), (300, 3), (2048, 4), (2049, 1), (5003, 40),
                                 (30011, 7), (4000, 3000)])
@pytest.mark.parametrize("kind", ["sigmoid", "ipo", "hinge"])
@pytest.mark.parametrize("average", [False, True])
def test_pref(kdkl, T, P, kind, average):
    _, f, got, want, arrays = _pref_case(kdkl, T, P, seed=T, kind=kind, average=average,
                                         halves=bool(T % 2), label_smoothing=0.1, margin=0.2)
    _pref_check(got, want, arrays, f)


@pytest.mark.parametrize("use_ref,use_mask", [(False, True), (True, False), (False, False)])
def test_pref_optional_inputs(kdkl, use_ref, use_mask):
    _, f, got, want, arrays = _pref_case(kdkl, 6007, 9, use_ref=use_ref, use_mask=use_mask)
    _pref_check(got, want, arrays, f)


def test_pref_nothing_counted(kdkl):
    T = 3000
    nan = torch.full((T,), float("nan"), device="cuda")
    cu = torch.tensor([0, 1000, 1000, 2000, T], dtype=torch.int32, device="cuda")
    loss, rewards, grad = kdkl.kd_pref_loss(nan, nan, cu, torch.zeros(T, dtype=torch.uint8,
                                                                      device="cuda"))
    assert abs(loss.item() - math.log(2)) < 1e-6 and not rewards.any() and not grad.any()
    e = torch.zeros(0, device="cuda")
    loss, rewards, grad = kdkl.kd_pref_loss(e, e, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert abs(loss.item() - math.log(2)) < 1e-6 and not rewards.any() and grad.numel() == 0
    loss, rewards, _ = kdkl.kd_pref_loss(e, e, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert loss.item() == 0 and rewards.shape == (0, 2)


def test_pref_extreme_margins(kdkl):
    """Log ratios far apart: no overflow, slopes 0 and 1."""
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for gap, want in ((1e5, 0.0), (-1e5, 1e4)):
        logp = torch.tensor([gap, 0.0], device="cuda")
        loss, _, grad = kdkl.kd_pref_loss(logp, None, cu, beta=0.1)
        assert abs(loss.item() - want) <= 1e-3
        assert abs(grad[0].item() + (0.0 if gap > 0 else 0.1)) <= 1e-7


def test_pref_nan_reaches_the_loss(kdkl):
    cu = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    logp = torch.tensor([float("nan"), -1.0, -1.0, -2.0], device="cuda")
    for kind in ("sigmoid", "ipo", "hinge"):
        loss, _, grad = kdkl.kd_pref_loss(logp, None, cu, kind=kind)
        assert loss.isnan().all() and grad.isnan().all()


def test_pref_unaligned_views_and_reruns(kdkl):
    ins, f, got, _, _ = _pref_case(kdkl, 5003, 11, average=True)
    shifted = list(ins)
    for i in (0, 1, 3):
        pad = torch.zeros(ins[i].numel() + 1, dtype=ins[i].dtype, device="cuda")
        pad[1:] = ins[i]
        shifted[i] = pad[1:]
    for other in (kdkl.kd_pref_loss(*shifted, grad_loss=0.6, **f),
                  kdkl.kd_pref_loss(*ins, grad_loss=0.6, **f)):
        for a, b in zip(got, other):
            assert torch.equal(a, b)


# ----------------------------------------------- streams, graphs, the whole step

class _Step:
    """One preference step of a head on static buffers: forward, loss, backward, optimizer."""

    def __init__(self, kdkl, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)
        T, d, V, P = 200, 64, 700, 4
        self.k = kdkl
        self.H = torch.randn(T, d, generator=g, device="cuda").bfloat16()
        self.master = torch.randn(V, d, generator=g, device="cuda") / 8
        self.W = self.master.bfloat16()
        self.ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.ref = -6 - torch.rand(T, generator=g, device="cuda")
        self.cu = torch.arange(0, T + 1, T // (2 * P), dtype=torch.int32, device="cuda")
        self.dW = torch.empty(V, d, device="cuda")
        self.m, self.v = torch.zeros_like(self.dW), torch.zeros_like(self.dW)
        self.opt = kdkl.kd_adamw_tensors([self.master], [self.dW], [self.m], [self.v],
                                         copies=[self.W])
        self.out = None

    def __call__(self, stream=None):
        k = self.k
        logp, lse = k.kd_logprob_forward(self.H, self.W, self.ids, stream=stream)
        loss, rewards, grad = k.kd_pref_loss(logp, self.ref, self.cu, beta=0.5, stream=stream)
        dH, _ = k.kd_logprob_backward(self.H, self.W, self.ids, lse, grad, dW=self.dW,
                                      stream=stream)
        k.kd_adamw_step(self.opt, lr=1e-2, step=1, stream=stream)
        self.out = (loss, rewards, dH)
        return self.out

    def state(self):
        return [t.clone() for t in (*self.out, self.dW, self.master, self.W, self.m, self.v)]


def test_step_on_a_side_stream_and_in_a_graph(kdkl):
    eager = _Step(kdkl)
    losses = [eager()[0].item() for _ in range(3)]
    assert losses[0] > losses[1] > losses[2]
    want = eager.state()

    side = _Step(kdkl)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        side(stream=stream)
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, side.state()))

    warm = _Step(kdkl)  # first launches outside the capture
    warm()
    captured = _Step(kdkl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, captured.state()))
