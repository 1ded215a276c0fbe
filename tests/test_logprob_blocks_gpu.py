"""dH cut into parts along the vocabulary together with several vocabulary blocks, the
last of them with fewer steps than there are parts; and logp and lse as exact as the
token's own fp32 logit makes them.

Bounds on dH and dW as in test_logprob_label_gpu: element by element, the entries that
pass through bf16 once, an output's own rounding, the own entries' fp32. fp32 sums over
the vocabulary or the tokens, in whatever parts: 2^-18 of the terms' magnitudes.

logp and lse at logits of 25, d = 2880: the own logit's fp32 sum is 1.6e-6 off (random
rounding of 90 products a lane and of 32 lanes), half a step of lse 1e-6, the sum of
exponentials 1e-6 or less: 1e-5 is 5 sigma, where the own logit carries all but 1 % of
the mass: the other logits keep the error of the products' accumulator (1e-5 of a logit
when all products have one sign, as here: 2.5e-4, times 1 %)."""
import pytest
import torch

from tests.test_logprob_label_gpu import _case, _delta, _hold, _want

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


# blocks of 2048 columns (32 steps, 4 parts), the 8th of 8 columns; four blocks of 32,000
SHAPES = [(300, 200, 14_344, 40), (2000, 1024, 128_000, 512)]


@pytest.mark.parametrize("T,d,V,chunk", SHAPES)
@pytest.mark.parametrize("form", ["fp32", "added", "bf16"])
@pytest.mark.parametrize("pairs", [True, False])
def test_parts_and_blocks(kdkl, monkeypatch, T, d, V, chunk, form, pairs):
    g = torch.Generator("cuda").manual_seed(T)
    ids = (torch.rand(T, generator=g, device="cuda") ** 3 * V).int().clamp_(max=V - 1)
    H, W, grad = _case(T, d, V, 1.0, ids, 8 * torch.rand(T, generator=g, device="cuda"))
    grad[::5] = 0
    if not pairs:
        monkeypatch.setenv("KDKL_CTA_PAIR", "0")
    _, lse = kdkl.kd_logprob_forward(H, W, ids)
    base = torch.zeros(V, d, device="cuda")
    kw = {"fp32": {}, "bf16": dict(dW_dtype=torch.bfloat16),
          "added": dict(dW=base, accumulate_dW=True)}[form]
    if form == "added":
        base[::3] = 0.5
    start = base.double()
    dH, dW = kdkl.kd_logprob_backward(H, W, ids, lse, grad, chunk=chunk, **kw)
    want_dH, want_dW, rest_dH, rest_dW, slope, logs = _want(H, W, ids, grad, 1.0)
    delta = grad.double().abs() * _delta(H, W, ids, 1.0, logs) + 2.0 ** -20 * slope.abs().sum(1)
    label = torch.zeros_like(want_dW).index_add_(0, ids.long(), delta[:, None] * H.double().abs())
    sums = 2.0 ** -18 * (slope.abs().t() @ H.double().abs())
    _hold(dW, start + want_dW, rest_dW, label + sums + 2.0 ** -20 * start, form == "bf16")
    _hold(dH, want_dH, rest_dH, delta[:, None] * W.double()[ids.long()].abs()
          + 2.0 ** -18 * (slope.abs() @ W.double().abs()), True)
    assert not dH[::5].any()


@pytest.mark.parametrize("rest", [1e-2, 1e-3, 1e-4])
@pytest.mark.parametrize("masked", [False, True])
def test_logp_and_lse_by_the_own_logit(kdkl, rest, masked):
    T, d, V = 64, 2880, 512
    g = torch.Generator("cuda").manual_seed(9)
    ids = torch.arange(0, 2 * T, 2, dtype=torch.int32, device="cuda")
    W = torch.randn(V, d, generator=g, device="cuda") / d ** 0.5
    H = 25 * W[ids.long()] / (W[ids.long()] ** 2).sum(1, keepdim=True)
    W[ids.long() + 1] = (1 + torch.log(torch.tensor(rest)) / 25) * W[ids.long()]
    H, W = H.bfloat16(), W.bfloat16()
    mask = (torch.arange(T, device="cuda") % 3 != 0).to(torch.uint8)
    logp, lse = kdkl.kd_logprob_forward(H, W, ids, mask if masked else None)
    z = H.double() @ W.double().t()
    want_lse = torch.logsumexp(z, 1)
    want = torch.log_softmax(z, 1).gather(1, ids.long()[:, None])[:, 0]
    on = mask != 0 if masked else torch.ones(T, dtype=torch.bool, device="cuda")
    assert (lse - want_lse)[on].abs().max().item() <= 1e-5
    assert (logp - want)[on].abs().max().item() <= 1e-5
    assert not lse[~on].any() and not logp[~on].any()
