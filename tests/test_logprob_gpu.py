"""Token log-probabilities of the LM head and their gradients against the fp64
oracle.

Tolerances. logp, lse: fp32 accumulation of d products and of V exponentials of
logits of a few tens, well within 1e-3 (the KL path's bound). dH, dW: each
logit gradient is rounded to bf16 once (relative 2^-8 at most) before the
product and a bf16 output once more (2^-8): in the 2-norm at most their sum,
2^-7, when the terms do not cancel, as random rows do not."""
import numpy as np
import pytest
import torch

import oracle.kl_oracle as ok
import oracle.tune_oracle as ot
from tests._helpers import LSE_ATOL, rel_l2

pytestmark = pytest.mark.gpu
GRAD_TOL = 2.0 ** -7


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _make(T, d, V, seed=0, off=0.4):
    r = np.random.default_rng(seed)
    W = r.normal(size=(V, d)) / np.sqrt(d)
    ids = (V * r.random(T) ** 2).astype(np.int32)
    H = r.normal(size=(T, d)) + 8 * r.random((T, 1)) * W[ids]
    mask = (r.random(T) >= off).astype(np.uint8)
    grad = np.where(mask != 0, r.normal(size=T), 0.0).astype(np.float32)
    return (torch.from_numpy(H).bfloat16(), torch.from_numpy(W).bfloat16(),
            torch.from_numpy(ids), torch.from_numpy(mask), torch.from_numpy(grad))


def _f64(t):
    return ok.bf16_bits_to_f64(t.view(torch.int16).numpy())


SHAPES = [(1, 8, 1), (1, 64, 700), (3, 8, 257), (64, 72, 256), (255, 72, 513), (257, 320, 1000),
          (300, 576, 4099), (700, 64, 100), (513, 256, 2050)]


@pytest.mark.parametrize("T,d,V", SHAPES)
@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("masked", [False, True])
def test_forward(kdkl, T, d, V, tau, masked):
    H, W, ids, mask, _ = _make(T, d, V)
    logp, lse = kdkl.kd_logprob_forward(H.cuda(), W.cuda(), ids.cuda(),
                                        mask.cuda() if masked else None, temperature=tau)
    r_logp, r_lse = ot.logprob_forward(_f64(H), _f64(W), ids.numpy(),
                                       mask.numpy() if masked else None, tau)
    assert np.abs(logp.cpu().numpy() - r_logp).max() <= LSE_ATOL
    assert np.abs(lse.cpu().numpy() - r_lse).max() <= LSE_ATOL


@pytest.mark.parametrize("T,d,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("chunk", [32, 4096])
def test_backward(kdkl, T, d, V, dtype, chunk):
    tau = 0.8
    H, W, ids, mask, grad = _make(T, d, V)
    g = [t.cuda() for t in (H, W, ids, grad)]
    _, lse = kdkl.kd_logprob_forward(*g[:3], temperature=tau)
    dH, dW = kdkl.kd_logprob_backward(*g[:3], lse, g[3], temperature=tau, chunk=chunk,
                                      dW_dtype=dtype)
    r_dH, r_dW = ot.logprob_backward(_f64(H), _f64(W), ids.numpy(), grad.numpy().astype(float), tau)
    assert dW.dtype == dtype
    if V == 1:  # one word: its probability is one and every gradient zero, up to lse's rounding
        assert np.abs(dH.float().cpu().numpy()).max() <= 1e-5 * np.abs(grad.numpy()).max() * 30
        return
    assert rel_l2(dH.float().cpu().numpy(), r_dH) <= GRAD_TOL
    assert rel_l2(dW.float().cpu().numpy(), r_dW) <= GRAD_TOL
    assert not dH.float().cpu().numpy()[grad.numpy() == 0].any()


def test_accumulates_into_fp32(kdkl):
    H, W, ids, mask, grad = [t.cuda() for t in _make(300, 128, 900)]
    _, lse = kdkl.kd_logprob_forward(H, W, ids)
    _, once = kdkl.kd_logprob_backward(H, W, ids, lse, grad, chunk=64)
    base = torch.randn_like(once)
    _, both = kdkl.kd_logprob_backward(H, W, ids, lse, grad, chunk=64, dW=base.clone(),
                                       accumulate_dW=True)
    # fp32 sums: the base is added last or first, one rounding of a value below ~8 each
    assert (both - base - once).abs().max().item() <= 2e-6 * 8
    with pytest.raises(ValueError):
        kdkl.kd_logprob_backward(H, W, ids, lse, grad, dW=base.bfloat16(), accumulate_dW=True)


def test_masked_places_are_not_read(kdkl):
    H, W, ids, mask, grad = _make(400, 96, 1000)
    clean = [t.cuda() for t in (H, W, ids, mask, grad)]
    logp, lse = kdkl.kd_logprob_forward(*clean[:4])
    dH, dW = kdkl.kd_logprob_backward(*clean[:3], lse, clean[4])
    off = mask == 0
    H2, ids2 = H.clone(), ids.clone()
    H2[off] = float("nan")
    ids2[off] = -7
    lse2 = lse.clone()
    lse2[off.cuda()] = float("inf")
    ws = torch.empty(kdkl.kd_logprob_workspace_size(400, 96, 1000), dtype=torch.uint8,
                     device="cuda")
    got = kdkl.kd_logprob_forward(H2.cuda(), clean[1], ids2.cuda(), clean[3], workspace=ws)
    assert torch.equal(got[0], logp) and torch.equal(got[1], lse)
    assert kdkl.kd_kl_check_status(ws) == 0
    got = kdkl.kd_logprob_backward(H2.cuda(), clean[1], ids2.cuda(), lse2, clean[4])
    assert torch.equal(got[0], dH) and torch.equal(got[1], dW)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nothing_counted_and_no_tokens(kdkl, dtype):
    H, W, ids, mask, grad = [t.cuda() for t in _make(130, 64, 500)]
    logp, lse = kdkl.kd_logprob_forward(H, W, ids, torch.zeros_like(mask))
    assert not logp.any() and not lse.any()
    dH, dW = kdkl.kd_logprob_backward(H, W, ids, lse, torch.zeros_like(grad), dW_dtype=dtype)
    assert not dH.any() and not dW.any()
    logp, lse = kdkl.kd_logprob_forward(H[:0], W, ids[:0], mask[:0])
    dH, dW = kdkl.kd_logprob_backward(H[:0], W, ids[:0], lse, grad[:0], dW_dtype=dtype)
    assert logp.numel() == 0 and dH.numel() == 0 and not dW.any()


@pytest.mark.parametrize("bad", [-1, 500])
def test_bad_id_is_reported(kdkl, bad):
    H, W, ids, mask, grad = [t.cuda() for t in _make(130, 64, 500)]
    ids[77] = bad
    ws = torch.empty(kdkl.kd_logprob_workspace_size(130, 64, 500), dtype=torch.uint8, device="cuda")
    kdkl.kd_logprob_forward(H, W, ids, workspace=ws)
    assert kdkl.kd_kl_check_status(ws) == 4
    ws = torch.empty(kdkl.kd_logprob_workspace_size(130, 64, 500, which=1), dtype=torch.uint8,
                     device="cuda")
    grad[77] = 1.0
    kdkl.kd_logprob_backward(H, W, ids, torch.zeros(130, device="cuda"), grad, workspace=ws)
    assert kdkl.kd_kl_check_status(ws) == 4


def test_small_workspace_is_refused(kdkl):
    H, W, ids, mask, grad = [t.cuda() for t in _make(130, 64, 500)]
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    with pytest.raises(kdkl.KDKLError):
        kdkl.kd_logprob_forward(H, W, ids, workspace=ws)


def test_gradient_nan_reaches_the_outputs(kdkl):
    H, W, ids, mask, grad = [t.cuda() for t in _make(130, 64, 500)]
    grad[5] = float("nan")
    _, lse = kdkl.kd_logprob_forward(H, W, ids)
    dH, dW = kdkl.kd_logprob_backward(H, W, ids, lse, grad)
    assert dH[5].isnan().all() and dW.isnan().any()


@pytest.mark.parametrize("T", [1, 5, 4097])
def test_large_vocabulary_rows(kdkl, T):
    """Many vocabulary splits per token, few and many tokens, against torch in 64 bits."""
    d, V = 128, 60000
    H, W, ids, mask, grad = [t.cuda() for t in _make(T, d, V, seed=3)]
    logp, lse = kdkl.kd_logprob_forward(H, W, ids)
    z = H.double() @ W.double().t()
    ref = torch.logsumexp(z, 1)
    assert (lse - ref).abs().max().item() <= LSE_ATOL
    assert (logp - (z.gather(1, ids.long()[:, None])[:, 0] - ref)).abs().max().item() <= LSE_ATOL


@pytest.mark.parametrize("T", [1024, 1025, 32768, 32769, 70001])
def test_compaction_over_many_tokens(kdkl, T):
    """Token counts around the compaction's tiles, most tokens without a gradient."""
    d, V = 8, 40
    H, W, ids, mask, grad = _make(T, d, V, seed=5, off=0.9)
    g = [t.cuda() for t in (H, W, ids, mask, grad)]
    logp, lse = kdkl.kd_logprob_forward(*g[:4])
    dH, dW = kdkl.kd_logprob_backward(*g[:3], lse, g[4])
    z = g[0].double() @ g[1].double().t()
    on = g[3] != 0
    ref = torch.where(on, z.gather(1, g[2].long()[:, None])[:, 0] - torch.logsumexp(z, 1), 0.0)
    assert (logp - ref).abs().max().item() <= LSE_ATOL
    slope = -torch.softmax(z, 1)
    slope[torch.arange(T, device="cuda"), g[2].long()] += 1
    slope *= g[4].double()[:, None]
    assert rel_l2(dH.float().cpu().numpy(), (slope @ g[1].double()).cpu().numpy()) <= GRAD_TOL
    assert rel_l2(dW.cpu().numpy(), (slope.t() @ g[0].double()).cpu().numpy()) <= GRAD_TOL
    assert not dH[~on].any()
