"""8-bit states: every code and scale is the elementwise formula's, each operation rounded to
fp32 by itself and the root correctly rounded, over enough elements for some roots to lie
next to halfway between two codes (8 halfway points in 2^23 floats: one in a million)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BLOCK, BORDER = 256, 0.904383


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _quantise(x, least):
    x = x.view(-1, BLOCK)
    half, e = torch.frexp(x.abs().amax(1))
    scale = torch.where(half > 0, torch.ldexp(torch.ones_like(half), (e - 9 + (half > BORDER)).clamp(min=-126)), 1.0)
    q = (x / scale[:, None]).view(-1).to(torch.float8_e4m3fn)
    if least:
        q = torch.where((x.view(-1) > 0) & (q.float() == 0), 2.0 ** -9, q.float()).to(torch.float8_e4m3fn)
    return q, scale


@pytest.mark.parametrize("seed", [0, 1, 2])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_codes_of_many_elements(kdkl, seed, grad):
    n = BLOCK * 100_000
    b1, b2, lr, t, eps = 0.9, 0.95, 3e-4, 7, 1e-8
    g = torch.Generator("cuda").manual_seed(seed)
    gr = (torch.randn(n, generator=g, device="cuda") * 1e-3).to(grad)
    p = torch.randn(n, generator=g, device="cuda") * 0.02
    m, ms = _quantise(torch.randn(n, generator=g, device="cuda") * 5e-4, False)
    r, rs = _quantise(torch.rand(n, generator=g, device="cuda") * 1e-3 + 1e-5, True)
    gf = gr.float()
    m32 = (m.float().view(-1, BLOCK) * ms[:, None]).view(-1) * b1 + gf * (1 - b1)
    v32 = (r.float().view(-1, BLOCK) * rs[:, None]).view(-1) ** 2 * b2 + gf * gf * (1 - b2)
    root = v32.sqrt()
    want_m, want_ms = _quantise(m32, False)
    want_r, want_rs = _quantise(root, True)
    want_p = p - m32 / (root * (1 / math.sqrt(1 - b2 ** t)) + eps) * (lr / (1 - b1 ** t))
    handle = kdkl.kd_adamw_tensors([p], [gr], [m], [r], m_scales=[ms], v_scales=[rs])
    kdkl.kd_adamw_step(handle, lr=lr, betas=(b1, b2), eps=eps, step=t)
    assert torch.equal(ms, want_ms) and torch.equal(rs, want_rs)
    assert torch.equal(m.view(torch.uint8), want_m.view(torch.uint8))
    assert torch.equal(r.view(torch.uint8), want_r.view(torch.uint8))
    # p: the quotient is an approximation of 2 ulp of the step, below 5e-2 here
    assert (p - want_p).abs().max().item() <= 2.0 ** -21 * 5e-2 + 2.0 ** -24 * 0.2
