"""Two steps of a tied student, each part against 64 bits: the first step's gradients, what the two
optimizers made of them, the copies that the next forward reads, and the second step's loss and
gradients from those. (How far a loss falls is not looked at.)"""
import os
import sys

import pytest
import torch

from oracle import body_oracle as bo
from test_train_tied_gpu import _graph

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
pytestmark = pytest.mark.gpu
U = 2.0 ** -24
GRAD_TOL = 0.02  # of a step's gradients in bf16: see test_train_tied_gpu.py
LR, WD, BETAS, EPS = 0.02, 0.1, (0.9, 0.95), 1e-8


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _adamw(p, g, m, v, step, decay):
    m = BETAS[0] * m.double() + (1 - BETAS[0]) * g.double()
    v = BETAS[1] * v.double() + (1 - BETAS[1]) * g.double() ** 2
    root = (v / (1 - BETAS[1] ** step)).sqrt()
    return p.double() * (1 - LR * decay) - LR / (1 - BETAS[0] ** step) * m / (root + EPS)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T,d,f,V,K", [(300, 96, 200, 1000, 16), (777, 264, 600, 3001, 8)])
def test_two_steps(kdkl, norm, T, d, f, V, K):
    from train_tied import Student
    s, teacher = Student(V, d, f, norm, 0), Student(V, d, f, norm, 1)
    g = torch.Generator("cuda").manual_seed(T)
    ids = (V * torch.rand(T, generator=g, device="cuda") ** 2).int().clamp_(max=V - 1)
    topk_idx, topk_logit = kdkl.kd_lmhead_topk(teacher.forward(ids), teacher.p["W"], K)
    mats = ["up", "down"]
    rest = [k for k in s.master if k not in mats]
    pick = lambda x, ks: [x[k] for k in ks]  # noqa: E731
    state = {name: {k: torch.zeros_like(v) for k, v in s.master.items()} for name in ("m", "v")}
    muon = kdkl.kd_muon_tensors(pick(s.master, mats), pick(s.grad, mats), pick(state["m"], mats), copies=pick(s.p, mats))
    adamw = kdkl.kd_adamw_tensors(pick(s.master, rest), pick(s.grad, rest), pick(state["m"], rest), pick(state["v"], rest),
                                  copies=pick(s.p, rest), decay=[k == "W" for k in rest])
    for step in (1, 2):
        H = s.forward(ids)
        loss, lse, _ = kdkl.kd_kl_forward(H, s.p["W"], topk_idx, topk_logit)
        dH, _ = kdkl.kd_kl_backward(H, s.p["W"], topk_idx, topk_logit, None, lse, dW=s.grad["W"])
        s.backward(dH)
        want_loss, want = _graph(s, ids, topk_idx, topk_logit)
        assert abs(loss.item() - want_loss) <= GRAD_TOL * abs(want_loss), step
        for k, t in want.items():
            off = float((s.grad[k].double() - t).norm() / t.norm())
            assert off <= GRAD_TOL, (step, k, off)
        before = {k: (s.master[k].clone(), s.grad[k].clone(), state["m"][k].clone(), state["v"][k].clone()) for k in s.master}
        kdkl.kd_muon_step(muon, lr=LR, weight_decay=WD)
        kdkl.kd_adamw_step(adamw, lr=LR, betas=BETAS, eps=EPS, weight_decay=WD, step=step)
        for k, (p0, g0, m0, v0) in before.items():
            assert torch.equal(s.grad[k], g0)
            if k in mats:
                p = bo.muon(p0, g0, m0, lr=LR, weight_decay=WD)[0]
                rel = 8.6e-4  # of the step: the bound of test_muon_gpu.py
            else:
                p = _adamw(p0, g0, m0, v0, step, WD if k == "W" else 0.0)
                rel = 16 * U  # m, v, their corrections, the root, the quotient, the product: a dozen roundings
            moved = float((p - p0.double()).norm())
            off = float((s.master[k].double() - p).norm())
            assert moved > 0 and off <= rel * moved + 3 * U * float(p0.double().norm()), (step, k, off, moved)
            assert torch.equal(s.p[k], s.master[k].bfloat16()), (step, k)
