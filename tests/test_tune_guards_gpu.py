"""The tuning calls write inside their outputs and workspaces and read nothing that they
have not written: workspaces of exactly the stated size and outputs lie between guard
regions that must survive, everything starts as 0xFF bytes (a NaN pattern), and the results
equal a clean call's bit for bit."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
GUARD = 1024


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


class _Guarded:
    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        n = 1
        for s in shape:
            n *= s
        size = n * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((2 * GUARD + -(-size // 256) * 256,), 0xFF, dtype=torch.uint8, device="cuda")
        room[:GUARD] = 0x5A
        room[GUARD + size:] = 0x5A
        self.all.append((room, size))
        return room[GUARD:GUARD + size].view(dtype).view(shape)

    def check(self):
        for room, size in self.all:
            assert (room[:GUARD] == 0x5A).all() and (room[GUARD + size:] == 0x5A).all()


@pytest.mark.parametrize("T,d,V,chunk", [(1, 8, 1, 4096), (130, 72, 513, 16), (700, 200, 9001, 100),
                                         (300, 2056, 40_001, 4096)])
@pytest.mark.parametrize("counted", ["some", "all", "none"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprob(kdkl, T, d, V, chunk, counted, dtype):
    g = torch.Generator("cuda").manual_seed(T)
    H = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=g, device="cuda") / d ** 0.5).bfloat16()
    ids = (torch.rand(T, generator=g, device="cuda") ** 3 * V).int()
    mask = {"some": (torch.rand(T, generator=g, device="cuda") < 0.4).to(torch.uint8),
            "all": None, "none": torch.zeros(T, dtype=torch.uint8, device="cuda")}[counted]
    grad = torch.randn(T, generator=g, device="cuda")
    if mask is not None:
        grad = torch.where(mask != 0, grad, 0.0)
    logp, lse = kdkl.kd_logprob_forward(H, W, ids, mask)
    want = (logp, lse) + kdkl.kd_logprob_backward(H, W, ids, lse, grad, dW_dtype=dtype, chunk=chunk)
    new = _Guarded()
    ws = new((kdkl.kd_logprob_workspace_size(T, d, V),), torch.uint8)
    got = kdkl.kd_logprob_forward(H, W, ids, mask, logp=new((T,), torch.float32),
                                  lse=new((T,), torch.float32), workspace=ws)
    wb = new((kdkl.kd_logprob_workspace_size(T, d, V, 1.0, chunk, 1, dtype),), torch.uint8)
    got += kdkl.kd_logprob_backward(H, W, ids, got[1], grad, chunk=chunk,
                                    dH=new((T, d), torch.bfloat16), dW=new((V, d), dtype),
                                    workspace=wb)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    new.check()
    assert kdkl.kd_kl_check_status(ws) == 0 and kdkl.kd_kl_check_status(wb) == 0


@pytest.mark.parametrize("T,S", [(1, 1), (100, 7), (4097, 50), (40_001, 3), (2_600_003, 400)])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy(kdkl, T, S, reduction):
    g = torch.Generator("cuda").manual_seed(T)
    x = [torch.randn(T, generator=g, device="cuda") for _ in range(3)]
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    cu = (torch.linspace(0, 1, S + 1, dtype=torch.double) * T).round().int().cuda()
    args = (x[0], x[0] + 0.2 * x[1], x[0] + 0.3 * x[2], x[1], mask, cu)
    kw = dict(kl_coef=0.1, reduction=reduction, dual_clip=2.0, advantage_per_sequence=False)
    want = kdkl.kd_policy_loss(*args, **kw)
    p = kdkl.kd_policy_problem(T, S, 0.2, 0.2, 2.0, 0.1, 1.0, kdkl.KD_REDUCTIONS[reduction], 0)
    new = _Guarded()
    ws = new((kdkl.load().kd_policy_workspace_size(ctypes.byref(p)),), torch.uint8)
    got = kdkl.kd_policy_loss(*args, loss=new((1,), torch.float32), stats=new((3,), torch.float32),
                              grad_logp=new((T,), torch.float32), workspace=ws, **kw)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    new.check()
    assert kdkl.kd_kl_check_status(ws) == 0


@pytest.mark.parametrize("T,P", [(2, 1), (100, 3), (8193, 40), (9000, 300), (2_600_003, 500)])
def test_pref(kdkl, T, P):
    g = torch.Generator("cuda").manual_seed(T)
    x = [torch.randn(T, generator=g, device="cuda") for _ in range(2)]
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8)
    cu = (torch.linspace(0, 1, 2 * P + 1, dtype=torch.double) ** 2 * T).round().int().cuda()
    want = kdkl.kd_pref_loss(*x, cu, mask, average=True)
    p = kdkl.kd_pref_problem(T, P, 0.1, 0.0, 0.0, 0, 1, 0, 0)
    new = _Guarded()
    ws = new((kdkl.load().kd_pref_workspace_size(ctypes.byref(p)),), torch.uint8)
    got = kdkl.kd_pref_loss(*x, cu, mask, average=True, loss=new((1,), torch.float32),
                            rewards=new((P, 2), torch.float32), grad_logp=new((T,), torch.float32),
                            workspace=ws)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    new.check()
    assert kdkl.kd_kl_check_status(ws) == 0
