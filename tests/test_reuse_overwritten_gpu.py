"""A backward does not reuse a forward workspace that another call has overwritten since:
every call that takes a workspace drops the record of the forward that filled it."""
import pytest
import torch

from lm_head_top_gb300.inputs import WORKLOADS, make_inputs

pytestmark = pytest.mark.gpu
T, d, V, K, CHUNK = 96, 64, 500, 8, 64
INVALID = 1


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


@pytest.fixture(scope="module")
def g():
    w = WORKLOADS["small"].with_(T=T, d=d, V=V, K=K, chunk=CHUNK, tau=1.0, seq_len=T, pad_frac=0.2)
    return {k: v.cuda() for k, v in make_inputs(w, seed=5).items()}


def _workspace(kdkl):
    """Enough for every call here."""
    n = (64 << 20) + kdkl.kd_lmhead_topk_workspace_size(T, d, V, K)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _calls(kdkl, g, ws, lse):
    H, W, idx, logit, mask = (g[k] for k in ("H", "W", "topk_idx", "topk_logit", "mask"))
    x = torch.zeros(T, device="cuda")
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
    return {
        "policy": lambda: kdkl.kd_policy_loss(x, None, None, x, workspace=ws),
        "pref": lambda: kdkl.kd_pref_loss(x, None, cu, workspace=ws),
        "logprob_forward": lambda: kdkl.kd_logprob_forward(H, W, ids, mask, workspace=ws),
        "logprob_backward": lambda: kdkl.kd_logprob_backward(H, W, ids, lse, x, workspace=ws),
        "kl_backward": lambda: kdkl.kd_kl_backward(H, W, idx, logit, mask, lse, chunk=CHUNK,
                                                   workspace=ws),
        "rkl_forward": lambda: kdkl.kd_rkl_forward(H, W, idx, logit, mask, workspace=ws),
        "rkl_backward": lambda: kdkl.kd_rkl_backward(H, W, idx, logit, mask, workspace=ws),
        "topk": lambda: kdkl.kd_lmhead_topk(H, W, K, workspace=ws),
    }


def _forward(kdkl, g, ws):
    loss, lse, _ = kdkl.kd_kl_forward(g["H"], g["W"], g["topk_idx"], g["topk_logit"], g["mask"],
                                      chunk=CHUNK, workspace=ws)
    return lse


def _reuse(kdkl, g, ws, lse, **kw):
    return kdkl.kd_kl_backward(g["H"], g["W"], g["topk_idx"], g["topk_logit"], g["mask"], lse,
                               chunk=CHUNK, fwd_workspace=ws, **kw)


@pytest.mark.parametrize("name", ["policy", "pref", "logprob_forward", "logprob_backward",
                                  "kl_backward", "rkl_forward", "rkl_backward", "topk"])
def test_overwritten_workspace_is_refused(kdkl, g, name):
    ws = _workspace(kdkl)
    lse = _forward(kdkl, g, ws)
    want = _reuse(kdkl, g, ws, lse)  # as often as one likes while nothing has overwritten it
    again = _reuse(kdkl, g, ws, lse)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    _calls(kdkl, g, ws, lse)[name]()
    with pytest.raises(kdkl.KDKLError) as e:
        _reuse(kdkl, g, ws, lse)
    assert e.value.code == INVALID
    lse = _forward(kdkl, g, ws)  # filled again
    assert all(torch.equal(a, b) for a, b in zip(want, _reuse(kdkl, g, ws, lse)))


def test_its_own_workspace_is_refused(kdkl, g):
    ws = _workspace(kdkl)
    lse = _forward(kdkl, g, ws)
    with pytest.raises(kdkl.KDKLError) as e:
        _reuse(kdkl, g, ws, lse, workspace=ws)
    assert e.value.code == INVALID
