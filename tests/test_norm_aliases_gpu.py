"""A norm written over its own input: what is returned for what was normed."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("d", [96, 501])
@pytest.mark.parametrize("view", [False, True])
def test_over_x_without_a_residual(kdkl, kind, d, view):
    x, w = torch.randn(33, d, device="cuda"), torch.randn(d, device="cuda")
    want, h, mean, rstd = kdkl.kd_norm_forward(x, w, kind=kind)
    assert h is x
    y, gone, mean2, rstd2 = kdkl.kd_norm_forward(x, w, kind=kind, y=x.view(33, d) if view else x)
    # x holds y now: it is not handed out as what the backward takes
    assert gone is None and torch.equal(y, want) and torch.equal(x, want)
    assert torch.equal(rstd, rstd2) and (mean is None or torch.equal(mean, mean2))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_over_x_and_residual(kdkl, kind):
    """With a residual the sum has its own place, whichever of the inputs that is."""
    x, r, w = torch.randn(33, 96, device="cuda"), torch.randn(33, 96, device="cuda"), torch.randn(96, device="cuda")
    want, h, _, _ = kdkl.kd_norm_forward(x, w, residual=r, kind=kind)
    for over in (("x", "r"), ("r", "x"), ("x", None), (None, "x")):
        t = {"x": x.clone(), "r": r.clone(), None: None}
        y2, h2, _, _ = kdkl.kd_norm_forward(t["x"], w, residual=t["r"], kind=kind, y=t[over[0]], h=t[over[1]])
        assert torch.equal(y2, want) and torch.equal(h2, h)


def test_no_rows(kdkl):
    x = torch.empty(0, 16, device="cuda")
    assert kdkl.kd_norm_forward(x, kind="rms")[1] is x
    assert kdkl.kd_norm_forward(x, kind="rms", y=x)[1] is None
