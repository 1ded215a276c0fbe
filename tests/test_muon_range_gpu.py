"""The Muon step over the whole range of 32 bits: momenta so small or so large that their squares
vanish or overflow there, against fp64."""
import pytest
import torch

from oracle import body_oracle as bo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# Of the orthogonalised matrix, in the 2-norm: three products of at most 96 terms each, a unit in
# the last place (2^-23) lost with each at most, 5 times and grown by up to 5 in one of them.
X_TOL = 8.6e-4
# A block's own (up to 128 x 256, alone in the list), one sum of squares and several of them.
LISTS = {"small": [(100, 100), (40, 70), (70, 40)], "one sum": [(140, 110)], "sums": [(300, 700), (700, 300), (100, 100)]}


@pytest.fixture(scope="module")
def kdkl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from lm_head_top_gb300 import kdkl as m
    m.load()
    return m


def _matrices(shapes, seed=0, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [r(*s) * size for s in shapes], [r(*s) * size for s in shapes]


def _check(kdkl, grads, momentum, eps, mu, nesterov=True):
    """From parameters of zero: what is left is the step alone."""
    params = [torch.zeros_like(g) for g in grads]
    before = [m.clone() for m in momentum]
    kdkl.kd_muon_step(kdkl.kd_muon_tensors(params, grads, momentum), lr=1.0, scale="spectral", eps=eps,
                      momentum=mu, nesterov=nesterov)
    for p, g, m0, m in zip(params, grads, before, momentum):
        want = bo.muon(torch.zeros_like(p), g, m0, lr=1.0, scale="spectral", eps=eps, mu=mu, nesterov=nesterov)[0]
        assert m.isfinite().all() and p.isfinite().all()
        err, size = float((p.double() - want).norm()), float(want.norm())
        assert err <= (X_TOL + 4 * U) * size, (tuple(p.shape), err, size)


@pytest.mark.parametrize("shapes", list(LISTS))
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("size", [2e-23, 1e-26, 1e-20, 1e-12, 1e12, 1e18, 1e20, 1e30, 2e37])
def test_a_step_does_not_depend_on_the_size(kdkl, shapes, nesterov, size):
    grads, momentum = _matrices(LISTS[shapes], size=size)
    # 1e-30, the least that is taken: 1e-26 times 70 or more elements' root is above it
    _check(kdkl, grads, momentum, 1e-30, 0.5, nesterov)


@pytest.mark.parametrize("shapes", list(LISTS))
@pytest.mark.parametrize("size,eps", [(1e-25, 1e-20), (1e-25, 1e-7), (1e-23, 1e-22), (1e-18, 1e-16), (1e-3, 1e25), (1e25, 1e30)])
def test_below_eps(kdkl, shapes, size, eps):
    """X = u / eps: as far below 1 as u is below eps. What fp16 halves times 2^13 hold of it ends
    at 2^-38, and five steps grow what is lost there by up to 3.4445^5 (as X itself)."""
    grads, momentum = _matrices(LISTS[shapes], size=size)
    params = [torch.zeros_like(g) for g in grads]
    before = [m.clone() for m in momentum]
    kdkl.kd_muon_step(kdkl.kd_muon_tensors(params, grads, momentum), lr=1.0, scale="spectral", eps=eps, momentum=0.5)
    for p, g, m0 in zip(params, grads, before):
        want = bo.muon(torch.zeros_like(p), g, m0, lr=1.0, scale="spectral", eps=eps, mu=0.5)[0]
        scale = max(1.0, p.shape[0] / p.shape[1]) ** 0.5
        lost = 2.0 ** -38 * 3.4445 ** 5 * 5 * scale * p.numel() ** 0.5
        assert float((p.double() - want).norm()) <= (X_TOL + 4 * U) * float(want.norm()) + lost


@pytest.mark.parametrize("sizes", [(1e-25, 1e-21), (1e-25, 1.0), (1.0, 1e25), (1e-25, 1e25), (1e-13, 1e-11), (1e11, 1e13)])
@pytest.mark.parametrize("where", ["first", "last", "one element"])
def test_parts_of_a_matrix_of_different_sizes(kdkl, sizes, where):
    """Sums of squares are taken by pieces of a matrix: pieces of different sizes meet."""
    shapes = [(300, 700), (700, 300), (90, 200), (200, 90)]
    grads, momentum = _matrices(shapes, size=sizes[0])
    for k, t in enumerate(grads):
        rows = t.view(-1) if where == "one element" else t
        n = 1 if where == "one element" else t.shape[0] // 3
        part = rows[:n] if where != "last" else rows[-n:]
        part.div_(sizes[0]).mul_(sizes[1])  # (their quotient may be beyond fp32)
    _check(kdkl, grads, momentum, 1e-30, 0.0)
    for g, m in zip(grads[2:], momentum[2:]):
        m.zero_()
    _check(kdkl, grads[2:], momentum[2:], 1e-30, 0.0)


@pytest.mark.parametrize("size", [1e-25, 1.0, 1e25])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_at_any_size(kdkl, size, bad):
    """It takes its own matrix and no other; in a list and in the small ones' launch."""
    for shapes in ([(300, 700)] * 3, [(100, 100)] * 3):
        grads, momentum = _matrices(shapes, size=size)
        grads[1][3, 5] = bad
        params = [torch.ones_like(g) for g in grads]
        kdkl.kd_muon_step(kdkl.kd_muon_tensors(params, grads, momentum), lr=0.1, eps=1e-30)
        assert params[0].isfinite().all() and params[2].isfinite().all()
        assert params[1].isnan().all()


def test_a_momentum_that_decays_away(kdkl):
    """A matrix without gradients: 3000 steps at 0.95 take its momentum from 1 to 1e-67, through all
    sizes that fp32 has, and out. Its parameters stay finite, and every step is at most a whole one."""
    for shapes in ([(40, 70)], [(140, 150)]):
        params, momentum = _matrices(shapes)
        grads = [torch.zeros_like(p) for p in params]
        h = kdkl.kd_muon_tensors(params, grads, momentum)
        ws = torch.empty(h.workspace_bytes, dtype=torch.uint8, device="cuda")
        last = params[0].clone()
        for step in range(3000):
            kdkl.kd_muon_step(h, lr=1e-3, scale="spectral", eps=1e-30, workspace=ws)
            if step % 100 == 99:
                assert params[0].isfinite().all(), step
                # singular values of X end up below 1.21, and |X| below that times r's root
                assert float((params[0] - last).norm()) <= 100 * 1e-3 * 1.21 * min(shapes[0]) ** 0.5 * 1.01
                last = params[0].clone()
        assert not momentum[0].any() or float(momentum[0].abs().max()) < 1e-37
